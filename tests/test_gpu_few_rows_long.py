"""Scores of few long rows: the few-row kernel's tokens take up to 96 KB of shared
memory, beside what the scores themselves take.  Each length runs in a process of
its own, so that no longer call has raised the kernel's limit before it."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Logits are exact sums times scales, 2u off as in the product's own tests; the
# scores are compared with 64-bit ones of the fp32 logits, tolerances as there:
# (7 |y| + 5 |b|) u a logit, (3 D + V / 256 + 160) u the sums.
CHILD = """
import sys
import torch
import attention_free_long_b200 as av
K = int(sys.argv[1])
dev = torch.device("cuda:0")
U = 2.0 ** -24
for rows, N in ((1, 1500), (8, 1500), (3, 9601)):
    g = torch.Generator(device=dev).manual_seed(rows)
    W = torch.randint(-127, 128, (N, (K + 15) // 16 * 16), device=dev, generator=g, dtype=torch.int8)
    lin = av.QuantLinear(W, torch.rand(N, device=dev, generator=g) / 40 / K ** 0.5, K)
    h = torch.randn(rows, K, device=dev, generator=g)
    ids = torch.randint(0, N, (rows,), device=dev, generator=g, dtype=torch.int32)
    for x in (h, h.to(torch.bfloat16), av.avey_quantize_rows(h)):
        r = av.avey_score_tokens_i8(x, lin, ids)
        y = av.avey_linear_i8(x, lin).double()
        torch.cuda.synchronize()
        lse = torch.logsumexp(y, 1)
        lp = y.gather(1, ids.long()[:, None])[:, 0] - lse
        big = 7 * y.abs().amax(1)
        far = (y.amax(1) - y.amin(1)).clamp(max=60.0)
        tol = (2 * big + 3 * far + N / 256 + 160) * U
        assert bool(((r.logprob.double() - lp).abs() <= 2 * tol + 4 * U * lp.abs()).all())
        assert bool(((r.stats[:, 0].double() - y.amax(1)).abs() <= U * big).all())
assert av.device_status() == 0
"""


@pytest.mark.parametrize("K", [5888, 5889, 6016, 6017, 12160])
def test_scores_of_few_long_rows(K, cuda_dev):
    r = subprocess.run([sys.executable, "-c", CHILD, str(K)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
