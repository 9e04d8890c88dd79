"""The gradient where the given word itself is masked: p = 0 there, and the formula
g (1[j = id] - p_j) - h p_j (log p_j + entropy) leaves g."""
import numpy as np
import pytest
import torch

import attention_free_long_b200 as av

pytestmark = pytest.mark.gpu
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,V", [(3, 7), (4, 4097), (2000, 250)])
def test_given_word_of_minus_infinity(rows, V, dtype, cuda_dev):
    g = torch.Generator(device=cuda_dev).manual_seed(V)
    x = (torch.randn(rows, V, device=cuda_dev, generator=g) * 2).to(dtype)
    ids = torch.randint(0, V, (rows,), device=cuda_dev, generator=g, dtype=torch.int32)
    at = ids.long()[:, None]
    x.scatter_(1, at, float("-inf"))
    x[1] = float("-inf")  # nothing left: zeros
    d = torch.randn(rows, device=cuda_dev, generator=g)
    for h in (None, torch.randn(rows, device=cuda_dev, generator=g)):
        r = av.avey_token_logprobs(x, ids)
        dx = av.avey_token_logprobs_backward(x, ids, r, d, h)
        torch.cuda.synchronize()
        assert av.device_status() == 0
        assert bool((r.logprob == float("-inf")).all())
        got = dx.gather(1, at)[:, 0]
        keep = torch.arange(rows, device=cuda_dev) != 1
        assert torch.equal(got[keep], d.to(dtype)[keep])
        assert bool((dx[1] == 0).all())
        # the others against the definition in 64 bits, D = max |x - m| < 20, H and z < 9: log p
        # is (3 D + 4 + V / 256 + 150) u + 3 D u < 300 u off and p as much, relative; with H,
        # 230 u (1 + 2 (H + z)) < 8100 u off, the term of h has 300 u 40 + 8100 u + 300 u
        # < 400 u 64; then half a step of the type
        p = torch.softmax(x.double(), 1)
        want = -p * d.double()[:, None]
        if h is not None:
            lp = torch.log_softmax(x.double(), 1)
            H = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(1, keepdim=True)
            want = want - h.double()[:, None] * torch.where(p > 0, p * (lp + H), torch.zeros_like(p))
        want.scatter_(1, at, d.double()[:, None])
        scale = p * (d.abs().double()[:, None] + (0 if h is None else h.abs().double()[:, None] * 64))
        tol = 400 * 2.0 ** -24 * scale + HALF[dtype] * want.abs() + 1e-37
        bad = ((dx.double() - want).abs() > tol)[keep]
        assert not bool(bad.any())
