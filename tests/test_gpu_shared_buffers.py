"""Operands that are columns of one wide buffer: their rows alternate in memory but
share no byte, so the calls take them, and touch nothing else of the buffer."""
import numpy as np
import pytest
import torch

import attention_free_long_b200 as av

pytestmark = pytest.mark.gpu


def _lin(N, K, dev):
    g = torch.Generator(device=dev).manual_seed(N + K)
    return av.quantize_linear(torch.randn(N, K, device=dev, generator=g), torch.randn(N, device=dev, generator=g))


@pytest.mark.parametrize("rows,K,N", [(2, 40, 24), (12, 96, 64), (40, 72, 5000), (300, 136, 272)])
def test_product_beside_its_input_and_residual(rows, K, N, cuda_dev):
    lin = _lin(N, K, cuda_dev)
    x = torch.randn(rows, K, device=cuda_dev)
    res = torch.randn(rows, N, device=cuda_dev)
    want = av.avey_linear_i8(x, lin, residual=res)
    wide = torch.full((rows, K + 2 * N + 8), 7.0, device=cuda_dev)
    xv, rv, ov = wide[:, :K], wide[:, K:K + N], wide[:, K + N:K + 2 * N]
    xv.copy_(x)
    rv.copy_(res)
    av.avey_linear_i8(xv, lin, residual=rv, out=ov)
    torch.cuda.synchronize()
    assert torch.equal(ov, want) and torch.equal(xv, x) and torch.equal(rv, res)
    assert bool((wide[:, K + 2 * N:] == 7).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,V", [(2, 50), (5, 3001), (2000, 96)])
def test_gradient_beside_the_logits(rows, V, dtype, cuda_dev):
    wide = torch.full((rows, 2 * V + 6), 7.0, device=cuda_dev, dtype=dtype)
    for x, out in ((wide[:, :V], wide[:, V:2 * V]), (wide[:, V + 5:2 * V + 5], wide[:, :V])):
        wide.fill_(7.0)
        x.copy_(torch.randn(rows, V, device=cuda_dev) * 3)
        kept = x.clone()
        ids = torch.randint(0, V, (rows,), device=cuda_dev, dtype=torch.int32)
        r = av.avey_token_logprobs(x, ids)
        d = torch.randn(rows, device=cuda_dev)
        want = av.avey_token_logprobs_backward(kept, ids, r, d, d)
        av.avey_token_logprobs_backward(x, ids, r, d, d, out=out)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(x, kept)
        left = torch.ones_like(wide, dtype=torch.bool)
        left[:, x.storage_offset():x.storage_offset() + V] = False
        left[:, out.storage_offset():out.storage_offset() + V] = False
        assert bool((wide[left] == 7).all())


def test_rounded_rows_beside_their_source(cuda_dev):
    # one byte buffer: 40 fp32 values, then 48 bytes of integers, a row
    rows, cols = 6, 40
    buf = torch.zeros(rows, 160 + 48, dtype=torch.uint8, device=cuda_dev)
    x = torch.randn(rows, cols, device=cuda_dev)
    buf[:, :160] = x.view(torch.uint8).view(rows, 160)
    want = av.avey_quantize_rows(x)
    scale = torch.zeros(rows, device=cuda_dev)
    code = av.lib().avey_quantize_rows(buf.data_ptr(), av.AVEY_F32, rows, cols, 52, 0, buf.data_ptr() + 160, 208,
                                       scale.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert code == 0
    np.testing.assert_array_equal(buf[:, 160:].view(torch.int8).cpu().numpy(), want.q.cpu().numpy())
    assert torch.equal(scale, want.scale)
    assert torch.equal(buf[:, :160].contiguous().view(torch.float32), x)
