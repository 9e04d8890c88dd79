"""RMS-normalised 8-bit rows whose squares leave fp32: finite rows have a finite,
non-zero scale, s / sqrt(mean(x^2) + 1e-6), however large their values."""
import numpy as np
import pytest
import torch

import attention_free_long_b200 as av

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _rows(cols, kind, dev):
    """(tensor, its values in 64 bits): rows around and far past 2^64, where squares
    overflow, among ordinary ones."""
    rng = np.random.default_rng(cols)
    x = rng.standard_normal((9, cols))
    x /= np.abs(x).max(1, keepdims=True)
    x *= np.array([1.0, 1e18, 1.8e19, 2e19, 1e20, 1e30, 3e38, 1e-20, 1.0])[:, None]
    x[8, cols // 2] = 3e38  # one value among ordinary ones
    t = torch.from_numpy(x.astype(np.float32)).to(dev)
    if kind == "bf16":
        t = t.to(torch.bfloat16)
    elif kind == "pair":
        hi = t.to(torch.bfloat16)
        t = torch.stack([hi, (t - hi.float()).to(torch.bfloat16)]).contiguous()
        return t, (t[0].float() + t[1].float()).double().cpu().numpy()
    elif kind == "strided":
        wide = torch.full((9, cols + 5), float("nan"), device=dev)
        wide[:, 3:3 + cols] = t
        t = wide[:, 3:3 + cols]
    return t, t.double().cpu().numpy()


# every number of threads to a row, and rows longer than their registers
@pytest.mark.parametrize("cols", [3, 64, 200, 300, 700, 1500, 3001, 5000, 20003])
@pytest.mark.parametrize("kind", ["f32", "bf16", "pair", "strided"])
@pytest.mark.parametrize("copies", [1, 40])  # a block to a row, and rows side by side in a block
def test_scales_of_large_rows(cols, kind, copies, cuda_dev):
    t, x = _rows(cols, kind, cuda_dev)
    if copies > 1:
        t = t.repeat(1, copies, 1) if kind == "pair" else t.repeat(copies, 1)
        x = np.tile(x, (copies, 1))
    r, n = av.avey_quantize_rows(t), av.avey_quantize_rows(t, prenorm=True)
    torch.cuda.synchronize()
    assert torch.equal(r.q, n.q)
    want = r.scale.double().cpu().numpy() / np.sqrt((x * x).mean(1) + 1e-6)
    # a lane adds at most cols / 32 squares (32 in rows of few threads), then ten partial
    # sums; half of that on the root, and five roundings
    tol = ((cols / 32 + 32) / 2 + 5) * U
    np.testing.assert_allclose(n.scale.double().cpu().numpy(), want, rtol=tol)


@pytest.mark.parametrize("kind", ["f32", "bf16", "pair", "strided"])
@pytest.mark.parametrize("cols", [64, 700, 3001])
def test_products_of_large_rows(cols, kind, cuda_dev):
    # nine rows are rounded by the few-row kernel (up to 768 columns) or before the product
    t, x = _rows(cols, kind, cuda_dev)
    t, x = (t[:, :8].contiguous() if kind == "pair" else t[:8]), x[:8]
    W = torch.randint(-127, 128, (100, (cols + 15) // 16 * 16), device=cuda_dev, dtype=torch.int8)
    lin = av.QuantLinear(W, torch.rand(100, device=cuda_dev), cols)
    got = av.avey_linear_i8(t, lin, prenorm=True).double().cpu().numpy()
    r = av.avey_quantize_rows(t)
    torch.cuda.synchronize()
    scale = r.scale.double().cpu().numpy() / np.sqrt((x * x).mean(1) + 1e-6)
    acc = r.q[:, :cols].double().cpu().numpy() @ lin.q[:, :cols].double().cpu().numpy().T
    y = acc * scale[:, None] * lin.scale.double().cpu().numpy()[None]
    # the scale as above, and three roundings of the product
    tol = ((cols / 32 + 32) / 2 + 5 + 3) * U
    np.testing.assert_allclose(got, y, rtol=tol)


def test_rows_that_are_not_finite_keep_a_nan_scale(cuda_dev):
    x = torch.randn(6, 100, device=cuda_dev)
    x[0] = 3e38
    x[1, 3], x[2, 5], x[3, 99] = float("inf"), float("nan"), -float("inf")
    x[3, 0] = 3e38
    s = av.avey_quantize_rows(x, prenorm=True).scale.cpu()
    assert bool(torch.isnan(s[1:4]).all()) and bool((s[[0, 4, 5]] > 0).all()) and bool(torch.isfinite(s[[0, 4, 5]]).all())
    assert abs(float(s[0]) * 127 - 1) < 1e-6  # equal values: |x| / rms = 1
