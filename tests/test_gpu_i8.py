"""8-bit rounding and products against the same definitions in 64 bits.

Tolerances count roundings: u = 2^-24 is half a step of fp32.
  rounding  q is a whole number defined exactly: equality.
  product   float(acc), its product with s_t and the fused multiply-add with
            w_n and b_n: at most 2u of |s_t w_n acc| and u of the result;
            one more u for the residual sum; ReLU^2 doubles the relative error
            and adds its own product.
"""
import numpy as np
import pytest
import torch

import attention_free_long_b200 as av

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _ref_rows(x):
    """(q, scale) of fp32 rows from the definition, in float64 / exact fp32."""
    x32 = x.astype(np.float32)
    amax = np.abs(x32).max(1)
    s = (amax * np.float32(np.float32(1) / np.float32(127))).astype(np.float32)
    ok = s > 0
    q = np.zeros_like(x32, dtype=np.float64)
    q[ok] = np.rint(x32[ok].astype(np.float64) / s[ok].astype(np.float64)[:, None])
    return np.clip(q, -127, 127).astype(np.int64), s


def _activations(rows, cols, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)))
    return x.astype(np.float32)


def _source(x, kind, dev):
    """(tensor, the fp32 values it stands for) as fp32, bf16, a pair, or with
    rows that start off the 16-byte boundary."""
    t = torch.from_numpy(x).to(dev)
    if kind == "bf16":
        t = t.to(torch.bfloat16)
        return t, t.float().cpu().numpy()
    if kind == "pair":
        hi = t.to(torch.bfloat16)
        p = torch.stack([hi, (t - hi.float()).to(torch.bfloat16)]).contiguous()
        return p, (p[0].float() + p[1].float()).cpu().numpy()
    if kind == "strided":
        wide = torch.full((x.shape[0], x.shape[1] + 5), float("nan"), device=dev)
        wide[:, 3:3 + x.shape[1]] = t
        return wide[:, 3:3 + x.shape[1]], x
    return t, x


@pytest.mark.parametrize("kind", ["f32", "bf16", "pair", "strided"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 768), (3, 7), (5, 129), (300, 40), (200, 1023), (150, 1025),
                                       (2, 8193), (2, 20003)])
def test_rows_are_rounded_as_defined(rows, cols, kind, cuda_dev):
    t, x = _source(_activations(rows, cols, rows * 7 + cols), kind, cuda_dev)
    r = av.avey_quantize_rows(t)
    n = av.avey_quantize_rows(t, prenorm=True)
    torch.cuda.synchronize()
    q, s = _ref_rows(x)
    np.testing.assert_array_equal(r.q[:, :cols].cpu().numpy().astype(np.int64), q)
    assert int(r.q[:, cols:].abs().sum()) == 0
    np.testing.assert_array_equal(r.scale.cpu().numpy(), s)
    assert torch.equal(n.q, r.q)
    x64 = x.astype(np.float64)
    want = s.astype(np.float64) / np.sqrt((x64 * x64).mean(1) + 1e-6)
    # a lane adds cols / 32 squares, then ten partial sums; half of that on the root, and five roundings
    tol = ((cols / 32 + 32) / 2 + 5) * U
    np.testing.assert_allclose(n.scale.cpu().numpy().astype(np.float64), want, rtol=tol)


def test_quotients_next_to_and_on_a_half(cuda_dev):
    # scales that are powers of two give exact halves (ties to even); x one
    # step beside them must go to the near side
    k = np.arange(-126, 126)
    half = (k + 0.5).astype(np.float32)
    # the largest value of a row whose scale is exactly 1: amax * fl(1/127) == 1
    inv = np.float32(np.float32(1) / np.float32(127))
    amax = next(np.float32(a) for a in (127.0, np.nextafter(np.float32(127), np.float32(0)),
                                        np.nextafter(np.float32(127), np.float32(200)))
                if np.float32(np.float32(a) * inv) == np.float32(1))
    base = np.concatenate([half, np.nextafter(half, np.float32(1e9)), np.nextafter(half, np.float32(-1e9)), [amax]])
    rows = np.stack([base, base * np.float32(2.0 ** -40), base * np.float32(2.0 ** 60), -base]).astype(np.float32)
    r = av.avey_quantize_rows(torch.from_numpy(rows).to(cuda_dev))
    q, s = _ref_rows(rows)
    np.testing.assert_array_equal(r.q[:, :rows.shape[1]].cpu().numpy().astype(np.int64), q)
    np.testing.assert_array_equal(r.scale.cpu().numpy(), s)
    assert (s == np.float32(1)).sum() == 2


def test_rows_of_zeros_tiny_values_and_what_is_not_finite(cuda_dev):
    x = _activations(9, 100, 3)
    x[0] = 0
    x[1] *= np.float32(1e-42)  # subnormal: the scale itself rounds coarsely
    x[2] = 0
    x[2, 5] = np.float32(1e-45)  # the scale underflows to 0
    x[3, 7] = np.nan
    x[4, 8] = np.inf
    x[5, 9] = -np.inf
    x[6] = np.float32(3e38)
    r = av.avey_quantize_rows(torch.from_numpy(x).to(cuda_dev))
    got, scale = r.q[:, :100].cpu().numpy().astype(np.int64), r.scale.cpu().numpy()
    ok = [0, 1, 2, 6, 7, 8]
    q, s = _ref_rows(x[ok])
    np.testing.assert_array_equal(got[ok], q)
    np.testing.assert_array_equal(scale[ok], s)
    assert np.isnan(scale[[3, 4, 5]]).all() and not got[[3, 4, 5]].any()
    assert (scale[[0, 2]] == 0).all() and not got[[0, 2]].any()


def test_quantize_leaves_columns_behind_the_padding(cuda_dev):
    x = torch.randn(5, 20, device=cuda_dev)
    q = torch.full((5, 64), 99, dtype=torch.int8, device=cuda_dev)
    scale = torch.full((7,), -1.0, device=cuda_dev)
    code = av.lib().avey_quantize_rows(x.data_ptr(), av.AVEY_F32, 5, 20, 20, 0, q.data_ptr(), 64, scale.data_ptr(),
                                       torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert code == 0
    assert bool((q[:, 32:] == 99).all()) and bool((q[:, 20:32] == 0).all())
    assert bool((scale[5:] == -1).all())


def _weights(N, K, seed, dev, bias):
    rng = np.random.default_rng(seed)
    q = rng.integers(-127, 128, (N, K))
    ld = (K + 15) // 16 * 16 + 16
    t = torch.full((N, ld), 77, dtype=torch.int8, device=dev)  # what lies behind K is not used
    t[:, :K] = torch.from_numpy(q.astype(np.int8)).to(dev)
    w = (np.exp(rng.standard_normal(N)) / 127 / np.sqrt(K)).astype(np.float32)
    b = rng.standard_normal(N).astype(np.float32) if bias else None
    lin = av.QuantLinear(t, torch.from_numpy(w).to(dev), K, None if b is None else torch.from_numpy(b).to(dev))
    return lin, q, w, b


def _product(x, q, w, b, act, res):
    """(y, bound of the fp32 kernel's error) in float64."""
    xq, s = _ref_rows(x)
    # float64 products of whole numbers are exact here
    p = (xq.astype(np.float64) @ q.T.astype(np.float64)) * s.astype(np.float64)[:, None] * w.astype(np.float64)[None]
    y = p + (0 if b is None else b.astype(np.float64))
    err = 2 * U * np.abs(p) + U * np.abs(y)
    if act:
        y = np.maximum(y, 0)
        err = 2 * y * err + err * err + U * y * y
        y = y * y
    if res is not None:
        y = y + res.astype(np.float64)
        err = err + U * np.abs(y)
    return y, err * (1 + 1e-6) + 1e-37


SHAPES = [(1, 768, 1000), (1, 5, 1), (2, 16, 7), (7, 31, 64), (8, 768, 257), (9, 127, 65), (16, 128, 8),
          (33, 129, 255), (64, 768, 1536), (129, 1000, 96), (257, 100, 300), (300, 2048, 33), (1025, 64, 513), (24, 500, 77),
          (30, 5000, 40), (12, 7000, 9700), (17, 64, 1), (32, 1025, 130)]
# tiles of 128 and of 256 columns, x resident or not, several row blocks to a pair of SMs
WIDE = [(700, 100, 4000), (2000, 300, 9001), (1500, 1100, 4004), (40000, 64, 300)]
# few tokens against many channels
SWAPPED = [(17, 768, 5001), (64, 1000, 9001), (33, 2100, 4743), (32, 15, 19000), (12, 1025, 4800), (9, 800, 25000),
           (11, 1000, 100)]


@pytest.mark.parametrize("rows,K,N", SHAPES + WIDE + SWAPPED)
@pytest.mark.parametrize("kind,out", [("f32", "f32"), ("bf16", "bf16"), ("pair", "pair"), ("strided", "f32")])
def test_product(rows, K, N, kind, out, cuda_dev):
    act, bias = (rows + N) % 2, K % 2 == 0
    lin, q, w, b = _weights(N, K, rows + K + N, cuda_dev, bias)
    t, x = _source(_activations(rows, K, K), kind, cuda_dev)
    y, err = _product(x, q, w, b, act, None)
    got = av.avey_linear_i8(t, lin, act=act, out_dtype=torch.bfloat16 if out == "bf16" else torch.float32,
                            pair=out == "pair")
    torch.cuda.synchronize()
    assert av.device_status() == 0
    if out == "pair":
        assert got.shape == (2, rows, N)
        got = got[0].double() + got[1].double()
        err = err + 2.0 ** -16 * np.abs(y)  # lo <= 2^-8 of the value, off by 2^-8 of itself
    elif out == "bf16":
        err = err + 2.0 ** -8 * (np.abs(y) + err)
    assert tuple(got.shape) == (rows, N)
    assert (np.abs(got.double().cpu().numpy() - y) <= err).all()


@pytest.mark.parametrize("rows,K,N", [(1, 64, 40), (5, 100, 13), (70, 768, 200), (300, 1536, 768),
                                      (600, 40, 4001), (3001, 100, 2050), (40, 100, 5003), (64, 65, 20000)])
def test_residual_alone_and_in_place(rows, K, N, cuda_dev):
    lin, q, w, b = _weights(N, K, 5, cuda_dev, True)
    x = _activations(rows, K, 6)
    res = np.random.default_rng(7).standard_normal((rows, N)).astype(np.float32)
    t, r = torch.from_numpy(x).to(cuda_dev), torch.from_numpy(res).to(cuda_dev)
    y, err = _product(x, q, w, b, 0, res)
    got = av.avey_linear_i8(t, lin, residual=r)
    assert (np.abs(got.double().cpu().numpy() - y) <= err).all()
    # rows of the residual that start anywhere
    loose = torch.full((rows * (N + 3) + 8,), float("nan"), device=cuda_dev)
    view = loose[1:1 + rows * (N + 3)].view(rows, N + 3)[:, :N]
    view.copy_(r)
    assert torch.equal(av.avey_linear_i8(t, lin, residual=view), got)
    ld = (N + 7) // 8 * 8
    wide = torch.full((rows + 2, ld + 8), 7.0, device=cuda_dev)  # rows and columns around the output
    wide[:rows, :N] = r
    av.avey_linear_i8(t, lin, residual=wide[:rows, :N], out=wide[:rows, :N])
    assert torch.equal(wide[:rows, :N], got)
    assert bool((wide[rows:] == 7).all()) and bool((wide[:, N:] == 7).all())


def test_prequantized_rows_and_extreme_integers(cuda_dev):
    rows, K, N = 40, 1100, 50
    lin, q, w, _ = _weights(N, K, 8, cuda_dev, False)
    lin.q.fill_(127)
    xq = torch.full((rows, 1104), 127, dtype=torch.int8, device=cuda_dev)  # sums past 2^24
    xq[1] = -128
    xq[:, K:] = 55
    scale = torch.rand(rows, device=cuda_dev) + 0.5
    for n in (rows, 3):
        r = av.QuantRows(xq[:n].contiguous(), scale[:n].contiguous(), K)
        got = av.avey_linear_i8(r, lin).double().cpu().numpy()
        acc = np.full((n, 1), 127.0 * 127 * K)
        acc[1] = -128.0 * 127 * K
        y = acc * scale[:n].double().cpu().numpy()[:, None] * w.astype(np.float64)[None]
        # float(acc) rounds too: 3u of the product, u of the result
        assert (np.abs(got - y) <= 4 * U * np.abs(y) * (1 + 1e-6)).all()


@pytest.mark.parametrize("rows,N", [(3, 33), (40, 33), (40, 4801)])
def test_a_row_that_is_not_finite_spoils_itself_alone(rows, N, cuda_dev):
    lin, q, w, b = _weights(N, 200, 9, cuda_dev, True)
    x = _activations(rows, 200, 10)
    clean, _ = _product(x, q, w, b, 1, None)
    x[1, 17] = np.nan
    x[2] = 0
    got = av.avey_linear_i8(torch.from_numpy(x).to(cuda_dev), lin, act=av.AVEY_ACT_RELU2).cpu().numpy()
    assert np.isnan(got[1]).all()
    np.testing.assert_allclose(got[2], np.maximum(b, 0) ** 2, rtol=2 * U)
    keep = [0] + list(range(3, rows))
    np.testing.assert_allclose(got[keep], clean[keep], rtol=1e-3, atol=1e-3)


@pytest.mark.parametrize("rows", [4, 130])
def test_rounding_error_stays_within_half_a_step(rows, cuda_dev):
    # |y - xW^T| <= s_t / 2 sum|W| + w_n / 2 sum|x_q| for weights and rows rounded here
    rng = np.random.default_rng(11)
    K, N = 384, 96
    W = (rng.standard_normal((N, K)) / np.sqrt(K)).astype(np.float32)
    x = _activations(rows, K, 12)
    lin = av.quantize_linear(torch.from_numpy(W).to(cuda_dev))
    got = av.avey_linear_i8(torch.from_numpy(x).to(cuda_dev), lin).double().cpu().numpy()
    xq, s = _ref_rows(x)
    y = x.astype(np.float64) @ W.astype(np.float64).T
    xa = np.abs(xq * s.astype(np.float64)[:, None]).sum(1)[:, None]
    bound = s[:, None] / 2 * np.abs(W).sum(1)[None] + lin.scale.cpu().numpy()[None] / 2 * xa
    assert (np.abs(got - y) <= bound * (1 + 1e-5)).all()


def test_streams_graphs_and_shared_weights(cuda_dev):
    lin, q, w, b = _weights(300, 256, 13, cuda_dev, True)
    xs = [torch.randn(n, 256, device=cuda_dev) for n in (2, 200, 500)]
    want = [av.avey_linear_i8(x, lin) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for x, s in zip(xs, streams):
        with torch.cuda.stream(s):
            got.append([av.avey_linear_i8(x, lin) for _ in range(3)])
    torch.cuda.synchronize()
    for g, e in zip(got, want):
        assert all(torch.equal(a, e) for a in g)
    for x, e in zip(xs, want):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = av.avey_linear_i8(x, lin)
        x.mul_(2.0)
        graph.replay()
        torch.cuda.synchronize()
        # doubling a row doubles its scale and leaves its integers
        bias = lin.bias[None]
        torch.testing.assert_close(y - bias, 2 * (e - bias), rtol=1e-5, atol=1e-5)
    assert av.device_status() == 0
