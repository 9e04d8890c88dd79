"""Token scoring (log probabilities, entropy, alternatives) and its gradient
against the definitions in 64 bits.

Tolerances, with u = 2^-24 (half a step of fp32), D = max |x_j - m| over the
entries that count (e^-D > u / V) and V words:
  e_j   the difference, its product with log2 e and the constant: 3u D; the
        exponential unit 4u                      -> E = (3 D + 4) u relative
  sums  a thread adds at most V / 256 + 32 terms, then 20 merges (each with
        one more exponential)                    -> S = E + (V/256 + 150) u
  z     S + 2u |z|;  logprob: that + u (|x - m| + |logprob|)
  H     z - t / s with |t / s| <= H + |z|:       S (1 + 2 (H + |z|)) + 4u (H + |z|)
"""
import numpy as np
import pytest
import torch

import attention_free_long_b200 as av

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def _logits(rows, V, dtype, seed, dev, masked=0.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, V)) * 2.0
    x[np.arange(rows), rng.integers(0, V, rows)] += 8.0
    if masked:
        x[rng.random((rows, V)) < masked] = -np.inf
    t = torch.from_numpy(x.astype(np.float32)).to(dev, dtype)
    return t, t.double().cpu().numpy()


def _ref(x, ids):
    """Per row: m, z, entropy, logprob in float64, and their tolerances."""
    rows, V = x.shape
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        m = x.max(1)
        d = x - m[:, None]
        e = np.exp(d)
        s = e.sum(1)
        z = np.log(s)
        H = z - np.where(e > 0, e * d, 0).sum(1) / s
    far = np.where(e > U / V, -d, 0).max(1)
    E = (3 * far + 4) * U
    S = E + (V / 256 + 150) * U
    tol_z = S + 2 * U * np.abs(z)
    tol_H = S * (1 + 2 * (H + np.abs(z))) + 4 * U * (H + np.abs(z))
    lp = np.where(ids >= 0, d[np.arange(rows), np.maximum(ids, 0)] - z, 0.0)
    with np.errstate(invalid="ignore"):
        tol_lp = np.where(np.isfinite(lp), tol_z + U * (np.abs(lp + z) + np.abs(lp)), 0)
    return dict(m=m, z=z, H=H, lp=lp, tz=tol_z, tH=tol_H, tlp=tol_lp, d=d)


def _top(x, k):
    """(ids, values) by (value desc, index asc); -1 past the entries above -inf."""
    order = np.argsort(-x, axis=1, kind="stable")[:, :k]
    val = np.take_along_axis(x, order, 1)
    ids = np.where(val > -np.inf, order, -1)
    pad = k - ids.shape[1]
    if pad > 0:
        ids = np.pad(ids, ((0, 0), (0, pad)), constant_values=-1)
        val = np.pad(val, ((0, 0), (0, pad)), constant_values=-np.inf)
    return ids, val


def _check(t, x, ids, top, r):
    ref = _ref(x, ids)
    got = lambda v: v.double().cpu().numpy()
    np.testing.assert_array_equal(got(r.stats[:, 0]), ref["m"])
    assert (np.abs(got(r.stats[:, 1]) - ref["z"]) <= ref["tz"]).all()
    assert (np.abs(got(r.entropy) - ref["H"]) <= ref["tH"]).all()
    lp = got(r.logprob)
    fin = np.isfinite(ref["lp"])
    np.testing.assert_array_equal(lp[~fin], ref["lp"][~fin])
    assert (np.abs(lp[fin] - ref["lp"][fin]) <= ref["tlp"][fin]).all()
    if top:
        ti, tv = _top(x, top)
        np.testing.assert_array_equal(r.top_ids.cpu().numpy(), ti)
        want = tv - ref["m"][:, None] - ref["z"][:, None]
        tl = got(r.top_logprobs)
        np.testing.assert_array_equal(tl[ti < 0], -np.inf)
        tol = ref["tz"][:, None] + U * (np.abs(want + ref["z"][:, None]) + np.abs(want))
        ok = ti >= 0
        assert (np.abs(tl[ok] - want[ok]) <= tol[ok]).all()


def _ids(rows, V, seed, dev):
    rng = np.random.default_rng(seed + 1)
    ids = rng.integers(0, V, rows)
    ids[rng.random(rows) < 0.2] = -1
    return ids, torch.from_numpy(ids.astype(np.int32)).to(dev)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,V,top", [
    (1, 1, 1), (3, 2, 2), (1, 50368, 8), (2, 50021, 32), (5, 7, 8), (40, 200, 3), (37, 999, 0), (150, 5003, 17),
    (300, 2048, 32), (700, 511, 5), (90, 12345, 1), (20, 131072, 4),
    (1500, 700, 9), (1203, 4001, 32), (1201, 1, 1), (2000, 33, 0), (640, 30011, 32)])
def test_scores(rows, V, top, dtype, cuda_dev):
    t, x = _logits(rows, V, dtype, rows + V, cuda_dev, masked=0.25 if V > 100 and rows % 2 else 0.0)
    ids, dids = _ids(rows, V, V, cuda_dev)
    r = av.avey_token_logprobs(t, dids, top=top)
    torch.cuda.synchronize()
    assert av.device_status() == 0
    _check(t, x, ids, top, r)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [2, 170])
@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 0), (3, 5), (5, 1)])
def test_rows_anywhere_in_memory(offset, pad, rows, dtype, cuda_dev):
    V = 3001
    t, x = _logits(rows, V, dtype, offset + pad, cuda_dev)
    wide = torch.full((rows * (V + pad) + offset + 16,), float("inf"), dtype=dtype, device=cuda_dev)
    view = wide[offset:offset + rows * (V + pad)].view(rows, V + pad)[:, :V]
    view.copy_(t)
    ids, dids = _ids(rows, V, 3, cuda_dev)
    r = av.avey_token_logprobs(view, dids, top=9)
    _check(view, x, ids, 9, r)
    # the gradient, to rows of other offsets, leaves what lies around them
    g = torch.randn(rows, device=cuda_dev)
    dense = av.avey_token_logprobs_backward(t, dids, r, g)
    for off2 in (offset, offset + 1):
        buf = torch.full((rows * (V + pad) + off2 + 16,), 5.0, dtype=dtype, device=cuda_dev)
        out = buf[off2:off2 + rows * (V + pad)].view(rows, V + pad)
        av.avey_token_logprobs_backward(view, dids, r, g, out=out[:, :V])
        assert torch.equal(out[:, :V], dense)
        assert bool((out[:, V:] == 5).all()) and bool((buf[:off2] == 5).all())
        assert bool((buf[off2 + rows * (V + pad):] == 5).all())


@pytest.mark.parametrize("rows", [3, 400])
@pytest.mark.parametrize("V", [40, 4099, 60000])
def test_ties_go_to_the_lower_index(V, rows, cuda_dev):
    if rows * V > 10_000_000:
        rows = 160
    elif rows > 3 and V == 40:
        rows = 1300  # a warp to a row
    rng = np.random.default_rng(V)
    x = rng.integers(0, 3, (rows, V)).astype(np.float32)  # thousands of equal values
    x[0] = 1.5  # all equal
    x[1, :] = -0.0
    x[1, V // 2] = 0.0  # equal to -0
    x[2] = np.arange(V, dtype=np.float32) / 64  # rising: the last vectors hold everything
    for dtype in (torch.float32, torch.bfloat16):
        t = torch.from_numpy(x).to(cuda_dev, dtype)
        ids, dids = _ids(rows, V, V, cuda_dev)
        r = av.avey_token_logprobs(t, dids, top=32)
        _check(t, t.double().cpu().numpy(), ids, 32, r)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [33, 5000])
@pytest.mark.parametrize("rows", [10, 600])
def test_masks_infinities_and_nan(rows, V, dtype, cuda_dev):
    t, x = _logits(rows, V, dtype, V, cuda_dev)
    low = torch.finfo(dtype).min
    t[0] = float("-inf")  # nothing left
    t[1] = float("-inf")
    t[1, 4] = 2.0  # one word left
    t[2] = low  # masked with the lowest value, all of it
    t[3, 10:] = low
    t[4, 5] = float("nan")
    t[5, 6] = float("inf")
    t[6, ::2] = float("-inf")
    t[7, 3:] = float("-inf")  # fewer words than alternatives
    t[8] *= 1e30 if dtype == torch.float32 else 1e3
    x = t.double().cpu().numpy()
    ids = np.full(rows, 4)
    ids[6] = 2  # a masked word
    r = av.avey_token_logprobs(t, torch.from_numpy(ids.astype(np.int32)).to(cuda_dev), top=8)
    torch.cuda.synchronize()
    assert r.stats[0].tolist() == [-np.inf, 0.0] and float(r.entropy[0]) == 0.0
    assert float(r.logprob[0]) == -np.inf and bool((r.top_ids[0] == -1).all())
    assert bool((r.top_logprobs[0] == -np.inf).all())
    for i in (4, 5):
        assert all(bool(torch.isnan(v[i]).all()) for v in (r.stats, r.entropy, r.logprob, r.top_logprobs))
        assert bool((r.top_ids[i] == -1).all())
    keep = np.array([i for i in range(rows) if i not in (0, 4, 5)])
    sel = torch.from_numpy(keep).to(cuda_dev)
    part = av.TokenLogprobs(r.logprob[sel], r.stats[sel], r.entropy[sel], r.top_ids[sel], r.top_logprobs[sel])
    _check(t[sel], x[keep], ids[keep], 8, part)
    assert float(r.entropy[1]) == 0.0 and float(r.logprob[1]) == 0.0 and r.top_ids[1].tolist()[:2] == [4, -1]
    # gradients: nothing for the empty row, NaN for the spoilt ones, 0 where masked
    g, h = torch.ones(rows, device=cuda_dev), torch.full((rows,), 0.5, device=cuda_dev)
    g[5], h[5] = 0.0, 0.0  # a spoilt row that does not count
    dids = torch.from_numpy(ids.astype(np.int32)).to(cuda_dev)
    dx = av.avey_token_logprobs_backward(t, dids, r, g, h)
    assert bool((dx[0] == 0).all()) and bool(torch.isnan(dx[4]).all()) and bool((dx[5] == 0).all())
    assert bool(torch.isfinite(dx[6:]).all())
    assert float(dx[1].abs().sum()) == 0.0
    assert bool((dx[7, 3:][torch.arange(3, V, device=cuda_dev) != 4] == 0).all())


def test_given_tokens_out_of_range_are_reported(cuda_dev):
    t, x = _logits(4, 100, torch.float32, 1, cuda_dev)
    ids = torch.tensor([3, 100, -7, 99], dtype=torch.int32, device=cuda_dev)
    assert av.device_status() == 0
    r = av.avey_token_logprobs(t, ids)
    assert av.device_status() == 5  # AVEY_ERR_DEVICE_BOUNDS
    assert av.device_status() == 0
    assert r.logprob[1] == 0 and r.logprob[2] == 0 and r.logprob[0] < 0 and r.logprob[3] < 0
    dx = av.avey_token_logprobs_backward(t, ids, r, torch.ones(4, device=cuda_dev))
    assert av.device_status() == 5
    assert bool((dx[1:3] == 0).all()) and bool((dx[0] != 0).any())


def _grad_ref(x, ids, g, h):
    """(gradient, tolerance before the output's rounding) in float64."""
    ref = _ref(x, ids)
    g = np.where(ids >= 0, g, 0.0)[:, None]
    h = h[:, None]
    with np.errstate(invalid="ignore"):
        lp = ref["d"] - ref["z"][:, None]
        p = np.exp(lp)
        lps = np.where(p > 0, lp, 0.0)
    H = ref["H"][:, None]
    dx = -p * (g + h * (lps + H))
    rows = np.arange(len(ids))
    has = ids >= 0
    dx[rows[has], ids[has]] += g[has, 0]
    elp = ref["tz"][:, None] + U * (np.abs(lps + ref["z"][:, None]) + np.abs(lps))
    ep = elp + (3 * np.abs(lps) + 4) * U  # relative error of p
    size = np.abs(g) + np.abs(h) * (np.abs(lps) + H)
    tol = p * (size * (ep + 4 * U) + np.abs(h) * (elp + ref["tH"][:, None])) + U * np.abs(dx)
    tol[rows[has], ids[has]] += U * np.abs(g[has, 0])
    return dx, tol * (1 + 1e-6) + 1e-37


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,V", [(1, 1), (2, 9), (3, 50021), (130, 4097), (500, 256), (61, 20000), (1300, 3)])
def test_gradient(rows, V, dtype, cuda_dev):
    t, x = _logits(rows, V, dtype, rows * V, cuda_dev, masked=0.3 if V > 100 else 0.0)
    ids, dids = _ids(rows, V, rows, cuda_dev)
    rng = np.random.default_rng(V)
    g, h = rng.standard_normal(rows).astype(np.float32), rng.standard_normal(rows).astype(np.float32)
    dg, dh = torch.from_numpy(g).to(cuda_dev), torch.from_numpy(h).to(cuda_dev)
    r = av.avey_token_logprobs(t, dids)
    for gg, hh in ((g, h), (g, None), (None, h)):
        zero = np.zeros(rows)
        dx, tol = _grad_ref(x, ids, zero if gg is None else gg, zero if hh is None else hh)
        got = av.avey_token_logprobs_backward(t, dids, r, None if gg is None else dg, None if hh is None else dh)
        assert got.dtype == dtype
        bound = tol + HALF[dtype] * (np.abs(dx) + tol)
        assert (np.abs(got.double().cpu().numpy() - dx) <= bound).all()
    # in place of the logits
    want = av.avey_token_logprobs_backward(t, dids, r, dg, dh)
    same = av.avey_token_logprobs_backward(t, dids, r, dg, dh, out=t)
    assert same.data_ptr() == t.data_ptr() and torch.equal(t, want)
    assert av.device_status() == 0


def test_gradient_against_differences(cuda_dev):
    rows, V = 4, 60
    t, x = _logits(rows, V, torch.float32, 5, cuda_dev)
    ids, dids = np.array([3, 0, 59, 7]), torch.tensor([3, 0, 59, 7], dtype=torch.int32, device=cuda_dev)
    g, h = np.array([1.0, -2.0, 0.5, 0.0]), np.array([0.3, 0.0, -1.0, 2.0])

    def value(v):
        ref = _ref(v, ids)
        return (g * ref["lp"] + h * ref["H"]).sum()

    r = av.avey_token_logprobs(t, dids)
    f32 = lambda a: torch.from_numpy(a.astype(np.float32)).to(cuda_dev)
    dx = av.avey_token_logprobs_backward(t, dids, r, f32(g), f32(h)).double().cpu().numpy()
    rng = np.random.default_rng(6)
    for _ in range(5):
        v = rng.standard_normal((rows, V))
        step = 1e-4
        diff = (value(x + step * v) - value(x - step * v)) / (2 * step)
        # third-order term of the difference about step^2, float64 noise 1e-15 / step
        assert abs(diff - (dx * v).sum()) <= 1e-5 * max(1.0, np.abs(dx).sum())


def test_shared_stream_graph_and_repeats(cuda_dev):
    t, _ = _logits(300, 9000, torch.bfloat16, 8, cuda_dev)
    few, _ = _logits(3, 60000, torch.float32, 9, cuda_dev)
    pick = lambda n, V: torch.randint(0, V, (n,), dtype=torch.int32, device=cuda_dev)
    ids, fids = pick(300, 9000), pick(3, 60000)
    want, wfew = av.avey_token_logprobs(t, ids, top=6), av.avey_token_logprobs(few, fids, top=6)
    torch.cuda.synchronize()
    flat = lambda r: [r.logprob, r.stats, r.entropy, r.top_ids, r.top_logprobs]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    out = []
    for _ in range(4):
        with torch.cuda.stream(a):
            out.append((want, av.avey_token_logprobs(t, ids, top=6)))
        with torch.cuda.stream(b):
            out.append((wfew, av.avey_token_logprobs(few, fids, top=6)))
    torch.cuda.synchronize()
    for w, g in out:  # the same bits every time
        assert all(torch.equal(p, q) for p, q in zip(flat(w), flat(g)))
    graph = torch.cuda.CUDAGraph()
    d = torch.ones(300, device=cuda_dev)
    with torch.cuda.graph(graph):
        g = av.avey_token_logprobs(t, ids, top=6)
        g2 = av.avey_token_logprobs(few, fids, top=6)
        dx = av.avey_token_logprobs_backward(t, ids, g, d)
    new, _ = _logits(300, 9000, torch.bfloat16, 10, cuda_dev)
    t.copy_(new)
    graph.replay()
    torch.cuda.synchronize()
    eager = av.avey_token_logprobs(t, ids, top=6)
    assert all(torch.equal(p, q) for p, q in zip(flat(eager), flat(g)))
    assert all(torch.equal(p, q) for p, q in zip(flat(wfew), flat(g2)))
    assert torch.equal(dx, av.avey_token_logprobs_backward(t, ids, eager, d))


def test_no_rows(cuda_dev):
    t = torch.empty((0, 50), device=cuda_dev)
    r = av.avey_token_logprobs(t, torch.empty((0,), dtype=torch.int32, device=cuda_dev), top=3)
    assert r.logprob.shape == (0,) and r.top_ids.shape == (0, 3)
    assert av.avey_token_logprobs_backward(t, None, r, None).shape == (0, 50)


def test_binding_refuses(cuda_dev):
    t = torch.zeros(4, 50, device=cuda_dev)
    ids = torch.zeros(4, dtype=torch.int32, device=cuda_dev)
    with pytest.raises(TypeError):
        av.avey_token_logprobs(t, ids.long())
    with pytest.raises(TypeError):
        av.avey_token_logprobs(t, ids[:3])
    with pytest.raises(TypeError):
        av.avey_token_logprobs(t.half())
    with pytest.raises(ValueError):
        av.avey_token_logprobs(t.t())
    with pytest.raises(ValueError):
        av.avey_token_logprobs(t[:1].expand(4, 50))
    with pytest.raises(ValueError):
        av.avey_token_logprobs(t, ids.cpu())
    with pytest.raises(av.AveyError):
        av.avey_token_logprobs(t, ids, top=33)
    r = av.avey_token_logprobs(t, ids)
    with pytest.raises(av.AveyError):  # d_logprob without ids
        av.avey_token_logprobs_backward(t, None, r, torch.ones(4, device=cuda_dev))
    with pytest.raises(TypeError):
        av.avey_token_logprobs_backward(t, ids, r, torch.ones(4, device=cuda_dev), out=t.bfloat16())


def _orders(rows, V, kind, dtype, dev):
    """Rows whose alternatives reach the selection in a hard order."""
    rng = np.random.default_rng(V)
    if kind == "ascending":
        x = np.sort(rng.standard_normal((rows, V)) * 3, axis=1)
    elif kind == "descending":
        x = -np.sort(rng.standard_normal((rows, V)) * 3, axis=1)
    elif kind == "constant":
        x = np.repeat(rng.standard_normal((rows, 1)), V, axis=1)
    else:  # "few": many equal values, the largest at the end
        x = rng.integers(-3, 3, (rows, V)).astype(np.float64)
        x[:, V - 1 - rng.integers(0, min(V, 40), rows)] = 4.0
    t = torch.from_numpy(x.astype(np.float32)).to(dev, dtype)
    return t, t.double().cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["ascending", "descending", "constant", "few"])
@pytest.mark.parametrize("rows,V", [
    (1190, 70), (1190, 512), (1190, 1025), (1190, 4090), (2, 700), (200, 6000), (700, 5000), (3, 40000)])
def test_alternatives_in_hard_orders(rows, V, kind, dtype, cuda_dev):
    t, x = _orders(rows, V, kind, dtype, cuda_dev)
    ids, dids = _ids(rows, V, V, cuda_dev)
    for top in (1, 4, 5, 32):
        _check(t, x, ids, top, av.avey_token_logprobs(t, dids, top=top))


def test_a_warp_to_each_of_many_rows(cuda_dev):
    rows, V = 7200, 4101
    t, x = _orders(rows, V, "few", torch.float32, cuda_dev)
    ids, dids = _ids(rows, V, V, cuda_dev)
    _check(t, x, ids, 7, av.avey_token_logprobs(t, dids, top=7))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,offset,pad", [(1, 0, 0), (5, 1, 2), (100, 3, 1), (517, 1, 0), (1000, 0, 8), (4085, 7, 3)])
def test_many_short_rows_anywhere(V, offset, pad, dtype, cuda_dev):
    rows = 1301
    t, x = _logits(rows, V, dtype, V, cuda_dev, masked=0.2 if V > 50 else 0.0)
    ids, dids = _ids(rows, V, 3, cuda_dev)
    wide = torch.full((rows * (V + pad) + offset + 16,), float("inf"), dtype=dtype, device=cuda_dev)
    view = wide[offset:offset + rows * (V + pad)].view(rows, V + pad)[:, :V]
    view.copy_(t)
    r = av.avey_token_logprobs(view, dids, top=8)
    _check(view, x, ids, 8, r)
    g, h = torch.randn(rows, device=cuda_dev), torch.randn(rows, device=cuda_dev)
    g[::7], h[::7] = 0, 0
    dense = av.avey_token_logprobs_backward(t, dids, r, g, h)
    want = torch.zeros(rows, V, dtype=torch.float64, device=cuda_dev)
    m, z = r.stats[:, 0].double(), r.stats[:, 1].double()
    lp = torch.clamp(t.double() - m[:, None] - z[:, None], min=-200)
    p = lp.exp()
    gg = torch.where(dids >= 0, g, 0).double()
    want = -p * (gg[:, None] + h.double()[:, None] * (lp + r.entropy.double()[:, None]))
    want[torch.arange(rows), dids.clamp(min=0).long()] += gg
    # p: its exponent has 3 roundings of |lp|, the unit 4u, the bracket 4 roundings
    # of the sum of its terms, the last addition and the output one each
    size = gg.abs()[:, None] + h.double().abs()[:, None] * (lp.abs() + r.entropy.double()[:, None])
    tol = U * (3 * lp.abs() + 12) * p * size + (HALF[dtype] + 2 * U) * want.abs() + 1e-37
    assert bool(((dense.double() - want).abs() <= tol).all())
    assert bool((dense[::7] == 0).all())
    for off2 in (offset, offset + 1):
        buf = torch.full((rows * (V + pad) + off2 + 16,), 5.0, dtype=dtype, device=cuda_dev)
        out = buf[off2:off2 + rows * (V + pad)].view(rows, V + pad)
        av.avey_token_logprobs_backward(view, dids, r, g, h, out=out[:, :V])
        assert torch.equal(out[:, :V], dense)
        assert bool((out[:, V:] == 5).all()) and bool((buf[:off2] == 5).all())
        assert bool((buf[off2 + rows * (V + pad):] == 5).all())
    av.avey_token_logprobs_backward(view, dids, r, g, h, out=view)  # in place
    assert torch.equal(view, dense)
    rest = wide[offset:offset + rows * (V + pad)].view(rows, V + pad)[:, V:]
    assert bool(torch.isinf(rest).all()) and bool(torch.isinf(wide[:offset]).all())
