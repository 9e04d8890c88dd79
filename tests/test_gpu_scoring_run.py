"""The 8-bit products and the token scoring as they are used together: an
encoder with 8-bit layers, a vocabulary head on its hidden states, the scores of
given words, the alternatives of masked ones and the gradient of the loss."""
import numpy as np
import pytest
import torch

import attention_free_long_b200 as av
import synthetic as sy

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _setup(dev, prenorm=True, S=64, N=1000, B=2):
    wl = sy.custom("scored", B=B, N=N, S=S, d=136, m=272, m_h=136, k=3,
                   pattern=(sy.STATIC, sy.DYNAMIC, sy.STATIC), centers=8, sigma=0.5, prenorm=prenorm)
    W = sy.gen_weights(wl)
    x = torch.from_numpy(sy.gen_embeddings(wl).X).to(dev, torch.bfloat16)
    P = torch.from_numpy(W.P).to(dev, torch.bfloat16)
    return wl, x, P, av.device_layers(W, torch.bfloat16, dev)


def _head(V, d, dev, seed=3):
    g = torch.Generator(device="cpu").manual_seed(seed)
    E = (torch.randn(V, d, generator=g) / d ** 0.5).to(dev)
    return av.quantize_linear(E, torch.randn(V, generator=g).to(dev) * 0.1)


@pytest.mark.parametrize("prenorm", [False, True])
@pytest.mark.parametrize("S", [16, 64])
def test_layers_are_their_products_and_mixes(S, prenorm, cuda_dev):
    wl, x, P, layers = _setup(cuda_dev, prenorm, S)
    q = av.quantize_layers(layers)
    ws = av.make_workspace(wl.B, wl.N, wl.d, wl.S, wl.k, wl.m, torch.bfloat16, prenorm, cuda_dev, quantized=True)
    out = av.encoder_forward(x, P, q, wl.S, wl.k, wl.m_h, wl.eps, prenorm, ws=ws)
    bare = av.encoder_forward(x, P, q, wl.S, wl.k, wl.m_h, wl.eps, prenorm)
    # the same, call by call
    idx, w = av.avey_rank(x, wl.S, wl.k)
    h, _ = av.avey_compress(x, wl.S, wl.k, idx, w, P, lowp=False)
    h = h.view(-1, wl.d)
    for lay in q:
        z = av.avey_linear_i8(h, lay.U, act=av.AVEY_ACT_RELU2, prenorm=prenorm, pair=True)
        tail = z[:, :, wl.m_h:].contiguous()
        c = (av.avey_static_mix(lay.V, tail, wl.S) if lay.kind == av.AVEY_STATIC
             else av.avey_dynamic_mix(tail, wl.S, wl.eps))
        z[:, :, wl.m_h:] = c
        h = av.avey_linear_i8(z, lay.O, residual=h)
    torch.cuda.synchronize()
    assert av.device_status() == 0
    assert torch.equal(out.reshape(-1, wl.d), h) and torch.equal(bare, out)


def test_one_layer_stays_near_the_16_bit_one(cuda_dev):
    # one static layer on the same input: the enricher's rounding moves Z by at
    # most dZ (half a step of x and of U, squared by ReLU^2), V and O carry it,
    # and the fuser rounds Z and O again
    wl, x, P, layers = _setup(cuda_dev, prenorm=False)
    lay, q = layers[0], av.quantize_layers(layers[:1])[0]
    T = 512
    h = torch.randn(T, wl.d, device=cuda_dev, generator=torch.Generator(device=cuda_dev).manual_seed(1))
    want, _ = av.avey_layer_forward(lay, wl.S, wl.m_h, wl.eps, False, h)
    z = av.avey_linear_i8(h, q.U, act=av.AVEY_ACT_RELU2, pair=True)
    z[:, :, wl.m_h:] = av.avey_static_mix(q.V, z[:, :, wl.m_h:].contiguous(), wl.S)
    got = av.avey_linear_i8(z, q.O, residual=h)
    D = lambda t: t.double().cpu().numpy()
    A, Ut, Ot, V = D(h), D(lay.Ut), D(lay.Ot), D(lay.V)
    s = np.abs(A).max(1)[:, None] / 127
    pre = A @ Ut.T + D(lay.bU)[None]
    xq = np.abs(A).sum(1)[:, None] + s / 2 * wl.d
    dpre = s / 2 * np.abs(Ut).sum(1)[None] + D(q.U.scale)[None] / 2 * xq
    zmax = np.maximum(pre + dpre, 0)
    zlo = np.maximum(pre, 0)
    dz, zz = zmax ** 2 - np.minimum(zlo, np.maximum(pre - dpre, 0)) ** 2, zmax ** 2
    blocks = dz[:, wl.m_h:].reshape(-1, wl.S, wl.m - wl.m_h)
    dz[:, wl.m_h:] = np.einsum("ij,bjf->bif", np.abs(V), blocks).reshape(T, -1)
    zb = zz[:, wl.m_h:].reshape(-1, wl.S, wl.m - wl.m_h)
    zz[:, wl.m_h:] = np.einsum("ij,bjf->bif", np.abs(V), zb).reshape(T, -1)
    s2 = zz.max(1)[:, None] / 127
    bound = (dz + s2 / 2) @ np.abs(Ot).T + D(q.O.scale)[None] / 2 * (zz + s2 / 2).sum(1)[:, None]
    # both layers round in fp32 and to pairs (2^-16) besides
    bound = bound * 1.001 + 1e-3 * np.abs(D(want)).max()
    assert (np.abs(D(got) - D(want)) <= bound).all()


@pytest.mark.parametrize("rows,V,d", [(r, V, 136) for r in (1, 9, 17, 32, 33, 700) for V in (1, 1000, 5003)]
                         + [(300, 3001, 1040), (2600, 700, 64), (40, 70000, 72), (1, 50368, 768), (8, 20011, 1025),
                            (16, 60001, 100), (12, 9000, 1100)])
def test_score_is_product_then_scores(rows, V, d, cuda_dev):
    head = _head(V, d, cuda_dev)
    g = torch.Generator(device=cuda_dev).manual_seed(rows)
    h = torch.randn(rows, d, device=cuda_dev, generator=g) * 4
    ids = torch.randint(-1, V, (rows,), device=cuda_dev, generator=g, dtype=torch.int32)
    for x in (h, h.to(torch.bfloat16), av.avey_quantize_rows(h)):
        logits = av.avey_linear_i8(x, head).double()
        r = av.avey_score_tokens_i8(x, head, ids)
        torch.cuda.synchronize()
        assert av.device_status() == 0
        lse = torch.logsumexp(logits, 1)
        p = torch.softmax(logits, 1)
        H = -(p * (logits - lse[:, None])).sum(1)
        lp = torch.where(ids >= 0, logits.gather(1, ids.clamp(min=0).long()[:, None])[:, 0] - lse,
                         torch.zeros_like(lse))
        # The kernel works on logits times log2 e, y = fma(acc (s log2 e), w, b log2 e), and
        # goes back with ln 2.  Either constant is off by u / 2 at most: 2.5u of the product
        # p = acc s w, 1.5u of b, 2.5u of y; the fp32 logits compared with are off by u of p
        # and u of y.  With |p| <= |y| + |b|: (7 |y| + 5 |b|) u for a logit.  Sums as in the
        # scoring's own tests: (3 D + V / 256 + 160) u, twice that times H + z for the entropy.
        big = 7 * (logits.abs().amax(1) + head.bias.double().abs().amax())
        far = (logits.amax(1) - logits.amin(1)).clamp(max=60.0)
        tol = (2 * big + 3 * far + V / 256 + 160) * U
        z = lse - logits.amax(1)
        assert bool(((r.stats[:, 0].double() - logits.amax(1)).abs() <= U * big).all())
        assert bool(((r.stats[:, 1].double() - z).abs() <= tol + 2 * U * z.abs()).all())
        assert bool(((r.logprob.double() - lp).abs() <= 2 * tol + 4 * U * lp.abs()).all())
        assert bool(((r.entropy.double() - H).abs() <= tol * (2 + 3 * (H + z.abs()))).all())


def test_score_many_rows_in_a_small_workspace(cuda_dev):
    head = _head(60000, 64, cuda_dev)
    h = torch.randn(3000, 64, device=cuda_dev) * 3
    ids = torch.randint(0, 60000, (3000,), device=cuda_dev, dtype=torch.int32)
    ws = av.score_workspace(3000, head)
    r = av.avey_score_tokens_i8(h, head, ids, ws=ws)
    parts = [av.avey_score_tokens_i8(h[i:i + 1000], head, ids[i:i + 1000], ws=ws) for i in (0, 1000, 2000)]
    for a, b in ((r.logprob, [p.logprob for p in parts]), (r.entropy, [p.entropy for p in parts]),
                 (r.stats, [p.stats for p in parts])):
        torch.testing.assert_close(a, torch.cat(b), rtol=1e-5, atol=1e-5)
    assert ws.numel() < 3000 * 60000 * 4


def test_score_spoilt_and_ignored_rows(cuda_dev):
    head = _head(2000, 64, cuda_dev)
    for rows in (4, 20, 300):
        h = torch.randn(rows, 64, device=cuda_dev)
        ids = torch.full((rows,), 5, dtype=torch.int32, device=cuda_dev)
        ids[1], ids[2] = -1, 2000
        clean = av.avey_score_tokens_i8(h, head, ids)
        assert av.device_status() == 5
        h[0, 3] = float("nan")
        h[3] = 0
        r = av.avey_score_tokens_i8(h, head, ids)
        assert av.device_status() == 5
        assert r.logprob[1] == 0 and r.logprob[2] == 0
        assert bool(torch.isnan(r.logprob[0])) and bool(torch.isnan(r.entropy[0])) and bool(torch.isnan(r.stats[0]).all())
        lp = torch.log_softmax(head.bias.double(), 0)[5]
        assert abs(float(r.logprob[3]) - float(lp)) <= 300 * U
        assert torch.equal(r.logprob[4:], clean.logprob[4:])


@pytest.mark.parametrize("rows", [5, 300])
def test_score_with_words_masked_by_the_bias(rows, cuda_dev):
    V, d = 2100, 64
    head = _head(V, d, cuda_dev)
    g = torch.Generator(device=cuda_dev).manual_seed(2)
    h = torch.randn(rows, d, device=cuda_dev, generator=g) * 3
    free = torch.rand(V, device=cuda_dev, generator=g) < 0.3
    free[1990:] = False  # a tile's last columns too
    free[7] = True
    open_words = torch.nonzero(free)[:, 0]
    part = av.QuantLinear(head.q[open_words].contiguous(), head.scale[open_words], d, head.bias[open_words])
    ids = torch.randint(0, open_words.numel(), (rows,), device=cuda_dev, generator=g, dtype=torch.int32)
    want = av.avey_score_tokens_i8(h, part, ids)
    for low in (float("-inf"), torch.finfo(torch.float32).min):
        bias = torch.where(free, head.bias, torch.full_like(head.bias, low))
        r = av.avey_score_tokens_i8(h, av.QuantLinear(head.q, head.scale, d, bias),
                                    open_words[ids.long()].to(torch.int32))
        for a, b in ((r.logprob, want.logprob), (r.stats, want.stats), (r.entropy, want.entropy)):
            assert bool(torch.isfinite(a).all())
            # the same terms added in another order: V / 256 + 160 roundings of sums near 1 .. 10
            torch.testing.assert_close(a, b, rtol=200 * U, atol=200 * U)
    none = av.QuantLinear(head.q, head.scale, d, torch.full_like(head.bias, float("-inf")))
    r = av.avey_score_tokens_i8(h, none, ids)
    assert bool((r.logprob == -np.inf).all()) and bool((r.entropy == 0).all())
    assert bool((r.stats[:, 0] == -np.inf).all()) and bool((r.stats[:, 1] == 0).all())


def test_rows_past_32_bit_offsets(cuda_dev):
    # 2.27e9 logits: the last rows lie past 2^31 elements and 2^32 bytes
    V, d, rows, tail = 50368, 64, 45000, 2000
    head = _head(V, d, cuda_dev)
    h = av.avey_quantize_rows(torch.randn(rows, d, device=cuda_dev))
    logits = av.avey_linear_i8(h, head, out_dtype=torch.bfloat16)
    end = av.QuantRows(h.q[-tail:].contiguous(), h.scale[-tail:].contiguous(), d)
    last = av.avey_linear_i8(end, head, out_dtype=torch.bfloat16)
    assert torch.equal(logits[-tail:], last)
    ids = torch.randint(0, V, (rows,), device=cuda_dev, dtype=torch.int32)
    r = av.avey_token_logprobs(logits, ids, top=2)
    e = av.avey_token_logprobs(last, ids[-tail:].contiguous(), top=2)
    for a, b in ((r.logprob, e.logprob), (r.stats, e.stats), (r.top_ids, e.top_ids)):
        assert torch.equal(a[-tail:], b)
    g = torch.ones(rows, device=cuda_dev)
    dlast = av.avey_token_logprobs_backward(last, ids[-tail:].contiguous(), e, g[-tail:].contiguous())
    av.avey_token_logprobs_backward(logits, ids, r, g, out=logits)
    assert torch.equal(logits[-tail:], dlast)
    assert av.device_status() == 0


def test_encoder_to_fill_mask_and_loss(cuda_dev):
    wl, x, P, layers = _setup(cuda_dev)
    q = av.quantize_layers(layers)
    V = 3001
    head = _head(V, wl.d, cuda_dev)
    hidden = av.encoder_forward(x, P, q, wl.S, wl.k, wl.m_h, wl.eps, wl.prenorm).reshape(-1, wl.d)
    rows = torch.arange(0, hidden.shape[0], 5, device=cuda_dev)  # every fifth token is masked
    ids = torch.randint(0, V, (rows.numel(),), device=cuda_dev, dtype=torch.int32)
    h = hidden[rows]
    scored = av.avey_score_tokens_i8(h, head, ids)
    logits = av.avey_linear_i8(h, head)
    assert logits.shape == (rows.numel(), V) and logits.stride(0) == 3008
    full = av.avey_token_logprobs(logits, ids, top=5)
    torch.testing.assert_close(scored.logprob, full.logprob, rtol=1e-5, atol=1e-5)
    torch.testing.assert_close(scored.entropy, full.entropy, rtol=1e-5, atol=1e-5)
    best = logits.double().topk(5, dim=1)
    assert torch.equal(logits.gather(1, full.top_ids.long()).double(), best.values)
    # the loss -mean(logprob) and its gradient, against autograd in 64 bits
    n = rows.numel()
    dx = av.avey_token_logprobs_backward(logits, ids, full, torch.full((n,), -1.0 / n, device=cuda_dev))
    ref = logits.double().requires_grad_()
    loss = torch.nn.functional.cross_entropy(ref, ids.long())
    loss.backward()
    assert abs(float(-full.logprob.mean()) - loss.item()) <= 1e-5 * loss.item()
    torch.testing.assert_close(dx.double(), ref.grad, rtol=1e-4, atol=1e-9)
    torch.cuda.synchronize()
    assert av.device_status() == 0


@pytest.mark.parametrize("world", [2, 3])
def test_sequence_shares_of_8_bit_layers(world, cuda_dev):
    wl, x, P, layers = _setup(cuda_dev, S=64, N=1000, B=2)
    q = av.quantize_layers(layers)
    full = av.encoder_forward(x, P, q, wl.S, wl.k, wl.m_h, wl.eps, wl.prenorm)
    _, _, scores = av.avey_rank(x, wl.S, wl.k, return_scores=True)
    n = scores.shape[1]
    for rank in range(world):
        # the sum over the ranks is the whole matrix
        out = av.encoder_forward_sharded(x, P, q, wl.S, wl.k, wl.m_h, wl.eps, wl.prenorm, rank, world,
                                         lambda s: s.copy_(scores))
        t0, t1 = av.shard_targets(n, world, rank)
        assert torch.equal(out, full[:, t0 * wl.S:t1 * wl.S])
    assert av.device_status() == 0


def test_captured_run(cuda_dev):
    wl, x, P, layers = _setup(cuda_dev, N=640)
    q = av.quantize_layers(layers)
    head = _head(999, wl.d, cuda_dev)
    ids = torch.randint(0, 999, (wl.B * 640,), device=cuda_dev, dtype=torch.int32)
    ws = av.make_workspace(wl.B, wl.N, wl.d, wl.S, wl.k, wl.m, torch.bfloat16, wl.prenorm, cuda_dev, quantized=True)
    sws = av.score_workspace(wl.B * 640, head)

    def step():
        h = av.encoder_forward(x, P, q, wl.S, wl.k, wl.m_h, wl.eps, wl.prenorm, ws=ws).reshape(-1, wl.d)
        return av.avey_score_tokens_i8(h, head, ids, ws=sws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = step()
    x.copy_(x.flip(1).contiguous())
    graph.replay()
    torch.cuda.synchronize()
    e = step()
    assert torch.equal(r.logprob, e.logprob) and torch.equal(r.entropy, e.entropy)


def test_stack_refuses(cuda_dev):
    wl, x, P, layers = _setup(cuda_dev)
    q = av.quantize_layers(layers)
    go = lambda xx, ll, m_h=wl.m_h: av.encoder_forward(xx, P, ll, wl.S, wl.k, m_h, wl.eps, False)
    with pytest.raises(TypeError):
        go(x, [q[0], layers[1]])
    with pytest.raises(ValueError):
        go(x, q, m_h=100)
    with pytest.raises(ValueError):
        go(x, [av.QuantLayer(av.AVEY_STATIC, q[0].U, None, q[0].O)])
    with pytest.raises(ValueError):
        av.avey_linear_i8(torch.zeros(3, 8, device=cuda_dev), q[0].U)
    with pytest.raises(TypeError):
        av.encoder_forward_uncompressed(x, q, wl.S, wl.k, wl.m_h, wl.eps, False)
