"""Workloads of the 8-bit products and of the token scoring of the encoder.

``listed()`` and ``draw()`` give cases, ``prepare()`` a case's inputs, ``run()``
one pass: in plain torch operations where ``own`` is false, through the
library where it is true.  ``exact()`` is the same pass from the definitions
in 64 bits, ``work()`` the bytes and operations a pass cannot do without.

Operators (one per case, field "op"):
  linear   y = act(x_q W_q^T * s_x s_w + b) + residual, x quantised per token
           inside the pass, W per output channel beforehand
  logprobs log probabilities of given tokens, row maxima and log sums,
           entropies and the top alternatives of a matrix of logits
  train    log probabilities and entropies, then the gradient of the logits
  score    the 8-bit product with the vocabulary matrix and the scoring of its
           rows in one call: logits are not an output
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the vocabulary head on one token: latency, and one read of the matrix
        dict(name="linear_one_token", op="linear", rows=1, K=768, N=50368, x="f32", out="f32", act=0,
             bias=True, residual=False, prenorm=False),
        # the enricher on one split of 64 tokens: a layer at its shortest sequence
        dict(name="linear_one_split", op="linear", rows=64, K=768, N=1536, x="f32", out="bf16", act=1,
             bias=True, residual=False, prenorm=True),
        # enricher of a batch of 8 sequences of 4096 tokens
        dict(name="linear_enrich", op="linear", rows=32768, K=768, N=1536, x="f32", out="bf16", act=1,
             bias=True, residual=False, prenorm=True),
        # fuser of a wide layer with its residual, whole in fp32
        dict(name="linear_fuse", op="linear", rows=16384, K=2048, N=1024, x="bf16", out="f32", act=0,
             bias=False, residual=True, prenorm=False),
        # ragged everywhere: an odd number of tokens, odd channel counts
        dict(name="linear_ragged", op="linear", rows=1003, K=999, N=2045, x="bf16", out="f32", act=0,
             bias=True, residual=False, prenorm=False),
        # the alternatives of one masked token
        dict(name="logprobs_one_token", op="logprobs", rows=1, V=50368, x="f32", top=8, masked=0.0),
        # every masked token (a fifth) of 8 sequences of 4096
        dict(name="logprobs_masked_lm", op="logprobs", rows=6554, V=50368, x="bf16", top=8, masked=0.0),
        # an odd vocabulary of which a third is excluded, many alternatives
        dict(name="logprobs_ragged", op="logprobs", rows=701, V=30011, x="f32", top=32, masked=0.3),
        # the loss of the same masked tokens and its gradient
        dict(name="train_masked_lm", op="train", rows=6554, V=50368, x="bf16", masked=0.0),
        dict(name="train_ragged", op="train", rows=517, V=50021, x="f32", masked=0.3),
        # scores of a few tokens, and of every masked token of 8 sequences
        dict(name="score_few", op="score", rows=12, K=768, N=50368, x="f32", bias=True),
        dict(name="score_masked_lm", op="score", rows=6554, K=768, N=50368, x="f32", bias=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "logprobs", "train", "score"])
    if op == "linear":
        K, N = _log_int(rng, 64, 2048), _log_int(rng, 96, 50368)
        rows = _log_int(rng, 1, min(32768, max(1, 300_000_000 // N)))
        residual = rng.random() < 0.3
        return dict(op=op, rows=rows, K=K, N=N, x=rng.choice(["f32", "bf16"]),
                    out="f32" if residual else rng.choice(["f32", "bf16"]),
                    act=0 if residual else rng.choice([0, 1]), bias=rng.random() < 0.6,
                    residual=residual, prenorm=rng.random() < 0.3)
    if op == "score":
        K, N = _log_int(rng, 64, 1024), _log_int(rng, 1000, 65536)
        rows = _log_int(rng, 1, min(16384, max(1, 250_000_000_000 // (K * N))))
        return dict(op=op, rows=rows, K=K, N=N, x=rng.choice(["f32", "bf16"]), bias=rng.random() < 0.6)
    V = _log_int(rng, 200, 131072)
    rows = _log_int(rng, 1, min(32768, max(1, 300_000_000 // V)))
    case = dict(op=op, rows=rows, V=V, x=rng.choice(["f32", "bf16"]),
                masked=rng.choice([0.0, 0.0, 0.3]))
    if op == "logprobs":
        case["top"] = rng.choice([0, 1, 3, 8, 17, 32])
    return case


def _weights(N, K, g):
    """Weights N(0, 1/K) as 8-bit integers with a scale for each channel; the
    storage rows are padded to 16 bytes."""
    W = torch.randn((N, K), generator=g, device=DEV) / math.sqrt(K)
    scale = W.abs().amax(1) / 127.0
    q = torch.zeros((N, (K + 15) // 16 * 16), dtype=torch.int8, device=DEV)
    q[:, :K] = torch.round(W.double() / scale.double()[:, None]).clamp(-127, 127).to(torch.int8)
    return q, scale


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    T, s = case["rows"], {"case": case}
    if case["op"] in ("linear", "score"):
        K, N = case["K"], case["N"]
        # activations of a residual stream: a few tokens and features much larger than the rest
        x = torch.randn((T, K), generator=g, device=DEV)
        x *= torch.exp(0.5 * torch.randn((T, 1), generator=g, device=DEV))
        x *= torch.exp(0.3 * torch.randn((1, K), generator=g, device=DEV))
        s["x"] = x.to(TYPES[case["x"]])
        s["wq"], s["ws"] = _weights(N, K, g)
        s["bias"] = torch.randn((N,), generator=g, device=DEV) * 0.1 if case["bias"] else None
        if case["op"] == "linear":
            s["residual"] = torch.randn((T, N), generator=g, device=DEV) if case["residual"] else None
        else:
            s["ids"] = torch.randint(0, N, (T,), generator=g, device=DEV, dtype=torch.int32)
            s["ids"][torch.rand((T,), generator=g, device=DEV) < 0.05] = -1
        if own:
            import attention_free_long_b200 as av
            s["av"] = av
            s["lin"] = av.QuantLinear(s["wq"], s["ws"], K, s["bias"])
            if case["op"] == "score":
                s["work"] = av.score_workspace(T, s["lin"])
        return s
    V = case["V"]
    # a masked token: most words unlikely, a few far ahead
    x = torch.randn((T, V), generator=g, device=DEV) * 2.0
    ahead = torch.randint(0, V, (T, 4), generator=g, device=DEV)
    x.scatter_add_(1, ahead, 10.0 * torch.rand((T, 4), generator=g, device=DEV))
    ids = torch.where(torch.rand((T,), generator=g, device=DEV) < 0.5, ahead[:, 0],
                      torch.randint(0, V, (T,), generator=g, device=DEV))
    if case["masked"]:
        out = torch.rand((V,), generator=g, device=DEV) < case["masked"]
        out[0] = False
        x.masked_fill_(out[None, :], float("-inf"))
        ids = torch.where(out[ids], torch.zeros_like(ids), ids)
    s["x"] = x.to(TYPES[case["x"]])
    ids = ids.to(torch.int32)
    ids[torch.rand((T,), generator=g, device=DEV) < 0.05] = -1  # rows without a given token
    s["ids"] = ids
    if case["op"] == "train":
        s["d_logprob"] = torch.randn((T,), generator=g, device=DEV) / T
        s["d_entropy"] = 0.01 * torch.randn((T,), generator=g, device=DEV) / T
    if own:
        import attention_free_long_b200 as av
        s["av"] = av
    return s


# ------------------------------------------------------------- plain forms --

def _plain_quantized(x, prenorm):
    """Whole numbers -127..127 as fp32, and the scale of each row."""
    xf = x.float()
    amax = xf.abs().amax(1)
    scale = amax / 127.0
    step = torch.where(scale > 0, scale, torch.ones_like(scale))
    q = torch.round(xf.double() / step.double()[:, None]).clamp(-127, 127).float()
    if prenorm:
        scale = scale / torch.sqrt((xf * xf).mean(1) + 1e-6)
    return q, scale


def _plain_product(s, prenorm):
    K = s["case"]["K"]
    q, scale = _plain_quantized(s["x"], prenorm)
    y = (q @ s["wq"][:, :K].float().t()) * scale[:, None] * s["ws"][None, :]
    return y if s["bias"] is None else y + s["bias"][None, :]


def _plain_stats(x):
    m = x.amax(1)
    e = torch.exp(x - m[:, None])
    z = e.sum(1)
    d = torch.where(e > 0, x - m[:, None], torch.zeros_like(x))
    entropy = torch.log(z) - (e * d).sum(1) / z
    return torch.stack([m, torch.log(z)], 1), entropy


def _plain_given(x, ids, stats):
    at = ids.long().clamp(min=0)
    lp = x.gather(1, at[:, None])[:, 0] - stats[:, 0] - stats[:, 1]
    return torch.where(ids >= 0, lp, torch.zeros_like(lp))


def _plain_top(x, stats, k):
    left = x.clone()
    place = torch.arange(x.shape[1], device=x.device)
    ids, lps = [], []
    for _ in range(k):
        v = left.amax(1)
        i = torch.where(left == v[:, None], place[None, :], x.shape[1]).amin(1)
        left.scatter_(1, i[:, None], float("-inf"))
        ids.append(i.to(torch.int32))
        lps.append(v - stats[:, 0] - stats[:, 1])
    return torch.stack(ids, 1), torch.stack(lps, 1)


def _plain(s):
    case = s["case"]
    if case["op"] == "linear":
        y = _plain_product(s, case["prenorm"])
        if case["act"]:
            y = torch.clamp(y, min=0.0) ** 2
        if s["residual"] is not None:
            y = y + s["residual"]
        return y.to(TYPES[case["out"]])
    if case["op"] == "score":
        x = _plain_product(s, False)
        stats, entropy = _plain_stats(x)
        return _plain_given(x, s["ids"], stats), stats, entropy
    x = s["x"].float()
    stats, entropy = _plain_stats(x)
    lp = _plain_given(x, s["ids"], stats)
    if case["op"] == "logprobs":
        out = [lp, stats, entropy]
        return out + list(_plain_top(x, stats, case["top"])) if case["top"] else out
    logp = x - stats[:, :1] - stats[:, 1:]
    p = torch.exp(logp)
    given = (s["ids"] >= 0).float()
    dl = s["d_logprob"] * given
    safe = torch.where(p > 0, logp, torch.zeros_like(logp))
    dx = -p * (dl[:, None] + s["d_entropy"][:, None] * (safe + entropy[:, None]))
    dx.scatter_add_(1, s["ids"].long().clamp(min=0)[:, None], dl[:, None])
    return lp, entropy, dx.to(s["x"].dtype)


# ------------------------------------------------------------------ a pass --

def run(s):
    if not own:
        return _plain(s)
    av, case = s["av"], s["case"]
    if case["op"] == "linear":
        return av.avey_linear_i8(s["x"], s["lin"], act=case["act"], residual=s["residual"],
                                 prenorm=case["prenorm"], out_dtype=TYPES[case["out"]])
    if case["op"] == "score":
        r = av.avey_score_tokens_i8(s["x"], s["lin"], s["ids"], ws=s["work"])
        return r.logprob, r.stats, r.entropy
    if case["op"] == "logprobs":
        r = av.avey_token_logprobs(s["x"], s["ids"], top=case["top"])
        out = [r.logprob, r.stats, r.entropy]
        return out + [r.top_ids, r.top_logprobs] if case["top"] else out
    r = av.avey_token_logprobs(s["x"], s["ids"])
    dx = av.avey_token_logprobs_backward(s["x"], s["ids"], r, s["d_logprob"], s["d_entropy"])
    return r.logprob, r.entropy, dx


# ------------------------------------------------------------------- exact --

def _exact_rows(case, s, lo, hi):
    """Rows lo..hi-1 of every output, in 64 bits from the definitions."""
    if case["op"] in ("linear", "score"):
        x = s["x"][lo:hi].double()
        # the scale of a row is an fp32 number by definition
        step = (s["x"][lo:hi].float().abs().max(1).values / 127.0).double()
        level = torch.round(x / step.clamp(min=1e-300)[:, None])
        level = torch.minimum(torch.maximum(level, torch.full_like(level, -127)), torch.full_like(level, 127))
        value = level * step[:, None]
        if case.get("prenorm"):
            value = value * (x.pow(2).sum(1) / case["K"] + 1e-6).rsqrt()[:, None]
        W = s["wq"][:, :case["K"]].double() * s["ws"].double()[:, None]
        y = torch.einsum("tk,nk->tn", value, W)
        if s["bias"] is not None:
            y += s["bias"].double()
        if case["op"] == "linear":
            if case["act"]:
                y = y.relu().square()
            if s["residual"] is not None:
                y = y + s["residual"][lo:hi].double()
            return [y]
    else:
        y = s["x"][lo:hi].double()
    ids = s["ids"][lo:hi].long()
    has = ids.ge(0)
    top = y.max(1).values
    lse = torch.logsumexp(y, 1)
    logp = y - lse[:, None]
    p = logp.exp()
    entropy = -torch.nan_to_num(p * logp, nan=0.0, posinf=0.0, neginf=0.0).sum(1)
    given = torch.where(has, logp[torch.arange(hi - lo, device=DEV), ids.clamp(min=0)], 0.0)
    stats = torch.stack([top, lse - top], 1)
    if case["op"] == "score":
        return [given, stats, entropy]
    if case["op"] == "logprobs":
        out = [given, stats, entropy]
        if case["top"]:
            v, i = torch.sort(logp, dim=1, descending=True, stable=True)
            out += [i[:, :case["top"]].to(torch.int32), v[:, :case["top"]].contiguous()]
        return out
    dl = s["d_logprob"][lo:hi].double() * has
    dh = s["d_entropy"][lo:hi].double()
    hot = torch.zeros_like(y)
    hot[has, ids[has]] = 1.0
    dx = dl[:, None] * (hot - p) - dh[:, None] * torch.nan_to_num(p * (logp + entropy[:, None]), nan=0.0,
                                                                posinf=0.0, neginf=0.0)
    return [given, entropy, dx]


def exact(case, seed):
    global own
    before, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = before
    width = case.get("V", case.get("N"))
    step = max(1, 60_000_000 // width)
    parts = [_exact_rows(case, s, lo, min(lo + step, case["rows"])) for lo in range(0, case["rows"], step)]
    out = [torch.cat(list(p), 0) for p in zip(*parts)]
    return out[0] if case["op"] == "linear" else out


# -------------------------------------------------------------------- work --

def work(case):
    T = case["rows"]
    size = {"f32": 4, "bf16": 2}
    if case["op"] in ("linear", "score"):
        K, N = case["K"], case["N"]
        b = T * K * size[case["x"]] + N * K + 4 * N + (4 * N if case["bias"] else 0)
        f = 2 * T * N * K
        if case["op"] == "linear":
            b += T * N * size[case["out"]] + (4 * T * N if case["residual"] else 0)
        else:
            b += T * 20
            f += 6 * T * N
        return {"bytes": b, "flops": f}
    V, e = case["V"], size[case["x"]]
    if case["op"] == "logprobs":
        return {"bytes": T * V * e + T * (20 + 8 * case["top"]), "flops": 6 * T * V}
    return {"bytes": 2 * T * V * e + T * 24, "flops": 14 * T * V}
