"""Refusals of the 8-bit products and of the token scoring that need no GPU:
every call below is rejected on the host, before CUDA is touched, and says why."""
import ctypes

import pytest
import torch

import attention_free_long_b200 as av

A = 0x100000  # 256-byte aligned addresses, never dereferenced
O = 0x900000
vp = ctypes.c_void_p


def _refused(code, want, word):
    assert code == want
    assert word in av.lib().avey_last_error_detail().decode()


def _quantize(**kw):
    a = dict(x=A, dt=av.AVEY_F32, rows=4, cols=40, ld=40, q=A, ld_q=48, scale=A)
    a.update(kw)
    return av.lib().avey_quantize_rows(a["x"], a["dt"], a["rows"], a["cols"], a["ld"], 0, a["q"], a["ld_q"],
                                       a["scale"], None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(x=None), 1, "null"), (dict(q=None), 1, "null"), (dict(scale=None), 1, "null"),
    (dict(rows=-1), 1, "rows"), (dict(cols=0), 1, "cols"), (dict(ld=39), 1, "ld_x"),
    (dict(ld_q=40), 1, "ld_q"), (dict(ld_q=32), 1, "ld_q"), (dict(dt=av.AVEY_I8), 2, "dtype"),
    (dict(x=A + 2), 1, "aligned"), (dict(q=A + 8), 1, "aligned"), (dict(scale=A + 2), 1, "aligned"),
    (dict(cols=(1 << 30) + 1, ld=1 << 31, ld_q=1 << 31), 2, "2^30"),
    (dict(), 1, "overlaps"), (dict(q=A + 512), 1, "overlaps"), (dict(q=A - 176), 1, "overlaps"),
    (dict(dt=av.AVEY_BF16X2, q=A + 624), 1, "overlaps"),
])
def test_quantize_rows_refuses(kw, code, word):
    _refused(_quantize(**kw), code, word)


def _params(**kw):
    a = dict(K=40, N=24, Wq=A, ld_w=48, w_scale=A, bias=None, act=0)
    a.update(kw)
    return av.LinearI8Params(a["K"], a["N"], a["Wq"], a["ld_w"], a["w_scale"], a["bias"], a["act"])


def _linear(p=None, **kw):
    a = dict(x=A, dt=av.AVEY_F32, ld=40, xs=None, prenorm=0, rows=40, res=None, ldr=24, out=O, odt=av.AVEY_F32, ldo=24,
             ws=A, wsb=1 << 20)
    a.update(kw)
    q = _params() if p is None else p
    return av.lib().avey_linear_i8(ctypes.byref(q), a["x"], a["dt"], a["ld"], a["xs"], a["prenorm"], a["rows"],
                                   a["res"], a["ldr"], a["out"], a["odt"], a["ldo"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("pk,kw,code,word", [
    (dict(K=0), {}, 1, "K"), (dict(N=0), {}, 1, "N"), (dict(act=2), {}, 1, "act"),
    (dict(K=131072, ld_w=131072), dict(ld=131072), 2, "int32"),
    (dict(ld_w=40), {}, 1, "ld_w"), (dict(ld_w=32), {}, 1, "ld_w"), (dict(Wq=None), {}, 1, "null"),
    (dict(w_scale=None), {}, 1, "null"), (dict(Wq=A + 8), {}, 1, "aligned"), (dict(bias=A + 4), {}, 1, "aligned"),
    (dict(w_scale=A + 4), {}, 1, "aligned"),
    ({}, dict(rows=-1), 1, "rows"), ({}, dict(x=None), 1, "null"), ({}, dict(out=None), 1, "null"),
    ({}, dict(ld=39), 1, "ld_x"), ({}, dict(xs=A), 1, "x_scale"),
    ({}, dict(dt=av.AVEY_I8, ld=48), 1, "x_scale"), ({}, dict(dt=av.AVEY_I8, ld=40, xs=A), 1, "ld_x"),
    ({}, dict(dt=av.AVEY_I8, ld=48, xs=A, prenorm=1), 1, "prenorm"),
    ({}, dict(dt=av.AVEY_I8, ld=48, xs=A, x=A + 8), 1, "aligned"),
    ({}, dict(dt=7), 2, "dtype"), ({}, dict(odt=av.AVEY_I8), 2, "output dtype"),
    ({}, dict(ldo=20), 1, "ld_out"), ({}, dict(ldo=16), 1, "ld_out"), ({}, dict(out=O + 8), 1, "aligned"),
    ({}, dict(out=A), 1, "overlap"), ({}, dict(out=A + 40 * 160 - 16), 1, "overlap"),
    ({}, dict(x=O + 40 * 96 - 16), 1, "overlap"), ({}, dict(res=O + 16), 1, "overlap"),
    ({}, dict(res=O - 16), 1, "overlap"),
    ({}, dict(res=A, odt=av.AVEY_BF16), 2, "residual"), (dict(act=1), dict(res=A), 2, "residual"),
    ({}, dict(res=A + 2), 1, "aligned"), ({}, dict(res=A, ldr=23), 1, "ld_res"), ({}, dict(res=O, ldr=32), 1, "overlap"), ({}, dict(ws=None), 1, "workspace"),
    ({}, dict(ws=A + 16), 1, "workspace"), ({}, dict(wsb=64), 1, "workspace"),
])
def test_linear_i8_refuses(pk, kw, code, word):
    _refused(_linear(_params(**pk), **kw), code, word)


def test_linear_i8_refuses_null_params_and_sizes_its_workspace():
    L = av.lib()
    assert L.avey_linear_i8(None, A, 0, 40, None, 0, 4, None, 0, A, 0, 24, A, 1 << 20, None) == 1
    assert L.avey_linear_i8_workspace_bytes(av.AVEY_I8, 100, 40) == 0
    assert L.avey_linear_i8_workspace_bytes(av.AVEY_F32, 0, 40) == 0
    # few rows are rounded by the product's own kernel
    assert L.avey_linear_i8_workspace_bytes(av.AVEY_F32, 16, 40) == 0
    assert L.avey_linear_i8_workspace_bytes(av.AVEY_F32, 17, 40) == (17 * 48 + 255) // 256 * 256 + 256
    assert L.avey_linear_i8_workspace_bytes(av.AVEY_F32, 100, 40) == (100 * 48 + 255) // 256 * 256 + 512


def _logprobs(**kw):
    a = dict(x=A, dt=av.AVEY_F32, rows=4, V=50, ld=50, ids=A, top=2, lp=A, st=A, en=A, ti=A, tl=A)
    a.update(kw)
    return av.lib().avey_token_logprobs(a["x"], a["dt"], a["rows"], a["V"], a["ld"], a["ids"], a["top"], a["lp"],
                                        a["st"], a["en"], a["ti"], a["tl"], None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(x=None), 1, "null"), (dict(dt=av.AVEY_BF16X2), 2, "dtype"), (dict(rows=-1), 1, "rows"),
    (dict(V=0), 1, "V"), (dict(ld=49), 1, "leading"), (dict(x=A + 2), 1, "aligned"),
    (dict(top=33), 2, "top"), (dict(top=-1), 1, "top"), (dict(ids=None), 1, "ids"), (dict(lp=None), 1, "ids"),
    (dict(top=0), 1, "top"), (dict(ti=None), 1, "top"), (dict(tl=None), 1, "top"),
    (dict(ids=None, lp=None, st=None, en=None, top=0, ti=None, tl=None), 1, "no output"),
    (dict(st=A + 4), 1, "8-byte"), (dict(ids=A + 2), 1, "4-byte"), (dict(rows=1 << 28), 2, "large"),
    (dict(V=(1 << 30) + 1, ld=1 << 31), 2, "large"),
])
def test_token_logprobs_refuses(kw, code, word):
    _refused(_logprobs(**kw), code, word)


def _grad(**kw):
    a = dict(x=A, dt=av.AVEY_BF16, rows=4, V=50, ld=50, ids=A, st=A, en=A, dl=A, de=A, dx=A, ld_d=50)
    a.update(kw)
    return av.lib().avey_token_logprobs_backward(a["x"], a["dt"], a["rows"], a["V"], a["ld"], a["ids"], a["st"],
                                                 a["en"], a["dl"], a["de"], a["dx"], a["ld_d"], None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(x=None), 1, "null"), (dict(st=None), 1, "null"), (dict(dx=None), 1, "null"),
    (dict(ids=None), 1, "ids"), (dict(en=None), 1, "entropy"), (dict(ld_d=49), 1, "leading"),
    (dict(dx=A + 2), 1, "overlap"), (dict(ld_d=64), 1, "overlap"), (dict(dx=A + 1), 1, "aligned"),
    (dict(dx=A + 398), 1, "overlap"), (dict(dt=av.AVEY_I8), 2, "dtype"),
])
def test_token_logprobs_backward_refuses(kw, code, word):
    _refused(_grad(**kw), code, word)


def _score(p=None, **kw):
    a = dict(x=A, dt=av.AVEY_F32, ld=40, xs=None, rows=4, ids=A, lp=A, st=A, en=A, ws=A, wsb=1 << 28)
    a.update(kw)
    q = _params() if p is None else p
    return av.lib().avey_score_tokens_i8(ctypes.byref(q), a["x"], a["dt"], a["ld"], a["xs"], 0, a["rows"],
                                         a["ids"], a["lp"], a["st"], a["en"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("pk,kw,code,word", [
    (dict(act=1), {}, 2, "act"), ({}, dict(ids=None), 1, "ids"), ({}, dict(lp=None), 1, "ids"),
    ({}, dict(ids=None, lp=None, st=None, en=None), 1, "no output"), ({}, dict(ws=None), 1, "workspace"),
    ({}, dict(wsb=16), 1, "workspace"), ({}, dict(st=A + 4), 1, "8-byte"), ({}, dict(x=None), 1, "null"),
    (dict(K=0), {}, 1, "K"),
])
def test_score_tokens_refuses(pk, kw, code, word):
    _refused(_score(_params(**pk), **kw), code, word)


def test_no_rows_is_no_work():
    # nothing is launched (there is no GPU here) and nothing is asked of the pointers
    assert _quantize(rows=0, x=None, q=None, scale=None) == 0
    assert _linear(rows=0, x=None, out=None, ws=None, wsb=0) == 0
    assert _logprobs(rows=0, x=None) == 0
    assert _grad(rows=0, x=None) == 0
    assert _score(rows=0, x=None, ws=None, wsb=0) == 0


def test_binding_refuses_before_the_library():
    x = torch.zeros(4, 40)
    with pytest.raises(ValueError, match="CUDA"):
        av.avey_token_logprobs(x)
    with pytest.raises(ValueError, match="CUDA"):
        av.avey_quantize_rows(x)
    with pytest.raises(ValueError, match="int8"):
        av.QuantLinear(torch.zeros(4, 48, dtype=torch.int8), torch.ones(4), 40)
    lay = av.DeviceLayer(av.AVEY_COUPLED_CAUSAL, x, x, x, x)
    with pytest.raises(ValueError, match="static or dynamic"):
        av.quantize_layers([lay])
    mixed = [lay, av.QuantLayer(av.AVEY_STATIC, None, None, None)]
    with pytest.raises(TypeError, match="not both"):
        av._quantized(mixed)
    with pytest.raises(TypeError, match="compression"):
        av.encoder_forward_uncompressed(x, mixed[1:], 16, 3, 64, 1e-8, False)
