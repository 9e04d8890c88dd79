"""The first CUDA call of a host thread may be one of the library's: a thread of a
server that was handed tensors, weights and workspaces made by another one."""
import threading

import pytest
import torch

import attention_free_long_b200 as av
import synthetic as sy

pytestmark = pytest.mark.gpu


def _in_a_new_thread(call):
    got = []

    def work():
        try:
            got.append(call())
        except Exception as e:  # shown by the assertion below
            got.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    return got[0]


@pytest.mark.parametrize("rows,N", [(3, 200), (40, 20000), (300, 5000)])
def test_product_and_scores(rows, N, cuda_dev):
    g = torch.Generator(device=cuda_dev).manual_seed(N)
    lin = av.quantize_linear(torch.randn(N, 100, device=cuda_dev, generator=g))
    x = av.avey_quantize_rows(torch.randn(rows, 100, device=cuda_dev, generator=g))
    want, scores = av.avey_linear_i8(x, lin), av.avey_score_tokens_i8(x, lin)
    out, ws = torch.empty_like(want), av.score_workspace(rows, lin)
    torch.cuda.synchronize()
    got = _in_a_new_thread(lambda: av.avey_linear_i8(x, lin, out=out))
    assert got is out and torch.equal(out, want)
    r = _in_a_new_thread(lambda: av.avey_score_tokens_i8(x, lin, ws=ws))
    assert torch.equal(r.stats, scores.stats) and torch.equal(r.entropy, scores.entropy)
    assert av.device_status() == 0


@pytest.mark.parametrize("quantized", [False, True])
def test_encoder(quantized, cuda_dev):
    wl = sy.custom("thread", B=2, N=500, S=64, d=128, m=256, k=3, pattern=(sy.STATIC, sy.DYNAMIC), centers=6,
                   sigma=0.5, prenorm=True)
    W = sy.gen_weights(wl)
    x = torch.from_numpy(sy.gen_embeddings(wl).X).to(cuda_dev, torch.bfloat16)
    P = torch.from_numpy(W.P).to(cuda_dev, torch.bfloat16)
    layers = av.device_layers(W, torch.bfloat16, cuda_dev)
    if quantized:
        layers = av.quantize_layers(layers)
    args = (x, P, layers, wl.S, wl.k, wl.m_h, wl.eps, True)
    want = av.encoder_forward(*args).clone()
    ws = av.make_workspace(wl.B, wl.N, wl.d, wl.S, wl.k, wl.m, torch.bfloat16, True, cuda_dev, quantized=quantized)
    torch.cuda.synchronize()
    got = _in_a_new_thread(lambda: av.encoder_forward(*args, ws=ws))
    assert torch.equal(got, want)
    idx, w = ws.idx.clone(), ws.w.clone()
    got = _in_a_new_thread(lambda: av.processor_forward(*args, idx, w, ws=ws).clone())
    assert torch.equal(got, want)
    assert av.device_status() == 0
