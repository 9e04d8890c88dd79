"""8-bit products and scores called by two host threads at once, on streams and
with weights of their own: one call's launch depends on nothing that another call
of the same kernel sets.  The two lengths of a pair need different amounts of
shared memory from one kernel."""
import ctypes
import threading

import pytest
import torch

import attention_free_long_b200 as av

pytestmark = pytest.mark.gpu


def _caller(op, rows, K, N, dev):
    """(call, outputs, tensors to keep): one call of the C entry, arguments laid out once."""
    g = torch.Generator(device=dev).manual_seed(K)
    W = torch.randint(-127, 128, (N, (K + 15) // 16 * 16), device=dev, generator=g, dtype=torch.int8)
    lin = av.QuantLinear(W, torch.rand(N, device=dev, generator=g) / K, K)
    r = av.avey_quantize_rows(torch.randn(rows, K, device=dev, generator=g))
    stream = torch.cuda.Stream(dev)
    p, st, ld = lin._params(av.AVEY_ACT_NONE), stream.cuda_stream, r.q.shape[1]
    if op == "product":
        out = torch.empty(rows, N, dtype=torch.bfloat16, device=dev)
        args = (ctypes.byref(p), r.q.data_ptr(), av.AVEY_I8, ld, r.scale.data_ptr(), 0, rows, None, 0,
                out.data_ptr(), av.AVEY_BF16, N, None, 0, st)
        fn = av.lib().avey_linear_i8
        ws = None
    else:
        out = torch.empty(rows, 2, device=dev)
        ws = av.score_workspace(rows, lin)
        args = (ctypes.byref(p), r.q.data_ptr(), av.AVEY_I8, ld, r.scale.data_ptr(), 0, rows, None, None,
                out.data_ptr(), None, ws.data_ptr(), ws.numel(), st)
        fn = av.lib().avey_score_tokens_i8
    return (lambda: fn(*args)), out, (lin, r, p, ws, stream)


@pytest.mark.parametrize("op,rows,N,lengths", [
    ("product", 256, 18944, (64, 768)),   # rows of x resident in shared memory
    ("score", 300, 5000, (64, 768)),
    ("product", 4, 1000, (6200, 12000)),  # the few-row kernel past 48 KB
    ("score", 4, 1000, (6200, 12000)),
])
def test_two_threads_with_unlike_lengths(op, rows, N, lengths, cuda_dev):
    calls = [_caller(op, rows, K, N, cuda_dev) for K in lengths]
    want = []
    torch.cuda.synchronize()
    for call, out, _ in calls:
        assert call() == 0
        torch.cuda.synchronize()
        want.append(out.clone())
    refused = []
    start = threading.Barrier(2)

    def work(call):
        start.wait()
        for _ in range(3000):
            code = call()
            if code:
                refused.append((code, av.lib().avey_last_error_detail()))
                return

    threads = [threading.Thread(target=work, args=(call,)) for call, _, _ in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert refused == []
    for (_, out, _), w in zip(calls, want):
        assert torch.equal(out, w)
    assert av.device_status() == 0
