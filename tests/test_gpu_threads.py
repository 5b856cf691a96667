"""Calls on distinct streams from two host threads: two calls of one kernel that
need different amounts of shared memory must not disturb each other."""
import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

tq = pytest.importorskip("kv_cache_vector_09_b200")
DEV = torch.device("cuda", 0)


def rows(n, d, seed):
    return torch.randn((n, d), generator=torch.Generator().manual_seed(seed)).to(DEV)


def cache(codec, n, seed):
    c = tq.Compressed.empty(codec, n)
    tq.tq_quantize(codec, rows(n, codec.d, seed), c)
    return c


# Each maker returns (C entry, arguments but the stream, output tensors, what
# the arguments refer to).
def quantize(d, bits, m, **kw):
    codec, x = tq.Codec(d, bits, m, 0, **kw), rows(40, d, 1)
    out = tq.Compressed.empty(codec, 40)
    st = out.struct()
    return (tq.c_api().tq_quantize, (codec.handle, x.data_ptr(), tq.TQ_F32, 40, d, ctypes.byref(st)),
            [t for t in (out.codes, out.signs, out.norms, out.rnorms) if t is not None], (codec, x, st))


def scores(d, bits, m, Hq, T, **kw):
    codec = tq.Codec(d, bits, m, 0, **kw)
    q, K, out = rows(Hq, d, 2), cache(codec, T, 3), torch.empty((1, Hq, T), device=DEV)
    ws, st = tq.workspace(tq.tq_scores_workspace_size(codec, 1, Hq, 1), DEV), K.struct()
    return (tq.c_api().tq_scores, (codec.handle, q.data_ptr(), tq.TQ_F32, 1, Hq, 1, T, ctypes.byref(st), out.data_ptr(),
                                   ws.data_ptr(), ws.numel() * ws.element_size()), [out], (codec, q, K, ws, st))


def attend(d, bits, m, Hq, T, vm=0, **kw):
    kc, vc = tq.Codec(d, bits, m, 0, **kw), tq.Codec(d, bits, vm, 1, **kw)
    q, K, V, out = rows(Hq, d, 2), cache(kc, T, 3), cache(vc, T, 4), torch.empty((1, Hq, d), device=DEV)
    ws = tq.workspace(tq.tq_attend_workspace_size(kc, vc, 1, Hq, 1, T), DEV)
    k, v = K.struct(), V.struct()
    return (tq.c_api().tq_attend, (kc.handle, vc.handle, q.data_ptr(), tq.TQ_F32, 1, Hq, 1, T, 0.0, ctypes.byref(k),
                                   ctypes.byref(v), ws.data_ptr(), ws.numel() * ws.element_size(), out.data_ptr()), [out],
            (kc, vc, q, K, V, ws, k, v))


def search(nq, k):
    codec = tq.Codec(512, (3,), 256, 0)
    q, X = rows(nq, 512, 2), cache(codec, 300, 3)
    idx, val = torch.empty((nq, k), dtype=torch.int32, device=DEV), torch.empty((nq, k), device=DEV)
    ws, st = tq.workspace(tq.tq_search_workspace_size(codec, nq, k), DEV), X.struct()
    return (tq.c_api().tq_search_topk, (codec.handle, q.data_ptr(), tq.TQ_F32, nq, ctypes.byref(st), 300, k, idx.data_ptr(),
                                        val.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size()), [idx, val],
            (codec, q, X, ws, st))


@pytest.mark.parametrize("pair", [
    (lambda: quantize(128, (3,), 64), lambda: quantize(128, (3,), 128)),
    (lambda: quantize(256, (3,), 0, rotation=1), lambda: quantize(256, (1,), 0, vq_bits=8)),
    (lambda: scores(128, (3,), 128, 1, 500), lambda: scores(128, (3,), 128, 8, 500)),
    (lambda: scores(256, (3,), 32, 4, 100), lambda: scores(256, (3,), 1024, 4, 100)),
    (lambda: attend(128, (3,), 64, 4, 64), lambda: attend(128, (3,), 128, 4, 30000)),
    (lambda: attend(256, (3,), 32, 4, 100), lambda: attend(256, (3,), 1024, 4, 3000)),
    (lambda: search(1, 1), lambda: search(16, 32)),
], ids=["quantize", "quantize_any", "scores", "scores_any", "attend", "attend_any", "search"])
def test_two_host_threads(pair):
    calls, want = [p() for p in pair], []
    for fn, args, outs, _ in calls:
        assert fn(*args, None) == 0, tq.tq_last_error_string()
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    failed, go = [], threading.Barrier(2)

    def work(i):
        fn, args, outs, _ = calls[i]
        torch.cuda.set_device(0)
        st = torch.cuda.Stream()
        torch.cuda.synchronize()
        go.wait()
        bad = sum(fn(*args, st.cuda_stream) != 0 for _ in range(8000))
        st.synchronize()
        if bad or not all(torch.equal(a, b) for a, b in zip(outs, want[i])):
            failed.append((i, bad, tq.tq_last_error_string()))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not failed, failed
