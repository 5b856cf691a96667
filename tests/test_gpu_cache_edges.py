"""Shared-prefix attention and bounded cache at the edges of their contract:
calls from several host threads, weights without a history or with infinite
statistics and logits, and the weights' way through eviction."""
import ctypes
import math
import threading

import numpy as np
import pytest
import torch

from test_gpu_cache import DEV, Case, evict_reference

pytestmark = pytest.mark.gpu

tq = pytest.importorskip("kv_cache_vector_09_b200")
U = 2.0 ** -24


# ------------------------------------------------------- several host threads
def test_calls_from_two_host_threads():
    # codecs of one kernel that need different amounts of shared memory: a call
    # must not depend on what another thread launches between its own steps
    V, VG = dict(bits=(4,), seed=4), dict(bits=(4,), seed=9)
    pairs = [[Case(128, dict(bits=(3,), m=m), V, 2, 8, 2, 200, 20, [20, 3], seed=m) for m in ms] for ms in ((128, 0), (96, 32))]
    pairs += [[Case(256, dict(bits=(3,), m=m), VG, 2, 4, 2, 70, 20, [20, 3], seed=m) for m in (1024, 32)]]
    for cases in pairs:
        want = [c.run()[0] for c in cases]
        torch.cuda.synchronize()
        failed, go = [], threading.Barrier(2)

        def work(c, w):
            # the C entry itself, its arguments made beforehand: calls overlap outside the interpreter's lock
            torch.cuda.set_device(0)
            st, ws, out, g = torch.cuda.Stream(), c.ws(), torch.empty_like(w), c.g
            rec = [g[k].struct() for k in ("Kp", "Vp", "K", "V")]
            Kp, Vp, K, V = (ctypes.byref(r) for r in rec)
            args = (c.kc.handle, c.vc.handle, g["q"].data_ptr(), tq.TQ_BF16, c.B, c.Hq, c.Hkv, c.scale, c.Tp, Kp, Vp, c.T,
                    g["lens"].data_ptr(), K, V, ws.data_ptr(), ws.numel() * ws.element_size(), out.data_ptr(), tq.TQ_F32,
                    None, st.cuda_stream)
            call = tq.c_api().tq_attend_prefix
            torch.cuda.synchronize()
            go.wait()
            bad = sum(call(*args) != 0 for _ in range(20000))
            st.synchronize()
            if bad or not torch.equal(out, w):
                failed.append((c.okc.m, bad, tq.tq_last_error_string()))

        threads = [threading.Thread(target=work, args=x) for x in zip(cases, want)]
        [t.start() for t in threads]
        [t.join() for t in threads]
        assert not failed, failed


# --------------------------------------------------------------------- weights
#         B, Hq, Hkv, T, lens, statistics given
WEIGHTS = [(2, 4, 2, 7, [7, 3], False), (2, 8, 2, 3000, None, False), (1, 8, 2, 4001, [4000], False),
           (1, 32, 1, 60001, [60000], False), (1, 32, 1, 65536, None, False),
           (2, 8, 2, 3000, [3000, 1], True), (2, 5, 5, 4097, None, True)]


def weights(B, Hq, Hkv, T, lens, with_lse, mass, decay, logits=None, lse=None, scale=0.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    kc = tq.Codec(128, (3,), 0, 0)
    if logits is None:
        logits = torch.randn((B, Hq, T), generator=g, device=DEV) * 20.0
    if with_lse and lse is None:
        lse = torch.logsumexp(logits.double() / math.sqrt(128), -1).float()
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    tq.tq_mass_update(kc, logits, B, Hq, Hkv, T, mass, lens=n, lse=lse, scale=scale, decay=decay)
    return mass


@pytest.mark.parametrize("B,Hq,Hkv,T,lens,with_lse", WEIGHTS)
def test_a_decay_of_zero_forgets_the_old_weight(B, Hq, Hkv, T, lens, with_lse):
    # whatever the buffer holds, NaN and infinities included
    want = weights(B, Hq, Hkv, T, lens, with_lse, torch.zeros((B, Hkv, T), device=DEV), 1.0)
    for old in (math.nan, math.inf, 3.0):
        got = weights(B, Hq, Hkv, T, lens, with_lse, torch.full((B, Hkv, T), old, device=DEV), 0.0)
        for b in range(B):
            n = T if lens is None else lens[b]
            assert torch.equal(got[b, :, :n], want[b, :, :n]) and torch.isfinite(got[b, :, :n]).all()
            assert torch.equal(got[b, :, n:].isnan(), torch.full_like(got[b, :, n:], old).isnan())  # left alone


@pytest.mark.parametrize("T", [8, 4097])
def test_a_statistic_of_infinity_adds_nothing(T):
    # e^(l - inf) = 0, as for a row without keys; 3e38 log2(e) is beyond fp32
    lse = torch.tensor([[math.inf, -math.inf, 9.0, 3e38]], device=DEV)
    logits = torch.randn((1, 4, T), generator=torch.Generator().manual_seed(T)).to(DEV) * 20.0
    got = weights(1, 4, 2, T, None, True, torch.ones((1, 2, T), device=DEV), 0.5, logits, lse)
    assert torch.all(got[0, 0] == 0.5)
    p = torch.exp(logits[0, 2].double() / math.sqrt(128) - 9.0)
    assert torch.all((got[0, 1].double() - 0.5 - p).abs() <= U * (1 + 40 * p))  # |exponent| <= 20: 20 u, exp2 4 u


@pytest.mark.parametrize("T", [8, 4097])
def test_infinite_logits_follow_the_definition(T):
    # e^(-inf) = 0 at every scale, and e^(inf) = inf
    lse = torch.zeros((1, 2), device=DEV)
    for scale in (1e-38, 0.5, 64.0):
        logits = torch.zeros((1, 2, T), device=DEV)
        logits[0, :, 0::3] = -math.inf
        logits[0, 0, 1] = math.inf
        got = weights(1, 2, 2, T, None, True, torch.ones((1, 2, T), device=DEV), 1.0, logits, lse, scale)
        want = torch.full((2, T), 2.0, device=DEV)
        want[:, 0::3] = 1.0
        want[0, 1] = math.inf
        assert torch.equal(got[0], want), scale


def test_weights_follow_their_keys_through_eviction():
    """Steps of a bounded cache: the accumulated weight of every key against the
    64-bit sum over that key's own logits and statistics, where it started and
    where eviction moved it; the move itself is exact."""
    d, B, Hq, Hkv, Tp, T, keep = 128, 3, 8, 2, 60, 24, 10
    G, R, sc = Hq // Hkv, B * Hkv, float(np.float32(1.0 / math.sqrt(d)))
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    f = lambda *s: 3.0 * torch.randn(s, generator=g, device=DEV)  # noqa: E731
    kc, vc = tq.Codec(d, (3,), 128, 0), tq.Codec(d, (4,), 0, 1)
    pre = [tq.Compressed.empty(c, Hkv * Tp) for c in (kc, vc)]
    for c, p in zip((kc, vc), pre):
        tq.tq_quantize(c, f(Hkv * Tp, d), p)
    caches = [[tq.Compressed.empty(c, R * T) for c in (kc, vc)] for _ in range(2)]
    new = [tq.Compressed.empty(c, R) for c in (kc, vc)]
    lens = torch.zeros((B,), dtype=torch.int32, device=DEV)
    lens2 = torch.empty_like(lens)
    mass, mass2 = torch.zeros((B, Hkv, T), device=DEV), torch.empty((B, Hkv, keep), device=DEV)
    idx = torch.empty((B, Hkv, keep), dtype=torch.int32, device=DEV)
    model, size = np.zeros((B, Hkv, T)), np.zeros((B, Hkv, T))   # the sums, and the sums of error bounds
    ws = tq.workspace(tq.tq_attend_prefix_workspace_size(kc, vc, B, Hq, Hkv, Tp, T), DEV)
    ws2 = tq.workspace(tq.tq_scores_workspace_size(kc, B, Hq, Hkv), DEV)
    out, lse, logits = (torch.empty(s, device=DEV) for s in ((B, Hq, d), (B, Hq), (B, Hq, T)))
    cuts = 0
    for step in range(60):
        # one sequence grows each step, the others every second or third
        grow = torch.tensor([True, step % 2 == 0, step % 3 == 0], device=DEV)
        at = torch.where(grow, lens, torch.full_like(lens, -1)).repeat_interleave(Hkv).contiguous()
        for c, cache, n in zip((kc, vc), caches[0], new):
            tq.tq_quantize(c, f(R, d), n)
            tq.tq_copy_rows(c, n, 1, cache, T, R, 1, dst_idx=at)
        lens += grow.to(torch.int32)
        q = f(B, Hq, d)
        tq.tq_attend_prefix(kc, vc, q, B, Hq, Hkv, Tp, *pre, T, *caches[0], out, ws, lens=lens, scale=sc, lse=lse)
        tq.tq_scores(kc, q, B, Hq, Hkv, T, caches[0][0], logits, ws2)
        tq.tq_mass_update(kc, logits, B, Hq, Hkv, T, mass, lens=lens, lse=lse, scale=sc)
        n = lens.cpu().numpy()
        l, s = logits.double().cpu().numpy() * sc, lse.double().cpu().numpy()
        for b in range(B):
            p = np.exp(l[b, :, :n[b]] - s[b][:, None])
            x = np.abs(l[b, :, :n[b]] - s[b][:, None])
            # of each weight p = e^-x: exp2 4 u, its argument 3 roundings of x; one rounding of the sum for each head
            model[b, :, :n[b]] += p.reshape(Hkv, G, -1).sum(1)
            size[b, :, :n[b]] += U * ((8 + 4 * x) * p).reshape(Hkv, G, -1).sum(1) + (G + 2) * U * model[b, :, :n[b]]
            got = mass[b, :, :n[b]].double().cpu().numpy()
            assert np.all(np.abs(got - model[b, :, :n[b]]) <= size[b, :, :n[b]]), step
        assert not torch.any(mass[torch.arange(T, device=DEV)[None, None] >= lens[:, None, None].expand(B, Hkv, 1)])
        if n.max() < T:
            continue
        cuts += 1
        m = mass.cpu().numpy()
        tq.tq_evict_select(kc, mass, B, Hkv, T, keep, idx, lens=lens, sink=1, recent=3, mass_out=mass2, lens_out=lens2)
        for c, a, z in zip((kc, vc), *caches):
            tq.tq_copy_rows(c, a, T, z, T, R, keep, src_idx=idx)
        caches.reverse()
        want, kept = evict_reference(m, n, keep, 1, 3)
        assert np.array_equal(idx.cpu().numpy(), want) and np.array_equal(mass2.cpu().numpy(), kept)
        mass.zero_()
        mass[..., :keep] = mass2
        lens.copy_(lens2)
        pick = np.maximum(want, 0)
        for a in (model, size):
            moved = np.where(want >= 0, np.take_along_axis(a, pick, 2), 0.0)
            a[:] = 0.0
            a[..., :keep] = moved
    assert cuts >= 2
    assert tq.tq_codec_device_error(kc) == 0 and tq.tq_codec_device_error(vc) == 0


def test_a_captured_step_replays_like_the_eager_one():
    """Append, attention, scores, weights, choice and copies of one step in a
    graph, replayed with other queries, lengths and contents."""
    d, B, Hq, Hkv, Tp, T, keep = 128, 3, 8, 2, 100, 2100, 600
    R = B * Hkv
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    f = lambda *s: 3.0 * torch.randn(s, generator=g, device=DEV)  # noqa: E731
    kc, vc = tq.Codec(d, (3,), 128, 0), tq.Codec(d, (4,), 0, 1)
    new = lambda n: [tq.tq_quantize(c, f(n, d), tq.Compressed.empty(c, n)) for c in (kc, vc)]  # noqa: E731
    pre, own, kept, row = new(Hkv * Tp), new(R * T), new(R * keep), new(R)
    x, q = [f(R, d) for _ in range(2)], f(B, Hq, d)
    lens, at = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(R, dtype=torch.int32, device=DEV)
    mass = torch.zeros((B, Hkv, T), device=DEV)
    out, lse, logits = (torch.zeros(s, device=DEV) for s in ((B, Hq, d), (B, Hq), (B, Hq, T)))
    idx = torch.zeros((B, Hkv, keep), dtype=torch.int32, device=DEV)
    mass2, lens2 = torch.zeros((B, Hkv, keep), device=DEV), torch.zeros_like(lens)
    ws = tq.workspace(tq.tq_attend_prefix_workspace_size(kc, vc, B, Hq, Hkv, Tp, T), DEV)
    ws2 = tq.workspace(tq.tq_scores_workspace_size(kc, B, Hq, Hkv), DEV)
    state = [t for c in own + kept for t in (c.codes, c.signs, c.norms, c.rnorms) if t is not None]
    state += [mass, out, lse, idx, mass2, lens2]

    def step():
        for c, v, r, cache in zip((kc, vc), x, row, own):
            tq.tq_quantize(c, v, r)
            tq.tq_copy_rows(c, r, 1, cache, T, R, 1, dst_idx=at)
        tq.tq_attend_prefix(kc, vc, q, B, Hq, Hkv, Tp, *pre, T, *own, out, ws, lens=lens, lse=lse)
        tq.tq_scores(kc, q, B, Hq, Hkv, T, own[0], logits, ws2)
        tq.tq_mass_update(kc, logits, B, Hq, Hkv, T, mass, lens=lens, lse=lse)
        tq.tq_mass_update(kc, logits, B, Hq, Hkv, T, mass, lens=lens, decay=0.5)
        tq.tq_evict_select(kc, mass, B, Hkv, T, keep, idx, lens=lens, sink=2, recent=9, mass_out=mass2, lens_out=lens2)
        for c, a, z in zip((kc, vc), own, kept):
            tq.tq_copy_rows(c, a, T, z, keep, R, keep, src_idx=idx)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in ([5, 1, 2100], [2100, 601, 600], [1, 1, 1]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        at.copy_((lens - 1).repeat_interleave(Hkv))
        q.copy_(f(B, Hq, d))
        for v in x:
            v.copy_(f(R, d))
        before = [t.clone() for t in state]
        step()
        want = [t.clone() for t in state]
        for t, b in zip(state, before):
            t.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(state, want)), n
    assert tq.tq_codec_device_error(kc) == 0 and tq.tq_codec_device_error(vc) == 0
