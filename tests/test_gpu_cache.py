"""Shared-prefix attention, accumulated attention weight, eviction and record
copies against 64-bit references on the same compressed records.

Records are drawn at random (any word is a code), so that norms, lengths and
garbage behind the lengths can be chosen freely; the oracle decodes them.

Tolerances, u = 2^-24 (derived, not fitted):

* a logit is a sum of d + m products in fp32 or of fp16 products of operands
  split in two parts (2^-22 relative), so |dl| <= E L with
  L = scale nu (sum |q'_i c_i| / sqrt(d) + gamma coef sum |w_j|) and
  E = (d + m + 32) u;
* softmax weights move by at most e^(2 max |dl|) - 1, the weighted sums of n
  values by n u more, both relative to A = sum p_t |v_t| (per coordinate in the
  rotated space; the inverse rotation keeps the 2-norm, so rows are compared
  in the 2-norm);
* outputs of fp16 or bf16 add their half step.  bf16 outputs may come from
  operands rounded once to fp16: E then is 2^-10 (q', c and w, half a step 2^-11
  each, on either factor), and p and v move by 2^-11 each.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu

tq = pytest.importorskip("kv_cache_vector_09_b200")
DEV = torch.device("cuda", 0)
U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


# ------------------------------------------------------------------- helpers
def make_codecs(d, spec):
    """(library codec, oracle codec) of a spec dict."""
    kw = dict(spec)
    bits, m, seed = kw.pop("bits"), kw.pop("m", 0), kw.pop("seed", 3)
    lib = tq.Codec(d, bits, m, seed, residual=1 if kw.get("residual") == "sign" else 0,
                   rotation=1 if kw.get("rotation") == "haar" else 0, vq_bits=kw.get("vq_bits", 0))
    return lib, O.make_codec(d, bits, m, seed, **kw)


def records(rng, n, codec, sigma=0.4, scale=3.0):
    """Random records of `codec` (oracle) with lognormal norms."""
    words = lambda w: rng.integers(0, 2 ** 32, (n, w), dtype=np.uint64).astype(np.uint32)  # noqa: E731
    rn = rng.uniform(0.1, 0.5, n).astype(np.float32)
    if codec.residual == "sign":
        rn[:] = np.float32(codec.mu * math.sqrt(2 * codec.d / math.pi))
    return O.Compressed(words(codec.words), words(codec.m // 32), (scale * np.exp(sigma * rng.standard_normal(n))
                                                                   ).astype(np.float32), rn if codec.m else rn[:0])


def up(rec, codec):
    g = lambda a: torch.from_numpy(np.ascontiguousarray(a).view(np.int32)).to(DEV)  # noqa: E731
    f = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    return tq.Compressed(g(rec.codes), g(rec.signs) if codec.m else None, f(rec.norms),
                         f(rec.rnorms) if codec.m else None)


def part(rec, a, b):
    return O.Compressed(rec.codes[a:b], rec.signs[a:b], rec.norms[a:b], rec.rnorms[a:b])


def spoil(rec, rows, rng):
    """Garbage in records that no call may read."""
    rec.norms[rows] = np.nan
    if rec.rnorms.size:
        rec.rnorms[rows] = np.inf
    return rec


class Case:
    """One attention problem, its inputs on both sides and its 64-bit result."""

    def __init__(self, d, ks, vs, B, Hq, Hkv, Tp, T, lens, qdt=torch.bfloat16, scale=0.0, seed=0, qscale=1.0):
        rng = np.random.default_rng(seed)
        self.d, self.B, self.Hq, self.Hkv, self.Tp, self.T, self.scale = d, B, Hq, Hkv, Tp, T, scale
        self.kc, self.okc = make_codecs(d, ks)
        self.vc, self.ovc = make_codecs(d, vs)
        self.q = torch.from_numpy(qscale * rng.standard_normal((B, Hq, d))).to(qdt)
        self.lens = np.asarray(lens if lens is not None else [T] * B)
        self.Kp, self.Vp = records(rng, Hkv * Tp, self.okc), records(rng, Hkv * Tp, self.ovc)
        self.K, self.V = records(rng, B * Hkv * T, self.okc), records(rng, B * Hkv * T, self.ovc)
        dead = (np.arange(T)[None, None] >= self.lens[:, None, None]).repeat(Hkv, 1).reshape(-1)
        spoil(self.K, dead, rng)
        spoil(self.V, dead, rng)
        self.g = dict(q=self.q.to(DEV), Kp=up(self.Kp, self.okc), Vp=up(self.Vp, self.ovc), K=up(self.K, self.okc),
                      V=up(self.V, self.ovc), lens=torch.from_numpy(self.lens.astype(np.int32)).to(DEV))
        if lens is None:
            self.g["lens"] = None

    def ws(self):
        return tq.workspace(tq.tq_attend_prefix_workspace_size(self.kc, self.vc, self.B, self.Hq, self.Hkv, self.Tp,
                                                               self.T), DEV)

    def run(self, out_dtype=torch.float32, lse=True, ws=None, out=None, stream=None):
        out = torch.full((self.B, self.Hq, self.d), 7.0, device=DEV, dtype=out_dtype) if out is None else out
        l = torch.full((self.B, self.Hq), 7.0, device=DEV) if lse else None
        g = self.g
        tq.tq_attend_prefix(self.kc, self.vc, g["q"], self.B, self.Hq, self.Hkv, self.Tp, g["Kp"], g["Vp"], self.T,
                            g["K"], g["V"], out, self.ws() if ws is None else ws, lens=g["lens"], scale=self.scale,
                            lse=l, stream=stream)
        return out, l

    def _decoded(self, lo, hi, rec, key):
        """Rotated rows lo..hi in double; for keys also their |centroids| and
        sketch weights, both times the norm (for the logits' error bound)."""
        r, c = part(rec, lo, hi), self.okc if key else self.ovc
        x = O.dequantize(r, c, rotated=True, qjl=True)
        if not key:
            return x
        nu = r.norms.astype(np.float64)
        mag = np.abs(c.coord_cen(O.unpack_codes(r.codes, c))) / math.sqrt(c.d) * nu[:, None]
        gam = r.rnorms.astype(np.float64) * math.sqrt(math.pi / 2) / c.m * nu if c.m else 0.0 * nu
        return x, mag, gam

    def reference(self, lens=None):
        """out, lse, and per row L (bound of the terms' sum over its logits), A
        (2-norm of sum p |v|) and the number of keys."""
        d, G = self.d, self.Hq // self.Hkv
        lens = self.lens if lens is None else lens
        sc = self.scale or 1.0 / math.sqrt(d)
        q = self.q.double().numpy() @ self.okc.Pi.T
        out, lse = np.zeros((self.B, self.Hq, d)), np.full((self.B, self.Hq), -np.inf)
        L, A, n = (np.zeros((self.B, self.Hq)) for _ in range(3))
        for h in range(self.Hkv):
            pre = self._decoded(h * self.Tp, (h + 1) * self.Tp, self.Kp, True)
            prev = self._decoded(h * self.Tp, (h + 1) * self.Tp, self.Vp, False)
            for b in range(self.B):
                r0 = (b * self.Hkv + h) * self.T
                k, mag, gam = (np.concatenate(t) for t in zip(pre, self._decoded(r0, r0 + lens[b], self.K, True)))
                v = np.concatenate([prev, self._decoded(r0, r0 + lens[b], self.V, False)])
                if not len(k):
                    continue
                for hq in range(h * G, (h + 1) * G):
                    l = k @ q[b, hq] * sc
                    w = np.abs(self.okc.S.astype(np.float64) @ q[b, hq]).sum() if self.okc.m else 0.0
                    L[b, hq] = sc * (mag @ np.abs(q[b, hq]) + gam * w).max()
                    p = np.exp(l - l.max())
                    lse[b, hq] = l.max() + math.log(p.sum())
                    p /= p.sum()
                    out[b, hq], A[b, hq], n[b, hq] = (p @ v) @ self.ovc.Pi, np.linalg.norm(p @ np.abs(v)), len(k)
        return out, lse, L, A, n

    def check(self, out, lse, ref):
        o, s, L, A, n = ref
        dt = out.dtype
        single = dt == torch.bfloat16 and lse is None
        E = (2.0 ** -10 if single else 0.0) + (self.d + self.okc.m + 32) * U
        err = np.linalg.norm(out.double().cpu().numpy() - o, axis=-1)
        tol = (np.expm1(2 * E * L) + (n + 32) * U + (2.0 ** -10 if single else 0.0)) * A \
            + HALF_STEP[dt] * np.linalg.norm(o, axis=-1) + 1e-30
        assert np.all(err <= tol), f"out: {(err / tol).max():.3g} of the tolerance at {np.argmax(err / tol)}"
        assert not np.any(out.cpu().numpy()[n == 0] if dt != torch.bfloat16 else out.float().cpu().numpy()[n == 0])
        if lse is not None:
            g = lse.double().cpu().numpy()
            assert np.array_equal(np.isneginf(g), n == 0)
            live = n > 0
            t = E * L[live] + 8 * U * (1 + np.abs(s[live])) + (n[live] + 32) * U
            off = np.abs(g[live] - s[live])
            assert np.all(off <= t), f"lse: {(off / t).max():.3g} of the tolerance"


K3 = dict(bits=(3,), m=128)
V4 = dict(bits=(4,), seed=4)
BF, HF, FL = torch.bfloat16, torch.float16, torch.float32


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("d,ks,vs,B,Hq,Hkv,Tp,T,lens,qdt,odt", [
    (128, K3, V4, 1, 4, 1, 1, 0, None, BF, FL),                      # one prefix key, nothing else
    (128, K3, V4, 2, 2, 2, 0, 1, [0, 1], BF, FL),                    # no prefix; an empty row and a single key
    (128, K3, V4, 3, 8, 2, 63, 65, [0, 64, 65], BF, FL),             # around a tile
    (128, K3, V4, 5, 32, 8, 129, 127, [127, 0, 1, 126, 63], BF, BF),
    (128, K3, V4, 40, 8, 2, 700, 33, list(range(34)) + [33] * 6, BF, HF),   # 160 rows a head: two row blocks
    (128, K3, V4, 4, 32, 1, 2500, 0, None, BF, FL),                  # 32 heads a group, 128 rows exactly
    (128, K3, V4, 17, 7, 1, 1001, 300, [0, 300, 299] + [100 + i for i in range(14)], FL, FL),
    (128, dict(bits=(2, 3), m=64), V4, 3, 8, 2, 1111, 257, [0, 257, 100], BF, FL),
    (128, dict(bits=(1,), m=32), dict(bits=(1,), seed=9), 3, 5, 1, 333, 99, [99, 7, 0], HF, FL),
    (128, dict(bits=(2,), m=64), dict(bits=(2, 3), seed=9), 2, 2, 1, 4100, 10, [10, 3], HF, BF),
    (128, dict(bits=(4,), m=256), dict(bits=(3,), seed=9), 9, 4, 2, 515, 130, None, BF, FL),
    (128, dict(bits=(4, 1), m=0), dict(bits=(1, 4), seed=9), 2, 4, 2, 200, 50, [50, 20], BF, FL),
    (64, dict(bits=(4,), m=0), dict(bits=(3,), seed=9), 16, 20, 20, 130, 40, [0] + [40] * 15, FL, FL),
    (64, dict(bits=(2,), m=64), dict(bits=(2,), seed=9), 3, 6, 2, 777, 129, [5, 129, 0], BF, BF),
    (64, dict(bits=(3,), m=128), dict(bits=(4,), seed=9), 33, 8, 2, 65, 64, [2 * i for i in range(33)], HF, HF),
    (64, dict(bits=(1, 2), m=32), dict(bits=(2, 3), seed=9), 2, 4, 4, 257, 31, [31, 30], BF, FL),
    (128, dict(bits=(3,), m=96), V4, 2, 6, 3, 200, 70, [70, 1], HF, FL),                # three sign words
    (64, dict(bits=(2,), m=32), dict(bits=(3,), seed=9), 300, 64, 2, 70, 5, [i % 6 for i in range(300)], BF, BF),  # more groups than SMs
    (256, dict(bits=(3,), m=64), dict(bits=(4,), seed=9), 2, 4, 2, 300, 70, [70, 0], BF, FL),
    (128, dict(bits=(2,), m=512), dict(bits=(2,), m=64, seed=9), 2, 4, 1, 200, 66, [0, 66], BF, FL),
    (128, K3, dict(bits=(3,), m=128, seed=9), 2, 4, 1, 200, 66, [0, 66], BF, BF),     # QJL-corrected values
    (128, dict(bits=(3,), m=128, residual="sign"), V4, 3, 4, 1, 300, 66, [0, 66, 9], BF, FL),
    (128, dict(bits=(3,), m=64, rotation="haar"), dict(bits=(3,), rotation="haar", seed=9), 2, 4, 2, 200, 20, [20, 1], BF, FL),
    (64, dict(bits=(1,), m=64, vq_bits=5), dict(bits=(1,), vq_bits=6, seed=9), 2, 4, 2, 200, 20, [20, 1], BF, FL),
])
@pytest.mark.parametrize("lse", [True, False])
def test_attend_prefix(d, ks, vs, B, Hq, Hkv, Tp, T, lens, qdt, odt, lse):
    c = Case(d, ks, vs, B, Hq, Hkv, Tp, T, lens, qdt, seed=B + Tp)
    out, l = c.run(odt, lse)
    torch.cuda.synchronize()
    assert tq.tq_codec_device_error(c.kc) == 0
    c.check(out, l, c.reference())
    again, l2 = c.run(odt, lse)
    assert torch.equal(out, again) and (not lse or torch.equal(l, l2))


def test_attend_prefix_explicit_scale_and_peaked_softmax():
    # logits of several hundred: one key takes nearly all weight
    c = Case(128, K3, V4, 3, 8, 2, 900, 130, [130, 0, 55], scale=0.5, qscale=4.0, seed=5)
    out, l = c.run()
    c.check(out, l, c.reference())


def test_attend_prefix_value_norms_of_any_size():
    # value norms over 60 binary orders of magnitude, some zero
    c = Case(128, K3, V4, 3, 8, 2, 900, 130, [130, 0, 55], seed=6)
    rng = np.random.default_rng(1)
    for r in (c.Vp, c.V):
        r.norms *= (2.0 ** rng.integers(-40, 20, r.norms.shape)).astype(np.float32)
        r.norms[rng.random(r.norms.shape) < 0.1] = 0.0
    c.g["Vp"], c.g["V"] = up(c.Vp, c.ovc), up(c.V, c.ovc)
    for odt in (FL, BF):
        out, l = c.run(odt, odt == FL)
        c.check(out, l, c.reference())


def test_attend_prefix_zero_values_and_keys():
    # all keys and values zero: uniform weights, zero output, lse = ln n
    c = Case(64, dict(bits=(2,), m=64), dict(bits=(2,), seed=9), 2, 4, 2, 70, 30, [0, 30], seed=7)
    for r in (c.Kp, c.Vp, c.K, c.V):
        r.norms[:] = 0.0
    c.g.update(Kp=up(c.Kp, c.okc), Vp=up(c.Vp, c.ovc), K=up(c.K, c.okc), V=up(c.V, c.ovc))
    out, l = c.run()
    assert not torch.any(out)
    want = torch.tensor([[math.log(70)] * 4, [math.log(100)] * 4], device=DEV)
    assert torch.all((l - want).abs() <= 8 * U * 6)


def test_attend_prefix_equals_tq_attend_without_a_prefix():
    # the same keys as one full-length cache through the earlier entry point
    c = Case(128, K3, V4, 3, 8, 2, 0, 500, None, seed=8)
    out, _ = c.run()
    o2 = torch.empty((3, 8, 128), device=DEV)
    tq.tq_attend(c.kc, c.vc, c.g["q"], 3, 8, 2, 500, c.g["K"], c.g["V"], o2,
                 tq.workspace(tq.tq_attend_workspace_size(c.kc, c.vc, 3, 8, 2, 500), DEV))
    o, s, L, A, n = c.reference()
    c.check(out, None, (o, s, L, A, n))
    c.check(o2, None, (o, s, L, A, n))


def test_attend_prefix_lengths_out_of_range_are_clamped_and_recorded():
    c = Case(128, K3, V4, 3, 4, 2, 100, 40, [40, 0, 17], seed=9)
    c.g["lens"] = torch.tensor([41, -1, 17], dtype=torch.int32, device=DEV)
    out, l = c.run()
    torch.cuda.synchronize()
    assert tq.tq_codec_device_error(c.kc) == 4
    assert tq.tq_codec_device_error(c.kc) == 0
    c.check(out, l, c.reference())


def test_attend_prefix_on_another_stream_and_in_a_graph():
    c = Case(128, K3, V4, 4, 8, 2, 600, 90, [90, 0, 45, 89], seed=10)
    want, wl = c.run()
    torch.cuda.synchronize()
    ws, out = c.ws(), torch.empty_like(want)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got, gl = c.run(ws=ws, out=out)
    st.synchronize()
    assert torch.equal(want, got) and torch.equal(wl, gl)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got, gl = c.run(ws=ws, out=out)
    for lens in ([90, 0, 45, 89], [1, 0, 3, 4], [0, 0, 0, 0]):   # records behind the first lengths hold garbage
        # the captured call reads the lengths at replay; the workspace may hold anything
        c.g["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        c2 = c.reference(np.array(lens)) if lens != [90, 0, 45, 89] else None
        if c2 is None:
            assert torch.equal(want, got) and torch.equal(wl, gl)
        else:
            c.check(got, gl, c2)


def test_attend_prefix_calls_that_overlap():
    # two calls in flight on two streams, a workspace each, over the same caches
    c = Case(128, K3, V4, 6, 8, 2, 3000, 90, [90, 0, 45, 89, 1, 64], seed=13)
    (want, wl), (want16, _) = c.run(), c.run(BF, False)
    torch.cuda.synchronize()
    streams, ws = [torch.cuda.Stream() for _ in range(2)], [c.ws() for _ in range(2)]
    outs = [torch.empty_like(want), torch.empty_like(want16)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got.append(c.run(outs[k].dtype, k == 0, ws=ws[k], out=outs[k]))
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want16) and torch.equal(got[-2][1], wl)


# ---------------------------------------------------------------------- mass
def mass_reference(logits, lens, lse, scale, decay, mass, Hkv):
    B, Hq, T = logits.shape
    out, add = mass.astype(np.float64), np.zeros(mass.shape)
    for b in range(B):
        n = lens[b]
        if not n:
            continue
        l = logits[b, :, :n].astype(np.float64) * scale
        with np.errstate(divide="ignore", invalid="ignore"):
            s = np.log(np.exp(l - l.max(1, keepdims=True)).sum(1)) + l.max(1) if lse is None else lse[b].astype(np.float64)
            p = np.where(np.isneginf(s)[:, None] | np.isnan(s)[:, None], 0.0, np.exp(l - s[:, None]))
        add[b, :, :n] = p.reshape(Hkv, -1, n).sum(1)
        out[b, :, :n] = out[b, :, :n] * decay + add[b, :, :n]
    return out, add


@pytest.mark.parametrize("B,Hq,Hkv,T,lens,with_lse,decay,scale", [
    (1, 1, 1, 1, None, False, 1.0, 0.0),
    (2, 8, 2, 5, [0, 5], False, 0.5, 0.0),
    (3, 32, 1, 1023, [1023, 1, 512], False, 1.0, 0.3),
    (2, 5, 5, 4097, [4097, 4096], True, 0.0, 0.0),
    (3, 32, 8, 2048, None, True, 0.96875, 0.0),
    (1, 8, 2, 40003, [39999], False, 1.0, 0.0),
    (1, 32, 1, 131072, None, False, 1.0, 0.0),
    (1, 32, 1, 60001, [60000], False, 1.0, 0.0),
    (1, 4, 1, 300001, [300000], True, 1.0, 0.0),
    (70, 4, 2, 333, [i * 333 // 69 for i in range(70)], False, 1.0, 0.0),
])
def test_mass_update(B, Hq, Hkv, T, lens, with_lse, decay, scale):
    rng = np.random.default_rng(T)
    kc = tq.Codec(128, (3,), 0, 0)
    sc = scale or 1.0 / math.sqrt(128)
    n = np.asarray(lens if lens is not None else [T] * B)
    logits = (rng.standard_normal((B, Hq, T)) * 2.0 / sc).astype(np.float32)
    logits[:, ::3, 0] += np.float32(20.0 / sc)
    if T > 4:
        logits[:, :, 3] = -np.inf                       # a masked key
    dead = np.arange(T)[None, :] >= n[:, None]
    mass = rng.random((B, Hkv, T)).astype(np.float32) * 5
    mass[dead[:, None].repeat(Hkv, 1)] = np.nan         # left as it was, NaN included
    lse = None
    if with_lse:
        lse = np.log(np.exp(logits.astype(np.float64) * sc).sum(-1)).astype(np.float32) + np.float32(0.5)
        lse[-1, 0] = -np.inf                            # a row without keys
    want, add = mass_reference(logits, n, lse, sc, decay, mass, Hkv)
    logits[dead[:, None].repeat(Hq, 1)] = np.nan
    up = lambda a, t=None: None if a is None else torch.from_numpy(np.asarray(a, t)).to(DEV)  # noqa: E731
    m = up(mass)
    tq.tq_mass_update(kc, up(logits), B, Hq, Hkv, T, m, lens=up(lens, np.int32), lse=up(lse), scale=scale, decay=decay)
    got = m.double().cpu().numpy()
    live = ~dead[:, None].repeat(Hkv, 1)
    assert np.array_equal(got[~live], mass.astype(np.float64)[~live], equal_nan=True)
    # exponent |x| <= 60 with 3 roundings of x 2^-x <= 0.54, exp2 within 4 u; the
    # row's own sum of exponentials carries n/512 + 40 roundings; G + 2 to add up
    G = Hq // Hkv
    tol = U * (8 * G + (T / 512 + 48) * add + (G + 2) * (np.abs(mass) * decay + add))
    assert np.all((np.abs(got - want) <= tol)[live]), (np.abs(got - want) / tol)[live].max()


def test_mass_update_rows_that_are_all_masked_add_nothing():
    kc = tq.Codec(128, (3,), 0, 0)
    for T in (7, 3000):
        logits = torch.full((2, 4, T), -math.inf, device=DEV)
        logits[1] = 0.0
        mass = torch.ones((2, 2, T), device=DEV)
        tq.tq_mass_update(kc, logits, 2, 4, 2, T, mass, decay=0.5)
        assert torch.all(mass[0] == 0.5)
        assert torch.all((mass[1] - (0.5 + 2.0 / T)).abs() <= 16 * U)


# ----------------------------------------------------------------- eviction
def evict_reference(mass, lens, keep, sink, recent):
    B, H, T = mass.shape
    idx, kept = np.full((B, H, keep), -1, np.int64), np.zeros((B, H, keep), mass.dtype)
    for b in range(B):
        for h in range(H):
            n = lens[b]
            if n <= keep:
                at = np.arange(n)
            else:
                mid = np.arange(sink, n - recent)
                v = mass[b, h, mid].astype(np.float64)
                order = np.lexsort((mid, -np.where(np.isnan(v), -np.inf, v), np.isnan(v)))
                at = np.concatenate([np.arange(sink), np.sort(mid[order[:keep - sink - recent]]), np.arange(n - recent, n)])
            idx[b, h, :len(at)], kept[b, h, :len(at)] = at, mass[b, h, at]
    return idx, kept


@pytest.mark.parametrize("B,H,T,keep,sink,recent,lens,kind", [
    (1, 1, 1, 1, 0, 0, None, "random"),
    (1, 1, 2, 1, 0, 0, None, "ties"),
    (2, 3, 100, 1, 0, 1, [100, 0], "random"),
    (2, 3, 100, 10, 10, 0, [100, 11], "random"),
    (2, 3, 100, 10, 3, 7, [100, 10], "random"),              # nothing to choose
    (2, 2, 1000, 1200, 4, 64, [1000, 5], "random"),          # more room than keys
    (3, 2, 1025, 513, 4, 64, [1025, 514, 513], "ties"),
    (2, 2, 4099, 1021, 1, 127, [4099, 1022], "special"),
    (1, 2, 20000, 19999, 0, 0, None, "equal"),
    (1, 2, 32768, 8192, 4, 1024, None, "ties"),
    (1, 1, 150001, 50000, 4, 100, [150000], "random"),
    (1, 1, 420001, 3000, 4, 100, [420000], "ties"),
    (70, 2, 300, 64, 2, 8, [i * 300 // 69 for i in range(70)], "ties"),
])
def test_evict_select(B, H, T, keep, sink, recent, lens, kind):
    rng = np.random.default_rng(T + keep)
    mass = np.exp(3 * rng.standard_normal((B, H, T))).astype(np.float32)
    if kind == "ties":
        mass = np.floor(rng.random((B, H, T)) * 4).astype(np.float32) / 4
    elif kind == "equal":
        mass[:] = 0.25
    elif kind == "special":
        mass[rng.random(mass.shape) < 0.2] = 0.0
        mass[rng.random(mass.shape) < 0.2] = -0.0
        for v in (np.nan, -np.nan, np.inf, -np.inf, -1.0, 1e-45, -1e-45):
            mass[rng.random(mass.shape) < 0.1] = v
    n = np.asarray(lens if lens is not None else [T] * B)
    want, kept = evict_reference(mass, n, keep, sink, recent)
    mass[(np.arange(T)[None, :] >= n[:, None])[:, None].repeat(H, 1)] = np.inf     # behind the length: not read
    kc = tq.Codec(128, (3,), 0, 0)
    up = lambda a, t=None: None if a is None else torch.from_numpy(np.asarray(a, t)).to(DEV)  # noqa: E731
    idx = torch.full((B, H, keep), 77, dtype=torch.int32, device=DEV)
    mo, lo = torch.full((B, H, keep), 7.0, device=DEV), torch.full((B,), 77, dtype=torch.int32, device=DEV)
    tq.tq_evict_select(kc, up(mass), B, H, T, keep, idx, lens=up(lens, np.int32), sink=sink, recent=recent, mass_out=mo,
                       lens_out=lo)
    assert np.array_equal(idx.cpu().numpy(), want)
    assert np.array_equal(mo.cpu().numpy(), kept, equal_nan=True)
    assert np.array_equal(lo.cpu().numpy(), np.minimum(n, keep))
    idx2 = torch.empty_like(idx)                                   # without the optional outputs
    tq.tq_evict_select(kc, up(mass), B, H, T, keep, idx2, lens=up(lens, np.int32), sink=sink, recent=recent)
    assert torch.equal(idx, idx2)
    assert tq.tq_codec_device_error(kc) == 0


@pytest.mark.parametrize("d,ks", [(128, K3), (128, V4), (64, dict(bits=(1,), m=32)), (64, dict(bits=(1,), m=0)),
                                  (128, dict(bits=(2, 3), m=64)), (1536, dict(bits=(3,), m=256)),
                                  (128, dict(bits=(1,), m=0, vq_bits=5))])
@pytest.mark.parametrize("R,src_T,dst_T,n", [(1, 1, 1, 1), (3, 50, 41, 33), (7, 9, 4, 20), (2, 1000, 777, 700)])
def test_copy_rows(d, ks, R, src_T, dst_T, n):
    c, oc = make_codecs(d, ks)
    rng = np.random.default_rng(n)
    src, dst = records(rng, R * src_T, oc), records(rng, R * dst_T, oc)
    si = rng.integers(-1, src_T, (R, n))
    di = np.full((R, n), -1)
    for r in range(R):                                             # distinct destinations, the rest skipped
        k = min(n, dst_T)
        di[r, rng.permutation(n)[:k]] = rng.permutation(dst_T)[:k]
    want = [a.copy() for a in (dst.codes, dst.signs, dst.norms, dst.rnorms)]
    for r in range(R):
        for i in range(n):
            if si[r, i] >= 0 and di[r, i] >= 0:
                for w, s in zip(want, (src.codes, src.signs, src.norms, src.rnorms)):
                    if s.size:
                        w[r * dst_T + di[r, i]] = s[r * src_T + si[r, i]]
    g = up(dst, oc)
    up_i = lambda a: torch.from_numpy(a.astype(np.int32)).to(DEV)  # noqa: E731
    tq.tq_copy_rows(c, up(src, oc), src_T, g, dst_T, R, n, src_idx=up_i(si), dst_idx=up_i(di))
    assert np.array_equal(g.codes.cpu().numpy().view(np.uint32), want[0])
    assert np.array_equal(g.norms.cpu().numpy(), want[2])
    if oc.m:
        assert np.array_equal(g.signs.cpu().numpy().view(np.uint32), want[1])
        assert np.array_equal(g.rnorms.cpu().numpy(), want[3])
    assert tq.tq_codec_device_error(c) == 0
    # without lists: record i to record i
    k, g = min(src_T, dst_T), up(dst, oc)
    tq.tq_copy_rows(c, up(src, oc), src_T, g, dst_T, R, k)
    got = g.codes.cpu().numpy().view(np.uint32).reshape(R, dst_T, -1)
    assert np.array_equal(got[:, :k], src.codes.reshape(R, src_T, -1)[:, :k])
    assert np.array_equal(got[:, k:], dst.codes.reshape(R, dst_T, -1)[:, k:])


def test_copy_rows_reports_an_index_outside():
    c, oc = make_codecs(128, K3)
    rng = np.random.default_rng(0)
    src, dst = records(rng, 10, oc), records(rng, 10, oc)
    for bad in ([10, 0], [-2, 0]):
        for kw in ("src_idx", "dst_idx"):
            g = up(dst, oc)
            tq.tq_copy_rows(c, up(src, oc), 10, g, 10, 1, 2, **{kw: torch.tensor([bad], dtype=torch.int32, device=DEV)})
            assert tq.tq_codec_device_error(c) == 5 and tq.tq_codec_device_error(c) == 0
            want = dst.codes.copy()
            want[0 if kw == "dst_idx" else 1] = src.codes[1 if kw == "dst_idx" else 0]
            assert np.array_equal(g.codes.cpu().numpy().view(np.uint32), want)


# ---------------------------------------------------------------- all of them
def test_a_bounded_shared_cache_over_decode_steps():
    """Decode steps of a ragged batch as a server runs them: quantise and append
    each sequence's new key and value at its own length, attend over the shared
    prefix and the own keys, score the own keys, add the weights, and cut the
    cache when a sequence is full; checked each step against 64 bits on the
    records that the cache should hold."""
    d, B, Hq, Hkv, Tp, T, keep = 128, 3, 8, 2, 150, 24, 10
    R = B * Hkv
    rng = np.random.default_rng(11)
    kc, okc = make_codecs(d, K3)
    vc, ovc = make_codecs(d, V4)
    f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32) * 3).to(DEV)  # noqa: E731
    pre = [tq.Compressed.empty(c, Hkv * Tp) for c in (kc, vc)]
    for c, p in zip((kc, vc), pre):
        tq.tq_quantize(c, f(Hkv * Tp, d), p)
    caches = [[tq.Compressed.empty(c, R * T) for c in (kc, vc)] for _ in range(2)]
    new = [tq.Compressed.empty(c, R) for c in (kc, vc)]
    mass, mass2 = torch.zeros((B, Hkv, T), device=DEV), torch.zeros((B, Hkv, keep), device=DEV)
    lens = torch.tensor([0, 7, 3], dtype=torch.int32, device=DEV)
    lens2 = torch.empty_like(lens)
    held = [[[] for _ in range(R)], [[] for _ in range(R)]]       # the host's model: records per block
    model = np.zeros((B, Hkv, T))

    def snapshot(c, rows):
        return [t[rows].cpu().numpy() for t in (c.codes, c.signs, c.norms, c.rnorms) if t is not None]

    def append(at):
        for c, cache, n in zip((kc, vc), caches[0], new):
            tq.tq_quantize(c, f(R, d), n)
            tq.tq_copy_rows(c, n, 1, cache, T, R, 1, dst_idx=at)
        for k in range(2):
            for r in range(R):
                held[k][r].append(snapshot(new[k], slice(r, r + 1)))

    for i in range(7):                                            # ragged starts: sequences 1 and 2 hold 7 and 3
        at = torch.tensor([i if i < n else -1 for n in (0, 7, 3)], dtype=torch.int32, device=DEV)
        append(at.repeat_interleave(Hkv).contiguous())
        for k in range(2):
            for r in range(R):
                if i >= (0, 7, 3)[r // Hkv]:
                    held[k][r].pop()
    cut = 0
    for step in range(40):
        append(lens.repeat_interleave(Hkv).contiguous())
        lens += 1
        n = lens.cpu().numpy()
        q = f(B, Hq, d)
        out, lse = torch.empty((B, Hq, d), device=DEV), torch.empty((B, Hq), device=DEV)
        ws = tq.workspace(tq.tq_attend_prefix_workspace_size(kc, vc, B, Hq, Hkv, Tp, T), DEV)
        tq.tq_attend_prefix(kc, vc, q, B, Hq, Hkv, Tp, *pre, T, *caches[0], out, ws, lens=lens, lse=lse)
        logits = torch.empty((B, Hq, T), device=DEV)
        tq.tq_scores(kc, q, B, Hq, Hkv, T, caches[0][0], logits, tq.workspace(tq.tq_scores_workspace_size(kc, B, Hq, Hkv), DEV))
        tq.tq_mass_update(kc, logits, B, Hq, Hkv, T, mass, lens=lens, lse=lse)
        # the host's side, from the records that each block should hold
        def rec(k, r, oc):
            a = [np.concatenate(x) for x in zip(*held[k][r])]
            u = lambda v: v.view(np.uint32)  # noqa: E731
            e = np.zeros((len(a[0]), 0), np.uint32)
            return O.Compressed(u(a[0]), u(a[1]) if oc.m else e, a[2] if oc.m else a[1], a[3] if oc.m else np.zeros(0, np.float32))
        dec = lambda r, c: O.dequantize(r, c, rotated=True, qjl=True)  # noqa: E731
        pk, pv = (O.Compressed(*(t.cpu().numpy().view(np.uint32) if t is not None and t.dtype == torch.int32 else
                                 (np.zeros((Hkv * Tp, 0), np.uint32) if t is None and j == 1 else
                                  np.zeros(0, np.float32) if t is None else t.cpu().numpy())
                                 for j, t in enumerate((c.codes, c.signs, c.norms, c.rnorms)))) for c in pre)
        qr = q.double().cpu().numpy() @ okc.Pi.T
        for b in range(B):
            for h in range(Hkv):
                r = b * Hkv + h
                assert len(held[0][r]) == n[b]
                k = np.concatenate([dec(pk, okc)[h * Tp:(h + 1) * Tp], dec(rec(0, r, okc), okc)])
                v = np.concatenate([dec(pv, ovc)[h * Tp:(h + 1) * Tp], dec(rec(1, r, ovc), ovc)])
                for hq in range(h * 4, h * 4 + 4):
                    l = k @ qr[b, hq] / math.sqrt(d)
                    p = np.exp(l - l.max())
                    s, p = l.max() + math.log(p.sum()), p / p.sum()
                    o = (p @ v) @ ovc.Pi
                    # |l| sums up to 2^9 here: E L <= 300 u 2^9 = 2^-7 in the worst case, 2^-12 for rounding
                    # errors that do not all agree; logits of tq_scores carry 2^-14 |q| nu of their own
                    assert np.abs(out[b, hq].double().cpu().numpy() - o).max() <= 2e-3 * np.abs(p @ np.abs(v)).max()
                    assert abs(lse[b, hq].item() - s) <= 1e-3
                    model[b, h, :n[b]] += p[Tp:]
                g = mass[b, h, :n[b]].double().cpu().numpy()
                assert np.all(np.abs(g - model[b, h, :n[b]]) <= 4 * 40 * 2e-3)
        if n.max() == T - 1:
            cut += 1
            idx = torch.empty((B, Hkv, keep), dtype=torch.int32, device=DEV)
            m = mass.cpu().numpy()
            tq.tq_evict_select(kc, mass, B, Hkv, T, keep, idx, lens=lens, sink=1, recent=3, mass_out=mass2, lens_out=lens2)
            for c, a, z in zip((kc, vc), *caches):
                tq.tq_copy_rows(c, a, T, z, T, R, keep, src_idx=idx)
            want, kept = evict_reference(m, n, keep, 1, 3)
            assert np.array_equal(idx.cpu().numpy(), want)
            caches.reverse()
            mass.zero_()
            mass[..., :keep] = mass2
            old, model = model, np.zeros((B, Hkv, T))
            lens.copy_(lens2)
            for r in range(R):
                at = [t for t in want[r // Hkv, r % Hkv] if t >= 0]
                model[r // Hkv, r % Hkv, :len(at)] = old[r // Hkv, r % Hkv, at]
                for k in range(2):
                    held[k][r] = [held[k][r][t] for t in at]
    assert cut >= 2
    assert tq.tq_codec_device_error(kc) == 0 and tq.tq_codec_device_error(vc) == 0


# ------------------------------------------------------------------- refusals
def test_refusals_leave_the_outputs_alone():
    c = Case(128, K3, V4, 2, 4, 2, 20, 10, [3, 10], seed=12)
    lib, g = tq.c_api(), c.g
    import ctypes
    R = ctypes.byref
    st = {k: g[k].struct() for k in ("Kp", "Vp", "K", "V")}
    out = torch.full((2, 4, 128), 7.0, device=DEV)
    ws = c.ws()
    good = dict(kc=c.kc.handle, vc=c.vc.handle, q=g["q"].data_ptr(), dt=1, B=2, Hq=4, Hkv=2, scale=0.0, Tp=20,
                Kp=R(st["Kp"]), Vp=R(st["Vp"]), T=10, lens=g["lens"].data_ptr(), K=R(st["K"]), V=R(st["V"]),
                ws=ws.data_ptr(), n=ws.numel(), out=out.data_ptr(), odt=0, lse=None, stream=None)
    call = lambda **kw: lib.tq_attend_prefix(*{**good, **kw}.values())  # noqa: E731
    d64, d512 = tq.Codec(64, (3,), 128, 0), tq.Codec(512, (3,), 0, 0)
    host = tq.Codec(128, (3,), 128, 0, device=-1)
    sketched = tq.Codec(128, (3,), 256, 0)
    for kw, want in ((dict(kc=None), 1), (dict(kc=host.handle), 1), (dict(kc=d64.handle), 1), (dict(dt=3), 1),
                     (dict(kc=d512.handle, vc=d512.handle), 2), (dict(vc=sketched.handle), 2), (dict(odt=-1), 1),
                     (dict(B=-1), 1), (dict(Hq=3), 1), (dict(Hq=0), 1), (dict(Hq=66, Hkv=2), 2), (dict(Tp=-1), 1),
                     (dict(T=-1), 1), (dict(T=2 ** 31), 2), (dict(Tp=2 ** 31), 2), (dict(B=2 ** 30), 2),
                     (dict(scale=-1.0), 1), (dict(scale=math.nan), 1), (dict(q=None), 1), (dict(out=None), 1),
                     (dict(q=g["q"].data_ptr() + 2), 1), (dict(out=out.data_ptr() + 4), 1), (dict(Kp=None), 1),
                     (dict(V=None), 1), (dict(ws=None), 1), (dict(ws=ws.data_ptr() + 4), 1), (dict(n=ws.numel() - 1), 1),
                     (dict(n=0), 1), (dict(lens=g["lens"].data_ptr() + 1), 1), (dict(lse=out.data_ptr() + 2), 1)):
        assert call(**kw) == want, (kw, tq.tq_last_error_string())
    assert torch.all(out == 7.0)
    assert call(B=0) == 0 and call(Tp=0, Kp=None, Vp=None) == 0 and call() == 0
    m = torch.zeros((2, 2, 10), device=DEV)
    i = torch.zeros((2, 2, 10), dtype=torch.int32, device=DEV)
    p, k = m.data_ptr(), c.kc.handle
    for args, want in (((None, p, 2, 2, 10, None, 5, 0, 0, i.data_ptr(), None, None, None), 1),
                       ((k, p, 2, 2, 10, None, 0, 0, 0, i.data_ptr(), None, None, None), 1),
                       ((k, p, 2, 2, 10, None, 5, 3, 3, i.data_ptr(), None, None, None), 1),
                       ((k, p, 2, 2, 10, None, 5, -1, 0, i.data_ptr(), None, None, None), 1),
                       ((k, p, 2, 2, 10, None, 5, 0, 2 ** 62, i.data_ptr(), None, None, None), 1),
                       ((k, None, 2, 2, 10, None, 5, 0, 0, i.data_ptr(), None, None, None), 1),
                       ((k, p, 2, 2, 10, None, 5, 0, 0, None, None, None, None), 1),
                       ((k, p, 2, 2, 10, None, 5, 0, 0, i.data_ptr(), p, None, None), 1),
                       ((k, p, 2, 2, 10, i.data_ptr(), 5, 0, 0, i.data_ptr(), None, i.data_ptr(), None), 1)):
        assert lib.tq_evict_select(*args) == want, tq.tq_last_error_string()
    for args, want in (((k, p, 2, 3, 2, 10, None, None, 0.0, 1.0, p, None), 1),
                       ((k, p, 2, 4, 2, 10, None, None, -1.0, 1.0, p, None), 1),
                       ((k, p, 2, 4, 2, 10, None, None, 0.0, math.inf, p, None), 1),
                       ((k, None, 2, 4, 2, 10, None, None, 0.0, 1.0, p, None), 1),
                       ((k, p, 2, 66, 2, 10, None, None, 0.0, 1.0, p, None), 2)):
        assert lib.tq_mass_update(*args) == want, tq.tq_last_error_string()
    s, t = R(st["K"]), R(st["Kp"])
    for args, want in (((k, None, 10, t, 20, 1, 1, None, None, None), 1), ((k, s, 10, t, 20, 1, 11, None, None, None), 1),
                       ((k, s, -1, t, 20, 1, 1, None, None, None), 1), ((k, s, 10, s, 10, 1, 1, None, None, None), 1),
                       ((k, s, 10, t, 20, -1, 1, None, None, None), 1), ((k, s, 0, t, 20, 1, 1, i.data_ptr(), None, None), 1),
                       ((k, s, 10, t, 20, 1, 1, i.data_ptr() + 2, None, None), 1)):
        assert lib.tq_copy_rows(*args) == want, tq.tq_last_error_string()
    assert not torch.any(m) and not torch.any(i)
    # the binding looks at types, devices and sizes before the library does
    for kw in (dict(out=out.double()), dict(q=g["q"].cpu())):
        with pytest.raises((AssertionError, KeyError)):
            tq.tq_attend_prefix(c.kc, c.vc, kw.get("q", g["q"]), 2, 4, 2, 20, g["Kp"], g["Vp"], 10, g["K"], g["V"],
                                kw.get("out", out), ws, lens=g["lens"])
    with pytest.raises(AssertionError):
        tq.tq_attend_prefix(c.kc, c.vc, g["q"], 2, 4, 2, 21, g["Kp"], g["Vp"], 10, g["K"], g["V"], out, ws)
    with pytest.raises(AssertionError):
        tq.tq_mass_update(c.kc, m, 2, 4, 2, 10, m)
