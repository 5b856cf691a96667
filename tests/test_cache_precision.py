"""Precision of the shared-prefix attention: tolerances that a single rounding of
an operand to fp16 exceeds.

A worst-case sum of d + m absolute terms hides a wrong precision, so rounding
errors are added here as root sums of squares.  Records and queries are random,
so that terms and their errors are independent; LAM = 6 standard deviations
bound a sum of them.  u = 2^-24, R_t = scale nu_t (|q| |c_t| / d + gamma_t coef |S q|),
the standard deviation of a logit over such records.

* A logit: q' and S q' in fp32 (7 u and 6 u of their rms), operands in two fp16
  parts (2^-22 = 4 u each, 4 u for lo lo), 40 accumulating steps whose truncation
  is at most 2 u of the running sum for the sum and each of 16 addends
  (sqrt(40 * 17 / 3) 2 u <= 31 u): together at most 64 u R_t; and, with one sign,
  40 u |l_t| (truncation towards zero at every step, the scalings, the argument
  of the exponential).
* The statistic: sum p_t dl_t, and 8 u (1 + |lse|) for the logarithm, 16 + tiles
  roundings of the sum of exponentials, 4 u each exponential.
* The output: sum p_t (dl_t - dlse) (v_t - o) for the logits; and of
  b = |o| + sqrt(sum p_t^2 |v_t|^2): 16 u for P and V in two parts and the 12
  accumulating steps of a tile, u a tile for the sums over tiles (random signs),
  64 u with one sign (truncation, the inverse rotation), 16 + tiles for the
  normalisation.  P ends at 2^-37 of its tile's largest value norm.
* A result of 16 bits adds its half step, 2^-8 (bf16) or 2^-11 (fp16) of |o|, and
  2^-25 a coordinate where fp16 ends.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from test_gpu_cache import DEV, make_codecs, part, records, up

tq = pytest.importorskip("kv_cache_vector_09_b200")
U, LAM = 2.0 ** -24, 6.0
FL, BF, HF = torch.float32, torch.bfloat16, torch.float16
HALF_STEP = {FL: 0.0, HF: 2.0 ** -11, BF: 2.0 ** -8}

#    d, keys, values, B, Hq, Hkv, Tp, T, lens, query type, scale, query size
CASES = [
    (128, dict(bits=(3,), m=128), dict(bits=(4,), seed=4), 3, 8, 2, 900, 130, [130, 0, 55], BF, 0.5, 3.0),
    (128, dict(bits=(3,), m=128), dict(bits=(4,), seed=4), 5, 32, 8, 129, 127, [127, 0, 1, 126, 63], FL, 0.0, 16.0),
    (128, dict(bits=(2, 3), m=64), dict(bits=(2, 3), seed=9), 2, 4, 2, 1111, 257, [257, 100], HF, 0.0, 12.0),
    (128, dict(bits=(4,), m=0), dict(bits=(3,), seed=9), 17, 7, 1, 0, 300, [0, 300, 299] + [100 + i for i in range(14)], BF, 1.0, 1.0),
    (64, dict(bits=(2,), m=64), dict(bits=(2,), seed=9), 3, 6, 2, 777, 129, [5, 129, 0], BF, 0.5, 3.0),
    (64, dict(bits=(4,), m=0), dict(bits=(3,), seed=9), 16, 20, 20, 130, 40, [0] + [40] * 15, FL, 0.0, 8.0),
]


def half(x):
    """x with one rounding to fp16, each row scaled by a power of two to fp16's range."""
    top = np.abs(x).max(-1, keepdims=True)
    s = 2.0 ** np.floor(np.log2(np.where(top > 0, top, 1.0)) - 9)
    return (x / s).astype(np.float16).astype(np.float64) * s


class Problem:
    """One attention problem on the host: its inputs and its result in 64 bits."""

    def __init__(self, d, ks, vs, B, Hq, Hkv, Tp, T, lens, qdt, scale, qsize):
        rng = np.random.default_rng(d + Tp + T)
        kw = [dict(s) for s in (ks, vs)]
        self.kc, self.vc = (O.make_codec(d, k.pop("bits"), k.pop("m", 0), k.pop("seed", 3), **k) for k in kw)
        self.d, self.B, self.Hq, self.Hkv, self.Tp, self.T, self.lens = d, B, Hq, Hkv, Tp, T, lens
        self.scale = scale
        self.q = torch.from_numpy(qsize * rng.standard_normal((B, Hq, d))).to(qdt)
        self.Kp, self.Vp = records(rng, Hkv * Tp, self.kc), records(rng, Hkv * Tp, self.vc)
        self.K, self.V = records(rng, B * Hkv * T, self.kc), records(rng, B * Hkv * T, self.vc)

    def _keys(self, b, h):
        r = (b * self.Hkv + h) * self.T
        k = [(self.Kp, h * self.Tp, (h + 1) * self.Tp), (self.K, r, r + self.lens[b])]
        v = [(self.Vp, h * self.Tp, (h + 1) * self.Tp), (self.V, r, r + self.lens[b])]
        return [part(*x) for x in k], [part(*x) for x in v]

    def solve(self, rnd=lambda x: x):
        """out, lse, and their error bounds; rnd is applied to every operand of the products."""
        d, G, kc, vc = self.d, self.Hq // self.Hkv, self.kc, self.vc
        sc = self.scale or 1.0 / math.sqrt(d)
        out, lse = np.zeros((self.B, self.Hq, d)), np.full((self.B, self.Hq), -np.inf)
        eo, el = np.zeros((self.B, self.Hq)), np.zeros((self.B, self.Hq))
        for b in range(self.B):
            for h in range(self.Hkv):
                ks, vs = self._keys(b, h)
                c = np.concatenate([kc.coord_cen(O.unpack_codes(r.codes, kc)) for r in ks])
                nu = np.concatenate([r.norms for r in ks]).astype(np.float64)
                gam = np.concatenate([r.rnorms for r in ks]).astype(np.float64) if kc.m else 0.0 * nu
                s = np.concatenate([2.0 * O.unpack_bits(r.signs, kc.m) - 1.0 for r in ks]) if kc.m else np.zeros((len(nu), 1))
                cv = np.concatenate([vc.coord_cen(O.unpack_codes(r.codes, vc)) for r in vs])
                nv = np.concatenate([r.norms for r in vs]).astype(np.float64)
                if not len(nu):
                    continue
                tiles = len(nu) // 64 + 2
                for hq in range(h * G, (h + 1) * G):
                    q = self.q[b, hq].double().numpy() @ kc.Pi.T
                    w = kc.S.astype(np.float64) @ q if kc.m else np.zeros(1)
                    coef = math.sqrt(math.pi / 2) / max(kc.m, 1)
                    l = sc * nu * (rnd(c) @ rnd(q) / math.sqrt(d) + gam * coef * (s @ rnd(w)))
                    R = sc * nu * (np.linalg.norm(q) * np.linalg.norm(c, axis=1) / d + gam * coef * np.linalg.norm(w))
                    e = np.exp(l - l.max())
                    p, z = e / e.sum(), e.sum()
                    v = cv * (nv / math.sqrt(d))[:, None]
                    o = (rnd(e * nv) @ rnd(cv)) / math.sqrt(d) / z
                    out[b, hq], lse[b, hq] = o @ vc.Pi, l.max() + math.log(z)
                    far, vn = np.linalg.norm(v - o, axis=1), np.linalg.norm(v, axis=1)
                    no = np.linalg.norm(o)
                    rms = lambda x: math.sqrt((x * x).sum())  # noqa: E731
                    el[b, hq] = U * (LAM * 64 * rms(p * R) + 40 * (p * np.abs(l)).sum() + 8 * (1 + abs(lse[b, hq]))
                                     + 20 + tiles)
                    eo[b, hq] = U * (LAM * 64 * rms(p * R * far) + 40 * (p * np.abs(l) * far).sum()
                                     + (LAM * (16 + math.sqrt(tiles)) + 64) * (no + rms(p * vn)) + (20 + tiles) * no) \
                        + LAM * math.sqrt(len(nu)) * 2.0 ** -37 * nv.max()
        return out, lse, eo, el


def ratio(err, tol):
    return np.max(err / np.maximum(tol, 1e-300))


@pytest.mark.parametrize("case", CASES)
def test_one_rounding_to_fp16_exceeds_the_tolerance(case):
    # the oracle with its operands rounded once: the bounds below would see it
    p = Problem(*case)
    (o, s, eo, el), (o1, s1, _, _) = p.solve(), p.solve(half)
    live = np.isfinite(s)
    assert ratio(np.linalg.norm(o1 - o, axis=-1), eo) > 2
    assert ratio(np.abs(s1[live] - s[live]), el[live]) > 2


class Device:
    """The same problem on the GPU."""

    def __init__(self, p, ks, vs):
        self.p = p
        (self.kc, okc), (self.vc, ovc) = make_codecs(p.d, ks), make_codecs(p.d, vs)
        self.rec = [up(r, c) for r, c in ((p.Kp, okc), (p.Vp, ovc), (p.K, okc), (p.V, ovc))]
        self.q, self.lens = p.q.to(DEV), torch.tensor(p.lens, dtype=torch.int32, device=DEV)
        self.ws = tq.workspace(tq.tq_attend_prefix_workspace_size(self.kc, self.vc, p.B, p.Hq, p.Hkv, p.Tp, p.T), DEV)

    def run(self, odt, with_lse):
        p = self.p
        out = torch.empty((p.B, p.Hq, p.d), device=DEV, dtype=odt)
        lse = torch.empty((p.B, p.Hq), device=DEV) if with_lse else None
        Kp, Vp, K, V = self.rec
        tq.tq_attend_prefix(self.kc, self.vc, self.q, p.B, p.Hq, p.Hkv, p.Tp, Kp, Vp, p.T, K, V, out, self.ws,
                            lens=self.lens, scale=p.scale, lse=lse)
        return out, lse


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_attend_prefix_precision(case):
    p = Problem(*case)
    g = Device(p, case[1], case[2])
    o, s, eo, el = p.solve()
    live, off = np.isfinite(s), []
    for odt in (FL, BF, HF):
        for with_lse in (True, False):
            out, lse = g.run(odt, with_lse)
            tol = eo + HALF_STEP[odt] * np.linalg.norm(o, axis=-1) + (2.0 ** -25 * math.sqrt(p.d) if odt == HF else 0.0)
            off.append((str(odt), with_lse, ratio(np.linalg.norm(out.double().cpu().numpy() - o, axis=-1), tol)))
            if with_lse:
                off.append(("lse", True, ratio(np.abs(lse.double().cpu().numpy()[live] - s[live]), el[live])))
    assert all(x[2] <= 1 for x in off), off


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_the_result_is_one_value_rounded_to_its_type(case):
    # neither the output's type nor asking for the statistic changes what is computed
    g = Device(Problem(*case), case[1], case[2])
    want, lse = g.run(FL, True)
    for odt in (FL, BF, HF):
        for with_lse in (True, False):
            out, l = g.run(odt, with_lse)
            assert torch.equal(out, want.to(odt)), (odt, with_lse)
            assert l is None or torch.equal(l, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("d,m", [(128, 128), (64, 0)])
@pytest.mark.parametrize("power", [10, 15, 20, 28])
def test_values_beside_a_norm_far_above_theirs(d, m, power):
    # in the tile of the heaviest key, a value of 2^power times the norm whose own key weighs nothing
    ks, vs = dict(bits=(3,), m=m), dict(bits=(4,), seed=4)
    case = (d, ks, vs, 1, 1, 1, 500, 0, [0], FL, 1.0, 4.0)
    p = Problem(*case)
    k = p.kc.coord_cen(O.unpack_codes(p.Kp.codes, p.kc)) / math.sqrt(d)
    if m:
        gam = p.Kp.rnorms.astype(np.float64)[:, None] * math.sqrt(math.pi / 2) / m
        k = k + gam * ((2.0 * O.unpack_bits(p.Kp.signs, m) - 1.0) @ p.kc.S.astype(np.float64))
    l = (k * p.Kp.norms.astype(np.float64)[:, None]) @ (p.kc.Pi @ p.q[0, 0].double().numpy())
    tile = np.arange(500) // 64
    near = np.flatnonzero(tile == tile[l.argmax()])
    far = near[l[near].argmin()]
    assert l[far] - l.max() < -(28 + 30) * math.log(2)
    p.Vp.norms[far] = 3.0 * 2.0 ** power
    o, s, eo, _ = p.solve()
    e, nv = np.exp(l - l.max()), p.Vp.norms.astype(np.float64)
    top = np.array([nv[tile == t].max() for t in range(tile.max() + 1)])[tile]
    lost = np.minimum(2.0 ** -37 * top, e * nv)
    eo = eo - LAM * math.sqrt(500) * 2.0 ** -37 * nv.max() + LAM * math.sqrt((lost * lost).sum()) / e.sum()
    out, _ = Device(p, ks, vs).run(FL, True)
    assert ratio(np.linalg.norm(out.double().cpu().numpy() - o, axis=-1), eo) <= 1


@pytest.mark.gpu
@pytest.mark.parametrize("d,m", [(128, 128), (64, 0)])
@pytest.mark.parametrize("power", [-105, 105])
def test_powers_of_two_pass_from_queries_to_keys(d, m, power):
    # q 2^k against norms 2^-k are the same logits, bit for bit: every scale is a power of two
    ks, vs = dict(bits=(3,), m=m), dict(bits=(4,), seed=4)
    p = Problem(d, ks, vs, 3, 8, 2, 300, 70, [70, 0, 33], FL, 0.0, 4.0)
    want, lse = Device(p, ks, vs).run(FL, True)
    p.q = p.q * 2.0 ** power
    for r in (p.Kp, p.K):
        r.norms *= np.float32(2.0 ** -power)
    out, l = Device(p, ks, vs).run(FL, True)
    assert torch.isfinite(want).all() and torch.equal(out, want) and torch.equal(l, lse)
