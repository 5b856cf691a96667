"""The operators of a shared, bounded compressed cache: their cases, their plain
form in elementary torch operations, and the calls a user makes.

  attend_prefix   decode attention of a batch whose sequences share one long
                  compressed prefix and each own a ragged compressed tail
                  (tq_attend_prefix)
  mass            accumulated attention weight per cached key
                  (tq_mass_update)
  evict           choice of the keys that stay and compaction of both caches
                  (tq_evict_select, tq_copy_rows)

Compressed rows follow include/tq.h: planar code words, sign words, norms and
residual norms, with the codec's D signs, sketch S and Lloyd-Max tables.
"""
import functools
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
K_SEED, V_SEED = 0, 1


# ----------------------------------------------------------------------- cases
def listed():
    att = dict(op="attend_prefix", Hq=32, Hkv=8, d=128, kbits="3", m=128, vbits="4", q="bf16")
    return [
        # one chat turn on a short system prompt: a single sequence, latency counts
        dict(att, name="attend one sequence", B=1, Tp=509, T=63, out="bf16", lse=False),
        # four samples of one long document, statistics kept for the eviction
        dict(att, name="attend 4 x 32k, lse", B=4, Tp=32768, T=512, out="f32", lse=True),
        # a served batch over a 32k system prompt, in the model's type
        dict(att, name="attend 32 x 32k", B=32, Tp=32768, T=1024, out="bf16", lse=False),
        # the same as fp32 with its statistics, odd lengths, many sequences
        dict(att, name="attend 64 x 16k, lse", B=64, Tp=16411, T=777, out="f32", lse=True),
        # the long-context codec (2.5 bits, m = 64) at 131,072 keys less one
        dict(att, name="attend 8 x 131k, 2.5 bit", B=8, Tp=131071, T=257, kbits="2+3", m=64, out="f16", lse=False),
        # the d = 64 codec without grouped heads and without a key sketch
        dict(att, name="attend d64 no groups", B=16, Hq=20, Hkv=20, d=64, kbits="4", m=0, vbits="3", Tp=4096, T=333,
             q="f32", out="f32", lse=False),
        # the tiny workload's shape: one KV head, 16 query heads
        dict(op="mass", name="mass 16 heads x 512", B=1, Hq=16, Hkv=1, T=512, d=128, lse=False, decay=1.0),
        # the decode layer at 32k keys, the softmax taken from the logits alone
        dict(op="mass", name="mass 8 x 32k", B=8, Hq=32, Hkv=8, T=32768, d=128, lse=False, decay=1.0),
        # a ragged batch with given statistics and a fading history
        dict(op="mass", name="mass 32 x 4k, lse", B=32, Hq=32, Hkv=8, T=4093, d=128, lse=True, decay=0.96875),
        # one short sequence over its budget
        dict(op="evict", name="evict 1 x 700 to 256", B=1, Hkv=8, T=700, keep=256, sink=4, recent=64, d=128, kbits="3",
             m=128, vbits="4"),
        # the decode layer's 32k cache cut to a quarter
        dict(op="evict", name="evict 8 x 32k to 8k", B=8, Hkv=8, T=32768, keep=8192, sink=4, recent=1024, d=128,
             kbits="3", m=128, vbits="4"),
        # many ragged sequences, odd sizes, the 2.5-bit codec
        dict(op="evict", name="evict 64 x 4k to 1k", B=64, Hkv=8, T=4099, keep=1021, sink=1, recent=127, d=128,
             kbits="2+3", m=64, vbits="4"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend_prefix", "attend_prefix", "mass", "evict"])
    if op == "attend_prefix":
        B = _log(rng, 1, 64)
        d = rng.choice([64, 128, 128])
        Hkv = rng.choice([1, 2, 8])
        G = rng.choice([1, 2, 4, 7, 8])
        Tp = _log(rng, 1, max(2, min(131072, (1 << 20) // B, (1 << 22) // (B * G))))
        T = _log(rng, 1, 1024)
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, kbits=rng.choice(["1", "2", "3", "4", "2+3"]),
                    m=rng.choice([0, 32, 64, 128]), vbits=rng.choice(["2", "3", "4", "2+3"]), Tp=Tp, T=T,
                    q=rng.choice(["bf16", "f16", "f32"]), out=rng.choice(["bf16", "f16", "f32"]),
                    lse=rng.random() < 0.3)
    B = _log(rng, 1, 64)
    Hkv = rng.choice([1, 2, 8])
    T = _log(rng, 1 if op == "mass" else 16, min(131072, (1 << 21) // (B * Hkv)))
    if op == "mass":
        return dict(op=op, B=B, Hq=Hkv * rng.choice([1, 2, 4, 5, 8]), Hkv=Hkv, T=T, d=rng.choice([64, 128]),
                    lse=rng.random() < 0.5, decay=rng.choice([1.0, 0.96875, 0.5, 0.0]))
    keep = _log(rng, 4, T)
    sink = rng.randint(0, min(4, keep))
    return dict(op=op, B=B, Hkv=Hkv, T=T, keep=keep, sink=sink, recent=rng.randint(0, (keep - sink) // 2), d=128,
                kbits=rng.choice(["2", "3", "2+3"]), m=rng.choice([0, 64, 128]), vbits=rng.choice(["3", "4"]))


def _bits(text):
    return tuple(int(v) for v in text.split("+"))


def _record_words(case, key):
    """32-bit words of one compressed key or value, norms included."""
    bits = _bits(case["kbits" if key else "vbits"])
    m = case["m"] if key else 0
    return sum(bits) * (case["d"] // len(bits)) // 32 + m // 32 + (2 if m else 1)


def _mean_len(case):
    lo, hi, n = case["T"] // 4, case["T"], case["B"]
    return hi if n == 1 else (hi + (n - 2) * (lo + hi) / 2) / n


def work(case):
    if case["op"] == "attend_prefix":
        size = {"f32": 4, "bf16": 2, "f16": 2}
        rows = case["B"] * case["Hq"]
        own_keys = case["B"] * case["Hkv"] * _mean_len(case)
        keys = case["Hkv"] * case["Tp"] + own_keys
        pairs = rows * case["Tp"] + own_keys * (case["Hq"] // case["Hkv"])
        return {"bytes": 4 * keys * (_record_words(case, True) + _record_words(case, False))
                + rows * (case["d"] * (size[case["q"]] + size[case["out"]]) + 4 * case["lse"]),
                "flops": pairs * 2 * (2 * case["d"] + case["m"])}
    keys = case["B"] * case["Hkv"] * _mean_len(case)
    if case["op"] == "mass":
        G = case["Hq"] // case["Hkv"]
        return {"bytes": 4 * keys * (G + (2 if case["decay"] else 1)), "flops": 4 * keys * G}
    kept = case["B"] * case["Hkv"] * min(case["keep"], _mean_len(case))
    return {"bytes": 4 * keys + 8 * kept + 8 * kept * (_record_words(case, True) + _record_words(case, False)),
            "flops": keys}


# ------------------------------------------------------------ the codec's tables
def _splitmix(seed, n):
    """The first n outputs of splitmix64."""
    z = np.uint64(seed) + np.arange(1, n + 1, dtype=np.uint64) * np.uint64(0x9E3779B97F4A7C15)
    z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
    z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
    return z ^ (z >> np.uint64(31))


@functools.lru_cache(None)
def _levels(bits, d):
    """Lloyd-Max centroids of f(z) ~ (1 - z^2/d)^((d-3)/2), |z| < sqrt(d), in double."""
    x, w = np.polynomial.legendre.leggauss(96)
    dens = lambda z: np.maximum(1.0 - z * z / d, 0.0) ** ((d - 3) / 2)  # noqa: E731
    h = 1 << (bits - 1)
    c = np.minimum((np.arange(h) + 0.5) * 2.5 / h, 0.9 * math.sqrt(d))
    top = min(math.sqrt(d), 12.0)  # the density is below e^-60 of its peak beyond
    for _ in range(20000):
        b = np.concatenate([[0.0], 0.5 * (c[1:] + c[:-1]), [top]])
        z = (0.5 * (b[1:] - b[:-1]))[:, None] * x + (0.5 * (b[1:] + b[:-1]))[:, None]
        f = dens(z) * w
        new = (f * z).sum(1) / f.sum(1)
        moved, c = np.abs(new - c).max(), new
        if moved < 1e-12:
            break
    return np.concatenate([-c[::-1], c])


@functools.lru_cache(None)
def _tables(d, bits, m, seed):
    """Pi [d, d], S [m, d], centroids and cell borders per segment, on the GPU."""
    neg = (_splitmix(seed, d) >> np.uint64(63)).astype(bool)
    H = np.ones((1, 1))
    while H.shape[0] < d:
        H = np.block([[H, H], [H, -H]])
    Pi = H * np.where(neg, -1.0, 1.0) / math.sqrt(d)
    o = _splitmix(seed ^ 0x5851F42D4C957F2D, 2 * m * d).reshape(-1, 2) >> np.uint64(11)
    u1, u2 = (o[:, 0].astype(np.float64) + 1) * 2.0 ** -53, o[:, 1].astype(np.float64) * 2.0 ** -53
    S = (np.sqrt(-2.0 * np.log(u1)) * np.cos(2.0 * math.pi * u2)).astype(np.float32).reshape(m, d)
    cen = [_levels(b, d).astype(np.float32) for b in bits]
    bnd = [(0.5 * (_levels(b, d)[1:] + _levels(b, d)[:-1])).astype(np.float32) for b in bits]
    put = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).to(DEV, t)  # noqa: E731
    return {"d": d, "bits": bits, "m": m, "Pi": put(Pi, torch.float64), "S": put(S, torch.float32),
            "cen": [put(c, torch.float32) for c in cen], "bnd": [put(b, torch.float32) for b in bnd]}


def _planes_to_words(b):
    """0/1 values [n, 32 w] to int32 words [n, w], the first in the lowest bit."""
    t = (b.to(torch.int64).view(b.shape[0], -1, 32) << torch.arange(32, device=b.device)).sum(-1)
    return torch.where(t >= 1 << 31, t - (1 << 32), t).to(torch.int32)


def _compress(x, tab):
    """The records of the rows x, by the definitions of include/tq.h."""
    d, n = tab["d"], x.shape[0]
    norms = x.norm(dim=1)
    y = (x / norms.clamp_min(1e-30)[:, None]) @ tab["Pi"].float().T
    seg = d // len(tab["bits"])
    words, hat = [], []
    for s, b in enumerate(tab["bits"]):
        ys = y[:, s * seg:(s + 1) * seg]
        code = torch.bucketize(ys.contiguous() * math.sqrt(d), tab["bnd"][s], right=True)
        words += [_planes_to_words((code >> p) & 1) for p in range(b)]
        hat.append(tab["cen"][s][code] / math.sqrt(d))
    rec = {"codes": torch.cat(words, 1), "norms": norms, "signs": None, "rnorms": None}
    if tab["m"]:
        r = y - torch.cat(hat, 1)
        rec["signs"] = _planes_to_words((r @ tab["S"].T) >= 0)
        rec["rnorms"] = r.norm(dim=1)
    return rec


# ----------------------------------------------------------------------- inputs
@functools.lru_cache(None)
def _codec(d, bits, m, seed):
    import kv_cache_vector_09_b200 as tq
    return tq.Codec(d, bits, m, seed)


def _as_cache(rec):
    import kv_cache_vector_09_b200 as tq
    return tq.Compressed(rec["codes"], rec["signs"], rec["norms"], rec["rnorms"])


def _lens(case, g):
    """Ragged lengths: T for the last sequence, none for the first of several."""
    n = torch.randint(case["T"] // 4, case["T"] + 1, (case["B"],), generator=g, device=DEV)
    n[0] = 0
    n[-1] = case["T"]
    return n.to(torch.int32)


def _rows(g, n, d, value):
    """Heavy-tailed keys or values: lognormal norms, a few strong channels."""
    x = torch.randn((n, d), generator=g, device=DEV)
    x[:, :2] *= 1.5 if value else 4.0
    return x * torch.exp(0.4 * torch.randn((n, 1), generator=g, device=DEV))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "mass":
        B, Hq, Hkv, T = case["B"], case["Hq"], case["Hkv"], case["T"]
        s["lens"] = _lens(case, g)
        s["logits"] = torch.randn((B, Hq, T), generator=g, device=DEV) * (1.5 * math.sqrt(case["d"]))
        s["logits"][..., :1] += 6.0 * math.sqrt(case["d"])  # the first token draws weight, as sinks do
        held = torch.arange(T, device=DEV) < s["lens"][:, None]
        s["lse"] = None
        if case["lse"]:  # statistics of these keys and of a prefix beside them
            l = (s["logits"].double() / math.sqrt(case["d"])).masked_fill(~held[:, None], -math.inf)
            s["lse"] = torch.logaddexp(torch.logsumexp(l, -1), torch.full_like(l[..., 0], 9.0)).float()
        s["logits"].masked_fill_(~held[:, None], math.nan)  # rows that were never written
        s["mass"] = torch.rand((B, Hkv, T), generator=g, device=DEV) * 4.0
        if own:
            s["kc"] = _codec(case["d"], (3,), 0, K_SEED)
        return s
    kb, vb, d, m = _bits(case["kbits"]), _bits(case["vbits"]), case["d"], case["m"]
    s["kt"], s["vt"] = _tables(d, kb, m, K_SEED), _tables(d, vb, 0, V_SEED)
    if own:
        s["kc"], s["vc"] = _codec(d, kb, m, K_SEED), _codec(d, vb, 0, V_SEED)
    s["lens"] = _lens(case, g)
    if case["op"] == "attend_prefix":
        B, Hq, Hkv, Tp, T = case["B"], case["Hq"], case["Hkv"], case["Tp"], case["T"]
        for name, n in (("p", Hkv * Tp), ("o", B * Hkv * T)):
            s["K" + name] = _compress(_rows(g, n, d, False), s["kt"])
            s["V" + name] = _compress(_rows(g, n, d, True), s["vt"])
        s["q"] = torch.randn((B, Hq, d), generator=g, device=DEV).to(DTYPES[case["q"]])
        s["out"] = torch.empty((B, Hq, d), device=DEV, dtype=DTYPES[case["out"]])
        s["lse"] = torch.empty((B, Hq), device=DEV) if case["lse"] else None
        if own:
            import kv_cache_vector_09_b200 as tq
            s["ws"] = tq.workspace(tq.tq_attend_prefix_workspace_size(s["kc"], s["vc"], B, Hq, Hkv, Tp, T), DEV)
            s["caches"] = [_as_cache(s[k]) for k in ("Kp", "Vp", "Ko", "Vo")]
        return s
    B, Hkv, T, keep = case["B"], case["Hkv"], case["T"], case["keep"]
    rows, Td = B * Hkv, keep + 64  # room for the tokens that follow
    mass = torch.exp(2.0 * torch.randn((B, Hkv, T), generator=g, device=DEV))
    s["mass"] = mass * (torch.rand((B, Hkv, T), generator=g, device=DEV) > 0.25)  # keys never looked at: ties
    word = lambda n, w: torch.randint(-2 ** 31, 2 ** 31, (n, w), generator=g, device=DEV).to(torch.int32)  # noqa: E731
    nrm = lambda n: torch.rand((n,), generator=g, device=DEV) + 0.5  # noqa: E731
    for name, bits, mm in (("K", kb, m), ("V", vb, 0)):
        W, MS = sum(bits) * (d // len(bits)) // 32, mm // 32
        s[name] = {"codes": word(rows * T, W), "norms": nrm(rows * T), "signs": word(rows * T, MS) if mm else None,
                   "rnorms": nrm(rows * T) if mm else None}
        s[name + "2"] = {k: None if v is None else torch.zeros((rows * Td,) + v.shape[1:], dtype=v.dtype, device=DEV)
                         for k, v in s[name].items()}
    s["idx"] = torch.empty((B, Hkv, keep), dtype=torch.int32, device=DEV)
    s["mass2"] = torch.empty((B, Hkv, keep), device=DEV)
    s["lens2"] = torch.empty((B,), dtype=torch.int32, device=DEV)
    if own:
        s["caches"] = [_as_cache(s[k]) for k in ("K", "V", "K2", "V2")]
    return s


# -------------------------------------------------------------- the plain forms
def _unpack(words, at, planes, per):
    """Integers of `planes` bit planes of `per` words each, from word `at` on."""
    w = words[..., at:at + planes * per]
    bits = ((w[..., None] >> torch.arange(32, device=w.device, dtype=torch.int32)) & 1).flatten(-2)
    bits = bits.unflatten(-1, (planes, per * 32))
    return (bits << torch.arange(planes, device=w.device, dtype=torch.int32)[:, None]).sum(-2)


def _centroids(codes, tab):
    """The decoded rotated coordinates (z units) of packed codes [..., W]."""
    per = tab["d"] // len(tab["bits"]) // 32
    at = [0, tab["bits"][0] * per]
    return torch.cat([tab["cen"][k][_unpack(codes, at[k], b, per)] for k, b in enumerate(tab["bits"])], -1)


def _scores(q, w, rec, tab, lead):
    """Estimates <q, x> of rotated queries q [.., r, d] and w = S q against the
    keys [.., t] of rec, whose rows are laid out as `lead`."""
    c = _centroids(rec["codes"].view(*lead, -1), tab)
    a = torch.matmul(q, c.transpose(-1, -2)) / math.sqrt(tab["d"])
    if tab["m"]:
        s = _unpack(rec["signs"].view(*lead, -1), 0, 1, tab["m"] // 32).float() * 2 - 1
        gam = rec["rnorms"].view(*lead) * (math.sqrt(math.pi / 2) / tab["m"])
        a = a + torch.matmul(w, s.transpose(-1, -2)) * gam[..., None, :]
    return a * rec["norms"].view(*lead)[..., None, :]


def _plain_attend(s):
    c = s["case"]
    B, Hq, Hkv, Tp, T, d = (c[k] for k in ("B", "Hq", "Hkv", "Tp", "T", "d"))
    G = Hq // Hkv
    q = s["q"].float().view(B, Hkv, G, d) @ s["kt"]["Pi"].float().T
    w = q @ s["kt"]["S"].T if c["m"] else None
    fold = lambda v: None if v is None else v.transpose(0, 1).reshape(Hkv, B * G, -1)  # noqa: E731
    lp = _scores(fold(q), fold(w), s["Kp"], s["kt"], (Hkv, Tp)).view(Hkv, B, G, Tp).transpose(0, 1)
    lo = _scores(q, w, s["Ko"], s["kt"], (B, Hkv, T))
    held = torch.arange(T, device=DEV) < s["lens"][:, None]
    lo = torch.where(held[:, None, None], lo, torch.full_like(lo, -math.inf))
    l = torch.cat([lp, lo], -1) / math.sqrt(d)
    top = l.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    e = torch.exp(l - top)
    z = e.sum(-1, keepdim=True)
    vp = _centroids(s["Vp"]["codes"].view(Hkv, Tp, -1), s["vt"]) * s["Vp"]["norms"].view(Hkv, Tp, 1)
    vo = _centroids(s["Vo"]["codes"].view(B, Hkv, T, -1), s["vt"]) * s["Vo"]["norms"].view(B, Hkv, T, 1)
    o = torch.matmul(e[..., :Tp].transpose(0, 1).reshape(Hkv, B * G, Tp), vp).view(Hkv, B, G, d).transpose(0, 1)
    o = (o + torch.matmul(e[..., Tp:], vo)) / math.sqrt(d) / torch.where(z > 0, z, torch.ones_like(z))
    o = (o @ s["vt"]["Pi"].float()).reshape(B, Hq, d)
    s["out"].copy_(o)
    if s["lse"] is None:
        return s["out"]
    s["lse"].copy_((top + torch.log(z)).view(B, Hq))
    return s["out"], s["lse"]


def _plain_mass(s):
    c = s["case"]
    B, Hq, Hkv, T = (c[k] for k in ("B", "Hq", "Hkv", "T"))
    held = (torch.arange(T, device=DEV) < s["lens"][:, None])[:, None]
    l = torch.where(held, s["logits"] / math.sqrt(c["d"]), torch.full_like(s["logits"], -math.inf))
    if s["lse"] is None:
        top = l.amax(-1, keepdim=True)
        top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
        p = torch.exp(l - top)
        z = p.sum(-1, keepdim=True)
        p = p / torch.where(z > 0, z, torch.ones_like(z))
    else:
        p = torch.exp(l - s["lse"][..., None])
    add = p.view(B, Hkv, Hq // Hkv, T).sum(2)
    s["mass"].copy_(torch.where(held, s["mass"] * c["decay"] + add, s["mass"]))
    return s["mass"]


def _plain_evict(s):
    c = s["case"]
    B, Hkv, T, keep = (c[k] for k in ("B", "Hkv", "T", "keep"))
    t = torch.arange(T, device=DEV, dtype=torch.int32)
    n = s["lens"][:, None, None]
    always = (t < c["sink"]) | (t >= n - c["recent"])
    rank = torch.where(always, torch.full_like(s["mass"], math.inf), s["mass"])
    rank = torch.where(t < n, rank, torch.full_like(rank, -math.inf))
    pick = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    pick = torch.sort(torch.where(pick < n, pick, torch.full_like(pick, T)), dim=-1).values
    if keep > T:
        pick = torch.cat([pick, torch.full((B, Hkv, keep - T), T, device=DEV, dtype=pick.dtype)], -1)
    held = pick < T
    s["idx"].copy_(torch.where(held, pick, torch.full_like(pick, -1)))
    at = torch.where(held, pick, torch.zeros_like(pick))
    s["mass2"].copy_(torch.where(held, torch.gather(s["mass"], -1, at), torch.zeros_like(s["mass2"])))
    s["lens2"].copy_(torch.clamp(s["lens"], max=keep))
    rows = B * Hkv
    src = (at.view(rows, keep) + torch.arange(rows, device=DEV)[:, None] * T).flatten()
    move = lambda a, b: b.unflatten(0, (rows, -1))[:, :keep].copy_(  # noqa: E731
        torch.where(held.view((rows, keep) + (1,) * (a.dim() - 1)), a[src].unflatten(0, (rows, keep)),
                    b.unflatten(0, (rows, -1))[:, :keep]))
    [move(s[k][f], s[k + "2"][f]) for k in ("K", "V") for f in s[k] if s[k][f] is not None]
    return _evict_outputs(s)


def _evict_outputs(s):
    caches = {k + f: v for k in ("K2", "V2") for f, v in s[k].items() if v is not None}
    return dict(caches, idx=s["idx"], mass=s["mass2"], lens=s["lens2"])


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"attend_prefix": _plain_attend, "mass": _plain_mass, "evict": _plain_evict}[c["op"]](s)
    import kv_cache_vector_09_b200 as tq
    if c["op"] == "attend_prefix":
        Kp, Vp, K, V = s["caches"]
        tq.tq_attend_prefix(s["kc"], s["vc"], s["q"], c["B"], c["Hq"], c["Hkv"], c["Tp"], Kp, Vp, c["T"], K, V,
                            s["out"], s["ws"], lens=s["lens"], lse=s["lse"])
        return s["out"] if s["lse"] is None else (s["out"], s["lse"])
    if c["op"] == "mass":
        return tq.tq_mass_update(s["kc"], s["logits"], c["B"], c["Hq"], c["Hkv"], c["T"], s["mass"], lens=s["lens"],
                                 lse=s["lse"], decay=c["decay"])
    K, V, K2, V2 = s["caches"]
    rows, Td = c["B"] * c["Hkv"], c["keep"] + 64
    tq.tq_evict_select(s["kc"], s["mass"], c["B"], c["Hkv"], c["T"], c["keep"], s["idx"], lens=s["lens"],
                       sink=c["sink"], recent=c["recent"], mass_out=s["mass2"], lens_out=s["lens2"])
    tq.tq_copy_rows(s["kc"], K, c["T"], K2, Td, rows, c["keep"], src_idx=s["idx"])
    tq.tq_copy_rows(s["vc"], V, c["T"], V2, Td, rows, c["keep"], src_idx=s["idx"])
    return _evict_outputs(s)


# ------------------------------------------------------------------- 64 bits
def _decode64(rec, tab, lo, hi):
    """Rows lo..hi of rec decoded back to the original coordinates in double."""
    d, n = tab["d"], hi - lo
    words = rec["codes"][lo:hi].long()
    bit = torch.arange(32, device=DEV)
    y = torch.zeros((n, d), dtype=torch.float64, device=DEV)
    col, at, per = 0, 0, d // len(tab["bits"]) // 32
    for s, b in enumerate(tab["bits"]):
        code = torch.zeros((n, per * 32), dtype=torch.long, device=DEV)
        for p in range(b):
            code += (((words[:, at:at + per, None] >> bit) & 1) << p).flatten(1)
            at += per
        y[:, col:col + per * 32] = tab["cen"][s].double()[code] / math.sqrt(d)
        col += per * 32
    if tab["m"]:
        sg = ((rec["signs"][lo:hi].long()[:, :, None] >> bit) & 1).flatten(1).double() * 2 - 1
        y += (sg @ tab["S"].double()) * (math.sqrt(math.pi / 2) / tab["m"] * rec["rnorms"][lo:hi].double())[:, None]
    return (y * rec["norms"][lo:hi].double()[:, None]) @ tab["Pi"]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "attend_prefix":
        B, Hq, Hkv, Tp, T, d = (case[k] for k in ("B", "Hq", "Hkv", "Tp", "T", "d"))
        G, lens = Hq // Hkv, s["lens"].tolist()
        out = torch.zeros((B, Hq, d), dtype=torch.float64, device=DEV)
        lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=DEV)
        for h in range(Hkv):
            kp, vp = (_decode64(s[k + "p"], s[k.lower() + "t"], h * Tp, (h + 1) * Tp) for k in "KV")
            for b in range(B):
                r = (b * Hkv + h) * T
                ko, vo = (_decode64(s[k + "o"], s[k.lower() + "t"], r, r + lens[b]) for k in "KV")
                q = s["q"][b, h * G:(h + 1) * G].double()
                l = torch.cat([q @ kp.T, q @ ko.T], 1) / math.sqrt(d)
                if l.shape[1]:
                    lse[b, h * G:(h + 1) * G] = torch.logsumexp(l, 1)
                    out[b, h * G:(h + 1) * G] = torch.softmax(l, 1) @ torch.cat([vp, vo])
        return (out, lse) if case["lse"] else out
    if case["op"] == "mass":
        G = case["Hq"] // case["Hkv"]
        mass = s["mass"].double()
        for b, n in enumerate(s["lens"].tolist()):
            if n:
                l = s["logits"][b, :, :n].double() / math.sqrt(case["d"])
                p = torch.softmax(l, -1) if s["lse"] is None else torch.exp(l - s["lse"][b].double()[:, None])
                mass[b, :, :n] = mass[b, :, :n] * case["decay"] + p.view(case["Hkv"], G, n).sum(1)
        return mass
    B, Hkv, T, keep = (case[k] for k in ("B", "Hkv", "T", "keep"))
    if B * Hkv * T > 3_000_000:
        return None
    mass, kept = s["mass"].double().cpu().numpy(), np.zeros((B, Hkv, keep))
    for b, n in enumerate(s["lens"].tolist()):
        for h in range(Hkv):
            must = [t for t in range(n) if t < case["sink"] or t >= n - case["recent"]] if n > keep else list(range(n))
            free = np.setdiff1d(np.arange(n), must)
            best = free[np.lexsort((free, -mass[b, h, free]))][:max(0, min(n, keep) - len(must))]
            at = np.sort(np.concatenate([np.array(must, dtype=np.int64), best.astype(np.int64)]))
            kept[b, h, :len(at)] = mass[b, h, at]
    outs = {k: None for k in ("idx", "lens")}
    outs.update({k + f: None for k in ("K2", "V2") for f, v in s[k].items() if v is not None})
    return dict(outs, mass=kept)
