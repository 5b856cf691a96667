// Argument checks and launch plans of the shared-prefix attention and of the
// bounded cache.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include "tq_cache.h"
#include "tq_trace.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return p && ((uintptr_t)p & (n - 1)) == 0; }

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

tq_status codec_here(const tq_codec* c, const char* name) {
  if (!c) return tq_fail(TQ_ERR_INVALID_ARG, "%s: null codec", name);
  if (c->device < 0) return tq_fail(TQ_ERR_INVALID_ARG, "%s: host-only codec", name);
  int cur = -1;
  const cudaError_t e = cudaGetDevice(&cur);
  if (e != cudaSuccess) return tq_fail(TQ_ERR_CUDA, "%s: cudaGetDevice: %s", name, cudaGetErrorString(e));
  if (cur != c->device)
    return tq_fail(TQ_ERR_INVALID_ARG, "%s: current device %d is not the codec's device %d", name, cur, c->device);
  return TQ_OK;
}

tq_status rows_ok(const tq_codec* c, const tq_compressed* t, const char* name, const char* what) {
  if (!t) return tq_fail(TQ_ERR_INVALID_ARG, "%s: null %s", name, what);
  if (!aligned(t->codes, 16) || !aligned(t->norms, 16))
    return tq_fail(TQ_ERR_INVALID_ARG, "%s: %s.codes / norms null or not 16-byte aligned", name, what);
  if (c->p.m > 0 && (!aligned(t->signs, 16) || !aligned(t->rnorms, 16)))
    return tq_fail(TQ_ERR_INVALID_ARG, "%s: %s.signs / rnorms null or not 16-byte aligned (m = %d)", name, what, c->p.m);
  return TQ_OK;
}

tq_status dtype_ok(tq_dtype dt, const char* name) {
  if (dt != TQ_F32 && dt != TQ_BF16 && dt != TQ_F16) return tq_fail(TQ_ERR_INVALID_ARG, "%s: dtype %d", name, (int)dt);
  return TQ_OK;
}

// heads, lengths and products that the kernels index with 32 bits
tq_status shape_ok(int B, int Hq, int Hkv, int64_t T, const char* name) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || T < 0)
    return tq_fail(TQ_ERR_INVALID_ARG, "%s: bad shape B=%d Hq=%d Hkv=%d T=%lld", name, B, Hq, Hkv, (long long)T);
  if (Hq % Hkv != 0) return tq_fail(TQ_ERR_INVALID_ARG, "%s: Hq %d not a multiple of Hkv %d", name, Hq, Hkv);
  if (Hq / Hkv > 32) return tq_fail(TQ_ERR_UNSUPPORTED, "%s: Hq/Hkv = %d above 32", name, Hq / Hkv);
  if ((int64_t)B * Hq > INT_MAX) return tq_fail(TQ_ERR_UNSUPPORTED, "%s: B*Hq above INT_MAX", name);
  if (T > INT_MAX) return tq_fail(TQ_ERR_UNSUPPORTED, "%s: T above INT_MAX", name);
  return TQ_OK;
}

tq_status done(cudaError_t e, const char* name) {
  if (e == cudaSuccess) return TQ_OK;
  if (e == cudaErrorNotSupported) return tq_fail(TQ_ERR_UNSUPPORTED, "%s: the shape needs more blocks than a grid has", name);
  return tq_fail(TQ_ERR_CUDA, "%s launch: %s", name, cudaGetErrorString(e));
}

int sms_of(int device) {
  int v = 0;
  if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || v <= 0) v = 148;
  return v;
}

// chunks of a part with `units` units of n keys: about two blocks an SM in all,
// at least 64 and at most 1024 keys each
int chunks_of(int64_t units, int64_t n, int sms) {
  if (n == 0 || units == 0) return 0;
  int64_t want = (2 * (int64_t)sms + units - 1) / units;
  want = std::min<int64_t>(want, (n + 63) / 64);
  return (int)std::max<int64_t>(std::max<int64_t>(want, 1), (n + 1023) / 1024);
}

// The tensor-core kernel runs one block an SM, each with the rows of one group
// (128 / G sequences of a KV head) and an equal share of its tiles: as many
// blocks as fit in one wave, or, with more groups than SMs, the split of each
// group that wastes the least of its last wave.
tq_prefix_plan plan_of(const tq_params& kp, const tq_params& vp, int B, int Hq, int Hkv, int64_t Tp, int64_t T,
                       int sms) {
  const int G = Hq / Hkv;
  tq_prefix_plan pl = {};
  pl.tc = tq_prefix_tc_supported(kp, vp);
  if (pl.tc) {
    const int SB = 128 / G;
    const int64_t groups = (int64_t)Hkv * ((B + SB - 1) / SB);
    const int64_t tiles = (Tp + 63) / 64 + (T + 63) / 64 * std::min(B, SB);
    if (groups == 0 || tiles == 0) return pl;
    int64_t best = std::max<int64_t>(1, sms / groups);
    if (groups > sms) {
      auto waves = [&](int64_t n) { return (double)((groups * n + sms - 1) / sms) / (double)n; };
      for (int64_t n = 2; n <= 4; ++n)
        if (waves(n) < 0.95 * waves(best)) best = n;
    }
    pl.nP = (int)std::min(best, tiles);
    return pl;
  }
  pl.nP = chunks_of((int64_t)Hkv * (((int64_t)B * G + 7) / 8), Tp, sms);
  pl.nO = chunks_of((int64_t)B * Hkv * ((G + 7) / 8), T, sms);
  return pl;
}

// the prepared queries, then the partials
size_t query_bytes(const tq_params& kp, int B, int Hq, int Hkv, const tq_prefix_plan& pl, size_t* scales_at) {
  *scales_at = 0;
  if (pl.tc) return align256(tq_prefix_tc_bytes(kp, B, Hkv, Hq / Hkv, scales_at));
  return align256(sizeof(float) * (size_t)B * Hq * (kp.d + kp.m));
}

size_t prefix_bytes(const tq_params& kp, const tq_params& vp, int B, int Hq, int Hkv, const tq_prefix_plan& pl) {
  size_t at;
  return query_bytes(kp, B, Hq, Hkv, pl, &at) +
         align256(sizeof(float) * (size_t)B * Hq * (pl.nP + pl.nO) * (size_t)(vp.d + 2 + vp.m));
}

tq_status prefix_shape(const tq_codec* kc, const tq_codec* vc, int B, int Hq, int Hkv, int64_t Tp, int64_t T,
                       const char* name) {
  if (kc->p.d != vc->p.d)
    return tq_fail(TQ_ERR_INVALID_ARG, "%s: key d %d != value d %d", name, kc->p.d, vc->p.d);
  if (kc->p.d > 256) return tq_fail(TQ_ERR_UNSUPPORTED, "%s: d = %d above 256", name, kc->p.d);
  if (vc->p.m > 128)
    return tq_fail(TQ_ERR_UNSUPPORTED, "%s: QJL-corrected values need a value sketch of m <= 128", name);
  tq_status st = shape_ok(B, Hq, Hkv, T, name);
  if (st != TQ_OK) return st;
  return shape_ok(B, Hq, Hkv, Tp, name);
}

}  // namespace

extern "C" tq_status tq_attend_prefix_workspace_size(const tq_codec* kc, const tq_codec* vc, int B, int Hq, int Hkv,
                                                     int64_t Tp, int64_t T, size_t* bytes) {
  const char* name = "tq_attend_prefix_workspace_size";
  if (!kc || !vc || !bytes) return tq_fail(TQ_ERR_INVALID_ARG, "%s: null argument", name);
  tq_status st = prefix_shape(kc, vc, B, Hq, Hkv, Tp, T, name);
  if (st != TQ_OK) return st;
  const tq_prefix_plan pl = plan_of(kc->p, vc->p, B, Hq, Hkv, Tp, T, sms_of(kc->device < 0 ? 0 : kc->device));
  *bytes = prefix_bytes(kc->p, vc->p, B, Hq, Hkv, pl);
  return TQ_OK;
}

extern "C" tq_status tq_attend_prefix(const tq_codec* kc, const tq_codec* vc, const void* q, tq_dtype dt, int B, int Hq,
                                      int Hkv, float scale, int64_t Tp, const tq_compressed* Kp,
                                      const tq_compressed* Vp, int64_t T, const int32_t* lens, const tq_compressed* K,
                                      const tq_compressed* V, void* workspace, size_t ws_bytes, void* out,
                                      tq_dtype out_dtype, float* lse, void* stream) {
  const char* name = "tq_attend_prefix";
  const tqtrace::Range trace(name);
  tq_status st = codec_here(kc, name);
  if (st != TQ_OK) return st;
  if ((st = codec_here(vc, name)) != TQ_OK) return st;
  if ((st = dtype_ok(dt, name)) != TQ_OK || (st = dtype_ok(out_dtype, name)) != TQ_OK) return st;
  if ((st = prefix_shape(kc, vc, B, Hq, Hkv, Tp, T, name)) != TQ_OK) return st;
  if (!std::isfinite(scale) || scale < 0)
    return tq_fail(TQ_ERR_INVALID_ARG, "%s: scale must be finite and >= 0", name);
  if (B == 0) return TQ_OK;
  if (!aligned(q, 16)) return tq_fail(TQ_ERR_INVALID_ARG, "%s: q null or not 16-byte aligned", name);
  if (!aligned(out, 16)) return tq_fail(TQ_ERR_INVALID_ARG, "%s: out null or not 16-byte aligned", name);
  if (lse && !aligned(lse, 4)) return tq_fail(TQ_ERR_INVALID_ARG, "%s: lse not 4-byte aligned", name);
  if (lens && !aligned(lens, 4)) return tq_fail(TQ_ERR_INVALID_ARG, "%s: lens not 4-byte aligned", name);
  if (Tp > 0 && ((st = rows_ok(kc, Kp, name, "Kp")) != TQ_OK || (st = rows_ok(vc, Vp, name, "Vp")) != TQ_OK)) return st;
  if (T > 0 && ((st = rows_ok(kc, K, name, "K")) != TQ_OK || (st = rows_ok(vc, V, name, "V")) != TQ_OK)) return st;
  const tq_prefix_plan pl = plan_of(kc->p, vc->p, B, Hq, Hkv, Tp, T, sms_of(kc->device));
  const size_t need = prefix_bytes(kc->p, vc->p, B, Hq, Hkv, pl);
  if (!aligned(workspace, 16) || ws_bytes < need)
    return tq_fail(TQ_ERR_INVALID_ARG, "%s: workspace null, misaligned or smaller than %zu bytes", name, need);
  const cudaStream_t s = (cudaStream_t)stream;
  tq_prefix_args a = {};
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.Tp = Tp;
  a.T = T;
  a.lens = lens;
  if (Tp > 0) a.Kp = *Kp, a.Vp = *Vp;
  if (T > 0) a.K = *K, a.V = *V;
  a.scale_log2e = (scale == 0.0f ? kc->p.inv_sqrt_d : scale) * 1.4426950408889634f;
  size_t scales_at;
  a.q = q;
  a.dtype = dt;
  a.partials = (float*)((char*)workspace + query_bytes(kc->p, B, Hq, Hkv, pl, &scales_at));
  cudaError_t e = cudaSuccess;
  if (pl.nP + pl.nO > 0 && pl.tc) {
    a.image = (unsigned char*)workspace;
    a.scales = (float*)((char*)workspace + scales_at);
    e = tq_launch_prefix_tc(kc->p, vc->p, a, pl, s);
  } else if (pl.nP + pl.nO > 0) {
    a.qprep = (const float*)workspace;
    e = tq_launch_qprep(kc->p, q, dt, B * Hq, (float*)workspace, s);
    if (e == cudaSuccess) e = tq_launch_prefix_any(kc->p, vc->p, a, pl, s);
  }
  if (e == cudaSuccess) e = tq_launch_prefix_combine(vc->p, a, pl, out, out_dtype, lse, s);
  return done(e, name);
}

extern "C" tq_status tq_mass_update(const tq_codec* kc, const float* logits, int B, int Hq, int Hkv, int64_t T,
                                    const int32_t* lens, const float* lse, float scale, float decay, float* mass,
                                    void* stream) {
  const char* name = "tq_mass_update";
  const tqtrace::Range trace(name);
  tq_status st = codec_here(kc, name);
  if (st != TQ_OK) return st;
  if ((st = shape_ok(B, Hq, Hkv, T, name)) != TQ_OK) return st;
  if (!std::isfinite(scale) || scale < 0)
    return tq_fail(TQ_ERR_INVALID_ARG, "%s: scale must be finite and >= 0", name);
  if (!std::isfinite(decay)) return tq_fail(TQ_ERR_INVALID_ARG, "%s: decay must be finite", name);
  if (B == 0 || T == 0) return TQ_OK;
  if (!aligned(logits, 16) || !aligned(mass, 16))
    return tq_fail(TQ_ERR_INVALID_ARG, "%s: logits or mass null or not 16-byte aligned", name);
  if (lens && !aligned(lens, 4)) return tq_fail(TQ_ERR_INVALID_ARG, "%s: lens not 4-byte aligned", name);
  if (lse && !aligned(lse, 4)) return tq_fail(TQ_ERR_INVALID_ARG, "%s: lse not 4-byte aligned", name);
  return done(tq_launch_mass(kc->p, logits, B, Hq, Hkv, T, lens, lse, scale == 0.0f ? kc->p.inv_sqrt_d : scale, decay,
                             mass, (cudaStream_t)stream),
              name);
}

extern "C" tq_status tq_evict_select(const tq_codec* kc, const float* mass, int B, int Hkv, int64_t T,
                                     const int32_t* lens, int64_t keep, int64_t sink, int64_t recent, int32_t* idx,
                                     float* mass_out, int32_t* lens_out, void* stream) {
  const char* name = "tq_evict_select";
  const tqtrace::Range trace(name);
  tq_status st = codec_here(kc, name);
  if (st != TQ_OK) return st;
  if ((st = shape_ok(B, Hkv, Hkv, T, name)) != TQ_OK) return st;
  if (keep < 1 || keep > INT_MAX || sink < 0 || recent < 0 || sink > keep || recent > keep - sink)
    return tq_fail(TQ_ERR_INVALID_ARG, "%s: keep %lld, sink %lld, recent %lld (needs 1 <= keep, sink + recent <= keep)",
                   name, (long long)keep, (long long)sink, (long long)recent);
  if (B == 0) return TQ_OK;
  if (T > 0 && !aligned(mass, 16)) return tq_fail(TQ_ERR_INVALID_ARG, "%s: mass null or not 16-byte aligned", name);
  if (!aligned(idx, 16)) return tq_fail(TQ_ERR_INVALID_ARG, "%s: idx null or not 16-byte aligned", name);
  if (mass_out && !aligned(mass_out, 16)) return tq_fail(TQ_ERR_INVALID_ARG, "%s: mass_out not 16-byte aligned", name);
  if ((lens && !aligned(lens, 4)) || (lens_out && !aligned(lens_out, 4)))
    return tq_fail(TQ_ERR_INVALID_ARG, "%s: lens or lens_out not 4-byte aligned", name);
  if (mass_out && mass_out == mass) return tq_fail(TQ_ERR_INVALID_ARG, "%s: mass_out must not be mass", name);
  if (lens_out && lens_out == lens) return tq_fail(TQ_ERR_INVALID_ARG, "%s: lens_out must not be lens", name);
  return done(tq_launch_evict(kc->p, mass, B, Hkv, T, lens, keep, sink, recent, idx, mass_out, lens_out,
                              (cudaStream_t)stream),
              name);
}

extern "C" tq_status tq_copy_rows(const tq_codec* c, const tq_compressed* src, int64_t src_T, const tq_compressed* dst,
                                  int64_t dst_T, int64_t rows, int64_t n, const int32_t* src_idx,
                                  const int32_t* dst_idx, void* stream) {
  const char* name = "tq_copy_rows";
  const tqtrace::Range trace(name);
  tq_status st = codec_here(c, name);
  if (st != TQ_OK) return st;
  if (src_T < 0 || dst_T < 0 || rows < 0 || n < 0 || src_T > INT_MAX || dst_T > INT_MAX || n > INT_MAX ||
      rows > INT_MAX)
    return tq_fail(TQ_ERR_INVALID_ARG, "%s: src_T %lld, dst_T %lld, rows %lld, n %lld outside [0, INT_MAX]", name,
                   (long long)src_T, (long long)dst_T, (long long)rows, (long long)n);
  if ((!src_idx && n > src_T) || (!dst_idx && n > dst_T))
    return tq_fail(TQ_ERR_INVALID_ARG, "%s: n = %lld records without an index list, caches of %lld and %lld", name,
                   (long long)n, (long long)src_T, (long long)dst_T);
  if (rows == 0 || n == 0) return TQ_OK;
  if (src_T == 0 || dst_T == 0) return tq_fail(TQ_ERR_INVALID_ARG, "%s: an empty cache", name);
  if ((st = rows_ok(c, src, name, "src")) != TQ_OK || (st = rows_ok(c, dst, name, "dst")) != TQ_OK) return st;
  if (src->codes == dst->codes || src->norms == dst->norms)
    return tq_fail(TQ_ERR_INVALID_ARG, "%s: src and dst must be different caches", name);
  if ((src_idx && !aligned(src_idx, 4)) || (dst_idx && !aligned(dst_idx, 4)))
    return tq_fail(TQ_ERR_INVALID_ARG, "%s: an index list is not 4-byte aligned", name);
  return done(tq_launch_copy_rows(c->p, *src, src_T, *dst, dst_T, rows, n, src_idx, dst_idx, (cudaStream_t)stream),
              name);
}
