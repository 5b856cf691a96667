// Decode attention over a prefix that the batch shares and ragged keys that
// each sequence owns.
//
// For query row (b, h) of KV head k = h / G the context is the prefix keys
// (k, t), t < Tp, and the sequence's own keys (b, k, t), t < len_b.  With
//   l_x = scale * nu_x (<q', cen[code_x]> / sqrt(d) + gamma_x sqrt(pi/2)/m <S q', s_x>)
// a chunk C of either part leaves M = max l_x, Z = sum 2^(l_x - M) (logits in
// log2 units) and A = sum 2^(l_x - M) v_x in the rotated space; softmax over
// the union is the merge
//   M* = max M_C,  out = Pi_v^T (sum 2^(M_C - M*) A_C) / (sum 2^(M_C - M*) Z_C),
// so a prefix key is read once for the whole batch, not once a sequence.
//
// This file holds the kernel for every codec (CUDA cores, eight query rows a
// block) and the merge.
#include <math.h>

#include <algorithm>

#include "tq_cache.h"
#include "tq_common.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kNG = 8;           // query rows of a block
// most dynamic shared memory of a block: d <= 256, m <= 1024, chunks of <= 1024
// keys.  The limit is set to it, the same for every call: the attribute is the
// process's, and one thread's launch may come between another's two steps
constexpr int kMostSmem = (int)sizeof(float) * kNG * (256 + 1024 + 1024);

// length of sequence b's own context, clamped to [0, T]; an entry outside is
// recorded in the codec's error word
__device__ __forceinline__ int64_t own_len(const int32_t* lens, int b, int64_t T, uint32_t* err) {
  if (!lens) return T;
  const int64_t n = __ldg(lens + b);
  if (n < 0 || n > T) {
    atomicMax(err, (uint32_t)kErrLength);
    return n < 0 ? 0 : T;
  }
  return n;
}

// code of coordinate i of a packed row and its reconstruction (z units)
__device__ __forceinline__ float decode(const tq_params& p, const uint32_t* __restrict__ cw, int i) {
  if (p.vq_bits) {
    const int j = i >> 1, w = j >> 5, bit = j & 31;
    int c = 0;
    for (int b = 0; b < p.vq_bits; ++b) c |= ((__ldg(cw + b * p.vq_pw + w) >> bit) & 1) << b;
    return __ldg(p.vq_cb + 2 * c + (i & 1));
  }
  const int s = i >= p.seg_len ? 1 : 0;
  const int il = i - s * p.seg_len, w = il >> 5, bit = il & 31;
  int c = 0;
  for (int b = 0; b < p.bits[s]; ++b) c |= ((__ldg(cw + p.segbase[s] + b * p.pw + w) >> bit) & 1) << b;
  return p.cen[s][c];
}

// One block: eight query rows of one unit against one chunk of its keys.
__global__ void __launch_bounds__(kThreads)
    prefix_any_kernel(const tq_params kp, const tq_params vp, const tq_prefix_args a, const int nP, const int nO,
                      const int subP, const int subO) {
  extern __shared__ __align__(16) float smem[];
  __shared__ float red[kWarps][kNG];
  __shared__ float s_max[kNG], s_sum[kNG];
  __shared__ int s_row[kNG];  // query row b * Hq + h of each of the block's rows, -1: none
  const int d = kp.d, m = kp.m, vm = vp.m;
  float* qs = smem;                    // [d + m][kNG]
  float* L = qs + (size_t)(d + m) * kNG;  // [chunk][kNG]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // which unit, rows and chunk
  int64_t blk = blockIdx.x;
  const int64_t nblkP = (int64_t)a.Hkv * subP * nP;
  const bool pre = blk < nblkP;
  int h, b = 0, sub, chunk, slot;
  int64_t n, base;
  tq_compressed K, V;
  if (pre) {
    chunk = (int)(blk % nP);
    sub = (int)(blk / nP % subP);
    h = (int)(blk / nP / subP);
    slot = chunk;
    n = a.Tp;
    base = (int64_t)h * a.Tp;
    K = a.Kp;
    V = a.Vp;
  } else {
    blk -= nblkP;
    chunk = (int)(blk % nO);
    sub = (int)(blk / nO % subO);
    h = (int)(blk / nO / subO % a.Hkv);
    b = (int)(blk / nO / subO / a.Hkv);
    slot = nP + chunk;
    n = own_len(a.lens, b, a.T, kp.err);
    base = ((int64_t)b * a.Hkv + h) * a.T;
    K = a.K;
    V = a.V;
  }
  const int64_t per = (n + (pre ? nP : nO) - 1) / (pre ? nP : nO);
  const int64_t t0 = min(n, chunk * per), t1 = min(n, t0 + per);
  if (tid < kNG) {
    int row = -1;
    const int r = sub * kNG + tid;
    if (pre) {
      if (r < a.B * a.G) row = (r / a.G) * a.Hq + h * a.G + r % a.G;
    } else if (r < a.G) {
      row = b * a.Hq + h * a.G + r;
    }
    s_row[tid] = row;
  }
  __syncthreads();
  for (int idx = tid; idx < (d + m) * kNG; idx += kThreads) {
    const int g = idx / (d + m), i = idx % (d + m);
    qs[i * kNG + g] = s_row[g] >= 0 ? a.qprep[(size_t)s_row[g] * (d + m) + i] * (i < d ? kp.inv_sqrt_d : 1.f) : 0.f;
  }
  __syncthreads();

  // logits in log2 units
  float lmax[kNG];
#pragma unroll
  for (int g = 0; g < kNG; ++g) lmax[g] = -INFINITY;
  for (int64_t t = t0 + tid; t < t1; t += kThreads) {
    const int64_t row = base + t;
    float acc[kNG], acq[kNG];
#pragma unroll
    for (int g = 0; g < kNG; ++g) acc[g] = acq[g] = 0.f;
    const uint32_t* cw = K.codes + row * kp.W;
    for (int i = 0; i < d; ++i) {
      const float c = decode(kp, cw, i);
#pragma unroll
      for (int g = 0; g < kNG; ++g) acc[g] = fmaf(c, qs[i * kNG + g], acc[g]);
    }
    float cq = 0.f;
    if (m > 0) {
      for (int j = 0; j < m; ++j) {
        const uint32_t neg = (~__ldg(K.signs + row * kp.MS + (j >> 5)) >> (j & 31) & 1u) << 31;
#pragma unroll
        for (int g = 0; g < kNG; ++g)
          acq[g] += __uint_as_float(__float_as_uint(qs[(d + j) * kNG + g]) ^ neg);
      }
      cq = __ldg(K.rnorms + row) * kp.qjl_coef;
    }
    const float nu = __ldg(K.norms + row);
#pragma unroll
    for (int g = 0; g < kNG; ++g) {
      const float l = nu * fmaf(cq, acq[g], acc[g]) * a.scale_log2e;
      L[(t - t0) * kNG + g] = l;
      lmax[g] = fmaxf(lmax[g], l);
    }
  }
#pragma unroll
  for (int g = 0; g < kNG; ++g) {
    const float v = tq_warp_max(lmax[g]);
    if (lane == 0) red[warp][g] = v;
  }
  __syncthreads();
  if (tid < kNG) {
    float v = -INFINITY;
    for (int w = 0; w < kWarps; ++w) v = fmaxf(v, red[w][tid]);
    s_max[tid] = v;
  }
  __syncthreads();
  // exponentials; L becomes 2^(l - M) nu_v
  float lsum[kNG];
#pragma unroll
  for (int g = 0; g < kNG; ++g) lsum[g] = 0.f;
  for (int64_t t = t0 + tid; t < t1; t += kThreads) {
    const float nv = __ldg(V.norms + base + t);
#pragma unroll
    for (int g = 0; g < kNG; ++g) {
      const float e = exp2f(L[(t - t0) * kNG + g] - (s_max[g] == -INFINITY ? 0.f : s_max[g]));
      lsum[g] += e;
      L[(t - t0) * kNG + g] = e * nv;
    }
  }
#pragma unroll
  for (int g = 0; g < kNG; ++g) {
    const float v = tq_warp_sum(lsum[g]);
    if (lane == 0) red[warp][g] = v;
  }
  __syncthreads();
  if (tid < kNG) {
    float v = 0.f;
    for (int w = 0; w < kWarps; ++w) v += red[w][tid];
    s_sum[tid] = v;
  }
  __syncthreads();
  // values: thread i < d a coordinate, then thread j < m_v a sketch entry
  const int nslot = nP + nO, ps = d + 2 + vm;
  for (int i = tid; i < d + vm; i += kThreads) {
    float acc[kNG];
#pragma unroll
    for (int g = 0; g < kNG; ++g) acc[g] = 0.f;
    for (int64_t t = t0; t < t1; ++t) {
      float v;
      if (i < d) {
        v = decode(vp, V.codes + (base + t) * vp.W, i) * vp.inv_sqrt_d;
      } else {
        const int j = i - d;
        v = __ldg(V.rnorms + base + t);
        if (!((__ldg(V.signs + (base + t) * vp.MS + (j >> 5)) >> (j & 31)) & 1u)) v = -v;
      }
#pragma unroll
      for (int g = 0; g < kNG; ++g) acc[g] = fmaf(L[(t - t0) * kNG + g], v, acc[g]);
    }
#pragma unroll
    for (int g = 0; g < kNG; ++g) {
      if (s_row[g] < 0) continue;
      float* pr = a.partials + ((size_t)s_row[g] * nslot + slot) * ps;
      pr[i < d ? i : i + 2] = acc[g];
      if (i == 0) {
        pr[d] = s_max[g];
        pr[d + 1] = s_sum[g];
      }
    }
  }
}

__device__ __forceinline__ void put(float* o, float v) { *o = v; }
__device__ __forceinline__ void put(__nv_bfloat16* o, float v) { *o = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* o, float v) { *o = __float2half_rn(v); }

// Merge of one query row's partials: the block's warps take chunks in turn,
// four at a time so that their loads overlap, each with its own maximum; warp 0
// merges the warps' sums in order, applies the values' QJL term and the inverse
// rotation, and writes the row in its type.  Launched as a programmatic
// dependent of the attention kernel.
template <int VPL, typename TOut>
__global__ void __launch_bounds__(kThreads)
    prefix_combine_kernel(const tq_params vp, const float* __restrict__ partials, const int nslot,
                          TOut* __restrict__ out, float* __restrict__ lse) {
  constexpr int d = 32 * VPL, kBatch = 4;
  __shared__ float s_acc[kWarps][d], s_as[kWarps][128], s_den[kWarps], s_m[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x, vm = vp.m, ps = d + 2 + vm;
  const float* pr = partials + (size_t)row * nslot * ps;
  float acc[VPL], as[4] = {0.f, 0.f, 0.f, 0.f}, den = 0.f, M = -INFINITY;
#pragma unroll
  for (int k = 0; k < VPL; ++k) acc[k] = 0.f;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int c0 = warp; c0 < nslot; c0 += kBatch * kWarps) {
    float m[kBatch], z[kBatch], x[kBatch][VPL];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int c = c0 + u * kWarps;
      const bool on = c < nslot;
      const float* pc = pr + (size_t)(on ? c : c0) * ps;
      m[u] = on ? pc[d] : -INFINITY;
      z[u] = on ? pc[d + 1] : 0.f;
#pragma unroll
      for (int k = 0; k < VPL; ++k) x[u][k] = pc[lane + 32 * k];
    }
    float top = M;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) top = fmaxf(top, m[u]);
    const float ref = top == -INFINITY ? 0.f : top, old = exp2f(M - ref);
    den *= old;
#pragma unroll
    for (int k = 0; k < VPL; ++k) acc[k] *= old;
#pragma unroll
    for (int u = 0; u < 4; ++u) as[u] *= old;
    M = top;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (z[u] == 0.f) continue;  // an empty chunk: nothing of it but z and the maximum is defined
      const float w = exp2f(m[u] - ref);
      den = fmaf(z[u], w, den);
#pragma unroll
      for (int k = 0; k < VPL; ++k) acc[k] = fmaf(x[u][k], w, acc[k]);
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (32 * v < vm) as[v] = fmaf(pr[(size_t)(c0 + u * kWarps) * ps + d + 2 + lane + 32 * v], w, as[v]);
    }
  }
#pragma unroll
  for (int k = 0; k < VPL; ++k) s_acc[warp][lane + 32 * k] = acc[k];
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (32 * u < vm) s_as[warp][lane + 32 * u] = as[u];
  if (lane == 0) {
    s_den[warp] = den;
    s_m[warp] = M;
  }
  __syncthreads();
  if (warp != 0) return;
  M = s_m[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
  const float ref = M == -INFINITY ? 0.f : M;
  den = 0.f;
#pragma unroll
  for (int k = 0; k < VPL; ++k) acc[k] = 0.f;
#pragma unroll
  for (int u = 0; u < 4; ++u) as[u] = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float f = exp2f(s_m[w] - ref);  // 0 for a warp without keys, whose sums are 0 too
    den = fmaf(s_den[w], f, den);
#pragma unroll
    for (int k = 0; k < VPL; ++k) acc[k] = fmaf(s_acc[w][lane + 32 * k], f, acc[k]);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (32 * u < vm) as[u] = fmaf(s_as[w][lane + 32 * u], f, as[u]);
  }
  if (lse && lane == 0) lse[row] = (ref + log2f(den)) * 0.693147180559945309f;
  const float inv = den == 0.f ? 0.f : 1.0f / den;  // a row without keys: zeros
#pragma unroll
  for (int k = 0; k < VPL; ++k) acc[k] *= inv;
  for (int j = 0; j < vm; ++j) {
    float aj = 0.f;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (u == (j >> 5)) aj = __shfl_sync(TQ_FULL_MASK, as[u], j & 31);
    aj *= inv * vp.qjl_coef;
    const float* Sj = vp.S + (size_t)j * d;
#pragma unroll
    for (int k = 0; k < VPL; ++k) acc[k] = fmaf(__ldg(Sj + lane + 32 * k), aj, acc[k]);
  }
  TOut* o = out + (size_t)row * d;
  if (vp.haar) {
    float y[VPL];
#pragma unroll
    for (int k = 0; k < VPL; ++k) y[k] = 0.f;
    for (int j = 0; j < d; ++j) {
      float aj = 0.f;
#pragma unroll
      for (int k = 0; k < VPL; ++k)
        if (k == (j >> 5)) aj = __shfl_sync(TQ_FULL_MASK, acc[k], j & 31);
#pragma unroll
      for (int k = 0; k < VPL; ++k) y[k] = fmaf(__ldg(vp.piT + (size_t)(lane + 32 * k) * d + j), aj, y[k]);
    }
#pragma unroll
    for (int k = 0; k < VPL; ++k) put(o + lane + 32 * k, y[k]);
    return;
  }
  tq_fwht_warp<VPL>(acc, lane);
#pragma unroll
  for (int k = 0; k < VPL; ++k) {
    const float v = acc[k] * vp.inv_sqrt_p;
    put(o + lane + 32 * k, tq_dneg(vp.dbits, k, lane) ? -v : v);
  }
}

template <int VPL, typename TOut>
cudaError_t launch_combine_t(const tq_params& vp, const tq_prefix_args& a, int nslot, void* out, float* lse,
                             cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(a.B * a.Hq));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_combine_kernel<VPL, TOut>, vp, (const float*)a.partials, nslot, (TOut*)out, lse);
}

template <int VPL>
cudaError_t launch_combine(const tq_params& vp, const tq_prefix_args& a, int nslot, void* out, tq_dtype dt, float* lse,
                           cudaStream_t st) {
  switch (dt) {
    case TQ_F32: return launch_combine_t<VPL, float>(vp, a, nslot, out, lse, st);
    case TQ_BF16: return launch_combine_t<VPL, __nv_bfloat16>(vp, a, nslot, out, lse, st);
    default: return launch_combine_t<VPL, __half>(vp, a, nslot, out, lse, st);
  }
}

}  // namespace

cudaError_t tq_launch_prefix_any(const tq_params& kp, const tq_params& vp, const tq_prefix_args& a,
                                 const tq_prefix_plan& plan, cudaStream_t st) {
  const int subP = (int)(((int64_t)a.B * a.G + kNG - 1) / kNG), subO = (a.G + kNG - 1) / kNG;
  const int64_t grid = (int64_t)a.Hkv * subP * plan.nP + (int64_t)a.B * a.Hkv * subO * plan.nO;
  if (grid == 0) return cudaSuccess;
  if (grid > 0x7fffffffll) return cudaErrorNotSupported;
  int64_t per = 0;
  if (plan.nP) per = std::max<int64_t>(per, (a.Tp + plan.nP - 1) / plan.nP);
  if (plan.nO) per = std::max<int64_t>(per, (a.T + plan.nO - 1) / plan.nO);
  const size_t smem = sizeof(float) * (size_t)kNG * (kp.d + kp.m + per);
  if (smem > (size_t)kMostSmem) return cudaErrorInvalidConfiguration;
  const cudaError_t e = cudaFuncSetAttribute(prefix_any_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
  if (e != cudaSuccess) return e;
  prefix_any_kernel<<<(unsigned)grid, kThreads, smem, st>>>(kp, vp, a, plan.nP, plan.nO, subP, subO);
  return cudaGetLastError();
}

cudaError_t tq_launch_prefix_combine(const tq_params& vp, const tq_prefix_args& a, const tq_prefix_plan& plan,
                                     void* out, tq_dtype dt, float* lse, cudaStream_t st) {
  const int nslot = plan.nP + plan.nO;
  switch (vp.d) {
    case 64: return launch_combine<2>(vp, a, nslot, out, dt, lse, st);
    case 128: return launch_combine<4>(vp, a, nslot, out, dt, lse, st);
    case 256: return launch_combine<8>(vp, a, nslot, out, dt, lse, st);
    default: return cudaErrorNotSupported;
  }
}
