// A bounded cache: accumulated attention weight per key, the choice of the
// keys that stay, and the copy of their compressed records.
#include <math.h>

#include <algorithm>

#include "tq_cache.h"
#include "tq_common.cuh"

namespace {

__device__ __forceinline__ int64_t held_len(const int32_t* lens, int b, int64_t T, uint32_t* err) {
  if (!lens) return T;
  const int64_t n = __ldg(lens + b);
  if (n < 0 || n > T) {
    atomicMax(err, (uint32_t)kErrLength);
    return n < 0 ? 0 : T;
  }
  return n;
}

// ---------------------------------------------------------------- mass
// mass_t <- decay mass_t + sum_g e^(scale l_gt - lse_g), t < len.  The exponent
// is taken in base 2 with c = scale log2(e) in two parts (ch + cl), so that
// the product's rounding does not grow with |l|.
struct Exponent {
  float ch, cl;  // scale * log2(e)
  __device__ __forceinline__ float of(float l, float hi, float lo) const {  // l * c - (hi + lo)
    l = l == -INFINITY ? -3.4028235e38f : l;  // a masked key: -inf * cl could be +inf or NaN
    return fmaf(l, cl, fmaf(l, ch, -hi) - lo);
  }
};

constexpr int kMassThreads = 512;

__global__ void __launch_bounds__(kMassThreads)
    mass_kernel(const tq_params p, const float* __restrict__ logits, const int Hq, const int Hkv, const int64_t T,
                const int32_t* __restrict__ lens, const float* __restrict__ lse, const Exponent ex, const float decay,
                float* __restrict__ mass) {
  __shared__ float s_hi[32], s_lo[32], s_red[kMassThreads / 32];
  const int h = blockIdx.x % Hkv, b = blockIdx.x / Hkv, G = Hq / Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t n = held_len(lens, b, T, p.err);
  const float* lg = logits + ((int64_t)b * Hq + h * G) * T;
  for (int g = 0; g < G; ++g) {
    double stat;  // log2 of the row's sum of exponentials
    if (lse) {
      stat = (double)lse[b * Hq + h * G + g] * 1.4426950408889634;
    } else {
      float mx = -INFINITY;
      for (int64_t t = tid; t < n; t += kMassThreads) mx = fmaxf(mx, lg[g * T + t]);
      mx = tq_warp_max(mx);
      __syncthreads();
      if (lane == 0) s_red[warp] = mx;
      __syncthreads();
      mx = -INFINITY;
      for (int w = 0; w < kMassThreads / 32; ++w) mx = fmaxf(mx, s_red[w]);
      float z = 0.f;
      for (int64_t t = tid; t < n; t += kMassThreads) z += exp2f((lg[g * T + t] - mx) * ex.ch);
      z = tq_warp_sum(z);
      __syncthreads();
      if (lane == 0) s_red[warp] = z;
      __syncthreads();
      z = 0.f;
      for (int w = 0; w < kMassThreads / 32; ++w) z += s_red[w];
      stat = mx == -INFINITY ? -INFINITY : (double)mx * ((double)ex.ch + (double)ex.cl) + log2((double)z);
    }
    if (tid == 0) {
      // a row without keys gives nothing: 2^(x - inf) = 0
      s_hi[g] = stat == -INFINITY ? INFINITY : (float)stat;
      s_lo[g] = stat == -INFINITY ? 0.f : (float)(stat - (double)(float)stat);
    }
  }
  __syncthreads();
  float* mr = mass + ((int64_t)b * Hkv + h) * T;
  for (int64_t t = tid; t < n; t += kMassThreads) {
    float add = 0.f;
    for (int g = 0; g < G; ++g) add += exp2f(ex.of(lg[g * T + t], s_hi[g], s_lo[g]));
    mr[t] = fmaf(mr[t], decay, add);
  }
}

// --------------------------------------------------------------- choice
// Order of the masses as unsigned keys: NaN below every number, -0 equal to 0.
__device__ __forceinline__ uint32_t mass_key(float v) {
  if (v != v) return 0u;
  const uint32_t u = __float_as_uint(v + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

constexpr int kEvThreads = 1024;

// One block: one (sequence, KV head).  A radix selection over the keys between
// the sinks and the recent ones finds the smallest kept key and how many of
// its equals stay (the lowest indices); an ordered pass writes the indices.
__global__ void __launch_bounds__(kEvThreads)
    evict_kernel(const tq_params p, const float* __restrict__ mass, const int Hkv, const int64_t T,
                 const int32_t* __restrict__ lens, const int64_t keep, const int64_t sink, const int64_t recent,
                 int32_t* __restrict__ idx, float* __restrict__ mass_out, int32_t* __restrict__ lens_out) {
  __shared__ int s_hist[256];
  __shared__ int s_w[32][2];
  __shared__ uint32_t s_key;
  __shared__ int s_need;
  const int b = blockIdx.x / Hkv, h = blockIdx.x % Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t n = held_len(lens, b, T, p.err);
  const float* mr = mass + (int64_t)blockIdx.x * T;
  int32_t* ir = idx + (int64_t)blockIdx.x * keep;
  float* mo = mass_out ? mass_out + (int64_t)blockIdx.x * keep : nullptr;
  const int64_t kept = n < keep ? n : keep;
  if (h == 0 && tid == 0 && lens_out) lens_out[b] = (int32_t)kept;
  for (int64_t i = kept + tid; i < keep; i += kEvThreads) {
    ir[i] = -1;
    if (mo) mo[i] = 0.f;
  }
  if (n <= keep) {
    for (int64_t i = tid; i < n; i += kEvThreads) {
      ir[i] = (int32_t)i;
      if (mo) mo[i] = mr[i];
    }
    return;
  }
  const int64_t lo = sink, hi = n - recent;  // the keys to choose from: more than `need` of them
  if (tid == 0) {
    s_key = 0u;
    s_need = (int)(keep - sink - recent);
  }
  __syncthreads();
  const bool any = s_need > 0;
  if (any) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) s_hist[tid] = 0;
      __syncthreads();
      const uint32_t want = s_key;
      for (int64_t t = lo + tid; t < hi; t += kEvThreads) {
        const uint32_t k = mass_key(mr[t]);
        if (shift == 24 || (k >> (shift + 8)) == (want >> (shift + 8))) atomicAdd(&s_hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int need = s_need, bin = 255;
        while (need > s_hist[bin]) need -= s_hist[bin--];
        s_need = need;
        s_key = want | ((uint32_t)bin << shift);
      }
      __syncthreads();
    }
  }
  const uint32_t key = s_key;
  const int ties = any ? s_need : 0;  // of the keys equal to `key`
  int64_t at = 0;
  int tied = 0;
  for (int64_t t0 = 0; t0 < n; t0 += kEvThreads) {
    const int64_t t = t0 + tid;
    const float v = t < n ? mr[t] : 0.f;
    const bool mid = t >= lo && t < hi;
    const uint32_t k = mass_key(v);
    const bool eq = t < n && mid && any && k == key;
    const uint32_t be = __ballot_sync(TQ_FULL_MASK, eq);
    if (lane == 0) s_w[warp][0] = __popc(be);
    __syncthreads();
    int e0 = tied, e1 = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) e0 += s_w[w][0];
      e1 += s_w[w][0];
    }
    const int rank = e0 + __popc(be & ((1u << lane) - 1u));
    const bool stay = t < n && (!mid || (any && (k > key || (eq && rank < ties))));
    const uint32_t bs = __ballot_sync(TQ_FULL_MASK, stay);
    if (lane == 0) s_w[warp][1] = __popc(bs);
    __syncthreads();
    int64_t c0 = at;
    int c1 = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) c0 += s_w[w][1];
      c1 += s_w[w][1];
    }
    if (stay) {
      const int64_t o = c0 + __popc(bs & ((1u << lane) - 1u));
      ir[o] = (int32_t)t;
      if (mo) mo[o] = v;
    }
    at += c1;
    tied += e1;
  }
}

// --------------------------------------------------------------- copies
// Record i of block r: source row r src_T + src_idx[r][i] to destination row
// r dst_T + dst_idx[r][i] (i itself where a list is null).  -1 skips the
// record; any other index outside its cache does too, and is recorded.
__global__ void __launch_bounds__(256)
    copy_rows_kernel(const tq_params p, const tq_compressed src, const int64_t src_T, const tq_compressed dst,
                     const int64_t dst_T, const int64_t total, const int64_t n, const int32_t* __restrict__ src_idx,
                     const int32_t* __restrict__ dst_idx) {
  const int lane = threadIdx.x & 31;
  const int64_t nw = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i < total; i += nw) {
    const int64_t r = i / n, c = i - r * n;
    const int64_t s = src_idx ? __ldg(src_idx + i) : c, t = dst_idx ? __ldg(dst_idx + i) : c;
    if (s < 0 || s >= src_T || t < 0 || t >= dst_T) {
      if (((s != -1 && (s < 0 || s >= src_T)) || (t != -1 && (t < 0 || t >= dst_T))) && lane == 0)
        atomicMax(p.err, (uint32_t)kErrRowIndex);
      continue;
    }
    const int64_t a = r * src_T + s, z = r * dst_T + t;
    for (int w = lane; w < p.W; w += 32) dst.codes[z * p.W + w] = __ldg(src.codes + a * p.W + w);
    for (int w = lane; w < p.MS; w += 32) dst.signs[z * p.MS + w] = __ldg(src.signs + a * p.MS + w);
    if (lane == 0) dst.norms[z] = __ldg(src.norms + a);
    if (lane == 1 && p.m > 0) dst.rnorms[z] = __ldg(src.rnorms + a);
  }
}

}  // namespace

cudaError_t tq_launch_mass(const tq_params& p, const float* logits, int B, int Hq, int Hkv, int64_t T,
                           const int32_t* lens, const float* lse, float scale, float decay, float* mass,
                           cudaStream_t st) {
  const double c = (double)scale * 1.4426950408889634;
  const Exponent ex = {(float)c, (float)(c - (double)(float)c)};
  mass_kernel<<<(unsigned)(B * Hkv), kMassThreads, 0, st>>>(p, logits, Hq, Hkv, T, lens, lse, ex, decay, mass);
  return cudaGetLastError();
}

cudaError_t tq_launch_evict(const tq_params& p, const float* mass, int B, int Hkv, int64_t T, const int32_t* lens,
                            int64_t keep, int64_t sink, int64_t recent, int32_t* idx, float* mass_out,
                            int32_t* lens_out, cudaStream_t st) {
  evict_kernel<<<(unsigned)(B * Hkv), kEvThreads, 0, st>>>(p, mass, Hkv, T, lens, keep, sink, recent, idx, mass_out,
                                                           lens_out);
  return cudaGetLastError();
}

cudaError_t tq_launch_copy_rows(const tq_params& p, const tq_compressed& src, int64_t src_T, const tq_compressed& dst,
                                int64_t dst_T, int64_t rows, int64_t n, const int32_t* src_idx,
                                const int32_t* dst_idx, cudaStream_t st) {
  const int64_t total = rows * n;
  const unsigned grid = (unsigned)std::min<int64_t>((total + 7) / 8, 148 * 16);
  copy_rows_kernel<<<grid, 256, 0, st>>>(p, src, src_T, dst, dst_T, total, n, src_idx, dst_idx);
  return cudaGetLastError();
}
