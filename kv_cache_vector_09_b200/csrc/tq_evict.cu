// A bounded cache: accumulated attention weight per key, the choice of the
// keys that stay, and the copy of their compressed records.
#include <math.h>

#include <algorithm>
#include <type_traits>

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
constexpr int kMassWarps = kMassThreads / 32;
constexpr size_t kMassSmem = 200 * 1024;  // most logits that a block keeps

// log2 of a row's sum of exponentials as hi + lo; a row without keys gives
// nothing: 2^(x - inf) = 0
__device__ __forceinline__ void split_stat(double stat, float& hi, float& lo) {
  hi = stat == -INFINITY ? INFINITY : (float)stat;
  lo = stat == -INFINITY ? 0.f : (float)(stat - (double)(float)stat);
}

// mass of V consecutive keys from logits at lg (heads `pitch` apart)
template <int V>
__device__ __forceinline__ void mass_add(const float* lg, int64_t pitch, int G, const Exponent& ex, const float* s_hi,
                                         const float* s_lo, float decay, float* mass) {
  float add[V], l[V], m[V];
#pragma unroll
  for (int i = 0; i < V; ++i) add[i] = 0.f;
#pragma unroll 4
  for (int g = 0; g < G; ++g) {
    if constexpr (V == 4) {
      *reinterpret_cast<float4*>(l) = *reinterpret_cast<const float4*>(lg + g * pitch);
    } else {
      l[0] = lg[g * pitch];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) add[i] += exp2f(ex.of(l[i], s_hi[g], s_lo[g]));
  }
  if constexpr (V == 4)
    *reinterpret_cast<float4*>(m) = *reinterpret_cast<const float4*>(mass);
  else
    m[0] = *mass;
#pragma unroll
  for (int i = 0; i < V; ++i) m[i] = fmaf(m[i], decay, add[i]);
  if constexpr (V == 4)
    *reinterpret_cast<float4*>(mass) = *reinterpret_cast<const float4*>(m);
  else
    *mass = m[0];
}

// Statistics given: one pass, a thread four keys (one when T % 4 leaves the
// rows unaligned), blocks over (sequence, KV head, piece of the keys).
template <int V>
__global__ void __launch_bounds__(256)
    mass_given_kernel(const tq_params p, const float* __restrict__ logits, const int Hq, const int Hkv, const int64_t T,
                      const int32_t* __restrict__ lens, const float* __restrict__ lse, const Exponent ex,
                      const float decay, float* __restrict__ mass) {
  __shared__ float s_hi[32], s_lo[32];
  const int64_t pieces = (T + 256 * V - 1) / (256 * V);
  const int64_t bh = blockIdx.x / pieces, piece = blockIdx.x % pieces;
  const int h = (int)(bh % Hkv), b = (int)(bh / Hkv), G = Hq / Hkv;
  const int64_t n = held_len(lens, b, T, p.err);
  if (piece * 256 * V >= n) return;
  if (threadIdx.x < G) split_stat((double)lse[b * Hq + h * G + threadIdx.x] * 1.4426950408889634, s_hi[threadIdx.x], s_lo[threadIdx.x]);
  __syncthreads();
  const float* lg = logits + ((int64_t)b * Hq + h * G) * T;
  float* mr = mass + bh * T;
  const int64_t t = (piece * 256 + threadIdx.x) * V;
  if (t + V <= n) {
    mass_add<V>(lg + t, T, G, ex, s_hi, s_lo, decay, mr + t);
  } else {
    for (int64_t u = t; u < n; ++u) mass_add<1>(lg + u, T, G, ex, s_hi, s_lo, decay, mr + u);
  }
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// a float in the shared memory of block `rank` of the cluster
__device__ __forceinline__ float peer_ld(const float* p, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// No statistics given: a cluster of blocks takes one (sequence, KV head), each
// an equal part of its keys.  A block brings its part of the G rows into shared
// memory once, leaves each row's maximum and sum of exponentials, and after one
// exchange over the cluster adds the weights: the logits are read once from
// memory.  A part that does not fit (KEEP false) is read again through the L2.
template <int V, bool KEEP>
__global__ void __launch_bounds__(kMassThreads)
    mass_kernel(const tq_params p, const float* __restrict__ logits, const int Hq, const int Hkv, const int64_t T,
                const int32_t* __restrict__ lens, const Exponent ex, const float decay, float* __restrict__ mass) {
  extern __shared__ __align__(16) float keep[];
  __shared__ float s_hi[32], s_lo[32], s_red[32][kMassWarps], s_m[32], s_z[32];
  const uint32_t rank = cluster_rank(), C = cluster_size();
  const int64_t bh = blockIdx.x / C;
  const int h = (int)(bh % Hkv), b = (int)(bh / Hkv), G = Hq / Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t n = held_len(lens, b, T, p.err);
  const int64_t per = ((n + C - 1) / C + 3) & ~(int64_t)3;
  const int64_t t0 = min(n, rank * per), len = min(n, t0 + per) - t0;
  const float* lg = logits + ((int64_t)b * Hq + h * G) * T + t0;
  int64_t pitch = T;
  if constexpr (KEEP) {
    pitch = per;
    const int64_t cnt = (len + V - 1) / V;  // copies a row: the last of four covers the row's end
    for (int g = 0; g < G; ++g) {
      for (int64_t i = tid; i < cnt; i += kMassThreads) {
        const uint32_t dst = (uint32_t)__cvta_generic_to_shared(keep + g * per + i * V);
        const float* src = lg + g * T + i * V;
        if (V == 4 && i * 4 + 4 <= len) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
        } else {
          for (int64_t u = i * V; u < len && u < i * V + V; ++u)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst + (uint32_t)(u - i * V) * 4), "l"(lg + g * T + u) : "memory");
        }
      }
    }
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
    lg = keep;
    __syncthreads();
  }
  for (int g = 0; g < G; ++g) {
    float mx = -INFINITY;
#pragma unroll 8
    for (int64_t t = tid; t < len; t += kMassThreads) mx = fmaxf(mx, lg[g * pitch + t]);
    mx = tq_warp_max(mx);
    if (lane == 0) s_red[g][warp] = mx;
  }
  __syncthreads();
  if (tid < G) {
    float mx = -INFINITY;
    for (int w = 0; w < kMassWarps; ++w) mx = fmaxf(mx, s_red[tid][w]);
    s_m[tid] = mx;
  }
  __syncthreads();
  for (int g = 0; g < G; ++g) {
    const float mx = s_m[g] == -INFINITY ? 0.f : s_m[g];
    float z = 0.f;
#pragma unroll 8
    for (int64_t t = tid; t < len; t += kMassThreads) z += exp2f((lg[g * pitch + t] - mx) * ex.ch);
    z = tq_warp_sum(z);
    if (lane == 0) s_red[g][warp] = z;
  }
  __syncthreads();
  if (tid < G) {
    float z = 0.f;
    for (int w = 0; w < kMassWarps; ++w) z += s_red[tid][w];
    s_z[tid] = z;
  }
  cluster_sync();
  if (tid < G) {
    float mx = -INFINITY;
    for (uint32_t r = 0; r < C; ++r) mx = fmaxf(mx, peer_ld(&s_m[tid], r));
    double z = 0.0;
    for (uint32_t r = 0; r < C; ++r) {
      const float m = peer_ld(&s_m[tid], r);
      const float zr = peer_ld(&s_z[tid], r);
      if (m != -INFINITY || zr != 0.f) z += (double)zr * exp2((double)(m - mx) * (double)ex.ch);
    }
    // all masked: nothing to add
    split_stat(mx == -INFINITY && z == 0.0 ? -INFINITY : (double)mx * ((double)ex.ch + (double)ex.cl) + log2(z), s_hi[tid], s_lo[tid]);
  }
  cluster_sync();  // nobody leaves while its statistics may be read
  float* mr = mass + bh * T + t0;
  if (V == 4) {
    for (int64_t t = (int64_t)tid * 4; t + 4 <= len; t += kMassThreads * 4)
      mass_add<4>(lg + t, pitch, G, ex, s_hi, s_lo, decay, mr + t);
    const int64_t tail = len & ~(int64_t)3;
    if (tid < len - tail) mass_add<1>(lg + tail + tid, pitch, G, ex, s_hi, s_lo, decay, mr + tail + tid);
  } else {
    for (int64_t t = tid; t < len; t += kMassThreads) mass_add<1>(lg + t, pitch, G, ex, s_hi, s_lo, decay, mr + t);
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
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvKeep = 50 * 1024;  // most keys that a block keeps in shared memory

// One block: one (sequence, KV head).  A radix selection over the keys between
// the sinks and the recent ones, eleven, eleven and ten bits, finds the
// smallest kept key and how many of its equals stay (the lowest indices); then
// every warp counts what stays in its contiguous piece, and after one scan
// over the warps writes it in order.  The masses are read once and kept as
// ordered keys in shared memory when they fit (KEEP).
template <bool KEEP>
__global__ void __launch_bounds__(kEvThreads)
    evict_kernel(const tq_params p, const float* __restrict__ mass, const int Hkv, const int64_t T,
                 const int32_t* __restrict__ lens, const int64_t keep, const int64_t sink, const int64_t recent,
                 int32_t* __restrict__ idx, float* __restrict__ mass_out, int32_t* __restrict__ lens_out) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ int s_hist[2048], s_sum[kEvWarps];
  __shared__ int64_t s_at[kEvWarps], s_tie[kEvWarps];
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
  if (KEEP) {
#pragma unroll 8
    for (int64_t t = tid; t < n; t += kEvThreads) keys[t] = mass_key(mr[t]);
  }
  auto key_of = [&](int64_t t) { return KEEP ? keys[t] : mass_key(mr[t]); };
  if (tid == 0) {
    s_key = 0u;
    s_need = (int)(keep - sink - recent);
  }
  __syncthreads();
  const bool any = s_need > 0;
  if (any) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, digits = pass == 2 ? 1024 : 2048;
      for (int i = tid; i < digits; i += kEvThreads) s_hist[i] = 0;
      __syncthreads();
      const uint32_t want = s_key, above = pass == 0 ? 0u : 0xffffffffu << (pass == 1 ? 21 : 10);
      const int need = s_need;
      for (int64_t t0 = lo; t0 < hi; t0 += kEvThreads) {
        const int64_t t = t0 + tid;
        const uint32_t k = t < hi ? key_of(t) : 0u;
        const bool in = t < hi && (k & above) == want;
        const int digit = (int)(k >> shift) & (digits - 1);
        // lanes with the first lane's digit count as one: untouched keys, all
        // of mass 0, would otherwise queue at a single counter
        const uint32_t on = __ballot_sync(TQ_FULL_MASK, in);
        if (on == 0u) continue;
        const int lead = __shfl_sync(TQ_FULL_MASK, digit, __ffs(on) - 1);
        const uint32_t same = __ballot_sync(TQ_FULL_MASK, in && digit == lead);
        if (lane == __ffs(on) - 1) atomicAdd(&s_hist[lead], __popc(same));
        if (in && digit != lead) atomicAdd(&s_hist[digit], 1);
      }
      __syncthreads();
      // the digit where the count from the top passes `need`: thread i sums
      // `digits` / 1024 counters from the top, then a scan over the block
      const int each = digits / kEvThreads, d0 = digits - 1 - tid * each;
      const int c0 = s_hist[d0], c1 = each == 2 ? s_hist[d0 - 1] : 0;
      int x = c0 + c1;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int y = __shfl_up_sync(TQ_FULL_MASK, x, s);
        if (lane >= s) x += y;
      }
      if (lane == 31) s_sum[warp] = x;
      __syncthreads();
      int base = 0;
      for (int w = 0; w < warp; ++w) base += s_sum[w];
      const int before = base + x - c0 - c1;  // greater digits than this thread's
      if (before < need && need <= before + c0) {
        s_key = want | ((uint32_t)d0 << shift);
        s_need = need - before;
      } else if (before + c0 < need && need <= before + c0 + c1) {
        s_key = want | ((uint32_t)(d0 - 1) << shift);
        s_need = need - before - c0;
      }
      __syncthreads();
    }
  }
  const uint32_t key = s_key;
  const int64_t ties = any ? s_need : 0;  // of the keys equal to `key`
  // a warp's contiguous piece: what stays for certain, and how many equal `key`
  const int64_t per = ((n + kEvWarps - 1) / kEvWarps + 31) & ~(int64_t)31;
  const int64_t w0 = min(n, warp * per), w1 = min(n, w0 + per);
  int sure = 0, equal = 0;
  for (int64_t t0 = w0; t0 < w1; t0 += 32) {
    const int64_t t = t0 + lane;
    const bool on = t < w1, mid = t >= lo && t < hi;
    const uint32_t k = on ? key_of(t) : 0u;
    sure += on && (!mid || (any && k > key));
    equal += on && mid && any && k == key;
  }
  sure = tq_warp_sum(sure);
  equal = tq_warp_sum(equal);
  if (lane == 0) {
    s_at[warp] = sure;
    s_tie[warp] = equal;
  }
  __syncthreads();
  int64_t at = 0, tied = 0;
  for (int w = 0; w < warp; ++w) {
    at += s_at[w];
    tied += s_tie[w];
  }
  at += min(tied, ties);  // the equal ones that stay before this piece
  for (int64_t t0 = w0; t0 < w1; t0 += 32) {
    const int64_t t = t0 + lane;
    const bool on = t < w1, mid = t >= lo && t < hi;
    const uint32_t k = on ? key_of(t) : 0u;
    const bool eq = on && mid && any && k == key;
    const uint32_t be = __ballot_sync(TQ_FULL_MASK, eq), below = (1u << lane) - 1u;
    const bool stay = on && (!mid || (any && (k > key || (eq && tied + __popc(be & below) < ties))));
    const uint32_t bs = __ballot_sync(TQ_FULL_MASK, stay);
    if (stay) {
      const int64_t o = at + __popc(bs & below);
      ir[o] = (int32_t)t;
      if (mo) mo[o] = mr[t];
    }
    at += __popc(bs);
    tied += __popc(be);
  }
}

// --------------------------------------------------------------- copies
// Record i of block r: source row r src_T + src_idx[r][i] to destination row
// r dst_T + dst_idx[r][i] (i itself where a list is null).  -1 skips the
// record; any other index outside its cache does too, and is recorded.
// Words of 32 records, `words` each, in units of V words: lane u of the units
// takes unit u % (words / V) of record u / (words / V), so that loads and
// stores run on along the records.
template <int V>
__device__ __forceinline__ void copy_words(uint32_t* __restrict__ dst, const uint32_t* __restrict__ src, int words,
                                           uint32_t magic, int64_t a, int64_t z, int lane) {
  using U = typename std::conditional<V == 4, uint4, typename std::conditional<V == 2, uint2, uint32_t>::type>::type;
  const int units = words / V;
#pragma unroll 4
  for (int i = 0; i < units; ++i) {
    const uint32_t u = i * 32 + lane, rec = (u * magic) >> 20, w = u - rec * units;  // rec = u / units
    const int64_t sa = __shfl_sync(TQ_FULL_MASK, a, rec), sz = __shfl_sync(TQ_FULL_MASK, z, rec);
    if (sa >= 0)
      reinterpret_cast<U*>(dst + sz * words)[w] = __ldg(reinterpret_cast<const U*>(src + sa * words) + w);
  }
}

// A warp moves 32 records at a time: a lane finds one record's places and
// moves its norms, then the warp moves the words of all 32 together.  VC, VS:
// words a lane moves at once of the codes and signs (by their rows' alignment).
template <int VC, int VS>
__global__ void __launch_bounds__(256)
    copy_rows_kernel(const tq_params p, const tq_compressed src, const int64_t src_T, const tq_compressed dst,
                     const int64_t dst_T, const int64_t total, const int64_t n, const int32_t* __restrict__ src_idx,
                     const int32_t* __restrict__ dst_idx, const uint32_t magic_c, const uint32_t magic_s) {
  const int lane = threadIdx.x & 31;
  const int64_t nw = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t i0 = ((int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * 32; i0 < total; i0 += nw * 32) {
    const int64_t i = i0 + lane;
    int64_t a = -1, z = -1;  // source and destination record, -1: none
    if (i < total) {
      const int64_t r = i / n, c = i - r * n;
      const int64_t s = src_idx ? __ldg(src_idx + i) : c, t = dst_idx ? __ldg(dst_idx + i) : c;
      if (s >= 0 && s < src_T && t >= 0 && t < dst_T) {
        a = r * src_T + s;
        z = r * dst_T + t;
        dst.norms[z] = __ldg(src.norms + a);
        if (VS) dst.rnorms[z] = __ldg(src.rnorms + a);
      } else if ((s != -1 && (s < 0 || s >= src_T)) || (t != -1 && (t < 0 || t >= dst_T))) {
        atomicMax(p.err, (uint32_t)kErrRowIndex);
      }
    }
    copy_words<VC>(dst.codes, src.codes, p.W, magic_c, a, z, lane);
    if constexpr (VS > 0) copy_words<VS>(dst.signs, src.signs, p.MS, magic_s, a, z, lane);
  }
}

template <int VC, int VS>
void launch_copy(const tq_params& p, const tq_compressed& src, int64_t src_T, const tq_compressed& dst, int64_t dst_T,
                 int64_t total, int64_t n, const int32_t* src_idx, const int32_t* dst_idx, cudaStream_t st) {
  // u / units for u < 32 units by a product: units <= 192, so 2^20 / units + 1 is exact enough
  const uint32_t mc = (1u << 20) / (uint32_t)(p.W / VC) + 1, ms = VS ? (1u << 20) / (uint32_t)(p.MS / (VS ? VS : 1)) + 1 : 0u;
  const unsigned grid = (unsigned)std::min<int64_t>((total + 255) / 256, 148 * 32);
  copy_rows_kernel<VC, VS><<<grid, 256, 0, st>>>(p, src, src_T, dst, dst_T, total, n, src_idx, dst_idx, mc, ms);
}

}  // namespace

cudaError_t tq_launch_mass(const tq_params& p, const float* logits, int B, int Hq, int Hkv, int64_t T,
                           const int32_t* lens, const float* lse, float scale, float decay, float* mass,
                           cudaStream_t st) {
  const double c = (double)scale * 1.4426950408889634;
  const Exponent ex = {(float)c, (float)(c - (double)(float)c)};
  const int64_t units = (int64_t)B * Hkv;
  const int G = Hq / Hkv;
  const bool vec = T % 4 == 0;  // every row then starts on 16 bytes
  if (lse) {
    const int64_t grid = units * ((T + (vec ? 1024 : 256) - 1) / (vec ? 1024 : 256));
    if (grid > 0x7fffffffll) return cudaErrorNotSupported;
    if (vec)
      mass_given_kernel<4><<<(unsigned)grid, 256, 0, st>>>(p, logits, Hq, Hkv, T, lens, lse, ex, decay, mass);
    else
      mass_given_kernel<1><<<(unsigned)grid, 256, 0, st>>>(p, logits, Hq, Hkv, T, lens, lse, ex, decay, mass);
    return cudaGetLastError();
  }
  // blocks of a cluster: about two an SM over all units, at least 512 keys each,
  // and enough of them to keep the rows in shared memory where eight can
  auto bytes = [&](int64_t C) { return sizeof(float) * (size_t)G * ((((T + C - 1) / C) + 3) & ~(int64_t)3); };
  int C = 1;
  while (C < 8 && ((units * C < 296 && T >= 1024 * C) || bytes(C) > kMassSmem)) C *= 2;
  if (units * C > 0x7fffffffll) return cudaErrorNotSupported;
  const size_t smem = bytes(C) <= kMassSmem ? bytes(C) : 0;
  auto go = [&](auto fn) -> cudaError_t {
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMassSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {(unsigned)C, 1, 1};
    cfg.gridDim = dim3((unsigned)(units * C));
    cfg.blockDim = dim3(kMassThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, p, logits, Hq, Hkv, T, lens, ex, decay, mass);
  };
  if (smem) return vec ? go(mass_kernel<4, true>) : go(mass_kernel<1, true>);
  return vec ? go(mass_kernel<4, false>) : go(mass_kernel<1, false>);
}

cudaError_t tq_launch_evict(const tq_params& p, const float* mass, int B, int Hkv, int64_t T, const int32_t* lens,
                            int64_t keep, int64_t sink, int64_t recent, int32_t* idx, float* mass_out,
                            int32_t* lens_out, cudaStream_t st) {
  const unsigned grid = (unsigned)(B * Hkv);
  if (T <= kEvKeep) {
    const cudaError_t e = cudaFuncSetAttribute(evict_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvKeep * 4);
    if (e != cudaSuccess) return e;
    evict_kernel<true><<<grid, kEvThreads, (size_t)T * 4, st>>>(p, mass, Hkv, T, lens, keep, sink, recent, idx, mass_out, lens_out);
  } else {
    evict_kernel<false><<<grid, kEvThreads, 0, st>>>(p, mass, Hkv, T, lens, keep, sink, recent, idx, mass_out, lens_out);
  }
  return cudaGetLastError();
}

cudaError_t tq_launch_copy_rows(const tq_params& p, const tq_compressed& src, int64_t src_T, const tq_compressed& dst,
                                int64_t dst_T, int64_t rows, int64_t n, const int32_t* src_idx,
                                const int32_t* dst_idx, cudaStream_t st) {
  const int64_t total = rows * n;
#define GO(VC) \
  if (p.MS == 0) launch_copy<VC, 0>(p, src, src_T, dst, dst_T, total, n, src_idx, dst_idx, st); \
  else if (p.MS % 4 == 0) launch_copy<VC, 4>(p, src, src_T, dst, dst_T, total, n, src_idx, dst_idx, st); \
  else if (p.MS % 2 == 0) launch_copy<VC, 2>(p, src, src_T, dst, dst_T, total, n, src_idx, dst_idx, st); \
  else launch_copy<VC, 1>(p, src, src_T, dst, dst_T, total, n, src_idx, dst_idx, st)
  if (p.W % 4 == 0) {
    GO(4);
  } else if (p.W % 2 == 0) {
    GO(2);
  } else {
    GO(1);
  }
#undef GO
  return cudaGetLastError();
}
