// A bounded cache: accumulated attention weight per key, the choice of the
// keys that stay, and the copy of their compressed records.
//
// Measured (B200): weights of 8 sequences, 32 heads, up to 32,768 keys (20 M
// logits) 17.5 us where reading and writing them is 4.6, bound by latency and a
// second wave of clusters; the choice of 8192 of up to 32,768 keys for 64 rows
// 36 us, bound by latency (issue slots 32% in use: reads, barriers and the three
// rounds); the copies of its records 4.0 (keys) and 4.2 TB/s (values), 1.28 times
// that in sectors.
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
// mass_t <- decay mass_t + sum_g e^(scale l_gt - lse_g), t < len; a decay of 0
// does not read the old weight, which may be anything.  The exponent
// is taken in base 2 with c = scale log2(e) in two parts (ch + cl), so that
// the product's rounding does not grow with |l|.
struct Exponent {
  float ch, cl;  // scale * log2(e)
  __device__ __forceinline__ float of(float l, float hi, float lo) const {  // l * c - (hi + lo)
    // a masked key: -inf * cl could be +inf or NaN
    return fabsf(l) == INFINITY ? l - hi : fmaf(l, cl, fmaf(l, ch, -hi) - lo);
  }
};

constexpr int kMassThreads = 512;
constexpr int kMassWarps = kMassThreads / 32;
constexpr size_t kMassSmem = 200 * 1024;  // most bytes of logits that a block keeps
constexpr int kGivenKeys = 1024;          // keys of a block when the statistics are given

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Statistics given: one pass, a thread four keys: consecutive ones by 16-byte
// loads (VEC), or, when T % 4 leaves the rows unaligned, 256 apart.
template <bool VEC>
__global__ void __launch_bounds__(256)
    mass_given_kernel(const tq_params p, const float* __restrict__ logits, const int Hq, const int Hkv, const int64_t T,
                      const int32_t* __restrict__ lens, const float* __restrict__ lse, const Exponent ex,
                      const float decay, float* __restrict__ mass) {
  __shared__ float s_hi[32], s_lo[32];
  const int64_t pieces = (T + kGivenKeys - 1) / kGivenKeys;
  const int64_t bh = blockIdx.x / pieces, t0 = blockIdx.x % pieces * kGivenKeys;
  const int h = (int)(bh % Hkv), b = (int)(bh / Hkv), G = Hq / Hkv;
  if (threadIdx.x < G) {
    // ln to log2 units, in two parts; a row without keys gives nothing, nor does
    // one whose sum is infinite: 2^(x - inf) = 0
    const double stat = (double)lse[b * Hq + h * G + threadIdx.x] * 1.4426950408889634;
    const float hi = stat == -INFINITY ? INFINITY : (float)stat;  // infinite beyond fp32 too
    s_hi[threadIdx.x] = hi;
    s_lo[threadIdx.x] = isinf(hi) ? 0.f : (float)(stat - (double)hi);
  }
  const int64_t n = held_len(lens, b, T, p.err);
  if (t0 >= n) return;
  __syncthreads();
  const float* lg = logits + ((int64_t)b * Hq + h * G) * T + t0;
  float* mr = mass + bh * T + t0;
  const int left = (int)min((int64_t)kGivenKeys, n - t0), tid = threadIdx.x;
  float add[4] = {0.f, 0.f, 0.f, 0.f};
  if (VEC && 4 * tid + 4 <= left) {
    const float4 m = decay != 0.f ? *reinterpret_cast<const float4*>(mr + 4 * tid) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int g = 0; g < G; ++g) {
      const float4 l = __ldg(reinterpret_cast<const float4*>(lg + g * T) + tid);
      add[0] += ex2(ex.of(l.x, s_hi[g], s_lo[g]));
      add[1] += ex2(ex.of(l.y, s_hi[g], s_lo[g]));
      add[2] += ex2(ex.of(l.z, s_hi[g], s_lo[g]));
      add[3] += ex2(ex.of(l.w, s_hi[g], s_lo[g]));
    }
    *reinterpret_cast<float4*>(mr + 4 * tid) = make_float4(fmaf(m.x, decay, add[0]), fmaf(m.y, decay, add[1]),
                                                           fmaf(m.z, decay, add[2]), fmaf(m.w, decay, add[3]));
    return;
  }
  const int first = VEC ? 4 * tid : tid, step = VEC ? 1 : 256;
#pragma unroll 2
  for (int g = 0; g < G; ++g) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (first + i * step < left) add[i] += ex2(ex.of(__ldg(lg + g * T + first + i * step), s_hi[g], s_lo[g]));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (first + i * step < left) mr[first + i * step] = decay != 0.f ? fmaf(mr[first + i * step], decay, add[i]) : add[i];
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
// a word in the shared memory of block `rank` of the cluster
__device__ __forceinline__ uint32_t peer_ld(const void* p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ uint4 peer_ld4(const void* p, uint32_t rank) {
  uint32_t a;
  uint4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// No statistics given: a cluster of blocks takes one (sequence, KV head), each
// an equal part of its keys, and each warp of a block one head's logits over a
// piece of that part: it fetches them into shared memory (KEEP), leaves the
// piece's maximum m and sum z = sum 2^(l - m), and 2^(l - m) in the logits'
// place.  After one exchange over the cluster the weight of a key is that
// exponential times the piece's factor 2^(m - M) / Z: the logits are read once
// and exponentiated once.  A part that does not fit is read again through the
// L2 and exponentiated twice.
template <int V, bool KEEP>
__global__ void __launch_bounds__(kMassThreads)
    mass_kernel(const tq_params p, const float* __restrict__ logits, const int Hq, const int Hkv, const int64_t T,
                const int32_t* __restrict__ lens, const Exponent ex, const float decay, float* __restrict__ mass) {
  extern __shared__ __align__(16) float keep[];
  __shared__ float s_m[32][kMassWarps], s_z[32][kMassWarps], s_f[32][kMassWarps];
  __shared__ float s_bm[32], s_bz[32], s_M[32], s_rz[32];
  const uint32_t rank = cluster_rank(), C = cluster_size();
  const int64_t bh = blockIdx.x / C;
  const int h = (int)(bh % Hkv), b = (int)(bh / Hkv), G = Hq / Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t n = held_len(lens, b, T, p.err);
  const int64_t per = ((n + C - 1) / C + 3) & ~(int64_t)3;
  const int64_t t0 = min(n, rank * per);
  const int len = (int)(min(n, t0 + per) - t0);
  const float* lg = logits + ((int64_t)b * Hq + h * G) * T + t0;
  const int nsub = G >= kMassWarps ? 1 : kMassWarps / G;         // pieces a head
  const int ps = ((len + nsub - 1) / nsub + 3) & ~3;             // keys a piece
  const int units = G * nsub;
  if constexpr (KEEP) {
    for (int u = warp; u < units; u += kMassWarps) {
      const int g = u / nsub, k0 = min(len, u % nsub * ps), k1 = min(len, k0 + ps);
      float* dst = keep + (size_t)g * per;
      const float* src = lg + g * T;
      for (int k = k0 + lane * V; k < k1; k += 32 * V) {
        if (V == 4 && k + 4 <= k1) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst + k)), "l"(src + k) : "memory");
        } else {
          for (int q = k; q < min(k1, k + V); ++q)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(dst + q)), "l"(src + q) : "memory");
        }
      }
    }
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
    __syncwarp();
  }
  for (int u = warp; u < units; u += kMassWarps) {
    const int g = u / nsub, sub = u % nsub, k0 = min(len, sub * ps), k1 = min(len, k0 + ps);
    float* row = keep + (size_t)g * per;
    const float* src = KEEP ? row : lg + g * T;
    float mx = -INFINITY, z = 0.f;
#pragma unroll 8
    for (int k = k0 + lane; k < k1; k += 32) mx = fmaxf(mx, src[k]);
    mx = tq_warp_max(mx);
    const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll 8
    for (int k = k0 + lane; k < k1; k += 32) {
      const float e = ex2((src[k] - ref) * ex.ch);
      z += e;
      if (KEEP) row[k] = e;
    }
    z = tq_warp_sum(z);
    if (lane == 0) {
      s_m[g][sub] = mx;
      s_z[g][sub] = z;
    }
  }
  __syncthreads();
  if (tid < G) {
    float mx = -INFINITY, z = 0.f;
    for (int q = 0; q < nsub; ++q) mx = fmaxf(mx, s_m[tid][q]);
    for (int q = 0; q < nsub; ++q)
      if (s_z[tid][q] != 0.f) z += s_z[tid][q] * ex2((s_m[tid][q] - mx) * ex.ch);
    s_bm[tid] = mx;
    s_bz[tid] = z;
  }
  cluster_sync();
  if (tid < G) {
    float mx = -INFINITY, z = 0.f, m[8], zr[8];
#pragma unroll
    for (uint32_t r = 0; r < 8; ++r) {
      m[r] = r < C ? __uint_as_float(peer_ld(&s_bm[tid], r)) : -INFINITY;
      zr[r] = r < C ? __uint_as_float(peer_ld(&s_bz[tid], r)) : 0.f;
      mx = fmaxf(mx, m[r]);
    }
#pragma unroll
    for (int r = 0; r < 8; ++r)
      if (zr[r] != 0.f) z += zr[r] * ex2((m[r] - mx) * ex.ch);
    s_M[tid] = mx == -INFINITY ? 0.f : mx;
    s_rz[tid] = z == 0.f ? 0.f : 1.f / z;  // all masked: nothing to add
  }
  cluster_sync();  // also: nobody leaves while its statistics may be read
  for (int u = tid; u < units; u += kMassThreads) {
    const int g = u / nsub, sub = u % nsub;
    s_f[g][sub] = s_z[g][sub] == 0.f ? 0.f : ex2((s_m[g][sub] - s_M[g]) * ex.ch) * s_rz[g];
  }
  __syncthreads();
  float* mr = mass + bh * T + t0;
  for (int k = tid * V; k < len; k += kMassThreads * V) {
    float add[V];
#pragma unroll
    for (int i = 0; i < V; ++i) add[i] = 0.f;
    const int sub = KEEP ? k / ps : 0;  // ps % 4 = 0: the V keys are of one piece
    if (V == 4 && k + 4 <= len) {
      float4 m = decay != 0.f ? *reinterpret_cast<const float4*>(mr + k) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int g = 0; g < G; ++g) {
        float4 e;
        float f;
        if constexpr (KEEP) {
          e = *reinterpret_cast<const float4*>(keep + (size_t)g * per + k);
          f = s_f[g][sub];
        } else {
          e = __ldg(reinterpret_cast<const float4*>(lg + g * T + k));
          const float M = s_M[g];
          e = make_float4(ex2((e.x - M) * ex.ch), ex2((e.y - M) * ex.ch), ex2((e.z - M) * ex.ch), ex2((e.w - M) * ex.ch));
          f = s_rz[g];
        }
        add[0] = fmaf(e.x, f, add[0]);
        add[V > 1 ? 1 : 0] = fmaf(e.y, f, add[V > 1 ? 1 : 0]);
        add[V > 2 ? 2 : 0] = fmaf(e.z, f, add[V > 2 ? 2 : 0]);
        add[V > 3 ? 3 : 0] = fmaf(e.w, f, add[V > 3 ? 3 : 0]);
      }
      m = make_float4(fmaf(m.x, decay, add[0]), fmaf(m.y, decay, add[V > 1 ? 1 : 0]),
                      fmaf(m.z, decay, add[V > 2 ? 2 : 0]), fmaf(m.w, decay, add[V > 3 ? 3 : 0]));
      *reinterpret_cast<float4*>(mr + k) = m;
    } else {
      for (int q = k; q < min(len, k + V); ++q) {
        float a = 0.f;
#pragma unroll 4
        for (int g = 0; g < G; ++g) {
          if constexpr (KEEP)
            a = fmaf(keep[(size_t)g * per + q], s_f[g][sub], a);
          else
            a = fmaf(ex2((__ldg(lg + g * T + q) - s_M[g]) * ex.ch), s_rz[g], a);
        }
        mr[q] = decay != 0.f ? fmaf(mr[q], decay, a) : a;
      }
    }
  }
}

// --------------------------------------------------------------- choice
// Order of the masses as unsigned keys: NaN below every number, -0 equal to 0.
__device__ __forceinline__ uint32_t mass_key(float v) {
  if (v != v) return 0u;
  const uint32_t u = __float_as_uint(v + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvKeep = 50 * 1024;  // most keys that a block keeps in shared memory

// sum of the first `warp` of kEvWarps counters, by one load and five shuffles
__device__ __forceinline__ int before_warp(const int* s, int warp, int lane) {
  return tq_warp_sum(lane < warp ? s[lane] : 0);
}

// A cluster of blocks: one (sequence, KV head), each block a contiguous part
// of its keys.  Sinks and recent keys get the key 2^32 - 1, which no mass has,
// so that the kept ones are the `keep` greatest of all.  A radix selection by
// eleven, eleven and ten bits finds the smallest kept key and how many of its
// equals stay (the lowest indices): every block counts its part's digits and
// sums the counters of all.  Then every warp counts what stays in its
// contiguous piece, and after one scan over warps and blocks writes it in order.
// The masses are read once and kept as ordered keys in shared memory when they
// fit (KEEP).  Bound by latency; 16-byte reads of the counters (4-byte: 54 us
// against 36) and of the keys leave fewer trips.
template <bool KEEP>
__global__ void __launch_bounds__(kEvThreads)
    evict_kernel(const tq_params p, const float* __restrict__ mass, const int Hkv, const int64_t T,
                 const int32_t* __restrict__ lens, const int64_t keep, const int64_t sink, const int64_t recent,
                 int32_t* __restrict__ idx, float* __restrict__ mass_out, int32_t* __restrict__ lens_out) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) int s_hist[3][2048];
  __shared__ int s_sum[kEvWarps], s_sure[kEvWarps], s_equal[kEvWarps], s_total[2], s_need;
  __shared__ uint32_t s_key;
  const uint32_t rank = cluster_rank(), C = cluster_size();
  const int64_t bh = blockIdx.x / C;
  const int b = (int)(bh / Hkv), h = (int)(bh % Hkv);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = (int)held_len(lens, b, T, p.err), room = (int)keep;
  int32_t* ir = idx + bh * keep;
  float* mo = mass_out ? mass_out + bh * keep : nullptr;
  const int kept = min(n, room);
  if (rank == 0 && h == 0 && tid == 0 && lens_out) lens_out[b] = kept;
  for (int64_t i = kept + (int64_t)(rank * kEvThreads + tid); i < room; i += C * kEvThreads) {
    ir[i] = -1;
    if (mo) mo[i] = 0.f;
  }
  if (n <= room) {  // for all blocks of the cluster alike
    for (int64_t i = rank * kEvThreads + tid; i < n; i += C * kEvThreads) {
      ir[i] = (int32_t)i;
      if (mo) mo[i] = mass[bh * T + i];
    }
    return;
  }
  // this block's keys: nk from key p0 on
  const int64_t part = (((int64_t)n + C - 1) / C + 31) & ~(int64_t)31;
  const int p0 = (int)min((int64_t)n, rank * part), nk = (int)min((int64_t)n - p0, part);
  const float* mr = mass + bh * T + p0;
  const int lo = (int)sink - p0, hi = n - (int)recent - p0;  // protected: below lo, from hi on
  auto make_key = [&](int i) { return i < lo || i >= hi ? 0xffffffffu : mass_key(__ldg(mr + i)); };
  if (KEEP) {
#pragma unroll 8
    for (int i = tid; i < nk; i += kEvThreads) keys[i] = make_key(i);
    if (tid < ((nk + 3) & ~3) - nk) keys[nk + tid] = 0u;  // the lowest key: the counters above it are right
  }
  for (int i = tid; i < 3 * 2048; i += kEvThreads) (&s_hist[0][0])[i] = 0;
  int need = room;
  uint32_t key = 0u;
  __syncthreads();
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, digits = pass == 2 ? 1024 : 2048;
    const uint32_t above = pass == 0 ? 0u : 0xffffffffu << (pass == 1 ? 21 : 10);
    int* hist = s_hist[pass];
    int zeros = 0;  // keys of mass 0 (never looked at) would queue at one counter: counted apart
    auto count = [&](uint32_t k) {
      if ((k & above) == key) {
        if (k == 0x80000000u)
          ++zeros;
        else
          atomicAdd(&hist[(k >> shift) & (digits - 1)], 1);
      }
    };
    if (KEEP) {
      for (int i = 4 * tid; i < nk; i += 4 * kEvThreads) {
        const uint4 k = *reinterpret_cast<const uint4*>(keys + i);
        count(k.x);
        count(k.y);
        count(k.z);
        count(k.w);
      }
    } else {
      for (int i = tid; i < nk; i += kEvThreads) count(make_key(i));
    }
    zeros = tq_warp_sum(zeros);
    if (lane == 0 && zeros) atomicAdd(&hist[(0x80000000u >> shift) & (digits - 1)], zeros);
    cluster_sync();
    // the digit where the count from the top passes `need`: a thread sums four
    // counters from the top (one 16-byte read a block), then a scan over the block
    const int top = 2047 - 4 * tid;
    int c[4] = {0, 0, 0, 0}, x = 0;
    for (uint32_t r = 0; r < C; ++r) {
      const uint4 y = peer_ld4(&hist[top - 3], r);
      c[0] += (int)y.w;
      c[1] += (int)y.z;
      c[2] += (int)y.y;
      c[3] += (int)y.x;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) x += c[q];
    const int own = x;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int y = __shfl_up_sync(TQ_FULL_MASK, x, s);
      if (lane >= s) x += y;
    }
    if (lane == 31) s_sum[warp] = x;
    __syncthreads();
    int before = before_warp(s_sum, warp, lane) + x - own;  // greater digits than this thread's
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (before < need && need <= before + c[q]) {
        s_key = key | ((uint32_t)(top - q) << shift);
        s_need = need - before;
      }
      before += c[q];
    }
    __syncthreads();
    key = s_key;
    need = s_need;
  }
  // a warp's contiguous piece: what stays for certain, and how many equal `key`
  // (of which the first `need` stay)
  const int per = ((nk + kEvWarps - 1) / kEvWarps + 31) & ~31;
  const int w0 = min(nk, warp * per), w1 = min(nk, w0 + per);
  int sure = 0, equal = 0;
#pragma unroll 4
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint32_t k = KEEP ? keys[i] : make_key(i);
    sure += k > key;
    equal += k == key;
  }
  sure = tq_warp_sum(sure);
  equal = tq_warp_sum(equal);
  if (lane == 0) {
    s_sure[warp] = sure;
    s_equal[warp] = equal;
  }
  __syncthreads();
  if (warp == 0) {
    const int a = tq_warp_sum(lane < kEvWarps ? s_sure[lane] : 0), e = tq_warp_sum(lane < kEvWarps ? s_equal[lane] : 0);
    if (lane == 0) {
      s_total[0] = a;
      s_total[1] = e;
    }
  }
  cluster_sync();
  int at = before_warp(s_sure, warp, lane), tied = before_warp(s_equal, warp, lane);
  for (uint32_t r = 0; r < rank; ++r) {
    at += (int)peer_ld(&s_total[0], r);
    tied += (int)peer_ld(&s_total[1], r);
  }
  cluster_sync();          // nobody leaves while its counters may be read
  at += min(tied, need);   // the equal ones that stay before this piece
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < w1 ? (KEEP ? keys[i] : make_key(i)) : 0u, below = (1u << lane) - 1u;
    const bool eq = i < w1 && k == key;
    const uint32_t be = __ballot_sync(TQ_FULL_MASK, eq);
    const bool stay = i < w1 && (k > key || (eq && tied + __popc(be & below) < need));
    const uint32_t bs = __ballot_sync(TQ_FULL_MASK, stay);
    if (stay) {
      const int o = at + __popc(bs & below);
      ir[o] = p0 + i;
      if (mo) mo[o] = __ldg(mr + i);
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

template <typename... P, typename... A>
cudaError_t launch_cluster(void (*fn)(P...), int64_t units, int C, int threads, size_t smem, size_t most,
                           cudaStream_t st, A... args) {
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(units * C));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, (P)args...);
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
    const int64_t grid = units * ((T + kGivenKeys - 1) / kGivenKeys);
    if (grid > 0x7fffffffll) return cudaErrorNotSupported;
    if (vec)
      mass_given_kernel<true><<<(unsigned)grid, 256, 0, st>>>(p, logits, Hq, Hkv, T, lens, lse, ex, decay, mass);
    else
      mass_given_kernel<false><<<(unsigned)grid, 256, 0, st>>>(p, logits, Hq, Hkv, T, lens, lse, ex, decay, mass);
    return cudaGetLastError();
  }
  // blocks of a cluster: about two an SM over all units, at least 512 keys each,
  // and enough of them to keep the rows in shared memory where eight can
  auto bytes = [&](int64_t C) { return sizeof(float) * (size_t)G * ((((T + C - 1) / C) + 3) & ~(int64_t)3); };
  int C = 1;
  while (C < 8 && ((units * C < 296 && T >= 1024 * C) || bytes(C) > kMassSmem)) C *= 2;
  if (units * C > 0x7fffffffll) return cudaErrorNotSupported;
  const size_t smem = bytes(C) <= kMassSmem ? bytes(C) : 0;
  auto go = [&](auto fn) {
    return launch_cluster(fn, units, C, kMassThreads, smem, kMassSmem, st, p, logits, Hq, Hkv, T, lens, ex, decay, mass);
  };
  if (smem) return vec ? go(mass_kernel<4, true>) : go(mass_kernel<1, true>);
  return vec ? go(mass_kernel<4, false>) : go(mass_kernel<1, false>);
}

cudaError_t tq_launch_evict(const tq_params& p, const float* mass, int B, int Hkv, int64_t T, const int32_t* lens,
                            int64_t keep, int64_t sink, int64_t recent, int32_t* idx, float* mass_out,
                            int32_t* lens_out, cudaStream_t st) {
  // blocks of a cluster: about two an SM over all units, at least 2048 keys
  // each, and enough of them to keep the keys in shared memory where eight can
  const int64_t units = (int64_t)B * Hkv;
  auto part = [&](int64_t C) { return ((T + C - 1) / C + 31) & ~(int64_t)31; };
  int C = 1;
  while (C < 8 && ((units * C < 148 && part(2 * C) >= 2048) || part(C) > kEvKeep)) C *= 2;
  if (units * C > 0x7fffffffll) return cudaErrorNotSupported;
  if (part(C) <= kEvKeep)
    return launch_cluster(evict_kernel<true>, units, C, kEvThreads, (size_t)part(C) * 4, kEvKeep * 4, st, p, mass, Hkv, T,
                          lens, keep, sink, recent, idx, mass_out, lens_out);
  return launch_cluster(evict_kernel<false>, units, C, kEvThreads, 0, 0, st, p, mass, Hkv, T, lens, keep, sink, recent,
                        idx, mass_out, lens_out);
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
