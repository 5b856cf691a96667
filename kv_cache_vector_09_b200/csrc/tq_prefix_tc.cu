// Shared-prefix decode attention on the tensor cores (kind::f16 tcgen05.mma),
// for scalar codes at d = 64 and 128, key sketches of m <= 128 and values
// without a sketch.
//
// The rows of a block are the query heads of one KV head over SB = 128 / G
// sequences: SB * G rows of an M = 128 tile.  Their keys are a list of tiles
// of 64: the prefix's tiles, which serve every row, then each sequence's own,
// which serve its G rows.  The list is cut into equal ranges, one per block;
// a block keeps its queries, walks its range, carries for each row the running
// maximum M, Z = sum 2^(l - M) and acc = sum 2^(l - M) v of the tiles that
// serve it, and leaves one partial per row.  A prefix key is so decoded once
// for 128 rows instead of once a query.
//
// Per tile, with c the centroids, s the signs, w = S q':
//   S = q' c^T (64 columns) and R = w s^T (64 more) into TMEM,
//   l = a_k S + b_k R,  a_k = nu scale log2(e) / sqrt(d), b_k = nu gamma coef scale log2(e)
//   P = 2^(l - M) nu_v 2^(14 - e) as fp16, back into TMEM over S,
//   O = P c_v into TMEM, added into acc in registers with the weight 2^(e - 14).
// 2^e bounds the tile's value norms, so that P uses fp16's range whatever the
// norms; its parts end at fp16's 2^-24, so a weighted norm is good to 2^-37 of
// the tile's largest norm where that is more than 2^-22 of itself (a scale by
// the row's largest product would need its maximum exchanged too).  O starts from zero each tile, so that the tensor core's truncating
// accumulation only ever spans one tile.
//
// Operands are two fp16 parts each (x = hi + lo, 2^-22 relative) and a product
// the three that matter, hi hi + hi lo + lo hi, the small ones first, whatever
// the result's type: one part (2^-11) would move a logit by its size times
// 2^-11, and a weight by e to that, which at logits of 100 is twice a bf16
// result's half step (32 sequences over 32,768 keys: 0.119 ms with one part,
// 0.136 with two).
//
// Operand bytes come from byte permutes: a code of up to three bits is a prmt
// selector into the eight low or high bytes of the codebook's fp16 values; the
// top bit of a 4-bit code is the sign of a symmetric codebook.  Selector word s
// of a 32-coordinate group holds the codes of coordinates s + 4 j in nibble j,
// so operand position 8 s + j of a group is coordinate s + 4 j; queries and the
// output columns use the same order.
//
// Warpgroups: 0-1 softmax (a thread half a row's keys), 2-3 accumulation (a
// thread half a row's columns), 4 expansion of keys, 5 of values, 6 MMA issue
// (one warp).  Keys of tile j + 1 are expanded and multiplied while tile j is in
// its softmax.  Seven roles share one instruction cache, so loops that need no
// unrolling stay loops: all unrolled, a tile took up to 6300 cycles.
//
// Measured (B200, d = 128, 8 KV heads, 32 query heads, 3-bit keys with m = 128,
// 4-bit values): 32 sequences over 32,768 + up to 1024 keys, bf16, 0.136 ms (193
// TFLOP/s); 64 over 16,411 + up to 777, fp32 with statistics, 0.166 ms.  Bound by
// the latency of one tile's chain through its warps, about 3500 cycles for 2300 of
// tensor-core time; reading the records is 9 us of it.
#include <math.h>

#include <algorithm>

#include "tq_cache.h"
#include "tq_common.cuh"
#include "tq_tc.cuh"

namespace {

constexpr int kKeys = 64;    // keys of a tile
constexpr int kRows = 128;   // rows of a block
constexpr int kThreads = 896;
// largest key sketch.  Limits of shared memory are set for it, the same for
// every call: the attribute is the process's, and one thread's launch may come
// between another's two steps
constexpr int kMostM = 128;
constexpr int kAccWarp0 = 8, kKeyWarp0 = 16, kValWarp0 = 20, kMmaWarp = 24;
// registers a thread after the roles have split the 72 of the launch:
// 2 * 80 + 2 * 88 + 72 + 72 + 24 = 7 * 72
constexpr int kRegSoft = 80, kRegAcc = 88, kRegMma = 24;
constexpr float kCenScale = 16.f;  // centroids as fp16: keeps the low parts out of the subnormals
constexpr uint32_t kColO = 256, kColQ = 384;

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
typedef unsigned long long u64;
__device__ __forceinline__ u64 pair(uint32_t lo, uint32_t hi) {
  u64 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ u64 pair(float x) { return pair(__float_as_uint(x), __float_as_uint(x)); }
__device__ __forceinline__ float2 parts(u64 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
  u64 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
  u64 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// one lane of a converged warp
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(addr)
               : "memory");
}
// exponent e of x = f 2^e, 1 <= f < 2 (subnormals: -127; infinities: 0), and 2^e
__device__ __forceinline__ int exponent_of(float x) {
  const int e = (int)(__float_as_uint(x) >> 23 & 255u);
  return e == 255 ? 0 : e - 127;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 <= e <= 127
// two floats to fp16x2 (lo in the low half), and back
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t v) { return __half22float2(*reinterpret_cast<__half2*>(&v)); }

// coordinate of operand position p
__host__ __device__ constexpr int coord_of(int p) { return (p & ~31) + ((p & 31) >> 3) + 4 * (p & 7); }
// sketch row of operand position p
__host__ __device__ constexpr int sketch_of(int p) { return (p & ~31) + ((p & 31) >> 1) + 16 * (p & 1); }

// prmt tables of one segment: bytes of the fp16 high and low parts
struct Tab {
  uint32_t hl[2], hh[2], ll[2], lh[2];
};

struct Smem {
  Tab tab[2][2];  // [keys, values][segment]
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2], sfull[2], pfull[2], pair[4], ofull, oempty, qfull, done;
  uint32_t tmem;
  int abort;
  alignas(16) float a[4][kKeys], b[4][kKeys], c[4][kKeys], v[4][kKeys];  // per key: a_k, b_k, 0 (-inf: no key), nu_v 2^(14 - e)
  float smax[2][2][kRows];                                   // a half tile's maximum
  float zsum[2][kRows];
  float f[8];                                                // 2^(e - 14) of a tile
  float mrow[4][kRows];                                      // running maximum after a tile
  int64_t len[kRows];                                        // keys of the block's sequences
};

template <int D>
struct Layout {
  static constexpr int NP = 2;                          // fp16 parts of an operand
  static constexpr int kpart = kKeys * D * 2;           // one part of a key or value tile
  int w, k, sg, v, total, kstage;
  int vst;  // value stages: two where they fit (all but d = 128 with m = 128)
  __host__ __device__ explicit Layout(int m) {
    w = 0;                                // W image: NP parts of [m / 8][128][16 bytes]
    const int wpart = kRows * m * 2;
    k = w + NP * wpart;                   // two key stages: centroid parts, then signs
    sg = NP * kpart;                      // offset of the signs in a key stage
    kstage = sg + kKeys * m * 2;
    v = k + 2 * kstage;
    vst = v + 2 * NP * kpart <= 216 * 1024 ? 2 : 1;
    total = v + vst * NP * kpart;
    const int rows_out = kRows * (D + 3) * 4;  // the block's result, over the same bytes
    if (total < rows_out) total = rows_out;
  }
};

// 32 coordinates of one key from their bit planes: 4 chunks of 16 bytes at
// `dst` + 1024 s, and the low parts at dst + lo_off
template <int P>
__device__ __forceinline__ void expand32(const uint32_t (&pl)[4], const Tab& t, unsigned char* dst, int lo_off) {
  const uint32_t neg = ~pl[3];  // P = 4: the top bit is the sign, the others the magnitude or its complement
  uint32_t w[3];
#pragma unroll
  for (int p = 0; p < 3; ++p) w[p] = P == 4 ? pl[p] ^ neg : pl[p];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    uint32_t sel = 0u;
#pragma unroll
    for (int p = 0; p < (P < 3 ? P : 3); ++p)
      sel |= (s >= p ? w[p] >> (s - p) : w[p] << (p - s)) & (0x11111111u << p);
    uint32_t sgn = 0u;  // 4 in a negative coordinate's nibble
    if constexpr (P == 4) sgn = (s >= 2 ? neg >> (s - 2) : neg << (2 - s)) & 0x44444444u;
    uint4 hi, lo;
    uint32_t* ph = reinterpret_cast<uint32_t*>(&hi);
    uint32_t* pw = reinterpret_cast<uint32_t*>(&lo);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t sl = h ? sel >> 16 : sel;
      uint32_t sg = 0u;
      if constexpr (P == 4) sg = prmt(0u, 0x80808080u, h ? sgn >> 16 : sgn);
      const uint32_t a = prmt(t.hl[0], t.hl[1], sl), b = prmt(t.hh[0], t.hh[1], sl) ^ sg;
      ph[2 * h] = prmt(a, b, 0x5140);
      ph[2 * h + 1] = prmt(a, b, 0x7362);
      const uint32_t c = prmt(t.ll[0], t.ll[1], sl), e = prmt(t.lh[0], t.lh[1], sl) ^ sg;
      pw[2 * h] = prmt(c, e, 0x5140);
      pw[2 * h + 1] = prmt(c, e, 0x7362);
    }
    *reinterpret_cast<uint4*>(dst + 1024 * s) = hi;
    *reinterpret_cast<uint4*>(dst + 1024 * s + lo_off) = lo;
  }
}

__device__ __forceinline__ void expand_group(int bits, const uint32_t (&pl)[4], const Tab& t, unsigned char* dst, int lo_off) {
  switch (bits) {
    case 1: expand32<1>(pl, t, dst, lo_off); break;
    case 2: expand32<2>(pl, t, dst, lo_off); break;
    case 3: expand32<3>(pl, t, dst, lo_off); break;
    default: expand32<4>(pl, t, dst, lo_off);
  }
}

// plane words of one key's half row: NWH words per plane from `src`
template <int NWH>
__device__ __forceinline__ void load_planes(uint32_t (&r)[4][NWH], const uint32_t* __restrict__ src, int pw, int bits,
                                            bool valid) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    if constexpr (NWH == 2) {
      const uint2 x = (valid && p < bits) ? __ldg(reinterpret_cast<const uint2*>(src + p * pw)) : make_uint2(0u, 0u);
      r[p][0] = x.x;
      r[p][1] = x.y;
    } else {
      r[p][0] = (valid && p < bits) ? __ldg(src + p * pw) : 0u;
    }
  }
}

// The block's tiles: prefix tiles, then every sequence's own.
struct Cursor {
  int seq;      // -1: prefix
  int64_t t0;   // first key
  __device__ void start(const Smem& s, int64_t tile, int64_t Tp) {
    const int64_t np = (Tp + kKeys - 1) / kKeys;
    seq = -1;
    if (tile < np) {
      t0 = tile * kKeys;
      return;
    }
    tile -= np;
    for (seq = 0;; ++seq) {
      const int64_t k = (s.len[seq] + kKeys - 1) / kKeys;
      if (tile < k) break;
      tile -= k;
    }
    t0 = tile * kKeys;
  }
  __device__ void next(const Smem& s, int64_t Tp) {
    t0 += kKeys;
    if (t0 < (seq < 0 ? Tp : s.len[seq])) return;
    t0 = 0;
    for (++seq; seq < kRows && s.len[seq] == 0; ++seq) {
    }
  }
};

// Query image of one group (KV head h, row block rb): for each of its kRows rows
// the fp16 parts of up * q' and of up * S q' in the order of the key operands,
//   [part][position / 8][row][8], positions [0, D) of q', then [0, m) of S q',
// and 1 / up, the power of two that brings the row's largest element to
// [2^9, 2^10).  Rows behind the last query are zero.
template <int D>
__host__ __device__ inline size_t image_part_bytes(int m) {
  return (size_t)kRows * (D + m) * 2;
}

// One block: 16 rows of one group.  Two warps of eight rotate a row pair each
// (Hadamard, or the dense Haar rotation), then thread (c, half) sums sketch row
// c for eight rows from the transposed sketch, whose columns are coalesced:
// the sketch is read once for 16 queries instead of once a query.
constexpr int kPrepRows = 16;

template <int D, typename TIn>
__global__ void __launch_bounds__(256)
    prefix_prep_kernel(const tq_params p, const TIn* __restrict__ q, const int B, const int Hq, const int G,
                       const int SB, unsigned char* __restrict__ img, float* __restrict__ scales) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int VPL = D / 32;
  __shared__ __align__(16) float qt[D][kPrepRows];  // q' transposed
  __shared__ float wt[128][kPrepRows + 1];          // S q' transposed
  __shared__ float buf[8][D], s_up[kPrepRows];
  extern __shared__ __align__(16) float sk[];  // transposed sketch [D][m]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nrb = (B + SB - 1) / SB;
  const int part = blockIdx.x % (kRows / kPrepRows), grp = blockIdx.x / (kRows / kPrepRows);
  const int rb = grp % nrb, h = grp / nrb, m = p.m;
  const int b0 = rb * SB, rows = min(SB, B - b0) * G, r0 = part * kPrepRows;
  for (int i = tid; i < D * m / 4; i += 256)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tqtc::smem_u32(sk + 4 * i)), "l"(p.St + 4 * i) : "memory");
  asm volatile("cp.async.commit_group;" ::: "memory");
  for (int i = warp; i < kPrepRows; i += 8) {
    const int r = r0 + i;
    float v[VPL];
#pragma unroll
    for (int k = 0; k < VPL; ++k) v[k] = 0.f;
    if (r < rows) {
      const TIn* src = q + (size_t)((b0 + r / G) * Hq + h * G + r % G) * D;
#pragma unroll
      for (int k = 0; k < VPL; ++k) {
        const float x = tq_to_f32(src[lane + 32 * k]);
        v[k] = tq_dneg(p.dbits, k, lane) ? -x : x;
      }
      if (p.haar) {
        tq_dense_rotate_warp<VPL>(v, lane, p.piT, buf[warp]);
      } else {
        tq_fwht_warp<VPL>(v, lane);
#pragma unroll
        for (int k = 0; k < VPL; ++k) v[k] *= p.inv_sqrt_p;
      }
    }
#pragma unroll
    for (int k = 0; k < VPL; ++k) qt[lane + 32 * k][i] = v[k];
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  for (int u = tid; u < 2 * m; u += 256) {
    const int c = u % m, half = u / m, Q = m / 32;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
#pragma unroll 4
    for (int i = 0; i < D; ++i) {
      const float s = sk[i * m + c];
      const float4 x = *reinterpret_cast<const float4*>(&qt[i][8 * half]);
      const float4 y = *reinterpret_cast<const float4*>(&qt[i][8 * half + 4]);
      acc[0] = fmaf(s, x.x, acc[0]);
      acc[1] = fmaf(s, x.y, acc[1]);
      acc[2] = fmaf(s, x.z, acc[2]);
      acc[3] = fmaf(s, x.w, acc[3]);
      acc[4] = fmaf(s, y.x, acc[4]);
      acc[5] = fmaf(s, y.y, acc[5]);
      acc[6] = fmaf(s, y.z, acc[6]);
      acc[7] = fmaf(s, y.w, acc[7]);
    }
    const int j = c / Q + 32 * (c % Q);  // St's column c is sketch row j
#pragma unroll
    for (int i = 0; i < 8; ++i) wt[j][8 * half + i] = acc[i];
  }
  __syncthreads();
  for (int i = warp; i < kPrepRows; i += 8) {
    float mx = 0.f;
    for (int k = lane; k < D; k += 32) mx = fmaxf(mx, fabsf(qt[k][i]));
    for (int k = lane; k < m; k += 32) mx = fmaxf(mx, fabsf(wt[k][i]));
    mx = tq_warp_max(mx);
    // 2^(9 - ex) and 2^(ex - 9) are normal numbers
    const int ex = mx > 0.f && mx < INFINITY ? max(-117, exponent_of(mx)) : 9;
    if (lane == 0) {
      s_up[i] = pow2(9 - ex);
      scales[(size_t)grp * kRows + r0 + i] = pow2(ex - 9);
    }
  }
  __syncthreads();
  unsigned char* out = img + (size_t)grp * 2 * image_part_bytes<D>(m);
  for (int u = tid; u < (D + m) / 8 * kPrepRows; u += 256) {
    const int i = u % kPrepRows, ch = u / kPrepRows;
    uint4 hi, lo;
    uint32_t* ph = reinterpret_cast<uint32_t*>(&hi);
    uint32_t* pl = reinterpret_cast<uint32_t*>(&lo);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int p0 = 8 * ch + 2 * k - (8 * ch < D ? 0 : D);
      const float x = (8 * ch < D ? qt[coord_of(p0)][i] : wt[sketch_of(p0)][i]) * s_up[i];
      const float y = (8 * ch < D ? qt[coord_of(p0 + 1)][i] : wt[sketch_of(p0 + 1)][i]) * s_up[i];
      ph[k] = pack_f16(x, y);
      const float2 f = unpack_f16(ph[k]);
      pl[k] = pack_f16(x - f.x, y - f.y);
    }
    const size_t at = ((size_t)ch * kRows + r0 + i) * 16;
    *reinterpret_cast<uint4*>(out + at) = hi;
    *reinterpret_cast<uint4*>(out + image_part_bytes<D>(m) + at) = lo;
  }
}

template <int D, bool SK>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc_kernel(const tq_params kp, const tq_params vp, const tq_prefix_args A, const int nC, const int SB) {
  using L = Layout<D>;
  constexpr int NWH = D / 64;
  extern __shared__ __align__(1024) unsigned char dyn[];
  __shared__ Smem sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const L lay(kp.m);
  const int nrb = (A.B + SB - 1) / SB;
  const int c = blockIdx.x % nC, rb = blockIdx.x / nC % nrb, h = blockIdx.x / nC / nrb;
  const int b0 = rb * SB, nb = min(SB, A.B - b0), rows = nb * A.G;

  // ---- prologue
  if (tid < kRows) {
    int64_t n = 0;
    if (tid < nb && A.T > 0) {
      n = A.lens ? __ldg(A.lens + b0 + tid) : A.T;
      if (n < 0 || n > A.T) {
        atomicMax(kp.err, (uint32_t)kErrLength);
        n = n < 0 ? 0 : A.T;
      }
    }
    sm.len[tid] = n;
  }
  if (tid >= 128 && tid < 132) {
    const int which = (tid - 128) >> 1, s = tid & 1;
    const tq_params& p = which ? vp : kp;
    Tab t = {};
    if (s < p.nseg) {
      for (int e = 0; e < 8; ++e) {
        const int code = p.bits[s] == 4 ? 8 + e : e;
        const float x = code < (1 << p.bits[s]) ? p.cen[s][code] * kCenScale : 0.f;
        const __half hi = __float2half_rn(x), lo = __float2half_rn(x - __half2float(hi));
        const uint32_t uh = __half_as_ushort(hi), ul = __half_as_ushort(lo);
        t.hl[e >> 2] |= (uh & 255u) << (8 * (e & 3));
        t.hh[e >> 2] |= (uh >> 8) << (8 * (e & 3));
        t.ll[e >> 2] |= (ul & 255u) << (8 * (e & 3));
        t.lh[e >> 2] |= (ul >> 8) << (8 * (e & 3));
      }
    }
    sm.tab[which][s] = t;
  }
  if (tid == 160) {
    for (int i = 0; i < 2; ++i) {
      tqtc::mbar_init(&sm.kfull[i], 128);
      tqtc::mbar_init(&sm.kempty[i], 1);
      tqtc::mbar_init(&sm.vfull[i], 128);
      tqtc::mbar_init(&sm.vempty[i], 1);
      tqtc::mbar_init(&sm.sfull[i], 1);
      tqtc::mbar_init(&sm.pfull[i], 8);
    }
    for (int i = 0; i < 4; ++i) tqtc::mbar_init(&sm.pair[i], 2);
    tqtc::mbar_init(&sm.ofull, 1);
    tqtc::mbar_init(&sm.oempty, 8);
    tqtc::mbar_init(&sm.qfull, 8);
    tqtc::mbar_init(&sm.done, 1);
    sm.abort = 0;
    tqtc::fence_mbar_init();
  }
  if (warp == kMmaWarp) tqtc::tmem_alloc(&sm.tmem, 512);
  tqtc::tc_fence_before();
  __syncthreads();
  tqtc::tc_fence_after();
  const uint32_t tm = sm.tmem;
  int64_t total = (A.Tp + kKeys - 1) / kKeys;
  for (int i = 0; i < nb; ++i) total += (sm.len[i] + kKeys - 1) / kKeys;
  const int64_t first = total * c / nC, last = total * (c + 1) / nC;
  const int nt = (int)(last - first);
  Cursor cur;
  cur.seq = -1;
  cur.t0 = 0;
  if (nt > 0) cur.start(sm, first, A.Tp);
  volatile int* abort = &sm.abort;
  auto fail = [&]() {
    atomicMax(kp.err, (uint32_t)tqtc::kErrMmaWait);
    *abort = 1;
  };
  // a wait that gives up ends its role's loop, for a whole warp at a time
#define WAIT_WARP(bar, parity)                                                               \
  if (!__all_sync(TQ_FULL_MASK, tqtc::mbar_wait_or_abort(&(bar), (parity), abort))) {        \
    fail();                                                                                  \
    break;                                                                                   \
  }

  if (warp < kAccWarp0) {
    // ------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegSoft));
    const int quad = warp & 3, half = warp >> 2, r = quad * 32 + lane;
    const uint32_t lane_base = tm + ((uint32_t)(quad * 32) << 16);
    const bool mine = r < rows;
    const int myseq = mine ? r / A.G : -2;
    float rs = 1.f, M = -INFINITY, Z = 0.f;
    int turn = 0;  // phases of this quadrant's pair of warps
    // the query image is the preceding launch's; every block waits for it, so
    // that this kernel never ends before that one
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (nt > 0) {
      const size_t grp = (size_t)h * nrb + rb;
      const unsigned char* img = A.image + grp * 2 * image_part_bytes<D>(kp.m);
      rs = A.scales[grp * kRows + r];
      // q' to TMEM: this half its share of the columns; S q' to shared memory
      if (quad * 32 < rows) {
#pragma unroll
        for (int part = 0; part < L::NP; ++part) {
#pragma unroll
          for (int g = 0; g < D / 64; ++g) {
            uint32_t x[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 v = *reinterpret_cast<const uint4*>(img + part * image_part_bytes<D>(kp.m) +
                                                              ((size_t)(4 * (half * (D / 64) + g) + i) * kRows + r) * 16);
              x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
            }
            tqtc::tmem_st16(lane_base + kColQ + part * (D / 2) + 16 * (half * (D / 64) + g), x);
          }
        }
        tqtc::tmem_wait_st();
        if (SK) {
#pragma unroll
          for (int part = 0; part < L::NP; ++part)
#pragma unroll 4
            for (int ch = half; ch < kp.m / 8; ch += 2)
              *reinterpret_cast<uint4*>(dyn + lay.w + part * kRows * kp.m * 2 + ch * 2048 + r * 16) =
                  *reinterpret_cast<const uint4*>(img + part * image_part_bytes<D>(kp.m) + ((size_t)(D / 8 + ch) * kRows + r) * 16);
          tqtc::fence_proxy_async_smem();
        }
      }
    }
    tqtc::tc_fence_before();
    __syncwarp();
    if (lane == 0) tqtc::mbar_arrive(&sm.qfull);
    for (int j = 0; j < nt; ++j) {
      const int s2 = j & 1, ph = (j >> 1) & 1;
      WAIT_WARP(sm.sfull[s2], ph);
      tqtc::tc_fence_after();
      const bool act = mine && (cur.seq < 0 || cur.seq == myseq);
      if (__any_sync(TQ_FULL_MASK, act)) {
        const uint32_t s_col = lane_base + 128 * s2 + 32 * half;
        u64 t[16];  // logits over the row's scale, in pairs of keys
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k0 = 0; k0 < 32; k0 += 16) {
          uint32_t x[16], y[16];
          tqtc::tmem_ld16(s_col + k0, x);
          if (SK) tqtc::tmem_ld16(s_col + 64 + k0, y);
          tqtc::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int k = 32 * half + k0 + 4 * i, o = k0 / 2 + 2 * i;
            const ulonglong2 a2 = *reinterpret_cast<const ulonglong2*>(&sm.a[j & 3][k]);
            const ulonglong2 c2 = *reinterpret_cast<const ulonglong2*>(&sm.c[j & 3][k]);
            t[o] = fma2(a2.x, pair(x[4 * i], x[4 * i + 1]), c2.x);
            t[o + 1] = fma2(a2.y, pair(x[4 * i + 2], x[4 * i + 3]), c2.y);
            if (SK) {
              const ulonglong2 b2 = *reinterpret_cast<const ulonglong2*>(&sm.b[j & 3][k]);
              t[o] = fma2(b2.x, pair(y[4 * i], y[4 * i + 1]), t[o]);
              t[o + 1] = fma2(b2.y, pair(y[4 * i + 2], y[4 * i + 3]), t[o + 1]);
            }
            const float2 f = parts(t[o]), g = parts(t[o + 1]);
            m4[i] = fmaxf(fmaxf(m4[i], fmaxf(f.x, f.y)), fmaxf(g.x, g.y));
          }
        }
        float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        sm.smax[turn & 1][half][r] = mx;
        __syncwarp();
        if (lane == 0) tqtc::mbar_arrive(&sm.pair[quad]);
        WAIT_WARP(sm.pair[quad], turn & 1);
        mx = fmaxf(M, fmaxf(mx, sm.smax[turn & 1][half ^ 1][r]) * rs);
        ++turn;
        const float ref = mx == -INFINITY ? 0.f : mx;
        const u64 rs2 = pair(rs), ref2 = pair(-ref);
        u64 z = 0ull;
        // P goes over the columns of S (high parts) and R (low parts) that this
        // warp has read
#pragma unroll
        for (int k0 = 0; k0 < 32; k0 += 16) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const ulonglong2 v2 = *reinterpret_cast<const ulonglong2*>(&sm.v[j & 3][32 * half + k0 + 2 * i]);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const float2 e = parts(fma2(t[k0 / 2 + i + w], rs2, ref2));
              const u64 p = pair(__float_as_uint(ex2(e.x)), __float_as_uint(ex2(e.y)));
              z = add2(z, p);
              const u64 pv = mul2(p, w ? v2.y : v2.x);
              // high part: the leading 11 bits; the rest is exact in fp32
              const u64 top = pv & 0xffffe000ffffe000ull;
              const float2 g = parts(top), q = parts(fma2(top, pair(-1.f), pv));
              hi[i + w] = pack_f16(g.x, g.y);
              lo[i + w] = pack_f16(q.x, q.y);
            }
          }
          tqtc::tmem_st8(s_col + k0 / 2, hi);
          tqtc::tmem_st8(s_col + 64 + k0 / 2, lo);
        }
        tqtc::tmem_wait_st();
        if (act) {
          const float2 f = parts(z);
          Z = fmaf(Z, M == -INFINITY ? 0.f : ex2(M - ref), f.x + f.y);
          M = mx;
        }
      }
      if (half == 0) sm.mrow[j & 3][r] = M;
      tqtc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tqtc::mbar_arrive(&sm.pfull[s2]);
      cur.next(sm, A.Tp);
    }
    sm.zsum[half][r] = Z;
  } else if (warp < kKeyWarp0) {
    // -------------------------------------------------------- accumulation
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegAcc));
    const int quad = warp & 3, half = (warp - kAccWarp0) >> 2;
    const int r = quad * 32 + lane;
    const bool mine = r < rows;
    const int myseq = mine ? r / A.G : -2;
    constexpr int NCOL = D / 2;
    const uint32_t o_base = tm + ((uint32_t)(quad * 32) << 16) + kColO + half * NCOL;
    u64 acc[NCOL / 2];
#pragma unroll
    for (int i = 0; i < NCOL / 2; ++i) acc[i] = 0ull;
    float M = -INFINITY;
    for (int j = 0; j < nt; ++j) {
      WAIT_WARP(sm.ofull, j & 1);
      tqtc::tc_fence_after();
      const bool act = mine && (cur.seq < 0 || cur.seq == myseq);
      if (__any_sync(TQ_FULL_MASK, act)) {
        const float m2 = sm.mrow[j & 3][r];
        const float al = act && m2 != M ? ex2(M - m2) : 1.f;
        if (__any_sync(TQ_FULL_MASK, al != 1.f)) {
          const u64 a2 = pair(al);
#pragma unroll
          for (int i = 0; i < NCOL / 2; ++i) acc[i] = mul2(acc[i], a2);
        }
        if (act) M = m2;
        const u64 f2 = pair(sm.f[j & 7]);
#pragma unroll
        for (int k0 = 0; k0 < NCOL; k0 += 8) {
          uint32_t x[8];
          tmem_ld8(o_base + k0, x);
          tqtc::tmem_wait_ld();
          if (act) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) acc[(k0 + i) / 2] = fma2(pair(x[i], x[i + 1]), f2, acc[(k0 + i) / 2]);
          }
          __syncwarp();  // the TMEM loads are whole-warp instructions
        }
      }
      tqtc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tqtc::mbar_arrive(&sm.oempty);
      cur.next(sm, A.Tp);
    }
    // rows to shared memory (the expanded tiles are spent: every product has
    // completed), one pad word a row; the block writes them out together
    if (mine) {
      float* row = reinterpret_cast<float*>(dyn) + r * (D + 3);
      const float k = vp.inv_sqrt_d / kCenScale;
#pragma unroll
      for (int i = 0; i < NCOL / 2; ++i) {
        const float2 f = parts(acc[i]);
        row[coord_of(half * NCOL + 2 * i)] = f.x * k;
        row[coord_of(half * NCOL + 2 * i + 1)] = f.y * k;
      }
      if (half == 0) row[D] = M;
    }
  } else if (warp < kValWarp0) {
    // --------------------------------------------------- expansion of keys
    const int te = tid - kKeyWarp0 * 32, key = te & 63, half = te >> 6;
    const int ks = kp.nseg == 2 ? half : 0;
    const int kw0 = kp.segbase[ks] + (kp.nseg == 2 ? 0 : half * NWH), kbits = kp.bits[ks];
    const Tab tk = sm.tab[0][ks];
    const int off = (key >> 3) * 128 + (key & 7) * 16;
    uint32_t kw[4][NWH], sg[2] = {0u, 0u};
    float nu = 0.f, gam = 0.f, nv0 = 0.f, nv1 = 0.f;
    bool kvalid = false;
    auto load = [&](const Cursor& cu) {
      const bool pre = cu.seq < 0;
      const int64_t n = pre ? A.Tp : sm.len[cu.seq];
      const tq_compressed& K = pre ? A.Kp : A.K;
      const float* vn = pre ? A.Vp.norms : A.V.norms;
      const int64_t first_row = (pre ? (int64_t)h * A.Tp : ((int64_t)(b0 + cu.seq) * A.Hkv + h) * A.T) + cu.t0;
      const bool valid = kvalid = cu.t0 + key < n;
      const int64_t row = first_row + key;
      load_planes<NWH>(kw, K.codes + row * kp.W + kw0, kp.pw, kbits, valid);
      if (SK) {
#pragma unroll
        for (int i = 0; i < 2; ++i) sg[i] = (valid && half + 2 * i < kp.MS) ? __ldg(K.signs + row * kp.MS + half + 2 * i) : 0u;
        gam = valid ? __ldg(K.rnorms + row) : 0.f;
      }
      nu = valid ? __ldg(K.norms + row) : 0.f;
      // value norms of keys lane and lane + 32: every warp sees the whole tile
      nv0 = cu.t0 + lane < n ? __ldg(vn + first_row + lane) : 0.f;
      nv1 = cu.t0 + 32 + lane < n ? __ldg(vn + first_row + 32 + lane) : 0.f;
    };
    if (nt > 0) load(cur);
    const float ca = A.scale_log2e * kp.inv_sqrt_d / kCenScale, cb = A.scale_log2e * kp.qjl_coef;
    for (int j = 0; j < nt; ++j) {
      const int s2 = j & 1;
      // QK(j - 2) done also means that softmax(j - 4) is: its product with the
      // values was issued before, so the scalars' slot j & 3 is free
      if (j >= 2) WAIT_WARP(sm.kempty[s2], ((j >> 1) & 1) ^ 1);
      unsigned char* st = dyn + lay.k + s2 * lay.kstage;
#pragma unroll 1
      for (int i = 0; i < NWH; ++i) {
        const uint32_t pl[4] = {kw[0][0], kw[1][0], kw[2][0], kw[3][0]};
        expand_group(kbits, pl, tk, st + (half * NWH + i) * 4096 + off, L::kpart);
#pragma unroll
        for (int p = 0; p < 4; ++p) kw[p][0] = kw[p][NWH - 1];
      }
      if (SK) {
#pragma unroll 1
        for (int w = half; w < kp.MS; w += 2) {
          const uint32_t y = sg[0];
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) {  // pairs (j, j + 16) to the sign bits of a word
            uint4 x;
            x.x = ((y << (15 - 4 * ch)) & 0x80008000u) ^ 0xBC00BC00u;
            x.y = ((y << (14 - 4 * ch)) & 0x80008000u) ^ 0xBC00BC00u;
            x.z = ((y << (13 - 4 * ch)) & 0x80008000u) ^ 0xBC00BC00u;
            x.w = ((y << (12 - 4 * ch)) & 0x80008000u) ^ 0xBC00BC00u;
            *reinterpret_cast<uint4*>(st + lay.sg + (4 * w + ch) * 1024 + off) = x;
          }
          sg[0] = sg[1];
        }
      }
      if (half == 0) {
        const float nm = tq_warp_max(fmaxf(fabsf(nv0), fabsf(nv1)));
        const int e = max(-100, exponent_of(nm) + 1);  // |nv| < 2^e
        sm.a[j & 3][key] = nu * ca;
        sm.b[j & 3][key] = nu * gam * cb;
        sm.c[j & 3][key] = kvalid ? 0.f : -INFINITY;
        sm.v[j & 3][key] = ((key & 32) ? nv1 : nv0) * pow2(14 - e);
        if (key == 0) sm.f[j & 7] = pow2(e - 14);
      }
      tqtc::fence_proxy_async_smem();
      tqtc::mbar_arrive(&sm.kfull[s2]);
      if (j + 1 < nt) {
        cur.next(sm, A.Tp);
        load(cur);
      }
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------- expansion of values
    const int te = tid - kValWarp0 * 32, key = te & 63, half = te >> 6;
    const int vs = vp.nseg == 2 ? half : 0;
    const int vw0 = vp.segbase[vs] + (vp.nseg == 2 ? 0 : half * NWH), vbits = vp.bits[vs];
    const Tab tv = sm.tab[1][vs];
    const int off = (key >> 3) * 128 + (key & 7) * 16;
    uint32_t vw[4][NWH];
    auto load = [&](const Cursor& cu) {
      const bool pre = cu.seq < 0;
      const int64_t n = pre ? A.Tp : sm.len[cu.seq];
      const int64_t base = pre ? (int64_t)h * A.Tp : ((int64_t)(b0 + cu.seq) * A.Hkv + h) * A.T;
      load_planes<NWH>(vw, (pre ? A.Vp : A.V).codes + (base + cu.t0 + key) * vp.W + vw0, vp.pw, vbits, cu.t0 + key < n);
    };
    if (nt > 0) load(cur);
    for (int j = 0; j < nt; ++j) {
      const int sv = lay.vst == 2 ? (j & 1) : 0, use = lay.vst == 2 ? (j >> 1) : j;
      if (use >= 1) WAIT_WARP(sm.vempty[sv], (use & 1) ^ 1);
      unsigned char* st = dyn + lay.v + sv * L::NP * L::kpart;
#pragma unroll 1
      for (int i = 0; i < NWH; ++i) {
        const uint32_t pl[4] = {vw[0][0], vw[1][0], vw[2][0], vw[3][0]};
        expand_group(vbits, pl, tv, st + (half * NWH + i) * 4096 + off, L::kpart);
#pragma unroll
        for (int p = 0; p < 4; ++p) vw[p][0] = vw[p][NWH - 1];
      }
      tqtc::fence_proxy_async_smem();
      tqtc::mbar_arrive(&sm.vfull[sv]);
      if (j + 1 < nt) {
        cur.next(sm, A.Tp);
        load(cur);
      }
    }
  } else {
    // ----------------------------------------------------------- MMA issue
    // The whole warp walks the loop with warp-uniform values and one elected
    // lane issues: an issue loop inside a single-lane branch costs 48 cycles
    // per 32-cycle product (measured), this one 33.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegMma));
    if (__shfl_sync(TQ_FULL_MASK, warp, 0) == kMmaWarp && nt > 0) {
      constexpr uint32_t idS = tqtc::instr_desc(1, 0, 0, 128, kKeys);
      constexpr uint32_t idO = tqtc::instr_desc(1, 0, 0, 128, D) | (1u << 16);  // B with its N index contiguous
      const uint32_t base = __shfl_sync(TQ_FULL_MASK, tqtc::smem_u32(dyn), 0);
      const uint32_t tu = __shfl_sync(TQ_FULL_MASK, tm, 0);
      const int ks = kp.m / 32;
      for (int j = 0; j <= nt; ++j) {
        if (j < nt) {
          const int s2 = j & 1, ph = (j >> 1) & 1;
          if (j == 0) WAIT_WARP(sm.qfull, 0);
          WAIT_WARP(sm.kfull[s2], ph);
          tqtc::tc_fence_after();
          if (elect()) {
            const uint32_t dS = tu + 128 * s2, kst = base + lay.k + s2 * lay.kstage;
            // parts: low queries, low keys, then the high product
#pragma unroll 1
            for (int pr = 0; pr < 3; ++pr) {
              const uint32_t qa = tu + kColQ + (pr == 0 ? D / 2 : 0);
              const uint64_t kd = tqtc::smem_desc(kst + (pr == 1 ? L::kpart : 0), 1024, 128);
#pragma unroll
              for (int k = 0; k < D / 16; ++k)
                tqtc::mma_f16_ts(dS, qa + 8 * k, kd + 128 * k, idS, !(k == 0 && pr == 0));
            }
            if (SK) {
              const uint64_t sd = tqtc::smem_desc(kst + lay.sg, 1024, 128);
#pragma unroll 1
              for (int pr = 0; pr < 2; ++pr) {
                const uint64_t wd = tqtc::smem_desc(base + lay.w + (pr == 0 ? kRows * kp.m * 2 : 0), 2048, 128);
#pragma unroll 1
                for (int k = 0; k < ks; ++k) {
                  tqtc::mma_f16_ss(dS + 64, wd + 512 * k, sd + 256 * k, idS, !(k == 0 && pr == 0));
                  tqtc::mma_f16_ss(dS + 64, wd + 512 * k + 256, sd + 256 * k + 128, idS, true);
                }
              }
            }
            tqtc::mma_commit(&sm.kempty[s2]);
            tqtc::mma_commit(&sm.sfull[s2]);
          }
          __syncwarp();
        }
        if (j > 0) {
          const int i0 = j - 1, s2 = i0 & 1, ph = (i0 >> 1) & 1;
          const int sv = lay.vst == 2 ? s2 : 0, use = lay.vst == 2 ? (i0 >> 1) : i0;
          WAIT_WARP(sm.pfull[s2], ph);
          WAIT_WARP(sm.vfull[sv], use & 1);
          if (i0 >= 1) WAIT_WARP(sm.oempty, (i0 & 1) ^ 1);
          tqtc::tc_fence_after();
          if (elect()) {
            const uint32_t dO = tu + kColO, pA = tu + 128 * s2, vst = base + lay.v + sv * L::NP * L::kpart;
#pragma unroll 1
            for (int pr = 0; pr < 3; ++pr) {
              const uint32_t pa = pA + (pr == 0 ? 64 : 0);
              const uint64_t vd = tqtc::smem_desc(vst + (pr == 1 ? L::kpart : 0), 128, 1024);
#pragma unroll
              for (int k = 0; k < kKeys / 16; ++k)
                tqtc::mma_f16_ts(dO, pa + 32 * (k >> 1) + 8 * (k & 1), vd + 16 * k, idO, !(k == 0 && pr == 0));
            }
            tqtc::mma_commit(&sm.vempty[sv]);
            tqtc::mma_commit(&sm.ofull);
          }
          __syncwarp();
        }
      }
      // every product and commit has landed before the block ends
      if (elect()) tqtc::mma_commit(&sm.done);
      __syncwarp();
      if (!tqtc::mbar_wait(&sm.done, 0)) fail();
    }
  }
#undef WAIT_WARP
  __syncwarp();
  tqtc::tc_fence_before();
  __syncthreads();
  for (int r = warp; r < rows; r += kThreads / 32) {
    float* pr = A.partials + ((size_t)((b0 + r / A.G) * A.Hq + h * A.G + r % A.G) * nC + c) * (D + 2);
    const float* row = reinterpret_cast<const float*>(dyn) + r * (D + 3);
#pragma unroll
    for (int k = 0; k < D / 32; ++k) pr[lane + 32 * k] = row[lane + 32 * k];
    // the two halves' sums: their exponentials refer to the same maxima
    if (lane < 2) pr[D + lane] = lane ? sm.zsum[0][r] + sm.zsum[1][r] : row[D];
  }
  if (warp == kMmaWarp) {
    tqtc::tc_fence_after();
    tqtc::tmem_dealloc(tm, 512);
  }
}

template <int D, typename TIn>
cudaError_t launch_prep(const tq_params& kp, const tq_prefix_args& a, int SB, unsigned groups, cudaStream_t st) {
  auto fn = prefix_prep_kernel<D, TIn>;
  const size_t smem = sizeof(float) * (size_t)D * kp.m;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(float) * D * kMostM);
  if (e != cudaSuccess) return e;
  fn<<<groups * (kRows / kPrepRows), 256, smem, st>>>(kp, (const TIn*)a.q, a.B, a.Hq, a.G, SB, a.image, a.scales);
  return cudaGetLastError();
}

template <int D, bool SK>
cudaError_t launch(const tq_params& kp, const tq_params& vp, const tq_prefix_args& a, int nC, int SB, unsigned groups,
                   cudaStream_t st) {
  const Layout<D> lay(kp.m);
  auto fn = prefix_tc_kernel<D, SK>;
  int most = 0;  // m = 96 needs more than m = 128, which has one value stage
  for (int m = 0; m <= kMostM; m += 32) most = std::max(most, Layout<D>(m).total);
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return e;
  e = a.dtype == TQ_F32    ? launch_prep<D, float>(kp, a, SB, groups, st)
      : a.dtype == TQ_BF16 ? launch_prep<D, __nv_bfloat16>(kp, a, SB, groups, st)
                           : launch_prep<D, __half>(kp, a, SB, groups, st);
  if (e != cudaSuccess) return e;
  // programmatic dependent launch: the blocks set up and expand their first
  // tiles while the queries are prepared, and wait for the image where they read it
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(groups * nC);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = lay.total;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, kp, vp, a, nC, SB);
}

}  // namespace

bool tq_prefix_tc_supported(const tq_params& kp, const tq_params& vp) {
  return (kp.d == 64 || kp.d == 128) && kp.m <= kMostM && vp.m == 0 && !kp.vq_bits && !vp.vq_bits;
}

static int64_t groups_of(int B, int Hkv, int G) { return (int64_t)Hkv * ((B + kRows / G - 1) / (kRows / G)); }

// query images (two fp16 parts), then the rows' scales
size_t tq_prefix_tc_bytes(const tq_params& kp, int B, int Hkv, int G, size_t* scales_at) {
  const size_t groups = (size_t)groups_of(B, Hkv, G);
  *scales_at = groups * 2 * kRows * (size_t)(kp.d + kp.m) * 2;
  return *scales_at + groups * kRows * sizeof(float);
}

cudaError_t tq_launch_prefix_tc(const tq_params& kp, const tq_params& vp, const tq_prefix_args& a,
                                const tq_prefix_plan& plan, cudaStream_t st) {
  const int SB = kRows / a.G;
  const int64_t groups = groups_of(a.B, a.Hkv, a.G);
  if (groups * std::max(plan.nP, kRows / kPrepRows) > 0x7fffffffll) return cudaErrorNotSupported;
  const unsigned g = (unsigned)groups;
  if (kp.d == 64)
    return kp.m ? launch<64, true>(kp, vp, a, plan.nP, SB, g, st) : launch<64, false>(kp, vp, a, plan.nP, SB, g, st);
  return kp.m ? launch<128, true>(kp, vp, a, plan.nP, SB, g, st) : launch<128, false>(kp, vp, a, plan.nP, SB, g, st);
}
