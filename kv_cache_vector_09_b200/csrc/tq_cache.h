// Internal declarations of the shared-prefix attention and of the bounded
// cache (accumulated attention weight, eviction, record copies).
#pragma once

#include "tq_internal.h"

// device error word: a length or a row index that a kernel found out of range
// (codes 1 to 3 are in tq_tc.cuh)
enum : uint32_t { kErrLength = 4, kErrRowIndex = 5 };

// How one tq_attend_prefix call is cut.  A unit is one KV head's prefix or one
// (sequence, KV head)'s own keys; each is cut into a fixed number of chunks,
// and every (query row, chunk) leaves a partial (acc[d], max, sum[, a[m_v]]).
struct tq_prefix_plan {
  int nP;   // chunks per prefix unit (0: no prefix); tc: blocks per group of rows
  int nO;   // chunks per own unit (0: no own keys, or tc)
  bool tc;  // tensor-core kernel (tq_prefix_tc.cu)
};

struct tq_prefix_args {
  int B, Hq, Hkv, G;
  int64_t Tp, T;
  const int32_t* lens;  // [B] or null (all T)
  tq_compressed Kp, Vp, K, V;
  float scale_log2e;
  const void* q;        // [B][Hq][d]
  tq_dtype dtype;
  const float* qprep;   // [B * Hq][d + m] (CUDA-core kernel)
  unsigned char* image; // query images and row scales (tensor-core kernel)
  float* scales;
  float* partials;     // [B * Hq][nP + nO][d + 2 + m_v]
};

cudaError_t tq_launch_prefix_any(const tq_params& kp, const tq_params& vp, const tq_prefix_args& a,
                                 const tq_prefix_plan& plan, cudaStream_t st);
// whether the codecs have the tensor-core kernel, its query images' bytes, and its launch
bool tq_prefix_tc_supported(const tq_params& kp, const tq_params& vp);
size_t tq_prefix_tc_bytes(const tq_params& kp, int B, int Hkv, int G, size_t* scales_at);
cudaError_t tq_launch_prefix_tc(const tq_params& kp, const tq_params& vp, const tq_prefix_args& a,
                                const tq_prefix_plan& plan, cudaStream_t st);
cudaError_t tq_launch_prefix_combine(const tq_params& vp, const tq_prefix_args& a, const tq_prefix_plan& plan,
                                     void* out, tq_dtype out_dtype, float* lse, cudaStream_t st);

cudaError_t tq_launch_mass(const tq_params& p, const float* logits, int B, int Hq, int Hkv, int64_t T,
                           const int32_t* lens, const float* lse, float scale, float decay, float* mass,
                           cudaStream_t st);
cudaError_t tq_launch_evict(const tq_params& p, const float* mass, int B, int Hkv, int64_t T, const int32_t* lens,
                            int64_t keep, int64_t sink, int64_t recent, int32_t* idx, float* mass_out,
                            int32_t* lens_out, cudaStream_t st);
cudaError_t tq_launch_copy_rows(const tq_params& p, const tq_compressed& src, int64_t src_T, const tq_compressed& dst,
                                int64_t dst_T, int64_t rows, int64_t n, const int32_t* src_idx,
                                const int32_t* dst_idx, cudaStream_t st);
