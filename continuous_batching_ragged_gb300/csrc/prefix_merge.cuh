// Joining a row's attention over its own keys with the shared prefix's state.
//
// With the softmax of a row cut into parts, part i leaves (acc_i, m_i, l_i): the
// sum of 2^(s - m_i) v, the part's reference maximum and the sum of 2^(s - m_i)
// (scores s in the exp2 domain).  The row is
//     sum_i 2^(m_i - M) acc_i / sum_i 2^(m_i - M) l_i,   M = max_i m_i.
// The prefix kernel leaves one record per row and KV segment; the kernels that
// run a row's own keys join them here, in the order of the segments, so a
// row's bits never depend on which piece finished first.
#pragma once

#include "device_common.cuh"
#include "kernels.h"

namespace cb {

// The prefix part of sequence s, as the prefix plan left it.
__device__ __forceinline__ int4 prefix_info(const AttnArgs& a, int s) {
  return __ldcg(reinterpret_cast<const int4*>(a.prefix.seq_info) + s);   // (skipped blocks, records, stride, -)
}
__device__ __forceinline__ const float* prefix_records(const AttnArgs& a, const int4& info, int token, int head) {
  return a.prefix.recs + (size_t(token) * a.num_heads + head) * info.z * kPrefixRec;
}

// One dimension d of a row: own state (o, M, L) joined with the records.
__device__ __forceinline__ float join_prefix_dim(const float* rec, int n, int d, float o, float M, float L) {
  float mx = M;
  for (int k = 0; k < n; ++k) mx = fmaxf(mx, __ldcg(rec + size_t(k) * kPrefixRec + kPrefixDim));
  const float f = ex2(M - mx);
  float num = o * f, den = L * f;
#pragma unroll 4
  for (int k = 0; k < n; ++k) {
    const float* r = rec + size_t(k) * kPrefixRec;
    const float w = ex2(__ldcg(r + kPrefixDim) - mx);
    num = fmaf(w, __ldcg(r + d), num);
    den = fmaf(w, __ldcg(r + kPrefixDim + 1), den);
  }
  return num / den;
}

// A row held by one thread: the common maximum and 1 / denominator for the own
// state (M, L) and the records.
__device__ __forceinline__ void prefix_row_scale(const float* rec, int n, float M, float L, float& mx, float& inv) {
  mx = M;
  for (int k = 0; k < n; ++k) mx = fmaxf(mx, __ldcg(rec + size_t(k) * kPrefixRec + kPrefixDim));
  float den = L * ex2(M - mx);
  for (int k = 0; k < n; ++k) {
    const float* r = rec + size_t(k) * kPrefixRec + kPrefixDim;
    den = fmaf(ex2(__ldcg(r) - mx), __ldcg(r + 1), den);
  }
  inv = 1.0f / den;
}
// acc[0..N) (own state, unscaled, of reference maximum M) -> the joined, normalised dims d0 .. d0 + N - 1.
template <int N>
__device__ __forceinline__ void join_prefix_row(const float* rec, int n, int d0, float M, float mx, float inv,
                                                float (&acc)[N]) {
  const float f = ex2(M - mx) * inv;
#pragma unroll
  for (int e = 0; e < N; ++e) acc[e] *= f;
  for (int k = 0; k < n; ++k) {
    const float* r = rec + size_t(k) * kPrefixRec;
    const float w = ex2(__ldcg(r + kPrefixDim) - mx) * inv;
#pragma unroll
    for (int e = 0; e < N; e += 4) {
      const float4 x = __ldcg(reinterpret_cast<const float4*>(r + d0 + e));
      acc[e] = fmaf(w, x.x, acc[e]);
      acc[e + 1] = fmaf(w, x.y, acc[e + 1]);
      acc[e + 2] = fmaf(w, x.z, acc[e + 2]);
      acc[e + 3] = fmaf(w, x.w, acc[e + 3]);
    }
  }
}

}  // namespace cb
