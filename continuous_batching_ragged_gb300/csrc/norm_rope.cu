// cb_norm_rope_append: RMS norm of each query and key head, the position
// rotation, and the append of keys and values to the paged cache, in one pass.
//
// Per token t and head, with x the head's row in fp32:
//     y = x * rsqrt(mean(x^2) + eps) * w           (norm; left out where w is null)
//     (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s)  for each pair (a, b) of the
//                                                   first rot_dim dimensions,
// c and s from the position's row of a fp32 table.  Queries go to q_out, keys
// to the token's cache slot, values to theirs unchanged.  Everything between
// the load and the one rounding at the store is fp32.
//
// Bound by HBM: every row is read once and written once, a few dozen fp32
// operations per 16 bytes in between.  A group of LPR lanes holds one row, 16
// bytes a lane, so that the mean is log2(LPR) shuffles, the half-split pair of
// an element sits in one other lane, and a lane's cosines, sines and weights
// are the same for every head of its token: they are loaded once and serve the
// kRows rows that the group keeps in flight.
#include <algorithm>
#include <cmath>

#include "device_common.cuh"
#include "runtime.h"

namespace {

using cb::Vec16;

constexpr int kThreads = 256;
constexpr int kSpreadCtasPerSm = 8;   // up to so many CTAs of one row per lane group, a token is spread over several

struct NormRopeArgs {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;   // 16-byte chunks between tokens
  const void *q_weight, *k_weight;
  const float* cos_sin;
  const int32_t* positions;
  const int64_t* slots;
  const int32_t* dims;
  uint4 *q_out, *k_pool, *v_pool;
  int64_t num_slots;
  int32_t num_tokens, num_q_heads, num_kv_heads, block_size, max_positions, rot_dim;
  float eps;
  unsigned* err;
};

__device__ __forceinline__ uint4 pack16(const float (&f)[8]) {
  uint4 r;
  uint32_t* w = &r.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return r;
}
__device__ __forceinline__ uint4 pack16(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

// blockIdx.y takes kRows rows per lane group of the token's num_q_heads query,
// num_kv_heads key and num_kv_heads value rows, in that order; blockIdx.x
// strides over tokens.
template <typename T, int LPR, int kRows, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) norm_rope_append_kernel(const NormRopeArgs a) {
  constexpr int EPV = Vec16<T>::N;              // elements per lane
  constexpr int A = LPR * EPV;                  // head_dim
  constexpr int kGroups = kThreads / LPR;       // rows side by side in the CTA
  int32_t n_tok = a.num_tokens;
  if (a.dims) {                                 // the step's token count, at most num_tokens (the capacity)
    const int32_t t = a.dims[1];
    if (t < 0 || t > a.num_tokens) {
      if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) cb::raise_error(a.err, cb::kErrInvalid);
      return;
    }
    n_tok = t;
  }
  const int lane = threadIdx.x & 31;
  const int c = threadIdx.x % LPR;              // this lane's 16-byte chunk of the row
  const int H = a.num_q_heads, K = a.num_kv_heads, n_rows = H + 2 * K;
  const int row0 = (blockIdx.y * kRows) * kGroups + threadIdx.x / LPR;
  const int half = a.rot_dim / 2;
  const bool turned = c * EPV < a.rot_dim;      // rot_dim is a multiple of 2 * EPV: a lane turns all or nothing
  // half-split pairs: element d of the first half pairs with d + rot_dim / 2
  const bool low = c * EPV < half;
  const int partner = INTERLEAVED || !turned ? lane : lane + (low ? 1 : -1) * (half / EPV);

  float wq[EPV], wk[EPV];
  if (a.q_weight) Vec16<T>::to_float(__ldg(static_cast<const uint4*>(a.q_weight) + c), wq);
  if (a.k_weight) Vec16<T>::to_float(__ldg(static_cast<const uint4*>(a.k_weight) + c), wk);

  for (int tok = blockIdx.x; tok < n_tok; tok += gridDim.x) {
    uint4 raw[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int r = row0 + u * kGroups;
      const uint4* src = r < H       ? static_cast<const uint4*>(a.q) + tok * a.q_stride + int64_t(r) * LPR
                         : r < H + K ? static_cast<const uint4*>(a.k) + tok * a.k_stride + int64_t(r - H) * LPR
                                     : static_cast<const uint4*>(a.v) + tok * a.v_stride + int64_t(r - H - K) * LPR;
      raw[u] = r < n_rows ? *(src + c) : make_uint4(0, 0, 0, 0);
    }
    const int64_t slot = a.slots[tok];
    float cs[EPV], sn[EPV];                     // interleaved: the first EPV / 2 hold the lane's pairs
#pragma unroll
    for (int e = 0; e < EPV; ++e) cs[e] = 1.f, sn[e] = 0.f;
    bool skip = false;
    if (a.rot_dim > 0) {
      const int pos = a.positions[tok];
      skip = pos < 0 || pos >= a.max_positions;
      if (skip && threadIdx.x == 0 && blockIdx.y == 0) cb::raise_error(a.err, cb::kErrBounds);
      if (!skip && turned) {
        const float* tab = a.cos_sin + int64_t(pos) * a.rot_dim;
        const int d0 = INTERLEAVED ? c * (EPV / 2) : (low ? c * EPV : c * EPV - half);
        // 16 bytes at a time, or 8 where an interleaved fp32 lane has only two pairs
        constexpr int kTab = INTERLEAVED ? EPV / 2 : EPV;
        if constexpr (kTab % 4 == 0) {
#pragma unroll
          for (int e = 0; e < kTab; e += 4) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(tab + d0 + e));
            const float4 y = __ldg(reinterpret_cast<const float4*>(tab + half + d0 + e));
            cs[e] = x.x, cs[e + 1] = x.y, cs[e + 2] = x.z, cs[e + 3] = x.w;
            sn[e] = y.x, sn[e + 1] = y.y, sn[e + 2] = y.z, sn[e + 3] = y.w;
          }
        } else {
          const float2 x = __ldg(reinterpret_cast<const float2*>(tab + d0));
          const float2 y = __ldg(reinterpret_cast<const float2*>(tab + half + d0));
          cs[0] = x.x, cs[1] = x.y, sn[0] = y.x, sn[1] = y.y;
        }
      }
    }
    if (skip) continue;                         // the same for the whole CTA
    const bool bad_slot = slot >= a.num_slots;
    if (bad_slot && threadIdx.x == 0 && blockIdx.y == 0) cb::raise_error(a.err, cb::kErrBounds);
    const bool cached = slot >= 0 && !bad_slot;
    const int64_t blk = cached ? slot / a.block_size : 0, off = cached ? slot - blk * a.block_size : 0;
    const int64_t dst0 = (blk * K * a.block_size + off) * LPR, head_step = int64_t(a.block_size) * LPR;
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int r = row0 + u * kGroups;
      float x[EPV];
      Vec16<T>::to_float(raw[u], x);
      const bool is_q = r < H, norm = is_q ? a.q_weight != nullptr : a.k_weight != nullptr;
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < EPV; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (norm) {
        const float inv = rsqrtf(ss * (1.0f / A) + a.eps);
#pragma unroll
        for (int e = 0; e < EPV; ++e) x[e] = x[e] * inv * (is_q ? wq[e] : wk[e]);
      }
      if (INTERLEAVED) {
        if (turned) {
#pragma unroll
          for (int p = 0; p < EPV / 2; ++p) {
            const float y = x[2 * p] * cs[p] - x[2 * p + 1] * sn[p];
            x[2 * p + 1] = x[2 * p + 1] * cs[p] + x[2 * p] * sn[p];
            x[2 * p] = y;
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
          const float other = __shfl_sync(0xffffffffu, x[e], partner);
          if (turned) x[e] = x[e] * cs[e] + (low ? -other : other) * sn[e];
        }
      }
      if (r < H) {
        a.q_out[(int64_t(tok) * H + r) * LPR + c] = pack16(x);
      } else if (r < n_rows && cached) {
        if (r < H + K)
          a.k_pool[dst0 + (r - H) * head_step + c] = pack16(x);
        else
          a.v_pool[dst0 + (r - H - K) * head_step + c] = raw[u];
      }
    }
  }
}

template <typename T, int LPR, int kRows>
void launch_rows(const NormRopeArgs& a, bool interleaved, dim3 grid, cudaStream_t stream) {
  if (interleaved)
    norm_rope_append_kernel<T, LPR, kRows, true><<<grid, kThreads, 0, stream>>>(a);
  else
    norm_rope_append_kernel<T, LPR, kRows, false><<<grid, kThreads, 0, stream>>>(a);
}

// Rows in flight per lane group.
template <typename T, int LPR>
void launch(const NormRopeArgs& a, bool interleaved, cudaStream_t stream) {
  constexpr int kGroups = kThreads / LPR;
  const int64_t rows = int64_t(a.num_q_heads) + 2 * int64_t(a.num_kv_heads);
  const int64_t per_group = (rows + kGroups - 1) / kGroups;   // rows of a token per lane group, if one CTA takes it whole
  int k = 1;
  if (int64_t(a.num_tokens) * per_group > int64_t(kSpreadCtasPerSm) * cb::sm_count())
    k = per_group <= 1 ? 1 : per_group == 2 ? 2 : per_group == 3 ? 3 : per_group == 4 ? 4 : 6;
  const dim3 grid(unsigned(a.num_tokens), unsigned((rows + int64_t(k) * kGroups - 1) / (int64_t(k) * kGroups)));
  switch (k) {
    case 6: return launch_rows<T, LPR, 6>(a, interleaved, grid, stream);
    case 4: return launch_rows<T, LPR, 4>(a, interleaved, grid, stream);
    case 3: return launch_rows<T, LPR, 3>(a, interleaved, grid, stream);
    case 2: return launch_rows<T, LPR, 2>(a, interleaved, grid, stream);
    default: return launch_rows<T, LPR, 1>(a, interleaved, grid, stream);
  }
}

}  // namespace

extern "C" cb_status cb_norm_rope_append(const cb_norm_rope* in, int32_t num_q_heads, const int32_t* positions,
                                         const int64_t* slot_mapping, const int32_t* dims, int32_t num_tokens,
                                         const cb_kv_cache* cache, void* q_out, void* stream) {
  const char* who = "cb_norm_rope_append";
  cb::NvtxRange nvtx("cb.norm_rope_append");
  if (!in || !cache) return cb::fail(CB_ERR_INVALID, "%s: null argument", who);
  if (num_tokens < 0) return cb::fail(CB_ERR_INVALID, "%s: num_tokens < 0", who);
  if (num_q_heads < 1) return cb::fail(CB_ERR_INVALID, "%s: num_q_heads < 1", who);
  if (cache->num_blocks < 1 || cache->block_size < 1 || cache->num_heads < 1 || cache->head_dim < 1)
    return cb::fail(CB_ERR_INVALID, "%s: cache dimensions must be >= 1", who);
  if (cache->dtype != CB_DTYPE_BF16 && cache->dtype != CB_DTYPE_F32)
    return cb::fail(CB_ERR_UNSUPPORTED, "%s: unknown dtype", who);
  const bool bf16 = cache->dtype == CB_DTYPE_BF16;
  const int A = cache->head_dim, elem = bf16 ? 2 : 4, epv = 16 / elem;
  if (A != 64 && A != 128 && !(bf16 && A == 256))
    return cb::fail(CB_ERR_UNSUPPORTED, "%s: head_dim must be 64 or 128 (or 256 in bf16)", who);
  if (in->rot_dim < 0 || in->rot_dim > A || in->rot_dim % (2 * epv) != 0)
    return cb::fail(CB_ERR_UNSUPPORTED, "%s: rot_dim must be a multiple of %d up to head_dim", who, 2 * epv);
  if ((in->q_weight || in->k_weight) && !(in->eps >= 0.f && std::isfinite(in->eps)))
    return cb::fail(CB_ERR_INVALID, "%s: eps must be finite and >= 0", who);
  if (in->rot_dim > 0 && in->max_positions < 1) return cb::fail(CB_ERR_INVALID, "%s: max_positions < 1", who);
  if (int64_t(num_q_heads) + 2 * int64_t(cache->num_heads) > 65535 * 8)
    return cb::fail(CB_ERR_UNSUPPORTED, "%s: too many heads", who);
  if (num_tokens == 0) return CB_OK;
  if (!in->q || !in->k || !in->v || !slot_mapping || !q_out || !cache->k || !cache->v ||
      (in->rot_dim > 0 && (!in->cos_sin || !positions)))
    return cb::fail(CB_ERR_INVALID, "%s: null pointer", who);
  const int64_t q_row = int64_t(num_q_heads) * A, kv_row = int64_t(cache->num_heads) * A;
  if (in->q_stride < q_row || in->k_stride < kv_row || in->v_stride < kv_row)
    return cb::fail(CB_ERR_INVALID, "%s: a token stride is shorter than the token's heads", who);
  if (in->q_stride % epv || in->k_stride % epv || in->v_stride % epv)
    return cb::fail(CB_ERR_INVALID, "%s: token strides must be multiples of 16 bytes", who);
  const void* buffers[] = {in->q, in->k, in->v, q_out, cache->k, cache->v, in->q_weight, in->k_weight, in->cos_sin};
  for (const void* p : buffers)
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0)
      return cb::fail(CB_ERR_INVALID, "%s: buffers must be 16-byte aligned", who);
  unsigned* err = cb::device_error_word();
  if (!err) return CB_ERR_CUDA;

  NormRopeArgs a;
  a.q = in->q, a.k = in->k, a.v = in->v;
  a.q_stride = in->q_stride / epv, a.k_stride = in->k_stride / epv, a.v_stride = in->v_stride / epv;
  a.q_weight = in->q_weight, a.k_weight = in->k_weight;
  a.cos_sin = in->cos_sin;
  a.positions = positions;
  a.slots = slot_mapping;
  a.dims = dims;
  a.q_out = static_cast<uint4*>(q_out);
  a.k_pool = static_cast<uint4*>(cache->k);
  a.v_pool = static_cast<uint4*>(cache->v);
  a.num_slots = int64_t(cache->num_blocks) * cache->block_size;
  a.num_tokens = num_tokens;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = cache->num_heads;
  a.block_size = cache->block_size;
  a.max_positions = in->max_positions;
  a.rot_dim = in->rot_dim;
  a.eps = in->eps;
  a.err = err;
  const bool il = in->interleaved != 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (bf16 && A == 64) launch<__nv_bfloat16, 8>(a, il, st);
  else if (bf16 && A == 128) launch<__nv_bfloat16, 16>(a, il, st);
  else if (bf16) launch<__nv_bfloat16, 32>(a, il, st);
  else if (A == 64) launch<float, 16>(a, il, st);
  else launch<float, 32>(a, il, st);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cb::cuda_fail(e, "norm and rotation: launch");
  return CB_OK;
}
