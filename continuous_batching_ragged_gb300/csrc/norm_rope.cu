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
// Every row is read once and written once, but with a few dozen fp32 operations per
// 16 bytes in between it is issue slots (half of them taken) and loads in flight that
// bound a step of thousands of tokens, before HBM does.  So a group of LPR lanes
// holds one row, 16 bytes a lane: the mean is log2(LPR) shuffles, a lane's cosines,
// sines and weights are the same for every head of its token, and where the whole
// head turns a lane takes 8 bytes of each half, so that both elements of a pair are
// its own.  A persistent grid keeps the next token's rows (up to three per lane
// group) on their way while it works on one; a warp of values only copies.
// 2048 tokens of 32 + 2 * 32 heads, bf16: 21.0 us over several sets of inputs in turn,
// 4.8 TB/s; 18.5 us on one set, whose writes stay in L2 (57 of its 102 MB pass DRAM).
// On one set: one row per lane group 42 us; several rows 30; pairs in one lane and the
// next token in flight 24; values only copied 21.9; three CTAs an SM 18.9.  Back to
// back it was 20.8 before it could be launched while the kernel in front ends; released
// to its own successor early, 20.4: that one's CTAs then wait where its own would run.
#include <algorithm>
#include <cmath>

#include "device_common.cuh"
#include "runtime.h"

namespace {

using cb::Vec16;

constexpr int kThreads = 256;
constexpr int kSpreadCtasPerSm = 1;   // up to so many CTAs of one row per lane group, a token is spread over several
constexpr int kCtasPerSm = 3;         // 80 registers a thread; 2 and 4 were slower (2048 tokens: 21.9, 21.4 against 18.9 us)

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

// How a lane's 16 bytes of a row lie, and where its pairs are.
enum RopeMode {
  kHalves,       // rot_dim = head_dim, pairs (i, i + A / 2): 8 bytes of each half, so a lane has whole pairs
  kPartial,      // pairs (i, i + rot_dim / 2): 16 bytes in order, the other element is in another lane
  kInterleaved   // pairs (2i, 2i + 1): 16 bytes in order
};

// blockIdx.y takes kRows rows per lane group of the token's num_q_heads query,
// num_kv_heads key and num_kv_heads value rows, in that order; blockIdx.x
// strides over tokens, the next token's rows already on their way while one is
// worked on.
template <typename T, int LPR, int kRows, int MODE>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) norm_rope_append_kernel(const NormRopeArgs a) {
  constexpr int EPV = Vec16<T>::N;              // elements per lane
  constexpr int A = LPR * EPV;                  // head_dim
  constexpr int kGroups = kThreads / LPR;       // rows side by side in the CTA
  constexpr int kTab = MODE == kPartial ? EPV : EPV / 2;   // cosines (and sines) that a lane needs
  asm volatile("griddepcontrol.wait;" ::: "memory");       // it may start while the stream's last kernel ends
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
  const int c = threadIdx.x % LPR;              // this lane's part of the row
  const int H = a.num_q_heads, K = a.num_kv_heads, n_rows = H + 2 * K;
  const int row0 = (blockIdx.y * kRows) * kGroups + threadIdx.x / LPR;
  const int half = a.rot_dim / 2;
  const bool turned = MODE == kHalves || c * EPV < a.rot_dim;   // rot_dim is a multiple of 2 * EPV: a lane turns all or nothing
  const bool low = c * EPV < half;              // kPartial: element d of the first half pairs with d + rot_dim / 2
  const int partner = MODE == kPartial && turned ? lane + (low ? 1 : -1) * (half / EPV) : lane;
  const int d0 = MODE == kPartial ? (low ? c * EPV : c * EPV - half) : c * (EPV / 2);   // its first table entry

  auto load16 = [&](const uint4* row) -> uint4 {
    if constexpr (MODE != kHalves) return row[c];
    const uint2* r = reinterpret_cast<const uint2*>(row);
    const uint2 x = r[c], y = r[LPR + c];
    return make_uint4(x.x, x.y, y.x, y.y);
  };
  auto store16 = [&](uint4* row, const uint4& v) {
    if constexpr (MODE != kHalves) {
      row[c] = v;
    } else {
      uint2* r = reinterpret_cast<uint2*>(row);
      r[c] = make_uint2(v.x, v.y);
      r[LPR + c] = make_uint2(v.z, v.w);
    }
  };
  auto load_rows = [&](int tok, uint4 (&raw)[kRows]) {
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int r = row0 + u * kGroups;
      const uint4* src = r < H       ? static_cast<const uint4*>(a.q) + tok * a.q_stride + int64_t(r) * LPR
                         : r < H + K ? static_cast<const uint4*>(a.k) + tok * a.k_stride + int64_t(r - H) * LPR
                                     : static_cast<const uint4*>(a.v) + tok * a.v_stride + int64_t(r - H - K) * LPR;
      raw[u] = r < n_rows ? load16(src) : make_uint4(0, 0, 0, 0);
    }
  };

  int tok = blockIdx.x;
  if (tok >= n_tok) return;
  uint4 next[kRows];
  load_rows(tok, next);
  int64_t next_slot = a.slots[tok];
  int next_pos = a.rot_dim > 0 ? a.positions[tok] : 0;
  const uint4 wq = a.q_weight ? load16(static_cast<const uint4*>(a.q_weight)) : make_uint4(0, 0, 0, 0);
  const uint4 wk = a.k_weight ? load16(static_cast<const uint4*>(a.k_weight)) : make_uint4(0, 0, 0, 0);

  for (; tok < n_tok; tok += gridDim.x) {
    uint4 raw[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) raw[u] = next[u];
    const int64_t slot = next_slot;
    const int pos = next_pos;
    const bool skip = a.rot_dim > 0 && (pos < 0 || pos >= a.max_positions);
    float cs[kTab], sn[kTab];
    if (a.rot_dim > 0 && !skip && turned) {
      const float* tab = a.cos_sin + int64_t(pos) * a.rot_dim + d0;
#pragma unroll
      for (int e = 0; e < kTab; e += 2) {       // 8 bytes each: merged to 16 where they are aligned
        const float2 x = __ldg(reinterpret_cast<const float2*>(tab + e));
        const float2 y = __ldg(reinterpret_cast<const float2*>(tab + half + e));
        cs[e] = x.x, cs[e + 1] = x.y, sn[e] = y.x, sn[e + 1] = y.y;
      }
    } else {
#pragma unroll
      for (int e = 0; e < kTab; ++e) cs[e] = 1.f, sn[e] = 0.f;
    }
    if (tok + int(gridDim.x) < n_tok) {
      const int t = tok + gridDim.x;
      load_rows(t, next);
      next_slot = a.slots[t];
      next_pos = a.rot_dim > 0 ? a.positions[t] : 0;
    }
    if (skip) {                                 // the same for the whole CTA
      if (threadIdx.x == 0 && blockIdx.y == 0) cb::raise_error(a.err, cb::kErrBounds);
      continue;
    }
    const bool bad_slot = slot >= a.num_slots;
    if (bad_slot && threadIdx.x == 0 && blockIdx.y == 0) cb::raise_error(a.err, cb::kErrBounds);
    const bool cached = slot >= 0 && !bad_slot;
    const int64_t blk = cached ? slot / a.block_size : 0, off = cached ? slot - blk * a.block_size : 0;
    const int64_t dst0 = (blk * K * a.block_size + off) * LPR, head_step = int64_t(a.block_size) * LPR;
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int r = row0 + u * kGroups;
      if (!__any_sync(0xffffffffu, r < H + K)) {  // values only: nothing to compute
        if (r < n_rows && cached) store16(a.v_pool + dst0 + (r - H - K) * head_step, raw[u]);
        continue;
      }
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
        float wt[EPV];
        Vec16<T>::to_float(is_q ? wq : wk, wt);
#pragma unroll
        for (int e = 0; e < EPV; ++e) x[e] = x[e] * inv * wt[e];
      }
      if constexpr (MODE == kPartial) {
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
          const float other = __shfl_sync(0xffffffffu, x[e], partner);
          if (turned) x[e] = x[e] * cs[e] + (low ? -other : other) * sn[e];
        }
      } else if (turned) {
#pragma unroll
        for (int p = 0; p < EPV / 2; ++p) {
          const int i = MODE == kHalves ? p : 2 * p, j = MODE == kHalves ? p + EPV / 2 : 2 * p + 1;
          const float y = x[i] * cs[p] - x[j] * sn[p];
          x[j] = x[j] * cs[p] + x[i] * sn[p];
          x[i] = y;
        }
      }
      if (r < H) {
        store16(a.q_out + (int64_t(tok) * H + r) * LPR, pack16(x));
      } else if (r < n_rows && cached) {
        if (r < H + K)
          store16(a.k_pool + dst0 + (r - H) * head_step, pack16(x));
        else
          store16(a.v_pool + dst0 + (r - H - K) * head_step, raw[u]);
      }
    }
  }
}

template <typename T, int LPR, int kRows>
cudaError_t launch_rows(const NormRopeArgs& a, bool interleaved, unsigned chunks, cudaStream_t stream) {
  const int64_t ctas = std::max<int64_t>(1, int64_t(kCtasPerSm) * cb::sm_count() / chunks);
  const dim3 grid(unsigned(std::min<int64_t>(a.num_tokens, ctas)), chunks);
  auto kernel = interleaved                         ? norm_rope_append_kernel<T, LPR, kRows, kInterleaved>
                : a.rot_dim == LPR * Vec16<T>::N ? norm_rope_append_kernel<T, LPR, kRows, kHalves>
                                                 : norm_rope_append_kernel<T, LPR, kRows, kPartial>;
  return cb::launch_kernel(kernel, grid, dim3(kThreads), 0, stream, true, a);
}

// Rows in flight per lane group: as many as a token has for each, where there are
// tokens enough to fill the GPU that way.
template <typename T, int LPR>
cudaError_t launch(const NormRopeArgs& a, bool interleaved, cudaStream_t stream) {
  constexpr int kGroups = kThreads / LPR;
  const int64_t rows = int64_t(a.num_q_heads) + 2 * int64_t(a.num_kv_heads);
  const int64_t per_group = (rows + kGroups - 1) / kGroups;
  int k = 1;
  if (int64_t(a.num_tokens) * per_group > int64_t(kSpreadCtasPerSm) * cb::sm_count())
    k = per_group <= 1 ? 1 : per_group % 3 != 0 && per_group % 2 == 0 ? 2 : 3;
  const unsigned chunks = unsigned((rows + int64_t(k) * kGroups - 1) / (int64_t(k) * kGroups));
  switch (k) {
    case 3: return launch_rows<T, LPR, 3>(a, interleaved, chunks, stream);
    case 2: return launch_rows<T, LPR, 2>(a, interleaved, chunks, stream);
    default: return launch_rows<T, LPR, 1>(a, interleaved, chunks, stream);
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
  const cudaError_t e = bf16 && A == 64    ? launch<__nv_bfloat16, 8>(a, il, st)
                        : bf16 && A == 128 ? launch<__nv_bfloat16, 16>(a, il, st)
                        : bf16             ? launch<__nv_bfloat16, 32>(a, il, st)
                        : A == 64          ? launch<float, 16>(a, il, st)
                                           : launch<float, 32>(a, il, st);
  if (e != cudaSuccess) return cb::cuda_fail(e, "norm and rotation: launch");
  return CB_OK;
}
