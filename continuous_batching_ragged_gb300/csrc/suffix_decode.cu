// The rows' own keys of a step with shared prefixes, and the join of every
// row's records (bf16, head_dim 128).
//
// Behind a shared prefix a decoding sequence has few keys of its own: the work
// is many short streams, one per (sequence, key/value head), each read once
// for the G query heads of the key/value head.  It is bound by HBM, so the
// design aims at bytes in flight from the first to the last microsecond:
//   * every warp is a stream of its own.  It claims units (row tile of 16 query
//     rows, key/value head, chunk of keys), copies their K and V in 16-key
//     tiles by TMA (128-byte swizzled, so that the matrix loads below hit every
//     bank once) into a private ring, and runs on into its next unit's tiles
//     before the current one ends.  Nothing in the CTA waits for anything else,
//     and a unit's end costs one warp's stores, no ticket and no CTA barrier;
//   * 1 to 16 rows would leave a 64- or 128-row tcgen05 tile nearly empty and
//     its accumulator a round trip through tensor memory away.  Here the warp's
//     16 x 16 score tile and 16 x 128 output tile stay in registers between
//     mma.sync m16n8k16 steps: 32 of them per 8 KB of keys and values, an
//     eighth of what that path could issue in the time HBM needs for the bytes;
//   * a unit leaves its rows unnormalised, (acc, max, sum) in fp32; the join
//     kernel reads a row's records, those of its prefix and its own, with one
//     warp per row, 512 coalesced bytes a record:
//         out = sum_i 2^(m_i - M) acc_i / sum_i 2^(m_i - M) l_i,  M = max_i m_i,
//     in a fixed order, so a row's bits never depend on who finished first.  A
//     row with a single record is written to out at once.
#include <algorithm>
#include <mutex>

#include <cuda.h>

#include "device_common.cuh"
#include "runtime.h"
#include "shared_prefix.h"
#include "sm100_ptx.cuh"

namespace cb {
namespace {

using namespace sm100;

constexpr int HD = kPrefixDim;
constexpr int kTileKeys = 16;
constexpr int kStages = 3;
constexpr uint32_t kBox = kTileKeys * 128;             // 16 keys x 64 dims, 128-byte rows: 2 KB
constexpr uint32_t kStageBytes = 4 * kBox;             // K and V, two 64-dim halves each
constexpr int kThreads = kSuffixWarps * 32;
constexpr uint32_t kOffBars = kSuffixWarps * kStages * kStageBytes;
constexpr uint32_t kSmemBytes = kOffBars + kSuffixWarps * kStages * 8 + 1024;   // + slack to align the base
static_assert(kSmemBytes <= 232448, "shared memory budget");

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// D(16 x 8, fp32) += A(16 x 16) B(16 x 8), bf16
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// One claimed unit, the same in every lane of its warp.
struct Unit {
  SuffixItem it;
  int hk;
  int n;                        // tiles; 0: no more work
  int z;                        // lane i: TMA box index of tile zt + i
  int zt;
};

__global__ void __launch_bounds__(kThreads, 1)
    suffix_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const AttnArgs a,
                  const PrefixWork w) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;         // 128B-swizzled boxes repeat every 1 KB
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = base + warp * kStages * kStageBytes;
  const uint32_t bars = base + kOffBars + warp * kStages * 8;
  if (lane == 0) {
    for (int st = 0; st < kStages; ++st) mbar_init(bars + 8 * st, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  __syncwarp();
  // The plan is complete: the kernel before this one released its dependents
  // after waiting for it.  The join may be set up now; it waits for this grid.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int n_items = __ldcg(w.header + 4);
  if (uint32_t(__ldcg(w.header + 2)) != w.tag || n_items < 0 || n_items > w.item_cap) {
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(a.err, kErrInvalid);
    n_items = 0;
  }
  const int H = a.num_heads, Hkv = a.num_kv_heads, G = H / Hkv, B = a.block_size;
  const int64_t n_units = int64_t(n_items) * Hkv;
  const int g = lane >> 2, t = lane & 3;                 // fragment row and column pair

  // pages of tiles zt .. zt + 31 of the unit, one per lane
  auto load_pages = [&](Unit& u, int zt) {
    u.zt = zt;
    u.z = a.num_blocks * Hkv;                            // out of range: TMA fills zeros
    const int i = zt + lane;
    if (i < u.n) {
      const int blk = a.block_tables[size_t(u.it.s) * a.max_blocks_per_seq + u.it.skip + (u.it.k0 + i * kTileKeys) / B];
      if (blk >= 0 && blk < a.num_blocks) u.z = blk * Hkv + u.hk;
      else raise_error(a.err, kErrBounds);
    }
  };
  auto load_unit = [&](int64_t idx, Unit& u) {
    u.n = 0;
    u.hk = 0;
    u.z = u.zt = 0;
    if (idx >= n_units) return;
    const int4* src = reinterpret_cast<const int4*>(w.items + idx / Hkv);
    int4* dst = reinterpret_cast<int4*>(&u.it);
    dst[0] = __ldcg(src);
    dst[1] = __ldcg(src + 1);
    dst[2] = __ldcg(src + 2);
    u.hk = int(idx % Hkv);
    u.n = (u.it.k1 - u.it.k0 + kTileKeys - 1) / kTileKeys;
    load_pages(u, 0);
  };
  // Every warp's first two units are given (neighbouring units to different
  // SMs), the later ones are claimed.
  const int n_warps = int(gridDim.x) * kSuffixWarps, me = warp * int(gridDim.x) + int(blockIdx.x);
  auto claim = [&]() -> int { return lane == 0 ? 2 * n_warps + atomicAdd(w.header + 5, 1) : 0; };

  uint32_t issued = 0, consumed = 0;                     // ring positions
  auto issue = [&](Unit& u, int i) {
    if (i - u.zt >= 32) load_pages(u, i);
    const int z = __shfl_sync(0xffffffffu, u.z, i - u.zt);
    if (lane == 0) {
      const int st = issued % kStages;
      const uint32_t dst = ring + st * kStageBytes, bar = bars + 8 * st;
      const int y = (u.it.k0 + i * kTileKeys) % B;
      mbar_arrive_expect_tx(bar, kStageBytes);
      tma_load_3d(dst, &tm_k, bar, 0, y, z);
      tma_load_3d(dst + kBox, &tm_k, bar, 64, y, z);
      tma_load_3d(dst + 2 * kBox, &tm_v, bar, 0, y, z);
      tma_load_3d(dst + 3 * kBox, &tm_v, bar, 64, y, z);
    }
    ++issued;
  };

  Unit cur, nxt;
  load_unit(me, cur);
  load_unit(me + n_warps, nxt);
  int i_cur = 0, i_nxt = 0;                              // tiles issued
  bool ok = true;
  const float sl2 = a.scale_log2;
  // this lane's part of an ldmatrix address: K as [key][dim], V transposed
  const int mi = lane >> 3, mr = lane & 7;
  const int k_row = (mi >> 1) * 8 + mr, v_row = (mi & 1) * 8 + mr;
  while (cur.n > 0) {
    auto top_up = [&]() {
      while (issued - consumed < uint32_t(kStages)) {
        if (i_cur < cur.n) issue(cur, i_cur++);
        else if (i_nxt < nxt.n) issue(nxt, i_nxt++);
        else break;
      }
    };
    top_up();
    const int ahead = claim();                           // for the unit after the next; read at this one's end
    const SuffixItem& it = cur.it;
    // the unit's query rows, as A fragments; rows past the sequence's are zero
    const int rows = min(16, it.q_len * G - it.row0);
    uint32_t qf[8][4];
    {
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
      const int r0 = it.row0 + g, r1 = r0 + 8;
      const __nv_bfloat16* p0 = q + (size_t(it.tok0 + r0 / G) * H + cur.hk * G + r0 % G) * HD + 2 * t;
      const __nv_bfloat16* p1 = q + (size_t(it.tok0 + r1 / G) * H + cur.hk * G + r1 % G) * HD + 2 * t;
      const bool in0 = g < rows, in1 = g + 8 < rows;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        qf[ks][0] = in0 ? *reinterpret_cast<const uint32_t*>(p0 + 16 * ks) : 0u;
        qf[ks][1] = in1 ? *reinterpret_cast<const uint32_t*>(p1 + 16 * ks) : 0u;
        qf[ks][2] = in0 ? *reinterpret_cast<const uint32_t*>(p0 + 16 * ks + 8) : 0u;
        qf[ks][3] = in1 ? *reinterpret_cast<const uint32_t*>(p1 + 16 * ks + 8) : 0u;
      }
    }
    // keys that a row sees: all before its own token's, and its own
    const int first = it.ctx - it.q_len;
    const int lim0 = min(it.k1, first + (it.row0 + g) / G + 1), lim1 = min(it.k1, first + (it.row0 + g + 8) / G + 1);
    const int lim_all = min(it.k1, first + it.row0 / G + 1);   // keys that every row sees
    float o[16][4];
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    for (int i = 0; i < cur.n; ++i) {
      const int st = consumed % kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(bars + 8 * st, (consumed / kStages) & 1))) {
        ok = false;
        break;
      }
      const uint32_t kt = ring + st * kStageBytes, vt = kt + 2 * kBox;
      const int kb = it.k0 + i * kTileKeys;
      if (kb + kTileKeys > it.ctx) {                     // rows behind the sequence's last key: P is 0, but 0 * NaN is not
        const int from = it.ctx - kb;
        for (int c = lane; c < (kTileKeys - from) * 16; c += 32) {
          const int r = from + c / 16, ch = c % 16;
          asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(vt + (ch >> 3) * kBox + r * 128 + (ch & 7) * 16), "r"(0)
                       : "memory");
        }
        fence_proxy_async_smem();                        // before the slot's next TMA write
        __syncwarp();
      }
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        uint32_t kf[4];
        const int ch = (ks & 3) * 2 + (mi & 1);
        ldmatrix4(kt + (ks >> 2) * kBox + k_row * 128 + ((ch ^ mr) << 4), kf);
        mma_bf16(s[0], qf[ks], kf[0], kf[1]);
        mma_bf16(s[1], qf[ks], kf[2], kf[3]);
      }
      if (kb + kTileKeys > lim_all) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = kb + 8 * x + 2 * t + e;
            if (key >= lim0) s[x][e] = -INFINITY;
            if (key >= lim1) s[x][2 + e] = -INFINITY;
          }
      }
      float t0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
      float t1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
      // keep a stale maximum while 2^x stays <= 2^8
      if (__any_sync(0xffffffffu, t0 * sl2 > m0 + 8.0f || t1 * sl2 > m1 + 8.0f)) {
#pragma unroll
        for (int x = 1; x <= 2; x <<= 1) {
          t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, x));
          t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, x));
        }
        const float n0 = fmaxf(m0, t0 * sl2), n1 = fmaxf(m1, t1 * sl2);
        const float f0 = n0 == -INFINITY ? 1.f : ex2(m0 - n0), f1 = n1 == -INFINITY ? 1.f : ex2(m1 - n1);
        m0 = n0, m1 = n1;
        l0 *= f0, l1 *= f1;
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j][0] *= f0, o[j][1] *= f0, o[j][2] *= f1, o[j][3] *= f1;
      }
      const float z0 = m0 == -INFINITY ? 0.f : -m0, z1 = m1 == -INFINITY ? 0.f : -m1;   // a row that sees no key yet
      uint32_t pf[4];                                    // P, rounded to bf16 for the tensor core
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float p0 = ex2(fmaf(s[x][0], sl2, z0)), p1 = ex2(fmaf(s[x][1], sl2, z0));
        const float p2 = ex2(fmaf(s[x][2], sl2, z1)), p3 = ex2(fmaf(s[x][3], sl2, z1));
        l0 += p0 + p1;
        l1 += p2 + p3;
        pf[2 * x] = pack_bf16x2(p0, p1);
        pf[2 * x + 1] = pack_bf16x2(p2, p3);
      }
#pragma unroll
      for (int jj = 0; jj < 8; ++jj) {
        uint32_t vf[4];
        const int ch = (jj & 3) * 2 + (mi >> 1);
        ldmatrix4_trans(vt + (jj >> 2) * kBox + v_row * 128 + ((ch ^ mr) << 4), vf);
        mma_bf16(o[2 * jj], pf, vf[0], vf[1]);
        mma_bf16(o[2 * jj + 1], pf, vf[2], vf[3]);
      }
      __syncwarp();                                      // every lane has read the slot
      ++consumed;
      top_up();
    }
    if (!ok) break;
#pragma unroll
    for (int x = 1; x <= 2; x <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, x);
      l1 += __shfl_xor_sync(0xffffffffu, l1, x);
    }
    // the rows' records, or, with nothing to join, the rows
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (g + 8 * half < rows) {
        const int r = it.row0 + g + 8 * half, tok = r / G, h = cur.hk * G + r % G;
        const float m = half ? m1 : m0, l = half ? l1 : l0;
        if (it.direct) {
          const float inv = 1.0f / l;
          uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + (size_t(it.tok0 + tok) * H + h) * HD) + t;
#pragma unroll
          for (int j = 0; j < 16; ++j) dst[4 * j] = pack_bf16x2(o[j][2 * half] * inv, o[j][2 * half + 1] * inv);
        } else {
          float* rec = w.own_recs + (size_t(it.base) + (size_t(tok) * H + h) * it.nch + it.chunk) * kPrefixRec;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            __stcg(reinterpret_cast<float2*>(rec + 8 * j + 2 * t), make_float2(o[j][2 * half], o[j][2 * half + 1]));
          if (t == 0) __stcg(reinterpret_cast<float2*>(rec + HD), make_float2(m, l));
        }
      }
    }
    cur = nxt;
    i_cur = i_nxt;
    i_nxt = 0;
    load_unit(__shfl_sync(0xffffffffu, ahead, 0), nxt);
  }
  if (!ok && lane == 0) raise_error(a.err, kErrTimeout | kSiteDecodeRing);
  // after a timeout some copies may still be in flight: wait for them (bounded) before exiting
  while (consumed < issued) {
    mbar_wait(bars + 8 * (consumed % kStages), (consumed / kStages) & 1);
    ++consumed;
  }
  // this grid ends after the kernel before it, so whoever waits for this grid finds its records too
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// One warp per (token, query head).
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const AttnArgs a, const PrefixWork w) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t(blockIdx.x) * kJoinThreads + threadIdx.x) >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row >= int64_t(a.num_tokens) * a.num_heads || uint32_t(__ldcg(w.header + 2)) != w.tag) return;
  const int tok = int(row / a.num_heads), h = int(row - int64_t(tok) * a.num_heads);
  const int4 ti = __ldcg(w.token_info + tok);
  const int np = ti.x, n = np + ti.z;
  if (n < 2) return;                                     // left out, or already written
  const float* pre = w.recs + size_t(row) * __ldcg(w.header + 1) * kPrefixRec;
  const float* own = w.own_recs + (size_t(ti.y) + size_t(h) * ti.z) * kPrefixRec;
  auto rec = [&](int k) { return k < np ? pre + size_t(k) * kPrefixRec : own + size_t(k - np) * kPrefixRec; };
  float mx = -INFINITY;
  for (int k = lane; k < n; k += 32) mx = fmaxf(mx, __ldcg(rec(k) + HD));
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float den = 0.f;
#pragma unroll 4
  for (int k = 0; k < n; ++k) {
    const float* r = rec(k);
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(r + HD));
    const float4 x = __ldcg(reinterpret_cast<const float4*>(r) + lane);
    const float f = ex2(ml.x - mx);
    den = fmaf(f, ml.y, den);
    acc.x = fmaf(f, x.x, acc.x);
    acc.y = fmaf(f, x.y, acc.y);
    acc.z = fmaf(f, x.z, acc.z);
    acc.w = fmaf(f, x.w, acc.w);
  }
  const float inv = 1.0f / den;
  uint2 v;
  v.x = pack_bf16x2(acc.x * inv, acc.y * inv);
  v.y = pack_bf16x2(acc.z * inv, acc.w * inv);
  *(reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + size_t(row) * HD) + lane) = v;
}

std::mutex g_attr_mutex;
bool g_attr_set[64] = {};

}  // namespace

cb_status launch_suffix(const AttnArgs& a, const PrefixWork& w, cudaStream_t stream) {
  NvtxRange nvtx("cb.suffix");
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return CB_ERR_CUDA;
  CUtensorMap tk, tv;
  const cuuint32_t ones[3] = {1, 1, 1};
  const cuuint64_t dims[3] = {cuuint64_t(HD), cuuint64_t(a.block_size), cuuint64_t(a.num_blocks) * a.num_kv_heads};
  const cuuint64_t strides[2] = {cuuint64_t(HD) * 2, cuuint64_t(a.block_size) * HD * 2};
  const cuuint32_t box[3] = {64, kTileKeys, 1};
  for (int i = 0; i < 2; ++i) {
    CUresult r = enc(i ? &tv : &tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(i ? a.v_pool : a.k_pool), dims,
                     strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(CB_ERR_CUDA, "shared prefixes: encoding a KV tensor map failed (%d)", int(r));
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
    return fail(CB_ERR_UNSUPPORTED, "shared prefixes: no usable current device");
  {
    std::lock_guard<std::mutex> lock(g_attr_mutex);
    if (!g_attr_set[dev]) {
      cudaError_t e = cudaFuncSetAttribute(suffix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmemBytes));
      if (e != cudaSuccess) return cuda_fail(e, "shared prefixes: shared memory attribute");
      g_attr_set[dev] = true;
    }
  }
  const int64_t max_units = int64_t(w.item_cap) * a.num_kv_heads;
  const int64_t grid = std::min<int64_t>(sm_count(), (max_units + kSuffixWarps - 1) / kSuffixWarps);
  cudaError_t e = launch_kernel(suffix_kernel, dim3(unsigned(grid)), dim3(kThreads), kSmemBytes, stream, true, tk, tv, a, w);
  return e == cudaSuccess ? CB_OK : cuda_fail(e, "shared prefixes: own keys launch");
}

cb_status launch_join(const AttnArgs& a, const PrefixWork& w, cudaStream_t stream) {
  const int64_t rows = int64_t(a.num_tokens) * a.num_heads;
  const unsigned grid = unsigned((rows * 32 + kJoinThreads - 1) / kJoinThreads);
  cudaError_t e = launch_kernel(join_kernel, dim3(grid), dim3(kJoinThreads), 0, stream, true, a, w);
  return e == cudaSuccess ? CB_OK : cuda_fail(e, "shared prefixes: join launch");
}

}  // namespace cb
