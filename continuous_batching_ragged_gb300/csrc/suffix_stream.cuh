// The rows' own keys of a step with shared prefixes (bf16, head_dim 128).
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
//     mma.sync m16n8k16 steps, 32 of them per 8 KB of keys and values;
//   * a unit leaves its rows unnormalised, (acc, max, sum) in fp32, for the join;
//     a row with a single record is written to out at once.
// Large steps stream at 6.4 to 6.8 TB/s.  One of 114 us took 163 with 4 warps of 6
// stages, 112 with both 64-dim halves in one box; its loads alone take 104.
#pragma once

#include <cuda.h>

#include "device_common.cuh"
#include "shared_prefix.h"
#include "sm100_ptx.cuh"

namespace cb {
namespace stream {

using namespace sm100;

constexpr int kDim = kPrefixDim;
constexpr int kTileKeys = 16;
constexpr int kStages = 3;
constexpr uint32_t kBox = kTileKeys * 128;             // 16 keys x 64 dims, 128-byte rows: 2 KB; a TMA box is both halves
constexpr uint32_t kStageBytes = 4 * kBox;             // K and V, two 64-dim halves each
constexpr uint32_t kRingBytes = kStreamWarps * kStages * kStageBytes;
constexpr uint32_t kBarBytes = kStreamWarps * kStages * 8;
constexpr uint32_t kSlotBytes = kStreamWarps * 2 * sizeof(SuffixItem);

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, uint32_t bar, int32_t x, int32_t y, int32_t z,
                                            int32_t w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
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
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// A claimed unit, the same in every lane of its warp but for `z`; its item is in
// the warp's shared slot.
struct Unit {
  int n;                        // tiles; 0: no more work
  int hk;
  int issued;                   // tiles requested
  int zt, z;                    // lane i: TMA box index of tile zt + i
};

// A sequence of a small step, in shared memory: every CTA works the whole plan of
// such a step out for itself.
struct SmallSeq {
  int item0, nch;               // its first item, chunks
  int tok0, q_len, keys;
  unsigned rec0;
};
struct SmallStep {
  const SmallSeq* seqs;
  int num_seqs;
  int len;                      // tiles of a chunk
};

// One warp (0 .. kStreamWarps - 1 of its CTA).  `ring`, `bars` (initialised) and
// `slots` are the warp's own.  `first`: its first two units, `first` and
// first + step, are given rather than claimed; -1: claimed like the later ones,
// which start at `claimed_from`.  kSmall: the items are those of `small`, and all
// units are given, `step` apart.
template <bool kSmall>
__device__ __noinline__ void run_warp(const CUtensorMap* tm_k, const CUtensorMap* tm_v, const AttnArgs& a,
                                         const PrefixWork& w, int n_items, uint32_t ring, uint32_t bars,
                                         SuffixItem* slots, int first, int step, int claimed_from, const SmallStep small) {
  const int lane = threadIdx.x & 31;
  const int H = a.num_heads, Hkv = a.num_kv_heads, G = H / Hkv, B = a.block_size;
  const int n_units = n_items * Hkv;
  const int g = lane >> 2, t = lane & 3;                 // fragment row and column pair

  // pages of tiles zt .. zt + 31 of the unit in slot `sl`, one per lane
  auto load_pages = [&](Unit& u, const SuffixItem& it, int zt) {
    u.zt = zt;
    u.z = a.num_blocks * Hkv;                            // out of range: TMA fills zeros
    const int i = zt + lane;
    if (i < u.n) {
      const int blk = a.block_tables[size_t(it.s) * a.max_blocks_per_seq + it.skip + (it.k0 + i * kTileKeys) / B];
      if (blk >= 0 && blk < a.num_blocks) u.z = blk * Hkv + u.hk;
      else raise_error(a.err, kErrBounds);
    }
  };
  auto load_unit = [&](int idx, Unit& u, SuffixItem& it) {
    u.n = u.hk = u.issued = u.zt = u.z = 0;
    if (idx >= n_units) return;
    __syncwarp();                                        // every lane is done with the slot's last item
    if (kSmall) {
      const int item = idx / Hkv;
      int s = 0;                                         // the last sequence that starts at or before it
      for (int hi = small.num_seqs - 1; s < hi;) {
        const int mid = (s + hi + 1) >> 1;
        if (small.seqs[mid].item0 <= item) s = mid; else hi = mid - 1;
      }
      if (lane == 0) {
        const SmallSeq q = small.seqs[s];
        const int local = item - q.item0, row = local / q.nch, chunk = local - row * q.nch;
        SuffixItem x = {};
        x.s = s, x.tok0 = q.tok0, x.q_len = q.q_len, x.row0 = 16 * row, x.ctx = q.keys;
        x.k0 = chunk * small.len * kTileKeys;
        x.k1 = x.k0 + min(q.keys - x.k0, small.len * kTileKeys);
        x.rec0 = q.rec0 + chunk, x.rec_step = q.nch, x.direct = q.nch == 1;
        it = x;
      }
    } else if (lane < int(sizeof(SuffixItem) / 16)) {
      reinterpret_cast<int4*>(&it)[lane] = __ldcg(reinterpret_cast<const int4*>(w.items + idx / Hkv) + lane);
    }
    __syncwarp();
    u.hk = idx % Hkv;
    u.n = (it.k1 - it.k0 + kTileKeys - 1) / kTileKeys;
    load_pages(u, it, 0);
  };
  auto claim = [&]() -> int { return lane == 0 ? claimed_from + atomicAdd(w.header + 5, 1) : 0; };

  uint32_t issued = 0, consumed = 0;                     // ring positions
  auto issue = [&](Unit& u, const SuffixItem& it) {
    const int i = u.issued++;
    if (i - u.zt >= 32) load_pages(u, it, i);
    const int z = __shfl_sync(0xffffffffu, u.z, i - u.zt);
    if (lane == 0) {
      const int st = issued % kStages;
      const uint32_t dst = ring + st * kStageBytes, bar = bars + 8 * st;
      const int y = (it.k0 + i * kTileKeys) & (B - 1);
      mbar_arrive_expect_tx(bar, kStageBytes);
      tma_load_4d(dst, tm_k, bar, 0, y, 0, z);
      tma_load_4d(dst + 2 * kBox, tm_v, bar, 0, y, 0, z);
    }
    ++issued;
  };

  Unit cur, nxt;
  int slot = 0;                                          // of the current unit; the next one's is the other
  int given = first + step;                              // kSmall: the last unit taken
  {
    int c0 = first, c1 = first + step;
    if (first < 0) {
      if (lane == 0) c0 = claimed_from + atomicAdd(w.header + 5, 2);
      c0 = __shfl_sync(0xffffffffu, c0, 0);
      c1 = c0 + 1;
    }
    load_unit(c0, cur, slots[0]);
    load_unit(c1, nxt, slots[1]);
  }
  bool ok = true;
  const float sl2 = a.scale_log2;
  // this lane's part of an ldmatrix address: K as [key][dim], V transposed
  const int mi = lane >> 3, mr = lane & 7;
  const int k_row = (mi >> 1) * 8 + mr, v_row = (mi & 1) * 8 + mr;
  while (cur.n > 0) {
    const SuffixItem& it = slots[slot];
    auto top_up = [&]() {
      while (issued - consumed < uint32_t(kStages)) {
        if (cur.issued < cur.n) issue(cur, it);
        else if (nxt.issued < nxt.n) issue(nxt, slots[slot ^ 1]);
        else break;
      }
    };
    top_up();
    int ahead = n_units;
    if (kSmall) ahead = given = min(given, n_units) + step;
    else if (nxt.n > 0) ahead = claim();                 // for the unit after the next; read at this one's end
    // the unit's query rows, as A fragments; rows past the sequence's are zero
    const int rows = min(16, it.q_len * G - it.row0);
    uint32_t qf[8][4];
    {
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
      const int r0 = it.row0 + g, r1 = r0 + 8;
      const __nv_bfloat16* p0 = q + (size_t(it.tok0 + r0 / G) * H + cur.hk * G + r0 % G) * kDim + 2 * t;
      const __nv_bfloat16* p1 = q + (size_t(it.tok0 + r1 / G) * H + cur.hk * G + r1 % G) * kDim + 2 * t;
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
    const int k0 = it.k0, k1 = it.k1, ctx = it.ctx, before = ctx - it.q_len;
    const int lim0 = min(k1, before + (it.row0 + g) / G + 1), lim1 = min(k1, before + (it.row0 + g + 8) / G + 1);
    const int lim_all = min(k1, before + it.row0 / G + 1);   // keys that every row sees
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
      const int kb = k0 + i * kTileKeys;
      if (kb + kTileKeys > ctx) {                        // rows behind the sequence's last key: P is 0, but 0 * NaN is not
        const int from = ctx - kb;
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
      uint32_t pf[4];                                    // P, rounded to bf16 as in the pieces: half a step of a weight
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float p0 = ex2(fmaf(s[x][0], sl2, z0)), p1 = ex2(fmaf(s[x][1], sl2, z0));
        const float p2 = ex2(fmaf(s[x][2], sl2, z1)), p3 = ex2(fmaf(s[x][3], sl2, z1));
        l0 += p0 + p1;
        l1 += p2 + p3;
        pf[2 * x] = pack2(p0, p1);
        pf[2 * x + 1] = pack2(p2, p3);
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
          uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + (size_t(it.tok0 + tok) * H + h) * kDim) + t;
#pragma unroll
          for (int j = 0; j < 16; ++j) dst[4 * j] = pack2(o[j][2 * half] * inv, o[j][2 * half + 1] * inv);
        } else {
          const size_t at = size_t(it.rec0) + (size_t(tok) * H + h) * it.rec_step;
          float* rec = w.recs + at * kDim;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            __stcg(reinterpret_cast<float2*>(rec + 8 * j + 2 * t), make_float2(o[j][2 * half], o[j][2 * half + 1]));
          if (t == 0) __stcg(w.rec_ml + at, make_float2(m, l));
        }
      }
    }
    cur = nxt;
    load_unit(__shfl_sync(0xffffffffu, ahead, 0), nxt, slots[slot]);
    slot ^= 1;
  }
  if (!ok && lane == 0) raise_error(a.err, kErrTimeout | kSiteDecodeRing);
  // after a timeout some copies may still be in flight: wait for them (bounded) before exiting
  while (consumed < issued) {
    mbar_wait(bars + 8 * (consumed % kStages), (consumed / kStages) & 1);
    ++consumed;
  }
}

}  // namespace stream
}  // namespace cb
