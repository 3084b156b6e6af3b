// Streams of single warps (suffix_stream.cuh) over a cache in 8 bits: e4m3 keys
// and values, a fp32 scale for each block and head.
//
// A tile is 16 keys of one block: 2 KB of keys and 2 KB of values by TMA, and the
// block's two scales by a 4-byte asynchronous copy each, all on the tile's barrier.
//   * Half the bytes a key leave half the time for its arithmetic: it is latency and
//     instructions that bound a stream, before HBM does.  So keys and dims are the 16
//     rows of the matrix steps (m16n8k16), S^T = K Q^T and O^T = V^T P^T, and the query
//     rows their 8 columns, in NT sets: a key's bytes are converted once for all rows,
//     and up to 8 rows (a decoding sequence's query heads of one key/value head) take
//     half the steps, registers and exponentials that 16 would.
//   * e4m3 numbers are exact in f16, so the matrix steps are f16's.  A query row is
//     scaled by a power of two that brings its largest number to 2^13 .. 2^14: its
//     bf16 numbers are then exact in f16 down to 2^-27 of that, and off by at most
//     2^-38 of it below.
//   * ldmatrix moves pairs of bytes as its 16-bit numbers.  For the scores a lane
//     gets four neighbouring dims of its key, and both operands take the dims of a
//     step in that order; for the output it gets two dims of two keys, one byte
//     permutation makes them two pairs of keys, and even and odd dims are the upper
//     and lower rows of a step.
//   * A block's key scale multiplies its scores.  Its value scale vs multiplies the
//     weights, of which the tensor core takes 11 bits and 2^-24 .. 2^16 in f16: so a
//     row keeps, beside its running maximum m of the scores (exp2 domain), the running
//     maximum M of score + log2(vs); the output's weights 2^(s - M) vs are at most
//     2^8 (stale maxima are kept as long as that holds), while the sum, in fp32, stays
//     that of 2^(s - m).
// Measured: 256 rows of 32 heads over 4096 keys 711 to 727 us, 0.98 to 1.0 of the copy
// rate; 201 rows, 32/8 heads, 152 to 155 us, 0.92; 140 rows of 32 heads on one 45 us, of
// which 12 are its bytes' and 17 a step's least time with its join: 8 warps an SM, and of
// a tile's instructions each waits for the last (issue 37 %, DRAM 26 %).
#pragma once

#include "e4m3.cuh"
#include "suffix_stream.cuh"

namespace cb {
namespace qstream {

using namespace sm100;
using stream::kDim;
using stream::kTileKeys;
using stream::ldmatrix4;
using stream::ldmatrix4_trans;
using stream::pack2;
using stream::Unit;

constexpr uint32_t kBox = kTileKeys * kDim;            // 2 KB, rows of 128 bytes, 128-byte swizzled
constexpr uint32_t kStageBytes = 2 * kBox;
constexpr int kBarArrivals = 3;                        // of a stage: the copies' bytes, and either scale

// Warps of a CTA, and 192 KB of tiles in flight.  Two tiles an iteration: more independent work between one matrix step and
// the next, and half the barriers' and maxima's part of it (256 rows of 32 heads at 4096 keys: 777 us one at a time, 727 so).
// 16 warps take 128 registers each, which hides most latency where streams are long and HBM bounds them (727 us; 12 warps 768);
// 12 warps start and end sooner (4 rows at 512 keys 8.7 us and, with 16, 9.5, 64 rows behind a shared prompt 37.3 and 39.3).  With 16 rows
// a unit 8 warps of 231 registers (140 rows of 32 heads on one: 44.9 us; 12 warps, which spill: 53.4).
template <int NT, int WARPS>
struct Shape {
  static constexpr int kSets = NT;
  static constexpr int kWarps = WARPS;
  static constexpr int kStages = 48 / kWarps;
  static constexpr int kAtOnce = 2;                    // tiles of an iteration
  static constexpr int kRows = 8 * NT;                 // query rows of a unit, at most
  static constexpr int kThreads = 32 * kWarps;
  static constexpr uint32_t kRingBytes = kWarps * kStages * kStageBytes;
  static constexpr uint32_t kWarpBarBytes = kStages * 16;   // barriers, then (key, value) scales of each stage
  static constexpr uint32_t kSlotBytes = kWarps * 2 * sizeof(SuffixItem);
  static constexpr uint32_t kOffBars = kRingBytes;
  static constexpr uint32_t kOffSlots = kOffBars + kWarps * kWarpBarBytes;
  static constexpr uint32_t kSmem = kOffSlots + kSlotBytes + 1024;   // + slack to align the ring
  static_assert(48 % kWarps == 0 && kStages >= kAtOnce && kOffSlots % 16 == 0 && kSmem <= 220 * 1024, "shared memory");
};
using SharesShape = Shape<1, 16>;                      // up to 8 rows, all tiles of a step dealt out
using FewShape = Shape<1, 12>;                         // up to 8 rows, a CTA to a stream, or listed units
using WideShape = Shape<2, 8>;                         // up to 16 rows

__device__ __forceinline__ void copy4_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives on `bar` once this thread's asynchronous copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}
// D(16 x 8, fp32) += A(16 x 16) B(16 x 8), f16
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Lane (g, t) gives row g, columns 2t and 2t + 1 of an 8 x 8 matrix and gets those of its transpose.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

// Where a warp's units come from: take() describes the next one in `it` (the warp is in step before and after) and
// returns its key/value head and tiles, no tiles if there is none; ahead() is called at a unit's beginning.
struct Taken {
  int hk, n;
};
__device__ __forceinline__ int tiles_of(const SuffixItem& it) { return (it.k1 - it.k0 + kTileKeys - 1) / kTileKeys; }

// Units (item, key/value head) that a plan kernel listed, all claimed: which CTAs start first is open.
struct ListedUnits {
  const PrefixWork& w;
  int kv_heads, n_units;
  int first = -1, given = 0, claimed = 0;   // the first two are claimed at once

  __device__ __forceinline__ void ahead(int lane, bool more) {
    claimed = n_units;
    if (more && lane == 0) claimed = atomicAdd(w.header + 5, 1);
  }
  __device__ __forceinline__ Taken take(SuffixItem& it, int lane) {
    if (first < 0) first = __shfl_sync(0xffffffffu, lane == 0 ? atomicAdd(w.header + 5, 2) : 0, 0);
    const int idx = given < 2 ? first + given++ : __shfl_sync(0xffffffffu, claimed, 0);
    if (idx >= n_units) return {0, 0};
    if (lane < int(sizeof(SuffixItem) / 16))
      reinterpret_cast<int4*>(&it)[lane] = __ldcg(reinterpret_cast<const int4*>(w.items + idx / kv_heads) + lane);
    __syncwarp();
    return {idx % kv_heads, tiles_of(it)};
  }
};

// A sequence of a step that every CTA plans for itself.  Its streams, one per (row tile, key/value head), are `tiles`
// tiles each, laid end to end from `off`; those of the sequences follow one another.
struct RangeSeq {
  int off, tiles;
  int stream0;                          // streams of the sequences before
  int tok0, q_len, keys;
};
// The warp's share of all tiles, [pos, end).  A stream that lies in several shares leaves a record of each row in each of
// them: a share begins and ends with at most one such part, so its records are rec0 .. rec0 + row_tile - 1 and the row_tile
// behind.
struct RangeUnits {
  const RangeSeq* seqs;
  int num_seqs, kv_heads, row_tile;
  int pos, end;
  unsigned rec0;
  bool begun = false;

  __device__ __forceinline__ void ahead(int, bool) {}
  __device__ __forceinline__ Taken take(SuffixItem& it, int lane) {
    if (pos >= end) return {0, 0};
    int s = 0;                          // the last sequence that starts at or before it; ones without tiles come before
    for (int hi = num_seqs - 1; s < hi;) {
      const int mid = (s + hi + 1) >> 1;
      if (seqs[mid].off <= pos) s = mid; else hi = mid - 1;
    }
    const RangeSeq q = seqs[s];
    const int local = pos - q.off, x = local / q.tiles, t0 = local - x * q.tiles, n = min(q.tiles - t0, end - pos);
    if (lane == 0) {
      SuffixItem u = {};
      u.s = s, u.tok0 = q.tok0, u.q_len = q.q_len, u.row0 = x / kv_heads * row_tile, u.ctx = q.keys;
      u.k0 = t0 * kTileKeys, u.k1 = min(q.keys, (t0 + n) * kTileKeys);
      u.direct = n == q.tiles;
      u.rec0 = rec0 + (begun ? row_tile : 0);
      it = u;
    }
    begun = true;
    pos += n;
    __syncwarp();
    return {x % kv_heads, n};
  }
};

// One warp.  `ring` and `slots` are its own, so are `bars`: kStages barriers (initialised for kBarArrivals), then kStages
// pairs of scales, which `scales` points to.
template <class Sh, class Units>
__device__ __forceinline__ void run_warp(const CUtensorMap* tm_k, const CUtensorMap* tm_v, const AttnArgs& a, float* recs,
                                         float2* rec_ml, uint32_t ring, uint32_t bars, const volatile float2* scales,
                                         SuffixItem* slots, Units& units) {
  constexpr int NT = Sh::kSets, kStages = Sh::kStages, kRows = Sh::kRows, kAtOnce = Sh::kAtOnce;
  const int lane = threadIdx.x & 31;
  const int H = a.num_heads, Hkv = a.num_kv_heads, G = H / Hkv, B = a.block_size;
  const int boxes = a.num_blocks * Hkv;
  const int g = lane >> 2, t = lane & 3;                 // fragment row and column pair
  const uint32_t scale_at = bars + 8 * kStages;

  // pages of tiles zt .. zt + 31 of a unit, one per lane
  auto load_pages = [&](const SuffixItem& it, int hk, int n, int zt) -> int {
    const int i = zt + lane;
    if (i >= n) return boxes;                            // out of range: TMA fills zeros
    const int blk = a.block_tables[size_t(it.s) * a.max_blocks_per_seq + it.skip + (it.k0 + i * kTileKeys) / B];
    if (blk >= 0 && blk < a.num_blocks) return blk * Hkv + hk;
    raise_error(a.err, kErrBounds);
    return boxes;
  };
  auto load_unit = [&](Unit& u, SuffixItem& it) {
    __syncwarp();                                        // every lane is done with the slot's last item
    const Taken next = units.take(it, lane);
    u.n = next.n, u.hk = next.hk;
    u.issued = u.zt = u.z = 0;
    if (u.n > 0) u.z = load_pages(it, u.hk, u.n, 0);
  };

  uint32_t issued = 0, consumed = 0;                     // ring positions
  int st_in = 0, st_out = 0;                             // their stages
  uint32_t phase = 0;                                    // of st_out

  Unit cur, nxt;
  int slot = 0;                                          // of the current unit; the next one's is the other
  load_unit(cur, slots[0]);
  load_unit(nxt, slots[1]);
  // Requests tiles of the current unit, then of the next, while stages are free.
  auto top_up = [&]() {
    while (issued - consumed < uint32_t(kStages)) {
      const bool ahead = cur.issued >= cur.n;
      if (ahead && nxt.issued >= nxt.n) break;
      const SuffixItem& it = slots[slot ^ int(ahead)];
      const int i = ahead ? nxt.issued : cur.issued;
      int zt = ahead ? nxt.zt : cur.zt, zs = ahead ? nxt.z : cur.z;
      if (i - zt >= 32) {
        zt = i;
        zs = load_pages(it, ahead ? nxt.hk : cur.hk, ahead ? nxt.n : cur.n, i);
        if (ahead) nxt.zt = zt, nxt.z = zs;
        else cur.zt = zt, cur.z = zs;
      }
      if (ahead) ++nxt.issued;
      else ++cur.issued;
      const int z = __shfl_sync(0xffffffffu, zs, i - zt);
      const uint32_t bar = bars + 8 * st_in;
      if (lane < 2) {
        copy4_async(scale_at + 8 * st_in + 4 * lane, (lane == 0 ? a.k_scale : a.v_scale) + (z < boxes ? z : 0));
        copies_arrive(bar);
      }
      if (lane == 0) {
        const uint32_t dst = ring + st_in * kStageBytes;
        const int y = (it.k0 + i * kTileKeys) & (B - 1);
        mbar_arrive_expect_tx(bar, kStageBytes);
        tma_load_3d(dst, tm_k, bar, 0, y, z);
        tma_load_3d(dst + kBox, tm_v, bar, 0, y, z);
      }
      ++issued;
      st_in = st_in + 1 == kStages ? 0 : st_in + 1;
    }
  };
  bool ok = true;
  // This lane's row in a tile's ldmatrix: four 8 x 16-byte matrices, of the keys' halves and two chunks of 16 dims; the j-th
  // pair of chunks is at `part ^ 32 * j`.
  const int mi = lane >> 3, mr = lane & 7;
  const uint32_t part = ((mi & 1) * 8 + mr) * 128 + (((mi >> 1) ^ mr) << 4);
  while (cur.n > 0) {
    const SuffixItem& it = slots[slot];
    top_up();
    units.ahead(lane, nxt.n > 0);                        // for the unit after the next, taken at this one's end
    // The unit's query rows as B fragments in f16 (columns past the sequence's are zero), and of this lane's two
    // columns per set the factor of a score without its block's scale, and the keys that the row sees: all before
    // its own token's, and its own.
    const int rows = min(kRows, it.q_len * G - it.row0);
    const int k0 = it.k0, k1 = it.k1, ctx = it.ctx, before = ctx - it.q_len;
    const int lim_all = min(k1, before + it.row0 / G + 1);   // keys that every row sees
    uint32_t qf[NT][8][2];
    float ef[NT][2];
    int lim[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = it.row0 + 8 * n + g;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + (size_t(it.tok0 + r / G) * H + cur.hk * G + r % G) * kDim + 4 * t;
      const bool in = 8 * n + g < rows;
      uint32_t top = 0;                                  // bits of the largest magnitude
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const uint2 x = in ? *reinterpret_cast<const uint2*>(src + 16 * ks) : make_uint2(0, 0);
        qf[n][ks][0] = x.x, qf[n][ks][1] = x.y;
        top = max(max(top, (x.x << 16) & 0x7fff0000u), max(x.x & 0x7fff0000u, max((x.y << 16) & 0x7fff0000u, x.y & 0x7fff0000u)));
      }
#pragma unroll
      for (int x = 1; x <= 2; x <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, x));
      const uint32_t ex = min(253u, 267u - (top >> 23));     // 2^13 / largest, as an exponent; its inverse is an ordinary number
      const float f = __uint_as_float(ex << 23), back = a.scale_log2 * __uint_as_float((254u - ex) << 23);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        qf[n][ks][0] = pack_f16(bf16_lo(qf[n][ks][0]) * f, bf16_hi(qf[n][ks][0]) * f);
        qf[n][ks][1] = pack_f16(bf16_lo(qf[n][ks][1]) * f, bf16_hi(qf[n][ks][1]) * f);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        ef[n][e] = __shfl_sync(0xffffffffu, back, 4 * (2 * t + e));
        lim[n][e] = min(k1, before + (it.row0 + 8 * n + 2 * t + e) / G + 1);
      }
    }
    float o[NT][8][4];                                   // [chunk of 16 dims]: dim 2g of rows 2t, 2t + 1, dim 2g + 1 of them
    // of rows 2t and 2t + 1 of each set: m, l, M and 2^(m - M)
    float m[NT][2], l[NT][2], mw[NT][2], fw[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) m[n][e] = mw[n][e] = -INFINITY, l[n][e] = 0.f, fw[n][e] = 1.f;
    }
    // Tiles i .. i + U - 1 of the unit; false after a timeout.
    auto tiles = [&](auto U_, int i) -> bool {
      constexpr int U = decltype(U_)::value;
      uint32_t kt[U];
      float ks[U], vs[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!__all_sync(0xffffffffu, mbar_wait(bars + 8 * st_out, phase))) {
          consumed += u;                                 // for the waits at the end
          return false;
        }
        ks[u] = scales[st_out].x, vs[u] = scales[st_out].y;
        kt[u] = ring + st_out * kStageBytes;
        if (++st_out == kStages) st_out = 0, phase ^= 1;
      }
      const int kb = k0 + i * kTileKeys;
      if (kb + U * kTileKeys > ctx) {                    // rows behind the sequence's last key: P is 0, but 0 * NaN is not
        const int from = ctx - kb - (U - 1) * kTileKeys;   // of the last tile, which has a key
        for (int c = lane; c < (kTileKeys - from) * 8; c += 32)
          asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(kt[U - 1] + kBox + (from + c / 8) * 128 + (c % 8) * 16), "r"(0)
                       : "memory");
        fence_proxy_async_smem();                        // before the slot's next TMA write
        __syncwarp();
      }
      float s[U][NT][4];                                 // keys g: rows 2t, 2t + 1; keys 8 + g
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n) s[u][n][0] = s[u][n][1] = s[u][n][2] = s[u][n][3] = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          uint32_t kf[4];
          ldmatrix4(kt[u] + (part ^ (32 * j)), kf);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t a0 = e4m3x2_to_f16x2(kf[2 * x]), a1 = e4m3x2_to_f16x2(kf[2 * x + 1]);
            const uint32_t a2 = e4m3x2_hi_to_f16x2(kf[2 * x]), a3 = e4m3x2_hi_to_f16x2(kf[2 * x + 1]);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(s[u][n], a0, a1, a2, a3, qf[n][2 * j + x][0], qf[n][2 * j + x][1]);
          }
        }
      if (kb + U * kTileKeys > lim_all) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (kb + u * kTileKeys + g >= lim[n][e]) s[u][n][e] = -INFINITY;
              if (kb + u * kTileKeys + 8 + g >= lim[n][e]) s[u][n][2 + e] = -INFINITY;
            }
      }
      float lv[U], af[U][NT][2], top[NT][2], topw[NT][2];
      bool grown = false;
#pragma unroll
      for (int u = 0; u < U; ++u) lv[u] = fmaxf(lg2(vs[u]), -126.f);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[n][e] = topw[n][e] = -INFINITY;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            af[u][n][e] = fmaxf(ef[n][e] * ks[u], 1.2e-38f);   // not 0: -inf stays
            const float x = fmaxf(s[u][n][e], s[u][n][2 + e]) * af[u][n][e];
            top[n][e] = fmaxf(top[n][e], x), topw[n][e] = fmaxf(topw[n][e], x + lv[u]);
          }
          grown = grown || top[n][e] > m[n][e] + 8.0f || topw[n][e] > mw[n][e] + 8.0f;
        }
      if (__any_sync(0xffffffffu, grown)) {              // stale maxima are kept while 2^x stays <= 2^8
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = top[n][e], y = topw[n][e];
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) {
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
              y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
            }
            x = fmaf(fabsf(x), 0x1p-22f, x), y = fmaf(fabsf(y), 0x1p-22f, y);   // above what fma makes of the scores
            const float to = fmaxf(m[n][e], x), tw = fmaxf(mw[n][e], y);
            if (to != -INFINITY) {                       // the row has seen a key
              l[n][e] *= ex2(m[n][e] - to);
              const float f = ex2(mw[n][e] - tw);
#pragma unroll
              for (int j = 0; j < 8; ++j) o[n][j][e] *= f, o[n][j][2 + e] *= f;
              fw[n][e] = ex2(fminf(to - tw, 126.f));
            }
            m[n][e] = to, mw[n][e] = tw;
          }
      }
      uint32_t pf[U][NT][2];                             // weights in f16: within 2^-11 of each, 2^-25 of 2^(M - m)
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float z = m[n][e] == -INFINITY ? 0.f : -m[n][e], c = fminf(vs[u] * fw[n][e], 3e38f);
            const float x = ex2(fmaf(s[u][n][e], af[u][n][e], z)), y = ex2(fmaf(s[u][n][2 + e], af[u][n][e], z));
            l[n][e] += x + y;
            p[e] = x * c, p[2 + e] = y * c;
          }
          pf[u][n][0] = transpose8(pack_f16(p[0], p[1]));
          pf[u][n][1] = transpose8(pack_f16(p[2], p[3]));
        }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          uint32_t vf[4];
          ldmatrix4_trans(kt[u] + kBox + (part ^ (32 * j)), vf);
#pragma unroll
          for (int x = 0; x < 4; ++x) vf[x] = __byte_perm(vf[x], 0, 0x3120);   // (key, key + 1) of the even dim, of the odd dim
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t a0 = e4m3x2_to_f16x2(vf[2 * x]), a1 = e4m3x2_hi_to_f16x2(vf[2 * x]);
            const uint32_t a2 = e4m3x2_to_f16x2(vf[2 * x + 1]), a3 = e4m3x2_hi_to_f16x2(vf[2 * x + 1]);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(o[n][2 * j + x], a0, a1, a2, a3, pf[u][n][0], pf[u][n][1]);
          }
        }
      __syncwarp();                                      // every lane has read the slots
      consumed += U;
      top_up();
      return true;
    };
    int i = 0;
    for (; ok && i + kAtOnce <= cur.n; i += kAtOnce) ok = tiles(std::integral_constant<int, kAtOnce>(), i);
    if (ok && i < cur.n) ok = tiles(std::integral_constant<int, 1>(), i);
    if (!ok) break;
    // the rows' records, or, with nothing to join, the rows; o is in units of 2^M, a record's in 2^m
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[n][e];
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (8 * n + 2 * t + e >= rows) continue;
        const int r = it.row0 + 8 * n + 2 * t + e, tok = r / G, h = cur.hk * G + r % G;
        const float to_m = m[n][e] == -INFINITY ? 0.f : ex2(mw[n][e] - m[n][e]);
        if (it.direct) {
          const float f = to_m / sum;
          uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + (size_t(it.tok0 + tok) * H + h) * kDim) + g;
#pragma unroll
          for (int j = 0; j < 8; ++j) dst[8 * j] = pack2(o[n][j][e] * f, o[n][j][2 + e] * f);
        } else {
          // records of a listed item's rows are `rec_step` apart in the order of tokens and heads, of a share's in the tile's
          const size_t at = size_t(it.rec0) + (it.rec_step ? (size_t(tok) * H + h) * it.rec_step : size_t(8 * n + 2 * t + e));
          float2* rec = reinterpret_cast<float2*>(recs + at * kDim) + g;
#pragma unroll
          for (int j = 0; j < 8; ++j) __stcg(rec + 8 * j, make_float2(o[n][j][e] * to_m, o[n][j][2 + e] * to_m));
          if (g == 0) __stcg(rec_ml + at, make_float2(m[n][e], sum));
        }
      }
    cur = nxt;
    load_unit(nxt, slots[slot]);
    slot ^= 1;
  }
  if (!ok && lane == 0) raise_error(a.err, kErrTimeout | kSiteDecodeRing);
  // after a timeout some copies may still be in flight: wait for them (bounded) before exiting
  while (consumed < issued) {
    mbar_wait(bars + 8 * st_out, phase);
    ++consumed;
    if (++st_out == kStages) st_out = 0, phase ^= 1;
  }
}

}  // namespace qstream
}  // namespace cb
