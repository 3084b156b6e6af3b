// Pieces of a step (shared_prefix.h) over a cache in 8 bits, on tcgen05: the query
// rows of one or two 128-row tiles against a KV segment, left as records.
//
// e4m3 tiles are exact in f16, so the tensor core multiplies f16 by f16 and the tiles
// are widened on their way: TMA brings half tiles (64 keys, 8 KB) into two staging
// buffers each for K and V, two warps each widen them into the swizzled tiles that the
// MMAs read, and L2 and DRAM see 8 bits.  (Widened to bf16, which takes four times the
// conversions, a tile took 4.1 us and, all else equal, 2.8 to f16.)  As in the streams
// (quant_stream.cuh), a query row is scaled by a power of two, on its way too, and the
// weights, of which f16 holds 2^-24 to 2^16, keep a running maximum M of score +
// log2(vs) of their own.  The scales of a tile's blocks go around the tensor core: the
// K loader puts 8 of K and the logarithms of 8 of V, one for each 16 keys, into a ring
// in shared memory; the softmax multiplies the scores by the ones and adds the others
// to the weights' exponents, and takes them out again of the sum.
//
// Warps 0 to 7 are the softmax of row tiles 0 and 1, 8 the K loader, 9 the MMA thread's,
// 10 the V loader, 12 and 13 widen K, 14 and 15 V; all with 128 registers.
//
// What bounds it: a KV tile for two row tiles takes 2.4 us, the pieces' ends included,
// where its four matrix products of 128^3 would take 1.3 at the measured bf16 rate.  A
// row tile's softmax, instructions that wait for one another, stands between its two
// products; the other tile's products fill a part of that, and the widening takes issue
// slots from the softmax.  Tensor pipe 46 %, issue 51 %, DRAM 6 %.  2048 tokens of 32
// heads behind 30,720 keys: 1005 us, 1060 TFLOP/s.  Measured against this, us: the maxima
// found first and half of the scores held, 1343; softmax warps with more registers from
// setmaxnreg, 1579, or 16 of them, 1470; the loop over 32 keys unrolled, 1358, the
// roles' code being more than the instruction caches hold; P V of the first 64 keys
// started before the last 64 have weights, 1049; three staging buffers, with V's ring in
// three halves, 1064.
#pragma once

#include <cuda.h>

#include "device_common.cuh"
#include "e4m3.cuh"
#include "packed.cuh"
#include "quant_stream.cuh"
#include "shared_prefix.h"
#include "sm100_ptx.cuh"

namespace cb {
namespace qpieces {

using namespace sm100;

constexpr int BM = 128;                          // query rows per tile = TMEM lanes
constexpr int BN = 128;                          // keys per KV tile
constexpr int HN = BN / 2;                       // of a staged half
constexpr int HD = kPrefixDim;
constexpr int kStages = 2;                       // K tiles, and V tiles
constexpr uint32_t kBufs = 2;                    // staged halves of K, and of V (with one, 1209 us of 1007)
constexpr int kThreads = 512;
constexpr int kWidenRows = 2;                    // that a lane widens at once (1: 1031 us of 1007, 4: 1021, 8: 1017)
constexpr int kWarpK = 8, kWarpMma = 9, kWarpV = 10, kWarpWiden = 12;
constexpr uint32_t kHalf = BM * 64 * 2;          // one 64-dim swizzled half of a bf16 tile: 16 KB
constexpr uint32_t kTile = 2 * kHalf;
constexpr uint32_t kStaged = HN * HD;            // 64 keys in 8 bits
constexpr uint32_t kTmemCols = 512;              // per slot t: S (then P) at 256t, O at 256t + 128
constexpr int kScaleSlots = 6;                   // tiles whose scales are kept: the softmax may be 4 behind the loader
constexpr int kTileScales = 16;                  // of K, and the logarithms of V's
constexpr float kNoScore = -3e38f;               // maxima before the first key

constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = kOffQ + 2 * kTile;
constexpr uint32_t kOffV = kOffK + kStages * kTile;
constexpr uint32_t kOffStaged = kOffV + kStages * kTile;   // K's two, V's two
constexpr uint32_t kOffBar = kOffStaged + 2 * kBufs * kStaged;
constexpr int kItemSlots = 2;
constexpr int kItemReaders = 1 + 1 + 8 + 4;      // V loader, MMA, softmax and widening warps
enum : int {
  BAR_Q = 0,                   // Q tiles landed
  BAR_QE = 1,                  // every S MMA of the piece has read Q, every softmax warp its rows' factors; a warp without rows
                               // arrives behind the piece's QF, or it could arrive for the next piece before this one's others
  BAR_QF = 2,                  // Q tiles in f16, their rows' factors written
  BAR_S = 3,                   // + slot: S ready
  BAR_P = BAR_S + 2,           // + slot: P written (128 arrivals)
  BAR_O = BAR_P + 2,           // + slot: the piece's last P V in the slot done
  BAR_F = BAR_O + 2,           // + 2 * (0: K, 1: V) + stage: widened
  BAR_E = BAR_F + 4,           // + the same: consumed
  BAR_SF = BAR_E + 4,          // + kBufs * (0: K, 1: V) + buffer: a half landed
  BAR_SE = BAR_SF + 2 * kBufs,   // + the same: read
  BAR_IF = BAR_SE + 2 * kBufs,   // + slot: piece published
  BAR_IE = BAR_IF + kItemSlots,  // + slot: piece read by every role
  BAR_DONE = BAR_IE + kItemSlots,
  NUM_BARS = BAR_DONE + 1
};
constexpr uint32_t kOffTmemSlot = kOffBar + 16 * ((NUM_BARS + 1) / 2);
constexpr uint32_t kOffItems = kOffTmemSlot + 16;
constexpr uint32_t kOffScales = kOffItems + kItemSlots * uint32_t(sizeof(Piece));
constexpr uint32_t kOffFactors = kOffScales + kScaleSlots * kTileScales * 4;   // of the query rows' scores
constexpr uint32_t kSmemBytes = kOffFactors + 2 * BM * 4 + 1024;   // + slack to align the base
static_assert(kOffItems % 16 == 0 && kOffScales % 16 == 0 && kSmemBytes <= 232448, "shared memory");

// idesc_bf16_f32 with f16 A and B
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return idesc_bf16_f32(M, N, b_mn_major) & ~((1u << 7) | (1u << 10));
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ float lds4(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ float2 lds8(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// The paged blocks of a piece's KV tiles, for one loader warp: the block table is read 32 entries at a time, one window ahead
// of the tiles, so that no load waits for it.  A lane issues each box.
struct BlockWindow {
  const int32_t* bt;           // the piece's first block
  int blocks;                  // blocks of the piece that hold keys
  int at;                      // first block of the window in `cur`
  int cur, next;               // lane i: box index of block at + i, at + 32 + i

  __device__ __forceinline__ int box(const AttnArgs& a, int hk, int i) const {
    const int none = a.num_blocks * a.num_kv_heads;            // out of range: TMA fills zeros
    if (i >= blocks) return none;
    const int blk = bt[i];
    if (blk >= 0 && blk < a.num_blocks) return blk * a.num_kv_heads + hk;
    raise_error(a.err, kErrBounds);
    return none;
  }
  __device__ __forceinline__ void start(const AttnArgs& a, const Piece& it, int lane) {
    const int bpt = BN / a.block_size;
    bt = a.block_tables + size_t(it.s0) * a.max_blocks_per_seq + it.skip + it.j0 * bpt;
    blocks = min((it.keys + a.block_size - 1) / a.block_size - it.j0 * bpt, it.nt * bpt);
    at = 0;
    cur = box(a, it.hk, lane);
    next = box(a, it.hk, 32 + lane);
  }
  // the window moves on to tile j
  __device__ __forceinline__ void advance(const AttnArgs& a, int hk, int j, int lane) {
    if (j * (BN / a.block_size) - at < 32) return;
    at += 32;
    cur = next;
    next = box(a, hk, at + 32 + lane);
  }
  // box index of the block that holds key `key` of tile j or j + 1
  __device__ __forceinline__ int of(int block_size, int j, int key) const {
    const int i = j * (BN / block_size) + key / block_size - at;
    const int x = __shfl_sync(0xffffffffu, cur, i & 31), y = __shfl_sync(0xffffffffu, next, i & 31);
    return i < 32 ? x : y;
  }
  // half hh of tile j (of the piece, in order) into dst
  __device__ __forceinline__ void load(uint32_t dst, const CUtensorMap* tm, uint32_t bar, const AttnArgs& a, int j, int hh,
                                       int lane) const {
    const int rows = min(a.block_size, HN), key = hh * HN + (lane * rows) % HN;
    const int z = of(a.block_size, j, key);
    if (lane == 0) mbar_arrive_expect_tx(bar, kStaged);
    if (lane < HN / rows) tma_load_3d(dst + lane * rows * HD, tm, bar, 0, key & (a.block_size - 1), z);
    __syncwarp();
  }
};

__device__ __forceinline__ void init_bars(uint32_t base) {
  auto bar = [&](int i) -> uint32_t { return base + kOffBar + 8u * uint32_t(i); };
  mbar_init(bar(BAR_Q), 1);
  mbar_init(bar(BAR_QE), 1 + 8);
  mbar_init(bar(BAR_QF), 4);
  for (int t = 0; t < 2; ++t) {
    mbar_init(bar(BAR_S + t), 1);
    mbar_init(bar(BAR_P + t), BM);
    mbar_init(bar(BAR_O + t), 1);
  }
  for (int i = 0; i < 4; ++i) {
    mbar_init(bar(BAR_F + i), 4);                  // two warps, two halves
    mbar_init(bar(BAR_E + i), 1);
  }
  for (int i = 0; i < 2 * kBufs; ++i) {
    mbar_init(bar(BAR_SF + i), 1);
    mbar_init(bar(BAR_SE + i), 2);                 // two warps
  }
  for (int i = 0; i < kItemSlots; ++i) {
    mbar_init(bar(BAR_IF + i), 1);
    mbar_init(bar(BAR_IE + i), kItemReaders);
  }
  mbar_init(bar(BAR_DONE), 1);
  fence_mbar_init();
}

// The pieces that this CTA claims through header[3], all its warps together.  Every wait is bounded; after a timeout the
// device error word is set, the roles wind down and the result is false.
__device__ __forceinline__ bool run_pieces(const CUtensorMap* tm_q, const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                                           const AttnArgs& a, const PrefixWork& w, uint8_t* gsm, uint32_t base, uint32_t tmem,
                                           int n_pieces, int with_pieces) {
  auto bar = [&](int i) -> uint32_t { return base + kOffBar + 8u * uint32_t(i); };
  Piece* items = reinterpret_cast<Piece*>(gsm + kOffItems);
  float* scales = reinterpret_cast<float*>(gsm + kOffScales);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int B = a.block_size;
  const int H = a.num_heads;
  const int G = H / a.num_kv_heads;                // query heads per key/value head
  const int TT = w.tile_tokens;
  bool ok = true;
  unsigned site = 0;

  auto warp_wait = [&](int b, uint32_t parity, unsigned where) -> bool {
    if (__all_sync(0xffffffffu, mbar_wait(bar(b), parity & 1u))) return true;
    ok = false;
    site = where;
    return false;
  };
  // a reading warp's view of piece n
  auto item_landed = [&](int n) -> bool { return warp_wait(BAR_IF + n % kItemSlots, n / kItemSlots, kSitePfItem); };
  auto item_read = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(BAR_IE + n % kItemSlots));
  };

  if (warp < kWarpK) {
    // ------------------------------------------------------------ softmax of slot t
    const int t = warp >> 2;
    const int wq = warp & 3;                       // TMEM lane quarter
    const int i = threadIdx.x - BM * t;            // tile row = TMEM lane
    const uint32_t lane_base = tmem + (uint32_t(wq * 32) << 16) + 256 * t;
    uint32_t cnt = 0, ocnt = 0;                    // S/P phases and O phases of this slot consumed
    uint32_t tiles = 0;                            // of the pieces before
    uint32_t qn = 0;                               // pieces before that have tiles, and so Q
    for (int n = 0; ok; ++n) {
      if (!item_landed(n)) break;
      // what the piece's end needs of it is read there: the slot is given back after that
      const volatile Piece* it = items + n % kItemSlots;
      if (it->flags & kPieceEnd) {
        item_read(n);
        break;
      }
      // this slot's rows and KV tiles j = first, first + step, ...
      const bool alt = it->flags & kPieceAlt;
      const int nt = it->nt;
      const int toff = alt ? 0 : t * TT;           // the slot's first token, within the piece
      const int rows = (alt ? it->ntok : min(TT, it->ntok - toff)) * G;
      const int step = alt ? 2 : 1;
      const int steps = alt ? (nt - t + 1) / 2 : nt;
      const bool work = wq * 32 < rows;            // some row of this warp is real
      if (nt > 0 && (steps == 0 || !work)) {       // no factor to read
        if (!warp_wait(BAR_QF, qn, kSitePfQ)) break;
        if (lane == 0) mbar_arrive(bar(BAR_QE));
      }
      qn += nt > 0;
      if (rows <= 0) {                             // no rows in the second tile
        tiles += nt;
        item_read(n);
        continue;
      }
      // keys of the current tile that this thread's row sees, and that every row of its warp does
      int lim, lim_warp;
      {
        const int k0 = (it->j0 + (alt ? t : 0)) * BN;
        lim = min(it->keys, it->lim0 + toff + i / G) - k0;
        lim_warp = min(it->keys, it->lim0 + toff + wq * 32 / G) - k0;
      }
      uint32_t tile = (tiles + (alt ? t : 0)) % kScaleSlots;
      tiles += nt;
      float m = kNoScore, l = 0.f, mw = kNoScore, sl2 = 0.f;   // mw: M
#pragma unroll 1
      for (int x = 0; x < steps; ++x) {
        if (!warp_wait(BAR_S + t, cnt + x, kSitePfS)) break;
        if (!work) {                               // rows of no token: their P may be anything
          mbar_arrive(bar(BAR_P + t));
          continue;
        }
        if (x == 0) {
          sl2 = a.scale_log2 * lds4(base + kOffFactors + ((alt ? 0 : BM * t) + i) * 4);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(BAR_QE));
        }
        tc_fence_after();
        // One pass, 32 keys at a time: weights by the maxima that the row has, which hold for nearly all keys behind the first;
        // where their sum shows a weight beyond f16, the maxima are raised, what they scaled so far is rescaled (M is whole, so that
        // is exact but for numbers below f16's normal ones), and the 32 keys are weighed again.
        const bool masked = BN > lim_warp;         // keys behind the last one, or the causal mask
        const uint32_t sc = base + kOffScales + tile * (kTileScales * 4);
        auto factor = [&](int g) { return fmaxf(sl2 * lds4(sc + 4 * g), 1.2e-38f); };   // of 16 keys' scores; not 0: -inf stays
        // Raises the maxima to those of keys 32 c .. 32 c + 31, with what they scaled so far.
        auto raise = [&](int c) {
          float mt = kNoScore, wt = kNoScore;
          uint32_t sr[32];
          tmem_ld32(lane_base + 32 * c, sr);
          tmem_wait_ld();
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float top = -INFINITY;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (!masked || 32 * c + 16 * g + e < lim) top = fmaxf(top, __uint_as_float(sr[16 * g + e]));
            top *= factor(2 * c + g);
            top = fmaf(fabsf(top), 0x1p-22f, top); // above what fma makes of the scores
            mt = fmaxf(mt, top);
            wt = fmaxf(wt, top + fmaxf(lds4(sc + 32 + 4 * (2 * c + g)), -126.f));
          }
          const float m_new = fmaxf(m, mt), w_new = fmaxf(mw, ceilf(wt) - 1.f), alpha = ex2(mw - w_new);
          l *= ex2(m - m_new);
          m = m_new, mw = w_new;
          tmem_wait_st();                          // of this tile's weights so far
#pragma unroll 1
          for (int k = 0; k < c; ++k) {
            uint32_t p[16];
            tmem_ld16(lane_base + 16 * k, p);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&p[e]));
              p[e] = qstream::pack_f16(v.x * alpha, v.y * alpha);
            }
            tmem_st16(lane_base + 16 * k, p);
          }
          // S done implies the slot's earlier P V done (one thread issues both, in order, and the commit behind S covers them):
          // O is stable
          if (x > 0) {
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
              uint32_t o[16];
              tmem_ld16(lane_base + 128 + 16 * k, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st16(lane_base + 128 + 16 * k, o);
            }
          }
        };
        // Weights times the values' scale, in units of 2^M and f16: within 2^-11 of each, 2^-25 of 2^M; `sum` is theirs, `add` that of
        // the weights alone, in units of 2^m.  A scale too small for any of its weights to count is raised to one whose weights' sum
        // is still in fp32's range.
        uint32_t sr[32];
        tmem_ld32(lane_base, sr);
        int raised = -1;                           // the last 32 keys that were; once each, whatever the scores
#pragma unroll 1
        for (int c = 0; c < 4;) {
          const float2 ks = lds8(sc + 8 * c), lg = lds8(sc + 32 + 8 * c);
          const float d = mw - m;
          float lv[2] = {fmaxf(lg.x, d - 60.f), fmaxf(lg.y, d - 60.f)};
          const float f[2] = {fmaxf(sl2 * ks.x, 1.2e-38f), fmaxf(sl2 * ks.y, 1.2e-38f)};   // not 0: -inf stays
          tmem_wait_ld();
          if (masked) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * c + e >= lim) sr[e] = __float_as_uint(-INFINITY);
          }
          uint64_t x2[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float z = lv[e >> 3] - mw;
            x2[e] = f2_fma(f2_pack(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1])), f2_pack(f[e >> 3], f[e >> 3]), f2_pack(z, z));
          }
          if (c < 3) tmem_ld32(lane_base + 32 * c + 32, sr);
          uint32_t p[16];
          uint64_t s2[2][2];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float x0, x1;
            f2_unpack(x2[e], x0, x1);
            x0 = ex2(x0), x1 = ex2(x1);
            p[e] = qstream::pack_f16(x0, x1);
            const uint64_t y = f2_pack(x0, x1);
            s2[e >> 3][e & 1] = (e & 7) < 2 ? y : f2_add(s2[e >> 3][e & 1], y);
          }
          float a0, a1, b0, b1;
          f2_unpack(f2_add(s2[0][0], s2[0][1]), a0, a1);
          f2_unpack(f2_add(s2[1][0], s2[1][1]), b0, b1);
          a0 += a1, b0 += b1;
          const float add = fmaf(a0, ex2(d - lv[0]), b0 * ex2(d - lv[1]));
          if (raised < c && __any_sync(0xffffffffu, a0 + b0 > 32768.f || add > 1e12f)) {
            tmem_wait_ld();
            raise(c);
            raised = c;
            tmem_ld32(lane_base + 32 * c, sr);     // once more
            continue;
          }
          l += add;
          tmem_st16(lane_base + 16 * c, p);        // over scores that are in registers
          ++c;
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(BAR_P + t));
        lim -= step * BN;
        lim_warp -= step * BN;
        tile = (tile + step) % kScaleSlots;
      }
      if (!ok) break;
      if (steps > 0) {
        if (!warp_wait(BAR_O + t, ocnt, kSitePfO)) break;
        tc_fence_after();
        ++ocnt;
      }
      cnt += steps;
      // The rows' records of this segment (in the alternating mode, of its even or odd tiles).  A lane holds one row; so that
      // a store is 8 whole lines, every 4 lanes first transpose their 4 rows of 32 dims in units of 32 bytes.
      const bool direct = it->flags & kPieceDirect;
      unsigned rec;
      {
        const int row_tok = toff + i / G, head = it->hk * G + i % G;
        rec = direct ? unsigned(it->tok0 + row_tok) * unsigned(H) + unsigned(head)
                     : it->rec0 + unsigned((row_tok * H + head) * it->rec_step + (alt ? t : 0));
      }
      item_read(n);
      const float to_m = ex2(mw - m);   // O is in units of 2^M, a record's in 2^m
      const float inv = direct ? to_m / l : to_m;
      if (work) {
        const int row4 = wq * 32 + (lane & ~3);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          if (steps > 0) {
            tmem_ld32(lane_base + 128 + 32 * c, o);
            tmem_wait_ld();
          } else {                                 // no tile: an empty record
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
#pragma unroll
          for (int d = 2; d > 0; d >>= 1) {
            const bool hi = lane & d;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              if (u & d) continue;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, hi ? o[8 * u + e] : o[8 * (u | d) + e], d);
                if (hi) o[8 * u + e] = got;
                else o[8 * (u | d) + e] = got;
              }
            }
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) {            // unit r now belongs to row r of these 4 lanes
            const unsigned at = __shfl_sync(0xffffffffu, rec, (lane & ~3) + r);
            const float f = __shfl_sync(0xffffffffu, inv, (lane & ~3) + r);
            if (row4 + r >= rows) continue;
            uint32_t* x = &o[8 * r];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
            if (direct) {
              auto two = [&](int e) { return pack_bf16x2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])); };
              *(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + size_t(at) * HD + 32 * c) + (lane & 3)) =
                  make_uint4(two(0), two(2), two(4), two(6));
            } else {
              store32(w.recs + size_t(at) * HD + 32 * c + 8 * (lane & 3), x);
            }
          }
        }
        if (i < rows && !direct) __stcg(w.rec_ml + rec, make_float2(m == kNoScore ? -INFINITY : m, l));
      }
      tc_fence_before();                           // O read before the next piece's first P V overwrites it
    }
    if (!ok && lane == 0) raise_error(a.err, kErrTimeout | site);
  } else if (warp < kWarpWiden) {
    if (warp == kWarpK) {
      // ---------------------------------------------------------- K loader (claims the pieces, brings the scales)
      uint32_t tc = 0, hc = 0, qc = 0;             // tiles, halves and Q loads requested
      int u = int(blockIdx.x);                     // the first piece is given, the later ones are claimed one ahead
      for (int n = 0; ok; ++n) {
        const int slot = n % kItemSlots;
        if (n >= kItemSlots && !warp_wait(BAR_IE + slot, (n / kItemSlots) - 1, kSitePfItemFree)) break;
        if (lane < int(sizeof(Piece) / 16)) {
          int4 part = make_int4(0, 0, 0, 0);
          if (u < n_pieces) part = __ldcg(reinterpret_cast<const int4*>(w.pieces + u) + lane);
          reinterpret_cast<int4*>(items + slot)[lane] = part;
        }
        __syncwarp();
        if (lane == 0) {
          if (u >= n_pieces) items[slot].flags = kPieceEnd;
          mbar_arrive(bar(BAR_IF + slot));         // release: the slot's contents are visible
        }
        if (u >= n_pieces) break;
        const int ahead = lane == 0 ? with_pieces + atomicAdd(w.header + 3, 1) : 0;
        const Piece it = items[slot];
        if (it.nt > 0) {
          const int nq = !(it.flags & kPieceAlt) && it.ntok > TT ? 2 : 1;
          auto load_q = [&]() -> bool {
            if (qc > 0 && !warp_wait(BAR_QE, qc - 1, kSitePfQFree)) return false;
            if (lane == 0) {
              mbar_arrive_expect_tx(bar(BAR_Q), uint32_t(nq) * 2u * uint32_t(G * TT) * 128u);
              for (int t = 0; t < nq; ++t) {
                tma_load_3d(base + kOffQ + t * kTile, tm_q, bar(BAR_Q), 0, it.hk * G, it.tok0 + t * TT);
                tma_load_3d(base + kOffQ + t * kTile + kHalf, tm_q, bar(BAR_Q), 64, it.hk * G, it.tok0 + t * TT);
              }
            }
            ++qc;
            __syncwarp();
            return true;
          };
          BlockWindow win;
          bool q_loaded = false;                   // the first piece's at once, later ones' behind a K tile: the last piece may still read Q
          if (n == 0) q_loaded = load_q();
          win.start(a, it, lane);
          // lanes 0 .. 7: a tile's K scales, 16 keys each; 8 .. 15: its V scales
          auto scale_of = [&](int j) -> float {
            const int z = win.of(B, j, (lane & 7) * 16);
            return lane < 16 && z < a.num_blocks * a.num_kv_heads ? (lane < 8 ? a.k_scale : a.v_scale)[z] : 1.0f;
          };
          float scale = scale_of(0);
          for (int j = 0; ok && j < it.nt; ++j) {
            if (j == 1 && !q_loaded && !load_q()) break;
            win.advance(a, it.hk, j, lane);
            for (int hh = 0; hh < 2; ++hh) {
              const int buf = hc % kBufs;
              if (hc >= kBufs && !warp_wait(BAR_SE + buf, hc / kBufs - 1, kSitePfKFree)) break;
              if (hh == 0) {                       // ahead of the half, which carries them to the softmax
                float* to = scales + (tc % kScaleSlots) * kTileScales + lane;
                if (lane < 16) to[0] = lane < 8 ? scale : qstream::lg2(scale);
                __syncwarp();
              }
              win.load(base + kOffStaged + buf * kStaged, tm_k, bar(BAR_SF + buf), a, j, hh, lane);
              ++hc;
            }
            ++tc;
            scale = scale_of(j + 1);
          }
          if (ok && it.nt == 1 && !q_loaded) load_q();
        }
        u = __shfl_sync(0xffffffffu, ahead, 0);
      }
      if (!ok && lane == 0) raise_error(a.err, kErrTimeout | site);
      if (lane == 0) {
        // (error path) let copies still in flight land before the memory is used again
        for (uint32_t x = hc > kBufs ? hc - kBufs : 0; x < hc; ++x) mbar_wait(bar(BAR_SF + x % kBufs), (x / kBufs) & 1);
        if (qc > 0) mbar_wait(bar(BAR_Q), (qc - 1) & 1);
      }
    } else if (warp == kWarpV) {
      // ---------------------------------------------------------- V loader
      uint32_t hc = 0;
      for (int n = 0; ok; ++n) {
        if (!item_landed(n)) break;
        const Piece it = items[n % kItemSlots];
        item_read(n);
        if (it.flags & kPieceEnd) break;
        if (it.nt == 0) continue;
        BlockWindow win;
        win.start(a, it, lane);
        for (int j = 0; ok && j < it.nt; ++j) {
          win.advance(a, it.hk, j, lane);
          for (int hh = 0; hh < 2; ++hh) {
            const int buf = kBufs + hc % kBufs;
            if (hc >= kBufs && !warp_wait(BAR_SE + buf, hc / kBufs - 1, kSitePfVFree)) break;
            win.load(base + kOffStaged + buf * kStaged, tm_v, bar(BAR_SF + buf), a, j, hh, lane);
            ++hc;
          }
        }
      }
      if (!ok && lane == 0) raise_error(a.err, kErrTimeout | site);
      if (lane == 0)                               // (error path) as above
        for (uint32_t x = hc > kBufs ? hc - kBufs : 0; x < hc; ++x) mbar_wait(bar(BAR_SF + kBufs + x % kBufs), (x / kBufs) & 1);
    } else if (warp == kWarpMma && lane == 0) {
      // ---------------------------------------------------------- MMA
      constexpr uint32_t idS = idesc_f16_f32(BM, BN, false);   // Q (K-major) x K (K-major)
      constexpr uint32_t idO = idesc_f16_f32(BM, HD, true);    // P (TMEM) x V (N-contiguous)
      const uint64_t dq0 = smem_desc(base + kOffQ, 16, 1024);
      const uint64_t dk0 = smem_desc(base + kOffK, 16, 1024);
      const uint64_t dv0 = smem_desc(base + kOffV, kHalf, 1024);
      // S of row tile `qt` into slot t
      auto issue_s = [&](int t, int qt, uint32_t gk) {
        const uint64_t kd = dk0 + (((gk % kStages) * kTile) >> 4);
        const uint64_t qd = dq0 + ((qt * kTile) >> 4);
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          const uint32_t off16 = ((k / 4) * kHalf + (k % 4) * 32) >> 4;
          mma_f16_ss(tmem + 256 * t, qd + off16, kd + off16, idS, k > 0);
        }
        mma_commit(bar(BAR_S + t));
      };
      auto issue_pv = [&](int t, uint32_t gv, bool accumulate, bool last) {
        const uint64_t vd = dv0 + (((gv % kStages) * kTile) >> 4);
#pragma unroll
        for (int k = 0; k < BN / 16; ++k)
          mma_f16_ts(tmem + 256 * t + 128, tmem + 256 * t + k * 8, vd + ((k * 2048) >> 4), idO, accumulate || k > 0);
        if (last) mma_commit(bar(BAR_O + t));
      };
      // Two row tiles, per KV tile j: P_0 V_j, S_0(j+1), P_1 V_j, S_1(j+1).
      // One row tile: P(j) V_j, S(j+2), both in slot j & 1.  Either way the S that
      // overwrites a slot comes right behind the P V that reads its P, which the
      // in-order execution of one thread's MMAs keeps safe.
      uint32_t kc = 0, vc = 0, qc = 0, cnt[2] = {0, 0};   // K, V tiles and Q loads consumed; S/P phases of the slots
      auto wait = [&](int b, uint32_t parity, unsigned where) -> bool {
        if (mbar_wait(bar(b), parity & 1u)) return true;
        ok = false;
        site = where;
        return false;
      };
      auto k_landed = [&](uint32_t gk) { return wait(BAR_F + gk % kStages, gk / kStages, kSitePfK); };
      auto v_landed = [&](uint32_t gv) { return wait(BAR_F + 2 + gv % kStages, gv / kStages, kSitePfV); };
      for (int n = 0; ok; ++n) {
        if (!wait(BAR_IF + n % kItemSlots, n / kItemSlots, kSitePfItem)) break;
        struct { int nt, ntok, flags; } it = {items[n % kItemSlots].nt, items[n % kItemSlots].ntok, items[n % kItemSlots].flags};
        mbar_arrive(bar(BAR_IE + n % kItemSlots));
        if (it.flags & kPieceEnd) break;
        if (it.nt == 0) continue;
        if (!wait(BAR_QF, qc++, kSitePfQ)) break;
        if (it.flags & kPieceAlt) {
          for (int j = 0; ok && j < min(2, it.nt); ++j) {
            const uint32_t gk = kc + j;
            if (!k_landed(gk)) break;
            tc_fence_after();
            issue_s(j, 0, gk);
            mma_commit(bar(BAR_E + gk % kStages));
            if (j + 1 == it.nt) mma_commit(bar(BAR_QE));
          }
          for (int j = 0; ok && j < it.nt; ++j) {
            const uint32_t gv = vc + j, t = j & 1;
            if (!v_landed(gv)) break;
            if (!wait(BAR_P + t, (t == 0 ? cnt[0] : cnt[1]) + (j >> 1), kSitePfP)) break;
            tc_fence_after();
            issue_pv(t, gv, j >= 2, j + 2 >= it.nt);
            mma_commit(bar(BAR_E + 2 + gv % kStages));
            if (j + 2 < it.nt) {
              const uint32_t gk = kc + j + 2;
              if (!k_landed(gk)) break;
              tc_fence_after();
              issue_s(t, 0, gk);
              mma_commit(bar(BAR_E + gk % kStages));
              if (j + 3 == it.nt) mma_commit(bar(BAR_QE));
            }
          }
          cnt[0] += (it.nt + 1) / 2;
          cnt[1] += it.nt / 2;
        } else {
          const int nq = it.ntok > TT ? 2 : 1;
          if (!k_landed(kc)) break;
          tc_fence_after();
          for (int t = 0; t < nq; ++t) issue_s(t, t, kc);
          mma_commit(bar(BAR_E + kc % kStages));
          if (it.nt == 1) mma_commit(bar(BAR_QE));
          for (int j = 0; ok && j < it.nt; ++j) {
            const bool next = j + 1 < it.nt;
            const uint32_t gv = vc + j, gk = kc + j + 1;
            if (!v_landed(gv)) break;
            for (int t = 0; t < nq; ++t) {
              if (!wait(BAR_P + t, (t == 0 ? cnt[0] : cnt[1]) + j, kSitePfP)) break;
              tc_fence_after();
              issue_pv(t, gv, j > 0, !next);
              if (t == nq - 1) mma_commit(bar(BAR_E + 2 + gv % kStages));
              if (next) {
                if (t == 0 && !k_landed(gk)) break;
                tc_fence_after();
                issue_s(t, t, gk);
                if (t == nq - 1) {
                  mma_commit(bar(BAR_E + gk % kStages));
                  if (j + 2 == it.nt) mma_commit(bar(BAR_QE));
                }
              }
            }
          }
          cnt[0] += it.nt;
          if (nq > 1) cnt[1] += it.nt;
        }
        kc += it.nt;
        vc += it.nt;
      }
      if (!ok) raise_error(a.err, kErrTimeout | site);
      mma_commit(bar(BAR_DONE));                   // every MMA issued so far has completed
      mbar_wait(bar(BAR_DONE), 0);
    }
  } else {
    // ------------------------------------------------------------ widening: two warps K, two V
    const int type = (warp - kWarpWiden) >> 1, sub = warp & 1;
    const uint32_t ring = base + (type ? kOffV : kOffK), staged = base + kOffStaged + type * kBufs * kStaged;
    // this lane: 16 dims (chunk c) of rows r0, r0 + 4, ... of its warp's 32; 8 lanes read a row's 128 bytes.  The lanes of the
    // upper 64 dims store their second 16 bytes first, so that 8 lanes' stores touch every bank once.
    const int c = lane & 7, r0 = sub * 32 + (lane >> 3), half = c >> 2, lo = 2 * (c & 3);
    uint32_t tc = 0, hc = 0, qc = 0;
    for (int n = 0; ok; ++n) {
      if (!item_landed(n)) break;
      const Piece it = items[n % kItemSlots];
      item_read(n);
      if (it.flags & kPieceEnd) break;
      if (it.nt == 0) continue;
      // the piece's Q tiles to f16, in place, a row a thread
      auto widen_q = [&]() -> bool {
        if (!warp_wait(BAR_Q, qc, kSitePfQ)) return false;
        ++qc;
        const int nq = !(it.flags & kPieceAlt) && it.ntok > TT ? 2 : 1, row = threadIdx.x - kWarpWiden * 32;
        for (int t = 0; t < nq; ++t) {
          const uint32_t at = base + kOffQ + t * kTile + row * 128;
          uint32_t top = 0;                        // bits of the largest magnitude
          const bool real = row < G * TT;          // the rows behind hold anything: zeros, whose scores raise no maximum
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const uint4 v = lds16(at + (k >> 3) * kHalf + (((k & 7) ^ (row & 7)) << 4));
            const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) top = max(top, max((in[e] << 16) & 0x7fff0000u, in[e] & 0x7fff0000u));
          }
          const uint32_t ex = real ? min(253u, 267u - (top >> 23)) : 127u;   // 2^13 / largest, as an exponent; its inverse is an ordinary number
          const float f = __uint_as_float(ex << 23);
          reinterpret_cast<float*>(gsm + kOffFactors)[t * BM + row] = __uint_as_float((254u - ex) << 23);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const uint32_t p = at + (k >> 3) * kHalf + (((k & 7) ^ (row & 7)) << 4);
            uint4 v = lds16(p);
            if (!real) v = make_uint4(0, 0, 0, 0);
            auto two = [&](uint32_t x) { return qstream::pack_f16(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xffff0000u) * f); };
            sts16(p, two(v.x), two(v.y), two(v.z), two(v.w));
          }
        }
        fence_proxy_async_smem();                  // for the tensor core
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_QF));
        return true;
      };
      if (n == 0 && !widen_q()) break;
      for (int j = 0; ok && j < it.nt; ++j, ++tc) {
        const int st = tc % kStages;
        if (tc >= kStages && !warp_wait(BAR_E + 2 * type + st, (tc / kStages) - 1, type ? kSitePfVFree : kSitePfKFree)) break;
        const int left = it.keys - (it.j0 + j) * BN;   // rows from there on may hold anything: V's are zeroed, since 0 * NaN is not 0
#pragma unroll 1
        for (int hh = 0; hh < 2; ++hh, ++hc) {
          const int buf = hc % kBufs;
          if (!warp_wait(BAR_SF + kBufs * type + buf, hc / kBufs, type ? kSitePfV : kSitePfK)) break;
#pragma unroll 1
          for (int k0 = 0; k0 < 8; k0 += kWidenRows) {
            uint4 x[kWidenRows];
#pragma unroll
            for (int k = 0; k < kWidenRows; ++k) {
              const int r = r0 + 4 * (k0 + k);
              x[k] = lds16(staged + buf * kStaged + r * HD + ((c ^ (r & 7)) << 4));
            }
            if (k0 + kWidenRows == 8) {
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(BAR_SE + kBufs * type + buf));
            }
#pragma unroll
            for (int k = 0; k < kWidenRows; ++k) {
              const int r = hh * HN + r0 + 4 * (k0 + k);
              if (type && r >= left) x[k] = make_uint4(0, 0, 0, 0);
              const uint32_t in[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
              uint32_t y[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) y[2 * e] = e4m3x2_to_f16x2(in[e]), y[2 * e + 1] = e4m3x2_hi_to_f16x2(in[e]);
              const uint32_t row = ring + st * kTile + half * kHalf + r * 128, at0 = row + ((lo ^ (r & 7)) << 4),
                             at1 = row + (((lo + 1) ^ (r & 7)) << 4);
              sts16(half ? at1 : at0, half ? y[4] : y[0], half ? y[5] : y[1], half ? y[6] : y[2], half ? y[7] : y[3]);
              sts16(half ? at0 : at1, half ? y[0] : y[4], half ? y[1] : y[5], half ? y[2] : y[6], half ? y[3] : y[7]);
            }
          }
          fence_proxy_async_smem();                // for the tensor core
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(BAR_F + 2 * type + st));
        }
        if (ok && j == 0 && n > 0) widen_q();      // requested behind the piece's first K tile, or, in the first piece, before
      }
    }
    if (!ok && lane == 0) raise_error(a.err, kErrTimeout | site);
  }
  __syncwarp();
  tc_fence_before();
  const bool failed = __syncthreads_or(ok ? 0 : 1);
  tc_fence_after();
  return !failed;
}

}  // namespace qpieces
}  // namespace cb
