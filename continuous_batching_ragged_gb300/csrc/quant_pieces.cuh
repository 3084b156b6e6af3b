// Pieces of a step (shared_prefix.h) over a cache in 8 bits, on tcgen05: the query
// rows of one or two 128-row tiles against a KV segment, left as records.
//
// The tensor core multiplies bf16 by bf16: queries are bf16, and weights need its
// range once the values' scales are in them.  So the e4m3 tiles, exact in bf16, are
// widened on their way: TMA brings half tiles (64 keys, 8 KB) into two staging
// buffers each for K and V, two warps each widen them into the swizzled tiles that the
// MMAs read (a quarter of the issue slots; the L2 and DRAM traffic stays that of 8
// bits), and everything behind is as over a bf16 cache (prefix_tc_kernel).  The scales
// of a tile's blocks go around the tensor core: the K loader puts 8 of K and 8 of V,
// one for each 16 keys, into a ring in shared memory, the softmax multiplies the
// scores by the ones and the weights by the others.
//
// Roles, in warpgroups whose registers are split by need: 0 and 1 softmax of row
// tiles 0 and 1, 2 K loader, MMA and V loader, 3 widening (two warps K, two V).
#pragma once

#include <cuda.h>

#include "device_common.cuh"
#include "e4m3.cuh"
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
constexpr int kThreads = 512;
constexpr int kWarpK = 8, kWarpMma = 9, kWarpV = 10, kWarpWiden = 12;
constexpr int kSoftmaxRegs = 184, kLoaderRegs = 56, kWidenRegs = 88;
static_assert(2 * kSoftmaxRegs + kLoaderRegs + kWidenRegs <= 512, "128 registers a thread in all");
constexpr uint32_t kHalf = BM * 64 * 2;          // one 64-dim swizzled half of a bf16 tile: 16 KB
constexpr uint32_t kTile = 2 * kHalf;
constexpr uint32_t kStaged = HN * HD;            // 64 keys in 8 bits
constexpr uint32_t kTmemCols = 512;              // per slot t: S (then P) at 256t, O at 256t + 128
constexpr int kScaleSlots = 8;                   // tiles whose scales are kept; the loader is at most 5 ahead of the softmax

constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = kOffQ + 2 * kTile;
constexpr uint32_t kOffV = kOffK + kStages * kTile;
constexpr uint32_t kOffStaged = kOffV + kStages * kTile;   // K's two, V's two
constexpr uint32_t kOffBar = kOffStaged + 4 * kStaged;
constexpr int kItemSlots = 2;
constexpr int kItemReaders = 1 + 1 + 8 + 4;      // V loader, MMA, softmax and widening warps
enum : int {
  BAR_Q = 0,                   // Q tiles landed
  BAR_QE = 1,                  // every S MMA of the piece has read Q
  BAR_S = 2,                   // + slot: S ready
  BAR_P = BAR_S + 2,           // + slot: P written (128 arrivals)
  BAR_O = BAR_P + 2,           // + slot: the piece's last P V in the slot done
  BAR_F = BAR_O + 2,           // + 2 * (0: K, 1: V) + stage: widened
  BAR_E = BAR_F + 4,           // + the same: consumed
  BAR_SF = BAR_E + 4,          // + 2 * (0: K, 1: V) + buffer: a half landed
  BAR_SE = BAR_SF + 4,         // + the same: read
  BAR_IF = BAR_SE + 4,         // + slot: piece published
  BAR_IE = BAR_IF + kItemSlots,  // + slot: piece read by every role
  BAR_DONE = BAR_IE + kItemSlots,
  NUM_BARS = BAR_DONE + 1
};
constexpr uint32_t kOffTmemSlot = kOffBar + 16 * ((NUM_BARS + 1) / 2);
constexpr uint32_t kOffItems = kOffTmemSlot + 16;
constexpr uint32_t kOffScales = kOffItems + kItemSlots * uint32_t(sizeof(Piece));
constexpr uint32_t kSmemBytes = kOffScales + kScaleSlots * 64 + 1024;   // + slack to align the base
static_assert(kOffItems % 16 == 0 && kOffScales % 16 == 0 && kSmemBytes <= 232448, "shared memory");

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
// Packed fp32 pairs: two lanes of work per instruction.
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
// 32 bytes in one store (aligned)
__device__ __forceinline__ void store32(float* p, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
               "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
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
  mbar_init(bar(BAR_QE), 1);
  for (int t = 0; t < 2; ++t) {
    mbar_init(bar(BAR_S + t), 1);
    mbar_init(bar(BAR_P + t), BM);
    mbar_init(bar(BAR_O + t), 1);
  }
  for (int i = 0; i < 4; ++i) {
    mbar_init(bar(BAR_F + i), 4);                  // two warps, two halves
    mbar_init(bar(BAR_E + i), 1);
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

  // A reader's view of piece n; `arrive`: this thread is its role's one arrival.
  auto read_item = [&](int n, bool arrive, Piece& it) -> bool {
    const int slot = n % kItemSlots;
    if (!mbar_wait(bar(BAR_IF + slot), (n / kItemSlots) & 1)) return false;
    it = items[slot];
    if (arrive) mbar_arrive(bar(BAR_IE + slot));
    return true;
  };
  // the same for a whole warp
  auto read_item_warp = [&](int n, Piece& it) -> bool {
    if (!__all_sync(0xffffffffu, read_item(n, false, it))) return false;
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(BAR_IE + n % kItemSlots));
    return true;
  };
  auto warp_wait = [&](int b, uint32_t parity, unsigned where) -> bool {
    if (__all_sync(0xffffffffu, mbar_wait(bar(b), parity & 1u))) return true;
    ok = false;
    site = where;
    return false;
  };

  if (warp < kWarpK) {
    // ------------------------------------------------------------ softmax of slot t
    regs_up<kSoftmaxRegs>();
    const int t = warp >> 2;
    const int wq = warp & 3;                       // TMEM lane quarter
    const int i = threadIdx.x - BM * t;            // tile row = TMEM lane
    const uint32_t lane_base = tmem + (uint32_t(wq * 32) << 16) + 256 * t;
    const float sl2 = a.scale_log2;
    uint32_t cnt = 0, ocnt = 0;                    // S/P phases and O phases of this slot consumed
    uint32_t tiles = 0;                            // of the pieces before
    for (int n = 0; ok; ++n) {
      Piece it;
      if (!read_item_warp(n, it)) {
        ok = false;
        site = kSitePfItem;
        break;
      }
      if (it.flags & kPieceEnd) break;
      // this slot's rows and KV tiles j = first, first + step, ...
      const bool alt = it.flags & kPieceAlt;
      const int toff = alt ? 0 : t * TT;           // the slot's first token, within the piece
      const int ntok = alt ? it.ntok : min(TT, it.ntok - toff);
      const int step = alt ? 2 : 1, first = alt ? t : 0;
      const uint32_t tile0 = tiles;
      tiles += it.nt;
      if (ntok <= 0) continue;                     // no rows in the second tile
      const int rows = ntok * G;
      const int steps = (it.nt - first + step - 1) / step;
      // keys that this thread's row sees, and that every row of its warp does
      const int lim = min(it.keys, it.lim0 + toff + i / G), lim_warp = min(it.keys, it.lim0 + toff + wq * 32 / G);
      const bool work = wq * 32 < rows;            // some row of this warp is real
      float m = -INFINITY, l = 0.f;
      for (int x = 0; x < steps; ++x) {
        if (!warp_wait(BAR_S + t, cnt + x, kSitePfS)) break;
        if (!work) {                               // rows of no token: their P may be anything
          mbar_arrive(bar(BAR_P + t));
          continue;
        }
        tc_fence_after();
        uint32_t sr[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(lane_base + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&sr[32 * c]));
        tmem_wait_ld();
        const int kb = (it.j0 + first + x * step) * BN;
        if (kb + BN > lim_warp) {                  // keys behind the last one, or the causal mask
#pragma unroll
          for (int c = 0; c < BN; ++c)
            if (kb + c >= lim) sr[c] = __float_as_uint(-INFINITY);
        }
        const float* sc = scales + ((tile0 + first + x * step) % kScaleSlots) * 16;
        float mt = -INFINITY;
#pragma unroll
        for (int c = 0; c < 8; ++c) {              // 16 keys of one block
          auto s = [&](int e) { return __uint_as_float(sr[16 * c + e]); };
          const float u = max3(max3(s(0), s(1), s(2)), max3(s(3), s(4), s(5)), max3(s(6), s(7), s(8)));
          const float v = max3(max3(s(9), s(10), s(11)), max3(s(12), s(13), s(14)), s(15));
          mt = fmaxf(mt, fmaxf(u, v) * fmaxf(sl2 * sc[c], 1.2e-38f));   // not 0: -inf stays
        }
        const float m_new = fmaxf(m, mt);
        const bool resc = m_new > m + 8.0f;        // keep a stale max while exp2 stays <= 2^8
        const float m_use = resc ? m_new : m;
        const float alpha = resc ? ex2(m - m_new) : 1.0f;
        const float m_sub = m_use == -INFINITY ? 0.f : m_use;   // scores all -inf so far
        const uint64_t neg_m2 = f2_pack(-m_sub, -m_sub);
        uint64_t sum2[4] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f), f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
        // weights times the values' scale over the scores, rounded to bf16 since the tensor core takes them no wider: half a
        // step, 2^-8, of each.  The sums are of the weights in fp32.
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float f = fmaxf(sl2 * sc[c], 1.2e-38f), vs = sc[8 + c];
          const uint64_t f2 = f2_pack(f, f), vs2 = f2_pack(vs, vs);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int k = 8 * c + e;
            float x0, x1, p0, p1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[2 * k]), __uint_as_float(sr[2 * k + 1])), f2, neg_m2), x0, x1);
            const uint64_t p2 = f2_pack(ex2(x0), ex2(x1));
            sum2[e & 3] = f2_add(sum2[e & 3], p2);
            f2_unpack(f2_mul(p2, vs2), p0, p1);
            sr[k] = pack_bf16x2(p0, p1);
          }
        }
        float r0, r1, r2, r3, r4, r5, r6, r7;
        f2_unpack(sum2[0], r0, r1);
        f2_unpack(sum2[1], r2, r3);
        f2_unpack(sum2[2], r4, r5);
        f2_unpack(sum2[3], r6, r7);
        l = l * alpha + (((r0 + r1) + (r2 + r3)) + ((r4 + r5) + (r6 + r7)));
        m = m_use;
        // S done implies the slot's earlier P V done (one thread issues both, in order,
        // and the commit behind S covers them): O is stable for the rescale
        if (x > 0 && __any_sync(0xffffffffu, resc)) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tmem_ld32(lane_base + 128 + 32 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(lane_base + 128 + 32 * c, o);
          }
        }
        tmem_st32(lane_base, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
        tmem_st32(lane_base + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(BAR_P + t));
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
      const bool direct = it.flags & kPieceDirect;
      const int row_tok = toff + i / G, head = it.hk * G + i % G;
      const unsigned rec = direct ? unsigned(it.tok0 + row_tok) * unsigned(H) + unsigned(head)
                                  : it.rec0 + unsigned((row_tok * H + head) * it.rec_step + (alt ? t : 0));
      const float inv = direct ? 1.0f / l : 1.0f;
      if (work) {
        unsigned at[4];                            // of the rows of this lane's 4
        float f[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          at[r] = __shfl_sync(0xffffffffu, rec, (lane & ~3) + r);
          f[r] = __shfl_sync(0xffffffffu, inv, (lane & ~3) + r);
        }
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
            if (row4 + r >= rows) continue;
            const uint32_t* x = &o[8 * r];
            if (direct) {
              auto two = [&](int e) { return pack_bf16x2(__uint_as_float(x[e]) * f[r], __uint_as_float(x[e + 1]) * f[r]); };
              *(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + size_t(at[r]) * HD + 32 * c) + (lane & 3)) =
                  make_uint4(two(0), two(2), two(4), two(6));
            } else {
              store32(w.recs + size_t(at[r]) * HD + 32 * c + 8 * (lane & 3), x);
            }
          }
        }
        if (i < rows && !direct) __stcg(w.rec_ml + rec, make_float2(m, l));
      }
      tc_fence_before();                           // O read before the next piece's first P V overwrites it
    }
    if (!ok && lane == 0) raise_error(a.err, kErrTimeout | site);
  } else if (warp < kWarpWiden) {
    regs_down<kLoaderRegs>();
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
          BlockWindow win;
          win.start(a, it, lane);
          // lanes 0 .. 7: a tile's K scales, 16 keys each; 8 .. 15: its V scales
          auto scale_of = [&](int j) -> float {
            const int z = win.of(B, j, (lane & 7) * 16);
            return lane < 16 && z < a.num_blocks * a.num_kv_heads ? (lane < 8 ? a.k_scale : a.v_scale)[z] : 1.0f;
          };
          float scale = scale_of(0);
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
          for (int j = 0; ok && j < it.nt; ++j) {
            if (j == 1 && !load_q()) break;
            win.advance(a, it.hk, j, lane);
            for (int hh = 0; hh < 2; ++hh) {
              const int buf = hc & 1;
              if (hc >= 2 && !warp_wait(BAR_SE + buf, (hc >> 1) - 1, kSitePfKFree)) break;
              if (hh == 0) {                       // ahead of the half, which carries them to the softmax
                if (lane < 16) scales[(tc % kScaleSlots) * 16 + lane] = scale;
                __syncwarp();
              }
              win.load(base + kOffStaged + buf * kStaged, tm_k, bar(BAR_SF + buf), a, j, hh, lane);
              ++hc;
            }
            ++tc;
            scale = scale_of(j + 1);
          }
          if (ok && it.nt == 1) load_q();
        }
        u = __shfl_sync(0xffffffffu, ahead, 0);
      }
      if (!ok && lane == 0) raise_error(a.err, kErrTimeout | site);
      if (lane == 0) {
        // (error path) let copies still in flight land before the memory is used again
        for (uint32_t x = hc > 2u ? hc - 2 : 0; x < hc; ++x) mbar_wait(bar(BAR_SF + (x & 1)), (x >> 1) & 1);
        if (qc > 0) mbar_wait(bar(BAR_Q), (qc - 1) & 1);
      }
    } else if (warp == kWarpV) {
      // ---------------------------------------------------------- V loader
      uint32_t hc = 0;
      for (int n = 0; ok; ++n) {
        Piece it;
        if (!read_item_warp(n, it)) {
          ok = false;
          site = kSitePfItem;
          break;
        }
        if (it.flags & kPieceEnd) break;
        if (it.nt == 0) continue;
        BlockWindow win;
        win.start(a, it, lane);
        for (int j = 0; ok && j < it.nt; ++j) {
          win.advance(a, it.hk, j, lane);
          for (int hh = 0; hh < 2; ++hh) {
            const int buf = hc & 1;
            if (hc >= 2 && !warp_wait(BAR_SE + 2 + buf, (hc >> 1) - 1, kSitePfVFree)) break;
            win.load(base + kOffStaged + (2 + buf) * kStaged, tm_v, bar(BAR_SF + 2 + buf), a, j, hh, lane);
            ++hc;
          }
        }
      }
      if (!ok && lane == 0) raise_error(a.err, kErrTimeout | site);
      if (lane == 0)                               // (error path) as above
        for (uint32_t x = hc > 2u ? hc - 2 : 0; x < hc; ++x) mbar_wait(bar(BAR_SF + 2 + (x & 1)), (x >> 1) & 1);
    } else if (warp == kWarpMma && lane == 0) {
      // ---------------------------------------------------------- MMA
      constexpr uint32_t idS = idesc_bf16_f32(BM, BN, false);   // Q (K-major) x K (K-major)
      constexpr uint32_t idO = idesc_bf16_f32(BM, HD, true);    // P (TMEM) x V (N-contiguous)
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
        Piece it;
        if (!read_item(n, true, it)) {
          ok = false;
          site = kSitePfItem;
          break;
        }
        if (it.flags & kPieceEnd) break;
        if (it.nt == 0) continue;
        if (!wait(BAR_Q, qc++, kSitePfQ)) break;
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
    regs_down<kWidenRegs>();
    const int type = (warp - kWarpWiden) >> 1, sub = warp & 1;
    const uint32_t ring = base + (type ? kOffV : kOffK), staged = base + kOffStaged + type * 2 * kStaged;
    // this lane: 16 dims (chunk c) of rows r0, r0 + 4, ... of its warp's 32; 8 lanes read a row's 128 bytes.  The lanes of the
    // upper 64 dims store their second 16 bytes first, so that 8 lanes' stores touch every bank once.
    const int c = lane & 7, r0 = sub * 32 + (lane >> 3), half = c >> 2, lo = 2 * (c & 3);
    uint32_t tc = 0, hc = 0;
    for (int n = 0; ok; ++n) {
      Piece it;
      if (!read_item_warp(n, it)) {
        ok = false;
        site = kSitePfItem;
        break;
      }
      if (it.flags & kPieceEnd) break;
      for (int j = 0; ok && j < it.nt; ++j, ++tc) {
        const int st = tc % kStages;
        if (tc >= kStages && !warp_wait(BAR_E + 2 * type + st, (tc / kStages) - 1, type ? kSitePfVFree : kSitePfKFree)) break;
        const int left = it.keys - (it.j0 + j) * BN;   // rows from there on may hold anything: V's are zeroed, since 0 * NaN is not 0
#pragma unroll 1
        for (int hh = 0; hh < 2; ++hh, ++hc) {
          const int buf = hc & 1;
          if (!warp_wait(BAR_SF + 2 * type + buf, hc >> 1, type ? kSitePfV : kSitePfK)) break;
          uint4 x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int r = r0 + 4 * k;
            x[k] = lds16(staged + buf * kStaged + r * HD + ((c ^ (r & 7)) << 4));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(BAR_SE + 2 * type + buf));
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int r = hh * HN + r0 + 4 * k;
            if (type && r >= left) x[k] = make_uint4(0, 0, 0, 0);
            const uint32_t in[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
            uint32_t y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float f[4];
              e4m3x4_to_float(in[e], f);
              y[2 * e] = pack_bf16x2(f[0], f[1]);
              y[2 * e + 1] = pack_bf16x2(f[2], f[3]);
            }
            const uint32_t row = ring + st * kTile + half * kHalf + r * 128, at0 = row + ((lo ^ (r & 7)) << 4),
                           at1 = row + (((lo + 1) ^ (r & 7)) << 4);
            if (half) {
              sts16(at1, y[4], y[5], y[6], y[7]);
              sts16(at0, y[0], y[1], y[2], y[3]);
            } else {
              sts16(at0, y[0], y[1], y[2], y[3]);
              sts16(at1, y[4], y[5], y[6], y[7]);
            }
          }
          fence_proxy_async_smem();                // for the tensor core
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(BAR_F + 2 * type + st));
        }
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
