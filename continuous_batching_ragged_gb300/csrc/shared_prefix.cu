// Attention over shared prefixes: the keys that every sequence of a group has
// in common, read once for all of its query rows (bf16, head_dim 128).
//
// A decode step reads every sequence's whole cache; where sequences continue
// one prompt, most of those bytes are the same pages again and again.  For a
// group of sequences with R query tokens and G query heads per key/value head,
// the prefix phase is, per key/value head, a dense product of R * G query rows
// with the prefix's keys, no mask: softmax(Q K^T) V over those keys, left
// unnormalised as one record (acc, max, sum) per row and KV segment.  The rows'
// own keys leave records too (suffix_decode.cu, or prefill_tc.cu for chunks of
// many query rows), and a last kernel joins each row's.
//
// What bounds it: the prefix's K and V once from HBM while R * G is below about
// 256 rows (the ridge of 4 flops per row and byte pair), the tensor cores
// above.  So the rows of all query heads of a key/value head are packed into
// the MMA tile (row = token * G + head), and
//   * a group of at most one tile of rows runs its KV tiles alternately on two
//     score/output buffers, the even tiles on one softmax warpgroup and the
//     odd ones on the other, each with its own record: the two halves of the
//     softmax work and the tensor core's overlap although there is one row tile;
//   * larger groups run two row tiles against every KV tile in ping-pong, as
//     the prefill kernel does.
// Pieces are (row tile pair, key/value head, KV segment).  The plan cuts the
// prefix into the number of segments that minimises the estimated time of the
// piece waves; every segment costs the join one more record per row.
#include <algorithm>
#include <atomic>
#include <mutex>

#include <cuda.h>

#include "device_common.cuh"
#include "kernels.h"
#include "runtime.h"
#include "shared_prefix.h"
#include "sm100_ptx.cuh"

namespace cb {
namespace {

using namespace sm100;

constexpr int BM = 128;                          // query rows per tile = TMEM lanes
constexpr int BN = 128;                          // keys per KV tile
constexpr int HD = kPrefixDim;
constexpr int kKStages = 2;
constexpr int kVStages = 3;
constexpr int kThreads = 352;                    // warps 0-7 softmax, 8 K loader, 9 MMA, 10 V loader
constexpr int kWarpK = 8, kWarpMma = 9, kWarpV = 10;
constexpr uint32_t kHalf = BM * 64 * 2;          // one 64-dim swizzled half of a tile: 16 KB
constexpr uint32_t kTile = 2 * kHalf;
constexpr uint32_t kTmemCols = 512;              // per slot t: S (then P) at 256t, O at 256t + 128

constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = kOffQ + 2 * kTile;
constexpr uint32_t kOffV = kOffK + kKStages * kTile;
constexpr uint32_t kOffBar = kOffV + kVStages * kTile;
constexpr int kItemSlots = 2;
constexpr int kItemReaders = 1 + 1 + 8;          // V loader, MMA, softmax warps
enum : int {
  BAR_Q = 0,                   // Q tiles landed
  BAR_QE = 1,                  // every S MMA of the piece has read Q
  BAR_S = 2,                   // + slot: S ready
  BAR_P = BAR_S + 2,           // + slot: P written (128 arrivals)
  BAR_O = BAR_P + 2,           // + slot: the piece's last P V in the slot done
  BAR_KF = BAR_O + 2,          // + stage: K landed
  BAR_KE = BAR_KF + kKStages,  // + stage: K consumed
  BAR_VF = BAR_KE + kKStages,  // + stage: V landed
  BAR_VE = BAR_VF + kVStages,  // + stage: V consumed
  BAR_IF = BAR_VE + kVStages,  // + slot: piece published
  BAR_IE = BAR_IF + kItemSlots,  // + slot: piece read by every role
  BAR_DONE = BAR_IE + kItemSlots,
  NUM_BARS = BAR_DONE + 1
};
constexpr uint32_t kOffTmemSlot = kOffBar + 16 * ((NUM_BARS + 1) / 2);
constexpr uint32_t kOffItems = kOffTmemSlot + 16;
constexpr int kLookAhead = 4;                    // tiles of block-table look-ahead and L2 prefetch
constexpr int kRing = 8;
constexpr uint32_t kOffRing = kOffItems + kItemSlots * 48;
constexpr uint32_t kSmemBytes = kOffRing + 2 * kRing * 8 * 4 + 1024;   // + slack to align the base
static_assert(kRing > kLookAhead, "ring must outlive the look-ahead");
static_assert(kOffItems % 16 == 0 && kOffRing % 16 == 0, "pieces are copied 16 bytes at a time");
static_assert(kSmemBytes <= 232448, "shared memory budget");

// ------------------------------------------------------------------ plan

constexpr int kPlanThreads = 512;
constexpr int kMaxSegs = 64;             // KV segments of a prefix
constexpr int kGroupCache = 512;         // groups kept in shared memory
constexpr int kExtraPieces = 1024;       // pieces beyond one per (row tile pair, key/value head)
constexpr int64_t kExtraRecs = 131072;   // prefix records beyond two per row (69 MB)
// Estimated cost of a piece beyond its KV tiles, in tiles: the Q load, the
// pipeline's fill and the records.
constexpr float kPieceTiles = 2.5f;
constexpr int kSuffixTile = 16;          // keys per tile of the suffix kernel
constexpr int kMinChunkTiles = 8;        // shortest chunk of own keys, in those tiles
constexpr int kSuffixRows = 16;          // query rows per row tile of the suffix kernel
constexpr int kUnitsPerWarp = 3;         // suffix units that each warp should get
constexpr int kMaxSms = 160;             // SMs that the lists are sized for
// Query rows per key/value head up to which a sequence's own keys go to the
// suffix kernel, which streams them once per 16 rows; beyond, to prefill tiles.
constexpr int kMaxWarpRows = 128;

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Exclusive block-wide scan; `total` receives the sum.  Contains __syncthreads.
__device__ int64_t block_scan(int64_t v, int64_t* warp_sums, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    all += warp_sums[w];
  }
  total = all;
  __syncthreads();
  return before + x - v;
}

// Whether a sequence's rows go to the prefill kernel, and its row tiles otherwise.
__device__ __forceinline__ bool is_chunk(const PrefixWork& w, int q_len, int G) {
  return q_len > 1 && int64_t(q_len) * G > w.max_warp_rows;
}

// One CTA.  Checks the groups, chooses the segments of the prefixes and the
// chunks of the own keys, lists the pieces and the items and gives every row
// its records.
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const AttnArgs a, const PrefixWork w) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // they wait for this grid on the device
  __shared__ int64_t warp_sums[kPlanThreads / 32];
  __shared__ float best_cost[kMaxSegs];
  __shared__ int4 gcache[kGroupCache];
  __shared__ int s_n, s_alt;
  const int tid = threadIdx.x;
  const int S = a.num_seqs, T = a.num_tokens, NG = w.num_groups, TT = w.tile_tokens;
  const int H = a.num_heads, Hkv = a.num_kv_heads, G = H / Hkv;
  const int32_t* cu = a.cu_seqlens_q;
  auto group = [&](int g) -> int4 { return g < kGroupCache ? gcache[g] : w.groups[g]; };
  auto set_header = [&](int pieces, int stride, int items) {
    w.header[0] = pieces;
    w.header[1] = stride;
    w.header[2] = int32_t(w.tag);
    w.header[3] = 0;
    w.header[4] = items;
    w.header[5] = 0;
  };
  // nothing runs and no row is written
  auto give_up = [&]() {
    for (int s = tid; s < S; s += kPlanThreads) {
      w.suffix_lens[s] = 0;
      w.seq_info[s] = make_int4(0, 0, 0, 0);
    }
    for (int t = tid; t < T; t += kPlanThreads) w.token_info[t] = make_int4(0, 0, 0, 0);
    if (tid == 0) {
      raise_error(a.err, kErrInvalid);
      set_header(0, 0, 0);
    }
  };

  // Each group's shared keys: whole blocks of its prefix, for at least two
  // sequences.  Where the first sequence, whose table names the blocks, does
  // not hold them, every sequence of the group reads its own.  The groups have
  // to cover the sequences in order.
  if (tid == 0) s_alt = 0;
  __syncthreads();
  int bad = 0;
  int64_t pairs_sum = 0;
  for (int g = tid; g < NG; g += kPlanThreads) {
    const int s0 = w.cu_groups[g], s1 = w.cu_groups[g + 1], p = w.prefix_lens[g];
    int t0 = 0, tokens = 0, shared = 0;
    if (s0 < 0 || s1 < s0 || s1 > S || (g == 0 && s0 != 0) || (g == NG - 1 && s1 != S)) {
      bad = 1;
    } else if (s1 - s0 >= 2 && p >= a.block_size) {
      t0 = cu[s0];
      const int t1 = cu[s1], q0 = cu[s0 + 1] - t0, ctx0 = w.context_lens[s0];
      if (t0 >= 0 && t1 <= T && t1 > t0 && q0 >= 1 && ctx0 <= a.max_context_len && ctx0 - q0 >= p &&
          int64_t(ctx0) <= int64_t(a.max_blocks_per_seq) * a.block_size) {
        tokens = t1 - t0;
        shared = p / a.block_size * a.block_size;
        pairs_sum += ceil_div(tokens, 2 * TT);
        if (tokens <= TT) s_alt = 1;
      }
    }
    const int4 gr = make_int4(s0, t0, tokens, shared);
    w.groups[g] = gr;
    if (g < kGroupCache) gcache[g] = gr;
  }
  if (__syncthreads_or(bad)) {                     // no sequence can be told its prefix
    give_up();
    return;
  }
  int64_t all_pairs;
  block_scan(pairs_sum, warp_sums, all_pairs);
  if (all_pairs * Hkv > w.piece_cap) {             // only if token ranges overlap (malformed metadata)
    give_up();
    return;
  }
  const int alt_recs = s_alt ? 2 : 1;

  // Segments: the n that minimises the estimated time, n by thread.
  if (all_pairs == 0) {
    if (tid == 0) s_n = 1;
  } else if (tid < kMaxSegs) {
    const int n = tid + 1;
    float cost = 3.0e38f;
    int64_t pieces = 0;
    float work = 0.f;
    int longest = 0;
    for (int g = 0; g < NG; ++g) {
      const int4 gr = group(g);
      if (gr.w == 0) continue;
      const int units = ceil_div(gr.z, 2 * TT) * Hkv, tiles = ceil_div(gr.w, BN);
      const int len = ceil_div(tiles, n), segs = ceil_div(tiles, len);
      pieces += int64_t(units) * segs;
      work += float(units) * (float(tiles) + kPieceTiles * segs);
      longest = max(longest, len);
    }
    if (pieces <= w.piece_cap && int64_t(T) * H * n * alt_recs <= w.rec_cap) {
      const float one = float(longest) + kPieceTiles;
      const float waves = float((unsigned(pieces) + unsigned(w.num_sms) - 1) / unsigned(w.num_sms));
      // pieces of one size run in whole waves; unequal ones fill the gaps
      const float even = waves * one, filled = __fdividef(work, float(w.num_sms)) + 0.5f * one;
      cost = (NG == 1 ? even : fminf(even, fmaxf(filled, one))) + 0.05f * float(n);
    }
    best_cost[tid] = cost;
  }
  __syncthreads();
  if (tid == 0 && all_pairs > 0) {
    int n = 1;
    for (int k = 1; k < kMaxSegs; ++k)
      if (best_cost[k] < best_cost[n - 1]) n = k + 1;
    s_n = n;
  }
  __syncthreads();
  const int n = s_n, stride = n * alt_recs;

  // Each sequence: what its prefix covers, and the tiles of its own keys.
  int64_t unit_tiles = 0;
  for (int s = tid; s < S; s += kPlanThreads) {
    int lo = 0, hi = NG - 1;                       // the last group starting at or before s (empty groups start there too)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (group(mid).x <= s) lo = mid; else hi = mid - 1;
    }
    const int4 gr = group(lo);
    const int p = w.prefix_lens[lo], ctx = w.context_lens[s], c0 = cu[s], q_len = cu[s + 1] - c0;
    if (p < 0 || q_len < 1 || c0 < 0 || c0 + q_len > T || q_len > a.max_q_len || ctx < q_len || p > ctx - q_len ||
        ctx > a.max_context_len || int64_t(ctx) > int64_t(a.max_blocks_per_seq) * a.block_size) {
      raise_error(a.err, kErrInvalid);             // left out
      w.suffix_lens[s] = 0;
      w.seq_info[s] = make_int4(0, 0, 0, 0);
      continue;
    }
    const int tiles = ceil_div(gr.w, BN), len = gr.w > 0 ? ceil_div(tiles, n) : 1;
    const int segs = ceil_div(tiles, len);
    const bool chunk = is_chunk(w, q_len, G);
    w.suffix_lens[s] = ctx - gr.w;
    w.seq_info[s] = make_int4(gr.w / a.block_size, segs * (gr.z <= TT ? 2 : 1), 0, chunk ? 1 : 0);
    if (!chunk) unit_tiles += int64_t(ceil_div(q_len * G, kSuffixRows)) * Hkv * ceil_div(ctx - gr.w, kSuffixTile);
  }
  int64_t all_tiles;
  block_scan(unit_tiles, warp_sums, all_tiles);
  // chunk length: the suffix kernel's units come out even over its warps
  const int64_t per = (all_tiles + w.suffix_units - 1) / w.suffix_units;
  const int L = int(per < kMinChunkTiles ? kMinChunkTiles : (per > (1 << 26) ? (1 << 26) : per));

  // Items and records.  (Each thread reads back its own sequences' entries.)
  int64_t base = 0;                                // items in the low, records in the high word
  for (int s0 = 0; s0 < S; s0 += kPlanThreads) {
    const int s = s0 + tid;
    int64_t n_items = 0, n_recs = 0;
    int4 info = make_int4(0, 0, 0, 0);
    int own = 0, c0 = 0, q_len = 0, rt = 0, nch = 0;
    if (s < S) {
      own = w.suffix_lens[s];
      if (own > 0) {
        info = w.seq_info[s];
        c0 = cu[s];
        q_len = cu[s + 1] - c0;
        nch = info.w ? 1 : ceil_div(ceil_div(own, kSuffixTile), L);
        rt = info.w ? 0 : ceil_div(q_len * G, kSuffixRows);
        n_items = int64_t(rt) * nch;
        n_recs = info.y + nch > 1 ? int64_t(q_len) * H * nch : 0;
      }
    }
    int64_t total;
    const int64_t at = base + block_scan(n_items | (n_recs << 32), warp_sums, total);
    base += total;
    if ((base & 0xffffffff) > w.item_cap || (base >> 32) > w.own_cap) {   // only if token ranges overlap
      __syncthreads();
      give_up();
      return;
    }
    if (own > 0) {
      info.z = int(at >> 32);
      w.seq_info[s] = info;
      SuffixItem it;
      it.s = s, it.tok0 = c0, it.q_len = q_len, it.ctx = own, it.skip = info.x, it.base = info.z, it.nch = nch;
      it.direct = n_recs == 0;
      SuffixItem* out = w.items + (at & 0xffffffff);
      for (int r = 0; r < rt; ++r)
        for (int c = 0; c < nch; ++c) {
          it.row0 = r * kSuffixRows;
          it.chunk = c;
          it.k0 = c * L * kSuffixTile;
          it.k1 = min(own, it.k0 + L * kSuffixTile);
          *out++ = it;
        }
    }
  }
  __syncthreads();                                 // every sequence's info is written
  for (int t = tid; t < T; t += kPlanThreads) {
    int lo = t < S ? t : S - 1;
    if (cu[lo] != t) {                             // not all sequences before have one token
      lo = 0;
      int hi = S - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid - 1;
      }
    }
    int4 ti = make_int4(0, 0, 0, 0);
    const int own = w.suffix_lens[lo];
    if (own > 0 && cu[lo] <= t && t < cu[lo + 1]) {
      const int4 info = w.seq_info[lo];
      const int nch = info.w ? 1 : ceil_div(ceil_div(own, kSuffixTile), L);
      ti = make_int4(info.y, info.z + (t - cu[lo]) * H * nch, nch, 0);
    }
    w.token_info[t] = ti;
  }

  // the pieces: by segment, key/value head and row tile pair, so that the
  // pairs of one (segment, head) run side by side and share its K/V in L2
  int64_t pbase = 0;
  if (all_pairs > 0) {
    for (int g0 = 0; g0 < NG; g0 += kPlanThreads) {
      const int g = g0 + tid;
      int64_t count = 0;
      if (g < NG) {
        const int4 gr = group(g);
        if (gr.w > 0) {
          const int tiles = ceil_div(gr.w, BN), len = ceil_div(tiles, n);
          count = int64_t(ceil_div(gr.z, 2 * TT)) * Hkv * ceil_div(tiles, len);
        }
      }
      int64_t total;
      const int64_t at = pbase + block_scan(count, warp_sums, total);
      if (g < NG) w.first_piece[g] = int(at);
      pbase += total;
    }
    __syncthreads();
  }
  const int n_pieces = int(pbase);
  for (int i = tid; i < n_pieces; i += kPlanThreads) {
    int lo = 0, hi = NG - 1;                       // the last group whose pieces start at or before i
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (w.first_piece[mid] <= i) lo = mid; else hi = mid - 1;
    }
    const int4 gr = group(lo);
    const int tiles = ceil_div(gr.w, BN), len = ceil_div(tiles, n), pairs = ceil_div(gr.z, 2 * TT);
    const int local = i - w.first_piece[lo];
    const int pair = local % pairs, hk = local / pairs % Hkv, seg = local / (pairs * Hkv);
    // tokens evenly over the pairs
    const int each = gr.z / pairs, more = gr.z - each * pairs;
    const bool alt = gr.z <= TT;
    Piece pc = {};
    pc.s0 = gr.x;
    pc.tok0 = gr.y + pair * each + min(pair, more);
    pc.ntok = each + (pair < more ? 1 : 0);
    pc.hk = hk;
    pc.j0 = seg * len;
    pc.nt = min(len, tiles - seg * len);
    pc.shared = gr.w;
    pc.rec = alt ? 2 * seg : seg;
    pc.alt = alt;
    w.pieces[i] = pc;
  }
  if (tid == 0) set_header(n_pieces, stride, int(base & 0xffffffff));
}

// ------------------------------------------------------------------ prefix phase

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
// Packed fp32 pairs (Blackwell f32x2 FMA / add): two lanes of work per instruction.
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

__device__ __forceinline__ void tma_prefetch_l2_3d(const void* tmap, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// Warp-wide: lane i < 128/B looks up paged block i of KV tile j, stores its box
// index (or an out-of-range one: TMA fills zeros) in the ring slot of the
// piece's jl-th tile and asks TMA to prefetch that box into L2.
__device__ __forceinline__ void stage_boxes(int j, int jl, int B, int keys, const int32_t* bt, const AttnArgs& a,
                                            int hk, int lane, int* ring, const CUtensorMap* tm) {
  if (lane < BN / B) {
    const int lb = j * (BN / B) + lane;
    int z = a.num_blocks * a.num_kv_heads;
    if (lb * B < keys) {
      const int blk = bt[lb];
      if (blk >= 0 && blk < a.num_blocks) {
        z = blk * a.num_kv_heads + hk;
        tma_prefetch_l2_3d(tm, 0, 0, z);
        tma_prefetch_l2_3d(tm, 64, 0, z);
      } else {
        raise_error(a.err, kErrBounds);
      }
    }
    ring[(jl % kRing) * 8 + lane] = z;
  }
  __syncwarp();
}

__device__ __forceinline__ void load_kv_tile(uint32_t dst, const CUtensorMap* tm, uint32_t bar, int B, const int* zs) {
  for (int bi = 0; bi < BN / B; ++bi) {
    tma_load_3d(dst + bi * B * 128, tm, bar, 0, 0, zs[bi]);
    tma_load_3d(dst + kHalf + bi * B * 128, tm, bar, 64, 0, zs[bi]);
  }
}

// Persistent, one CTA per SM; pieces are claimed through header[3].  Roles and
// hand-offs as in the prefill kernel; every wait is bounded, and a timeout sets
// the device error word and winds the CTA down.
__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const AttnArgs a, const PrefixWork w) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;    // 128B-swizzled tiles need 1 KB alignment
  uint8_t* gsm = smem_raw + (base - raw);
  auto bar = [&](int i) -> uint32_t { return base + kOffBar + 8u * uint32_t(i); };
  Piece* items = reinterpret_cast<Piece*>(gsm + kOffItems);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int B = a.block_size;
  const int H = a.num_heads;
  const int G = H / a.num_kv_heads;                // query heads per key/value head
  const int TT = w.tile_tokens;

  asm volatile("griddepcontrol.wait;" ::: "memory");   // the plan kernels have finished
  int n_pieces = __ldcg(w.header);
  const int stride = __ldcg(w.header + 1);
  if (uint32_t(__ldcg(w.header + 2)) != w.tag || n_pieces < 0 || n_pieces > w.piece_cap) {
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(a.err, kErrInvalid);
    n_pieces = 0;
  }
  // the plan is complete: the kernel behind this one may start on the SMs that
  // this grid leaves
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (int(blockIdx.x) >= n_pieces) return;

  if (threadIdx.x == 0) {
    mbar_init(bar(BAR_Q), 1);
    mbar_init(bar(BAR_QE), 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(BAR_S + t), 1);
      mbar_init(bar(BAR_P + t), BM);
      mbar_init(bar(BAR_O + t), 1);
    }
    for (int st = 0; st < kKStages; ++st) {
      mbar_init(bar(BAR_KF + st), 1);
      mbar_init(bar(BAR_KE + st), 1);
    }
    for (int st = 0; st < kVStages; ++st) {
      mbar_init(bar(BAR_VF + st), 1);
      mbar_init(bar(BAR_VE + st), 1);
    }
    for (int i = 0; i < kItemSlots; ++i) {
      mbar_init(bar(BAR_IF + i), 1);
      mbar_init(bar(BAR_IE + i), kItemReaders);
    }
    mbar_init(bar(BAR_DONE), 1);
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(base + kOffTmemSlot, kTmemCols);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gsm + kOffTmemSlot);

  // A reader's view of piece n (nt = 0: no more pieces); `arrive`: this thread is its role's one arrival.
  auto read_item = [&](int n, bool arrive, Piece& it) -> bool {
    const int slot = n % kItemSlots;
    if (!mbar_wait(bar(BAR_IF + slot), (n / kItemSlots) & 1)) return false;
    it = items[slot];
    if (arrive) mbar_arrive(bar(BAR_IE + slot));
    return true;
  };

  if (warp == kWarpK) {
    // ------------------------------------------------------------ K loader (claims the pieces)
    int* ring = reinterpret_cast<int*>(gsm + kOffRing);
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
    }
    uint32_t kc = 0;
    int n = 0;
    bool ok = true;
    unsigned site = 0;
    for (;; ++n) {
      const int slot = n % kItemSlots;
      if (n >= kItemSlots && !__all_sync(0xffffffffu, mbar_wait(bar(BAR_IE + slot), ((n / kItemSlots) - 1) & 1))) {
        ok = false;
        site = kSitePfItemFree;
        break;
      }
      if (lane == 0) {
        Piece it = {};
        const int u = atomicAdd(w.header + 3, 1);
        if (u < n_pieces) {
          const int4* src = reinterpret_cast<const int4*>(w.pieces + u);
          int4* dst = reinterpret_cast<int4*>(&it);
          dst[0] = __ldcg(src);
          dst[1] = __ldcg(src + 1);
          dst[2] = __ldcg(src + 2);
        }
        items[slot] = it;
        mbar_arrive(bar(BAR_IF + slot));
      }
      __syncwarp();
      const Piece it = items[slot];
      if (it.nt == 0) break;
      const int nq = !it.alt && it.ntok > TT ? 2 : 1;
      const int32_t* bt = a.block_tables + size_t(it.s0) * a.max_blocks_per_seq;
      auto load_q = [&]() -> bool {
        if (n > 0 && !__all_sync(0xffffffffu, mbar_wait(bar(BAR_QE), (n - 1) & 1))) return false;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(BAR_Q), uint32_t(nq) * 2u * uint32_t(G * TT) * 128u);
          for (int t = 0; t < nq; ++t) {
            tma_load_3d(base + kOffQ + t * kTile, &tm_q, bar(BAR_Q), 0, it.hk * G, it.tok0 + t * TT);
            tma_load_3d(base + kOffQ + t * kTile + kHalf, &tm_q, bar(BAR_Q), 64, it.hk * G, it.tok0 + t * TT);
          }
        }
        __syncwarp();
        return true;
      };
      const int q_at = min(kKStages - 1, it.nt);   // K tiles requested before the Q load
      for (int j = 0; j < min(kLookAhead, it.nt); ++j)
        stage_boxes(it.j0 + j, j, B, it.shared, bt, a, it.hk, lane, ring, &tm_k);
      for (int j = 0; j < it.nt; ++j) {
        if (j == q_at && !load_q()) {
          ok = false;
          site = kSitePfQFree;
          break;
        }
        if (j + kLookAhead < it.nt)
          stage_boxes(it.j0 + j + kLookAhead, j + kLookAhead, B, it.shared, bt, a, it.hk, lane, ring, &tm_k);
        const uint32_t gk = kc + j;
        const int st = gk % kKStages;
        if (gk >= kKStages && !__all_sync(0xffffffffu, mbar_wait(bar(BAR_KE + st), ((gk / kKStages) - 1) & 1))) {
          ok = false;
          site = kSitePfKFree;
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(BAR_KF + st), kTile);
          load_kv_tile(base + kOffK + st * kTile, &tm_k, bar(BAR_KF + st), B, ring + (j % kRing) * 8);
        }
        __syncwarp();
      }
      if (ok && q_at == it.nt && !load_q()) {
        ok = false;
        site = kSitePfQFree;
      }
      if (!ok) break;
      kc += it.nt;
    }
    if (!ok && lane == 0) raise_error(a.err, kErrTimeout | site);
    if (lane == 0) {
      // (error path) let copies still in flight land before the CTA exits
      for (uint32_t gk = kc > uint32_t(kKStages) ? kc - kKStages : 0; gk < kc; ++gk)
        mbar_wait(bar(BAR_KF + gk % kKStages), (gk / kKStages) & 1);
      if (n > 0) mbar_wait(bar(BAR_Q), (n - 1) & 1);
    }
  } else if (warp == kWarpV) {
    // ------------------------------------------------------------ V loader
    int* ring = reinterpret_cast<int*>(gsm + kOffRing) + kRing * 8;
    if (lane == 0) tma_prefetch_desc(&tm_v);
    uint32_t vc = 0;
    bool ok = true;
    unsigned site = 0;
    for (int n = 0;; ++n) {
      Piece it;
      if (!__all_sync(0xffffffffu, read_item(n, false, it))) {
        ok = false;
        site = kSitePfItem;
        break;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_IE + n % kItemSlots));
      if (it.nt == 0) break;
      const int32_t* bt = a.block_tables + size_t(it.s0) * a.max_blocks_per_seq;
      for (int j = 0; j < min(kLookAhead, it.nt); ++j)
        stage_boxes(it.j0 + j, j, B, it.shared, bt, a, it.hk, lane, ring, &tm_v);
      for (int j = 0; j < it.nt; ++j) {
        if (j + kLookAhead < it.nt)
          stage_boxes(it.j0 + j + kLookAhead, j + kLookAhead, B, it.shared, bt, a, it.hk, lane, ring, &tm_v);
        const uint32_t gv = vc + j;
        const int st = gv % kVStages;
        if (gv >= kVStages && !__all_sync(0xffffffffu, mbar_wait(bar(BAR_VE + st), ((gv / kVStages) - 1) & 1))) {
          ok = false;
          site = kSitePfVFree;
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(BAR_VF + st), kTile);
          load_kv_tile(base + kOffV + st * kTile, &tm_v, bar(BAR_VF + st), B, ring + (j % kRing) * 8);
        }
        __syncwarp();
      }
      if (!ok) break;
      vc += it.nt;
    }
    if (!ok && lane == 0) raise_error(a.err, kErrTimeout | site);
    if (lane == 0)                                 // (error path) copies in flight land before the CTA exits
      for (uint32_t gv = vc > uint32_t(kVStages) ? vc - kVStages : 0; gv < vc; ++gv)
        mbar_wait(bar(BAR_VF + gv % kVStages), (gv / kVStages) & 1);
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ MMA
    if (lane == 0) {
      constexpr uint32_t idS = idesc_bf16_f32(BM, BN, false);   // Q (K-major) x K (K-major)
      constexpr uint32_t idO = idesc_bf16_f32(BM, HD, true);    // P (TMEM) x V (N-contiguous)
      const uint64_t dq0 = smem_desc(base + kOffQ, 16, 1024);
      const uint64_t dk0 = smem_desc(base + kOffK, 16, 1024);
      const uint64_t dv0 = smem_desc(base + kOffV, kHalf, 1024);
      // S of row tile `qt` into slot t
      auto issue_s = [&](int t, int qt, uint32_t gk) {
        const uint64_t kd = dk0 + (((gk % kKStages) * kTile) >> 4);
        const uint64_t qd = dq0 + ((qt * kTile) >> 4);
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          const uint32_t off16 = ((k / 4) * kHalf + (k % 4) * 32) >> 4;
          mma_f16_ss(tmem + 256 * t, qd + off16, kd + off16, idS, k > 0);
        }
        mma_commit(bar(BAR_S + t));
      };
      auto issue_pv = [&](int t, uint32_t gv, bool accumulate, bool last) {
        const uint64_t vd = dv0 + (((gv % kVStages) * kTile) >> 4);
#pragma unroll
        for (int k = 0; k < BN / 16; ++k)
          mma_f16_ts(tmem + 256 * t + 128, tmem + 256 * t + k * 8, vd + ((k * 2048) >> 4), idO, accumulate || k > 0);
        if (last) mma_commit(bar(BAR_O + t));
      };
      // Two row tiles, per KV tile j: P_0 V_j, S_0(j+1), P_1 V_j, S_1(j+1).
      // One row tile: P(j) V_j, S(j+2), both in slot j & 1.  Either way the S that
      // overwrites a slot comes right behind the P V that reads its P, which the
      // in-order execution of one thread's MMAs keeps safe.
      uint32_t kc = 0, vc = 0, cnt[2] = {0, 0};    // K, V tiles consumed; S/P phases of the slots
      bool ok = true;
      unsigned site = 0;
      auto wait = [&](int b, uint32_t parity, unsigned where) -> bool {
        if (mbar_wait(bar(b), parity & 1u)) return true;
        ok = false;
        site = where;
        return false;
      };
      for (int n = 0; ok; ++n) {
        Piece it;
        if (!read_item(n, true, it)) {
          ok = false;
          site = kSitePfItem;
          break;
        }
        if (it.nt == 0) break;
        if (!wait(BAR_Q, n, kSitePfQ)) break;
        if (it.alt) {
          for (int j = 0; ok && j < min(2, it.nt); ++j) {
            const uint32_t gk = kc + j;
            if (!wait(BAR_KF + gk % kKStages, gk / kKStages, kSitePfK)) break;
            tc_fence_after();
            issue_s(j, 0, gk);
            mma_commit(bar(BAR_KE + gk % kKStages));
            if (j + 1 == it.nt) mma_commit(bar(BAR_QE));
          }
          for (int j = 0; ok && j < it.nt; ++j) {
            const uint32_t gv = vc + j, t = j & 1;
            if (!wait(BAR_VF + gv % kVStages, gv / kVStages, kSitePfV)) break;
            if (!wait(BAR_P + t, (t == 0 ? cnt[0] : cnt[1]) + (j >> 1), kSitePfP)) break;
            tc_fence_after();
            issue_pv(t, gv, j >= 2, j + 2 >= it.nt);
            mma_commit(bar(BAR_VE + gv % kVStages));
            if (j + 2 < it.nt) {
              const uint32_t gk = kc + j + 2;
              if (!wait(BAR_KF + gk % kKStages, gk / kKStages, kSitePfK)) break;
              tc_fence_after();
              issue_s(t, 0, gk);
              mma_commit(bar(BAR_KE + gk % kKStages));
              if (j + 3 == it.nt) mma_commit(bar(BAR_QE));
            }
          }
          cnt[0] += (it.nt + 1) / 2;
          cnt[1] += it.nt / 2;
        } else {
          const int nq = it.ntok > TT ? 2 : 1;
          if (!wait(BAR_KF + kc % kKStages, kc / kKStages, kSitePfK)) break;
          tc_fence_after();
          for (int t = 0; t < nq; ++t) issue_s(t, t, kc);
          mma_commit(bar(BAR_KE + kc % kKStages));
          if (it.nt == 1) mma_commit(bar(BAR_QE));
          for (int j = 0; ok && j < it.nt; ++j) {
            const bool next = j + 1 < it.nt;
            const uint32_t gv = vc + j, gk = kc + j + 1;
            if (!wait(BAR_VF + gv % kVStages, gv / kVStages, kSitePfV)) break;
            for (int t = 0; t < nq; ++t) {
              if (!wait(BAR_P + t, (t == 0 ? cnt[0] : cnt[1]) + j, kSitePfP)) break;
              tc_fence_after();
              issue_pv(t, gv, j > 0, !next);
              if (t == nq - 1) mma_commit(bar(BAR_VE + gv % kVStages));
              if (next) {
                if (t == 0 && !wait(BAR_KF + gk % kKStages, gk / kKStages, kSitePfK)) break;
                tc_fence_after();
                issue_s(t, t, gk);
                if (t == nq - 1) {
                  mma_commit(bar(BAR_KE + gk % kKStages));
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
    // ------------------------------------------------------------ softmax of slot t
    const int t = warp >> 2;
    const int wq = warp & 3;                       // TMEM lane quarter
    const int i = threadIdx.x - BM * t;            // tile row = TMEM lane
    const uint32_t lane_base = tmem + (uint32_t(wq * 32) << 16) + 256 * t;
    const float sl2 = a.scale_log2;
    uint32_t cnt = 0, ocnt = 0;                    // S/P phases and O phases of this slot consumed
    bool ok = true;
    unsigned site = 0;
    for (int n = 0; ok; ++n) {
      Piece it;
      if (!__all_sync(0xffffffffu, read_item(n, false, it))) {
        ok = false;
        site = kSitePfItem;
        break;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_IE + n % kItemSlots));
      if (it.nt == 0) break;
      // this slot's rows and KV tiles j = first, first + step, ...
      const int tok0 = it.alt ? it.tok0 : it.tok0 + t * TT;
      const int ntok = it.alt ? it.ntok : min(TT, it.ntok - t * TT);
      const int step = it.alt ? 2 : 1, first = it.alt ? t : 0;
      if (ntok <= 0) continue;                     // no rows in the second tile
      const int rows = ntok * G;
      const int steps = (it.nt - first + step - 1) / step;
      const bool work = wq * 32 < rows;            // some row of this warp is real
      float m = -INFINITY, l = 0.f;
      for (int x = 0; x < steps; ++x) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar(BAR_S + t), (cnt + x) & 1))) {
          ok = false;
          site = kSitePfS;
          break;
        }
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
        if (kb + BN > it.shared) {                 // keys behind the prefix
#pragma unroll
          for (int c = 0; c < BN; ++c)
            if (kb + c >= it.shared) sr[c] = __float_as_uint(-INFINITY);
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < BN; c += 8)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            m4[u] = max3(m4[u], __uint_as_float(sr[c + 2 * u]), __uint_as_float(sr[c + 2 * u + 1]));
        const float mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        const float m_new = fmaxf(m, mt * sl2);
        const bool resc = m_new > m + 8.0f;        // keep a stale max while exp2 stays <= 2^8
        const float m_use = resc ? m_new : m;
        const float alpha = resc ? ex2(m - m_new) : 1.0f;
        const float m_sub = m_use == -INFINITY ? 0.f : m_use;   // scores all -inf so far
        const uint64_t scale2 = f2_pack(sl2, sl2), neg_m2 = f2_pack(-m_sub, -m_sub);
        uint64_t sum2[4] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f), f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 64; ++c) {             // P, rounded to bf16 for the tensor core, over the scores
          float x0, x1;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[2 * c]), __uint_as_float(sr[2 * c + 1])), scale2, neg_m2), x0, x1);
          const float p0 = ex2(x0), p1 = ex2(x1);
          sum2[c & 3] = f2_add(sum2[c & 3], f2_pack(p0, p1));
          sr[c] = pack_bf16x2(p0, p1);
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
        if (!__all_sync(0xffffffffu, mbar_wait(bar(BAR_O + t), ocnt & 1))) {
          ok = false;
          site = kSitePfO;
          break;
        }
        tc_fence_after();
        ++ocnt;
      }
      cnt += steps;
      // the row's record of this segment (in the alternating mode, of its even or odd tiles)
      const bool real = i < rows;
      float* rec = w.recs + ((size_t(tok0 + i / G) * H + it.hk * G + i % G) * stride + it.rec + (it.alt ? t : 0)) * kPrefixRec;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        if (steps > 0) {
          tmem_ld32(lane_base + 128 + 32 * c, o);
          tmem_wait_ld();
        } else {                                   // no odd tile: an empty record
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        if (real) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            __stcg(reinterpret_cast<uint4*>(rec + 32 * c + e), make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]));
        }
      }
      if (real) __stcg(reinterpret_cast<float2*>(rec + HD), make_float2(m, l));
      tc_fence_before();                           // O read before the next piece's first P V overwrites it
    }
    if (!ok && lane == 0) raise_error(a.err, kErrTimeout | site);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

std::mutex g_attr_mutex;
bool g_attr_set[64] = {};

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Capacities of a step's lists, and whether the step may hold prefill chunks.
struct PrefixSizes {
  size_t S, T, NG, pieces, items, recs, own, units;
  bool chunks;
};
PrefixSizes prefix_sizes(int32_t num_q_heads, int32_t num_kv_heads, int32_t num_seqs, int32_t num_tokens, int32_t num_groups) {
  PrefixSizes z;
  z.S = size_t(num_seqs), z.T = size_t(num_tokens), z.NG = size_t(num_groups);
  const size_t G = size_t(num_q_heads / num_kv_heads), rows = z.T * size_t(num_q_heads);
  // a group that shares has two sequences or more
  z.pieces = size_t(num_kv_heads) * (z.T / (2 * size_t(prefix_tile_tokens(int(G)))) + std::min(z.NG, z.S / 2) + 1) + kExtraPieces;
  z.recs = std::min(rows * 2 * kMaxSegs, rows * 2 + size_t(kExtraRecs));
  z.units = size_t(kMaxSms) * kSuffixWarps * kUnitsPerWarp;
  // ceil(x / L) <= x / L + 1 for every sequence, and all x / L together are at most `units`
  z.items = z.T * G / kSuffixRows + z.S + z.units + 1;
  z.own = rows + kSuffixRows * z.units;
  z.chunks = z.T > z.S && (z.T - z.S + 1) * G > size_t(kMaxWarpRows);
  return z;
}

}  // namespace

int prefix_tile_tokens(int group_heads) { return BM / group_heads; }

size_t prefix_workspace_bytes(int32_t num_q_heads, int32_t num_kv_heads, int32_t num_seqs, int32_t num_tokens,
                              int32_t num_groups, int32_t head_dim, int32_t max_context_len) {
  const PrefixSizes z = prefix_sizes(num_q_heads, num_kv_heads, num_seqs, num_tokens, num_groups);
  return 256 + align256(z.S * 4) + align256(z.S * 16) + align256(z.NG * 16) + align256((z.NG + 1) * 4) +
         align256(z.pieces * sizeof(Piece)) + align256(z.items * sizeof(SuffixItem)) + align256(z.T * 16) +
         align256(z.recs * kPrefixRec * sizeof(float)) + align256(z.own * kPrefixRec * sizeof(float)) +
         (z.chunks ? step_workspace_bytes(num_seqs, num_tokens, num_q_heads, head_dim, max_context_len) : 0);
}

static cb_status launch_prefix_tc(const AttnArgs& a, const PrefixWork& w, cudaStream_t stream) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return CB_ERR_CUDA;
  const int G = a.num_heads / a.num_kv_heads, B = a.block_size;
  CUtensorMap tq, tk, tv;
  const cuuint32_t ones[3] = {1, 1, 1};
  {
    // q as [tokens][heads][128]: a box is one key/value head's query heads of tile_tokens tokens, one 64-dim half
    const cuuint64_t dims[3] = {cuuint64_t(HD), cuuint64_t(a.num_heads), cuuint64_t(a.num_tokens)};
    const cuuint64_t strides[2] = {cuuint64_t(HD) * 2, cuuint64_t(a.num_heads) * HD * 2};
    const cuuint32_t box[3] = {64, cuuint32_t(G), cuuint32_t(w.tile_tokens)};
    CUresult r = enc(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides, box, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(CB_ERR_CUDA, "shared prefixes: encoding the Q tensor map failed (%d)", int(r));
  }
  const cuuint64_t dims[3] = {cuuint64_t(HD), cuuint64_t(B), cuuint64_t(a.num_blocks) * a.num_kv_heads};
  const cuuint64_t strides[2] = {cuuint64_t(HD) * 2, cuuint64_t(B) * HD * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(B), 1};
  CUresult r = enc(&tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.k_pool), dims, strides, box, ones,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r == CUDA_SUCCESS)
    r = enc(&tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.v_pool), dims, strides, box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(CB_ERR_CUDA, "shared prefixes: encoding the KV tensor maps failed (%d)", int(r));
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
    return fail(CB_ERR_UNSUPPORTED, "shared prefixes: no usable current device");
  {
    std::lock_guard<std::mutex> lock(g_attr_mutex);
    if (!g_attr_set[dev]) {
      cudaError_t e = cudaFuncSetAttribute(prefix_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmemBytes));
      if (e != cudaSuccess) return cuda_fail(e, "shared prefixes: shared memory attribute");
      g_attr_set[dev] = true;
    }
  }
  const int64_t grid = std::min<int64_t>(w.num_sms, w.piece_cap);
  cudaError_t e = launch_kernel(prefix_tc_kernel, dim3(unsigned(grid)), dim3(kThreads), kSmemBytes, stream, true, tq, tk, tv,
                                a, w);
  return e == cudaSuccess ? CB_OK : cuda_fail(e, "shared prefixes: launch");
}

// A step with shared prefixes on one stream: the plan, the prefix kernel, the
// kernels of the rows' own keys and the join.  Each starts as a programmatic
// dependent of the one before: the own keys' kernel runs beside the prefix
// kernel on the SMs that one leaves, and ends only after it.
cb_status run_shared_prefix(AttnArgs a, const int32_t* cu_groups, const int32_t* prefix_lens, int32_t num_groups,
                            void* workspace, cudaStream_t stream) {
  NvtxRange nvtx("cb.shared_prefix");
  if (int64_t(a.num_blocks) * a.num_kv_heads >= (int64_t(1) << 31))
    return fail(CB_ERR_UNSUPPORTED, "shared prefixes: num_blocks * num_kv_heads must fit in int32");
  const int G = a.num_heads / a.num_kv_heads;
  const PrefixSizes z = prefix_sizes(a.num_heads, a.num_kv_heads, a.num_seqs, a.num_tokens, num_groups);
  if (z.pieces > 0x7FFFFFFF || z.items > size_t(0x7FFFFFFF / a.num_kv_heads) || z.own > 0x7FFFFFFF)
    return fail(CB_ERR_UNSUPPORTED, "shared prefixes: too many tokens");
  PrefixWork w;
  w.cu_groups = cu_groups;
  w.prefix_lens = prefix_lens;
  w.context_lens = a.context_lens;
  w.num_groups = num_groups;
  w.num_sms = sm_count();
  w.tile_tokens = prefix_tile_tokens(G);
  // a sequence has at most num_tokens - num_seqs + 1 tokens, which z.chunks says
  const bool chunks = z.chunks && a.max_q_len > 1 && int64_t(a.max_q_len) * G > kMaxWarpRows;
  w.max_warp_rows = chunks ? kMaxWarpRows : INT32_MAX;
  w.suffix_units = std::min(w.num_sms, kMaxSms) * kSuffixWarps * kUnitsPerWarp;
  w.piece_cap = int32_t(z.pieces);
  w.item_cap = int32_t(z.items);
  w.rec_cap = int64_t(z.recs);
  w.own_cap = int64_t(z.own);
  char* p = static_cast<char*>(workspace);
  auto take = [&p](size_t bytes) {
    char* at = p;
    p += align256(bytes);
    return at;
  };
  w.header = reinterpret_cast<int32_t*>(take(256));
  w.suffix_lens = reinterpret_cast<int32_t*>(take(z.S * 4));
  w.seq_info = reinterpret_cast<int4*>(take(z.S * 16));
  w.groups = reinterpret_cast<int4*>(take(z.NG * 16));
  w.first_piece = reinterpret_cast<int32_t*>(take((z.NG + 1) * 4));
  w.pieces = reinterpret_cast<Piece*>(take(z.pieces * sizeof(Piece)));
  w.items = reinterpret_cast<SuffixItem*>(take(z.items * sizeof(SuffixItem)));
  w.token_info = reinterpret_cast<int4*>(take(z.T * 16));
  w.recs = reinterpret_cast<float*>(take(z.recs * kPrefixRec * sizeof(float)));
  w.own_recs = reinterpret_cast<float*>(take(z.own * kPrefixRec * sizeof(float)));
  static std::atomic<uint32_t> next_tag{1};
  w.tag = next_tag.fetch_add(1);

  prefix_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a, w);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "shared prefixes: plan launch");
  AttnArgs own = a;                                // the prefill chunks' view of the step
  StepPlan plan;
  cb_status st;
  if (chunks) {
    const size_t bytes = step_workspace_bytes(a.num_seqs, a.num_tokens, a.num_heads, a.head_dim, a.max_context_len);
    st = step_plan_layout(p, bytes, a.num_seqs, a.num_tokens, a.num_heads, a.head_dim, a.max_context_len, &plan);
    if (st != CB_OK) return st;
    own.context_lens = w.suffix_lens;
    own.prefix.seq_info = reinterpret_cast<const int32_t*>(w.seq_info);
    own.prefix.recs = w.own_recs;
    set_decode_plan(own, &plan);
    st = launch_plan(own, plan, stream);
    if (st != CB_OK) return st;
  }
  st = launch_prefix_tc(a, w, stream);
  if (st != CB_OK) return st;
  if (chunks) {
    st = launch_prefill_tc(own, plan, true, stream);
    if (st != CB_OK) return st;
  }
  st = launch_suffix(a, w, stream);
  if (st != CB_OK) return st;
  return launch_join(a, w, stream);
}

}  // namespace cb
