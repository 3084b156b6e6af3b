// Attention of a step whose sequences share prefixes: the keys that every
// sequence of a group has in common are read once for all of its query rows
// (bf16, head_dim 128).
//
// A decode step reads every sequence's whole cache; where sequences continue
// one prompt, most of those bytes are the same pages again and again.  For a
// group of sequences with R query tokens and G query heads per key/value head,
// the prefix phase is, per key/value head, a dense product of R * G query rows
// with the prefix's keys: softmax(Q K^T) V over those keys, left unnormalised
// as one record (acc, max, sum) per row and KV segment.  A sequence's own keys,
// behind the prefix, leave records too, and a last kernel joins each row's.
//
// What bounds it: the prefix's K and V once from HBM while R * G is below about
// 256 rows (the ridge of 4 flops per row and byte pair), the tensor cores
// above; the own keys once from HBM.  So
//   * the rows of all query heads of a key/value head are packed into the
//     128-row tcgen05 tile (row = token * G + head).  A piece of work is two row
//     tiles against a KV segment, in ping-pong as in the prefill kernel; where
//     there is only one row tile, its KV tiles alternate over the two score and
//     output buffers, the even ones on one softmax warpgroup and the odd ones on
//     the other, each with its own record, so that the two halves of the softmax
//     work and the tensor core's overlap all the same;
//   * own keys of sequences with many query rows (chunks) are pieces too, with
//     their causal mask; those of the few rows of a decoding sequence are streams
//     of single warps (suffix_stream.cuh);
//   * both run in one launch: some CTAs take pieces first, the others stream own
//     keys at once, and whoever runs out of pieces goes on to the streams;
//   * the plan, one CTA, cuts the pieces' KV ranges and splits the SMs by
//     estimated time.  Every segment costs the join one more record per row.
#include <algorithm>
#include <atomic>
#include <mutex>

#include <cuda.h>

#include "device_common.cuh"
#include "kernels.h"
#include "runtime.h"
#include "shared_prefix.h"
#include "sm100_ptx.cuh"
#include "suffix_stream.cuh"

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
  BAR_VTAIL = BAR_VE + kVStages,   // V landed, its stale rows still to be zeroed
  BAR_IF = BAR_VTAIL + 1,      // + slot: piece published
  BAR_IE = BAR_IF + kItemSlots,  // + slot: piece read by every role
  BAR_DONE = BAR_IE + kItemSlots,
  NUM_BARS = BAR_DONE + 1
};
constexpr uint32_t kOffTmemSlot = kOffBar + 16 * ((NUM_BARS + 1) / 2);
constexpr uint32_t kOffItems = kOffTmemSlot + 16;
constexpr int kLookAhead = 4;                    // tiles ahead of the loads that are prefetched into L2
constexpr uint32_t kOffOwnBars = kOffItems + kItemSlots * uint32_t(sizeof(Piece));   // streams: barriers, items;
constexpr uint32_t kOffOwnSlots = kOffOwnBars + stream::kBarBytes;                  // their rings lie over the tiles
constexpr uint32_t kSmemBytes = kOffOwnSlots + stream::kSlotBytes + 1024;   // + slack to align the base
static_assert(kOffItems % 16 == 0 && kOffOwnSlots % 16 == 0, "pieces and items are copied 16 bytes at a time");
static_assert(stream::kRingBytes <= kOffBar, "the streams' rings");
static_assert(kSmemBytes <= 232448, "shared memory budget");

// ------------------------------------------------------------------ plan

constexpr int kPlanThreads = 512;
constexpr int kMaxSegs = 64;             // KV segments of a prefix, or of a chunk's own keys
constexpr int kGroupCache = 512;         // groups kept in shared memory
constexpr int kSeqCache = 1024;          // sequences kept in shared memory
constexpr int kExtraPieces = 1024;       // pieces beyond one per (row tile pair, key/value head)
constexpr int64_t kExtraRecs = 131072;   // records beyond two per row (69 MB)
constexpr int kMinChunkTiles = 8;        // shortest chunk of streamed keys, in 16-key tiles
constexpr int kStreamRows = 16;          // query rows per row tile of a stream
constexpr int kUnitsPerWarp = 3;         // streamed units that each warp should get
constexpr int kMaxSms = 160;             // SMs that the lists are sized for
// Query rows per key/value head up to which a sequence's own keys are streamed,
// once per 16 rows; beyond, they are pieces.
constexpr int kMaxStreamRows = 64;
// Cost model of the segments and of the SM split, in microseconds and bytes.
constexpr float kTileUsTwo = 1.95f;      // a KV tile against two row tiles, one SM
constexpr float kTileUsOne = 1.2f;       // a KV tile against one row tile
constexpr float kPieceUs = 3.0f;         // a piece beyond its tiles: Q, the pipeline's fill, the records
constexpr float kBytesPerUs = 6.4e6f;    // HBM
constexpr float kStreamBytesPerUsPerSm = 6.0e4f;
constexpr float kJoinBytesPerUs = 4.0e6f;
constexpr int kSmSteps = 19;             // SM splits that are scored: 1/19 .. 19/19 of the SMs

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

// Block-wide sums of three values, in every thread.  Contains __syncthreads;
// `sums` holds 3 per warp.
__device__ void block_sums(int64_t& x, int64_t& y, int64_t& z, int64_t* sums) {
  constexpr int kW = kPlanThreads / 32;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    x += __shfl_xor_sync(0xffffffffu, x, o);
    y += __shfl_xor_sync(0xffffffffu, y, o);
    z += __shfl_xor_sync(0xffffffffu, z, o);
  }
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) sums[warp] = x, sums[kW + warp] = y, sums[2 * kW + warp] = z;
  __syncthreads();
  x = y = z = 0;
#pragma unroll
  for (int w = 0; w < kW; ++w) x += sums[w], y += sums[kW + w], z += sums[2 * kW + w];
  __syncthreads();
}

// The segments of a range of keys where none is longer than `longest` KV tiles:
// their number and length.
__device__ __forceinline__ int2 segments(int keys, int longest) {
  const int tiles = ceil_div(keys, BN);
  const int len = ceil_div(tiles, ceil_div(tiles, longest));
  return make_int2(ceil_div(tiles, len), len);
}

// A sequence as the plan sees it; own = 0: left out.
struct SeqPlan {
  int own, c0, q_len, group;
};

// Rows that a set of pieces has in common: a group's over its prefix, or a
// chunk's over its own keys.  keys = 0: none.
struct Job {
  int keys, tok0, tokens, s0, skip, lim0;
};

// One CTA.  Checks the groups, chooses the segments of the pieces and the
// chunks of the streams, lists both and gives every row its records.
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const AttnArgs a, const PrefixWork w) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // they wait for this grid on the device
  __shared__ int64_t warp_sums[3 * (kPlanThreads / 32)];
  __shared__ float n_work[kMaxSegs], n_piece[kMaxSegs];
  __shared__ int n_pieces_of[kMaxSegs];
  __shared__ int4 gcache[kGroupCache];
  __shared__ SeqPlan scache[kSeqCache];
  __shared__ unsigned long long s_best;
  __shared__ int s_alt, s_tiles;
  const int tid = threadIdx.x;
  const int S = a.num_seqs, T = a.num_tokens, NG = w.num_groups, TT = w.tile_tokens;
  const int H = a.num_heads, Hkv = a.num_kv_heads, G = H / Hkv;
  const int32_t* cu = a.cu_seqlens_q;
  const bool chunks = int64_t(a.max_q_len) * G > kMaxStreamRows && a.max_q_len > 1;   // some sequence's own keys may be pieces
  auto group = [&](int g) -> int4 { return g < kGroupCache ? gcache[g] : w.groups[g]; };
  auto set_header = [&](int pieces, int stride, int items, int working) {
    w.header[0] = pieces;
    w.header[1] = stride;
    w.header[2] = int32_t(w.tag);
    w.header[3] = 0;
    w.header[4] = items;
    w.header[5] = 0;
    w.header[6] = working;
  };
  // nothing runs and no row is written
  auto give_up = [&]() {
    __syncthreads();
    for (int t = tid; t < T; t += kPlanThreads) w.token_info[t] = make_int4(0, 0, 0, 0);
    if (tid == 0) {
      raise_error(a.err, kErrInvalid);
      set_header(0, 0, 0, 0);
    }
  };

  // Each group's shared keys: whole blocks of its prefix, for at least two
  // sequences.  Where the first sequence, whose table names the blocks, does
  // not hold them, every sequence of the group reads its own.  The groups have
  // to cover the sequences in order.
  if (tid == 0) {
    s_alt = 0;
    s_tiles = 1;
    s_best = ~0ull;
  }
  __syncthreads();
  int bad = 0, tiles_max = 1;
  int64_t n_first = 0;                             // pieces if nothing is cut, per key/value head
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
        n_first += ceil_div(tokens, 2 * TT);
        tiles_max = max(tiles_max, ceil_div(shared, BN));
        if (tokens <= TT) s_alt = 1;
      }
    }
    const int4 gr = make_int4(s0, t0, tokens, shared);
    if (g < kGroupCache) gcache[g] = gr;
    else w.groups[g] = gr;
  }
  if (__syncthreads_or(bad)) {                     // no sequence can be told its prefix
    give_up();
    return;
  }

  // Each sequence: its group and own keys.
  auto seq_plan = [&](int s) -> SeqPlan {
    int lo = 0, hi = NG - 1;                       // the last group starting at or before s (empty groups start there too)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (group(mid).x <= s) lo = mid; else hi = mid - 1;
    }
    const int p = w.prefix_lens[lo], ctx = w.context_lens[s], c0 = cu[s], q_len = cu[s + 1] - c0;
    const bool ok = p >= 0 && q_len >= 1 && c0 >= 0 && c0 + q_len <= T && q_len <= a.max_q_len && ctx >= q_len &&
                    p <= ctx - q_len && ctx <= a.max_context_len &&
                    int64_t(ctx) <= int64_t(a.max_blocks_per_seq) * a.block_size;
    return SeqPlan{ok ? ctx - group(lo).w : 0, c0, q_len, lo};
  };
  auto seq = [&](int s) -> SeqPlan { return s < kSeqCache ? scache[s] : seq_plan(s); };
  auto is_chunk = [&](const SeqPlan& q) { return q.own > 0 && q.q_len > 1 && int64_t(q.q_len) * G > kMaxStreamRows; };
  // job j: group j's prefix, then sequence (j - NG)'s own keys
  const int jobs = NG + (chunks ? S : 0);
  auto job = [&](int j) -> Job {
    if (j < NG) {
      const int4 gr = group(j);
      return Job{gr.w, gr.y, gr.z, gr.x, 0, gr.w};
    }
    const SeqPlan q = seq(j - NG);
    if (!is_chunk(q)) return Job{0, 0, 0, 0, 0, 0};
    return Job{q.own, q.c0, q.q_len, j - NG, group(q.group).w / a.block_size, q.own - q.q_len + 1};
  };
  int64_t unit_tiles = 0, own_keys = 0;            // streamed units' tiles and keys
  for (int s = tid; s < S; s += kPlanThreads) {
    const SeqPlan q = seq_plan(s);
    if (s < kSeqCache) scache[s] = q;
    if (q.own == 0) {
      raise_error(a.err, kErrInvalid);             // left out
    } else if (!is_chunk(q)) {
      unit_tiles += int64_t(ceil_div(q.q_len * G, kStreamRows)) * Hkv * ceil_div(q.own, stream::kTileKeys);
      own_keys += q.own;
    } else {
      n_first += ceil_div(q.q_len, 2 * TT);
      tiles_max = max(tiles_max, ceil_div(q.own, BN));
    }
  }
  for (int t = tid; t < T; t += kPlanThreads) w.token_info[t] = make_int4(0, 0, 0, 0);
  tiles_max = __reduce_max_sync(0xffffffffu, tiles_max);
  if ((tid & 31) == 0) atomicMax(&s_tiles, tiles_max);
  int64_t all_first = n_first, all_tiles = unit_tiles, all_keys = own_keys;
  block_sums(all_first, all_tiles, all_keys, warp_sums);
  if (all_first * Hkv > w.piece_cap) {             // only if token ranges overlap (malformed metadata)
    give_up();
    return;
  }
  const int alt_recs = s_alt ? 2 : 1;
  tiles_max = s_tiles;

  // Segments: no longer than the longest range / n, and the SMs that take pieces
  // first; the rest streams own keys beside them, which leaves the tensor cores
  // idle as large groups' pieces do HBM.  First the pieces of every n, then
  // every (n, SMs) is scored.
  int longest = 1, working = w.num_sms, n_segs = 1;
  if (all_first > 0) {
    constexpr int kLanes = kPlanThreads / kMaxSegs;   // threads per n, each with a share of the jobs
    {
      const int n = tid / kLanes + 1, len = ceil_div(tiles_max, n);
      int64_t pieces = 0, own_recs = 0;
      float work = 0.f, piece = 0.f;
      for (int j = tid % kLanes; j < jobs; j += kLanes) {
        const Job jb = job(j);
        if (jb.keys == 0) continue;
        const int2 sg = segments(jb.keys, len);
        const int64_t units = int64_t(ceil_div(jb.tokens, 2 * TT)) * Hkv * sg.x;
        const bool alt = jb.tokens <= TT;
        const float us = float(sg.y) * (alt ? kTileUsOne : kTileUsTwo) + kPieceUs;
        pieces += units;
        if (j >= NG) own_recs += int64_t(jb.tokens) * H * sg.x * (alt ? 2 : 1);
        work += float(units) * us;
        piece = fmaxf(piece, us);
      }
#pragma unroll
      for (int x = kLanes / 2; x > 0; x >>= 1) {
        pieces += __shfl_xor_sync(0xffffffffu, pieces, x);
        own_recs += __shfl_xor_sync(0xffffffffu, own_recs, x);
        work += __shfl_xor_sync(0xffffffffu, work, x);
        piece = fmaxf(piece, __shfl_xor_sync(0xffffffffu, piece, x));
      }
      if (tid % kLanes == 0) {
        const bool fits = pieces <= w.piece_cap && int64_t(T) * H * n * alt_recs <= w.prefix_rec_cap &&
                          own_recs <= w.piece_rec_cap;
        n_pieces_of[n - 1] = fits ? int(pieces) : 0;
        n_work[n - 1] = work;
        n_piece[n - 1] = piece;
      }
    }
    float piece_bytes = 0.f;                       // K and V bytes of the pieces, once
    for (int j = tid & 31; j < jobs; j += 32) piece_bytes += float(job(j).keys);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) piece_bytes += __shfl_xor_sync(0xffffffffu, piece_bytes, x);
    const float key_bytes = 4.0f * HD * float(Hkv);
    piece_bytes *= key_bytes;
    const float own_bytes = float(all_keys) * key_bytes;
    __syncthreads();
    unsigned long long best = ~0ull;
    for (int i = tid; i < kMaxSegs * kSmSteps; i += kPlanThreads) {
      const int n = i / kSmSteps, k = (i % kSmSteps + 1) * w.num_sms / kSmSteps;
      const int pieces = n_pieces_of[n];
      if (pieces == 0 || k < 1 || (own_bytes == 0.f && k < w.num_sms)) continue;
      // pieces of one size run in whole waves; unequal ones fill the gaps
      const float waves = ceilf(__fdividef(float(pieces), float(k))) * n_piece[n];
      float us = fminf(waves, __fdividef(n_work[n], float(k)) + n_piece[n]);
      us = fmaxf(us, piece_bytes * (1.0f / kBytesPerUs));
      const float beside = fminf(kBytesPerUs * us - piece_bytes, float(w.num_sms - k) * kStreamBytesPerUsPerSm * us);
      us += fmaxf(0.f, own_bytes - beside) * (1.0f / kBytesPerUs);
      us += float(T) * float(H) * float((n + 1) * alt_recs) * (kPrefixRec * 4.0f / kJoinBytesPerUs);
      const unsigned long long key = ((unsigned long long)(__float_as_uint(us)) << 32) | unsigned(i);
      best = key < best ? key : best;
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
      const unsigned long long other = __shfl_xor_sync(0xffffffffu, best, x);
      best = other < best ? other : best;
    }
    if ((tid & 31) == 0) atomicMin(&s_best, best);
    __syncthreads();
    if (s_best == ~0ull) {                         // n = 1 fits unless token ranges overlap
      give_up();
      return;
    }
    const int i = int(unsigned(s_best));
    n_segs = i / kSmSteps + 1;
    working = (i % kSmSteps + 1) * w.num_sms / kSmSteps;
    longest = ceil_div(tiles_max, n_segs);
  }
  const int stride = n_segs * alt_recs;
  const unsigned own_rec0 = unsigned(w.prefix_rec_cap);
  // chunk length: the streamed units come out even over the warps
  const int64_t per = (all_tiles + w.stream_units - 1) / w.stream_units;
  const int L = int(per < kMinChunkTiles ? kMinChunkTiles : (per > (1 << 26) ? (1 << 26) : per));
  // records per (token, head) of a group's prefix and of a sequence's own keys
  auto prefix_recs = [&](int g) -> int {
    const int4 gr = group(g);
    return gr.w > 0 ? segments(gr.w, longest).x * (gr.z <= TT ? 2 : 1) : 0;
  };
  auto own_recs_of = [&](const SeqPlan& q) -> int {
    return is_chunk(q) ? segments(q.own, longest).x * (q.q_len <= TT ? 2 : 1) : ceil_div(ceil_div(q.own, stream::kTileKeys), L);
  };

  // Streamed items, and every sequence's own records.
  int64_t base = 0;                                // items in the low, records in the high word
  for (int s0 = 0; s0 < S; s0 += kPlanThreads) {
    const int s = s0 + tid;
    int64_t n_items = 0, n_recs = 0;
    SeqPlan q = {0, 0, 0, 0};
    int pre = 0, rt = 0, nch = 0;
    if (s < S) q = seq(s);
    if (q.own > 0) {
      pre = prefix_recs(q.group);
      nch = own_recs_of(q);
      rt = is_chunk(q) ? 0 : ceil_div(q.q_len * G, kStreamRows);
      n_items = int64_t(rt) * nch;
      n_recs = pre + nch > 1 ? int64_t(q.q_len) * H * nch : 0;
    }
    int64_t total;
    const int64_t at = base + block_scan(n_items | (n_recs << 32), warp_sums, total);
    base += total;
    if ((base & 0xffffffff) > w.item_cap || (base >> 32) > w.own_rec_cap) {   // only if token ranges overlap
      give_up();
      return;
    }
    if (q.own > 0) {
      const unsigned rec = own_rec0 + unsigned(at >> 32);
      if (a.max_q_len > 1) w.seq_rec[s] = rec;
      if (a.max_q_len == 1) w.token_info[q.c0] = make_int4(pre, int(rec), nch, 0);
      SuffixItem it = {};
      it.s = s, it.tok0 = q.c0, it.q_len = q.q_len, it.ctx = q.own, it.skip = group(q.group).w / a.block_size;
      it.rec_step = nch;
      it.direct = n_recs == 0;
      SuffixItem* out = w.items + (at & 0xffffffff);
      for (int r = 0; r < rt; ++r)
        for (int c = 0; c < nch; ++c) {
          it.row0 = r * kStreamRows;
          it.rec0 = rec + c;
          it.k0 = c * L * stream::kTileKeys;
          it.k1 = min(q.own, it.k0 + L * stream::kTileKeys);
          *out++ = it;
        }
    }
  }
  if (a.max_q_len > 1) {                           // every token's sequence by search
    __syncthreads();
    for (int t = tid; t < T; t += kPlanThreads) {
      int lo = 0, hi = S - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((mid < kSeqCache ? scache[mid].c0 : cu[mid]) <= t) lo = mid; else hi = mid - 1;
      }
      const SeqPlan q = seq(lo);
      if (q.own > 0 && q.c0 <= t && t < q.c0 + q.q_len) {
        const int nch = own_recs_of(q);
        w.token_info[t] = make_int4(prefix_recs(q.group), int(w.seq_rec[lo] + unsigned((t - q.c0) * H * nch)), nch, 0);
      }
    }
  }

  // the pieces: by segment, key/value head and row tile pair, so that the
  // pairs of one (segment, head) run side by side and share its K/V in L2
  int64_t pbase = 0;
  if (all_first > 0) {
    for (int j0 = 0; j0 < jobs; j0 += kPlanThreads) {
      const int j = j0 + tid;
      int64_t count = 0;
      if (j < jobs) {
        const Job jb = job(j);
        if (jb.keys > 0) count = int64_t(ceil_div(jb.tokens, 2 * TT)) * Hkv * segments(jb.keys, longest).x;
      }
      int64_t total;
      const int64_t at = pbase + block_scan(count, warp_sums, total);
      if (j < jobs) w.first_piece[j] = int(at);
      pbase += total;
    }
    __syncthreads();
  }
  const int n_pieces = int(pbase);
  for (int i = tid; i < n_pieces; i += kPlanThreads) {
    int lo = 0, hi = jobs - 1;                     // the last job whose pieces start at or before i
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (w.first_piece[mid] <= i) lo = mid; else hi = mid - 1;
    }
    const Job jb = job(lo);
    const int2 sg = segments(jb.keys, longest);
    const int pairs = ceil_div(jb.tokens, 2 * TT);
    const int local = i - w.first_piece[lo];
    const int pair = local % pairs, hk = local / pairs % Hkv, seg = local / (pairs * Hkv);
    // tokens evenly over the pairs
    const int each = jb.tokens / pairs, more = jb.tokens - each * pairs;
    const int off = pair * each + min(pair, more);
    const bool alt = jb.tokens <= TT;
    Piece pc = {};
    pc.s0 = jb.s0;
    pc.skip = jb.skip;
    pc.tok0 = jb.tok0 + off;
    pc.ntok = each + (pair < more ? 1 : 0);
    pc.hk = hk;
    pc.keys = jb.keys;
    pc.lim0 = jb.lim0 + off;
    // tiles of the segment that some row of the pair sees
    const int seen = min(jb.keys, pc.lim0 + pc.ntok - 1);
    pc.j0 = seg * sg.y;
    pc.nt = max(0, min(sg.y, ceil_div(seen, BN) - pc.j0));
    const int recs = sg.x * (alt ? 2 : 1);
    pc.rec_step = lo < NG ? stride : recs;
    pc.rec0 = (lo < NG ? unsigned(pc.tok0) * unsigned(H) * unsigned(stride)
                       : w.seq_rec[lo - NG] + unsigned(off * H * recs)) + (alt ? 2 * seg : seg);
    // one record in all: only a chunk without a prefix, in one segment of two row tiles
    const bool direct = lo >= NG && recs == 1 && jb.skip == 0;
    pc.flags = (alt ? kPieceAlt : 0) | (direct ? kPieceDirect : 0);
    w.pieces[i] = pc;
  }
  if (tid == 0) set_header(n_pieces, stride, int(base & 0xffffffff), working);
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

// The paged blocks of a piece's KV tiles, for one loader warp: the block table is
// read 32 entries at a time, one window ahead of the tiles, so that no load waits
// for it, and each tile's boxes are prefetched into L2 kLookAhead tiles before
// their load.
struct BlockWindow {
  const int32_t* bt;           // the piece's first block
  int blocks;                  // blocks of the piece that hold keys
  int at;                      // first block of the window in `cur`
  int cur, next;               // lane i: box index of block at + i, at + 32 + i

  __device__ __forceinline__ int box(const AttnArgs& a, int hk, int i) const {
    if (i >= blocks) return a.num_blocks * a.num_kv_heads;     // out of range: TMA fills zeros
    const int blk = bt[i];
    if (blk >= 0 && blk < a.num_blocks) return blk * a.num_kv_heads + hk;
    raise_error(a.err, kErrBounds);
    return a.num_blocks * a.num_kv_heads;
  }
  __device__ __forceinline__ void start(const AttnArgs& a, const Piece& it, int lane) {
    const int bpt = BN / a.block_size;
    bt = a.block_tables + size_t(it.s0) * a.max_blocks_per_seq + it.skip + it.j0 * bpt;
    blocks = min(ceil_div(it.keys, a.block_size) - it.j0 * bpt, it.nt * bpt);
    at = 0;
    cur = box(a, it.hk, lane);
    next = box(a, it.hk, 32 + lane);
  }
  // the window holds block i from now on (i grows by tiles)
  __device__ __forceinline__ void move_to(const AttnArgs& a, int hk, int i, int lane) {
    if (i - at >= 32) {
      at += 32;
      cur = next;
      next = box(a, hk, at + 32 + lane);
    }
  }
  // tile j's boxes into L2: lane i those of its block i
  __device__ __forceinline__ void prefetch(const CUtensorMap* tm, const AttnArgs& a, int j, int lane) const {
    const int bpt = BN / a.block_size, i = j * bpt + lane - at;    // within the two windows
    const int z0 = __shfl_sync(0xffffffffu, cur, i & 31), z1 = __shfl_sync(0xffffffffu, next, i & 31);
    const int z = i < 32 ? z0 : z1;
    if (lane < bpt && z < a.num_blocks * a.num_kv_heads) {
      tma_prefetch_l2_3d(tm, 0, 0, z);
      tma_prefetch_l2_3d(tm, 64, 0, z);
    }
  }
  // warp-wide; lane 0 loads tile j
  __device__ __forceinline__ void load(uint32_t dst, const CUtensorMap* tm, uint32_t bar, const AttnArgs& a, int j,
                                       int lane) const {
    const int B = a.block_size, bpt = BN / B;
    if (lane == 0) mbar_arrive_expect_tx(bar, kTile);
    for (int bi = 0; bi < bpt; ++bi) {
      const int z = __shfl_sync(0xffffffffu, cur, j * bpt + bi - at);
      if (lane == 0) {
        tma_load_3d(dst + bi * B * 128, tm, bar, 0, 0, z);
        tma_load_3d(dst + kHalf + bi * B * 128, tm, bar, 64, 0, z);
      }
    }
    __syncwarp();
  }
};

// The pieces that this CTA claims through header[3], all its warps together
// (roles and hand-offs as in the prefill kernel).  Every wait is bounded; after
// a timeout the device error word is set, the roles wind down and the result is
// false.
__device__ __forceinline__ bool run_pieces(const CUtensorMap* tm_q, const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                                           const AttnArgs& a, const PrefixWork& w, uint8_t* gsm, uint32_t base, int n_pieces,
                                           int with_pieces) {
  auto bar = [&](int i) -> uint32_t { return base + kOffBar + 8u * uint32_t(i); };
  Piece* items = reinterpret_cast<Piece*>(gsm + kOffItems);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int B = a.block_size;
  const int H = a.num_heads;
  const int G = H / a.num_kv_heads;                // query heads per key/value head
  const int TT = w.tile_tokens;
  const int bpt = BN / B;                          // blocks per KV tile
  bool role_ok = true;

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
    mbar_init(bar(BAR_VTAIL), 1);
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

  // A reader's view of piece n; `arrive`: this thread is its role's one arrival.
  auto read_item = [&](int n, bool arrive, Piece& it) -> bool {
    const int slot = n % kItemSlots;
    if (!mbar_wait(bar(BAR_IF + slot), (n / kItemSlots) & 1)) return false;
    it = items[slot];
    if (arrive) mbar_arrive(bar(BAR_IE + slot));
    return true;
  };

  if (warp == kWarpK) {
    // ------------------------------------------------------------ K loader (claims the pieces)
    if (lane == 0) {
      tma_prefetch_desc(tm_q);
      tma_prefetch_desc(tm_k);
    }
    uint32_t kc = 0;                               // K tiles requested
    uint32_t qc = 0;                               // Q loads requested
    bool ok = true;
    unsigned site = 0;
    // the first piece is given, the later ones are claimed one ahead
    int u = int(blockIdx.x);
    for (int n = 0; ok; ++n) {
      const int slot = n % kItemSlots;
      if (n >= kItemSlots && !__all_sync(0xffffffffu, mbar_wait(bar(BAR_IE + slot), ((n / kItemSlots) - 1) & 1))) {
        ok = false;
        site = kSitePfItemFree;
        break;
      }
      if (lane < int(sizeof(Piece) / 16)) {
        int4 part = make_int4(0, 0, 0, 0);
        if (u < n_pieces) part = __ldcg(reinterpret_cast<const int4*>(w.pieces + u) + lane);
        reinterpret_cast<int4*>(items + slot)[lane] = part;
      }
      __syncwarp();
      if (lane == 0) {
        if (u >= n_pieces) items[slot].flags = kPieceEnd;
        mbar_arrive(bar(BAR_IF + slot));           // release: the slot's contents are visible
      }
      if (u >= n_pieces) break;
      const int ahead = lane == 0 ? with_pieces + atomicAdd(w.header + 3, 1) : 0;
      const Piece it = items[slot];
      if (it.nt > 0) {
        const int nq = !(it.flags & kPieceAlt) && it.ntok > TT ? 2 : 1;
        BlockWindow win;
        win.start(a, it, lane);
        auto load_q = [&]() -> bool {
          if (qc > 0 && !__all_sync(0xffffffffu, mbar_wait(bar(BAR_QE), (qc - 1) & 1))) return false;
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
        const int q_at = min(kKStages - 1, it.nt);   // K tiles requested before the Q load
        for (int j = 1; j < min(kLookAhead, it.nt); ++j) win.prefetch(tm_k, a, j, lane);
        for (int j = 0; j < it.nt; ++j) {
          if (j == q_at && !load_q()) {
            ok = false;
            site = kSitePfQFree;
            break;
          }
          win.move_to(a, it.hk, j * bpt, lane);
          if (j + kLookAhead < it.nt) win.prefetch(tm_k, a, j + kLookAhead, lane);
          const int st = kc % kKStages;
          if (kc >= kKStages && !__all_sync(0xffffffffu, mbar_wait(bar(BAR_KE + st), ((kc / kKStages) - 1) & 1))) {
            ok = false;
            site = kSitePfKFree;
            break;
          }
          win.load(base + kOffK + st * kTile, tm_k, bar(BAR_KF + st), a, j, lane);
          ++kc;
        }
        if (ok && q_at == it.nt && !load_q()) {
          ok = false;
          site = kSitePfQFree;
        }
      }
      u = __shfl_sync(0xffffffffu, ahead, 0);
    }
    if (!ok && lane == 0) raise_error(a.err, kErrTimeout | site);
    role_ok = ok;
    if (lane == 0) {
      // (error path) let copies still in flight land before the memory is used again
      for (uint32_t gk = kc > uint32_t(kKStages) ? kc - kKStages : 0; gk < kc; ++gk)
        mbar_wait(bar(BAR_KF + gk % kKStages), (gk / kKStages) & 1);
      if (qc > 0) mbar_wait(bar(BAR_Q), (qc - 1) & 1);
    }
  } else if (warp == kWarpV) {
    // ------------------------------------------------------------ V loader
    if (lane == 0) tma_prefetch_desc(tm_v);
    uint32_t vc = 0, tails = 0;                    // V tiles requested, of which tails
    bool ok = true, tail_pending = false;
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
      if (it.flags & kPieceEnd) break;
      if (it.nt == 0) continue;
      BlockWindow win;
      win.start(a, it, lane);
      for (int j = 1; j < min(kLookAhead, it.nt); ++j) win.prefetch(tm_v, a, j, lane);
      for (int j = 0; j < it.nt; ++j) {
        win.move_to(a, it.hk, j * bpt, lane);
        if (j + kLookAhead < it.nt) win.prefetch(tm_v, a, j + kLookAhead, lane);
        const int st = vc % kVStages;
        if (vc >= kVStages && !__all_sync(0xffffffffu, mbar_wait(bar(BAR_VE + st), ((vc / kVStages) - 1) & 1))) {
          ok = false;
          site = kSitePfVFree;
          break;
        }
        // rows of the last block behind the last key may hold anything: P is 0 there, but 0 * NaN is not
        const int kb = (it.j0 + j) * BN, r0 = it.keys - kb, r1 = min(BN, ceil_div(it.keys, B) * B - kb);
        const bool tail = r0 < r1;
        win.load(base + kOffV + st * kTile, tm_v, tail ? bar(BAR_VTAIL) : bar(BAR_VF + st), a, j, lane);
        ++vc;
        if (tail) {
          if (!__all_sync(0xffffffffu, mbar_wait(bar(BAR_VTAIL), tails & 1))) {
            ok = false;
            tail_pending = true;
            site = kSitePfVTail;
            break;
          }
          ++tails;
          uint8_t* vt = gsm + kOffV + st * kTile;
          for (int c = lane; c < (r1 - r0) * 16; c += 32) {
            const int r = r0 + c / 16, wd = c % 16;
            *reinterpret_cast<uint4*>(vt + (wd / 8) * kHalf + r * 128 + (wd % 8) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(BAR_VF + st));
        }
      }
    }
    if (!ok && lane == 0) raise_error(a.err, kErrTimeout | site);
    role_ok = ok;
    if (lane == 0) {                               // (error path) as above
      if (tail_pending) mbar_wait(bar(BAR_VTAIL), tails & 1);
      const uint32_t landed = tail_pending ? vc - 1 : vc;
      for (uint32_t gv = landed > uint32_t(kVStages) ? landed - kVStages : 0; gv < landed; ++gv)
        mbar_wait(bar(BAR_VF + gv % kVStages), (gv / kVStages) & 1);
    }
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
      uint32_t kc = 0, vc = 0, qc = 0, cnt[2] = {0, 0};   // K, V tiles and Q loads consumed; S/P phases of the slots
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
        if (it.flags & kPieceEnd) break;
        if (it.nt == 0) continue;
        if (!wait(BAR_Q, qc++, kSitePfQ)) break;
        if (it.flags & kPieceAlt) {
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
      role_ok = ok;
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
      if (it.flags & kPieceEnd) break;
      // this slot's rows and KV tiles j = first, first + step, ...
      const bool alt = it.flags & kPieceAlt;
      const int toff = alt ? 0 : t * TT;           // the slot's first token, within the piece
      const int ntok = alt ? it.ntok : min(TT, it.ntok - toff);
      const int step = alt ? 2 : 1, first = alt ? t : 0;
      if (ntok <= 0) continue;                     // no rows in the second tile
      const int rows = ntok * G;
      const int steps = (it.nt - first + step - 1) / step;
      // keys that this thread's row sees, and that every row of its warp does
      const int lim = min(it.keys, it.lim0 + toff + i / G), lim_warp = min(it.keys, it.lim0 + toff + wq * 32 / G);
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
        if (kb + BN > lim_warp) {                  // keys behind the last one, or the causal mask
#pragma unroll
          for (int c = 0; c < BN; ++c)
            if (kb + c >= lim) sr[c] = __float_as_uint(-INFINITY);
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
      // The rows' records of this segment (in the alternating mode, of its even
      // or odd tiles).  A lane holds one row; stored as it is, each store of the
      // warp would touch 32 lines.  So every 8 lanes first transpose their 8
      // rows of 32 dims in units of 16 bytes: a store is then 4 whole lines.
      const bool direct = it.flags & kPieceDirect;
      const int row_tok = toff + i / G, head = it.hk * G + i % G;
      const unsigned rec = direct ? unsigned(it.tok0 + row_tok) * unsigned(H) + unsigned(head)
                                  : it.rec0 + unsigned((row_tok * H + head) * it.rec_step + (alt ? t : 0));
      const float inv = direct ? 1.0f / l : 1.0f;
      if (work) {
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
          for (int d = 4; d > 0; d >>= 1) {
            const bool hi = lane & d;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              if (u & d) continue;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, hi ? o[4 * u + e] : o[4 * (u | d) + e], d);
                if (hi) o[4 * u + e] = got;
                else o[4 * (u | d) + e] = got;
              }
            }
          }
#pragma unroll
          for (int r = 0; r < 8; ++r) {            // unit r now belongs to row r of these 8 lanes
            const int from = (lane & ~7) + r;
            const unsigned at = __shfl_sync(0xffffffffu, rec, from);
            const float f = __shfl_sync(0xffffffffu, inv, from);
            if (wq * 32 + from >= rows) continue;
            if (direct) {
              const float* x = reinterpret_cast<const float*>(&o[4 * r]);
              *(reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + size_t(at) * HD + 32 * c) + (lane & 7)) =
                  make_uint2(pack_bf16x2(x[0] * f, x[1] * f), pack_bf16x2(x[2] * f, x[3] * f));
            } else {
              __stcg(reinterpret_cast<uint4*>(w.recs + size_t(at) * kPrefixRec + 32 * c) + (lane & 7),
                     make_uint4(o[4 * r], o[4 * r + 1], o[4 * r + 2], o[4 * r + 3]));
            }
          }
        }
        if (i < rows && !direct) __stcg(reinterpret_cast<float2*>(w.recs + size_t(rec) * kPrefixRec + HD), make_float2(m, l));
      }
      tc_fence_before();                           // O read before the next piece's first P V overwrites it
    }
    if (!ok && lane == 0) raise_error(a.err, kErrTimeout | site);
    role_ok = ok;
  }
  tc_fence_before();
  const bool failed = __syncthreads_or(role_ok ? 0 : 1);
  if (warp == kWarpMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  return !failed;
}

// Persistent, one CTA per SM.  The first header[6] CTAs take pieces, then stream
// own keys like the rest, each of their first eight warps on its own.
__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_k16,
                     const __grid_constant__ CUtensorMap tm_v16, const AttnArgs a, const PrefixWork w) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;    // 128B-swizzled tiles need 1 KB alignment
  uint8_t* gsm = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  asm volatile("griddepcontrol.wait;" ::: "memory");   // the plan kernels have finished
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int n_pieces = __ldcg(w.header), n_items = __ldcg(w.header + 4);
  const int working = __ldcg(w.header + 6);
  if (uint32_t(__ldcg(w.header + 2)) != w.tag || n_pieces < 0 || n_pieces > w.piece_cap || n_items < 0 ||
      n_items > w.item_cap) {                      // a plan of another call: no work
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(a.err, kErrInvalid);
    return;
  }
  const int with_pieces = min(n_pieces, min(int(gridDim.x), working));   // CTAs that take pieces first
  const bool pieces_first = int(blockIdx.x) < with_pieces;
  if (pieces_first && !run_pieces(&tm_q, &tm_k, &tm_v, a, w, gsm, base, n_pieces, with_pieces)) return;

  // own keys: each streaming warp's ring (over the tiles, which the pieces are
  // done with), barriers and item slots
  if (warp >= kStreamWarps) return;
  const uint32_t bars = base + kOffOwnBars + warp * stream::kStages * 8;
  if (lane == 0) {
    for (int st = 0; st < stream::kStages; ++st) mbar_init(bars + 8 * st, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tm_k16);
    tma_prefetch_desc(&tm_v16);
  }
  __syncwarp();
  // The first units are given to the CTAs that start with them, neighbouring
  // units to different SMs; the rest is claimed.
  const int others = int(gridDim.x) - with_pieces, warps = others * kStreamWarps;
  stream::run_warp(&tm_k16, &tm_v16, a, w, n_items, base + warp * stream::kStages * stream::kStageBytes, bars,
                   reinterpret_cast<SuffixItem*>(gsm + kOffOwnSlots) + 2 * warp,
                   pieces_first ? -1 : warp * others + int(blockIdx.x) - with_pieces, warps, 2 * warps);
}

// One warp per kJoinRows query heads of a token: their records are loaded four
// at a time for all of them, one pass with a running maximum.
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 2;
constexpr int kJoinRecs = 4;
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const AttnArgs a, const PrefixWork w) {
  const int lane = threadIdx.x & 31;
  const unsigned unit = blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
  const unsigned per_token = unsigned(a.num_heads + kJoinRows - 1) / kJoinRows;
  const int tok = int(unit / per_token);
  const int h0 = int(unit - unsigned(tok) * per_token) * kJoinRows;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tok >= a.num_tokens) return;
  const uint32_t tag = uint32_t(__ldcg(w.header + 2));
  const int stride = __ldcg(w.header + 1);
  const int4 ti = __ldcg(w.token_info + tok);
  const int np = ti.x, n = np + ti.z;
  if (tag != w.tag || n < 2) return;                     // left out, or already written
  float4 acc[kJoinRows];
  float mx[kJoinRows], den[kJoinRows];
  const float *pre[kJoinRows], *own[kJoinRows];
#pragma unroll
  for (int r = 0; r < kJoinRows; ++r) {
    const int h = min(h0 + r, a.num_heads - 1);
    pre[r] = w.recs + (size_t(tok) * a.num_heads + h) * stride * kPrefixRec;
    own[r] = w.recs + (size_t(unsigned(ti.y)) + size_t(h) * ti.z) * kPrefixRec;
    acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    mx[r] = -INFINITY;
    den[r] = 0.f;
  }
  for (int k0 = 0; k0 < n; k0 += kJoinRecs) {
    float4 x[kJoinRows][kJoinRecs];
    float2 ml[kJoinRows][kJoinRecs];
#pragma unroll
    for (int k = 0; k < kJoinRecs; ++k)
#pragma unroll
      for (int r = 0; r < kJoinRows; ++r) {
        const int kk = k0 + k;
        x[r][k] = make_float4(0.f, 0.f, 0.f, 0.f);
        ml[r][k] = make_float2(-INFINITY, 0.f);
        if (kk < n) {
          const float* p = kk < np ? pre[r] + size_t(kk) * kPrefixRec : own[r] + size_t(kk - np) * kPrefixRec;
          x[r][k] = __ldcg(reinterpret_cast<const float4*>(p) + lane);
          ml[r][k] = __ldcg(reinterpret_cast<const float2*>(p + HD));
        }
      }
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r) {
      float top = mx[r];
#pragma unroll
      for (int k = 0; k < kJoinRecs; ++k) top = fmaxf(top, ml[r][k].x);
      const float ref = top == -INFINITY ? 0.f : top;    // no key seen so far
      const float old = ex2(mx[r] - ref);
      acc[r].x *= old, acc[r].y *= old, acc[r].z *= old, acc[r].w *= old;
      den[r] *= old;
      mx[r] = top;
#pragma unroll
      for (int k = 0; k < kJoinRecs; ++k) {
        const float f = ex2(ml[r][k].x - ref);
        den[r] = fmaf(f, ml[r][k].y, den[r]);
        acc[r].x = fmaf(f, x[r][k].x, acc[r].x);
        acc[r].y = fmaf(f, x[r][k].y, acc[r].y);
        acc[r].z = fmaf(f, x[r][k].z, acc[r].z);
        acc[r].w = fmaf(f, x[r][k].w, acc[r].w);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kJoinRows; ++r) {
    if (h0 + r >= a.num_heads) break;
    const float inv = 1.0f / den[r];
    uint2 v;
    v.x = pack_bf16x2(acc[r].x * inv, acc[r].y * inv);
    v.y = pack_bf16x2(acc[r].z * inv, acc[r].w * inv);
    *(reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + (size_t(tok) * a.num_heads + h0 + r) * HD) + lane) = v;
  }
}

std::mutex g_attr_mutex;
bool g_attr_set[64] = {};

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Capacities of a step's lists.
struct PrefixSizes {
  size_t S, T, NG, pieces, items, prefix_recs, piece_recs, own_recs;
};
int tile_tokens(int group_heads) { return BM / group_heads; }
PrefixSizes prefix_sizes(int32_t num_q_heads, int32_t num_kv_heads, int32_t num_seqs, int32_t num_tokens, int32_t num_groups) {
  PrefixSizes z;
  z.S = size_t(num_seqs), z.T = size_t(num_tokens), z.NG = size_t(num_groups);
  const size_t G = size_t(num_q_heads / num_kv_heads), rows = z.T * size_t(num_q_heads);
  const bool chunks = z.T > z.S && (z.T - z.S + 1) * G > size_t(kMaxStreamRows);
  // uncut: groups that share have two sequences or more; chunks are all of their tokens
  const size_t pairs = z.T / (2 * size_t(tile_tokens(int(G))));
  z.pieces = size_t(num_kv_heads) * (pairs + std::min(z.NG, z.S / 2) + 1 + (chunks ? pairs + z.S : 0)) + kExtraPieces;
  z.prefix_recs = std::min(rows * 2 * kMaxSegs, rows * 2 + size_t(kExtraRecs));
  z.piece_recs = chunks ? rows * 2 + size_t(kExtraRecs) : 0;
  // ceil(x / L) <= x / L + 1 for every streamed sequence, and all x / L together are at most `units`
  const size_t units = size_t(kMaxSms) * kStreamWarps * kUnitsPerWarp;
  z.items = z.T * G / kStreamRows + z.S + units + 1;
  z.own_recs = z.piece_recs + rows + kStreamRows * units;
  return z;
}

}  // namespace

size_t shared_prefix_workspace_bytes(int32_t num_q_heads, int32_t num_kv_heads, int32_t num_seqs, int32_t num_tokens,
                                     int32_t num_groups) {
  const PrefixSizes z = prefix_sizes(num_q_heads, num_kv_heads, num_seqs, num_tokens, num_groups);
  return 256 + align256(z.NG * 16) + align256((z.NG + z.S) * 4) + align256(z.S * 4) + align256(z.pieces * sizeof(Piece)) +
         align256(z.items * sizeof(SuffixItem)) + align256(z.T * 16) +
         align256((z.prefix_recs + z.own_recs) * kPrefixRec * sizeof(float));
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
  auto encode_kv = [&](CUtensorMap* tm, const void* pool, int rows) -> CUresult {
    const cuuint32_t box[3] = {64, cuuint32_t(rows), 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(pool), dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  // the pieces load whole blocks, the own keys 16 rows at a time
  CUtensorMap tk16, tv16;
  CUresult r = encode_kv(&tk, a.k_pool, B);
  if (r == CUDA_SUCCESS) r = encode_kv(&tv, a.v_pool, B);
  tk16 = tk;
  tv16 = tv;
  if (B != stream::kTileKeys) {
    if (r == CUDA_SUCCESS) r = encode_kv(&tk16, a.k_pool, stream::kTileKeys);
    if (r == CUDA_SUCCESS) r = encode_kv(&tv16, a.v_pool, stream::kTileKeys);
  }
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
  cudaError_t e = launch_kernel(prefix_tc_kernel, dim3(unsigned(w.num_sms)), dim3(kThreads), kSmemBytes, stream, true, tq, tk,
                                tv, tk16, tv16, a, w);
  return e == cudaSuccess ? CB_OK : cuda_fail(e, "shared prefixes: launch");
}

static cb_status launch_join(const AttnArgs& a, const PrefixWork& w, cudaStream_t stream) {
  const int64_t warps = int64_t(a.num_tokens) * ((a.num_heads + kJoinRows - 1) / kJoinRows);
  const unsigned grid = unsigned((warps * 32 + kJoinThreads - 1) / kJoinThreads);
  cudaError_t e = launch_kernel(join_kernel, dim3(grid), dim3(kJoinThreads), 0, stream, true, a, w);
  return e == cudaSuccess ? CB_OK : cuda_fail(e, "shared prefixes: join launch");
}

// A step with shared prefixes on one stream: the plan, the pieces and streams, and
// the join, each a programmatic dependent of the one before.
cb_status run_shared_prefix(const AttnArgs& a, const int32_t* cu_groups, const int32_t* prefix_lens, int32_t num_groups,
                            void* workspace, cudaStream_t stream) {
  NvtxRange nvtx("cb.shared_prefix");
  if (int64_t(a.num_blocks) * a.num_kv_heads >= (int64_t(1) << 31))
    return fail(CB_ERR_UNSUPPORTED, "shared prefixes: num_blocks * num_kv_heads must fit in int32");
  const PrefixSizes z = prefix_sizes(a.num_heads, a.num_kv_heads, a.num_seqs, a.num_tokens, num_groups);
  if (z.pieces > 0x7FFFFFFF || z.items > size_t(0x7FFFFFFF / a.num_kv_heads) || z.prefix_recs > 0x7FFFFFFF ||
      z.own_recs > 0x7FFFFFFF)
    return fail(CB_ERR_UNSUPPORTED, "shared prefixes: too many tokens");
  PrefixWork w;
  w.cu_groups = cu_groups;
  w.prefix_lens = prefix_lens;
  w.context_lens = a.context_lens;
  w.num_groups = num_groups;
  w.num_sms = sm_count();
  w.tile_tokens = tile_tokens(a.num_heads / a.num_kv_heads);
  w.stream_units = std::min(w.num_sms, kMaxSms) * kStreamWarps * kUnitsPerWarp;
  w.piece_cap = int32_t(z.pieces);
  w.item_cap = int32_t(z.items);
  w.prefix_rec_cap = int64_t(z.prefix_recs);
  w.piece_rec_cap = int64_t(z.piece_recs);
  w.own_rec_cap = int64_t(z.own_recs);
  char* p = static_cast<char*>(workspace);
  auto take = [&p](size_t bytes) {
    char* at = p;
    p += align256(bytes);
    return at;
  };
  w.header = reinterpret_cast<int32_t*>(take(256));
  w.groups = reinterpret_cast<int4*>(take(z.NG * 16));
  w.first_piece = reinterpret_cast<int32_t*>(take((z.NG + z.S) * 4));
  w.seq_rec = reinterpret_cast<unsigned*>(take(z.S * 4));
  w.pieces = reinterpret_cast<Piece*>(take(z.pieces * sizeof(Piece)));
  w.items = reinterpret_cast<SuffixItem*>(take(z.items * sizeof(SuffixItem)));
  w.token_info = reinterpret_cast<int4*>(take(z.T * 16));
  w.recs = reinterpret_cast<float*>(take((z.prefix_recs + z.own_recs) * kPrefixRec * sizeof(float)));
  static std::atomic<uint32_t> next_tag{1};
  w.tag = next_tag.fetch_add(1);

  prefix_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a, w);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "shared prefixes: plan launch");
  cb_status st = launch_prefix_tc(a, w, stream);
  if (st != CB_OK) return st;
  return launch_join(a, w, stream);
}

}  // namespace cb
