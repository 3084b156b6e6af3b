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
//     estimated time.  Every segment costs the join one more record per row;
//   * a step whose keys are too few for sharing to pay is streams alone, and every
//     CTA plans it for itself.
// Measured (graph replays; behind the bar, with every sequence reading its whole
// context): 64 sequences behind 2048 keys of 32 heads 75 us | 286; 256 behind 8192
// keys of 8 heads 129 to 133 | 1590; 24 prompts of up to 7 samples 69 | 101; 12 chunks
// of up to 200 tokens behind 4096 keys 164 | 220; 4 behind 512 keys 9 | 27.
#include <algorithm>
#include <atomic>
#include <cmath>
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
constexpr uint32_t kOffOwnBars = kOffItems + kItemSlots * uint32_t(sizeof(Piece));   // streams: barriers, items;
constexpr uint32_t kOffOwnSlots = kOffOwnBars + stream::kBarBytes;                  // their rings lie over the tiles
constexpr uint32_t kSmemBytes = kOffOwnSlots + stream::kSlotBytes + 1024;   // + slack to align the base
static_assert(kOffItems % 16 == 0 && kOffOwnSlots % 16 == 0, "pieces and items are copied 16 bytes at a time");
static_assert(stream::kRingBytes <= kOffBar, "the streams' rings");
static_assert(kSmemBytes <= 232448, "shared memory budget");

// ------------------------------------------------------------------ plan

constexpr int kPlanThreads = 512;
constexpr int kMaxSegs = 64;             // KV segments of a prefix, or of a chunk's own keys
constexpr int kSegChoices = 32;          // numbers of segments that are scored: 1 .. 24, then every fifth to 64
constexpr int kGroupCache = 512;         // groups kept in shared memory
constexpr int kSeqCache = 768;           // sequences kept in shared memory
constexpr int kJobCache = 768;           // jobs whose first piece is kept in shared memory
constexpr int kExtraPieces = 1024;       // pieces beyond one per (row tile pair, key/value head)
constexpr int64_t kExtraRecs = 131072;   // records beyond two per row (69 MB)
constexpr int kMinChunkTiles = 4;        // shortest chunk of streamed keys, in 16-key tiles
constexpr int kStreamRows = 16;          // query rows per row tile of a stream
constexpr int kUnitsPerWarp = 3;         // streamed units that each warp should get
constexpr int kMaxSms = 160;             // SMs that the lists are sized for
// Query rows per key/value head up to which a sequence's own keys are streamed,
// once per 16 rows; beyond, they are pieces.
constexpr int kMaxStreamRows = 64;
// Cost model of the segments and of the SM split, in microseconds and bytes.
constexpr float kTileUsTwo = 1.8f;       // a KV tile against two row tiles, one SM
constexpr float kTileUsOne = 1.4f;       // a KV tile against one row tile, at an SM's share of HBM (0.85 alone)
constexpr float kPieceUs = 5.0f;         // a piece beyond its tiles: Q, the pipeline's fill, the records
constexpr float kBytesPerUs = 6.7e6f;    // HBM
constexpr float kStreamBytesPerUsPerSm = 4.2e4f;   // streams of one SM
constexpr float kJoinBytesPerUs = 4.0e6f;
constexpr float kShareUs = 6.0f;          // what a step's pieces and join take at least
constexpr float kSmallUs = 28.0f;         // the same with the plan, for steps that can do without
constexpr int kWaveSteps = 16;           // SM splits that are scored: those that the pieces fill in 1 .. 16 waves
static_assert(kSegChoices * kWaveSteps == kPlanThreads, "a thread scores one choice");

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// The plan is one CTA that runs every line once: what it costs is latency, of the
// instruction fetches first of all (some 10 us for 200 sequences).  So its
// helpers are functions of their own, and its arrays are reached through one
// generic pointer each, in shared memory where they fit and in the workspace else.

// ceil(a / b) through one approximate quotient, corrected to be exact; a, b >= 1.
__device__ __noinline__ int ceil_div_fast(int a, int b) {
  if (a >= (1 << 22)) return (a - 1) / b + 1;
  int q = int(__fdividef(float(a), float(b)));
  const int r = a - q * b;                         // the quotient is off by one at most
  if (r < 0) --q;
  else if (r >= b) ++q;
  return q * b < a ? q + 1 : q;
}

// The segments of a range of keys where none is longer than `longest` KV tiles:
// their number and length.
__device__ __noinline__ int2 segments(int keys, int longest) {
  const int tiles = (keys + BN - 1) / BN;
  const int len = ceil_div_fast(tiles, ceil_div_fast(tiles, longest));
  return make_int2(ceil_div_fast(tiles, len), len);
}

// The last i < n with p[i * stride] <= v; 0 if there is none.
__device__ __noinline__ int last_at_or_before(const int* p, int stride, int n, int v) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p[mid * stride] <= v) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The plan's last lists, the streamed items and the pieces, are made side by side,
// by half of the threads each.
constexpr int kHalfThreads = kPlanThreads / 2;
__device__ __forceinline__ void half_sync(int half) { asm volatile("bar.sync %0, %1;" ::"r"(1 + half), "n"(kHalfThreads) : "memory"); }

// Exclusive scan over a half's threads; `total` receives the sum.  Contains half_sync.
__device__ __noinline__ int64_t half_scan(int64_t v, int64_t* warp_sums, int half, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = half * (kHalfThreads / 32);
  int64_t x = v;
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  half_sync(half);
  int64_t before = 0, all = 0;
  for (int w = first; w < first + kHalfThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    all += warp_sums[w];
  }
  *total = all;
  half_sync(half);
  return before + x - v;
}

// Sums over the CTA without shared atomics, which are slow in 64 bits: every
// warp's part (0 <= v < 2^60), 20 bits at a time through the warp's reduction, ...
__device__ __noinline__ void put_warp_sum(int64_t* parts, int64_t v) {
  const unsigned lo = __reduce_add_sync(0xffffffffu, unsigned(v & 0xfffff));
  const unsigned mid = __reduce_add_sync(0xffffffffu, unsigned((v >> 20) & 0xfffff));
  const unsigned hi = __reduce_add_sync(0xffffffffu, unsigned((v >> 40) & 0xfffff));
  if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = int64_t(lo) + (int64_t(mid) << 20) + (int64_t(hi) << 40);
}
// ... and, after a __syncthreads, their sum.
__device__ __noinline__ int64_t sum_parts(const int64_t* parts) {
  int64_t x = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) x += parts[w];
  return x;
}

__device__ __forceinline__ int sms_of(int pieces, int waves, int num_sms) { return min(num_sms, (pieces + waves - 1) / waves); }
__device__ __forceinline__ int seg_choice(int i) { return i < 24 ? i + 1 : 24 + (i - 23) * 5; }

// Rows that a set of pieces has in common: a group's over its prefix, or a
// chunk's over its own keys.  keys = 0: none.
struct Job {
  int keys, tok0, tokens, s0, skip, lim0;
};

// What the plan knows of the groups and sequences.
struct PlanView {
  const int4* groups;          // (first sequence, first token, tokens, shared keys)
  const int4* seqs;            // (own keys, 0: left out; first token; tokens; group)
  int num_groups, block_shift, group_heads;
  int stream_rows;             // query rows per key/value head up to which own keys are streamed
};
__device__ __forceinline__ bool is_chunk(const int4& q, const PlanView& v) {
  return q.x > 0 && q.z > 1 && int64_t(q.z) * v.group_heads > v.stream_rows;
}
// Job j: group j's prefix, then sequence (j - num_groups)'s own keys.
__device__ __noinline__ Job get_job(const PlanView v, int j) {
  if (j < v.num_groups) {
    const int4 gr = v.groups[j];
    return Job{gr.w, gr.y, gr.z, gr.x, 0, gr.w};
  }
  const int4 q = v.seqs[j - v.num_groups];
  if (!is_chunk(q, v)) return Job{0, 0, 0, 0, 0, 0};
  return Job{q.x, q.y, q.z, j - v.num_groups, v.groups[q.w].w >> v.block_shift, q.x - q.z + 1};
}

// One CTA.  Checks the groups, chooses the segments of the pieces and the
// chunks of the streams, lists both and gives every row its records.
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const AttnArgs a, const PrefixWork w) {
  __shared__ int64_t warp_sums[kPlanThreads / 32];
  __shared__ int64_t sums[4][kPlanThreads / 32];
  __shared__ unsigned long long best[kPlanThreads / 32];
  __shared__ int4 gcache[kGroupCache], scache[kSeqCache];
  __shared__ int m_cu[kSeqCache + 1], m_ctx[kSeqCache], p_first[kJobCache];
  __shared__ int s_alt, s_tiles;
  const int tid = threadIdx.x;
  const int S = a.num_seqs, T = a.num_tokens, NG = w.num_groups, TT = w.tile_tokens;
  const int H = a.num_heads, Hkv = a.num_kv_heads, G = H / Hkv, block_shift = __ffs(a.block_size) - 1;
  // no room for chunks' records: a step that has one all the same (others have no token) streams it
  const int stream_rows = w.piece_rec_cap > 0 ? kMaxStreamRows : 0x7fffffff;
  const bool chunks = int64_t(a.max_q_len) * G > stream_rows && a.max_q_len > 1;   // some sequence's own keys may be pieces
  const int jobs = NG + (chunks ? S : 0);
  int4* groups = NG <= kGroupCache ? gcache : w.groups;
  int4* seqs = S <= kSeqCache ? scache : w.seqs;
  int* first_piece = jobs <= kJobCache ? p_first : w.first_piece;
  const int* cu = S <= kSeqCache ? m_cu : a.cu_seqlens_q;
  const int* ctx = S <= kSeqCache ? m_ctx : w.context_lens;
  const PlanView view = {groups, seqs, NG, block_shift, G, stream_rows};
  if (tid == 0) {
    s_alt = 0;
    s_tiles = 1;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");   // it may start while the stream's last kernel ends
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // they wait for this grid on the device
  if (w.max_sharers >= 0 && __ldcg(w.header + 7) != 0) {             // the small step's kernel ran it: nothing to do
    if (tid == 0) {
      w.header[0] = w.header[1] = w.header[4] = w.header[6] = 0;
      w.header[2] = int32_t(w.tag);
    }
    return;
  }
  int g_s0 = 0, g_s1 = 0, g_p = 0;                 // group tid, requested along with the sequences
  if (tid < NG) g_s0 = w.cu_groups[tid], g_s1 = w.cu_groups[tid + 1], g_p = w.prefix_lens[tid];
  if (S <= kSeqCache) {
    for (int i = tid; i <= S; i += kPlanThreads) {
      m_cu[i] = a.cu_seqlens_q[i];
      if (i < S) m_ctx[i] = w.context_lens[i];
    }
  }
  for (int t = tid; t < T; t += kPlanThreads) w.token_info[t] = make_int4(0, 0, 0, 0);
  __syncthreads();

  // Each group's shared keys: whole blocks of its prefix, for at least two
  // sequences.  Where the first sequence, whose table names the blocks, does
  // not hold them, every sequence of the group reads its own.  The groups have
  // to cover the sequences in order.
  const float key_bytes = 4.0f * HD * float(Hkv);  // K and V of a key
  int bad = 0;
  int64_t saved = 0;                               // keys that are not read again
  for (int g = tid; g < NG; g += kPlanThreads) {
    if (g != tid) g_s0 = w.cu_groups[g], g_s1 = w.cu_groups[g + 1], g_p = w.prefix_lens[g];
    const int s0 = g_s0, s1 = g_s1, p = g_p;
    int t0 = 0, tokens = 0, shared = 0;
    if (s0 < 0 || s1 < s0 || s1 > S || (g == 0 && s0 != 0) || (g == NG - 1 && s1 != S)) {
      bad = 1;
    } else if (s1 - s0 >= 2 && p >= a.block_size) {
      t0 = cu[s0];
      const int t1 = cu[s1], q0 = cu[s0 + 1] - t0, ctx0 = ctx[s0];
      if (t0 >= 0 && t1 <= T && t1 > t0 && q0 >= 1 && ctx0 <= a.max_context_len && ctx0 - q0 >= p &&
          int64_t(ctx0) <= int64_t(a.max_blocks_per_seq) * a.block_size) {
        tokens = t1 - t0;
        shared = (p >> block_shift) << block_shift;
        const float keys = float(shared) * float(s1 - s0 - 1);
        const float cost = float(ceil_div_fast(tokens, 2 * TT) * Hkv) *
                           (float((shared + BN - 1) / BN) * (tokens <= TT ? kTileUsOne : kTileUsTwo) + kPieceUs);
        // many small groups' pieces take longer than the reads that they save
        // (150 pairs behind 96 keys of 8 heads: 97 us shared, 50 not); the rows of a
        // group that can hold a chunk, more query tokens than one a sequence, are pieces either way
        const int most = tokens - (s1 - s0 - 1);
        const bool chunk = most > 1 && int64_t(most) * G > stream_rows;
        if (!chunk && keys * key_bytes * float(w.num_sms) < cost * kBytesPerUs) shared = 0;
        else saved += int64_t(keys);
      }
    }
    groups[g] = make_int4(s0, t0, tokens, shared);
  }
  put_warp_sum(sums[3], saved);
  bad = __syncthreads_or(bad);
  // Sharing takes the pieces and the join, one after the other: where the bytes
  // that it saves take HBM less time than that, every sequence reads its own
  // table (4 samples behind 512 keys of 8 heads: 25.1 us shared, 17.4 not).
  if (float(sum_parts(sums[3])) * key_bytes < kShareUs * kBytesPerUs) {
    for (int g = tid; g < NG; g += kPlanThreads) groups[g].w = 0;
  }
  __syncthreads();

  // Each sequence: its group and own keys.
  int tiles_max = 1;
  int64_t n_first = 0, unit_tiles = 0, own_keys = 0;   // pieces if nothing is cut, per key/value head; streamed
                                                       // units' tiles, and keys
  for (int g = tid; g < NG && !bad; g += kPlanThreads) {
    const int4 gr = groups[g];
    if (gr.w == 0) continue;
    n_first += ceil_div_fast(gr.z, 2 * TT);
    tiles_max = max(tiles_max, (gr.w + BN - 1) / BN);
    if (gr.z <= TT) s_alt = 1;
  }
  for (int s = tid; s < S && !bad; s += kPlanThreads) {
    const int g = last_at_or_before(&groups[0].x, 4, NG, s);   // empty groups start there too, and come before
    const int p = w.prefix_lens[g], n = ctx[s], c0 = cu[s], q_len = cu[s + 1] - c0;
    const bool ok = p >= 0 && q_len >= 1 && c0 >= 0 && c0 + q_len <= T && q_len <= a.max_q_len && n >= q_len &&
                    p <= n - q_len && n <= a.max_context_len && int64_t(n) <= int64_t(a.max_blocks_per_seq) * a.block_size;
    const int4 q = make_int4(ok ? n - groups[g].w : 0, c0, q_len, g);
    seqs[s] = q;
    if (!ok) {
      raise_error(a.err, kErrInvalid);             // left out
    } else if (is_chunk(q, view)) {
      n_first += ceil_div_fast(q_len, 2 * TT);
      tiles_max = max(tiles_max, (q.x + BN - 1) / BN);
    } else {
      unit_tiles += int64_t((q_len * G + kStreamRows - 1) / kStreamRows) * Hkv * ((q.x + stream::kTileKeys - 1) / stream::kTileKeys);
      own_keys += q.x;
    }
  }
  tiles_max = __reduce_max_sync(0xffffffffu, tiles_max);
  if ((tid & 31) == 0) atomicMax(&s_tiles, tiles_max);
  put_warp_sum(sums[0], n_first);
  put_warp_sum(sums[1], unit_tiles);
  put_warp_sum(sums[2], own_keys);
  __syncthreads();
  const int64_t all_first = sum_parts(sums[0]), all_tiles = sum_parts(sums[1]);
  bad |= all_first * Hkv > w.piece_cap;            // only if token ranges overlap (malformed metadata)
  const int alt_recs = s_alt ? 2 : 1;
  tiles_max = s_tiles;

  // Segments: no longer than the longest range / n, and the SMs that take pieces
  // first; the rest streams own keys beside them, which leaves the tensor cores
  // idle as large groups' pieces do HBM.  A thread scores one (n, SMs).
  int longest = 1, working = w.num_sms, n_segs = 1;
  if (all_first > 0 && !bad) {
    constexpr int kLanes = kPlanThreads / kSegChoices;   // threads per n, each with a share of the jobs
    const int c = tid / kLanes, n = seg_choice(c), len = ceil_div_fast(tiles_max, n);
    float bytes = 0.f, work = 0.f, piece = 0.f;
    int64_t pieces = 0, own_recs = 0;
#pragma unroll 1
    for (int j = tid % kLanes; j < jobs; j += kLanes) {
      const Job jb = get_job(view, j);
      if (jb.keys == 0) continue;
      const int2 sg = segments(jb.keys, len);
      const int64_t units = int64_t(ceil_div_fast(jb.tokens, 2 * TT)) * Hkv * sg.x;
      const bool alt = jb.tokens <= TT;
      const float us = float(sg.y) * (alt ? kTileUsOne : kTileUsTwo) + kPieceUs;
      pieces += units;
      if (j >= NG) own_recs += int64_t(jb.tokens) * H * sg.x * (alt ? 2 : 1);
      work += float(units) * us;
      piece = fmaxf(piece, us);
      bytes += float(jb.keys);
    }
#pragma unroll 1
    for (int x = kLanes / 2; x > 0; x >>= 1) {
      pieces += __shfl_xor_sync(0xffffffffu, pieces, x);
      own_recs += __shfl_xor_sync(0xffffffffu, own_recs, x);
      work += __shfl_xor_sync(0xffffffffu, work, x);
      piece = fmaxf(piece, __shfl_xor_sync(0xffffffffu, piece, x));
      bytes += __shfl_xor_sync(0xffffffffu, bytes, x);
    }
    const int64_t recs = int64_t(T) * H * n * alt_recs;
    static_assert(kLanes == kWaveSteps, "the thread's n is the one that it scores");
    const float piece_bytes = bytes * key_bytes, own_bytes = float(sum_parts(sums[2])) * key_bytes;
    unsigned long long key = ~0ull;
    if (pieces > 0 && pieces <= w.piece_cap && recs <= w.prefix_rec_cap && own_recs <= w.piece_rec_cap) {
      // as many SMs as the pieces fill in 1 .. 16 waves; those of one size run in whole waves, unequal ones fill the gaps
      const int k = sms_of(int(pieces), tid % kWaveSteps + 1, w.num_sms);
      const float per_sm = __fdividef(1.0f, float(k));
      float us = fminf(ceilf(float(pieces) * per_sm) * piece, work * per_sm + piece);
      us = fmaxf(us, piece_bytes * (1.0f / kBytesPerUs));
      const float beside = fminf(kBytesPerUs * us - piece_bytes, float(w.num_sms - k) * kStreamBytesPerUsPerSm * us);
      us += __fdividef(fmaxf(0.f, own_bytes - beside), fminf(kBytesPerUs, float(w.num_sms) * kStreamBytesPerUsPerSm));
      us += float(recs) * (kPrefixRecBytes / kJoinBytesPerUs);
      key = ((unsigned long long)(__float_as_uint(us)) << 32) | unsigned(k << 16 | n);
    }
#pragma unroll 1
    for (int x = 16; x > 0; x >>= 1) {
      const unsigned long long other = __shfl_xor_sync(0xffffffffu, key, x);
      key = other < key ? other : key;
    }
    if ((tid & 31) == 0) best[tid >> 5] = key;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kPlanThreads / 32; ++x) key = best[x] < key ? best[x] : key;
    bad |= key == ~0ull;                           // n = 1 fits unless token ranges overlap
    n_segs = bad ? 1 : int(key & 0xffff);
    working = bad ? w.num_sms : int(unsigned(key) >> 16);
    longest = ceil_div_fast(tiles_max, n_segs);
  }
  const int stride = n_segs * alt_recs;
  const unsigned own_rec0 = unsigned(w.prefix_rec_cap);
  // chunk length: the streamed units come out even over the warps
  const int64_t per = (all_tiles + w.stream_units - 1) / w.stream_units;
  const int L = int(per < kMinChunkTiles ? kMinChunkTiles : (per > (1 << 26) ? (1 << 26) : per));

  // Streamed items, and every sequence's records: its rows have `pre` of the
  // prefix and `nch` own ones each.
  const int half = tid / kHalfThreads, htid = tid - half * kHalfThreads;
  int64_t base = 0;                                // items in the low, own records in the high word
  for (int s0 = 0; half == 0 && s0 < S && !bad; s0 += kHalfThreads) {
    const int s = s0 + htid;
    int4 q = make_int4(0, 0, 0, 0), gr = q;
    int pre = 0, rt = 0, nch = 0;
    // units are claimed in the order of the sequences: the last quarter's are half as long, so that the
    // warps end closer together
    const int Ls = s < S - S / 4 ? L : max(kMinChunkTiles, (L + 1) / 2);
    if (s < S) q = seqs[s];
    if (q.x > 0) {
      gr = groups[q.w];
      if (gr.w > 0) pre = segments(gr.w, longest).x * (gr.z <= TT ? 2 : 1);
      if (is_chunk(q, view)) {
        nch = segments(q.x, longest).x * (q.z <= TT ? 2 : 1);
      } else {
        nch = ceil_div_fast((q.x + stream::kTileKeys - 1) / stream::kTileKeys, Ls);
        rt = (q.z * G + kStreamRows - 1) / kStreamRows;
      }
    }
    const int64_t n_items = int64_t(rt) * nch, n_recs = pre + nch > 1 ? int64_t(q.z) * H * nch : 0;
    int64_t total;
    const int64_t at = base + half_scan(n_items | (n_recs << 32), warp_sums, half, &total);
    base += total;
    bad |= (base & 0xffffffff) > w.item_cap || (base >> 32) > w.own_rec_cap;   // only if token ranges overlap
    if (q.x > 0 && !bad) {
      const unsigned rec = own_rec0 + unsigned(at >> 32);
      if (a.max_q_len > 1) w.seq_recs[s] = make_int4(pre, int(rec), nch, 0);
      else w.token_info[q.y] = make_int4(pre, int(rec), nch, 0);
      SuffixItem it = {};
      it.s = s, it.tok0 = q.y, it.q_len = q.z, it.ctx = q.x, it.skip = gr.w >> block_shift;
      it.rec_step = nch;
      it.direct = n_recs == 0;
      SuffixItem* out = w.items + (at & 0xffffffff);
#pragma unroll 1
      for (int i = 0; i < int(n_items); ++i) {
        it.rec0 = rec + it.pad;                    // `pad` counts the chunks
        it.k0 = it.pad * Ls * stream::kTileKeys;
        it.k1 = it.k0 + min(q.x - it.k0, Ls * stream::kTileKeys);
        *out++ = it;
        if (++it.pad == nch) it.pad = 0, it.row0 += kStreamRows;
      }
    }
  }
  // the pieces: by segment, key/value head and row tile pair, so that the
  // pairs of one (segment, head) run side by side and share its K/V in L2
  int64_t pbase = 0;
  if (half == 1 && all_first > 0 && !bad) {
    for (int j0 = 0; j0 < jobs; j0 += kHalfThreads) {
      const int j = j0 + htid;
      int64_t count = 0;
      if (j < jobs) {
        const Job jb = get_job(view, j);
        if (jb.keys > 0) count = int64_t(ceil_div_fast(jb.tokens, 2 * TT)) * Hkv * segments(jb.keys, longest).x;
      }
      int64_t total;
      const int64_t at = pbase + half_scan(count, warp_sums, half, &total);
      if (j < jobs) first_piece[j] = int(at);
      pbase += total;
    }
    half_sync(half);
  }
  if (a.max_q_len > 1) __syncthreads();            // the sequences' records are known
  if (half == 0 && a.max_q_len > 1 && !bad) {      // every token's sequence by search
    for (int t = htid; t < T; t += kHalfThreads) {
      const int s = last_at_or_before(cu, 1, S, t);
      const int4 q = seqs[s];
      if (q.x > 0 && q.y <= t && t < q.y + q.z) {
        int4 info = w.seq_recs[s];
        info.y += (t - q.y) * H * info.z;
        w.token_info[t] = info;
      }
    }
  }
  const int n_pieces = int(pbase);
  for (int i = htid; i < n_pieces; i += kHalfThreads) {   // none in the other half
    const int j = last_at_or_before(first_piece, 1, jobs, i);   // jobs without pieces start there too, and come before
    const Job jb = get_job(view, j);
    const int2 sg = segments(jb.keys, longest);
    const int pairs = ceil_div_fast(jb.tokens, 2 * TT);
    const int local = i - first_piece[j];
    const int rest = local / pairs, pair = local - rest * pairs, seg = rest / Hkv, hk = rest - seg * Hkv;
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
    pc.nt = max(0, min(sg.y, (seen + BN - 1) / BN - pc.j0));
    const int recs = sg.x * (alt ? 2 : 1);
    pc.rec_step = j < NG ? stride : recs;
    pc.rec0 = (j < NG ? unsigned(pc.tok0) * unsigned(H) * unsigned(stride)
                      : unsigned(w.seq_recs[j - NG].y) + unsigned(off * H * recs)) + (alt ? 2 * seg : seg);
    // one record in all: only a chunk without a prefix, in one segment of two row tiles
    const bool direct = j >= NG && recs == 1 && jb.skip == 0;
    pc.flags = (alt ? kPieceAlt : 0) | (direct ? kPieceDirect : 0);
    w.pieces[i] = pc;
  }
  bad = __syncthreads_or(bad);
  if (bad)                                         // nothing runs and no row is written
    for (int t = tid; t < T; t += kPlanThreads) w.token_info[t] = make_int4(0, 0, 0, 0);
  if (tid == 0) {
    if (bad) raise_error(a.err, kErrInvalid);
    w.header[1] = stride;
    w.header[2] = int32_t(w.tag);
    w.header[3] = 0;
    w.header[4] = bad ? 0 : int(base & 0xffffffff);
    w.header[5] = 0;
    w.header[6] = working;
  }
  if (tid == kHalfThreads) w.header[0] = bad ? 0 : n_pieces;
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
// 32 bytes in one store (aligned)
__device__ __forceinline__ void store32(float* p, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
               "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

// The paged blocks of a piece's KV tiles, for one loader warp.  The block table is
// read 32 entries at a time, one window ahead of the tiles, so that no load waits
// for it.  A tile is up to 16 TMA boxes (8 blocks of 16 keys, two 64-dim halves),
// and issuing them is what bounds a piece with one row tile: from one lane in
// turn, with an L2 prefetch of each box before, a tile took 1.64 us at 16 keys a
// block; without the prefetches 1.26; with a lane for each box 0.85, against 0.78
// at 128 keys a block (152 such pieces at once: 1.70, 1.36, 1.35 us, the last
// 7.4 TB/s).
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
  // tile j (of the piece, in order) into dst: a lane per box
  __device__ __forceinline__ void load(uint32_t dst, const CUtensorMap* tm, uint32_t bar, const AttnArgs& a, int hk, int j,
                                       int lane) {
    const int B = a.block_size, bpt = BN / B;
    if (j * bpt - at >= 32) {
      at += 32;
      cur = next;
      next = box(a, hk, at + 32 + lane);
    }
    if (lane == 0) mbar_arrive_expect_tx(bar, kTile);
    const int bi = lane >> 1, half = lane & 1;
    const int z = __shfl_sync(0xffffffffu, cur, (j * bpt + bi - at) & 31);
    if (bi < bpt) tma_load_3d(dst + half * kHalf + bi * B * 128, tm, bar, 64 * half, 0, z);
    __syncwarp();
  }
};

// The pieces that this CTA claims through header[3], all its warps together
// (roles and hand-offs as in the prefill kernel).  Every wait is bounded; after
// a timeout the device error word is set, the roles wind down and the result is
// false.
__device__ __forceinline__ bool run_pieces(const CUtensorMap* tm_q, const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                                           const AttnArgs& a, const PrefixWork& w, uint8_t* gsm, uint32_t base, uint32_t tmem,
                                           int n_pieces, int with_pieces, int4 first_part) {
  auto bar = [&](int i) -> uint32_t { return base + kOffBar + 8u * uint32_t(i); };
  Piece* items = reinterpret_cast<Piece*>(gsm + kOffItems);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int B = a.block_size;
  const int H = a.num_heads;
  const int G = H / a.num_kv_heads;                // query heads per key/value head
  const int TT = w.tile_tokens;
  bool role_ok = true;

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
        int4 part = first_part;
        if (n > 0 && u < n_pieces) part = __ldcg(reinterpret_cast<const int4*>(w.pieces + u) + lane);
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
        for (int j = 0; j < it.nt; ++j) {
          if (j == q_at && !load_q()) {
            ok = false;
            site = kSitePfQFree;
            break;
          }
          const int st = kc % kKStages;
          if (kc >= kKStages && !__all_sync(0xffffffffu, mbar_wait(bar(BAR_KE + st), ((kc / kKStages) - 1) & 1))) {
            ok = false;
            site = kSitePfKFree;
            break;
          }
          win.load(base + kOffK + st * kTile, tm_k, bar(BAR_KF + st), a, it.hk, j, lane);
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
      for (int j = 0; j < it.nt; ++j) {
        const int st = vc % kVStages;
        if (vc >= kVStages && !__all_sync(0xffffffffu, mbar_wait(bar(BAR_VE + st), ((vc / kVStages) - 1) & 1))) {
          ok = false;
          site = kSitePfVFree;
          break;
        }
        // rows of the last block behind the last key may hold anything: P is 0 there, but 0 * NaN is not
        const int kb = (it.j0 + j) * BN, r0 = it.keys - kb, r1 = min(BN, ceil_div(it.keys, B) * B - kb);
        const bool tail = r0 < r1;
        win.load(base + kOffV + st * kTile, tm_v, tail ? bar(BAR_VTAIL) : bar(BAR_VF + st), a, it.hk, j, lane);
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
        // P over the scores, rounded to bf16 since the tensor core takes it no wider: half a step, 2^-8, of each
        // weight.  Outputs are off by 0.0023 of 64 bits where their own rounding is 0.0017; the sums stay in fp32.
#pragma unroll
        for (int c = 0; c < 64; ++c) {
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
      // warp would touch 32 lines.  So every 4 lanes first transpose their 4
      // rows of 32 dims in units of 32 bytes: a store is then 8 whole lines (2.4 to
      // 3.5 us a piece; in units of 16 bytes over 8 lanes, 3.5 to 4.8).
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
    role_ok = ok;
  }
  tc_fence_before();
  const bool failed = __syncthreads_or(role_ok ? 0 : 1);
  tc_fence_after();
  return !failed;
}

// Persistent, one CTA per SM.  The first header[6] CTAs take pieces, then stream
// own keys like the rest, each of their first eight warps on its own.
__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_k16,
                     const __grid_constant__ CUtensorMap tm_v16, const __grid_constant__ AttnArgs a,
                     const __grid_constant__ PrefixWork w) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;    // 128B-swizzled tiles need 1 KB alignment
  uint8_t* gsm = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // Set up while the plan still runs: barriers, and tensor memory for pieces
  auto bar = [&](int i) -> uint32_t { return base + kOffBar + 8u * uint32_t(i); };
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
  const uint32_t bars = base + kOffOwnBars + warp * stream::kStages * 8;   // a streaming warp's own
  if (warp < kStreamWarps && lane == 0) {
    for (int st = 0; st < stream::kStages; ++st) mbar_init(bars + 8 * st, 1);
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(base + kOffTmemSlot, kTmemCols);
    tmem_relinquish();
  } else if (warp == kWarpK && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_k16);
    tma_prefetch_desc(&tm_v16);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the plan has finished
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int4 first_part = make_int4(0, 0, 0, 0);         // the first piece, requested along with the header
  if (warp == kWarpK && lane < int(sizeof(Piece) / 16) && int(blockIdx.x) < w.piece_cap)
    first_part = __ldcg(reinterpret_cast<const int4*>(w.pieces + blockIdx.x) + lane);
  int n_pieces = __ldcg(w.header), n_items = __ldcg(w.header + 4);
  const int working = __ldcg(w.header + 6);
  if (uint32_t(__ldcg(w.header + 2)) != w.tag || n_pieces < 0 || n_pieces > w.piece_cap || n_items < 0 ||
      n_items > w.item_cap) {                      // a plan of another call: no work
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(a.err, kErrInvalid);
    n_pieces = n_items = 0;
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gsm + kOffTmemSlot);
  const int with_pieces = min(n_pieces, min(int(gridDim.x), working));   // CTAs that take pieces first
  const bool pieces_first = int(blockIdx.x) < with_pieces;
  const bool ok = !pieces_first || run_pieces(&tm_q, &tm_k, &tm_v, a, w, gsm, base, tmem, n_pieces, with_pieces,
                                             first_part);
  if (warp == kWarpMma) {
    __syncwarp();
    tmem_dealloc(tmem, kTmemCols);
  }

  // own keys: each streaming warp's ring lies over the tiles, which the pieces are done with
  if (!ok || warp >= kStreamWarps) return;
  // The first units are given to the CTAs that start with them, neighbouring
  // units to different SMs; the rest is claimed.
  const int others = int(gridDim.x) - with_pieces, warps = others * kStreamWarps;
  stream::run_warp<false>(&tm_k16, &tm_v16, a, w, n_items, base + warp * stream::kStages * stream::kStageBytes, bars,
                          reinterpret_cast<SuffixItem*>(gsm + kOffOwnSlots) + 2 * warp,
                          pieces_first ? -1 : warp * others + int(blockIdx.x) - with_pieces, warps, 2 * warps,
                          stream::SmallStep{});
}

// Small steps: too few keys for sharing to pay, and a thread of a CTA for each
// sequence.  The plan of such a step costs a CTA less than waiting for another
// kernel's, so every CTA makes its own, with the same checks, chunks and records
// (4 samples behind 512 keys 8.7 us, with the plan kernel 17.4).  That also holds
// where sharing would save some bytes, which are in L2 after the first reader: 32
// sequences behind 1024 keys, 137 MB in all, 20.0 us and 25.1 with sharing; 24 behind
// 2048, 203 MB, 25.2 and 25.5; 100 behind 1024, 271 MB, 35.8 and 28.2.
// How many sequences could share depends on the groups that are empty.  Where that
// decides, this kernel counts them and runs the step or leaves it to the kernels behind
// it, which have no work in the one case (64 sequences of 1000 keys, a group each, 58 us;
// 51 without them, 69 by the plan) and are late in the other (200 behind 4096 keys among
// empty groups 55 us; 51 by the plan alone, 269 here).
constexpr int kSmallThreads = 32 * kStreamWarps;
constexpr int kSmallSeqs = kSmallThreads;
constexpr int kSmallTokens = 4096;
// Contexts up to which a small step's rows are one chunk each, written at once, where the
// join and its launch cost more than the longer chunks: few units wait for every
// tile of theirs, some 0.6 us each, many fill the GPU all the same.  4 sequences of 8
// heads, 128 keys: 9.1 us and 8.7 with a join (called one after the other, from the host,
// 10.8 and 13.7); 192 keys 11.5 and 9.1.  214 of 4 heads, 190 keys: 13.4 and 21.0; 120 of
// 240 keys 13.8 and 15.2.
constexpr int kOneChunkKeysFew = 128, kOneChunkKeysMany = 384;
constexpr int kManyUnitsPerSm = 2;
// Shortest chunk: all of it in flight at once (2 rows of 320 keys: 8.7 us, 9.1 with one more tile).
constexpr int kSmallChunkTiles = stream::kStages;
constexpr uint32_t kSmallOffBars = stream::kRingBytes, kSmallOffSlots = kSmallOffBars + stream::kBarBytes;
constexpr uint32_t kSmallSmem = kSmallOffSlots + stream::kSlotBytes + 1024;
static_assert(kSmallOffSlots % 16 == 0 && kSmallSmem <= 220 * 1024, "shared memory");

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__global__ void __launch_bounds__(kSmallThreads, 1)
    small_step_kernel(const __grid_constant__ CUtensorMap tm_k16, const __grid_constant__ CUtensorMap tm_v16,
                      const __grid_constant__ AttnArgs a, const __grid_constant__ PrefixWork w) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ stream::SmallSeq seqs[kSmallSeqs];
  __shared__ int group_s0[kSmallSeqs], group_p[kSmallSeqs];
  __shared__ int64_t sums[4][kStreamWarps];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* gsm = smem_raw + (base - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool writer = blockIdx.x == 0;             // of what the join reads, and of the errors
  const uint32_t bars = base + kSmallOffBars + warp * stream::kStages * 8;
  const int S = a.num_seqs, T = a.num_tokens, NG = w.num_groups, H = a.num_heads, Hkv = a.num_kv_heads, G = H / Hkv;

  if (lane == 0) {
    for (int st = 0; st < stream::kStages; ++st) mbar_init(bars + 8 * st, 1);
    fence_mbar_init();
    if (warp == 0) {
      tma_prefetch_desc(&tm_k16);
      tma_prefetch_desc(&tm_v16);
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");   // it may start while the stream's last kernel ends
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int s0 = 0, s1 = 0, p = 0, c0 = 0, q_len = 0, n = 0;
  if (tid < NG) s0 = w.cu_groups[tid], s1 = w.cu_groups[tid + 1], p = w.prefix_lens[tid];
  if (tid < S) c0 = a.cu_seqlens_q[tid], q_len = a.cu_seqlens_q[tid + 1] - c0, n = w.context_lens[tid];
  if (writer)
    for (int t = tid; t < T; t += kSmallThreads) w.token_info[t] = make_int4(0, 0, 0, 0);
  group_s0[tid] = s0;
  group_p[tid] = p;
  int bad = tid < NG && (s0 < 0 || s1 < s0 || s1 > S || (tid == 0 && s0 != 0) || (tid == NG - 1 && s1 != S));
  bad = __syncthreads_or(bad);
  if (w.max_sharers >= 0) {
    const bool leave = S - __syncthreads_count(tid < NG && s1 > s0) > w.max_sharers;   // all but one of each group
    if (writer && tid == 0) w.header[7] = leave ? 0 : 1;
    if (leave) return;
  }
  int g = 0;                                       // the sequence's group: the last that starts at or before it
  for (int hi = NG - 1; g < hi;) {
    const int mid = (g + hi + 1) >> 1;
    if (group_s0[mid] <= tid) g = mid; else hi = mid - 1;
  }
  p = group_p[g];
  const bool ok = tid < S && p >= 0 && q_len >= 1 && c0 >= 0 && c0 + q_len <= T && q_len <= a.max_q_len && n >= q_len &&
                  p <= n - q_len && n <= a.max_context_len && int64_t(n) <= int64_t(a.max_blocks_per_seq) * a.block_size;
  const int tiles = ok ? (n - 1) / stream::kTileKeys + 1 : 0, rt = ok ? (q_len * G + kStreamRows - 1) / kStreamRows : 0;
  const int64_t my_tiles = warp_sum(int64_t(tiles) * rt * Hkv), my_rows = warp_sum(int64_t(rt) * Hkv);
  if (lane == 0) sums[0][warp] = my_tiles, sums[3][warp] = my_rows;
  __syncthreads();
  const int warps = int(gridDim.x) * kStreamWarps;
  int64_t all_tiles = 0, spare = warps;            // ceil(x / L) is less than x / L + 1 for each row tile and head
#pragma unroll
  for (int i = 0; i < kStreamWarps; ++i) all_tiles += sums[0][i], spare -= sums[3][i];
  // One unit a warp, where there are warps enough: a unit's beginning and end cost as much as some tiles (6 sequences
  // behind 4900 keys 13.2 us, with kUnitsPerWarp units a warp 18.5; one of 130,000 keys 89 and 99)
  const int64_t units = spare > 0 ? spare : w.stream_units, per = (all_tiles + units - 1) / units;
  const int L = int(per < w.min_chunk_tiles ? w.min_chunk_tiles : (per > (1 << 26) ? (1 << 26) : per));
  const int nch = ok ? (tiles - 1) / L + 1 : 0;
  const int64_t items = int64_t(rt) * nch, recs = nch > 1 ? int64_t(q_len) * H * nch : 0;
  int64_t item0 = items, rec0 = recs;              // exclusive scans over the CTA
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, item0, o), y = __shfl_up_sync(0xffffffffu, rec0, o);
    if (lane >= o) item0 += x, rec0 += y;
  }
  if (lane == 31) sums[1][warp] = item0, sums[2][warp] = rec0;
  __syncthreads();
  item0 -= items, rec0 -= recs;
  int64_t all_items = 0, all_recs = 0;
#pragma unroll
  for (int i = 0; i < kStreamWarps; ++i) {
    if (i < warp) item0 += sums[1][i], rec0 += sums[2][i];
    all_items += sums[1][i], all_recs += sums[2][i];
  }
  bad |= all_items > w.item_cap || all_recs > w.own_rec_cap;   // only if token ranges overlap
  seqs[tid] = stream::SmallSeq{int(item0), nch, c0, q_len, n, unsigned(w.prefix_rec_cap + rec0)};
  if (writer) {
    if (bad || (tid < S && !ok)) raise_error(a.err, kErrInvalid);
    if (ok && !bad)
      for (int t = 0; t < q_len; ++t)
        w.token_info[c0 + t] = make_int4(0, int(unsigned(w.prefix_rec_cap + rec0 + int64_t(t) * H * nch)), nch, 0);
    if (tid == 0) {
      w.header[1] = 0;
      w.header[2] = int32_t(w.tag);
    }
  }
  __syncthreads();
  stream::run_warp<true>(&tm_k16, &tm_v16, a, w, bad ? 0 : int(all_items), base + warp * stream::kStages * stream::kStageBytes,
                         bars, reinterpret_cast<SuffixItem*>(gsm + kSmallOffSlots) + 2 * warp,
                         warp * int(gridDim.x) + int(blockIdx.x), warps, 0, stream::SmallStep{seqs, S, L});
}

// A warp joins kJoinRows query heads of a token at a time and goes on to the next
// ones a grid further.  The records come from L2: what counts is bytes in flight,
// so 8 records are requested at once, two of each of four rows or four of each of
// two, and the next rows' description before them.  55,040 rows of 3 records: 23 us,
// 3.7 TB/s of them.  More CTAs an SM leave too few registers for that: the step of 12 prompt
// chunks takes 166 us with two, 167 with three, 183 with four.
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 4;
constexpr int kJoinCtasPerSm = 2;

// Rows h0 .. h0 + R - 1 of token tok, K records at a time, one pass with a running maximum.
template <int R, int K>
__device__ __forceinline__ void join_rows(const AttnArgs& a, const PrefixWork& w, int tok, int h0, int4 ti, int stride,
                                          int lane) {
  const int np = ti.x, n = np + ti.z;
  float4 acc[R];
  float mx[R], den[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    mx[r] = -INFINITY;
    den[r] = 0.f;
  }
  const size_t pre = (size_t(tok) * a.num_heads + h0) * stride, own = size_t(unsigned(ti.y)) + size_t(h0) * ti.z;
  const int rows = min(R, a.num_heads - h0);
  for (int k0 = 0; k0 < n; k0 += K) {
    float4 x[R][K];
    float2 ml[R][K];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int kk = k0 + k;
        x[r][k] = make_float4(0.f, 0.f, 0.f, 0.f);
        ml[r][k] = make_float2(-INFINITY, 0.f);
        if (kk < n && r < rows) {
          const size_t at = kk < np ? pre + size_t(r * stride + kk) : own + size_t(r * ti.z + kk - np);
          x[r][k] = __ldcg(reinterpret_cast<const float4*>(w.recs + at * HD) + lane);
          ml[r][k] = __ldcg(w.rec_ml + at);
        }
      }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float top = mx[r];
#pragma unroll
      for (int k = 0; k < K; ++k) top = fmaxf(top, ml[r][k].x);
      const float ref = top == -INFINITY ? 0.f : top;    // no key seen so far
      const float old = ex2(mx[r] - ref);
      acc[r].x *= old, acc[r].y *= old, acc[r].z *= old, acc[r].w *= old;
      den[r] *= old;
      mx[r] = top;
#pragma unroll
      for (int k = 0; k < K; ++k) {
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
  for (int r = 0; r < R; ++r) {
    if (r >= rows) break;
    const float inv = 1.0f / den[r];
    uint2 v;
    v.x = pack_bf16x2(acc[r].x * inv, acc[r].y * inv);
    v.y = pack_bf16x2(acc[r].z * inv, acc[r].w * inv);
    *(reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + (size_t(tok) * a.num_heads + h0 + r) * HD) + lane) = v;
  }
}

// ROWS: kJoinRows, or 1 where there are few rows, which then need the fewest steps in turn.
template <int ROWS>
__global__ void __launch_bounds__(kJoinThreads, kJoinCtasPerSm) join_kernel(const AttnArgs a, const PrefixWork w) {
  const int lane = threadIdx.x & 31;
  const unsigned per_token = unsigned(a.num_heads + ROWS - 1) / ROWS;
  const unsigned units = unsigned(a.num_tokens) * per_token, step = gridDim.x * (kJoinThreads / 32);
  unsigned u = blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (u >= units) return;
  int4 ti = __ldcg(w.token_info + u / per_token);
  const int stride = __ldcg(w.header + 1);
  if (uint32_t(__ldcg(w.header + 2)) != w.tag) return;
  while (u < units) {
    const unsigned next = u + step;
    const int4 ti_next = next < units ? __ldcg(w.token_info + next / per_token) : make_int4(0, 0, 0, 0);
    const int tok = int(u / per_token), h0 = int(u - unsigned(tok) * per_token) * ROWS;
    const int n = ti.x + ti.z;                           // below 2: left out, or already written
    if (ROWS == 1) {
      if (n > 1) join_rows<1, 8>(a, w, tok, h0, ti, stride, lane);
    } else if (n == 2) {
      join_rows<4, 2>(a, w, tok, h0, ti, stride, lane);
    } else if (n > 2) {
      join_rows<2, 4>(a, w, tok, h0, ti, stride, lane);
      if (h0 + 2 < a.num_heads) join_rows<2, 4>(a, w, tok, h0 + 2, ti, stride, lane);
    }
    ti = ti_next;
    u = next;
  }
}

// Very few rows, which may have very many records: a CTA to a row.  Each warp joins its
// share of the records, the first warp the eight results (a row of 8000 keys of 8 heads:
// the step 12 us, 29 with a warp to the row; 32,000 keys 31 and 72).
constexpr int kWideCtasPerSm = 4;
constexpr int kWideWarps = kJoinThreads / 32;
__global__ void __launch_bounds__(kJoinThreads, kWideCtasPerSm) join_wide_kernel(const AttnArgs a, const PrefixWork w) {
  constexpr int K = 4;                             // records in flight per warp
  __shared__ float4 part_acc[kWideWarps][32];
  __shared__ float2 part_ml[kWideWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tok = int(blockIdx.x) / a.num_heads, h = int(blockIdx.x) - tok * a.num_heads;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 ti = __ldcg(w.token_info + tok);
  const int stride = __ldcg(w.header + 1);
  if (uint32_t(__ldcg(w.header + 2)) != w.tag) return;
  const int np = ti.x, n = np + ti.z;
  if (n < 2) return;                               // left out, or already written
  const size_t pre = (size_t(tok) * a.num_heads + h) * stride, own = size_t(unsigned(ti.y)) + size_t(h) * ti.z;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float mx = -INFINITY, den = 0.f;
  auto add = [&](float top, const float4& x, float2 ml) {   // top: a maximum of at least ml.x
    const float f = ex2(ml.x - (top == -INFINITY ? 0.f : top));
    den = fmaf(f, ml.y, den);
    acc.x = fmaf(f, x.x, acc.x);
    acc.y = fmaf(f, x.y, acc.y);
    acc.z = fmaf(f, x.z, acc.z);
    acc.w = fmaf(f, x.w, acc.w);
  };
  auto raise = [&](float top) {
    const float old = ex2(mx - (top == -INFINITY ? 0.f : top));
    acc.x *= old, acc.y *= old, acc.z *= old, acc.w *= old;
    den *= old;
    mx = top;
  };
  for (int k0 = warp; k0 < n; k0 += kWideWarps * K) {
    float4 x[K];
    float2 ml[K];
    float top = mx;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int kk = k0 + k * kWideWarps;
      x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      ml[k] = make_float2(-INFINITY, 0.f);
      if (kk < n) {
        const size_t at = kk < np ? pre + kk : own + kk - np;
        x[k] = __ldcg(reinterpret_cast<const float4*>(w.recs + at * HD) + lane);
        ml[k] = __ldcg(w.rec_ml + at);
      }
      top = fmaxf(top, ml[k].x);
    }
    raise(top);
#pragma unroll
    for (int k = 0; k < K; ++k) add(top, x[k], ml[k]);
  }
  part_acc[warp][lane] = acc;
  if (lane == 0) part_ml[warp] = make_float2(mx, den);
  __syncthreads();
  if (warp > 0) return;
  float top = mx;
#pragma unroll
  for (int k = 1; k < kWideWarps; ++k) top = fmaxf(top, part_ml[k].x);
  raise(top);
#pragma unroll
  for (int k = 1; k < kWideWarps; ++k) add(top, part_acc[k][lane], part_ml[k]);
  const float inv = 1.0f / den;
  uint2 v;
  v.x = pack_bf16x2(acc.x * inv, acc.y * inv);
  v.y = pack_bf16x2(acc.z * inv, acc.w * inv);
  *(reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + size_t(blockIdx.x) * HD) + lane) = v;
}
bool wide_join(const AttnArgs& a, const PrefixWork& w) {
  return int64_t(a.num_tokens) * a.num_heads <= int64_t(w.num_sms) * kWideCtasPerSm;
}

std::mutex g_attr_mutex;
bool g_attr_set[64] = {};

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Capacities of a step's lists.
struct PrefixSizes {
  size_t S, T, NG, pieces, items, prefix_recs, piece_recs, own_recs;
};
int tile_tokens(int group_heads) { return BM / group_heads; }
PrefixSizes prefix_sizes(int32_t num_q_heads, int32_t num_kv_heads, int32_t num_seqs, int32_t num_tokens, int32_t num_groups,
                         int32_t max_context_len) {
  PrefixSizes z;
  z.S = size_t(num_seqs), z.T = size_t(num_tokens), z.NG = size_t(num_groups);
  const size_t G = size_t(num_q_heads / num_kv_heads), rows = z.T * size_t(num_q_heads);
  const bool chunks = z.T > z.S && (z.T - z.S + 1) * G > size_t(kMaxStreamRows);   // where every sequence has a token
  // uncut: groups that share have two sequences or more; chunks are all of their tokens
  const size_t pairs = z.T / (2 * size_t(tile_tokens(int(G))));
  z.pieces = size_t(num_kv_heads) * (pairs + std::min(z.NG, z.S / 2) + 1 + (chunks ? pairs + z.S : 0)) + kExtraPieces;
  z.prefix_recs = std::min(rows * 2 * kMaxSegs, rows * 2 + size_t(kExtraRecs));
  z.piece_recs = chunks ? rows * 2 + size_t(kExtraRecs) : 0;
  // ceil(x / L) <= x / L + 1 for every streamed sequence, and all x / L together are at most the units aimed for,
  // twice that where L is halved
  const size_t units = 2 * size_t(kMaxSms) * kStreamWarps * kUnitsPerWarp;
  const size_t shortest = size_t(stream::kTileKeys) * std::min(kMinChunkTiles, kSmallChunkTiles);
  const size_t chunks_of_row = (size_t(max_context_len) + shortest - 1) / shortest;
  z.items = z.T * G / kStreamRows + z.S + units + 1;
  z.own_recs = z.piece_recs + std::min(rows * chunks_of_row, rows + kStreamRows * units);
  return z;
}

}  // namespace

size_t shared_prefix_workspace_bytes(int32_t num_q_heads, int32_t num_kv_heads, int32_t num_seqs, int32_t num_tokens,
                                     int32_t num_groups, int32_t max_context_len) {
  const PrefixSizes z = prefix_sizes(num_q_heads, num_kv_heads, num_seqs, num_tokens, num_groups, max_context_len);
  return 256 + align256(z.NG * 16) + 2 * align256(z.S * 16) + align256((z.NG + z.S) * 4) + align256(z.pieces * sizeof(Piece)) +
         align256(z.items * sizeof(SuffixItem)) + align256(z.T * 16) +
         align256((z.prefix_recs + z.own_recs) * kPrefixRecBytes);
}

// The tensor maps of the K and V pools, boxes of one block and head.
static cb_status encode_pools(const AttnArgs& a, EncodeTiledFn enc, bool tiles16, CUtensorMap* tk, CUtensorMap* tv) {
  const cuuint64_t B = cuuint64_t(a.block_size), boxes = cuuint64_t(a.num_blocks) * a.num_kv_heads;
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  CUresult r = CUDA_SUCCESS;
  for (int v = 0; v < 2 && r == CUDA_SUCCESS; ++v) {
    void* pool = const_cast<void*>(v ? a.v_pool : a.k_pool);
    CUtensorMap* tm = v ? tv : tk;
    if (tiles16) {                                 // both 64-dim halves of 16 rows at a time, for the streams
      const cuuint64_t dims[4] = {64, B, 2, boxes}, strides[3] = {HD * 2, 128, B * HD * 2};
      const cuuint32_t box[4] = {64, cuuint32_t(stream::kTileKeys), 2, 1};
      r = enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, pool, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    } else {                                       // a block's 64-dim half, for the pieces
      const cuuint64_t dims[3] = {cuuint64_t(HD), B, boxes}, strides[2] = {HD * 2, B * HD * 2};
      const cuuint32_t box[3] = {64, cuuint32_t(B), 1};
      r = enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, pool, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    }
  }
  return r == CUDA_SUCCESS ? CB_OK : fail(CB_ERR_CUDA, "shared prefixes: encoding the KV tensor maps failed (%d)", int(r));
}

// Lets the kernels take their dynamic shared memory on the current device.
static cb_status allow_shared_memory() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
    return fail(CB_ERR_UNSUPPORTED, "shared prefixes: no usable current device");
  std::lock_guard<std::mutex> lock(g_attr_mutex);
  if (g_attr_set[dev]) return CB_OK;
  cudaError_t e = cudaFuncSetAttribute(prefix_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmemBytes));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(small_step_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmallSmem));
  if (e != cudaSuccess) return cuda_fail(e, "shared prefixes: shared memory attribute");
  g_attr_set[dev] = true;
  return CB_OK;
}

static cb_status launch_prefix_tc(const AttnArgs& a, const PrefixWork& w, cudaStream_t stream) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return CB_ERR_CUDA;
  const int G = a.num_heads / a.num_kv_heads;
  CUtensorMap tq, tk, tv, tk16, tv16;
  // q as [tokens][heads][128]: a box is one key/value head's query heads of tile_tokens tokens, one 64-dim half
  const cuuint64_t dims[3] = {cuuint64_t(HD), cuuint64_t(a.num_heads), cuuint64_t(a.num_tokens)};
  const cuuint64_t strides[2] = {cuuint64_t(HD) * 2, cuuint64_t(a.num_heads) * HD * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(G), cuuint32_t(w.tile_tokens)}, ones[3] = {1, 1, 1};
  CUresult r = enc(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides, box, ones,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(CB_ERR_CUDA, "shared prefixes: encoding the Q tensor map failed (%d)", int(r));
  cb_status st = encode_pools(a, enc, false, &tk, &tv);
  if (st == CB_OK) st = encode_pools(a, enc, true, &tk16, &tv16);
  if (st == CB_OK) st = allow_shared_memory();
  if (st != CB_OK) return st;
  cudaError_t e = launch_kernel(prefix_tc_kernel, dim3(unsigned(w.num_sms)), dim3(kThreads), kSmemBytes, stream, true, tq, tk,
                                tv, tk16, tv16, a, w);
  return e == cudaSuccess ? CB_OK : cuda_fail(e, "shared prefixes: launch");
}

static cb_status launch_small_step(const AttnArgs& a, const PrefixWork& w, cudaStream_t stream) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return CB_ERR_CUDA;
  CUtensorMap tk16, tv16;
  cb_status st = encode_pools(a, enc, true, &tk16, &tv16);
  if (st == CB_OK) st = allow_shared_memory();
  if (st != CB_OK) return st;
  cudaError_t e = launch_kernel(small_step_kernel, dim3(unsigned(w.num_sms)), dim3(kSmallThreads), kSmallSmem, stream, true,
                                tk16, tv16, a, w);
  return e == cudaSuccess ? CB_OK : cuda_fail(e, "shared prefixes: launch");
}

static cb_status launch_join(const AttnArgs& a, const PrefixWork& w, cudaStream_t stream) {
  if (wide_join(a, w)) {
    cudaError_t e = launch_kernel(join_wide_kernel, dim3(unsigned(a.num_tokens) * unsigned(a.num_heads)), dim3(kJoinThreads), 0,
                                  stream, true, a, w);
    return e == cudaSuccess ? CB_OK : cuda_fail(e, "shared prefixes: join launch");
  }
  const int64_t slots = int64_t(w.num_sms) * kJoinCtasPerSm, per_cta = kJoinThreads / 32;
  const bool few = int64_t(a.num_tokens) * a.num_heads <= slots * per_cta;
  const int64_t warps = int64_t(a.num_tokens) * (few ? a.num_heads : (a.num_heads + kJoinRows - 1) / kJoinRows);
  const int64_t grid = std::min<int64_t>(slots, (warps + per_cta - 1) / per_cta);
  cudaError_t e = launch_kernel(few ? join_kernel<1> : join_kernel<kJoinRows>, dim3(unsigned(grid)), dim3(kJoinThreads), 0,
                                stream, true, a, w);
  return e == cudaSuccess ? CB_OK : cuda_fail(e, "shared prefixes: join launch");
}

// A step with shared prefixes on one stream: the plan, the pieces and streams (a small
// step's streams alone), and the join, each a programmatic dependent of the one before.
cb_status run_shared_prefix(const AttnArgs& a, const int32_t* cu_groups, const int32_t* prefix_lens, int32_t num_groups,
                            void* workspace, cudaStream_t stream) {
  NvtxRange nvtx("cb.shared_prefix");
  if (int64_t(a.num_blocks) * a.num_kv_heads >= (int64_t(1) << 31))
    return fail(CB_ERR_UNSUPPORTED, "shared prefixes: num_blocks * num_kv_heads must fit in int32");
  const PrefixSizes z = prefix_sizes(a.num_heads, a.num_kv_heads, a.num_seqs, a.num_tokens, num_groups, a.max_context_len);
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
  w.seqs = reinterpret_cast<int4*>(take(z.S * 16));
  w.first_piece = reinterpret_cast<int32_t*>(take((z.NG + z.S) * 4));
  w.seq_recs = reinterpret_cast<int4*>(take(z.S * 16));
  w.pieces = reinterpret_cast<Piece*>(take(z.pieces * sizeof(Piece)));
  w.items = reinterpret_cast<SuffixItem*>(take(z.items * sizeof(SuffixItem)));
  w.token_info = reinterpret_cast<int4*>(take(z.T * 16));
  w.recs = reinterpret_cast<float*>(p);
  w.rec_ml = reinterpret_cast<float2*>(w.recs + (z.prefix_recs + z.own_recs) * HD);
  static std::atomic<uint32_t> next_tag{1};
  w.tag = next_tag.fetch_add(1);

  // Small: what sharing could save does not pay for it, and no sequence's own keys are pieces.  All sequences but
  // one of each group could share, at most their whole contexts, and any group but one may be empty.  With at
  // least two sequences a group, counting all groups misses half of the sharers at most (84 behind 1024 keys
  // among 41 empty groups 53 us, 28 without those); with fewer, the device counts.
  const int64_t row_tiles = (int64_t(a.max_q_len) * (a.num_heads / a.num_kv_heads) + kStreamRows - 1) / kStreamRows;
  const double each = double(a.max_context_len) * a.num_kv_heads * (4.0 * HD) * row_tiles;
  const int sharers = int(std::min(double(kSmallSeqs), std::ceil(double(kSmallUs) * kBytesPerUs / each) - 1.0));
  const bool fits = a.num_seqs <= kSmallSeqs && num_groups <= kSmallSeqs && a.num_tokens <= kSmallTokens &&
                    (a.max_q_len == 1 || int64_t(a.max_q_len) * (a.num_heads / a.num_kv_heads) <= kMaxStreamRows);
  const bool maybe = fits && a.num_seqs - num_groups <= sharers;
  const bool small = maybe && (a.num_seqs - 1 <= sharers || num_groups <= a.num_seqs / 2);
  const bool both = maybe && !small;
  w.max_sharers = both ? sharers : -1;
  const bool many = int64_t(a.num_seqs) * a.num_kv_heads >= int64_t(kManyUnitsPerSm) * w.num_sms;
  const bool one_chunk = maybe && a.max_context_len <= (many ? kOneChunkKeysMany : kOneChunkKeysFew);
  w.min_chunk_tiles = one_chunk ? kOneChunkKeysMany / stream::kTileKeys : kSmallChunkTiles;
  cb_status st = CB_OK;
  if (maybe) st = launch_small_step(a, w, stream);
  if (st == CB_OK && !small) {
    cudaError_t e = launch_kernel(prefix_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, true, a, w);
    if (e != cudaSuccess) return cuda_fail(e, "shared prefixes: plan launch");
    st = launch_prefix_tc(a, w, stream);
  }
  if (st != CB_OK || (small && one_chunk)) return st;
  return launch_join(a, w, stream);
}

}  // namespace cb
