// cb_ragged_attention_q8: attention of a packed step over a cache in 8 bits (e4m3
// pages, a fp32 scale for each page and key/value head; head_dim 128).
//
//     out = sum_j p_j vs_j v_j / sum_j p_j,  p_j = exp(scale * ks_j q . k_j),
// ks_j, vs_j the scales of key j's page, k_j and v_j its e4m3 numbers.
//
// Rows are streams of single warps (quant_stream.cuh).  A step without chunks and
// without a plan kernel: every CTA lays the step's streams end to end for itself and
// every warp of the grid takes an equal share of all tiles, whatever the lengths of
// the contexts.  A share begins and ends inside a stream at most, so a warp leaves at
// most two records a row, and the join reads what it needs: 2 records for each warp
// of the grid, however many sequences there are.  Where the streams are no more than
// the SMs and short, each is a CTA's, in equal parts to its warps, and the CTA joins
// them: one launch.  Steps of more sequences than a CTA has threads, with chunks, or
// whose prefixes are worth sharing, are listed by a plan kernel (shared_prefix.h) as
// pieces (quant_pieces.cuh) and streams.
#include <algorithm>
#include <mutex>

#include <cuda.h>

#include "device_common.cuh"
#include "kernels.h"
#include "quant_pieces.cuh"
#include "quant_stream.cuh"
#include "runtime.h"
#include "shared_prefix.h"
#include "sm100_ptx.cuh"

namespace cb {
namespace {

using namespace sm100;
using qstream::RangeSeq;
using qstream::RangeUnits;
using qstream::FewShape;
using qstream::SharesShape;
using qstream::WideShape;

constexpr int HD = kPrefixDim;
constexpr int kMaxSms = 160;             // SMs that the records are sized for
constexpr int kStepTokens = 4096;        // of a step without a plan kernel
// Tiles of a warp's shortest share: more warps load sooner, but leave more records.  4 rows of 1300 keys, 20 of 400 and 8 of
// 2000, 32/8 heads, us: with 1 10.7, 14.5, 14.6; 3 11.7, 14.1, 14.6; 8 14.6, 15.6, 16.2.
constexpr int kMinShareTiles = 3;
// Tiles a warp, at most, of a step whose streams are a CTA's each, which needs no join kernel.  1, 4 and 16 tokens of 32/8 heads,
// 12 warps, us, so and in shares: contexts of 512 7.3, 7.8, 8.0 and 10.7, 11.4, 12.4; of 1280 (6.7 tiles) 10.7, 11.1, 12.3 and
// 11.0, 11.8, 14.7; of 1536 11.6, 12.0, 13.9 and 9.8, 11.9, 16.2; 4 of 32 heads on one, 8 warps: of 768 (6 tiles) 12.1 and 13.7,
// of 1024 13.6 and 13.8, of 1280 15.3 and 14.1.
constexpr int kApartTiles = 7;
// Bytes that sharing has to be able to save for the plan, the pieces and the larger join to be worth their time, by the host's
// bound on the contexts.  Chats of 32/8 heads with up to 512 keys of their own, us, with the plan and without: 32 behind 2000
// shared ones (1.6e8 bytes) 32.6, 29.8; 64 behind 1000 (1.95e8) 35.0, 31.5; 48 behind 2000 (2.4e8) 34.7, 37.7; 64 behind 2000
// (3.2e8) 37.1, 45.9.
constexpr double kSharingBytes = 2.3e8;
// What the plan's estimates go by, in microseconds and bytes: a KV tile for two row tiles and for one (2.2, ends
// included: either is widened alike), and what an SM's streams read beside pieces.  3 chunks of 662 tokens behind 2048 keys with
// 64 decode rows, and with 200, 32/8 heads, us: these 146, 236; tiles of 1.7 153, 315; streams of 2.4e4 153, 315; of 4.2e4 146,
// 239.
constexpr float kTileUsTwo = 2.0f, kTileUsOne = 2.0f, kStreamBytesPerUsPerSm = 3.6e4f;

// What the CTAs of a step without a plan kernel make of it, for the join.
struct StepWork {
  const int32_t* cu_groups;              // null: none
  const int32_t* prefix_lens;
  int32_t num_groups;
  int32_t* header;                       // [0] tiles of a share
  int4* token_info;                      // [num_tokens] (first tile of its sequence's streams, tiles of each, token of the
                                         // sequence, 1: there is something to join)
  float* recs;                           // [2 * warps][row tile][HD]
  float2* rec_ml;
};

// The weighted sum of a row's records, by the lanes of a warp, 4 dims each.
struct Joined {
  float4 acc;
  float mx, den;
  __device__ __forceinline__ void raise(float top) {
    const float old = ex2(mx - (top == -INFINITY ? 0.f : top));
    acc.x *= old, acc.y *= old, acc.z *= old, acc.w *= old;
    den *= old;
    mx = top;
  }
  __device__ __forceinline__ void add(const float4& x, float2 ml) {   // mx is at least ml.x
    const float f = ex2(ml.x - (mx == -INFINITY ? 0.f : mx));
    den = fmaf(f, ml.y, den);
    acc.x = fmaf(f, x.x, acc.x);
    acc.y = fmaf(f, x.y, acc.y);
    acc.z = fmaf(f, x.z, acc.z);
    acc.w = fmaf(f, x.w, acc.w);
  }
};
constexpr int kJoinFlight = 4;           // records of a row requested at once

// Adds the records of parts k0 .. k0 + K - 1 of n to j; at(k) is where part k's is.
template <int K, class At>
__device__ __forceinline__ void join_parts(Joined& j, const float* recs, const float2* rec_ml, int k0, int n, int lane, const At& at) {
  float4 x[K];
  float2 ml[K];
  float top = j.mx;
#pragma unroll
  for (int i = 0; i < K; ++i) {
    x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    ml[i] = make_float2(-INFINITY, 0.f);
    if (k0 + i < n) {
      const size_t rec = at(k0 + i);
      x[i] = __ldcg(reinterpret_cast<const float4*>(recs + rec * HD) + lane);
      ml[i] = __ldcg(rec_ml + rec);
    }
    top = fmaxf(top, ml[i].x);
  }
  j.raise(top);
#pragma unroll
  for (int i = 0; i < K; ++i) j.add(x[i], ml[i]);
}
__device__ __forceinline__ void write_row(const AttnArgs& a, size_t row, const Joined& j, int lane) {
  const float inv = 1.0f / j.den;
  *(reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * HD) + lane) =
      make_uint2(stream::pack2(j.acc.x * inv, j.acc.y * inv), stream::pack2(j.acc.z * inv, j.acc.w * inv));
}

template <class Sh>
__device__ __forceinline__ void init_bars(uint32_t bars) {
  for (int st = 0; st < Sh::kStages; ++st) mbar_init(bars + 8 * st, qstream::kBarArrivals);
  fence_mbar_init();
}

// APART: a CTA to a stream, whose warps' parts it joins itself; else every warp of the grid takes its share of all tiles.
template <class Sh, bool APART>
__global__ void __launch_bounds__(Sh::kThreads, 1)
    q8_step_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ AttnArgs a, const __grid_constant__ StepWork w) {
  constexpr int kWarps = Sh::kWarps, kThreads = Sh::kThreads, kSeqs = kThreads;   // a thread for each sequence
  extern __shared__ uint8_t smem_raw[];
  __shared__ RangeSeq seqs[kSeqs];
  __shared__ int group_s0[kSeqs], group_p[kSeqs];
  __shared__ int2 sums[kWarps];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* gsm = smem_raw + (base - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool writer = blockIdx.x == 0;             // of what the join reads, and of the errors
  const uint32_t bars = base + Sh::kOffBars + warp * Sh::kWarpBarBytes;
  const int S = a.num_seqs, T = a.num_tokens, NG = w.num_groups, H = a.num_heads, Hkv = a.num_kv_heads, G = H / Hkv;

  if (lane == 0) {
    init_bars<Sh>(bars);
    if (warp == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");   // it may start while the stream's last kernel ends
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int s0 = 0, s1 = 0, p = 0, c0 = 0, c1 = 0, n = 0;
  if (tid < NG) s0 = w.cu_groups[tid], s1 = w.cu_groups[tid + 1], p = w.prefix_lens[tid];
  if (tid < S) c0 = a.cu_seqlens_q[tid], c1 = a.cu_seqlens_q[tid + 1], n = a.context_lens[tid];
  const int q_len = c1 - c0;
  if (writer)
    for (int t = tid; t < T; t += kThreads) w.token_info[t] = make_int4(0, 0, 0, 0);
  bool bad = false;
  if (NG > 0) {                                    // nothing is shared here, but what does not hold is reported
    group_s0[tid] = s0;
    group_p[tid] = p;
    bad = tid < NG && (s0 < 0 || s1 < s0 || s1 > S || (tid == 0 && s0 != 0) || (tid == NG - 1 && s1 != S));
    bad = __syncthreads_or(bad);
    int g = 0;                                     // the sequence's group: the last that starts at or before it
    for (int hi = NG - 1; g < hi;) {
      const int mid = (g + hi + 1) >> 1;
      if (group_s0[mid] <= tid) g = mid; else hi = mid - 1;
    }
    p = group_p[g];
  }
  const bool ok = tid < S && p >= 0 && c1 > c0 && c0 >= 0 && c1 <= T && q_len <= a.max_q_len && n >= q_len &&
                  p <= n - q_len && n <= a.max_context_len && int64_t(n) <= int64_t(a.max_blocks_per_seq) * a.block_size;
  const int tiles = ok && !bad ? (n - 1) / qstream::kTileKeys + 1 : 0;
  const int streams = tiles > 0 ? (q_len * G + Sh::kRows - 1) / Sh::kRows * Hkv : 0;
  int off = tiles * streams, st0 = streams;        // exclusive scans over the CTA (the host has checked their range)
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, off, o), y = __shfl_up_sync(0xffffffffu, st0, o);
    if (lane >= o) off += x, st0 += y;
  }
  if (lane == 31) sums[warp] = make_int2(off, st0);
  __syncthreads();
  off -= tiles * streams, st0 -= streams;
  int all_tiles = 0, all_streams = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) off += sums[i].x, st0 += sums[i].y;
    all_tiles += sums[i].x, all_streams += sums[i].y;
  }
  const int id = warp * int(gridDim.x) + int(blockIdx.x);
  seqs[tid] = RangeSeq{off, tiles, st0, c0, q_len, n};
  if (writer && ((bad && tid == 0) || (tid < S && !ok))) raise_error(a.err, kErrInvalid);
  int per, begin = 0, limit = all_tiles, k = id;   // tiles of a share; the tiles that are shared; the warp's share of them
  RangeSeq own = {};                               // the sequence of the CTA's one stream
  if (!APART) {
    per = max(kMinShareTiles, (all_tiles - 1) / (int(gridDim.x) * kWarps) + 1);
    if (writer) {
      if (tiles > 0)
        for (int t = 0; t < q_len; ++t) w.token_info[c0 + t] = make_int4(off, tiles, t, 1);
      if (tid == 0) w.header[0] = per;
    }
    __syncthreads();
  } else {
    __syncthreads();
    if (int(blockIdx.x) >= all_streams) return;
    int s = 0;                                     // the last sequence whose streams begin at or before it
    for (int hi = S - 1; s < hi;) {
      const int mid = (s + hi + 1) >> 1;
      if (seqs[mid].stream0 <= int(blockIdx.x)) s = mid; else hi = mid - 1;
    }
    own = seqs[s];
    per = (own.tiles - 1) / kWarps + 1;
    begin = own.off + (int(blockIdx.x) - own.stream0) * own.tiles, limit = begin + own.tiles, k = warp;
  }
  RangeUnits units{seqs, S, Hkv, Sh::kRows, int(min(int64_t(limit), begin + int64_t(k) * per)),
                   int(min(int64_t(limit), begin + int64_t(k + 1) * per)), unsigned(2 * id * Sh::kRows)};
  qstream::run_warp<Sh>(&tm_k, &tm_v, a, w.recs, w.rec_ml, base + warp * Sh::kStages * qstream::kStageBytes, bars,
                        reinterpret_cast<const float2*>(gsm + (bars - base) + 8 * Sh::kStages),
                        reinterpret_cast<SuffixItem*>(gsm + Sh::kOffSlots) + 2 * warp, units);
  if (!APART || own.tiles <= 1) return;
  __syncthreads();                                 // the warps' records are written
  const int x = int(blockIdx.x) - own.stream0, hk = x % Hkv, row0 = x / Hkv * Sh::kRows, parts = (own.tiles - 1) / per + 1;
  for (int r = warp; r < min(Sh::kRows, own.q_len * G - row0); r += kWarps) {
    Joined j{make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.f};
    join_parts<kWarps>(j, w.recs, w.rec_ml, 0, parts, lane,
                       [&](int part) { return size_t(2 * (part * int(gridDim.x) + int(blockIdx.x))) * Sh::kRows + r; });
    write_row(a, size_t(own.tok0 + (row0 + r) / G) * H + hk * G + (row0 + r) % G, j, lane);
  }
}

// The pieces of a step as the plan lists them, one CTA per SM; those beyond the header[6] that take pieces leave their SMs to
// the streams behind.
__global__ void __launch_bounds__(qpieces::kThreads, 1)
    q8_pieces_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ AttnArgs a, const __grid_constant__ PrefixWork w) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* gsm = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Set up while the plan still runs: barriers, and tensor memory
  if (threadIdx.x == 0) qpieces::init_bars(base);
  if (warp == qpieces::kWarpMma) {
    tmem_alloc(base + qpieces::kOffTmemSlot, qpieces::kTmemCols);
    tmem_relinquish();
  } else if (warp == qpieces::kWarpK && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the plan has finished
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int n_pieces = __ldcg(w.header);
  const int working = __ldcg(w.header + 6);
  if (uint32_t(__ldcg(w.header + 2)) != w.tag || n_pieces < 0 || n_pieces > w.piece_cap) {   // a plan of another call: no work
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(a.err, kErrInvalid);
    n_pieces = 0;
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gsm + qpieces::kOffTmemSlot);
  const int with_pieces = min(n_pieces, min(int(gridDim.x), working));
  if (int(blockIdx.x) < with_pieces) qpieces::run_pieces(&tm_q, &tm_k, &tm_v, a, w, gsm, base, tmem, n_pieces, with_pieces);
  if (warp == qpieces::kWarpMma) {
    __syncwarp();
    tmem_dealloc(tmem, qpieces::kTmemCols);
  }
}

// The streams of a step as the plan lists them.  wait_previous 0: behind the pieces' kernel, which lets this one start once
// the plan has finished, on the SMs without pieces and, as those end, on theirs.  The grid ends no sooner than that one.
template <class Sh>
__global__ void __launch_bounds__(Sh::kThreads, 1)
    q8_streams_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ AttnArgs a, const __grid_constant__ PrefixWork w, int wait_previous) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* gsm = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = base + Sh::kOffBars + warp * Sh::kWarpBarBytes;
  if (lane == 0) init_bars<Sh>(bars);
  if (wait_previous) asm volatile("griddepcontrol.wait;" ::: "memory");   // the plan has finished
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const EndAfterPrevious end{!wait_previous && blockIdx.x == 0};
  int n_items = __ldcg(w.header + 4);
  if (uint32_t(__ldcg(w.header + 2)) != w.tag || n_items < 0 || n_items > w.item_cap) {   // a plan of another call: no work
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(a.err, kErrInvalid);
    n_items = 0;
  }
  __syncwarp();
  qstream::ListedUnits units{w, a.num_kv_heads, n_items * a.num_kv_heads};
  qstream::run_warp<Sh>(&tm_k, &tm_v, a, w.recs, w.rec_ml, base + warp * Sh::kStages * qstream::kStageBytes, bars,
                        reinterpret_cast<const float2*>(gsm + (bars - base) + 8 * Sh::kStages),
                        reinterpret_cast<SuffixItem*>(gsm + Sh::kOffSlots) + 2 * warp, units);
}

constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;

// Joins the rows that lie in several shares.  WIDE: a CTA to a row, each warp with its part of the records, where rows are
// few (4 an SM at most) and may have very many; else a warp to a row.  A step with one and the other, 32/8 heads, us: 1 row of
// 8000 keys 15.6, 34.8; of 60,000 37, 91; 16 of 4000 25.5, 32.6; 19 of 1500 17.3, 21.4.
template <bool WIDE>
__global__ void __launch_bounds__(kJoinThreads) q8_join_kernel(const AttnArgs a, const StepWork w, int row_tile) {
  __shared__ float4 part_acc[WIDE ? kJoinWarps : 1][32];
  __shared__ float2 part_ml[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H = a.num_heads, Hkv = a.num_kv_heads, G = H / Hkv;
  const int rows = a.num_tokens * H, step = WIDE ? int(gridDim.x) : int(gridDim.x) * kJoinWarps;
  int row = WIDE ? int(blockIdx.x) : int(blockIdx.x) * kJoinWarps + warp;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int per = __ldcg(w.header);
  for (; row < rows; row += step) {
    const int tok = row / H, h = row - tok * H;
    const int4 ti = __ldcg(w.token_info + tok);
    if (ti.w == 0) continue;                       // left out
    const int hk = h / G, r = ti.z * G + h - hk * G, rt = r / row_tile;
    const int begin = ti.x + (rt * Hkv + hk) * ti.y;   // of the row's stream, in tiles
    const int f = begin / per, n = (begin + ti.y - 1) / per - f + 1;   // its first share, and shares
    if (n == 1) continue;                          // written already
    const int in_tile = r - rt * row_tile;
    const int first = (2 * f + (begin > f * per ? 1 : 0)) * row_tile + in_tile;   // the last part of share f, or its first
    Joined j{make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.f};
    for (int k0 = WIDE ? warp * kJoinFlight : 0; k0 < n; k0 += WIDE ? kJoinThreads / 32 * kJoinFlight : kJoinFlight) {
      join_parts<kJoinFlight>(j, w.recs, w.rec_ml, k0, n, lane, [&](int k) { return k == 0 ? size_t(first) : size_t(2 * (f + k)) * row_tile + in_tile; });
    }
    if (WIDE) {
      part_acc[warp][lane] = j.acc;
      if (lane == 0) part_ml[warp] = make_float2(j.mx, j.den);
      __syncthreads();
      if (warp == 0) {
        float top = j.mx;
#pragma unroll
        for (int k = 1; k < kJoinWarps; ++k) top = fmaxf(top, part_ml[k].x);
        j.raise(top);
#pragma unroll
        for (int k = 1; k < kJoinWarps; ++k) j.add(part_acc[k][lane], part_ml[k]);
      }
    }
    if (!WIDE || warp == 0) write_row(a, size_t(row), j, lane);
    if (WIDE) __syncthreads();                     // the parts are read before the next row's
  }
}

// Joins the rows of a listed step, a warp to every W-th row.  Its lanes look 32 rows ahead for those with records to join:
// in a step of prompts and decode rows most have none, and the others have many, so that what bounds it is the steps that
// one row's records take in turn.  3 chunks of 662 tokens and 64 decode rows of up to 26 records, 32/8 heads: the step 172 us,
// 190 with units of 4 neighbouring rows a warp, which few warps then hold; 4 CTAs an SM, of 64 registers, 175.
constexpr int kListedFlight = 8, kListedCtasPerSm = 2;
__global__ void __launch_bounds__(kJoinThreads, kListedCtasPerSm) q8_listed_join_kernel(const AttnArgs a, const PrefixWork w) {
  const int lane = threadIdx.x & 31, H = a.num_heads;
  const int64_t rows = int64_t(a.num_tokens) * H;
  const int warps = int(gridDim.x) * kJoinWarps, first = int(threadIdx.x >> 5) * int(gridDim.x) + int(blockIdx.x);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int stride = __ldcg(w.header + 1);
  if (uint32_t(__ldcg(w.header + 2)) != w.tag) return;   // a plan of another call
  for (int64_t r0 = first; r0 < rows; r0 += int64_t(warps) * 32) {
    const int64_t mine = r0 + int64_t(lane) * warps;
    const int4 ti = mine < rows ? __ldcg(w.token_info + mine / H) : make_int4(0, 0, 0, 0);
    unsigned two = __ballot_sync(0xffffffffu, ti.x + ti.z == 2);    // below 2: left out, or already written
    unsigned more = __ballot_sync(0xffffffffu, ti.x + ti.z > 2);
    // where record k of the row in lane `from` is
    int np, own, n;
    size_t row, own0;
    auto look = [&](int from) {
      np = __shfl_sync(0xffffffffu, ti.x, from), own = __shfl_sync(0xffffffffu, ti.y, from);
      n = __shfl_sync(0xffffffffu, ti.z, from);
      row = size_t(r0 + int64_t(from) * warps);
      own0 = size_t(unsigned(own)) + row % unsigned(H) * size_t(n);
      n += np;
    };
    auto at = [&](int k) { return k < np ? row * size_t(stride) + k : own0 + (k - np); };
    while (two) {                                        // 4 at once
      float4 x[4][2];
      float2 ml[4][2];
      const unsigned these = two;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (!two) break;
        look(__ffs(two) - 1);
        two &= two - 1;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          x[i][k] = __ldcg(reinterpret_cast<const float4*>(w.recs + at(k) * HD) + lane);
          ml[i][k] = __ldcg(w.rec_ml + at(k));
        }
      }
      unsigned left = these;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (left == two) break;
        Joined j{make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.f};
        j.raise(fmaxf(ml[i][0].x, ml[i][1].x));
        j.add(x[i][0], ml[i][0]);
        j.add(x[i][1], ml[i][1]);
        write_row(a, size_t(r0 + int64_t(__ffs(left) - 1) * warps), j, lane);
        left &= left - 1;
      }
    }
    for (; more; more &= more - 1) {
      look(__ffs(more) - 1);
      Joined j{make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.f};
      for (int k0 = 0; k0 < n; k0 += kListedFlight) join_parts<kListedFlight>(j, w.recs, w.rec_ml, k0, n, lane, at);
      write_row(a, row, j, lane);
    }
  }
}

std::mutex g_attr_mutex;
bool g_attr_set[64] = {};

// Lets the kernels take their dynamic shared memory on the current device.
cb_status allow_shared_memory() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
    return fail(CB_ERR_UNSUPPORTED, "8-bit attention: no usable current device");
  std::lock_guard<std::mutex> lock(g_attr_mutex);
  if (g_attr_set[dev]) return CB_OK;
  cudaError_t e = cudaSuccess;
  const auto allow = [&e](const void* kernel, uint32_t bytes) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
  };
  allow(reinterpret_cast<const void*>(q8_step_kernel<SharesShape, false>), SharesShape::kSmem);
  allow(reinterpret_cast<const void*>(q8_step_kernel<FewShape, true>), FewShape::kSmem);
  allow(reinterpret_cast<const void*>(q8_step_kernel<WideShape, false>), WideShape::kSmem);
  allow(reinterpret_cast<const void*>(q8_step_kernel<WideShape, true>), WideShape::kSmem);
  allow(reinterpret_cast<const void*>(q8_streams_kernel<FewShape>), FewShape::kSmem);
  allow(reinterpret_cast<const void*>(q8_streams_kernel<WideShape>), WideShape::kSmem);
  allow(reinterpret_cast<const void*>(q8_pieces_kernel), qpieces::kSmemBytes);
  if (e != cudaSuccess) return cuda_fail(e, "8-bit attention: shared memory attribute");
  g_attr_set[dev] = true;
  return CB_OK;
}

// The tensor maps of the K and V pools: boxes of `rows` rows of one block and head.
cb_status encode_pools(const AttnArgs& a, int rows, CUtensorMap* tk, CUtensorMap* tv) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return CB_ERR_CUDA;
  const cuuint64_t B = cuuint64_t(a.block_size), boxes = cuuint64_t(a.num_blocks) * a.num_kv_heads;
  const cuuint64_t dims[3] = {HD, B, boxes}, strides[2] = {HD, B * HD};
  const cuuint32_t box[3] = {HD, cuuint32_t(rows), 1}, ones[3] = {1, 1, 1};
  for (int v = 0; v < 2; ++v) {
    const CUresult r = enc(v ? tv : tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(v ? a.v_pool : a.k_pool), dims, strides,
                           box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(CB_ERR_CUDA, "8-bit attention: encoding the KV tensor maps failed (%d)", int(r));
  }
  return CB_OK;
}

// Sets of 8 query rows of a stream's units.
int stream_sets(const AttnArgs& a) { return int64_t(a.max_q_len) * (a.num_heads / a.num_kv_heads) <= 8 ? 1 : 2; }
// Of a listed step's, whose sequences may have more rows than one unit: small units, of up to 8 rows, where one token's rows
// fit them.  600 rows at 2000 keys, 32 heads on 4 and on 2, us: units of 8 rows 152, 131, of 16 179, 116.
int listed_sets(int group_heads) { return group_heads <= 8 ? 1 : 2; }
int listed_warps(int sets) { return sets == 1 ? FewShape::kWarps : WideShape::kWarps; }

// Records of a step without a plan kernel: two of a row tile for each warp that may have a share.
size_t step_records(int num_sms) {
  return size_t(num_sms) * std::max({2 * SharesShape::kWarps * SharesShape::kRows, 2 * FewShape::kWarps * FewShape::kRows,
                                     2 * WideShape::kWarps * WideShape::kRows});
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }
size_t step_workspace_bytes(int32_t num_tokens) {
  return 256 + align256(size_t(num_tokens) * 16) + align256(step_records(kMaxSms) * kPrefixRecBytes);
}
PrefixSizes listed_sizes(int32_t num_q_heads, int32_t num_kv_heads, int32_t num_seqs, int32_t num_tokens, int32_t num_groups,
                         int32_t max_context_len) {
  const int sets = listed_sets(num_q_heads / num_kv_heads);
  return prefix_sizes(num_q_heads, num_kv_heads, num_seqs, num_tokens, num_groups, max_context_len, listed_warps(sets), 8 * sets);
}

cb_status run_step(const AttnArgs& a, const int32_t* cu_groups, const int32_t* prefix_lens, int32_t num_groups, void* workspace,
                   cudaStream_t stream) {
  const int sets = stream_sets(a), sms = std::min(sm_count(), kMaxSms);
  StepWork w;
  w.cu_groups = cu_groups;
  w.prefix_lens = prefix_lens;
  w.num_groups = num_groups;
  const int64_t streams = int64_t(a.num_seqs) * a.num_kv_heads *
                          ((int64_t(a.max_q_len) * (a.num_heads / a.num_kv_heads) + 8 * sets - 1) / (8 * sets));
  const bool apart = streams <= sms && num_groups <= (sets == 1 ? FewShape::kThreads : WideShape::kThreads) &&
                     a.max_context_len <= kApartTiles * qstream::kTileKeys * listed_warps(sets);
  char* p = static_cast<char*>(workspace);
  w.header = reinterpret_cast<int32_t*>(p);
  w.token_info = reinterpret_cast<int4*>(p + 256);
  w.recs = reinterpret_cast<float*>(p + 256 + align256(size_t(a.num_tokens) * 16));
  w.rec_ml = reinterpret_cast<float2*>(w.recs + step_records(kMaxSms) * HD);
  CUtensorMap tk, tv;
  cb_status st = encode_pools(a, qstream::kTileKeys, &tk, &tv);
  if (st == CB_OK) st = allow_shared_memory();
  if (st != CB_OK) return st;
  cudaError_t e;
  if (sets == 1 && !apart)
    e = launch_kernel(q8_step_kernel<SharesShape, false>, dim3(unsigned(sms)), dim3(SharesShape::kThreads), SharesShape::kSmem,
                      stream, true, tk, tv, a, w);
  else if (sets == 1)
    e = launch_kernel(q8_step_kernel<FewShape, true>, dim3(unsigned(streams)), dim3(FewShape::kThreads), FewShape::kSmem, stream,
                      true, tk, tv, a, w);
  else
    e = launch_kernel(apart ? q8_step_kernel<WideShape, true> : q8_step_kernel<WideShape, false>,
                      dim3(unsigned(apart ? streams : sms)), dim3(WideShape::kThreads), WideShape::kSmem, stream, true, tk, tv, a, w);
  if (e != cudaSuccess) return cuda_fail(e, "8-bit attention: launch");
  if (apart) return CB_OK;
  const int64_t rows = int64_t(a.num_tokens) * a.num_heads;
  const int row_tile = 8 * sets;
  if (rows <= int64_t(sms) * 4)
    e = launch_kernel(q8_join_kernel<true>, dim3(unsigned(rows)), dim3(kJoinThreads), 0, stream, true, a, w, row_tile);
  else
    e = launch_kernel(q8_join_kernel<false>, dim3(unsigned(std::min<int64_t>((rows + kJoinWarps - 1) / kJoinWarps, int64_t(sms) * 8))),
                      dim3(kJoinThreads), 0, stream, true, a, w, row_tile);
  return e == cudaSuccess ? CB_OK : cuda_fail(e, "8-bit attention: join launch");
}

}  // namespace

size_t quant_attention_workspace_bytes(int32_t num_q_heads, int32_t num_kv_heads, int32_t num_seqs, int32_t num_tokens,
                                       int32_t num_groups, int32_t max_context_len) {
  return std::max(step_workspace_bytes(num_tokens), prefix_workspace_bytes(listed_sizes(num_q_heads, num_kv_heads, num_seqs,
                                                                                        num_tokens, num_groups, max_context_len)));
}

cb_status run_quant_attention(const AttnArgs& a, const int32_t* cu_groups, const int32_t* prefix_lens, int32_t num_groups,
                              void* workspace, cudaStream_t stream) {
  NvtxRange nvtx("cb.ragged_attention_q8");
  if (int64_t(a.num_blocks) * a.num_kv_heads >= (int64_t(1) << 31))
    return fail(CB_ERR_UNSUPPORTED, "8-bit attention: num_blocks * num_kv_heads must fit in int32");
  const int G = a.num_heads / a.num_kv_heads, sets = stream_sets(a), threads = sets == 1 ? SharesShape::kThreads : WideShape::kThreads;
  const int64_t rows = int64_t(a.max_q_len) * G, row_tiles = (rows + 8 * sets - 1) / (8 * sets);
  const int64_t tiles = (int64_t(a.max_context_len) + qstream::kTileKeys - 1) / qstream::kTileKeys;
  const float key_bytes = 2.0f * HD * float(a.num_kv_heads);
  // sequences that may share (all but one of each group), and what sharing may save
  const double saved = num_groups == 0 ? 0.0 : double(a.num_seqs - num_groups) * double(a.max_context_len) * key_bytes;
  const bool fits = a.num_seqs <= threads && num_groups <= threads && a.num_tokens <= kStepTokens &&
                    (a.max_q_len == 1 || rows <= kMaxStreamRows) && saved <= kSharingBytes &&
                    double(tiles) * double(row_tiles) * a.num_kv_heads * a.num_seqs < double(1 << 30);
  if (fits) return run_step(a, cu_groups, prefix_lens, num_groups, workspace, stream);

  const PrefixSizes z = listed_sizes(a.num_heads, a.num_kv_heads, a.num_seqs, a.num_tokens, num_groups, a.max_context_len);
  PrefixWork w;
  const int lsets = listed_sets(G);
  cb_status st = prefix_work(a, cu_groups, prefix_lens, num_groups, z, listed_warps(lsets), 8 * lsets, workspace, &w);
  if (st != CB_OK) return st;
  w.key_bytes = key_bytes;
  w.tile_us_two = kTileUsTwo;
  w.tile_us_one = kTileUsOne;
  w.stream_rate = kStreamBytesPerUsPerSm;
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return CB_ERR_CUDA;
  CUtensorMap tq, tk64, tv64, tk16, tv16;
  // q as [tokens][heads][128]: a box is one key/value head's query heads of tile_tokens tokens, one 64-dim half
  const cuuint64_t dims[3] = {cuuint64_t(HD), cuuint64_t(a.num_heads), cuuint64_t(a.num_tokens)};
  const cuuint64_t strides[2] = {cuuint64_t(HD) * 2, cuuint64_t(a.num_heads) * HD * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(G), cuuint32_t(w.tile_tokens)}, ones[3] = {1, 1, 1};
  const CUresult r = enc(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides, box, ones,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(CB_ERR_CUDA, "8-bit attention: encoding the Q tensor map failed (%d)", int(r));
  st = encode_pools(a, std::min(a.block_size, qpieces::HN), &tk64, &tv64);
  if (st == CB_OK) st = encode_pools(a, qstream::kTileKeys, &tk16, &tv16);
  if (st == CB_OK) st = allow_shared_memory();
  if (st == CB_OK) st = launch_prefix_plan(a, w, stream);
  if (st != CB_OK) return st;
  const bool pieces = num_groups > 0 || (a.max_q_len > 1 && rows > kMaxStreamRows);
  cudaError_t e = cudaSuccess;
  if (pieces)
    e = launch_kernel(q8_pieces_kernel, dim3(unsigned(w.num_sms)), dim3(qpieces::kThreads), qpieces::kSmemBytes, stream, true, tq, tk64,
                      tv64, a, w);
  if (e == cudaSuccess)
    e = lsets == 1 ? launch_kernel(q8_streams_kernel<FewShape>, dim3(unsigned(w.num_sms)), dim3(FewShape::kThreads), FewShape::kSmem,
                                   stream, true, tk16, tv16, a, w, pieces ? 0 : 1)
                   : launch_kernel(q8_streams_kernel<WideShape>, dim3(unsigned(w.num_sms)), dim3(WideShape::kThreads), WideShape::kSmem,
                                   stream, true, tk16, tv16, a, w, pieces ? 0 : 1);
  if (e != cudaSuccess) return cuda_fail(e, "8-bit attention: launch");
  const int64_t rows_all = int64_t(a.num_tokens) * a.num_heads;
  if (rows_all <= int64_t(w.num_sms) * 4) return launch_prefix_join(a, w, stream);
  e = launch_kernel(q8_listed_join_kernel,
                    dim3(unsigned(std::min<int64_t>((rows_all + kJoinWarps - 1) / kJoinWarps, int64_t(w.num_sms) * kListedCtasPerSm))),
                    dim3(kJoinThreads), 0, stream, true, a, w);
  return e == cudaSuccess ? CB_OK : cuda_fail(e, "8-bit attention: join launch");
}

}  // namespace cb
