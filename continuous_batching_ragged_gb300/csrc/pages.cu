// Page operations of the paged cache: cb_fork_sequences and cb_compact_blocks.
//
// Both move whole rows of pages and nothing else, so both are bound by HBM:
// each byte that has to move is read once and written once, 16 bytes a thread,
// several loads in flight.  A page of one layer is num_heads * block_size *
// head_dim contiguous elements of the K and of the V pool.
// 256 forks over 16 layers: 47.5 us, 5.4 TB/s, most of it writes of parts of pages.
// 2,500 pages of 6 layers moved in a pool of 10,240: 317 us, 6.2 TB/s, of which the plan 15.
#include <algorithm>
#include <mutex>

#include "device_common.cuh"
#include "runtime.h"

namespace {

constexpr int kMaxLayers = 128;        // layers per launch; more take several launches
constexpr int kThreads = 256;
constexpr int kVec = 8;                // 16-byte loads in flight per thread
constexpr int kMaxForks = 1 << 16;     // every fork's CTA checks it against all others: so many take 21 ms

// The K and V pools of up to kMaxLayers layers: p[2 * layer] and p[2 * layer + 1].
struct Pools {
  uint4* p[2 * kMaxLayers];
};

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ------------------------------------------------------------------ fork

struct ForkArgs {
  int32_t* block_tables;
  int32_t* context_lens;
  const int32_t *parents, *children, *new_blocks;
  int32_t table_rows, max_blocks_per_seq, num_forks, num_blocks, num_heads, block_size;
  int32_t row_chunks;                  // 16-byte chunks of one (token, head) row
  int32_t num_pools;                   // 2 * layers
  unsigned* err;
};

// A fork's own description: what its parent holds.
struct Fork {
  int parent, child, len, full, part, src, dst;   // src, dst: the copied page (-1: none)
  unsigned bad;                                   // error bits
};

__device__ __forceinline__ Fork read_fork(const ForkArgs& a, int f) {
  Fork k;
  k.parent = a.parents[f];
  k.child = a.children[f];
  k.src = k.dst = -1;
  k.len = k.full = k.part = 0;
  k.bad = 0;
  if (k.parent < 0 || k.parent >= a.table_rows || k.child < 0 || k.child >= a.table_rows) {
    k.bad = cb::kErrInvalid;
    return k;
  }
  k.len = a.context_lens[k.parent];
  if (k.len < 0 || k.len > int64_t(a.max_blocks_per_seq) * a.block_size) {
    k.bad = cb::kErrInvalid;
    return k;
  }
  k.full = k.len / a.block_size;
  k.part = k.len - k.full * a.block_size;
  if (k.part > 0) {
    k.src = a.block_tables[int64_t(k.parent) * a.max_blocks_per_seq + k.full];
    k.dst = a.new_blocks[f];
    if (k.src < 0 || k.src >= a.num_blocks || k.dst < 0 || k.dst >= a.num_blocks) {
      k.bad = cb::kErrBounds;
      k.src = k.dst = -1;
    }
  }
  return k;
}

// blockIdx.x = fork, blockIdx.y = a share of its layers' pools.  Every CTA
// checks its fork against all others first: a child row that is also a parent
// or another fork's child, or a new page that another fork writes or copies
// from, would make the result depend on who runs first, so such a fork is
// left out.  That is quadratic in the forks (kMaxForks).  What the check reads
// (parents' rows and lengths) is written by no fork that passes it.
__global__ void __launch_bounds__(kThreads) fork_kernel(const ForkArgs a, const Pools pools) {
  const int f = blockIdx.x;
  grid_dependency_wait();              // it may start while the stream's last kernel ends
  const Fork me = read_fork(a, f);
  unsigned bad = me.bad;
  if (!bad) {
    for (int g = threadIdx.x; g < a.num_forks; g += kThreads) {
      const Fork o = read_fork(a, g);
      if (me.child == o.parent || (g != f && me.child == o.child)) bad |= cb::kErrInvalid;
      if (me.dst >= 0 && (me.dst == o.src || (g != f && me.dst == o.dst))) bad |= cb::kErrInvalid;
    }
  }
  bad = __syncthreads_or(int(bad)) ? (bad | cb::kErrInvalid) : 0u;
  if (me.bad) bad = me.bad;
  if (bad) {
    if (threadIdx.x == 0 && blockIdx.y == 0) cb::raise_error(a.err, bad);
    return;
  }
  if (blockIdx.y == 0) {
    const int32_t* from = a.block_tables + int64_t(me.parent) * a.max_blocks_per_seq;
    int32_t* to = a.block_tables + int64_t(me.child) * a.max_blocks_per_seq;
    for (int i = threadIdx.x; i < a.max_blocks_per_seq; i += kThreads)
      to[i] = i < me.full ? from[i] : (i == me.full && me.part > 0 ? me.dst : -1);
    if (threadIdx.x == 0) a.context_lens[me.child] = me.len;
  }
  if (me.part == 0) return;
  // The page's first `part` rows of every head, in every pool of this share: a
  // head's are contiguous, and a warp takes a head, or a part of one where there
  // are fewer heads than warps, kVec loads in flight per lane.
  const int head_chunks = a.block_size * a.row_chunks;     // one head's page
  const int used = me.part * a.row_chunks;                 // of which are copied
  const int64_t page = int64_t(a.num_heads) * head_chunks;
  constexpr int kWarps = kThreads / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int parts = a.num_heads >= kWarps ? 1 : kWarps / a.num_heads, len = (used + parts - 1) / parts;
  for (int j = blockIdx.y; j < a.num_pools; j += gridDim.y) {
    for (int item = warp; item < a.num_heads * parts; item += kWarps) {
      const int h = item / parts, begin = (item - h * parts) * len, end = min(used, begin + len);
      const uint4* src = pools.p[j] + me.src * page + int64_t(h) * head_chunks;
      uint4* dst = pools.p[j] + me.dst * page + int64_t(h) * head_chunks;
      for (int i0 = begin + lane; i0 < end; i0 += 32 * kVec) {
        uint4 v[kVec];
#pragma unroll
        for (int k = 0; k < kVec; ++k)
          if (i0 + 32 * k < end) v[k] = src[i0 + 32 * k];
#pragma unroll
        for (int k = 0; k < kVec; ++k)
          if (i0 + 32 * k < end) dst[i0 + 32 * k] = v[k];
      }
    }
  }
}

// ------------------------------------------------------------------ compact

constexpr int kPlanThreads = 1024;
constexpr int kMaxBlocks = 1 << 20;    // the plan's bitmap of live pages stays in shared memory (128 KB)

struct CompactArgs {
  const int32_t *block_tables, *context_lens;
  int32_t *new_tables, *remap, *num_live;
  int32_t num_seqs, max_blocks_per_seq, num_blocks, block_size;
  int64_t page_chunks;                 // 16-byte chunks of a page in one pool
  int32_t num_pools;
  // workspace
  int32_t* header;                     // [0] live pages (-1: bad metadata, do nothing), [1] moves
  uint32_t* live;                      // bitmap, one word per 32 pages
  int32_t* before;                     // live pages before each word
  int32_t *holes, *movers;             // the k-th mover goes to the k-th hole
  unsigned* err;
};

__device__ __forceinline__ int block_sum_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = lane < kPlanThreads / 32 ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  total = warp_sums[kPlanThreads / 32 - 1];
  const int r = (warp == 0 ? 0 : warp_sums[warp - 1]) + x - v;
  __syncthreads();
  return r;
}

// One CTA: marks the pages that some table uses, counts them (n), and pairs
// the k-th live page at or above n with the k-th free page below it.  There
// are as many of the one as of the other, and no page is on both sides, so
// the moves need no order.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const CompactArgs a) {
  grid_dependency_wait();              // it may start while the stream's last kernel ends
  launch_dependents();                 // they wait for this grid on the device
  extern __shared__ uint32_t bits[];
  __shared__ int warp_sums[32];
  const int tid = threadIdx.x;
  const int words = (a.num_blocks + 31) / 32;
  for (int i = tid; i < words; i += kPlanThreads) bits[i] = 0;
  __syncthreads();
  // 32 threads to a sequence, kMark pages of it in flight per thread
  constexpr int kMark = 4;
  const int B = a.block_size, W = a.max_blocks_per_seq, lane = tid & 31;
  unsigned bad = 0;
  for (int s = tid >> 5; s < a.num_seqs; s += kPlanThreads / 32) {
    const int ctx = a.context_lens[s];
    if (ctx < 0 || ctx > int64_t(W) * B) {
      bad |= cb::kErrInvalid;
      continue;
    }
    const int used = int((int64_t(ctx) + B - 1) / B);
    const int32_t* row = a.block_tables + int64_t(s) * W;
    for (int b0 = lane; b0 < used; b0 += 32 * kMark) {
      int blk[kMark];
#pragma unroll
      for (int k = 0; k < kMark; ++k) blk[k] = b0 + 32 * k < used ? row[b0 + 32 * k] : 0;
#pragma unroll
      for (int k = 0; k < kMark; ++k) {
        if (b0 + 32 * k >= used) break;
        if (blk[k] < 0 || blk[k] >= a.num_blocks)
          bad |= cb::kErrBounds;
        else
          atomicOr(&bits[blk[k] >> 5], 1u << (blk[k] & 31));
      }
    }
  }
  if (bad) cb::raise_error(a.err, bad);
  if (__syncthreads_or(int(bad))) {
    if (tid == 0) a.header[0] = -1, a.header[1] = 0;
    return;
  }
  const int per = (words + kPlanThreads - 1) / kPlanThreads, w0 = min(words, tid * per), w1 = min(words, w0 + per);
  int mine = 0, n;
  for (int w = w0; w < w1; ++w) mine += __popc(bits[w]);
  const int base = block_sum_scan(mine, warp_sums, n);
  // live pages below id n: the rank of the first mover
  int below = 0, low;
  for (int w = w0; w < w1; ++w) {
    const int first = w * 32;
    const uint32_t m = first + 32 <= n ? 0xffffffffu : (first >= n ? 0u : (1u << (n - first)) - 1u);
    below += __popc(bits[w] & m);
  }
  block_sum_scan(below, warp_sums, low);
  int run = base;
  for (int w = w0; w < w1; ++w) {
    const uint32_t word = bits[w];
    a.live[w] = word;
    a.before[w] = run;
    int seen = run;                    // live pages below id
    for (int b = 0; b < 32; ++b) {
      const int id = w * 32 + b;
      if (id >= a.num_blocks) break;
      const bool live = (word >> b) & 1u;
      if (live && id >= n) a.movers[seen - low] = id;
      if (!live && id < n) a.holes[id - seen] = id;
      seen += live;
    }
    run = seen;
  }
  if (tid == 0) {
    a.header[0] = n;
    a.header[1] = n - low;
    a.header[2] = low;
  }
}

constexpr int kMoveCtasPerSm = 3;    // 200 pages of 2 layers: 8.9 us with the plan, at 8 CTAs 13.0; 10,240 pages 317 and 315

// Moves the pages and rewrites the tables, from the plan's lists.
__global__ void __launch_bounds__(kThreads) compact_move_kernel(const CompactArgs a, const Pools pools, int first) {
  grid_dependency_wait();              // the plan has finished
  const int n = __ldcg(a.header), moves = __ldcg(a.header + 1), low = __ldcg(a.header + 2);
  if (n < 0) {
    if (first && blockIdx.x == 0 && threadIdx.x == 0) *a.num_live = n;
    return;
  }
  // a unit is kThreads * kVec chunks of one page of one pool
  const int64_t per_page = (a.page_chunks + kThreads * kVec - 1) / (kThreads * kVec);
  const int64_t units = int64_t(moves) * a.num_pools * per_page;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t part = u % per_page, rest = u / per_page;
    const int pool = int(rest % a.num_pools), mv = int(rest / a.num_pools);
    const uint4* src = pools.p[pool] + __ldcg(a.movers + mv) * a.page_chunks;
    uint4* dst = pools.p[pool] + __ldcg(a.holes + mv) * a.page_chunks;
    const int64_t i0 = part * (kThreads * kVec) + threadIdx.x;
    uint4 v[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k)
      if (i0 + k * kThreads < a.page_chunks) v[k] = cb::ldg_stream(src + i0 + k * kThreads);
#pragma unroll
    for (int k = 0; k < kVec; ++k)
      if (i0 + k * kThreads < a.page_chunks) dst[i0 + k * kThreads] = v[k];
  }
  if (!first) return;
  // the tables, from the last CTA backwards: where there are few pages to move, the first ones move them
  const int64_t gtid = int64_t(gridDim.x - 1 - blockIdx.x) * kThreads + threadIdx.x, gsize = int64_t(gridDim.x) * kThreads;
  if (gtid == 0) *a.num_live = n;
  auto where = [&](int id) -> int {
    const uint32_t word = __ldcg(a.live + (id >> 5));
    if (!((word >> (id & 31)) & 1u)) return -1;
    if (id < n) return id;
    return __ldcg(a.holes + (__ldcg(a.before + (id >> 5)) + __popc(word & ((1u << (id & 31)) - 1u)) - low));
  };
  for (int64_t i = gtid; i < a.num_blocks; i += gsize) a.remap[i] = where(int(i));
  const int W = a.max_blocks_per_seq;
  const int64_t entries = int64_t(a.num_seqs) * W;
  for (int64_t i = gtid; i < entries; i += gsize) {
    const int s = int(i / W), b = int(i - int64_t(s) * W);
    a.new_tables[i] = int64_t(b) * a.block_size < a.context_lens[s] ? where(a.block_tables[i]) : -1;
  }
}

// Checks that the layers are alike and gives 16-byte chunks per row.
cb_status check_layers(const char* who, const cb_kv_cache* layers, int32_t num_layers, int32_t* row_chunks) {
  if (num_layers < 1) return cb::fail(CB_ERR_INVALID, "%s: num_layers < 1", who);
  if (!layers) return cb::fail(CB_ERR_INVALID, "%s: null layers", who);
  const cb_kv_cache& c = layers[0];
  if (c.num_blocks < 1 || c.block_size < 1 || c.num_heads < 1 || c.head_dim < 1)
    return cb::fail(CB_ERR_INVALID, "%s: cache dimensions must be >= 1", who);
  if (c.dtype != CB_DTYPE_BF16 && c.dtype != CB_DTYPE_F32) return cb::fail(CB_ERR_UNSUPPORTED, "%s: unknown dtype", who);
  const int64_t row = int64_t(c.head_dim) * (c.dtype == CB_DTYPE_BF16 ? 2 : 4);
  if (row % 16 != 0)
    return cb::fail(CB_ERR_UNSUPPORTED, "%s: head_dim * element size must be a multiple of 16", who);
  if (row / 16 * c.block_size > 0x7FFFFFFF / c.num_heads)
    return cb::fail(CB_ERR_UNSUPPORTED, "%s: pages too large", who);
  for (int32_t i = 0; i < num_layers; ++i) {
    const cb_kv_cache& l = layers[i];
    if (l.num_blocks != c.num_blocks || l.block_size != c.block_size || l.num_heads != c.num_heads ||
        l.head_dim != c.head_dim || l.dtype != c.dtype)
      return cb::fail(CB_ERR_INVALID, "%s: layer %d has another shape or dtype than layer 0", who, i);
    if (!l.k || !l.v) return cb::fail(CB_ERR_INVALID, "%s: null pool in layer %d", who, i);
    if ((reinterpret_cast<uintptr_t>(l.k) | reinterpret_cast<uintptr_t>(l.v)) % 16 != 0)
      return cb::fail(CB_ERR_INVALID, "%s: pools must be 16-byte aligned", who);
  }
  *row_chunks = int32_t(row / 16);
  return CB_OK;
}

int fill_pools(const cb_kv_cache* layers, int32_t first, int32_t num_layers, Pools* pools) {
  const int n = std::min(num_layers - first, kMaxLayers);
  for (int i = 0; i < n; ++i) {
    pools->p[2 * i] = static_cast<uint4*>(layers[first + i].k);
    pools->p[2 * i + 1] = static_cast<uint4*>(layers[first + i].v);
  }
  return n;
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

extern "C" cb_status cb_fork_sequences(const cb_kv_cache* layers, int32_t num_layers, int32_t* block_tables,
                                       int32_t* context_lens, int32_t table_rows, int32_t max_blocks_per_seq,
                                       const int32_t* parents, const int32_t* children, const int32_t* new_blocks,
                                       int32_t num_forks, void* stream) {
  const char* who = "cb_fork_sequences";
  cb::NvtxRange nvtx("cb.fork_sequences");
  int32_t row_chunks = 0;
  cb_status st = check_layers(who, layers, num_layers, &row_chunks);
  if (st != CB_OK) return st;
  if (num_forks < 0 || table_rows < 0 || max_blocks_per_seq < 0) return cb::fail(CB_ERR_INVALID, "%s: negative size", who);
  if (num_forks > kMaxForks) return cb::fail(CB_ERR_UNSUPPORTED, "%s: more than %d forks", who, kMaxForks);
  if (num_forks == 0) return CB_OK;
  if (!block_tables || !context_lens || !parents || !children || !new_blocks)
    return cb::fail(CB_ERR_INVALID, "%s: null pointer", who);
  unsigned* err = cb::device_error_word();
  if (!err) return CB_ERR_CUDA;
  ForkArgs a;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.parents = parents;
  a.children = children;
  a.new_blocks = new_blocks;
  a.table_rows = table_rows;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.num_forks = num_forks;
  a.num_blocks = layers[0].num_blocks;
  a.num_heads = layers[0].num_heads;
  a.block_size = layers[0].block_size;
  a.row_chunks = row_chunks;
  a.err = err;
  for (int32_t first = 0; first < num_layers; first += kMaxLayers) {
    Pools pools;
    a.num_pools = 2 * fill_pools(layers, first, num_layers, &pools);
    // 16 CTAs an SM in all: 256 forks over 16 layers took 47.7 us, at 4, 8 and 32 CTAs 55.9, 51.3 and 49.5
    const int64_t want = (int64_t(cb::sm_count()) * 16 + num_forks - 1) / num_forks;
    const unsigned y = unsigned(std::max<int64_t>(1, std::min<int64_t>(a.num_pools, want)));
    cudaError_t e = cb::launch_kernel(fork_kernel, dim3(unsigned(num_forks), y), dim3(kThreads), 0,
                                      static_cast<cudaStream_t>(stream), true, a, pools);
    if (e != cudaSuccess) return cb::cuda_fail(e, "fork: launch");
  }
  return CB_OK;
}

extern "C" size_t cb_compact_workspace_size(int32_t num_blocks) {
  if (num_blocks < 1) return 0;
  const size_t words = (size_t(num_blocks) + 31) / 32, half = size_t(num_blocks) / 2 + 1;
  return 256 + 2 * align256(words * 4) + 2 * align256(half * 4);
}

extern "C" cb_status cb_compact_blocks(const cb_kv_cache* layers, int32_t num_layers, const int32_t* block_tables,
                                       const int32_t* context_lens, int32_t num_seqs, int32_t max_blocks_per_seq,
                                       int32_t* new_block_tables, int32_t* remap, int32_t* num_live, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  const char* who = "cb_compact_blocks";
  cb::NvtxRange nvtx("cb.compact_blocks");
  int32_t row_chunks = 0;
  cb_status st = check_layers(who, layers, num_layers, &row_chunks);
  if (st != CB_OK) return st;
  const cb_kv_cache& c = layers[0];
  if (num_seqs < 0 || max_blocks_per_seq < 0) return cb::fail(CB_ERR_INVALID, "%s: negative size", who);
  if (c.num_blocks > kMaxBlocks)
    return cb::fail(CB_ERR_UNSUPPORTED, "%s: pools of more than %d blocks", who, kMaxBlocks);
  const bool some = num_seqs > 0 && max_blocks_per_seq > 0;
  if (!remap || !num_live || (num_seqs > 0 && !context_lens) || (some && (!block_tables || !new_block_tables)))
    return cb::fail(CB_ERR_INVALID, "%s: null pointer", who);
  const size_t need = cb_compact_workspace_size(c.num_blocks);
  if (!workspace || workspace_bytes < need)
    return cb::fail(CB_ERR_INVALID, "%s: workspace too small: %zu bytes given, %zu needed", who, workspace_bytes, need);
  if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
    return cb::fail(CB_ERR_INVALID, "%s: workspace must be 256-byte aligned", who);
  unsigned* err = cb::device_error_word();
  if (!err) return CB_ERR_CUDA;
  const size_t words = (size_t(c.num_blocks) + 31) / 32, half = size_t(c.num_blocks) / 2 + 1;
  CompactArgs a;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.new_tables = new_block_tables;
  a.remap = remap;
  a.num_live = num_live;
  a.num_seqs = num_seqs;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.num_blocks = c.num_blocks;
  a.block_size = c.block_size;
  a.page_chunks = int64_t(c.num_heads) * c.block_size * row_chunks;
  char* w = static_cast<char*>(workspace);
  a.header = reinterpret_cast<int32_t*>(w);
  w += 256;
  a.live = reinterpret_cast<uint32_t*>(w);
  w += align256(words * 4);
  a.before = reinterpret_cast<int32_t*>(w);
  w += align256(words * 4);
  a.holes = reinterpret_cast<int32_t*>(w);
  w += align256(half * 4);
  a.movers = reinterpret_cast<int32_t*>(w);
  a.err = err;
  const size_t smem = words * 4;
  if (smem > 48 * 1024 - 256) {
    static std::mutex mu;
    static bool ready[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return cb::fail(CB_ERR_CUDA, "%s: no usable current device", who);
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev]) {
      e = cudaFuncSetAttribute(compact_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxBlocks / 8);
      if (e != cudaSuccess) return cb::cuda_fail(e, "compact: shared memory attribute");
      ready[dev] = true;
    }
  }
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e = cb::launch_kernel(compact_plan_kernel, dim3(1), dim3(kPlanThreads), smem, cs, true, a);
  if (e != cudaSuccess) return cb::cuda_fail(e, "compact: plan launch");
  for (int32_t first = 0; first < num_layers; first += kMaxLayers) {
    Pools pools;
    a.num_pools = 2 * fill_pools(layers, first, num_layers, &pools);
    e = cb::launch_kernel(compact_move_kernel, dim3(unsigned(cb::sm_count() * kMoveCtasPerSm)), dim3(kThreads), 0, cs, first == 0, a,
                          pools, first == 0 ? 1 : 0);
    if (e != cudaSuccess) return cb::cuda_fail(e, "compact: move launch");
  }
  return CB_OK;
}
