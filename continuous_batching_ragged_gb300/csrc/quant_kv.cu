// The paged cache in 8 bits: e4m3 pages with a fp32 scale for each page and head.
//
// cb_append_kv_q8 writes a step's keys and values.  For each page that gets
// tokens and each head,
//     need = 2^e, e the least integer (at least kLeastExp) with max |x| <= 448 * 2^e
//     s    = max(need, the page's scale) if the page held tokens before, else need
//     new tokens: RN(x / s);  tokens before them, where s grew: RN(old * s_old / s).
// Powers of two: dividing by s is exact, so every number is rounded once, by at
// most half a step (2^-4 of it), and a page that is scaled anew loses nothing but
// the last bits of its smallest numbers.  e4m3's steps are relative, so a finer
// scale would gain nothing but the range between 224 and 448 steps.  A kept scale of
// the caller's own may be no power of two: then quotients are cut off to fp32 with the
// last bit set where bits were cut off, and rounded once all the same, apart from the
// others.
//
// cb_gather_kv_q8 reads tokens back: q * s, in bf16 or fp32.
//
// What bounds them: a large read-back HBM, a third of it reads (24 sequences of 4096
// keys, 24 heads: 234 us, 0.82 of the copy rate, with scales that are no powers of two 244;
// 32-byte stores, more or fewer warps and loads in flight change nothing).  An append is bound
// by its dependent steps: slots, page and scale, rows, their maximum, stores.  2048 tokens of
// 32 heads take 22.1 us of 7.5 at the copy rate, 2.5 of them the scan of the slots; warps wait
// for loads half of the time and issue a third of it.  64 decode rows: 4.8 us in a graph, a
// launch.
#include <algorithm>

#include "device_common.cuh"
#include "e4m3.cuh"
#include "runtime.h"

namespace {

using cb::Vec16;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kLeastExp = -100;          // 448 * 2^-100 is beyond any key or value in use; 2^100 and 2^-100 are ordinary fp32 numbers
constexpr int kMaxTokens = 65536;        // of a call: their bits are kept in shared memory
constexpr int kPageBits = 65536;         // pages told apart at once where a step's runs are looked over for one that comes again
constexpr int kAppendCtasPerSm = 2;
constexpr int kGatherCtasPerSm = 4;

struct AppendArgs {
  const void *k_new, *v_new;
  int64_t k_stride, v_stride;            // 16-byte chunks between tokens
  const int64_t* slots;
  const int32_t* dims;
  uint8_t *k, *v;
  float *k_scale, *v_scale;
  int64_t num_slots;
  int32_t num_tokens, num_heads, num_blocks, block_shift;
  unsigned* err;
};

// The scale that numbers of up to `amax` need.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);            // 448 = 1.75 * 2^8
  const int e = int(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float(uint32_t(max(e, kLeastExp) + 127) << 23);
}

// The largest magnitude of a lane's numbers: NaN does not count, an infinity shows and is left out by a second pass.
template <typename T>
struct Largest;
template <>
struct Largest<__nv_bfloat16> {
  uint32_t m = 0;                                      // two numbers of any sign
  __device__ __forceinline__ void add(const uint4& x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
  }
  __device__ __forceinline__ void add_finite(const uint4& x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t y = w[i];
      if ((y & 0x7f80u) == 0x7f80u) y &= 0xffff0000u;
      if ((y & 0x7f800000u) == 0x7f800000u) y &= 0xffffu;
      asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(y));
    }
  }
  __device__ __forceinline__ float get() const {
    return fmaxf(__uint_as_float((m << 16) & 0x7fff0000u), __uint_as_float(m & 0x7fff0000u));
  }
};
template <>
struct Largest<float> {
  float m = 0.f;
  __device__ __forceinline__ void add(const uint4& x) {
    m = fmaxf(fmaxf(m, fabsf(__uint_as_float(x.x))), fabsf(__uint_as_float(x.y)));
    m = fmaxf(fmaxf(m, fabsf(__uint_as_float(x.z))), fabsf(__uint_as_float(x.w)));
  }
  __device__ __forceinline__ void add_finite(const uint4& x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((w[i] & 0x7f800000u) != 0x7f800000u) m = fmaxf(m, fabsf(__uint_as_float(w[i])));
  }
  __device__ __forceinline__ float get() const { return m; }
};

// x / s as e4m3, `inv` = 1 / s.  FINITE: no infinity among the numbers; else one becomes NaN, as x - x is where x is not finite.
template <bool FINITE>
__device__ __forceinline__ float scaled(float x, float inv) {
  const float y = x * inv;
  return FINITE ? y : y + (y - y);
}
template <bool FINITE>
__device__ __forceinline__ uint2 to_e4m3(const float (&x)[8], float inv) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = scaled<FINITE>(x[i], inv);
  return make_uint2(cb::float_to_e4m3x4(y[0], y[1], y[2], y[3]), cb::float_to_e4m3x4(y[4], y[5], y[6], y[7]));
}
template <bool FINITE>
__device__ __forceinline__ uint32_t to_e4m3(const float (&x)[4], float inv) {
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = scaled<FINITE>(x[i], inv);
  return cb::float_to_e4m3x4(y[0], y[1], y[2], y[3]);
}
// A row's lane of numbers, for a scale that is no power of two: x / s to odd, from the remainder of a quotient that is off by less
// than one step.  Numbers that are not finite become NaN.
template <int N>
__device__ __forceinline__ void store_quotients(uint8_t* to, const float (&x)[N], float s) {
  const float up = s < 0x1p-40f ? 0x1p60f : 1.0f;   // remainders that count are ordinary fp32 numbers, and exact
  const float su = s * up, inv = 1.0f / su;
  float y[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float xu = x[i] * up, q = xu * inv, near = fmaf(fmaf(-q, su, xu), inv, q);
    y[i] = cb::to_odd(near + (near - near), fmaf(-near, su, xu));
  }
#pragma unroll
  for (int i = 0; i < N; i += 4) reinterpret_cast<uint32_t*>(to)[i / 4] = cb::float_to_e4m3x4(y[i], y[i + 1], y[i + 2], y[i + 3]);
}
__device__ __forceinline__ void store_lane(uint8_t* row, int c, const uint2& v) { reinterpret_cast<uint2*>(row)[c] = v; }
__device__ __forceinline__ void store_lane(uint8_t* row, int c, uint32_t v) { reinterpret_cast<uint32_t*>(row)[c] = v; }

// The first n 16-byte chunks of a head's page, times `ratio`: by `lanes` lanes, of which this is `lane`.
__device__ __forceinline__ void rescale_rows(uint8_t* rows, int n, int lane, int lanes, float ratio) {
  if (!cb::is_power_of_two(ratio)) {             // from a scale of the caller's own
#pragma unroll 1
    for (int i = lane; i < 4 * n; i += lanes) {
      uint32_t* w = reinterpret_cast<uint32_t*>(rows) + i;
      float f[4];
      cb::e4m3x4_to_float(*w, f);
      *w = cb::float_to_e4m3x4(cb::product_to_odd(f[0], ratio), cb::product_to_odd(f[1], ratio), cb::product_to_odd(f[2], ratio),
                               cb::product_to_odd(f[3], ratio));
    }
    return;
  }
  for (int i = lane; i < n; i += lanes) {
    uint4 old = reinterpret_cast<uint4*>(rows)[i];
    uint32_t* w = &old.x;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float f[4];
      cb::e4m3x4_to_float(w[e], f);
      w[e] = cb::float_to_e4m3x4(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
    }
    reinterpret_cast<uint4*>(rows)[i] = old;
  }
}

// The tokens of one page follow one another in a step: a run.  A warp takes a run's
// rows of one head at a time, keys or values, LPR lanes to a row, and holds 32 rows in
// registers between the maximum and the rounding (longer runs are read again), or with
// pages of up to 16 tokens 16 rows of two heads.  A run of one token, as decode rows
// are, has four heads for each row that the warp holds side by side.  It goes on to as
// many heads of its run as there are for each warp of the grid, so that finding the
// run, its slots and offsets is paid for once.  Which tokens begin a run, every CTA finds out for
// itself from the slots, so that the warps of the whole grid share the runs evenly
// whatever mix of decode rows and chunks they come from.  Two runs of one page would
// scale its rows at the same time: each CTA marks the runs' pages, and those that were
// marked before, whose runs it leaves out; a pool of more pages than there are marks has
// several to a mark, whose runs are compared one by one.  (Of 2048 tokens of 32 heads, all
// else equal, the marks take 0.9 us; in a pass of their own 1.0, in one pass with a second
// where marks are fewer than runs 1.1.)
template <typename T, int LPR, bool LONG>
__global__ void __launch_bounds__(kThreads, kAppendCtasPerSm) append_q8_kernel(const AppendArgs a) {
  constexpr int EPV = Vec16<T>::N;               // elements per lane
  constexpr int A = LPR * EPV;                   // head_dim
  constexpr int RPW = 32 / LPR;                  // rows side by side in the warp
  constexpr int kSpan = LONG && LPR < 32 ? 32 : 16;   // positions that the warp holds at a time
  constexpr int kHeld = kSpan / RPW;             // rows of them a lane
  constexpr int kHeads = !LONG && LPR < 32 ? 2 : 1;   // heads (keys or values) at a time
  constexpr int kWords = kMaxTokens / 32;
  __shared__ uint32_t kept[kWords], lead[kWords], before[kWords + 1];   // tokens that are cached; that begin a run; runs before the word
  __shared__ uint32_t marked[kPageBits / 32], again[kPageBits / 32];    // pages that runs are of; that were marked before
  __shared__ uint32_t warp_sum[kWarps];
  for (int w = threadIdx.x; w < (min(a.num_blocks, kPageBits) + 31) / 32; w += kThreads) marked[w] = again[w] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // it may start while the stream's last kernel ends
  int n_tok = a.num_tokens;
  if (a.dims) {                                  // the step's token count, at most num_tokens (the capacity)
    const int32_t t = a.dims[1];
    if (t < 0 || t > a.num_tokens) {
      if (blockIdx.x == 0 && threadIdx.x == 0) cb::raise_error(a.err, cb::kErrInvalid);
      return;
    }
    n_tok = t;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int words = (n_tok + 31) / 32;
#pragma unroll 4
  for (int w = warp; w < words; w += kWarps) {
    const int t = 32 * w + lane;
    const int64_t slot = t < n_tok ? a.slots[t] : -1;
    if (slot >= a.num_slots && blockIdx.x == 0) cb::raise_error(a.err, cb::kErrBounds);
    const uint32_t m = __ballot_sync(0xffffffffu, slot >= 0 && slot < a.num_slots);
    if (lane == 0) kept[w] = m;
  }
  __syncthreads();
  // a kept token begins a run if the last kept one before it is of another page
#pragma unroll 4
  for (int w = warp; w < words; w += kWarps) {
    const int t = 32 * w + lane;
    const uint32_t mine = kept[w];
    bool is_lead = false;
    if (mine >> lane & 1) {
      uint32_t m = mine & ((1u << lane) - 1);
      int x = w;
      while (m == 0 && x > 0) m = kept[--x];
      const int64_t page = a.slots[t] >> a.block_shift;
      is_lead = m == 0 || (a.slots[32 * x + 31 - __clz(m)] >> a.block_shift) != page;
      if (is_lead) {
        const unsigned at = unsigned(page) % kPageBits, bit = 1u << (at & 31);
        if (atomicOr(&marked[at / 32], bit) & bit) atomicOr(&again[at / 32], bit);
      }
    }
    const uint32_t m = __ballot_sync(0xffffffffu, is_lead);
    if (lane == 0) lead[w] = m;
  }
  __syncthreads();
  // runs before each word
  const int per = (words + kThreads - 1) / kThreads;
  uint32_t mine = 0;
  for (int i = 0; i < per; ++i)
    if (tid * per + i < words) mine += __popc(lead[tid * per + i]);
  uint32_t x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  uint32_t at = x - mine, runs = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) at += warp_sum[i];
    runs += warp_sum[i];
  }
  for (int i = 0; i < per; ++i)
    if (tid * per + i < words) {
      before[tid * per + i] = at;
      at += __popc(lead[tid * per + i]);
    }
  __syncthreads();

  const int K = a.num_heads, B = 1 << a.block_shift;
  const int c = lane % LPR, r0 = lane / LPR;
  const unsigned warps = gridDim.x * kWarps, parts = unsigned(2 * K);
  // as few heads to a warp as leave no warp with a second run, where there are warps enough
  const unsigned most = runs == 0 ? parts : max(1u, min(parts, warps / runs));
  const unsigned per_warp = (parts + most - 1) / most, groups = (parts + per_warp - 1) / per_warp;
  for (unsigned u = blockIdx.x * kWarps + warp; u < runs * groups; u += warps) {
    const unsigned run = u / groups;
    const int part0 = int((u - run * groups) * per_warp), part1 = min(int(parts), part0 + int(per_warp));
    // the run's first token, and the next run's
    int lo = 0;
    for (int hi = words - 1; lo < hi;) {
      const int mid = (lo + hi + 1) >> 1;
      if (before[mid] <= run) lo = mid; else hi = mid - 1;
    }
    uint32_t m = lead[lo];
    for (unsigned i = before[lo]; i < run; ++i) m &= m - 1;
    const int t0 = 32 * lo + __ffs(m) - 1;
    m &= m - 1;
    int w1 = lo;
    while (m == 0 && ++w1 < words) m = lead[w1];
    int t1 = m ? 32 * w1 + __ffs(m) - 1 : n_tok;
    {                                              // behind the run's last kept token, whatever is skipped behind it
      int w = (t1 - 1) >> 5;
      uint32_t k = kept[w] & (0xffffffffu >> (31 - ((t1 - 1) & 31)));
      while (k == 0) k = kept[--w];                // it has t0 at least
      t1 = 32 * w + 32 - __clz(k);
    }
    const int64_t slot0 = a.slots[t0];
    const int64_t page = slot0 >> a.block_shift;
    const int first = int(slot0) & (B - 1);

    if (again[unsigned(page) % kPageBits / 32] >> (unsigned(page) & 31) & 1) {
      int of_page = 2;                             // runs; at least two
      if (a.num_blocks > kPageBits) {              // or of pages that have one mark
        of_page = 0;
        for (int w = lane; w < words; w += 32)
          for (uint32_t l = lead[w]; l; l &= l - 1) of_page += (a.slots[32 * w + __ffs(l) - 1] >> a.block_shift) == page;
        of_page = __reduce_add_sync(0xffffffffu, of_page);
      }
      if (of_page > 1) {                           // left out
        if (lane == 0 && part0 == 0) cb::raise_error(a.err, cb::kErrInvalid);
        continue;
      }
    }

    if (t1 - t0 == 1) {                            // one token: a head for each row of the warp, four times
      for (int q = part0; q < part1; q += 4 * RPW) {
        uint4 raw[4];
        float *scale[4], held[4];
        uint8_t* rows[4];
        bool mine[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int part = q + i * RPW + r0, h = part % K;
          const bool is_v = part >= K;
          mine[i] = part < part1;
          scale[i] = (is_v ? a.v_scale : a.k_scale) + page * K + h;
          rows[i] = (is_v ? a.v : a.k) + (page * K + h) * int64_t(B) * A;
          const uint4* src = static_cast<const uint4*>(is_v ? a.v_new : a.k_new) + int64_t(h) * LPR + c;
          raw[i] = mine[i] ? src[int64_t(t0) * (is_v ? a.v_stride : a.k_stride)] : make_uint4(0, 0, 0, 0);
          held[i] = mine[i] && first > 0 ? *scale[i] : 0.f;
        }
        unsigned odd = 0;                          // heads whose scale is no power of two, and so the one that they had
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float f[EPV];
          Vec16<T>::to_float(raw[i], f);
          Largest<T> top;
          top.add_finite(raw[i]);
          float amax = top.get();
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          const float s = fmaxf(scale_for(amax), held[i]), inv = 1.0f / s;
          if (!mine[i]) continue;
          if (!cb::is_power_of_two(s)) {
            odd |= 1u << i;
            continue;
          }
          if (first > 0 && s > held[i]) rescale_rows(rows[i], first * (A / 16), c, LPR, held[i] * inv);
          if (c == 0) *scale[i] = s;
          store_lane(rows[i] + first * A, c, to_e4m3<false>(f, inv));
        }
#pragma unroll 1
        for (; odd; odd &= odd - 1) {
          const int part = q + (__ffs(odd) - 1) * RPW + r0, h = part % K;
          const bool is_v = part >= K;
          float f[EPV];
          Vec16<T>::to_float((static_cast<const uint4*>(is_v ? a.v_new : a.k_new) + int64_t(h) * LPR + c)[int64_t(t0) * (is_v ? a.v_stride : a.k_stride)], f);
          store_quotients(static_cast<uint8_t*>(is_v ? a.v : a.k) + ((page * K + h) * int64_t(B) + first) * A + EPV * c, f,
                          (is_v ? a.v_scale : a.k_scale)[page * K + h]);
        }
      }
      continue;
    }

    // lane i's offset in the page, of position p + i of the run; -1 if its token is not cached
    auto offsets = [&](int p) -> int {
      const int t = t0 + p + lane;
      if (t >= t1 || lane >= kSpan) return -1;
      const int64_t s = a.slots[t];
      return s >= 0 && s < a.num_slots ? int(s) & (B - 1) : -1;
    };
    int offs = -1;
    {
      bool rising = true;
      int top = -1;
      for (int p = 0; t0 + p < t1; p += kSpan) {   // each kept token's offset has to be above all before it
        const int o = offsets(p);
        if (p == 0) offs = o;
        int upto = o;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, upto, d);
          if (lane >= d) upto = max(upto, y);
        }
        int prev = __shfl_up_sync(0xffffffffu, upto, 1);
        prev = lane == 0 ? top : max(prev, top);
        rising = rising && __all_sync(0xffffffffu, o < 0 || o > prev);
        top = max(top, __shfl_sync(0xffffffffu, upto, 31));
      }
      if (!rising) {                               // left out
        if (lane == 0 && part0 == 0) cb::raise_error(a.err, cb::kErrInvalid);
        continue;
      }
    }
    const bool held_all = t1 - t0 <= kSpan;

    for (int q = part0; q < part1; q += kHeads) {
      const int n = min(kHeads, part1 - q);
      const uint4* src[kHeads];
      int64_t stride[kHeads];
      float *scale[kHeads], held[kHeads], amax[kHeads];
      Largest<T> top[kHeads];
      uint8_t* rows[kHeads];
      uint4 raw[kHeads][kHeld];
#pragma unroll
      for (int v = 0; v < kHeads; ++v) {
        const int part = v < n ? q + v : q, h = part % K;
        const bool is_v = part >= K;
        src[v] = static_cast<const uint4*>(is_v ? a.v_new : a.k_new) + int64_t(h) * LPR + c;
        stride[v] = is_v ? a.v_stride : a.k_stride;
        scale[v] = (is_v ? a.v_scale : a.k_scale) + page * K + h;
        held[v] = first > 0 ? *scale[v] : 0.f;     // tokens before the first new one, with this scale
        rows[v] = (is_v ? a.v : a.k) + (page * K + h) * int64_t(B) * A;
      }
      // rows of positions p .. p + kSpan - 1 of the run
      auto load = [&](int p, int o16) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
          if (t0 + p + i * RPW >= t1) break;
          const int j = i * RPW + r0;
          const int o = __shfl_sync(0xffffffffu, o16, j);
#pragma unroll
          for (int v = 0; v < kHeads; ++v) raw[v][i] = o >= 0 && v < n ? src[v][int64_t(t0 + p + j) * stride[v]] : make_uint4(0, 0, 0, 0);
        }
      };
      for (int p = 0; t0 + p < t1; p += kSpan) {
        if (p > 0) offs = offsets(p);
        load(p, offs);
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
          if (t0 + p + i * RPW >= t1) break;
#pragma unroll
          for (int v = 0; v < kHeads; ++v) top[v].add(raw[v][i]);
        }
      }
      bool finite = true;
#pragma unroll
      for (int v = 0; v < kHeads; ++v) {
        amax[v] = top[v].get();
        finite = finite && amax[v] <= 3.402823466e38f;
      }
      finite = __all_sync(0xffffffffu, finite);
      if (!finite) {                               // rare: once more, without what is not finite
#pragma unroll
        for (int v = 0; v < kHeads; ++v) top[v] = Largest<T>();
        for (int p = 0; t0 + p < t1; p += kSpan) {
          offs = offsets(p);
          load(p, offs);
#pragma unroll
          for (int i = 0; i < kHeld; ++i) {
            if (t0 + p + i * RPW >= t1) break;
#pragma unroll
            for (int v = 0; v < kHeads; ++v) top[v].add_finite(raw[v][i]);
          }
        }
#pragma unroll
        for (int v = 0; v < kHeads; ++v) amax[v] = top[v].get();
      }
      float inv[kHeads];
      bool even = finite;                          // and the scales are powers of two
#pragma unroll
      for (int v = 0; v < kHeads; ++v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax[v] = fmaxf(amax[v], __shfl_xor_sync(0xffffffffu, amax[v], o));
        const float s = fmaxf(scale_for(amax[v]), held[v]);
        inv[v] = 1.0f / s;
        even = even && cb::is_power_of_two(s);
        if (v >= n) continue;
        if (first > 0 && s > held[v]) rescale_rows(rows[v], first * (A / 16), lane, 32, held[v] * inv[v]);
        if (lane == 0) *scale[v] = s;
      }
      if (!even) {                                 // rare: the rows once more, four at a time
        __syncwarp();                              // the scales are written
#pragma unroll 1
        for (int v = 0; v < n; ++v) {
          const int part = q + v, h = part % K;
          const bool is_v = part >= K;
          const uint4* from = static_cast<const uint4*>(is_v ? a.v_new : a.k_new) + int64_t(h) * LPR + c;
          uint8_t* to = static_cast<uint8_t*>(is_v ? a.v : a.k) + (page * K + h) * int64_t(B) * A + EPV * c;
          const int64_t step = is_v ? a.v_stride : a.k_stride;
          const float s = static_cast<volatile float*>(is_v ? a.v_scale : a.k_scale)[page * K + h];
#pragma unroll 1
          for (int p = r0; t0 + p < t1; p += 4 * RPW) {
            uint4 x[4];
            int64_t slot[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int t = t0 + p + i * RPW;
              slot[i] = t < t1 ? a.slots[t] : -1;
              x[i] = t < t1 ? from[int64_t(t) * step] : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float f[EPV];
              Vec16<T>::to_float(x[i], f);
              if (slot[i] >= 0 && slot[i] < a.num_slots) store_quotients(to + int(slot[i] & (B - 1)) * A, f, s);
            }
          }
        }
        if (!held_all) offs = offsets(0);
        continue;
      }
      for (int p = 0; t0 + p < t1; p += kSpan) {
        if (!held_all) {
          offs = offsets(p);
          load(p, offs);
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
          if (t0 + p + i * RPW >= t1) break;
          const int o = __shfl_sync(0xffffffffu, offs, i * RPW + r0);
#pragma unroll
          for (int v = 0; v < kHeads; ++v) {
            float f[EPV];
            Vec16<T>::to_float(raw[v][i], f);
            if (o >= 0 && v < n) store_lane(rows[v] + o * A, c, to_e4m3<true>(f, inv[v]));
          }
        }
      }
      if (!held_all) offs = offsets(0);
    }
  }
}

struct GatherArgs {
  const uint8_t *k, *v;
  const float *k_scale, *v_scale;
  const int32_t *tables, *cu, *starts;
  void *k_out, *v_out;
  int32_t num_rows, num_seqs, max_blocks, num_blocks, num_heads, block_shift, chunk_shift;   // chunks of 16 elements a head
  unsigned* err;
};

// f * s cut off to fp32 as product_to_odd does, however small.
__device__ __forceinline__ float small_to_odd(float f, float s) {
  const double p = double(f) * double(s);          // exact
  const float y = __double2float_rz(p);
  return double(y) == p ? y : __uint_as_float(__float_as_uint(y) | 1u);
}
// Rounded once: four bits times a power of two are exact in fp32; times another scale they have up to 28 bits.
__device__ __forceinline__ void store_row(__nv_bfloat16* dst, const uint4& x, float s) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r[8];
  auto row = [&](auto times) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[4];
      cb::e4m3x4_to_float(w[i], f);
      const __nv_bfloat162 lo = __floats2bfloat162_rn(times(f[0]), times(f[1])), hi = __floats2bfloat162_rn(times(f[2]), times(f[3]));
      r[2 * i] = *reinterpret_cast<const uint32_t*>(&lo);
      r[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&hi);
    }
  };
  if (cb::is_power_of_two(s)) row([&](float f) { return f * s; });
  else if (s >= 0x1p-90f) row([&](float f) { return cb::product_to_odd(f, s); });
  else row([&](float f) { return small_to_odd(f, s); });
  reinterpret_cast<uint4*>(dst)[0] = make_uint4(r[0], r[1], r[2], r[3]);
  reinterpret_cast<uint4*>(dst)[1] = make_uint4(r[4], r[5], r[6], r[7]);
}
__device__ __forceinline__ void store_row(float* dst, const uint4& x, float s) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[4];
    cb::e4m3x4_to_float(w[i], f);
    reinterpret_cast<float4*>(dst)[i] = make_float4(f[0] * s, f[1] * s, f[2] * s, f[3] * s);
  }
}

// A warp to a token's keys and values of all heads: its output rows are whole,
// and the tokens beside it, in other warps, read the lines beside its own.
template <typename T>
__global__ void __launch_bounds__(kThreads, kGatherCtasPerSm) gather_q8_kernel(const GatherArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int K = a.num_heads, chunks = K << a.chunk_shift, B = 1 << a.block_shift;
  const int total = min(a.num_rows, a.cu[a.num_seqs]);
  for (int r = blockIdx.x * kWarps + (threadIdx.x >> 5); r < total; r += gridDim.x * kWarps) {
    int s = 0;                                       // the last sequence that starts at or before the row
    for (int hi = a.num_seqs - 1; s < hi;) {
      const int mid = (s + hi + 1) >> 1;
      if (a.cu[mid] <= r) s = mid; else hi = mid - 1;
    }
    const int c0 = a.cu[s], start = a.starts ? a.starts[s] : 0;
    const int64_t pos = int64_t(start) + r - c0, lb = pos >> a.block_shift;
    if (c0 > r || a.cu[s + 1] <= r || start < 0 || lb >= a.max_blocks) {
      if (lane == 0) cb::raise_error(a.err, cb::kErrInvalid);
      continue;
    }
    const int blk = a.tables[int64_t(s) * a.max_blocks + lb];
    if (blk < 0 || blk >= a.num_blocks) {
      if (lane == 0) cb::raise_error(a.err, cb::kErrBounds);
      continue;
    }
    const int64_t src0 = ((int64_t(blk) * K << a.block_shift) + (pos & (B - 1))) << a.chunk_shift;
    const int64_t dst0 = int64_t(r) * chunks;
#pragma unroll 4
    for (int i = lane; i < 2 * chunks; i += 32) {
      const bool is_v = i >= chunks;
      const int j = is_v ? i - chunks : i, h = j >> a.chunk_shift, part = j - (h << a.chunk_shift);
      T* out = static_cast<T*>(is_v ? a.v_out : a.k_out);
      if (!out) continue;
      const uint4 x = cb::ldg_stream(reinterpret_cast<const uint4*>(is_v ? a.v : a.k) + src0 + (int64_t(h) << (a.block_shift + a.chunk_shift)) + part);
      const float sc = (is_v ? a.v_scale : a.k_scale)[int64_t(blk) * K + h];
      store_row(out + (dst0 + j) * 16, x, sc);
    }
  }
}

cb_status check_q8(const cb_kv_cache_q8* c, const char* who) {
  if (!c) return cb::fail(CB_ERR_INVALID, "%s: null cache", who);
  if (c->num_blocks < 1 || c->block_size < 1 || c->num_heads < 1 || c->head_dim < 1)
    return cb::fail(CB_ERR_INVALID, "%s: cache dimensions must be >= 1", who);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return cb::fail(CB_ERR_UNSUPPORTED, "%s: head_dim must be 64, 128 or 256", who);
  if (c->block_size & (c->block_size - 1) || c->block_size > 1024)
    return cb::fail(CB_ERR_UNSUPPORTED, "%s: block_size must be a power of two up to 1024", who);
  if (c->num_heads > 65536) return cb::fail(CB_ERR_UNSUPPORTED, "%s: too many heads", who);
  return CB_OK;
}
int log2_of(int32_t x) { return __builtin_ctz(unsigned(x)); }

bool aligned16(std::initializer_list<const void*> buffers) {
  for (const void* p : buffers)
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return false;
  return true;
}

template <typename T, int LPR>
cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream) {
  const int64_t units = int64_t(a.num_tokens) * 2 * a.num_heads;      // at most: a run for each token
  const int64_t grid = std::min<int64_t>((units + kWarps - 1) / kWarps, int64_t(kAppendCtasPerSm) * cb::sm_count());
  // Pages of more than 16 tokens: 32 positions of one head a warp, else 16 of two.  661 tokens of 8 heads and 2048 of 32, us, so
  // and the other way: pages of 32 7.6, 24.0 and 10.3, 25.3; of 128 19.0, 57 and 25.3, 59; of 16 7.3, 22.1 and 6.6, 25.1.
  return cb::launch_kernel(a.block_shift > 4 ? append_q8_kernel<T, LPR, true> : append_q8_kernel<T, LPR, false>, dim3(unsigned(grid)),
                           dim3(kThreads), 0, stream, true, a);
}

}  // namespace

extern "C" cb_status cb_append_kv_q8(const void* k_new, const void* v_new, cb_dtype dtype, int64_t k_stride,
                                     int64_t v_stride, const int64_t* slot_mapping, const int32_t* dims, int32_t num_tokens,
                                     const cb_kv_cache_q8* cache, void* stream) {
  const char* who = "cb_append_kv_q8";
  cb::NvtxRange nvtx("cb.append_kv_q8");
  cb_status st = check_q8(cache, who);
  if (st != CB_OK) return st;
  if (num_tokens < 0) return cb::fail(CB_ERR_INVALID, "%s: num_tokens < 0", who);
  if (dtype != CB_DTYPE_BF16 && dtype != CB_DTYPE_F32) return cb::fail(CB_ERR_UNSUPPORTED, "%s: unknown dtype", who);
  const bool bf16 = dtype == CB_DTYPE_BF16;
  if (!bf16 && cache->head_dim == 256) return cb::fail(CB_ERR_UNSUPPORTED, "%s: head_dim 256 needs bf16", who);
  if (num_tokens > kMaxTokens) return cb::fail(CB_ERR_UNSUPPORTED, "%s: more than %d tokens", who, kMaxTokens);
  if (int64_t(num_tokens) * 2 * cache->num_heads > 0x7fffffff) return cb::fail(CB_ERR_UNSUPPORTED, "%s: too many heads", who);
  if (num_tokens == 0) return CB_OK;
  if (!k_new || !v_new || !slot_mapping || !cache->k || !cache->v || !cache->k_scale || !cache->v_scale)
    return cb::fail(CB_ERR_INVALID, "%s: null pointer", who);
  const int epv = bf16 ? 8 : 4;
  const int64_t row = int64_t(cache->num_heads) * cache->head_dim;
  if (k_stride < row || v_stride < row)
    return cb::fail(CB_ERR_INVALID, "%s: a token stride is shorter than the token's heads", who);
  if (k_stride % epv || v_stride % epv)
    return cb::fail(CB_ERR_INVALID, "%s: token strides must be multiples of 16 bytes", who);
  if (!aligned16({k_new, v_new, cache->k, cache->v}))
    return cb::fail(CB_ERR_INVALID, "%s: k_new, v_new and the pools must be 16-byte aligned", who);
  unsigned* err = cb::device_error_word();
  if (!err) return CB_ERR_CUDA;
  AppendArgs a;
  a.k_new = k_new, a.v_new = v_new;
  a.k_stride = k_stride / epv, a.v_stride = v_stride / epv;
  a.slots = slot_mapping;
  a.dims = dims;
  a.k = static_cast<uint8_t*>(cache->k), a.v = static_cast<uint8_t*>(cache->v);
  a.k_scale = cache->k_scale, a.v_scale = cache->v_scale;
  a.num_slots = int64_t(cache->num_blocks) * cache->block_size;
  a.num_tokens = num_tokens;
  a.num_heads = cache->num_heads;
  a.num_blocks = cache->num_blocks;
  a.block_shift = log2_of(cache->block_size);
  a.err = err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int A = cache->head_dim;
  const cudaError_t e = bf16 && A == 64    ? launch_append<__nv_bfloat16, 8>(a, s)
                        : bf16 && A == 128 ? launch_append<__nv_bfloat16, 16>(a, s)
                        : bf16             ? launch_append<__nv_bfloat16, 32>(a, s)
                        : A == 64          ? launch_append<float, 16>(a, s)
                                           : launch_append<float, 32>(a, s);
  return e == cudaSuccess ? CB_OK : cb::cuda_fail(e, "8-bit append: launch");
}

extern "C" cb_status cb_gather_kv_q8(const cb_kv_cache_q8* cache, const int32_t* block_tables, const int32_t* cu_keys,
                                     const int32_t* starts, int32_t num_seqs, int32_t max_blocks_per_seq, int32_t num_rows,
                                     cb_dtype dtype, void* k_out, void* v_out, void* stream) {
  const char* who = "cb_gather_kv_q8";
  cb::NvtxRange nvtx("cb.gather_kv_q8");
  cb_status st = check_q8(cache, who);
  if (st != CB_OK) return st;
  if (num_seqs < 0 || max_blocks_per_seq < 0 || num_rows < 0) return cb::fail(CB_ERR_INVALID, "%s: negative size", who);
  if (dtype != CB_DTYPE_BF16 && dtype != CB_DTYPE_F32) return cb::fail(CB_ERR_UNSUPPORTED, "%s: unknown dtype", who);
  if (num_seqs == 0 || num_rows == 0) return CB_OK;
  if (!block_tables || !cu_keys || (k_out && (!cache->k || !cache->k_scale)) || (v_out && (!cache->v || !cache->v_scale)))
    return cb::fail(CB_ERR_INVALID, "%s: null pointer", who);
  if (!k_out && !v_out) return CB_OK;
  if (!aligned16({k_out, v_out, cache->k, cache->v}))
    return cb::fail(CB_ERR_INVALID, "%s: the outputs and the pools must be 16-byte aligned", who);
  unsigned* err = cb::device_error_word();
  if (!err) return CB_ERR_CUDA;
  GatherArgs a;
  a.k = static_cast<const uint8_t*>(cache->k), a.v = static_cast<const uint8_t*>(cache->v);
  a.k_scale = cache->k_scale, a.v_scale = cache->v_scale;
  a.tables = block_tables, a.cu = cu_keys, a.starts = starts;
  a.k_out = k_out, a.v_out = v_out;
  a.num_rows = num_rows, a.num_seqs = num_seqs, a.max_blocks = max_blocks_per_seq;
  a.num_blocks = cache->num_blocks, a.num_heads = cache->num_heads;
  a.block_shift = log2_of(cache->block_size), a.chunk_shift = log2_of(cache->head_dim / 16);
  a.err = err;
  const int64_t grid = std::min<int64_t>((int64_t(num_rows) + kWarps - 1) / kWarps, int64_t(kGatherCtasPerSm) * cb::sm_count());
  const cudaError_t e = cb::launch_kernel(dtype == CB_DTYPE_BF16 ? gather_q8_kernel<__nv_bfloat16> : gather_q8_kernel<float>,
                                          dim3(unsigned(grid)), dim3(kThreads), 0, static_cast<cudaStream_t>(stream), true, a);
  return e == cudaSuccess ? CB_OK : cb::cuda_fail(e, "8-bit read-back: launch");
}
