// Streams of single warps (suffix_stream.cuh) over a cache in 8 bits: e4m3 keys
// and values, a fp32 scale for each block and head.
//
// A tile is 16 keys of one block: 2 KB of keys and 2 KB of values by TMA, and the
// block's two scales by a 4-byte asynchronous copy each, all on the tile's barrier.
//   * e4m3 numbers are exact in f16, so the matrix steps are f16's.  A query row is
//     scaled by a power of two that brings its largest number to 2^13 .. 2^14: its
//     bf16 numbers are then exact in f16 down to 2^-27 of that, and off by at most
//     2^-38 of it below.
//   * ldmatrix moves pairs of bytes as its 16-bit numbers.  For the scores a lane
//     gets four neighbouring dims of its key, and both operands take the dims of a
//     step in that order; for the output it gets two dims of two keys, one byte
//     permutation makes them two pairs of keys, and even and odd dims are columns of
//     different tiles.
//   * A block's key scale multiplies its scores.  Its value scale vs multiplies the
//     weights, of which the tensor core takes 11 bits and 2^-24 .. 2^16 in f16: so a
//     row keeps, beside its running maximum m of the scores (exp2 domain), the running
//     maximum M of score + log2(vs); the output's weights 2^(s - M) vs are at most
//     2^8 (stale maxima are kept as long as that holds), while the sum, in fp32, stays
//     that of 2^(s - m).
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
using stream::SmallStep;
using stream::Unit;

constexpr int kStages = 6;
constexpr uint32_t kBox = kTileKeys * kDim;            // 2 KB, rows of 128 bytes, 128-byte swizzled
constexpr uint32_t kStageBytes = 2 * kBox;
constexpr uint32_t kRingBytes = kStreamWarps * kStages * kStageBytes;
constexpr uint32_t kBarBytes = kStreamWarps * kStages * 16;   // per warp: barriers, then (key, value) scales of each stage
constexpr int kBarArrivals = 3;                        // of a stage: the copies' bytes, and either scale

__device__ __forceinline__ void tma_load_3d_tile(uint32_t dst, const void* tmap, uint32_t bar, int32_t y, int32_t z) {
  tma_load_3d(dst, tmap, bar, 0, y, z);
}
__device__ __forceinline__ void copy4_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives on `bar` once this thread's asynchronous copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}
// D(16 x 8, fp32) += A(16 x 16) B(16 x 8), f16
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// As stream::run_warp.  `bars`: kStages barriers (initialised for kBarArrivals),
// then kStages pairs of scales, which `scales` points to.
template <bool kSmall>
__device__ __forceinline__ void run_warp(const CUtensorMap* tm_k, const CUtensorMap* tm_v, const AttnArgs& a,
                                         const PrefixWork& w, int n_items, uint32_t ring, uint32_t bars,
                                         const volatile float2* scales, SuffixItem* slots, int first, int step,
                                         int claimed_from, const SmallStep small) {
  const int lane = threadIdx.x & 31;
  const int H = a.num_heads, Hkv = a.num_kv_heads, G = H / Hkv, B = a.block_size;
  const int n_units = n_items * Hkv;
  const int boxes = a.num_blocks * Hkv;
  const int g = lane >> 2, t = lane & 3;                 // fragment row and column pair
  const uint32_t scale_at = bars + 8 * kStages;

  // pages of tiles zt .. zt + 31 of the unit in slot `sl`, one per lane
  auto load_pages = [&](Unit& u, const SuffixItem& it, int zt) {
    u.zt = zt;
    u.z = boxes;                                         // out of range: TMA fills zeros
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
        const stream::SmallSeq q = small.seqs[s];
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
    const int st = issued % kStages;
    const uint32_t bar = bars + 8 * st;
    if (lane < 2) {
      const float* scale = lane == 0 ? a.k_scale : a.v_scale;
      copy4_async(scale_at + 8 * st + 4 * lane, scale + (z < boxes ? z : 0));
      copies_arrive(bar);
    }
    if (lane == 0) {
      const uint32_t dst = ring + st * kStageBytes;
      const int y = (it.k0 + i * kTileKeys) & (B - 1);
      mbar_arrive_expect_tx(bar, kStageBytes);
      tma_load_3d_tile(dst, tm_k, bar, y, z);
      tma_load_3d_tile(dst + kBox, tm_v, bar, y, z);
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
  // this lane's part of an ldmatrix address: matrix mi, its row mr
  const int mi = lane >> 3, mr = lane & 7;
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
    // The unit's query rows, as A fragments in f16; rows past the sequence's are zero.
    const int rows = min(16, it.q_len * G - it.row0);
    uint32_t qf[8][4];
    float e0, e1;                                        // a score's factor, without its block's scale
    {
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
      const int r0 = it.row0 + g, r1 = r0 + 8;
      const __nv_bfloat16* p0 = q + (size_t(it.tok0 + r0 / G) * H + cur.hk * G + r0 % G) * kDim + 4 * t;
      const __nv_bfloat16* p1 = q + (size_t(it.tok0 + r1 / G) * H + cur.hk * G + r1 % G) * kDim + 4 * t;
      const bool in0 = g < rows, in1 = g + 8 < rows;
      uint32_t top0 = 0, top1 = 0;                       // bits of the largest magnitude
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const uint2 x = in0 ? *reinterpret_cast<const uint2*>(p0 + 16 * ks) : make_uint2(0, 0);
        const uint2 y = in1 ? *reinterpret_cast<const uint2*>(p1 + 16 * ks) : make_uint2(0, 0);
        qf[ks][0] = x.x, qf[ks][1] = y.x, qf[ks][2] = x.y, qf[ks][3] = y.y;
        top0 = max(max(top0, (x.x << 16) & 0x7fff0000u), max(x.x & 0x7fff0000u, max((x.y << 16) & 0x7fff0000u, x.y & 0x7fff0000u)));
        top1 = max(max(top1, (y.x << 16) & 0x7fff0000u), max(y.x & 0x7fff0000u, max((y.y << 16) & 0x7fff0000u, y.y & 0x7fff0000u)));
      }
#pragma unroll
      for (int x = 1; x <= 2; x <<= 1) {
        top0 = max(top0, __shfl_xor_sync(0xffffffffu, top0, x));
        top1 = max(top1, __shfl_xor_sync(0xffffffffu, top1, x));
      }
      const uint32_t x0 = min(254u, 267u - (top0 >> 23)), x1 = min(254u, 267u - (top1 >> 23));   // 2^13 / largest, as exponents
      const float f0 = __uint_as_float(x0 << 23), f1 = __uint_as_float(x1 << 23);
      e0 = a.scale_log2 * __uint_as_float((254u - x0) << 23);
      e1 = a.scale_log2 * __uint_as_float((254u - x1) << 23);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        qf[ks][0] = pack_f16(bf16_lo(qf[ks][0]) * f0, bf16_hi(qf[ks][0]) * f0);
        qf[ks][1] = pack_f16(bf16_lo(qf[ks][1]) * f1, bf16_hi(qf[ks][1]) * f1);
        qf[ks][2] = pack_f16(bf16_lo(qf[ks][2]) * f0, bf16_hi(qf[ks][2]) * f0);
        qf[ks][3] = pack_f16(bf16_lo(qf[ks][3]) * f1, bf16_hi(qf[ks][3]) * f1);
      }
    }
    // keys that a row sees: all before its own token's, and its own
    const int k0 = it.k0, k1 = it.k1, ctx = it.ctx, before = ctx - it.q_len;
    const int lim0 = min(k1, before + (it.row0 + g) / G + 1), lim1 = min(k1, before + (it.row0 + g + 8) / G + 1);
    const int lim_all = min(k1, before + it.row0 / G + 1);   // keys that every row sees
    float o[16][4];                                      // [2 * chunk of 16 dims + odd dims]
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float w0 = -INFINITY, w1 = -INFINITY, f0 = 1.f, f1 = 1.f;   // M of either row, and 2^(m - M)
    for (int i = 0; i < cur.n; ++i) {
      const int st = consumed % kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(bars + 8 * st, (consumed / kStages) & 1))) {
        ok = false;
        break;
      }
      const float ks = scales[st].x, vs = scales[st].y;
      const uint32_t kt = ring + st * kStageBytes, vt = kt + kBox;
      const int kb = k0 + i * kTileKeys;
      if (kb + kTileKeys > ctx) {                        // rows behind the sequence's last key: P is 0, but 0 * NaN is not
        const int from = ctx - kb;
        for (int c = lane; c < (kTileKeys - from) * 8; c += 32)
          asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(vt + (from + c / 8) * 128 + (c % 8) * 16), "r"(0) : "memory");
        fence_proxy_async_smem();                        // before the slot's next TMA write
        __syncwarp();
      }
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t kf[4];
          ldmatrix4(kt + (8 * x + mr) * 128 + (((4 * c + mi) ^ mr) << 4), kf);
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_f16(s[x], qf[4 * c + j], e4m3x2_to_f16x2(kf[j]), e4m3x2_hi_to_f16x2(kf[j]));
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
      const float a0 = fmaxf(e0 * ks, 1.2e-38f), a1 = fmaxf(e1 * ks, 1.2e-38f);   // not 0: -inf stays
      const float lv = fmaxf(lg2(vs), -126.f);
      float t0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1])) * a0;
      float t1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3])) * a1;
      // keep stale maxima while 2^x stays <= 2^8
      if (__any_sync(0xffffffffu, t0 > m0 + 8.0f || t1 > m1 + 8.0f || t0 + lv > w0 + 8.0f || t1 + lv > w1 + 8.0f)) {
#pragma unroll
        for (int x = 1; x <= 2; x <<= 1) {
          t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, x));
          t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, x));
        }
        const float n0 = fmaxf(m0, t0), n1 = fmaxf(m1, t1), v0 = fmaxf(w0, t0 + lv), v1 = fmaxf(w1, t1 + lv);
        if (n0 != -INFINITY) {
          l0 *= ex2(m0 - n0);
          const float x = ex2(w0 - v0);
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j][0] *= x, o[j][1] *= x;
          f0 = ex2(fminf(n0 - v0, 126.f));
        }
        if (n1 != -INFINITY) {
          l1 *= ex2(m1 - n1);
          const float x = ex2(w1 - v1);
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j][2] *= x, o[j][3] *= x;
          f1 = ex2(fminf(n1 - v1, 126.f));
        }
        m0 = n0, m1 = n1, w0 = v0, w1 = v1;
      }
      const float z0 = m0 == -INFINITY ? 0.f : -m0, z1 = m1 == -INFINITY ? 0.f : -m1;   // a row that sees no key yet
      const float c0 = fminf(vs * f0, 3e38f), c1 = fminf(vs * f1, 3e38f);
      uint32_t pf[4];                                    // weights in f16: within 2^-12 of each, 2^-25 of 2^(M - m)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float p0 = ex2(fmaf(s[x][0], a0, z0)), p1 = ex2(fmaf(s[x][1], a0, z0));
        const float p2 = ex2(fmaf(s[x][2], a1, z1)), p3 = ex2(fmaf(s[x][3], a1, z1));
        l0 += p0 + p1;
        l1 += p2 + p3;
        pf[2 * x] = pack_f16(p0 * c0, p1 * c0);
        pf[2 * x + 1] = pack_f16(p2 * c1, p3 * c1);
      }
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        uint32_t vf[4];
        ldmatrix4_trans(vt + ((mi & 1) * 8 + mr) * 128 + (((2 * jj + (mi >> 1)) ^ mr) << 4), vf);
#pragma unroll
        for (int x = 0; x < 4; ++x) vf[x] = __byte_perm(vf[x], 0, 0x3120);   // (key, key + 1) of the even dim, of the odd dim
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          mma_f16(o[4 * jj + 2 * x], pf, e4m3x2_to_f16x2(vf[2 * x]), e4m3x2_to_f16x2(vf[2 * x + 1]));
          mma_f16(o[4 * jj + 2 * x + 1], pf, e4m3x2_hi_to_f16x2(vf[2 * x]), e4m3x2_hi_to_f16x2(vf[2 * x + 1]));
        }
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
    // the rows' records, or, with nothing to join, the rows; o is in units of 2^M, a record's in 2^m
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (g + 8 * half < rows) {
        const int r = it.row0 + g + 8 * half, tok = r / G, h = cur.hk * G + r % G;
        const float m = half ? m1 : m0, l = half ? l1 : l0, top = half ? w1 : w0;
        const float to_m = m == -INFINITY ? 0.f : ex2(top - m);
        if (it.direct) {
          const float f = to_m / l;
          uint2* dst = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + (size_t(it.tok0 + tok) * H + h) * kDim) + t;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float *even = &o[2 * j][2 * half], *odd = &o[2 * j + 1][2 * half];
            dst[4 * j] = make_uint2(pack2(even[0] * f, odd[0] * f), pack2(even[1] * f, odd[1] * f));
          }
        } else {
          const size_t at = size_t(it.rec0) + (size_t(tok) * H + h) * it.rec_step;
          float4* rec = reinterpret_cast<float4*>(w.recs + at * kDim) + t;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float *even = &o[2 * j][2 * half], *odd = &o[2 * j + 1][2 * half];
            __stcg(rec + 4 * j, make_float4(even[0] * to_m, odd[0] * to_m, even[1] * to_m, odd[1] * to_m));
          }
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

}  // namespace qstream
}  // namespace cb
