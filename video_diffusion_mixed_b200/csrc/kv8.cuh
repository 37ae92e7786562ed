// kv8.cuh -- what the FP8 cache's kernels share: number formats, a sequence's spans, masks, and the
// layout of partial results.
#pragma once

#include <cuda_fp16.h>

#include "e4m3.cuh"
#include "sb_device.cuh"
#include "sb_kernels.h"

namespace sb {
namespace kv8 {

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16x2(uint32_t lo, uint32_t hi) {  // FP32 bit patterns
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float(hi)), "f"(__uint_as_float(lo)));
  return r;
}
// A softmax weight is rounded to fp16 times 2^kShift: relative to the running maximum it is 2^kRise at most
// before the maximum moves, 2^(kRise + kShift) stays in fp16's range, and the smallest weights, of which a long
// cache has many, are rounded at 2^-(25 + kShift) of the largest. A rise of 4 and a shift of 11 would keep
// sixteen times smaller ones, but the maximum moves more often: 2047 causal rows of 16 heads of 128 took 202 us
// instead of 189, 17776 x 17776 of 30 heads of 64 3.54 ms instead of 3.46.
constexpr float kRise = 8.0f;
constexpr int kShift = 7;
constexpr int kFewRows = 16;   // rows of a key head up to which the streaming kernel serves

// The power of two (at most 2^126) that brings a row of queries with largest magnitude `a` (bf16 bits) to
// [2^14, 2^15), and the factor of the scores that takes it back, times scale and log2(e). An Inf or NaN
// stays one.
__device__ __forceinline__ float query_scale(float scale, uint32_t a, float& factor) {
  const int e = min(141 - (int)(a >> 7), 126);  // 14 - floor(log2 a)
  factor = __uint_as_float((uint32_t)(e + 127) << 23);
  return scale * __uint_as_float((uint32_t)(127 - e) << 23) * 1.4426950408889634f;
}

__device__ __forceinline__ float fast_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A row's running statistics. With s the scores (log2) and ev the exponents of the values' blocks, weights are
// 2^(s + ev - m), m the running maximum of s + ev over the keys that the row sees, and the sum is l = sum of
// 2^(s - m + e): a weight times 2^(e - ev), which is exact. e is the exponent of the block that moved m last, so
// blocks that the row does not see have no part in it. Scales differ by up to 2^254 and scores undo that, so
// e gives way wherever l would leave FP32's range.
struct RowStats {
  float m, l;
  int e;
};

// m moves to mn, set by a block of exponent ev. l loses 2^(m - mn), and counts by the new exponent.
__device__ __forceinline__ void move_max(RowStats& r, float mn, int ev) {
  const float y = r.m - mn + (float)(ev - r.e);
  const int k = y > 0.0f ? min(__float2int_ru(y), 512) : 0;  // l must not rise
  r.l *= fast_ex2(y - (float)k);
  r.e = ev - k;
  r.m = mn;
}

// A block more than kFar below e: its weights vanish where their part of the sum may not, so that is taken by
// itself, in terms 2^(s + far_base). top: the block's largest score before c.
constexpr int kFar = 64;
__device__ __forceinline__ float far_base(RowStats& r, float top, float c) {
  float base = (float)r.e - (r.m == -INFINITY ? 0.0f : r.m);
  const float most = fmaf(top, c, base);
  if (most > 64.0f) {
    const int k = min(__float2int_ru(most), 512);
    r.e -= k;
    r.l *= fast_ex2(-(float)k);
    base -= (float)k;
  }
  return base;
}

// The factor of a sum of shifted weights of a block `d` below e (at most kFar; what is 2^-119 times a weight
// adds nothing).
__device__ __forceinline__ float sum_factor(int d) {
  return __uint_as_float((uint32_t)(max(d, -119) - kShift + 127) << 23);
}

// The outputs' unit 2^(e - kShift), e relative to exponent byte e0, as two factors; the reciprocal of l goes
// between them, and no product on the way leaves the normal range.
__device__ __forceinline__ float2 output_unit(int e, int e0) {
  const int u = min(max(e + e0 - 127 - kShift, -252), 252), h = u >> 1;
  return make_float2(__uint_as_float((uint32_t)(h + 127) << 23), __uint_as_float((uint32_t)(u - h + 127) << 23));
}

// One sequence: tokens held, queries, and the position of a query token.
struct Span {
  int len, nq, causal;
  bool bad;  // a length on the device was out of range (and clamped)
  __device__ __forceinline__ int pos(int tok) const { return causal ? len - nq + tok : len - 1; }
};
__device__ __forceinline__ Span sequence_span(const Kv8Attn& p, int64_t b) {
  Span s;
  const int len = p.c.lens[b], nq = p.q_lens ? p.q_lens[b] : (int)p.n_q;
  s.len = max(0, min(len, (int)p.c.capacity));
  s.nq = max(0, min(nq, (int)p.n_q));
  s.bad = s.len != len || s.nq != nq;
  s.causal = p.causal;
  return s;
}

// window and sinks are clamped to 2^30 by the host: positions are below it.
__device__ __forceinline__ bool key_visible(const Kv8Attn& p, int pos, int j) {
  return j <= pos && (p.window == 0 || pos - j < (int)p.window || j < (int)p.sinks);
}

// The key tiles of `size` tokens that rows at positions pmin .. pmax may see: the first `head` ones, then
// those from `first` on.
struct KeyTiles {
  int head, first, n;
  __device__ __forceinline__ int tile(int i) const { return i < head ? i : i - head + first; }
};
__device__ __forceinline__ KeyTiles key_tiles(const Kv8Attn& p, int pmin, int pmax, int size) {
  KeyTiles k;
  const int end = pmax < 0 ? 0 : pmax / size + 1;
  k.first = 0;
  k.head = 0;
  if (p.window > 0) {
    k.first = min(end, max(0, pmin - (int)p.window + 1) / size);
    k.head = min(k.first, ((int)p.sinks + size - 1) / size);
  }
  k.n = k.head + end - k.first;
  return k;
}
// Whether some row at pmin .. pmax does not see every key of the tile.
__device__ __forceinline__ bool tile_needs_mask(const Kv8Attn& p, int j0, int size, int pmin, int pmax) {
  return j0 + size - 1 > pmin ||
         (p.window > 0 && pmax - j0 >= (int)p.window && j0 + size > (int)p.sinks);
}

// sb_kv8_store gives a block that holds a NaN or an Inf an exponent byte of at least this one (that of the largest
// finite values, from 1.75 * 2^127 on). A weight of zero does not hide a NaN in the products.
constexpr int kNanExp = 247;

// One row by itself, a warp's work, in FP32 throughout: for what the kernels' products cannot hold. Values of keys that
// the row does not see are not touched, so a NaN among them stays there. Rare, and some hundred times slower than the
// tensor cores: a lane takes a key's score, then D / 32 channels of the output.
template <int D>
struct ExactRow {
  float y[D / 32];  // this lane's channels
  float lse2;
};
template <int D>
__device__ __forceinline__ void exact_row(const Kv8Attn& p, int64_t b, int64_t hk, int64_t tok, int64_t hq, int len,
                                          int pos, KeyTiles kt, int size, int i0, int i1, float* qs,
                                          ExactRow<D>& out) {
  constexpr int kE = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t head = b * p.c.heads + hk;
  const uint8_t* kx = p.c.k_exp + head * (p.c.capacity / 64);
  const uint8_t* vx = p.c.v_exp + head * (p.c.capacity / 64);
  const uint8_t* kc = p.c.k_codes + head * p.c.capacity * D;
  const uint8_t* vc = p.c.v_codes + head * p.c.capacity * D + lane * kE;
  const uint16_t* q = static_cast<const uint16_t*>(p.q) + b * p.qs[0] + tok * p.qs[1] + hq * p.qs[2] + lane * kE;
  uint32_t a = 0;
  for (int i = 0; i < kE; ++i) a = max(a, (uint32_t)q[i] & 0x7fffu);
  float f;
  const float back = query_scale(p.scale, __reduce_max_sync(0xffffffffu, a), f);
  __syncwarp();  // the row before has been read
  for (int i = 0; i < kE; ++i) qs[lane * kE + i] = __uint_as_float((uint32_t)q[i] << 16) * f;
  __syncwarp();
  RowStats st{-INFINITY, 0.0f, 0};  // l: this lane's keys
  float acc[kE] = {};
  const int e0 = i0 < i1 ? (int)vx[(int64_t)kt.tile(i0) * size / 64] : 0;
#pragma unroll 1
  for (int i = i0; i < i1; ++i) {
#pragma unroll 1
    for (int j0 = kt.tile(i) * size, end = min(len, j0 + size); j0 < end; j0 += 32) {
      const int j = j0 + lane, ev = (int)vx[j0 >> 6] - e0;
      const bool see = j < len && key_visible(p, pos, j);
      const float c = fminf(fmaxf(back * pow2_byte((int)kx[j0 >> 6]), 0x1p-126f), 0x1p126f);
      float s = -INFINITY;
      if (see) {
        float dot = 0.0f;
#pragma unroll 1
        for (int d = 0; d < D; d += 4) {
          const uint32_t k = *reinterpret_cast<const uint32_t*>(kc + (int64_t)j * D + d);
          for (int e = 0; e < 4; ++e) dot = fmaf(qs[d + e], e4m3_to_f32(k >> (8 * e)), dot);
        }
        s = dot * c;
      }
      const float top = warp_max_f32(s), mn = fmaxf(st.m, top + (float)ev);
      if (mn > st.m + kRise) {
        const float g = fast_ex2(st.m - mn);
        for (int e = 0; e < kE; ++e) acc[e] *= g;
        move_max(st, mn, ev);
      }
      const int below = st.e - ev;
      if (below > kFar) st.l += fast_ex2(s + far_base(st, top, 1.0f));
      const float w = fast_ex2(s + ((float)(ev + kShift) - (st.m == -INFINITY ? 0.0f : st.m)));
      if (below <= kFar) st.l = fmaf(w, sum_factor(below), st.l);
      for (uint32_t seen = __ballot_sync(0xffffffffu, see); seen; seen &= seen - 1) {
        const int jj = __ffs(seen) - 1;
        const float wj = __shfl_sync(0xffffffffu, w, jj);
        for (int e = 0; e < kE; ++e) acc[e] = fmaf(wj, e4m3_to_f32(vc[(int64_t)(j0 + jj) * D + e]), acc[e]);
      }
    }
  }
#pragma unroll
  for (int s = 16; s >= 1; s >>= 1) st.l += __shfl_xor_sync(0xffffffffu, st.l, s);
  const float inv = st.l > 0.0f ? 1.0f / st.l : st.l;
  const float2 unit = output_unit(st.e, e0);
  for (int e = 0; e < kE; ++e) out.y[e] = acc[e] * unit.x * inv * unit.y;
  out.lse2 = st.l > 0.0f ? st.m - (float)st.e + log2f(st.l) : st.l == 0.0f ? -INFINITY : st.l;
}

// Partial results of `splits` parts of the keys: for every part and row (row = token * group + head in
// the group, of a sequence and key head) D normalised outputs, and the log2 of the sum.
__host__ __device__ inline int64_t part_rows(const Kv8Attn& p) {
  return p.c.batch * p.n_q * p.heads_q;
}
__device__ __forceinline__ int64_t part_index(const Kv8Attn& p, int split, int64_t b, int64_t hk, int64_t r) {
  return (split * p.c.batch * p.c.heads + b * p.c.heads + hk) * (p.n_q * (p.heads_q / p.c.heads)) + r;
}
__device__ __forceinline__ float* part_row(const Kv8Attn& p, float* part, int split, int64_t b, int64_t hk, int64_t r) {
  return part + part_index(p, split, b, hk, r) * p.c.dim;
}
__device__ __forceinline__ float* part_lse(const Kv8Attn& p, float* part, int splits, int split, int64_t b, int64_t hk,
                                           int64_t r) {
  return part + splits * part_rows(p) * p.c.dim + part_index(p, split, b, hk, r);
}

}  // namespace kv8
}  // namespace sb
