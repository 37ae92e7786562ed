// kv8.cuh -- what the FP8 cache's kernels share: number formats, a sequence's spans, masks, and the
// layout of partial results.
#pragma once

#include <cuda_fp16.h>

#include "sb_device.cuh"
#include "sb_kernels.h"

namespace sb {
namespace kv8 {

__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t b) {  // exact
  uint32_t h;
  const uint16_t in = (uint16_t)b;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(in));
  return h;
}
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
__device__ __forceinline__ float pow2_byte(int byte) {  // 2^(byte - 127)
  return byte <= 0 ? 0x1p-127f : __uint_as_float((uint32_t)byte << 23);
}

// A softmax weight is rounded to fp16 times 2^kShift: relative to the running maximum it is 2^kRise at most
// before the maximum moves, 2^(kRise + kShift) stays in fp16's range, and the smallest weights, of which a long
// cache has many, are rounded at 2^-(25 + kShift) of the largest. A rise of 4 and a shift of 11 would keep
// sixteen times smaller ones, but the maximum moves more often: 2047 causal rows of 16 heads of 128 took 202 us
// instead of 189, 17776 x 17776 of 30 heads of 64 3.54 ms instead of 3.46.
constexpr float kRise = 8.0f;
constexpr int kShift = 7;
constexpr float kUnshift = 1.0f / (1 << kShift);
constexpr int kFewRows = 16;   // rows of a key head up to which the streaming kernel serves

// The power of two (at most 2^126) that brings a row of queries with largest magnitude `a` (bf16 bits) to
// [2^14, 2^15), and the factor of the scores that takes it back, times scale and log2(e). An Inf or NaN
// stays one.
__device__ __forceinline__ float query_scale(float scale, uint32_t a, float& factor) {
  const int e = min(141 - (int)(a >> 7), 126);  // 14 - floor(log2 a)
  factor = __uint_as_float((uint32_t)(e + 127) << 23);
  return scale * __uint_as_float((uint32_t)(127 - e) << 23) * 1.4426950408889634f;
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
