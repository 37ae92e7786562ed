// gemm_epi.cuh -- what the tensor-core GEMM kernels share: FP32x2 epilogue arithmetic, the GELU, the
// tile order and the staging of bf16 output rows for TMA stores.
#pragma once

#include "sb_device.cuh"

namespace sb {

__device__ __forceinline__ float tanh_approx(float x) {
  float y;
  asm("tanh.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// FP32x2 arithmetic for the epilogue (one instruction, two lanes of FP32 work; the epilogue's
// outputs are compared with a tolerance, so contraction is allowed here).
__device__ __forceinline__ uint64_t ep_bits(float2 a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 ep_f2(uint64_t r) {
  float2 a;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
  return a;
}
__device__ __forceinline__ float2 ep_mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(ep_bits(a)), "l"(ep_bits(b)));
  return ep_f2(r);
}
__device__ __forceinline__ float2 ep_fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(ep_bits(a)), "l"(ep_bits(b)), "l"(ep_bits(c)));
  return ep_f2(r);
}
__device__ __forceinline__ float2 ep_add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(ep_bits(a)), "l"(ep_bits(b)));
  return ep_f2(r);
}

// tanh-form GELU, 0.5 v (1 + tanh(sqrt(2/pi) (v + 0.044715 v^3))), with the SFU's tanh
// approximation, on two values at a time. Its error (relative about 2^-11) is absolute in the result, about
// 2^-12 |v|: below the bf16 rounding for positive v, but up to a fifth of the value at v = -3 and more
// beyond, where the two terms cancel.
__device__ __forceinline__ float2 gelu_tanh2(float2 v) {
  const float2 c1 = make_float2(0.7978845608028654f * 0.044715f, 0.7978845608028654f * 0.044715f);
  const float2 c0 = make_float2(0.7978845608028654f, 0.7978845608028654f);
  const float2 u = ep_mul2(v, ep_fma2(c1, ep_mul2(v, v), c0));
  const float2 h = ep_mul2(make_float2(0.5f, 0.5f), v);
  return ep_fma2(h, make_float2(tanh_approx(u.x), tanh_approx(u.y)), h);
}

// The same GELU as v / (1 + 2^(-2 log2(e) sqrt(2/pi) (v + 0.044715 v^3))), whose relative error stays near
// 2^-20 in the negative tail: an exponential and a reciprocal for the tanh.
__device__ __forceinline__ float2 gelu_exp2(float2 v) {
  constexpr float kA = -2.0f * 1.4426950408889634f * 0.7978845608028654f;
  const float2 a = ep_mul2(v, ep_fma2(make_float2(kA * 0.044715f, kA * 0.044715f), ep_mul2(v, v), make_float2(kA, kA)));
  float ex, ey, rx, ry;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(ex) : "f"(a.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(ey) : "f"(a.y));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rx) : "f"(1.0f + ex));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(ry) : "f"(1.0f + ey));
  return make_float2(v.x * rx, v.y * ry);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Grouped tile order: group_m consecutive M-tiles are swept across all N-tiles before the next
// group starts (M-tile fastest inside a group), so the A rows of a group stay in L2 while every
// N-tile reuses them (A of the second FFN layer is larger than L2 and would otherwise be re-read
// from HBM for each N-tile). The host picks group_m (pick_group_m).
__device__ __forceinline__ void tile_coords(int t, int m_tiles, int n_tiles, int group_m, int* mt, int* nt) {
  const int group = group_m * n_tiles;
  const int g = t / group, r = t - g * group;
  const int first = g * group_m;
  const int gm = min(group_m, m_tiles - first);
  *mt = first + r % gm;
  *nt = r / gm;
}

// bf16 row chunk into a 32 x 32 staging box (row = lane, 64 bytes): 16-byte granule g of row r
// sits at granule g ^ ((r >> 1) & 3), the TMA 64B swizzle, so the 32 lanes' writes hit distinct
// banks in groups of eight.
__device__ __forceinline__ void stage_bf16_row(uint32_t box, int lane, const uint32_t (&y)[32]) {
  const uint32_t row = box + 64u * (uint32_t)lane;
  const uint32_t sw = ((uint32_t)lane >> 1) & 3u;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const float* v = reinterpret_cast<const float*>(&y[8 * g]);
    st_shared_v4(row + 16u * ((uint32_t)g ^ sw), pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                 pack_bf16(v[6], v[7]));
  }
}

}  // namespace sb
