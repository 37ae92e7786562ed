// fp8.cu -- linear layer in 8-bit floating point: E4M3 codes with one E8M0 scale per 128 channels.
#include "launch_util.h"
#include "sb_device.cuh"
#include "sb_kernels.h"

namespace sb {

// Exponent byte of a block with largest magnitude a, given as bf16 bits: the smallest e with
// a <= 448 * 2^e (448 = 1.75 * 2^8), plus 127; a is 1.m * 2^(field - 127). Subnormal and zero a
// give 0.
__device__ __forceinline__ uint32_t e8m0_of_amax(uint32_t bits) {
  const int b = (int)(bits >> 7) - 8 + ((bits & 0x7fu) > 0x60u ? 1 : 0);
  return (uint32_t)max(b, 0);
}

// 2^-e for an exponent byte e + 127 (byte <= 253, which every finite bf16 amax gives).
__device__ __forceinline__ float e8m0_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

__device__ __forceinline__ uint32_t cvt_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// One warp per (row, 512 channels): a lane takes 16 channels, eight lanes a block.
__global__ void __launch_bounds__(256) k_fp8_encode(const __nv_bfloat16* __restrict__ X, int64_t M, int K,
                                                    const int32_t* prec, uint8_t* __restrict__ codes,
                                                    uint32_t* __restrict__ sf, WsHeader* hdr) {
  if (prec && *prec == SB_SKIP) return;
  const int lane = threadIdx.x & 31;
  const int groups = (K + 511) / 512;
  const int64_t tasks = ceil_div(M, 128) * 128 * groups;
  for (int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); t < tasks; t += (int64_t)gridDim.x * 8) {
    const int64_t m = t / groups;
    const int g = (int)(t - m * groups);
    const int k = g * 512 + lane * 16;
    uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
    const bool live = m < M && k < K;
    if (live) {
      const uint4* src = reinterpret_cast<const uint4*>(X + m * K + k);
      u0 = __ldg(src);
      u1 = __ldg(src + 1);
    }
    uint32_t a = __vmaxu2(__vmaxu2(__vmaxu2(u0.x & 0x7fff7fffu, u0.y & 0x7fff7fffu),
                                   __vmaxu2(u0.z & 0x7fff7fffu, u0.w & 0x7fff7fffu)),
                          __vmaxu2(__vmaxu2(u1.x & 0x7fff7fffu, u1.y & 0x7fff7fffu),
                                   __vmaxu2(u1.z & 0x7fff7fffu, u1.w & 0x7fff7fffu)));
    a = max(a & 0xffffu, a >> 16);
#pragma unroll
    for (int s = 1; s < 8; s <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, s));
    if (a >= 0x7f80u) set_error(hdr, SB_ENONFINITE);
    const uint32_t byte = e8m0_of_amax(a);
    const float inv = e8m0_inverse(byte);
    if (live) {
      float v[16];
      float v0[8], v1[8];
      unpack8(u0, v0);
      unpack8(u1, v1);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v0[i] * inv, v[8 + i] = v1[i] * inv;
      *reinterpret_cast<uint4*>(codes + m * K + k) =
          make_uint4(cvt_e4m3x4(v[0], v[1], v[2], v[3]), cvt_e4m3x4(v[4], v[5], v[6], v[7]),
                     cvt_e4m3x4(v[8], v[9], v[10], v[11]), cvt_e4m3x4(v[12], v[13], v[14], v[15]));
    }
    const uint32_t w = __shfl_sync(0xffffffffu, byte, 0) | (__shfl_sync(0xffffffffu, byte, 8) << 8) |
                       (__shfl_sync(0xffffffffu, byte, 16) << 16) | (__shfl_sync(0xffffffffu, byte, 24) << 24);
    if (lane == 0) sf[((m >> 7) * groups + g) * 128 + (m & 31) * 4 + ((m & 127) >> 5)] = w;
  }
}

cudaError_t launch_fp8_encode(const void* X, int64_t M, int64_t K, const int32_t* prec, uint8_t* codes, uint8_t* sf,
                              void* hdr, cudaStream_t s) {
  const int64_t tasks = ceil_div(M, 128) * 128 * ceil_div(K, 512);
  const int64_t want = ceil_div(tasks, 8), most = (int64_t)device_sm_count() * 8;
  k_fp8_encode<<<(unsigned)(want < most ? want : most), 256, 0, s>>>(
      static_cast<const __nv_bfloat16*>(X), M, (int)K, prec, codes, reinterpret_cast<uint32_t*>(sf),
      static_cast<WsHeader*>(hdr));
  return cudaGetLastError();
}

__device__ __forceinline__ float sf_value(const uint8_t* sf, int64_t row, int k, int groups) {
  const uint32_t b = sf[((row >> 7) * groups + k / 512) * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4 + (k / 128 & 3)];
  return b == 0 ? 0x1p-127f : __uint_as_float(b << 23);
}

__device__ __forceinline__ float gelu_tanh(float v) {
  return 0.5f * v * (1.0f + tanhf(0.7978845608028654f * (v + 0.044715f * v * v * v)));
}

// One 64 x 64 output tile per block, 4 x 4 outputs per thread, both operands decoded to FP32.
__global__ void __launch_bounds__(256) k_fp8_linear(Fp8Linear p) {
  if (p.prec && *p.prec == SB_SKIP) return;
  __shared__ float As[64][65], Bs[64][65];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t m0 = (int64_t)blockIdx.x * 64;
  const int n0 = blockIdx.y * 64;
  const int K = (int)p.K, groups = (K + 511) / 512;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += 64) {
    for (int i = threadIdx.x; i < 64 * 64; i += 256) {
      const int r = i >> 6, c = i & 63;
      const int64_t m = m0 + r;
      const int64_t n = n0 + r;
      As[r][c] = m < p.M ? e4m3_to_f32(p.A[m * K + k0 + c]) * sf_value(p.sfA, m, k0, groups) : 0.0f;
      Bs[r][c] = n < p.N ? e4m3_to_f32(p.W[n * K + k0 + c]) * sf_value(p.sfW, n, k0, groups) : 0.0f;
    }
    __syncthreads();
    for (int c = 0; c < 64; ++c) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += As[ty * 4 + i][c] * Bs[tx * 4 + j][c];
    }
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m >= p.M || n >= p.N) continue;
      float y = acc[i][j] + (p.bias ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[n]) : 0.0f);
      if (p.epilogue == SB_EPI_GELU_TANH) y = gelu_tanh(y);
      if (p.out_dtype == SB_OUT_F32)
        static_cast<float*>(p.Y)[m * p.N + n] = y;
      else
        static_cast<__nv_bfloat16*>(p.Y)[m * p.N + n] = __float2bfloat16_rn(y);
    }
  }
}

cudaError_t launch_fp8_linear(const Fp8Linear& p, cudaStream_t s, const char** why) {
  *why = "sb_linear_fp8 (encode)";
  if (p.X) {
    const cudaError_t e = launch_fp8_encode(p.X, p.M, p.K, p.prec, p.A, p.sfA, p.hdr, s);
    if (e != cudaSuccess) return e;
  }
  *why = "sb_linear_fp8";
  k_fp8_linear<<<dim3((unsigned)ceil_div(p.M, 64), (unsigned)ceil_div(p.N, 64)), 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace sb
