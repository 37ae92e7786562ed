// fp8.cu -- linear layer in 8-bit floating point: E4M3 codes with one E8M0 scale per 128 channels.
#include "e4m3.cuh"
#include "gemm_epi.cuh"
#include "launch_util.h"
#include "sb_device.cuh"
#include "sb_kernels.h"

namespace sb {

// One warp per (row, 512 channels): a lane takes 16 channels (two 16-byte loads, one 16-byte store of codes),
// eight lanes a block, whose maximum takes three shuffles; four blocks make one 32-bit word of scales. Rows past
// M up to the end of their atom get zero scales. Bound by memory (2 bytes read, 1 written an element):
// 17776 x 1920 19.6 us (5.2 TB/s).
__global__ void __launch_bounds__(256) k_fp8_encode(const __nv_bfloat16* __restrict__ X, int64_t M, int K,
                                                    const int32_t* prec, uint8_t* __restrict__ codes,
                                                    uint32_t* __restrict__ sf, WsHeader* hdr) {
  asm volatile("griddepcontrol.launch_dependents;");  // the product's launch waits for this one's writes itself
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

// ------------------------------------------------------------------------------------------------
// Few rows (M <= 8): a stream over the weight
// ------------------------------------------------------------------------------------------------

// 2^(a + b - 254) as two factors, so that no product in between leaves the range of FP32 when the
// result does not.
__device__ __forceinline__ float2 pow2_factors(uint32_t a, uint32_t b) {
  const int e = (int)(a + b) - 254, h = e >> 1;
  return make_float2(__uint_as_float((uint32_t)(h + 127) << 23), __uint_as_float((uint32_t)(e - h + 127) << 23));
}

// The product is bound by reading the weight once (N K bytes), so the tensor core's rows are weight
// rows and its eight columns are tokens: a block takes 16 weight rows, its four warps take the
// 128-channel blocks in turn, and the warps' sums meet in shared memory in a fixed order. Codes become
// fp16 (exact); a 128-channel sum is scaled by its two power-of-two scales when it is complete.
//
// A thread reads 16 consecutive channels of two weight rows and of one token: the order in which a
// product's channels are summed is free, so the fragment's channels 2t, 2t+1, 2t+8, 2t+9 of step i are
// channels 16t + 4i .. + 3 of both sides. The weight's codes go through shared memory only to be in flight
// without registers: each thread copies (cp.async) and reads back its own pieces, so no barrier is
// needed, and four K-blocks a warp, all of a block's with K up to 2048, are on their way at once; the scales
// and the tokens' codes follow in registers. 1 x 11520 x 1920 with the weight out of L2's reach: 8.2 us (2.7
// TB/s; 6.7 us from L2), 1 x 7680 x 16384 30 us (4.2 TB/s). With the tokens' codes and the scales in the ring
// too, which leaves room for two K-blocks in flight: 8.7 and 38 us; with all in registers 11.4.
constexpr int kRowWarps = 4;
constexpr int kRowThreads = kRowWarps * 32;
constexpr int kRowSlots = 4;

__global__ void __launch_bounds__(kRowThreads) k_fp8_rows(Fp8Linear p) {
  __shared__ uint4 wbuf[kRowSlots][4][kRowThreads];  // piece 2c + r: chunk c (64 channels), weight row g + 8r
  __shared__ float red[kRowWarps][8][17];
  if (p.prec && *p.prec == SB_SKIP) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int K = (int)p.K, M = (int)p.M, nkb = (K + 127) / 128, groups = (K + 511) / 512;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const uint8_t* w0 = p.W + (n0 + g) * K + 16 * t;
  const uint8_t* w1 = w0 + (int64_t)8 * K;
  const uint32_t* sfw = reinterpret_cast<const uint32_t*>(p.sfW) + (n0 >> 7) * groups * 128 + ((n0 & 31) + g) * 4 +
                        ((n0 & 127) >> 5);  // row n0 + g; row n0 + g + 8 is 32 words on
  const uint32_t* sfx = reinterpret_cast<const uint32_t*>(p.sfA);
  auto fetch_w = [&](int slot, int kb) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int k = kb * 128 + c * 64;
      if (k < K) {
        cp_async16(smem_u32(&wbuf[slot][2 * c][tid]), w0 + k);
        cp_async16(smem_u32(&wbuf[slot][2 * c + 1][tid]), w1 + k);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int u = 0; u < kRowSlots; ++u) fetch_w(u, warp + u * kRowWarps);
  float total[4] = {};
  bool waited = false;
  for (int kb0 = warp; kb0 < nkb; kb0 += kRowSlots * kRowWarps) {
    uint32_t sw[kRowSlots][2], sx[kRowSlots][2];
    uint4 x[kRowSlots][2];
#pragma unroll
    for (int u = 0; u < kRowSlots; ++u) {  // kb >> 2 is kb0 / 4 + u: a warp takes every fourth K-block
      const int kb = kb0 + u * kRowWarps;
      sw[u][0] = kb < nkb ? __ldg(sfw + (int64_t)(kb >> 2) * 128) : 0u;
      sw[u][1] = kb < nkb ? __ldg(sfw + (int64_t)(kb >> 2) * 128 + 32) : 0u;
    }
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");  // the tokens' codes come from the launch before
    waited = true;
#pragma unroll
    for (int u = 0; u < kRowSlots; ++u) {  // tokens past M read as zero
      const int kb = kb0 + u * kRowWarps;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int k = kb * 128 + c * 64, e = 2 * t + c;
        x[u][c] = k < K && g < M ? ldg_v4(p.A + (int64_t)g * K + k + 16 * t) : make_uint4(0, 0, 0, 0);
        sx[u][c] = kb < nkb && e < M ? __ldcg(sfx + (int64_t)(kb >> 2) * 128 + e * 4) : 0u;
      }
    }
#pragma unroll
    for (int u = 0; u < kRowSlots; ++u) {
      const int kb = kb0 + u * kRowWarps;
      asm volatile("cp.async.wait_group %0;" ::"n"(kRowSlots - 1) : "memory");
      if (kb < nkb) {
        float acc[4] = {};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (kb * 128 + c * 64 >= K) break;
          const uint4 wa = wbuf[u][2 * c][tid], wb = wbuf[u][2 * c + 1][tid], q = x[u][c];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a = i == 0 ? wa.x : i == 1 ? wa.y : i == 2 ? wa.z : wa.w;
            const uint32_t b = i == 0 ? wb.x : i == 1 ? wb.y : i == 2 ? wb.z : wb.w;
            const uint32_t y = i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w;
            mma_16816(acc, e4m3x2_f16x2(a), e4m3x2_f16x2(b), e4m3x2_f16x2(a >> 16), e4m3x2_f16x2(b >> 16),
                    e4m3x2_f16x2(y), e4m3x2_f16x2(y >> 16));
          }
        }
        const int sh = 8 * (kb & 3);
        const uint32_t e0 = (sw[u][0] >> sh) & 0xffu, e1 = (sw[u][1] >> sh) & 0xffu;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t ex = (sx[u][j] >> sh) & 0xffu;
          const float2 f0 = pow2_factors(ex, e0), f1 = pow2_factors(ex, e1);
          total[j] = fmaf(acc[j] * f0.x, f0.y, total[j]);
          total[2 + j] = fmaf(acc[2 + j] * f1.x, f1.y, total[2 + j]);
        }
      }
      fetch_w(u, kb + kRowSlots * kRowWarps);  // this thread has read its pieces of the slot
    }
  }
  cp_async_wait_all();
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    red[warp][2 * t + j][g] = total[j];
    red[warp][2 * t + j][g + 8] = total[2 + j];
  }
  __syncthreads();
  const int m = tid >> 4, r = tid & 15;  // 128 threads: 8 tokens x 16 outputs
  if (m >= M) return;
  float y = 0.0f;
#pragma unroll
  for (int w = 0; w < kRowWarps; ++w) y += red[w][m][r];
  if (p.bias) y += __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[n0 + r]);
  if (p.epilogue == SB_EPI_GELU_TANH) y = gelu_exp2(make_float2(y, 0.0f)).x;
  const int64_t o = (int64_t)m * p.N + n0 + r;
  if (p.out_dtype == SB_OUT_F32)
    static_cast<float*>(p.Y)[o] = y;
  else
    static_cast<__nv_bfloat16*>(p.Y)[o] = __float2bfloat16_rn(y);
}

cudaError_t launch_fp8_linear(const Fp8Linear& p, cudaStream_t s, const char** why) {
  *why = "sb_linear_fp8 (encode)";
  if (p.X) {
    const cudaError_t e = launch_fp8_encode(p.X, p.M, p.K, p.prec, p.A, p.sfA, p.hdr, s);
    if (e != cudaSuccess) return e;
  }
  // Up to one tile of tokens the stream wins: 4 x 1920 x 1920 4.2 us against 7.9 in the single form of
  // the tensor-core product, 1 x 11520 x 1920 8.2 against 9.2, 8 x 7680 x 1920 7.8 against 9.1; two tiles lost
  // (16 x 7680 x 1920: 11.0 against 8.3).
  if (p.M > 8) return launch_fp8_gemm(p, s, why);
  *why = "sb_linear_fp8";
  const LaunchAfter L((unsigned)(p.N / 16), kRowThreads, 0, s, p.X != nullptr);
  return cudaLaunchKernelEx(&L.cfg, k_fp8_rows, p);
}

}  // namespace sb
