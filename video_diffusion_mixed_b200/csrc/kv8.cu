// kv8.cu -- FP8 key/value cache: the store of new tokens.
#include "launch_util.h"
#include "sb_device.cuh"
#include "sb_kernels.h"

namespace sb {

__device__ __forceinline__ uint32_t kv_e8m0(uint32_t bits) {
  return (uint32_t)max((int)(bits >> 7) - 8 + ((bits & 0x7fu) > 0x60u ? 1 : 0), 0);
}
__device__ __forceinline__ float kv_pow2(int byte) {  // 2^(byte - 127)
  return byte <= 0 ? 0x1p-127f : __uint_as_float((uint32_t)byte << 23);
}
__device__ __forceinline__ uint32_t kv_codes4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

constexpr int kKvBlock = 64;  // positions that share a scale

// One block of 128 threads per (cache block, keys or values, head, sequence). A thread keeps its
// share of the block's new elements (at most 64 x 128 / 128 = 64 of them, 8 at a time) in registers
// between the maximum and the codes. The block owns its 64 positions and their exponent, so no two
// blocks write the same bytes.
__global__ void __launch_bounds__(128) k_kv8_store(Kv8Store p) {
  __shared__ uint32_t red[4];
  if (p.prec && *p.prec == SB_SKIP) return;
  const int D = p.c.dim, vec = D / 8;
  const int which = blockIdx.y & 1;
  const int64_t h = blockIdx.y >> 1, b = blockIdx.z;
  const int held = __ldcg(p.c.lens + b);
  const int64_t st = p.start ? p.start[b] : held, cnt = p.counts ? p.counts[b] : p.n;
  const bool good = held >= 0 && held <= p.c.capacity && st >= 0 && st <= held && cnt >= 0 && cnt <= p.n &&
                    st + cnt <= p.c.capacity;
  const int64_t blk = st / kKvBlock + blockIdx.x;
  const int64_t lo = max(st, blk * kKvBlock), hi = min(st + cnt, (blk + 1) * kKvBlock);
  if (good && lo < hi) {
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(which ? p.v : p.k);
    const int64_t sb = which ? p.vs[0] : p.ks[0], stok = which ? p.vs[1] : p.ks[1], sh = which ? p.vs[2] : p.ks[2];
    src += b * sb + h * sh;
    uint8_t* codes = (which ? p.c.v_codes : p.c.k_codes) + ((b * p.c.heads + h) * p.c.capacity + blk * kKvBlock) * D;
    uint8_t* ep = (which ? p.c.v_exp : p.c.k_exp) + (b * p.c.heads + h) * (p.c.capacity / kKvBlock) + blk;
    uint4 u[8];
    uint32_t a = 0;
    const int first = (int)(lo - blk * kKvBlock), last = (int)(hi - blk * kKvBlock);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = threadIdx.x + 128 * i, tok = e / vec;
      u[i] = make_uint4(0, 0, 0, 0);
      if (tok >= first && tok < last)
        u[i] = __ldg(reinterpret_cast<const uint4*>(src + (blk * kKvBlock + tok - st) * stok + (e - tok * vec) * 8));
      const uint32_t m = __vmaxu2(__vmaxu2(u[i].x & 0x7fff7fffu, u[i].y & 0x7fff7fffu),
                                  __vmaxu2(u[i].z & 0x7fff7fffu, u[i].w & 0x7fff7fffu));
      a = max(a, max(m & 0xffffu, m >> 16));
    }
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, s));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
    const int old = first > 0 ? *ep : 0;  // before the barrier: thread 0 writes it below
    __syncthreads();
    a = max(max(red[0], red[1]), max(red[2], red[3]));
    const int need = (int)kv_e8m0(a);
    const int e8 = first > 0 ? max(old, need) : need;
    const float inv = __uint_as_float((254u - (uint32_t)e8) << 23);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = threadIdx.x + 128 * i, tok = e / vec;
      uint2* dst = reinterpret_cast<uint2*>(codes + (int64_t)e * 8);
      if (tok >= first && tok < last) {
        float v[8];
        unpack8(u[i], v);
        *dst = make_uint2(kv_codes4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                          kv_codes4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
      } else if (tok < first && e8 > old) {  // earlier tokens of the block, to the larger exponent
        const uint2 c = *dst;
        const float f = kv_pow2(127 + old - e8);
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] = e4m3_to_f32(c.x >> (8 * j)) * f;
          v[4 + j] = e4m3_to_f32(c.y >> (8 * j)) * f;
        }
        *dst = make_uint2(kv_codes4(v[0], v[1], v[2], v[3]), kv_codes4(v[4], v[5], v[6], v[7]));
      }
    }
    if (threadIdx.x == 0) {
      *ep = (uint8_t)e8;
      if (a >= 0x7f80u) set_error(p.hdr, SB_ENONFINITE);
    }
  }
  // The last block of the launch moves the lengths: every thread of every block has read them by
  // then (the barrier, before the block's ticket).
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    if (!good && blockIdx.x == 0 && blockIdx.y == 0) set_error(p.hdr, SB_ESHAPE);
    const uint32_t all = gridDim.x * gridDim.y * gridDim.z;
    red[0] = atomicAdd(&p.hdr->ticket[TICKET_KV], 1u) == all - 1 ? 1u : 0u;
    if (red[0]) p.hdr->ticket[TICKET_KV] = 0;
  }
  __syncthreads();
  if (red[0]) {
    for (int64_t i = threadIdx.x; i < p.c.batch; i += 128) {
      const int held_i = p.c.lens[i];
      const int64_t s_i = p.start ? p.start[i] : held_i, c_i = p.counts ? p.counts[i] : p.n;
      if (held_i >= 0 && held_i <= p.c.capacity && s_i >= 0 && s_i <= held_i && c_i >= 0 && c_i <= p.n &&
          s_i + c_i <= p.c.capacity)
        p.c.lens[i] = (int)(s_i + c_i);
    }
  }
}

cudaError_t launch_kv8_store(const Kv8Store& p, cudaStream_t s) {
  const dim3 grid((unsigned)((p.n + 62) / 64 + 1), (unsigned)(2 * p.c.heads), (unsigned)p.c.batch);
  k_kv8_store<<<grid, 128, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace sb
