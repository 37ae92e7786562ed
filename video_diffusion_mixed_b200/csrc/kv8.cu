// kv8.cu -- FP8 key/value cache: the store of new tokens.
#include "e4m3.cuh"
#include "launch_util.h"
#include "sb_device.cuh"
#include "sb_kernels.h"

namespace sb {

constexpr int kKvBlock = 64;  // positions that share a scale

// An item is one cache block (64 positions) of the keys or the values of one head of one sequence, taken
// by 128 threads; neighbouring items are the heads of the same tokens, whose rows lie next to one another
// in k and v. Each new element is read once (2 bytes) and written once (1 byte); DRAM is at two fifths of its
// rate, since a block has no load in flight while its warps meet and write. A thread
// keeps its share of the item's new elements (at most 64 x 128 / 128 = 64 of them, 8 at a time) in registers
// between the maximum and the codes. An item owns its positions and their exponent, so no two write the
// same bytes. Blocks loop over the items: one ticket an item (for the lengths, below) cost more than the
// copy, 67 us for 17550 tokens of 30 heads of 64 against 43 us
// (4.6 TB/s).
constexpr int kStoreThreads = 128;

struct StoreSpan {
  int64_t st, cnt;
  bool good;
};
__device__ __forceinline__ StoreSpan store_span(const Kv8Store& p, int64_t b) {
  StoreSpan s;
  const int held = __ldcg(p.c.lens + b);
  s.st = p.start ? p.start[b] : held;
  s.cnt = p.counts ? p.counts[b] : p.n;
  s.good = held >= 0 && held <= p.c.capacity && s.st >= 0 && s.st <= held && s.cnt >= 0 && s.cnt <= p.n &&
           s.st + s.cnt <= p.c.capacity;
  return s;
}

template <int D>
__global__ void __launch_bounds__(kStoreThreads) k_kv8_store(Kv8Store p, int64_t items) {
  __shared__ uint32_t red[2][4];
  if (p.prec && *p.prec == SB_SKIP) return;
  constexpr int kVec = D / 8, kPer = kKvBlock * kVec / kStoreThreads;
  const int64_t heads2 = 2 * p.c.heads, per_seq = ((p.n + 62) / 64 + 1) * heads2;
  int turn = 0;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t b = item / per_seq, in = item - b * per_seq, nth = in / heads2, hw = in - nth * heads2;
    const bool values = hw >= p.c.heads;
    const int64_t h = values ? hw - p.c.heads : hw;
    const StoreSpan sp = store_span(p, b);
    if (!sp.good) {
      if (in == 0 && threadIdx.x == 0) set_error(p.hdr, SB_ESHAPE);
      continue;
    }
    const int64_t blk = sp.st / kKvBlock + nth;
    const int64_t lo = max(sp.st, blk * kKvBlock), hi = min(sp.st + sp.cnt, (blk + 1) * kKvBlock);
    if (lo >= hi) continue;
    const int64_t* strides = values ? p.vs : p.ks;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(values ? p.v : p.k) + b * strides[0] + h * strides[2];
    const int64_t stok = strides[1];
    uint8_t* codes = (values ? p.c.v_codes : p.c.k_codes) + ((b * p.c.heads + h) * p.c.capacity + blk * kKvBlock) * D;
    uint8_t* ep = (values ? p.c.v_exp : p.c.k_exp) + (b * p.c.heads + h) * (p.c.capacity / kKvBlock) + blk;
    const int first = (int)(lo - blk * kKvBlock), last = (int)(hi - blk * kKvBlock);
    uint4 u[kPer];
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = threadIdx.x + kStoreThreads * i, tok = e / kVec;
      u[i] = make_uint4(0, 0, 0, 0);
      if (tok >= first && tok < last)
        u[i] = ldg_nc_v4(src + (blk * kKvBlock + tok - sp.st) * stok + (e - tok * kVec) * 8);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t m = __vmaxu2(__vmaxu2(u[i].x & 0x7fff7fffu, u[i].y & 0x7fff7fffu),
                                  __vmaxu2(u[i].z & 0x7fff7fffu, u[i].w & 0x7fff7fffu));
      a = max(a, max(m & 0xffffu, m >> 16));
    }
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, s));
    if ((threadIdx.x & 31) == 0) red[turn][threadIdx.x >> 5] = a;
    const int old = first > 0 ? *ep : 0;  // before the barrier: thread 0 writes it below
    __syncthreads();                      // two sets of maxima in turn: one barrier an item
    a = max(max(red[turn][0], red[turn][1]), max(red[turn][2], red[turn][3]));
    const int need = (int)e8m0_of_amax(a);
    const int e8 = first > 0 ? max(old, need) : need;
    const float inv = e8m0_inverse((uint32_t)e8);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = threadIdx.x + kStoreThreads * i, tok = e / kVec;
      uint2* dst = reinterpret_cast<uint2*>(codes + (int64_t)e * 8);
      if (tok >= first && tok < last) {
        float v[8];
        unpack8(u[i], v);
        *dst = make_uint2(cvt_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                          cvt_e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
      } else if (tok < first && e8 > old) {  // earlier tokens of the block, to the larger exponent
        const uint2 c = *dst;
        const float f = pow2_byte(127 + old - e8);
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] = e4m3_to_f32(c.x >> (8 * j)) * f;
          v[4 + j] = e4m3_to_f32(c.y >> (8 * j)) * f;
        }
        *dst = make_uint2(cvt_e4m3x4(v[0], v[1], v[2], v[3]), cvt_e4m3x4(v[4], v[5], v[6], v[7]));
      }
    }
    if (threadIdx.x == 0) {
      *ep = (uint8_t)e8;
      if (a >= 0x7f80u) set_error(p.hdr, SB_ENONFINITE);
    }
    turn ^= 1;  // only where the barrier was passed
  }
  // The last block of the launch moves the lengths: every thread of every block has read them by
  // then (the barrier, before the block's ticket).
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    red[0][0] = atomicAdd(&p.hdr->ticket[TICKET_KV], 1u) == gridDim.x - 1 ? 1u : 0u;
    if (red[0][0]) p.hdr->ticket[TICKET_KV] = 0;
  }
  __syncthreads();
  if (red[0][0]) {
    for (int64_t i = threadIdx.x; i < p.c.batch; i += kStoreThreads) {
      const StoreSpan sp = store_span(p, i);
      if (sp.good) p.c.lens[i] = (int)(sp.st + sp.cnt);
    }
  }
}

cudaError_t launch_kv8_store(const Kv8Store& p, cudaStream_t s) {
  const int64_t items = ((p.n + 62) / 64 + 1) * 2 * p.c.heads * p.c.batch, most = (int64_t)device_sm_count() * 12;
  const unsigned grid = (unsigned)(items < most ? items : most);
  if (p.c.dim == 64)
    k_kv8_store<64><<<grid, kStoreThreads, 0, s>>>(p, items);
  else
    k_kv8_store<128><<<grid, kStoreThreads, 0, s>>>(p, items);
  return cudaGetLastError();
}

}  // namespace sb
