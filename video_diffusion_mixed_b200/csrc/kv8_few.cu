// kv8_few.cu -- attention over the FP8 key/value cache for few query rows (at most 16 for a key head:
// the tokens being generated), and the join of partial results.
//
// Bound by reading the visible part of the cache once (2 D bytes a token and head), so the keys are
// split over many blocks and each warp streams 32-token steps of its block's share on its own: a thread
// copies (cp.async) and reads back its own pieces, three steps deep, with no barrier before the end.
// The products run on 16-row matrix instructions in fp16 (codes are exact there) with FP32 sums:
//
//   S [16 rows x 8 tokens] += Q K^T: a thread's fragment holds one token's channels 16t + 4i .. + 3 of a
//      64-channel chunk (the order of a contraction is free), 16 contiguous bytes of the cache;
//   O [16 rows x 8 channels] += w V: the weights are already the left operand's fragment; on the right a
//      thread takes D / 8 contiguous channels of four tokens, so column g of tile i is channel
//      g D / 8 + i, and the bytes of two neighbouring tokens are interleaved to fp16 pairs.
//
// Block scales, the running maximum and its rare moves are those of the tensor-core kernel beside it.
#include "kv8.cuh"
#include "launch_util.h"
#include "sb_device.cuh"
#include "sb_kernels.h"

namespace sb {
namespace kv8 {

constexpr int kFewWarps = 4;
constexpr int kFewThreads = kFewWarps * 32;
constexpr int kFewSlots = 3;
constexpr int kStep = 32;  // tokens

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float fast_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <int BYTES>
__device__ __forceinline__ void cp_async_or_zero(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(live ? BYTES : 0)
               : "memory");
}

template <int D>
struct FewSlot {  // one step of every warp; [thread] is that thread's own
  uint4 k[4][D / 64][kFewThreads];                    // token 8j + g, channels 64c + 16t .. + 15
  uint8_t v[2][4][kFewThreads][D / 8];                // tokens 16s + {2t, 2t+1, 2t+8, 2t+9}, channels g D/8 ..
};

// WIDE: 9 to 16 rows; otherwise the lower half of the matrix instruction's rows stays empty.
template <int D, bool WIDE>
__global__ void __launch_bounds__(kFewThreads) k_kv8_few(const Kv8Attn p, int splits, float* part) {
  extern __shared__ __align__(16) uint8_t few_smem[];
  FewSlot<D>* ring = reinterpret_cast<FewSlot<D>*>(few_smem);
  constexpr int kR = WIDE ? 2 : 1;  // rows g (and g + 8) of this thread
  constexpr int kC = D / 64, kN = D / 8;
  if (p.prec && *p.prec == SB_SKIP) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int group = (int)(p.heads_q / p.c.heads);
  const int split = blockIdx.x;
  const int64_t hk = blockIdx.y, b = blockIdx.z;
  const Span sp = sequence_span(p, b);
  if (split == 0 && hk == 0 && tid == 0 && sp.bad) set_error(p.hdr, SB_ESHAPE);
  const int rows = sp.nq * group;
  if (rows == 0) return;
  const int pmin = sp.pos(0), pmax = sp.pos(sp.nq - 1);
  const KeyTiles kt = key_tiles(p, pmin, pmax, 64);
  const int i0 = (int)((int64_t)kt.n * split / splits), i1 = (int)((int64_t)kt.n * (split + 1) / splits);
  const int steps = 2 * (i1 - i0);
  const int64_t head0 = (b * p.c.heads + hk) * p.c.capacity;
  const uint8_t* kc = p.c.k_codes + head0 * D;
  const uint8_t* vc = p.c.v_codes + head0 * D;
  const uint8_t* kx = p.c.k_exp + head0 / 64;
  const uint8_t* vx = p.c.v_exp + head0 / 64;

  auto fetch = [&](int slot, int q) {
    if (q < steps) {
      FewSlot<D>& o = ring[slot];
      const int j0 = kt.tile(i0 + (q >> 1)) * 64 + (q & 1) * kStep;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int tok = j0 + 8 * j + g;
#pragma unroll
        for (int c = 0; c < kC; ++c)
          cp_async_or_zero<16>(smem_u32(&o.k[j][c][tid]), kc + (int64_t)tok * D + 64 * c + 16 * t, tok < sp.len);
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = j0 + 16 * s + 2 * t + (i & 1) + 8 * (i >> 1);
          cp_async_or_zero<kN>(smem_u32(&o.v[s][i][tid][0]), vc + (int64_t)tok * D + kN * g, tok < sp.len);
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int u = 0; u < kFewSlots; ++u) fetch(u, warp + u * kFewWarps);

  // queries: rows g and g + 8 as the left operand
  uint32_t qf[kC][4][2][kR];
  float qc[kR];
  int pos[kR];
#pragma unroll
  for (int h = 0; h < kR; ++h) {
    const int r = g + 8 * h;
    const bool live = r < rows;
    const int tok = live ? r / group : 0;
    const int64_t hq = hk * group + (live ? r - tok * group : 0);
    pos[h] = live ? sp.pos(tok) : -1;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + b * p.qs[0] + tok * p.qs[1] + hq * p.qs[2];
    uint4 u[kC][2];
    uint32_t a = 0;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        u[c][i] = live ? __ldg(reinterpret_cast<const uint4*>(q + 64 * c + 16 * t) + i) : make_uint4(0, 0, 0, 0);
        a = __vmaxu2(a, __vmaxu2(__vmaxu2(u[c][i].x & 0x7fff7fffu, u[c][i].y & 0x7fff7fffu),
                                 __vmaxu2(u[c][i].z & 0x7fff7fffu, u[c][i].w & 0x7fff7fffu)));
      }
    }
    a = max(a & 0xffffu, a >> 16);
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
    float f;
    qc[h] = query_scale(p.scale, a, f);
#pragma unroll
    for (int c = 0; c < kC; ++c) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v[8];
        unpack8(u[c][i], v);
        qf[c][2 * i][0][h] = pack_f16(v[0] * f, v[1] * f);
        qf[c][2 * i][1][h] = pack_f16(v[2] * f, v[3] * f);
        qf[c][2 * i + 1][0][h] = pack_f16(v[4] * f, v[5] * f);
        qf[c][2 * i + 1][1][h] = pack_f16(v[6] * f, v[7] * f);
      }
    }
  }
  // the largest exponent of V over the block's share (after the first copies are on their way)
  const int blocks = (sp.len + 63) >> 6;
  int evmax = 0;
  for (int i = lane; i < i1 - i0; i += 32) {
    const int blk = kt.tile(i0 + i);
    if (blk < blocks) evmax = max(evmax, (int)vx[blk]);
  }
#pragma unroll
  for (int s = 16; s >= 1; s >>= 1) evmax = max(evmax, __shfl_xor_sync(0xffffffffu, evmax, s));

  float m[kR], l[kR], o[kN][2 * kR];
#pragma unroll
  for (int h = 0; h < kR; ++h) m[h] = -INFINITY, l[h] = 0.0f;
#pragma unroll
  for (int i = 0; i < kN; ++i)
#pragma unroll
    for (int h = 0; h < 2 * kR; ++h) o[i][h] = 0.0f;

  int slot = 0;
  for (int q = warp; q < steps; q += kFewWarps) {
    const int blk = kt.tile(i0 + (q >> 1)), j0 = blk * 64 + (q & 1) * kStep;
    const int ke = blk < blocks ? (int)__ldg(kx + blk) : 127, ve = blk < blocks ? (int)__ldg(vx + blk) : 0;
    asm volatile("cp.async.wait_group %0;" ::"n"(kFewSlots - 1) : "memory");
    const FewSlot<D>& d = ring[slot];
    float x[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float acc[4] = {};
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const uint4 w = d.k[j][c][tid];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t k = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
          mma_16816(acc, qf[c][i][0][0], WIDE ? qf[c][i][0][kR - 1] : 0u, qf[c][i][1][0],
                    WIDE ? qf[c][i][1][kR - 1] : 0u, e4m3x2_f16x2(k), e4m3x2_f16x2(k >> 16));
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) x[j][i] = acc[i];
    }
    const int rel = max(ve - evmax, -64);
    const float ev = (float)rel, iv = __uint_as_float((uint32_t)(127 - rel) << 23);
    const bool mask = tile_needs_mask(p, j0, kStep, pmin, pmax);
    uint32_t w[4][kR];
#pragma unroll
    for (int h = 0; h < kR; ++h) {
      if (mask) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (!key_visible(p, pos[h], j0 + 8 * j + 2 * t + i)) x[j][2 * h + i] = -INFINITY;
      }
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) mx = max3(mx, x[j][2 * h], x[j][2 * h + 1]);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float c = fminf(fmaxf(qc[h] * pow2_byte(ke), 0x1p-126f), 0x1p126f);
      const float mn = fmaxf(m[h], fmaf(mx, c, ev));
      if (__any_sync(0xffffffffu, mn > m[h] + kRise)) {
        const float f = mn == m[h] ? 1.0f : fast_ex2(m[h] - mn);
        m[h] = mn;
        l[h] *= f;
#pragma unroll
        for (int i = 0; i < kN; ++i) o[i][2 * h] *= f, o[i][2 * h + 1] *= f;
      }
      const float add = ev - (m[h] == -INFINITY ? 0.0f : m[h]);
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = fast_ex2(fmaf(x[j][2 * h], c, add)), e = fast_ex2(fmaf(x[j][2 * h + 1], c, add));
        sum += a + e;
        w[j][h] = pack_f16(a, e);
      }
      l[h] = fmaf(sum, iv, l[h]);
    }
    const bool far = ve < evmax - 64;  // more than 2^64 below the largest block: counts as zero
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int c = 0; c < kN / 4; ++c) {  // four channels of four tokens
        uint32_t e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = far ? 0u : *reinterpret_cast<const uint32_t*>(&d.v[s][i][tid][4 * c]);
        const uint32_t p0 = __byte_perm(e[0], e[1], 0x5140), p1 = __byte_perm(e[0], e[1], 0x7362);
        const uint32_t r0 = __byte_perm(e[2], e[3], 0x5140), r1 = __byte_perm(e[2], e[3], 0x7362);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t lo = i < 2 ? p0 : p1, hi = i < 2 ? r0 : r1;
          float acc[4];
#pragma unroll
          for (int h = 0; h < 4; ++h) acc[h] = h < 2 * kR ? o[4 * c + i][h < 2 * kR ? h : 0] : 0.0f;
          mma_16816(acc, w[2 * s][0], WIDE ? w[2 * s][kR - 1] : 0u, w[2 * s + 1][0], WIDE ? w[2 * s + 1][kR - 1] : 0u,
                    e4m3x2_f16x2(i & 1 ? lo >> 16 : lo), e4m3x2_f16x2(i & 1 ? hi >> 16 : hi));
#pragma unroll
          for (int h = 0; h < 2 * kR; ++h) o[4 * c + i][h] = acc[h];
        }
      }
    }
    fetch(slot, q + kFewSlots * kFewWarps);  // this thread has read its pieces of the slot
    slot = slot + 1 == kFewSlots ? 0 : slot + 1;
  }
  cp_async_wait_all();

  // join the warps: sums over the lanes of a row, then warp after warp in shared memory
#pragma unroll
  for (int h = 0; h < kR; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
  }
  __syncthreads();  // the ring's memory is reused
  float* sm = reinterpret_cast<float*>(few_smem);  // [warp][row] m, then l, then [warp][row][D] outputs
  float* sl = sm + kFewWarps * 16;
  float* so = sl + kFewWarps * 16;
#pragma unroll
  for (int h = 0; h < kR; ++h) {
    const int r = g + 8 * h;
    if (t == 0) sm[warp * 16 + r] = m[h], sl[warp * 16 + r] = l[h];
#pragma unroll
    for (int i = 0; i < kN; ++i)  // accumulator columns 2t, 2t + 1 of tile i: channels kN * column + i
#pragma unroll
      for (int e = 0; e < 2; ++e) so[(warp * 16 + r) * (D + 4) + kN * (2 * t + e) + i] = o[i][2 * h + e];
  }
  __syncthreads();
  const float unit = __uint_as_float((uint32_t)max(evmax, 1) << 23);
  for (int i = tid; i < rows * (D / 4); i += kFewThreads) {
    const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) mx = fmaxf(mx, sm[w * 16 + r]);
    float tot = 0.0f, y[4] = {};
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      const float mw = sm[w * 16 + r], f = mw == -INFINITY ? 0.0f : fast_ex2(mw - mx);
      const float* src = so + (w * 16 + r) * (D + 4) + c;
      tot = fmaf(sl[w * 16 + r], f, tot);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = fmaf(src[e], f, y[e]);
    }
    // nothing visible: zeros and -inf; a NaN row has a NaN sum and stays NaN
    const float inv = tot > 0.0f ? unit / tot : tot;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] *= inv;
    const float lse2 = tot > 0.0f ? mx + log2f(tot) : tot == 0.0f ? -INFINITY : tot;
    const int tok = r / group;
    const int64_t hq = hk * group + r - tok * group;
    if (splits == 1) {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + b * p.os[0] + tok * p.os[1] + hq * p.os[2] + c;
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(__float_as_uint(y[0]), __float_as_uint(y[1])),
                                                  pack_bf16x2(__float_as_uint(y[2]), __float_as_uint(y[3])));
      if (p.lse && c == 0) p.lse[(b * p.heads_q + hq) * p.n_q + tok] = lse2 * 0.6931471805599453f;
    } else {
      *reinterpret_cast<float4*>(part_row(p, part, split, b, hk, r) + c) = make_float4(y[0], y[1], y[2], y[3]);
      if (c == 0) *part_lse(p, part, splits, split, b, hk, r) = lse2;
    }
  }
}

// Joins the parts of a row: out = sum 2^(lse_s - max) o_s / sum 2^(lse_s - max). A warp per row, a lane D / 32
// channels; parts that saw no key have lse -inf.
template <int D>
__global__ void __launch_bounds__(128) k_kv8_join(const Kv8Attn p, int splits, float* part) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (p.prec && *p.prec == SB_SKIP) return;
  const int lane = threadIdx.x & 31;
  const int group = (int)(p.heads_q / p.c.heads);
  const int64_t per = p.n_q * group;  // rows of a sequence and key head
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (i >= part_rows(p)) return;
  const int64_t bh = i / per, r = i - bh * per, b = bh / p.c.heads, hk = bh - b * p.c.heads;
  const int64_t tok = r / group, hq = hk * group + r - tok * group;
  if (tok >= sequence_span(p, b).nq) return;
  float mx = -INFINITY;
  bool nan = false;
  for (int s = lane; s < splits; s += 32) {
    const float v = __ldcg(part_lse(p, part, splits, s, b, hk, r));
    nan = nan || v != v;
    mx = fmaxf(mx, v);
  }
  mx = warp_max_f32(mx);
  nan = __any_sync(0xffffffffu, nan);
  float tot = 0.0f, y[D / 32] = {};
  if (mx != -INFINITY || nan) {
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      const float f = fast_ex2(__ldcg(part_lse(p, part, splits, s, b, hk, r)) - mx);
      const float* src = part_row(p, part, s, b, hk, r) + lane * (D / 32);
      tot += f;
      if constexpr (D == 128) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
        y[0] = fmaf(v.x, f, y[0]), y[1] = fmaf(v.y, f, y[1]), y[2] = fmaf(v.z, f, y[2]), y[3] = fmaf(v.w, f, y[3]);
      } else {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
        y[0] = fmaf(v.x, f, y[0]), y[1] = fmaf(v.y, f, y[1]);
      }
    }
  }
  const float inv = tot > 0.0f ? 1.0f / tot : tot;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + b * p.os[0] + tok * p.os[1] + hq * p.os[2] + lane * (D / 32);
#pragma unroll
  for (int c = 0; c < D / 64; ++c)
    reinterpret_cast<uint32_t*>(dst)[c] =
        pack_bf16x2(__float_as_uint(y[2 * c] * inv), __float_as_uint(y[2 * c + 1] * inv));
  if (p.lse && lane == 0)
    p.lse[(b * p.heads_q + hq) * p.n_q + tok] =
        tot > 0.0f ? (mx + log2f(tot)) * 0.6931471805599453f : nan ? NAN : -INFINITY;
}

template <int D, bool WIDE>
static cudaError_t launch_few(const Kv8Attn& p, int splits, float* part, cudaStream_t s) {
  constexpr int kBytes = (int)(kFewSlots * sizeof(FewSlot<D>));
  static_assert(kBytes >= (int)sizeof(float) * (kFewWarps * 16 * 2 + kFewWarps * 16 * (D + 4)), "join in the ring");
  static std::atomic<uint64_t> attr{0};
  const cudaError_t e = smem_attr_once(k_kv8_few<D, WIDE>, kBytes, attr);
  if (e != cudaSuccess) return e;
  k_kv8_few<D, WIDE><<<dim3((unsigned)splits, (unsigned)p.c.heads, (unsigned)p.c.batch), kFewThreads, kBytes, s>>>(
      p, splits, part);
  return cudaGetLastError();
}

// How the keys of a call are split. Few rows: enough blocks that their reads fill the memory's queue on
// every SM, at least 256 tokens each. Many rows: the number of parts with the shortest schedule of 148
// CTAs, a part costing its key tiles and about three more for its start and its join.
static int plan_splits(int64_t batch, int64_t heads, int64_t heads_q, int64_t n_q, int dim, int64_t keys) {
  const int64_t rows = n_q * (heads_q / heads), units = batch * heads;
  const int64_t most = ((int64_t)128 << 20) / (batch * n_q * heads_q * dim * 4);  // 128 MB of partial results
  if (rows <= kFewRows) {
    const int64_t want = ceil_div(1184, units), fit = keys / 256;
    int64_t s = want < fit ? want : fit;
    s = s < most ? s : most;
    return (int)(s > 1 ? s : 1);
  }
  const int64_t tiles = ceil_div(rows, 256) * units, len = ceil_div(keys, 128);
  int best = 1;
  int64_t cost = ceil_div(tiles, 148) * len * 16;
  for (int s = 2; s <= 16 && s <= most && s * 4 <= len; ++s) {
    const int64_t c = ceil_div(tiles * s, 148) * (len * 16 / s + 48) + 48;
    if (c < cost) cost = c, best = s;
  }
  return best;
}

}  // namespace kv8

cudaError_t launch_kv8_attention(const Kv8Attn& p, void* part_, cudaStream_t s, const char** why) {
  using namespace kv8;
  *why = "sb_kv8_attention";
  float* part = static_cast<float*>(part_);
  const int64_t rows = p.n_q * (p.heads_q / p.c.heads);
  int64_t keys = p.c.capacity;
  if (p.window > 0 && p.window + p.sinks + p.n_q < keys) keys = p.window + p.sinks + p.n_q;
  const int splits = plan_splits(p.c.batch, p.c.heads, p.heads_q, p.n_q, p.c.dim, keys);
  cudaError_t e;
  if (rows <= kFewRows) {
    if (p.c.dim == 64)
      e = rows <= 8 ? launch_few<64, false>(p, splits, part, s) : launch_few<64, true>(p, splits, part, s);
    else
      e = rows <= 8 ? launch_few<128, false>(p, splits, part, s) : launch_few<128, true>(p, splits, part, s);
  } else {
    e = launch_kv8_tiles(p, splits, part, s, why);
  }
  if (e != cudaSuccess || splits == 1) return e;
  *why = "sb_kv8_attention (join)";
  const LaunchAfter L((unsigned)ceil_div(part_rows(p), 4), 128, 0, s, true);
  return p.c.dim == 64 ? cudaLaunchKernelEx(&L.cfg, k_kv8_join<64>, p, splits, part)
                       : cudaLaunchKernelEx(&L.cfg, k_kv8_join<128>, p, splits, part);
}

// The most that any number of key heads and any capacity need.
size_t kv8_workspace_bytes(int64_t batch, int64_t heads_q, int64_t n_q, int dim) {
  int64_t most = 0;
  for (int64_t heads = 1; heads <= heads_q; ++heads) {
    if (heads_q % heads) continue;
    const int64_t s = kv8::plan_splits(batch, heads, heads_q, n_q, dim, (int64_t)1 << 30);
    if (s > most) most = s;
  }
  const int64_t rows = batch * n_q * heads_q;
  return kKv8PartOffset + (most > 1 ? (size_t)(most * rows * (dim + 1) * 4 + 15) / 16 * 16 : 0);
}

}  // namespace sb
