// kv8_few.cu -- attention over the FP8 key/value cache for few query rows (at most 16 for a key head:
// the tokens being generated), and the join of partial results.
//
// Bound by reading the visible part of the cache once (2 D bytes a token and head). The 64-token tiles of
// all sequences and key heads, one after the other, are dealt out evenly to one wave of blocks, whatever
// the lengths: a block's share may end in the middle of a head (the parts are joined afterwards) and hold
// several heads. Within a share of a head each warp streams 32-token steps on its own: one TMA box of keys
// and one of values a step, three steps deep, no barrier between warps before the end.
// The products run on 16 x 8 matrix instructions in fp16 (codes are exact there) with FP32 sums, with the
// cache on the side of 16 and the query rows on the side of 8, so that few rows waste little:
//
//   S^T [16 tokens x 8 rows] += K Q^T: a thread's fragment holds a token's channels 16t + 4i .. + 3 of a
//      64-channel chunk (the order of a contraction is free), 16 contiguous bytes of the cache;
//   O^T [16 channels x 8 rows] += V^T w^T: a thread takes D / 8 contiguous channels of four tokens; the bytes
//      of two neighbouring tokens are interleaved to fp16 pairs, and the weights change from S^T's
//      fragment to a right operand by 8 x 8 transposes in the register file.
//
// Block scales, the running maximum and its rare moves are those of the tensor-core kernel beside it.
//
// Measured (32 query heads, 8 key heads of 128, one token): 131071 tokens of one sequence 56 us (4.8 TB/s, the
// join included), 32 sequences of 8191 tokens 95 us (5.7 TB/s), of 1 to 8191 tokens 75; 30 heads of 64, 17776
// tokens 24 us. A block a head, with no join, takes 86 us for the 32 equal sequences but 84 for the mixed ones
// (the longest block sets the time) and leaves most of the chip idle with few sequences. A long cache's
// stream runs at 5.6 TB/s; the start and the join are 8 us of the 56.
#include <cudaTypedefs.h>

#include <algorithm>

#include "kv8.cuh"
#include "launch_util.h"
#include "sb_device.cuh"
#include "sb_kernels.h"
#include "tmap.h"

namespace sb {
namespace kv8 {

constexpr int kFewWarps = 4;
constexpr int kFewThreads = kFewWarps * 32;
constexpr int kFewSlots = 3;
constexpr int kStep = 32;  // tokens
constexpr uint64_t kFewWaitNs = 2000000000ull;  // far above any legitimate wait
constexpr uint64_t kFewDrainNs = 20000000ull;

__device__ __forceinline__ uint32_t transpose8(uint32_t a) {  // 8 x 8 matrix of 16-bit values
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

struct FewMaps {
  CUtensorMap k, v;  // {dim, capacity, batch * heads}, box of kStep tokens
};

// Byte `c` of token row `r` in a box: rows of 128 bytes under the 128B swizzle, of 64 under the 64B one.
template <int D>
__device__ __forceinline__ uint32_t box_addr(uint32_t box, int r, int c) {
  const int x = D == 128 ? r & 7 : (r >> 1) & 3;
  return box + (uint32_t)(r * D + (((c >> 4) ^ x) << 4) + (c & 15));
}

// The tiles of one sequence's key head: at least one, which shows a query that it sees nothing.
__device__ __forceinline__ int few_tiles(const Kv8Attn& p, const Span& sp) {
  if (sp.nq == 0) return 0;
  return max(1, key_tiles(p, sp.pos(0), sp.pos(sp.nq - 1), 64).n);
}

// Blocks that get a share: one for every four tiles, as far as they go. Block c begins at tile floor(c total /
// shares), which spreads the larger shares over the chip: with all of them in front the long sequence above
// took 56 us. In 32 bits where they do (a cache has fewer than 2^31 tiles, rem c is below 592^2).
struct FewDeal {
  int total, shares, base, rem;
  __device__ __forceinline__ FewDeal(int total_, int blocks) : total(total_) {
    shares = max(1, min(blocks, (total - 1) / 4 + 1));
    base = total / shares;
    rem = total - base * shares;
  }
  __device__ __forceinline__ int first(int c) const { return c * base + c * rem / shares; }
  __device__ __forceinline__ int owner(int t) const {  // the largest c with first(c) <= t
    return (int)((((int64_t)t + 1) * shares - 1) / total);
  }
};

// A place in the row of all tiles (sequence after sequence, key head after key head).
struct FewPlace {
  int total;   // tiles of all
  int before;  // tiles before sequence b
  int b, n;    // the sequence, and the tiles of one of its key heads
};
// Thirty-two sequences from b0 on, one a lane: its tiles, and the range of all its heads' tiles behind `base`.
struct FewLane {
  int n, start, end;
};
__device__ __forceinline__ FewLane few_lane(const Kv8Attn& p, int b0, int base, int lane, bool report) {
  FewLane f;
  const int b = b0 + lane;
  f.n = 0;
  if (b < p.c.batch) {
    const Span sp = sequence_span(p, b);
    if (report && sp.bad) set_error(p.hdr, SB_ESHAPE);
    f.n = few_tiles(p, sp);
  }
  int sum = f.n;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, sum, s);
    if (lane >= s) sum += v;
  }
  f.end = base + sum * (int)p.c.heads;
  f.start = f.end - f.n * (int)p.c.heads;
  return f;
}
__device__ __forceinline__ void few_pick(const FewLane& l, int b0, bool here, FewPlace& f) {
  const unsigned hit = __ballot_sync(0xffffffffu, here);
  if (hit) {
    const int src = __ffs(hit) - 1;
    f.b = b0 + src;
    f.n = __shfl_sync(0xffffffffu, l.n, src);
    f.before = __shfl_sync(0xffffffffu, l.start, src);
  }
}
// Whole warps: the place of tile t, or (seq >= 0) of a sequence. Reads every length: the host deals out
// at most kFewUnits sequences.
__device__ __forceinline__ FewPlace few_place(const Kv8Attn& p, int t, int seq, int lane) {
  FewPlace f{0, 0, -1, 0};
  for (int b0 = 0; b0 < (int)p.c.batch; b0 += 32) {
    const FewLane l = few_lane(p, b0, f.total, lane, false);
    few_pick(l, b0, seq >= 0 ? b0 + lane == seq : t >= l.start && t < l.end, f);
    f.total = __shfl_sync(0xffffffffu, l.end, 31);
  }
  return f;
}
// Block c of `blocks`: its share [at, at_end) of all tiles and the place of the first; false when it has none.
__device__ __forceinline__ bool few_deal(const Kv8Attn& p, int c, int blocks, int lane, bool report, int& at,
                                         int& at_end, FewPlace& f) {
  FewLane l;
  f = FewPlace{0, 0, -1, 0};
  for (int b0 = 0; b0 < (int)p.c.batch; b0 += 32) {
    l = few_lane(p, b0, f.total, lane, report);
    f.total = __shfl_sync(0xffffffffu, l.end, 31);
  }
  const FewDeal d(f.total, blocks);
  if (c >= d.shares) return false;
  at = d.first(c);
  at_end = d.first(c + 1);
  if (at >= at_end) return false;
  if (p.c.batch <= 32)
    few_pick(l, 0, at >= l.start && at < l.end, f);
  else
    f = few_place(p, at, -1, lane);
  return true;
}
// Partial results: a block has at most two, of the head that it takes over and of the one it hands on.
__device__ __forceinline__ float* few_part(float* part, int D, int64_t block, int side, int r) {
  return part + ((block * 2 + side) * kFewRows + r) * D;
}
__device__ __forceinline__ float* few_part_lse(float* part, int D, int blocks, int64_t block, int side, int r) {
  return part + (int64_t)blocks * 2 * kFewRows * D + (block * 2 + side) * kFewRows + r;
}

template <int D>
constexpr int few_smem() {
  return kFewWarps * kFewSlots * 2 * kStep * D + 1024 + kFewWarps * kFewSlots * 8;
}

// A share's rows again, one by one in FP32: its values may hold a NaN, which only rows that see it may meet. A warp
// takes every fourth row.
template <int D>
__device__ __noinline__ void few_redo(const Kv8Attn& p, int64_t b, int64_t hk, KeyTiles kt, int i0, int i1, int tiles,
                                      float* qs, float* part) {
  const int lane = threadIdx.x & 31, c = lane * (D / 32);
  const Span sp = sequence_span(p, b);
  const int group = (int)(p.heads_q / p.c.heads), rows = sp.nq * group;
#pragma unroll 1
  for (int r = (int)threadIdx.x >> 5; r < rows; r += kFewWarps) {
    const int64_t tok = r / group, hq = hk * group + r - tok * group;
    ExactRow<D> row;
    exact_row<D>(p, b, hk, tok, hq, sp.len, sp.pos((int)tok), kt, 64, i0, i1, qs, row);
    if (i1 - i0 == tiles) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + b * p.os[0] + tok * p.os[1] +
                                                  hq * p.os[2] + c);
#pragma unroll
      for (int e = 0; e < D / 64; ++e)
        dst[e] = pack_bf16x2(__float_as_uint(row.y[2 * e]), __float_as_uint(row.y[2 * e + 1]));
      if (p.lse && lane == 0) p.lse[(b * p.heads_q + hq) * p.n_q + tok] = row.lse2 * 0.6931471805599453f;
    } else {
      const int side = i0 > 0 ? 0 : 1;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) few_part(part, D, blockIdx.x, side, r)[c + e] = row.y[e];
      if (lane == 0) *few_part_lse(part, D, gridDim.x, blockIdx.x, side, r) = row.lse2;
    }
  }
}

// NT tiles of eight query rows. deal: the tiles are dealt out as above; otherwise a block takes one head.
template <int D, int NT>
__global__ void __launch_bounds__(kFewThreads) k_kv8_few(const __grid_constant__ FewMaps tm,
                                                         const __grid_constant__ Kv8Attn p, int deal, float* part) {
  extern __shared__ uint8_t few_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(few_smem_raw) + 1023) & ~(uintptr_t)1023);
  constexpr int kC = D / 64, kN = D / 8, kBox = kStep * D;
  if (p.prec && *p.prec == SB_SKIP) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int group = (int)(p.heads_q / p.c.heads);
  int at = 0, at_end = 0;
  FewPlace place{0, 0, 0, 0};
  if (deal && !few_deal(p, blockIdx.x, gridDim.x, lane, blockIdx.x == 0 && warp == 0, at, at_end, place)) return;

  // this warp's ring: slot s holds a box of keys, then one of values
  const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * kFewSlots * 2 * kBox);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kFewWarps * kFewSlots * 2 * kBox) + warp * kFewSlots;
  if (lane == 0) {
    for (int u = 0; u < kFewSlots; ++u) mbar_init(&full[u], 1);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  __syncwarp();
  int slot = 0;  // the ring goes on from head to head
  uint32_t ph = 0;
  bool late = false;

  while (true) {
    // this head's share: tiles i0 .. i1 - 1 of its `tiles`
    int64_t hk, b;
    int i0, i1, tiles;
    if (deal) {
      if (at >= place.before + place.n * (int)p.c.heads) place = few_place(p, at, -1, lane);  // the next sequence
      const int in = at - place.before, h = in / place.n;
      b = place.b;
      hk = h;
      tiles = place.n;
      i0 = in - h * tiles;
      i1 = min(tiles, i0 + (at_end - at));
    } else {
      b = blockIdx.x / p.c.heads;
      hk = blockIdx.x - b * p.c.heads;
      const Span sp = sequence_span(p, b);
      if (hk == 0 && tid == 0 && sp.bad) set_error(p.hdr, SB_ESHAPE);
      tiles = few_tiles(p, sp);
      if (tiles == 0) return;
      i0 = 0;
      i1 = tiles;
    }
    const Span sp = sequence_span(p, b);
    const int rows = sp.nq * group;
    const int pmin = sp.pos(0), pmax = sp.pos(sp.nq - 1);
    const KeyTiles kt = key_tiles(p, pmin, pmax, 64);  // none: tile 0, where every key is masked
    const int steps = 2 * (i1 - i0);
    const int head = (int)(b * p.c.heads + hk);
    const uint8_t* kx = p.c.k_exp + (int64_t)head * (p.c.capacity / 64);
    const uint8_t* vx = p.c.v_exp + (int64_t)head * (p.c.capacity / 64);
    auto fetch = [&](int into, int q) {  // one lane
      if (q >= steps) return;
      const int j0 = kt.tile(i0 + (q >> 1)) * 64 + (q & 1) * kStep;
      const uint32_t box = ring + (uint32_t)(into * 2 * kBox), bar = smem_u32(&full[into]);
      mbar_arrive_expect_tx(&full[into], 2 * kBox);
      tma_load_3d(box, &tm.k, bar, 0, j0, head);
      tma_load_3d(box + kBox, &tm.v, bar, 0, j0, head);
    };
    if (lane == 0) {
      for (int u = 0; u < kFewSlots; ++u) fetch((slot + u) % kFewSlots, warp + u * kFewWarps);
    }
    __syncwarp();

    // queries as the right operand: row 8n + g, channels 64c + 16t + 4i .. + 3
    uint32_t qf[NT][kC][4][2];
    float qc[NT][2];  // rows 8n + 2t, 8n + 2t + 1
    int pos[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = g + 8 * n;
      const bool live = r < rows;
      const int tok = live ? r / group : 0;
      const int64_t hq = hk * group + (live ? r - tok * group : 0);
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
      const float back = query_scale(p.scale, a, f);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = 8 * n + 2 * t + e;
        qc[n][e] = __shfl_sync(0xffffffffu, back, 4 * (2 * t + e));
        pos[n][e] = rr < rows ? sp.pos(rr / group) : -1;
      }
#pragma unroll
      for (int c = 0; c < kC; ++c) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float v[8];
          unpack8(u[c][i], v);
          qf[n][c][2 * i][0] = pack_f16(v[0] * f, v[1] * f);
          qf[n][c][2 * i][1] = pack_f16(v[2] * f, v[3] * f);
          qf[n][c][2 * i + 1][0] = pack_f16(v[4] * f, v[5] * f);
          qf[n][c][2 * i + 1][1] = pack_f16(v[6] * f, v[7] * f);
        }
      }
    }
    const int e0 = (int)__ldg(vx + kt.tile(i0));  // exponents of V are taken relative to the share's first
    float o[kN / 2][NT][4];
    RowStats st[NT][2];  // l: this lane's tokens
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) st[n][e] = RowStats{-INFINITY, 0.0f, 0};
#pragma unroll
    for (int i = 0; i < kN / 2; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][n][e] = 0.0f;

    bool redo = false;
    for (int q = warp; q < steps; q += kFewWarps) {
      const int blk = kt.tile(i0 + (q >> 1)), j0 = blk * 64 + (q & 1) * kStep;
      const int ke = (int)__ldg(kx + blk), ve = (int)__ldg(vx + blk);  // a tile starts below len
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full[slot], ph, nullptr, kFewWaitNs))) {
        if (lane == 0) set_error(p.hdr, SB_ETIMEOUT);
        late = true;
        break;
      }
      const uint32_t kbox = ring + (uint32_t)(slot * 2 * kBox), vbox = kbox + kBox;
      float x[2][NT][4];  // tokens 16a + g (rows 2t, 2t + 1), 16a + g + 8
#pragma unroll
      for (int a = 0; a < 2; ++a) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[a][n][e] = 0.0f;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          const uint4 lo = ld_shared_v4(box_addr<D>(kbox, 16 * a + g, 64 * c + 16 * t));
          const uint4 hi = ld_shared_v4(box_addr<D>(kbox, 16 * a + g + 8, 64 * c + 16 * t));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t k0 = i == 0 ? lo.x : i == 1 ? lo.y : i == 2 ? lo.z : lo.w;
            const uint32_t k1 = i == 0 ? hi.x : i == 1 ? hi.y : i == 2 ? hi.z : hi.w;
            const uint32_t a0 = e4m3x2_f16x2(k0), a1 = e4m3x2_f16x2(k1);
            const uint32_t a2 = e4m3x2_f16x2(k0 >> 16), a3 = e4m3x2_f16x2(k1 >> 16);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_16816(x[a][n], a0, a1, a2, a3, qf[n][c][i][0], qf[n][c][i][1]);
          }
        }
      }
      const int rel = ve - e0;
      redo |= ve >= kNanExp;
      const float ev = (float)rel, ks = pow2_byte(ke);
      const bool mask = tile_needs_mask(p, j0, kStep, pmin, pmax);
      uint32_t w[2][NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (mask) {
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (!key_visible(p, pos[n][e], j0 + 16 * a + 8 * h + g)) x[a][n][2 * h + e] = -INFINITY;
          }
          float mx = fmaxf(fmaxf(x[0][n][e], x[0][n][2 + e]), fmaxf(x[1][n][e], x[1][n][2 + e]));
#pragma unroll
          for (int s = 4; s < 32; s <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
          const float c = fminf(fmaxf(qc[n][e] * ks, 0x1p-126f), 0x1p126f);
          RowStats& r = st[n][e];
          const float mn = fmaxf(r.m, fmaf(mx, c, ev));
          f[e] = 1.0f;
          if (mn > r.m + kRise) {
            f[e] = fast_ex2(r.m - mn);
            move_max(r, mn, rel);
          }
          const int below = r.e - rel;
          float sum = 0.0f;
          if (below > kFar) {
            const float base = far_base(r, mx, c);
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
              for (int h = 0; h < 2; ++h) r.l += fast_ex2(fmaf(x[a][n][2 * h + e], c, base));
          }
          const float add = ev + (float)kShift - (r.m == -INFINITY ? 0.0f : r.m);
#pragma unroll
          for (int a = 0; a < 2; ++a) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              x[a][n][2 * h + e] = fast_ex2(fmaf(x[a][n][2 * h + e], c, add));
              sum += x[a][n][2 * h + e];
            }
          }
          if (below <= kFar) r.l = fmaf(sum, sum_factor(below), r.l);
        }
        if (__any_sync(0xffffffffu, f[0] != 1.0f || f[1] != 1.0f)) {
#pragma unroll
          for (int i = 0; i < kN / 2; ++i) {
            o[i][n][0] *= f[0], o[i][n][1] *= f[1];
            o[i][n][2] *= f[0], o[i][n][3] *= f[1];
          }
        }
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int h = 0; h < 2; ++h) w[a][n][h] = transpose8(pack_f16(x[a][n][2 * h], x[a][n][2 * h + 1]));
      }
      const int fine = sp.len - j0;  // codes past the end are zeroed: they may be NaN, which no weight of zero hides
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        uint32_t e[4][kN / 4];  // tokens 16a + {2t, 2t+1, 2t+8, 2t+9}, channels kN g ..
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = 16 * a + 2 * t + (i & 1) + 8 * (i >> 1);
          const uint32_t addr = box_addr<D>(vbox, tok, kN * g);
          if constexpr (D == 128) {
            const uint4 v = ld_shared_v4(addr);
            e[i][0] = v.x, e[i][1] = v.y, e[i][2] = v.z, e[i][3] = v.w;
          } else {
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(e[i][0]), "=r"(e[i][1]) : "r"(addr));
          }
          if (fine < kStep && tok >= fine) {
#pragma unroll
            for (int c = 0; c < kN / 4; ++c) e[i][c] = 0u;
          }
        }
#pragma unroll
        for (int c = 0; c < kN / 4; ++c) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // channels 4c + 2h (row g) and 4c + 2h + 1 (row g + 8)
            const uint32_t lo = __byte_perm(e[0][c], e[1][c], h ? 0x7362 : 0x5140);
            const uint32_t hi = __byte_perm(e[2][c], e[3][c], h ? 0x7362 : 0x5140);
            const uint32_t a0 = e4m3x2_f16x2(lo), a1 = e4m3x2_f16x2(lo >> 16);
            const uint32_t a2 = e4m3x2_f16x2(hi), a3 = e4m3x2_f16x2(hi >> 16);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_16816(o[2 * c + h][n], a0, a1, a2, a3, w[a][n][0], w[a][n][1]);
          }
        }
      }
      __syncwarp();  // every lane has read the slot
      if (lane == 0) fetch(slot, q + kFewSlots * kFewWarps);
      if (++slot == kFewSlots) slot = 0, ph ^= 1u;
    }
    if (late) {  // what is still in flight lands before the memory is used again
      for (int u = 0; u < kFewSlots; ++u, ph ^= slot == kFewSlots - 1, slot = slot + 1 == kFewSlots ? 0 : slot + 1)
        mbar_wait_bounded(&full[slot], ph, nullptr, kFewDrainNs);
    }
    // the last share: the joining launch may come up (it waits for this one's end itself)
    if (deal && at + (i1 - i0) >= at_end) asm volatile("griddepcontrol.launch_dependents;");

    // join the warps: sums over the lanes of a row, then warp after warp in shared memory
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) st[n][e].l += __shfl_xor_sync(0xffffffffu, st[n][e].l, s);
    const bool again = __syncthreads_or(redo);  // the ring's memory is reused
    constexpr int kRows = 8 * NT;
    float* so = reinterpret_cast<float*>(smem);  // [warp][row][D + 4] outputs, then [warp][row] statistics
    RowStats* ss = reinterpret_cast<RowStats*>(so + kFewWarps * kRows * (D + 4));
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * n + 2 * t + e;
        if (g == 0) ss[warp * kRows + r] = st[n][e];
#pragma unroll
        for (int i = 0; i < kN / 2; ++i)
          *reinterpret_cast<float2*>(&so[(warp * kRows + r) * (D + 4) + kN * g + 2 * i]) =
              make_float2(o[i][n][e], o[i][n][2 + e]);
      }
    }
    __syncthreads();
    for (int i = again ? rows * (D / 4) : tid; i < rows * (D / 4); i += kFewThreads) {
      const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
      RowStats all{-INFINITY, 0.0f, 0};
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) {
        const RowStats one = ss[w * kRows + r];
        if (one.m > all.m) all.m = one.m, all.e = one.e;
      }
      int down = 0;  // the joint sum's exponent gives way to the warp whose sum counts most
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) {
        const RowStats one = ss[w * kRows + r];
        const float y = one.m - all.m + (float)(all.e - one.e);
        if (one.m != -INFINITY && y > 0.0f) down = max(down, min(__float2int_ru(y), 512));
      }
      all.e -= down;
      float y[4] = {};
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) {
        const RowStats one = ss[w * kRows + r];
        const bool none = one.m == -INFINITY;  // a sum of zero, or NaN
        const float f = none ? 0.0f : fast_ex2(one.m - all.m);
        const float4 v = *reinterpret_cast<const float4*>(so + (w * kRows + r) * (D + 4) + c);
        all.l = fmaf(one.l, none ? 0.0f : fast_ex2(one.m - all.m + (float)(all.e - one.e)), all.l);
        y[0] = fmaf(v.x, f, y[0]), y[1] = fmaf(v.y, f, y[1]), y[2] = fmaf(v.z, f, y[2]), y[3] = fmaf(v.w, f, y[3]);
      }
      // nothing visible: zeros and -inf; a NaN row has a NaN sum and stays NaN
      const float inv = all.l > 0.0f ? 1.0f / all.l : all.l;
      const float2 unit = output_unit(all.e, e0);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = y[e] * unit.x * inv * unit.y;
      const float lse2 = all.l > 0.0f ? all.m - (float)all.e + log2f(all.l) : all.l == 0.0f ? -INFINITY : all.l;
      const int tok = r / group;
      const int64_t hq = hk * group + r - tok * group;
      if (i1 - i0 == tiles) {  // the whole head
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + b * p.os[0] + tok * p.os[1] + hq * p.os[2] + c;
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(__float_as_uint(y[0]), __float_as_uint(y[1])),
                                                    pack_bf16x2(__float_as_uint(y[2]), __float_as_uint(y[3])));
        if (p.lse && c == 0) p.lse[(b * p.heads_q + hq) * p.n_q + tok] = lse2 * 0.6931471805599453f;
      } else {
        const int side = i0 > 0 ? 0 : 1;  // taken over from the block before, or handed on
        *reinterpret_cast<float4*>(few_part(part, D, blockIdx.x, side, r) + c) = make_float4(y[0], y[1], y[2], y[3]);
        if (c == 0) *few_part_lse(part, D, gridDim.x, blockIdx.x, side, r) = lse2;
      }
    }
    if (again) {
      float* qs = reinterpret_cast<float*>(ss + kFewWarps * kRows) + warp * D;
      few_redo<D>(p, b, hk, kt, i0, i1, tiles, qs, part);
    }
    at += i1 - i0;
    if (!deal || at >= at_end) break;
    fence_proxy_async_smem();  // the join's memory is the ring's again
    if (__syncthreads_or(late)) break;
  }
}

// One joined row: a lane writes its D / 32 channels.
template <int D>
__device__ __forceinline__ void put_joined(const Kv8Attn& p, int64_t b, int64_t hq, int64_t tok, int lane,
                                           const float (&y)[D / 32], float tot, float mx) {
  const float inv = tot > 0.0f ? 1.0f / tot : tot;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + b * p.os[0] + tok * p.os[1] +
                                              hq * p.os[2] + lane * (D / 32));
#pragma unroll
  for (int c = 0; c < D / 64; ++c)
    dst[c] = pack_bf16x2(__float_as_uint(y[2 * c] * inv), __float_as_uint(y[2 * c + 1] * inv));
  if (p.lse && lane == 0)
    p.lse[(b * p.heads_q + hq) * p.n_q + tok] =
        tot > 0.0f ? (mx + log2f(tot)) * 0.6931471805599453f : tot == 0.0f ? -INFINITY : tot;
}

// Joins the parts of a dealt-out head: out = sum 2^(lse - max) o / sum 2^(lse - max). A block per row; its
// warps take the parts in turn, a lane D / 32 channels, and meet in shared memory in a fixed order. Parts
// that saw no key have lse -inf.
template <int D>
__global__ void __launch_bounds__(256) k_kv8_join_few(const Kv8Attn p, int blocks, float* part) {
  __shared__ float sy[8][D], st[8];
  constexpr int kE = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (p.prec && *p.prec == SB_SKIP) return;
  const int group = (int)(p.heads_q / p.c.heads);
  const int64_t per = p.n_q * group;  // rows of a sequence and key head
  const int64_t bh = blockIdx.x / per, b = bh / p.c.heads, hk = bh - b * p.c.heads;
  const int r = (int)(blockIdx.x - bh * per), tok = r / group;
  const int64_t hq = hk * group + r - tok * group;
  if (tok >= sequence_span(p, b).nq) return;
  const FewPlace f = few_place(p, -1, (int)b, lane);
  const FewDeal d(f.total, blocks);
  const int t0 = f.before + (int)hk * f.n, c0 = d.owner(t0), c1 = d.owner(t0 + f.n - 1);
  if (c0 == c1) return;  // one block had the whole head
  const int parts = c1 - c0 + 1;
  float mx = -INFINITY;
  for (int s = lane; s < parts; s += 32) mx = fmaxf(mx, __ldcg(few_part_lse(part, D, blocks, c0 + s, s == 0, r)));
  mx = warp_max_f32(mx);  // NaN parts are ignored here and make the sums NaN below
  const float base = mx == -INFINITY ? 0.0f : mx;
  float tot = 0.0f, y[kE] = {};
#pragma unroll 4
  for (int s = warp; s < parts; s += 8) {
    const float w = fast_ex2(__ldcg(few_part_lse(part, D, blocks, c0 + s, s == 0, r)) - base);
    const float* src = few_part(part, D, c0 + s, s == 0, r) + lane * kE;
    tot += w;
    if constexpr (D == 128) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
      y[0] = fmaf(v.x, w, y[0]), y[1] = fmaf(v.y, w, y[1]), y[2] = fmaf(v.z, w, y[2]), y[3] = fmaf(v.w, w, y[3]);
    } else {
      const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
      y[0] = fmaf(v.x, w, y[0]), y[1] = fmaf(v.y, w, y[1]);
    }
  }
#pragma unroll
  for (int e = 0; e < kE; ++e) sy[warp][lane * kE + e] = y[e];
  if (lane == 0) st[warp] = tot;
  __syncthreads();
  if (warp != 0) return;
  tot = 0.0f;
#pragma unroll
  for (int e = 0; e < kE; ++e) y[e] = 0.0f;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    tot += st[w];
#pragma unroll
    for (int e = 0; e < kE; ++e) y[e] += sy[w][lane * kE + e];
  }
  put_joined<D>(p, b, hq, tok, lane, y, tot, mx);
}

// The same for the parts of the tensor-core kernel: many rows, few parts, a warp a row.
template <int D>
__global__ void __launch_bounds__(256) k_kv8_join(const Kv8Attn p, int splits, float* part) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (p.prec && *p.prec == SB_SKIP) return;
  constexpr int kE = D / 32;
  const int lane = threadIdx.x & 31;
  const int group = (int)(p.heads_q / p.c.heads);
  const int64_t per = p.n_q * group;  // rows of a sequence and key head
  const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= part_rows(p)) return;
  const int64_t bh = i / per, r = i - bh * per, b = bh / p.c.heads, hk = bh - b * p.c.heads;
  const int64_t tok = r / group, hq = hk * group + r - tok * group;
  if (tok >= sequence_span(p, b).nq) return;
  const float mine = lane < splits ? __ldcg(part_lse(p, part, splits, lane, b, hk, r)) : -INFINITY;
  const float mx = warp_max_f32(mine);  // NaN parts are ignored here and make the sums NaN below
  const float weight = fast_ex2(mine - (mx == -INFINITY ? 0.0f : mx));
  float tot = 0.0f, y[kE] = {};
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {  // at most 16
    const float w = __shfl_sync(0xffffffffu, weight, s);
    const float* src = part_row(p, part, s, b, hk, r) + lane * kE;
    tot += w;
    if constexpr (D == 128) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
      y[0] = fmaf(v.x, w, y[0]), y[1] = fmaf(v.y, w, y[1]), y[2] = fmaf(v.z, w, y[2]), y[3] = fmaf(v.w, w, y[3]);
    } else {
      const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
      y[0] = fmaf(v.x, w, y[0]), y[1] = fmaf(v.y, w, y[1]);
    }
  }
  put_joined<D>(p, b, hq, tok, lane, y, tot, mx);
}

static bool cache_map(CUtensorMap* m, const uint8_t* base, const sb_kv8& c) {
  auto fn = tmap_encoder();
  cuuint64_t dims[3] = {(cuuint64_t)c.dim, (cuuint64_t)c.capacity, (cuuint64_t)(c.batch * c.heads)};
  cuuint64_t strides[2] = {(cuuint64_t)c.dim, (cuuint64_t)(c.dim * c.capacity)};
  cuuint32_t box[3] = {(cuuint32_t)c.dim, kStep, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, c.dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NT>
static cudaError_t launch_few(const Kv8Attn& p, int deal, unsigned grid, float* part, cudaStream_t s) {
  constexpr int kBytes = few_smem<D>() + 1024;  // + alignment of the dynamic base
  static_assert(kFewSlots * kFewWarps * 2 * kStep * D >=
                    kFewWarps * (8 * NT * ((int)sizeof(RowStats) + 4 * (D + 4)) + 4 * D),
                "the join fits the ring");
  static std::atomic<uint64_t> attr{0};
  const cudaError_t e = smem_attr_once(k_kv8_few<D, NT>, kBytes, attr);
  if (e != cudaSuccess) return e;
  FewMaps tm;
  if (!cache_map(&tm.k, p.c.k_codes, p.c) || !cache_map(&tm.v, p.c.v_codes, p.c)) return cudaErrorInvalidValue;
  k_kv8_few<D, NT><<<grid, kFewThreads, kBytes, s>>>(tm, p, deal, part);
  return cudaGetLastError();
}

// Few rows: one wave of the blocks that fit (two an SM with heads of 128, four with 64); with many heads
// (four waves of them) a block each, which is as even and needs no join: 200 sequences of 4096 tokens with 8
// key heads of 128 259 us (6.5 TB/s).
constexpr int64_t kFewUnits = 1184;
static int few_blocks(int dim) { return dim == 64 ? 592 : 296; }

// Many rows: the number of parts of the keys, as many as the capacity and the window allow (the lengths are on the
// device), with the shortest schedule of 148 CTAs; a part costs its key
// tiles and about six more (10 us) for its start and its end, and its results two passes over memory. 1350
// tokens of 30 heads of 64 that see 11026 keys: 1 / 2 / 3 / 4 / 6 / 8 parts took 332 / 289 / 281 / 284 / 312 / 338 us.
constexpr int kMaxSplits = 16;
constexpr int64_t kPartBytes = (int64_t)128 << 20;  // of partial outputs, at most
static int plan_splits(int64_t batch, int64_t heads, int64_t heads_q, int64_t n_q, int dim, int64_t keys) {
  const int64_t rows = n_q * (heads_q / heads), tiles = ceil_div(rows, 256) * batch * heads, len = ceil_div(keys, 128);
  const int64_t most = kPartBytes / (batch * n_q * heads_q * dim * 4);
  const int64_t join = batch * n_q * heads_q * dim * 4 / 400000;                  // of a part, in 1/16 key tiles (0.1 us)
  int best = 1;
  int64_t cost = ceil_div(tiles, 148) * (len * 16 + 96);
  for (int s = 2; s <= kMaxSplits && s <= most && s * 4 <= len; ++s) {
    const int64_t c = ceil_div(tiles * s, 148) * (len * 16 / s + 96) + 40 + s * join;
    if (c < cost) cost = c, best = s;
  }
  return best;
}

}  // namespace kv8

Kv8Plan kv8_plan(const Kv8Attn& p) {
  using namespace kv8;
  Kv8Plan plan{p.n_q * (p.heads_q / p.c.heads) <= kFewRows, false, 1, kKv8PartOffset};
  int64_t floats = 0;
  if (plan.few) {
    plan.deal = p.c.batch * p.c.heads < kFewUnits;
    if (plan.deal) floats = (int64_t)few_blocks(p.c.dim) * 2 * kFewRows * (p.c.dim + 1);
  } else {
    int64_t keys = p.c.capacity;
    if (p.window > 0 && p.window + p.sinks + p.n_q < keys) keys = p.window + p.sinks + p.n_q;
    plan.splits = plan_splits(p.c.batch, p.c.heads, p.heads_q, p.n_q, p.c.dim, keys);
    if (plan.splits > 1) floats = plan.splits * part_rows(p) * (p.c.dim + 1);
  }
  plan.bytes += (size_t)(floats * 4 + 15) / 16 * 16;
  return plan;
}

cudaError_t launch_kv8_attention(const Kv8Attn& p, const Kv8Plan& plan, void* part_, cudaStream_t s, const char** why) {
  using namespace kv8;
  *why = "sb_kv8_attention";
  float* part = static_cast<float*>(part_);
  const int64_t rows = p.n_q * (p.heads_q / p.c.heads), all = part_rows(p);
  if (plan.few) {
    const int deal = plan.deal;
    const unsigned grid = deal ? (unsigned)few_blocks(p.c.dim) : (unsigned)(p.c.batch * p.c.heads);
    cudaError_t e;
    if (p.c.dim == 64)
      e = rows <= 8 ? launch_few<64, 1>(p, deal, grid, part, s) : launch_few<64, 2>(p, deal, grid, part, s);
    else
      e = rows <= 8 ? launch_few<128, 1>(p, deal, grid, part, s) : launch_few<128, 2>(p, deal, grid, part, s);
    if (e != cudaSuccess || !deal) return e;
    *why = "sb_kv8_attention (join)";
    const LaunchAfter L((unsigned)all, 256, 0, s, true);
    return p.c.dim == 64 ? cudaLaunchKernelEx(&L.cfg, k_kv8_join_few<64>, p, (int)grid, part)
                         : cudaLaunchKernelEx(&L.cfg, k_kv8_join_few<128>, p, (int)grid, part);
  }
  const int splits = plan.splits;
  const cudaError_t e = launch_kv8_tiles(p, splits, part, s, why);
  if (e != cudaSuccess || splits == 1) return e;
  *why = "sb_kv8_attention (join)";
  const LaunchAfter L((unsigned)ceil_div(all, 8), 256, 0, s, true);
  return p.c.dim == 64 ? cudaLaunchKernelEx(&L.cfg, k_kv8_join<64>, p, splits, part)
                       : cudaLaunchKernelEx(&L.cfg, k_kv8_join<128>, p, splits, part);
}

// What any call of at most these sizes may need, whatever its key heads, capacity and window. A smaller call may
// need more than a larger one (it is split where the larger one fills the chip), so this is a bound over all of
// them: the dealt-out parts of a few rows, which a single token of a single sequence needs already, and as many parts
// of many rows as kMaxSplits and kPartBytes allow.
size_t kv8_workspace_bytes(int64_t batch, int64_t heads_q, int64_t n_q, int dim) {
  using namespace kv8;
  int64_t floats = (int64_t)few_blocks(dim) * 2 * kFewRows * (dim + 1);
  if (n_q * heads_q > kFewRows) {
    const int64_t rows = batch * n_q * heads_q, most = kPartBytes / (dim * 4);
    floats = std::max(floats, std::min(kMaxSplits * rows, most) * (dim + 1));
  }
  return kKv8PartOffset + (size_t)(floats * 4 + 15) / 16 * 16;
}

}  // namespace sb
