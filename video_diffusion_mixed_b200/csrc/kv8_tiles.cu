// kv8_tiles.cu -- attention over the FP8 key/value cache for many query rows, on the tensor cores.
//
// A row is one query token of one query head; the rows of all query heads that share a key head stand
// together (row = token * group + head in the group), so a key tile serves all of them. A CTA takes 256
// rows (two tiles of 128, one warpgroup each) of one key head and a run of 128-token key tiles:
//
//   S = Q K^T       tcgen05 kind::f16, Q (fp16) in tensor memory, K in shared memory, S (FP32) in tensor memory
//   w = 2^(c S + ev - m), running maximum m and sum, one row a thread
//   O += w V        tcgen05 kind::f16, w (fp16) from tensor memory, O (FP32) in tensor memory
//
// Keys and values are E4M3 codes, which fp16 holds exactly, so a warpgroup turns each tile's codes into
// fp16 operands once for the 256 rows. The block scales are powers of two and never touch the tiles:
// the keys' enters c, the values' exponent ev the exponent of w, and with it the running maximum, which is
// that of what w V sums; the row sum takes it out again by an exact factor (RowStats in kv8.cuh). A block of
// values 2^64 below the largest before it is left out of the product, and if it holds anything but zeros, or if
// a block may hold a NaN, the CTA computes its rows again one by one in FP32: a branch for that in the
// softmax's loop, taken or not, cost a tenth of the time of 17776 x 17776, a second loop behind it as much.
// Queries are scaled by a power of two to [2^14, 2^15) and rounded to fp16, exact for every component within
// 2^-31 of the row's largest. The maximum moves only when it would rise by more than 2^8, so the accumulator is
// rescaled rarely; the rest of fp16's range, 2^7, is given to small weights.
//
// Warps: 0-3 and 4-7 softmax of the two row tiles, 8-11 codes -> fp16, 12 MMA issue. A key tile is taken in
// two steps of 64 keys (a scale block each); the weights overwrite their scores. The shared memory that
// feeds the MMAs is the scarcest resource, so Q, which every step multiplies, lives in tensor memory. With
// heads of 64 there is room for two score buffers a row tile, used in turn: the scores of step u + 2 are
// computed as soon as the weights of step u have been multiplied, and a softmax finds its next scores
// ready. With heads of 128 there is one. Every wait is bounded (SB_ETIMEOUT).
//
// Measured: 17776 tokens of 30 heads of 64 over 17776 keys 3.4 ms (710 TFLOP/s); 8192 over 8192 of 8 heads of 128
// 870 TFLOP/s, 980 with whole waves of CTAs. Bound by the hand-offs between a row tile's softmax and its two
// products, 110 to 220 cycles each way, which two row tiles and two buffers hide only in part: a probe without
// the exponentials (16 a clock and SM, three fifths of the time with heads of 64, a third with 128) was 13
// percent faster with heads of 64 and no faster with 128. A CTA's start and end (10 us, one CTA an SM) weigh on
// short key ranges. Where a block of values 2^100 larger sends the CTAs of 1350 tokens over 17776 keys to the
// row-by-row form, the call takes 72 ms instead of 0.37. With Q in shared memory it took 3.8 ms (772 TFLOP/s
// with heads of 128), with one score buffer besides 5.4. Tried and not kept: a second thread that issues MMAs, a
// fifth slower with 128; the two softmax groups taking turns and scores loaded a step ahead in registers, no
// faster; two threads a row, 535 TFLOP/s; the running maximum behind the exponentials, 622 (with heads of 128
// 887); one wave of CTAs with the tiles dealt out, whose inner loop was 12 percent slower: 3.9 ms.
#include "kv8.cuh"
#include "launch_util.h"
#include "sb_device.cuh"
#include "sb_kernels.h"

namespace sb {

namespace kv8 {

constexpr int kThreads = 512;
constexpr uint32_t kRegsSoft = 192, kRegsConv = 88, kRegsMma = 40;
constexpr int kRegsNeeded = (int)(kRegsSoft * 256 + kRegsConv * 128 + kRegsMma * 128);
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kSlab = 16384;  // 128 rows x 64 fp16, 128B swizzle

struct TileExp {  // a scale block: 2^ek, and ev relative to the first block's
  float k, v;
  int e, pad;
};

struct TileShared {
  uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], drain;
  uint64_t s_full[2][2];  // row tile, score buffer: the step's scores are complete
  uint64_t p_full[2][2];  // its weights are written (two buffers: a softmax may be two steps ahead of the MMAs)
  uint64_t o_done[2];     // and multiplied
  uint64_t o_full[2];     // those of the last step are

  uint32_t tmem;
  int abort;
  int e0;    // the exponent byte of V's first block
  int redo;  // the rows are computed again, one by one
  TileExp exps[4][2];
  float q[8][128];  // a softmax warp's row
};

template <int D>
constexpr int tile_smem() {
  return 4 * (D / 64) * kSlab + (int)sizeof(TileShared) + 1024;
}

// B operand whose rows are the contraction axis (V: token rows of 64 channels): 128B swizzle, 8-token
// groups 1024 B apart, 64-channel slabs kSlab apart.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3ffffu) >> 4);
  d |= (uint64_t)(kSlab >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// FP32 pairs, one instruction for two.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t pack2u(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// A row of a 128-row operand tile: 8 channels (16 bytes) at chunk c.
__device__ __forceinline__ uint32_t tile_addr(uint32_t base, int row, int c) {
  return base + (uint32_t)((c >> 3) * kSlab + row * 128 + (((c & 7) ^ (row & 7)) << 4));
}

// The accumulator of row tile t is complete up to step u - 1 once that step's product is done; the phase before
// is behind the scores just read, so the parity is not ambiguous.
template <int D>
__device__ __forceinline__ bool rescale(TileShared& sh, int t, int u, uint32_t o_col, float f) {
  const bool done = mbar_wait_bounded(&sh.o_done[t], (uint32_t)((u - 1) & 1), &sh.abort, kWaitNs);
  if (!__all_sync(0xffffffffu, done)) return false;
  tc_fence_after();
#pragma unroll 1
  for (int h = 0; h < D / 16; ++h) {
    uint32_t o[16];
    tmem_ld16(o_col + 16u * h, o);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
    tmem_st16(o_col + 16u * h, o);
  }
  return true;
}

// Rows r .. r + 31 of a CTA again, one by one: a warp's work, behind its own results.
template <int D>
__device__ __noinline__ void redo_rows(const Kv8Attn& p, int splits, float* part, float* qs, int64_t r) {
  const int64_t b = blockIdx.z, hk = blockIdx.y, group = p.heads_q / p.c.heads;
  const Span sp = sequence_span(p, b);
  const int split = (int)blockIdx.x % splits, c = (threadIdx.x & 31) * (D / 32);
  const int64_t rows = sp.nq * group, r0 = r / 256 * 256, end = min(rows, r + 32);
  const KeyTiles kt = key_tiles(p, sp.pos((int)(r0 / group)), sp.pos((int)((min(rows, r0 + 256) - 1) / group)), 128);
  const int i0 = (int)((int64_t)kt.n * split / splits), i1 = (int)((int64_t)kt.n * (split + 1) / splits);
  __syncwarp();
#pragma unroll 1
  for (; r < end; ++r) {
    const int64_t tok = r / group, hq = hk * group + r - tok * group;
    ExactRow<D> row;
    exact_row<D>(p, b, hk, tok, hq, sp.len, sp.pos((int)tok), kt, 128, i0, i1, qs, row);
    if (splits == 1) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + b * p.os[0] + tok * p.os[1] +
                                                  hq * p.os[2] + c);
#pragma unroll
      for (int e = 0; e < D / 64; ++e)
        dst[e] = pack_bf16x2(__float_as_uint(row.y[2 * e]), __float_as_uint(row.y[2 * e + 1]));
      if (p.lse && c == 0) p.lse[(b * p.heads_q + hq) * p.n_q + tok] = row.lse2 * 0.6931471805599453f;
    } else {
#pragma unroll
      for (int e = 0; e < D / 32; ++e) part_row(p, part, split, b, hk, r)[c + e] = row.y[e];
      if (c == 0) *part_lse(p, part, splits, split, b, hk, r) = row.lse2;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_kv8_tiles(const __grid_constant__ Kv8Attn p, int splits, float* part) {
  extern __shared__ uint8_t smem_raw[];
  if (p.prec && *p.prec == SB_SKIP) return;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  constexpr int kOp = (D / 64) * kSlab;  // one operand tile
  // tensor memory: score buffers of 64 columns, outputs, queries (fp16 pairs); 448 or 512 columns
  constexpr int kBufs = D == 64 ? 2 : 1;
  constexpr uint32_t kSCols = 64 * kBufs, kOCol = 2 * kSCols, kQCol = kOCol + 2 * D;
  static_assert(kQCol + D <= 512, "tensor memory");
  TileShared& sh = *reinterpret_cast<TileShared*>(smem + 4 * kOp);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t k_s = sbase, v_s = sbase + 2 * kOp;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // this CTA's rows and key tiles
  const int group = (int)(p.heads_q / p.c.heads);
  const int64_t b = blockIdx.z, hk = blockIdx.y;
  const Span sp = sequence_span(p, b);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && sp.bad) set_error(p.hdr, SB_ESHAPE);
  const int row_tiles = gridDim.x / splits, split = (int)blockIdx.x % splits;
  const int rt = row_tiles - 1 - (int)blockIdx.x / splits;  // causal: the longest first
  const int64_t rows = (int64_t)sp.nq * group;
  const int64_t r0 = (int64_t)rt * 256;
  if (r0 >= rows) return;
  const int nrow = (int)min((int64_t)256, rows - r0);
  const bool two = nrow > 128;
  const int pmin = sp.pos((int)(r0 / group)), pmax = sp.pos((int)((r0 + nrow - 1) / group));
  const KeyTiles kt = key_tiles(p, pmin, pmax, 128);
  const int i0 = (int)((int64_t)kt.n * split / splits), i1 = (int)((int64_t)kt.n * (split + 1) / splits);
  const int n = i1 - i0;

  if (threadIdx.x == 0) {
    mbar_init(&sh.q_full, two ? 256 : 128);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.k_full[s], 128);
      mbar_init(&sh.k_empty[s], 1);
      mbar_init(&sh.v_full[s], 128);
      mbar_init(&sh.v_empty[s], 1);
      mbar_init(&sh.s_full[s][0], 1);
      mbar_init(&sh.s_full[s][1], 1);
      mbar_init(&sh.p_full[s][0], 128);
      mbar_init(&sh.p_full[s][1], 128);
      mbar_init(&sh.o_done[s], 1);
      mbar_init(&sh.o_full[s], 1);
    }
    mbar_init(&sh.drain, 1);
    sh.abort = 0;
    sh.e0 = sh.redo = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 12) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  volatile int* abort = &sh.abort;

  if (warp < 8) {
    // ------------------------------------------------------------------ softmax, one row a thread
    setmaxnreg_inc<kRegsSoft>();
    const int t = warp >> 2, row = threadIdx.x & 127;
    if (t == 0 || two) {
      const int64_t r = r0 + t * 128 + row;
      const bool live = r < rows;
      const int64_t tok = live ? r / group : 0;
      const int64_t hq = hk * group + (live ? r - tok * group : 0);
      const int pos = sp.pos((int)tok);
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      float qc;
      {
        uint4 u[D / 8];
        uint32_t a = 0;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + b * p.qs[0] +
                                                          tok * p.qs[1] + hq * p.qs[2]);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          u[c] = live ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
          a = __vmaxu2(a, __vmaxu2(__vmaxu2(u[c].x & 0x7fff7fffu, u[c].y & 0x7fff7fffu),
                                   __vmaxu2(u[c].z & 0x7fff7fffu, u[c].w & 0x7fff7fffu)));
        }
        a = max(a & 0xffffu, a >> 16);
        float f;
        qc = query_scale(p.scale, a, f);
#pragma unroll
        for (int h = 0; h < D / 32; ++h) {
          uint32_t w[16];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float v[8];
            unpack8(u[4 * h + c], v);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[4 * c + i] = pack_f16(v[2 * i] * f, v[2 * i + 1] * f);
          }
          tmem_st16(tmem + lanes + kQCol + (uint32_t)(D / 2 * t) + 16u * h, w);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&sh.q_full);
      }
      const uint32_t s_col = tmem + lanes + kSCols * t, o_col = tmem + lanes + kOCol + (uint32_t)(D * t);
      RowStats st{-INFINITY, 0.0f, 0};
      bool ok = true;
      for (int u = 0; u < 2 * n; ++u) {
        const int buf = kBufs == 2 ? u & 1 : 0;
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.s_full[t][buf], (uint32_t)((u / kBufs) & 1), abort, kWaitNs));
        if (!ok) break;
        tc_fence_after();
        const uint32_t col = s_col + 64u * buf;
        uint32_t x[64];
        tmem_ld64(col, x);
        const TileExp te = sh.exps[(u >> 1) & 3][u & 1];
        const float c = fminf(fmaxf(qc * te.k, 0x1p-126f), 0x1p126f);
        const int j0 = kt.tile(i0 + (u >> 1)) * 128 + (u & 1) * 64;
        const bool mask = tile_needs_mask(p, j0, 64, pmin, pmax);
        tmem_ld_wait();
        if (mask) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (!key_visible(p, pos, j0 + i)) x[i] = 0xff800000u;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 64; i += 2)
          mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
        const float mn = fmaxf(st.m, fmaf(fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]), c, te.v));
        if (__any_sync(0xffffffffu, mn > st.m + kRise)) {
          const float f = mn == st.m ? 1.0f : fast_ex2(st.m - mn);
          if (mn > st.m) move_max(st, mn, te.e);
          if (u > 0) {
            ok = rescale<D>(sh, t, u, o_col, f);
            if (!ok) break;
          }
        }
        const float add = te.v + (float)kShift - (st.m == -INFINITY ? 0.0f : st.m);
        const uint64_t cc = pack2(c, c), aa = pack2(add, add);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float y0, y1;
            unpack2(fma2(pack2u(x[32 * h + i], x[32 * h + i + 1]), cc, aa), y0, y1);
            y0 = fast_ex2(y0);
            y1 = fast_ex2(y1);
            sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], pack2(y0, y1));
            w[i / 2] = pack_f16(y0, y1);
          }
          tmem_st16(col + 16u * h, w);
        }
        float s0, s1;
        unpack2(add2(sum[0], sum[1]), s0, s1);
        st.l = fmaf(s0 + s1, sum_factor(st.e - te.e), st.l);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&sh.p_full[t][buf]);
      }
      if (ok && n > 0) ok = mbar_wait_bounded(&sh.o_full[t], 0u, abort, kWaitNs);
      if (!ok) {
        set_error(p.hdr, SB_ETIMEOUT);
        *abort = 1;
      } else {
        tc_fence_after();
        // nothing visible: zeros and -inf; a NaN row has a NaN sum and stays NaN
        const float inv = st.l > 0.0f ? 1.0f / st.l : st.l;
        const float lse2 = st.l > 0.0f ? st.m - (float)st.e + log2f(st.l) : st.l == 0.0f ? -INFINITY : st.l;
        const float2 unit = output_unit(st.e, sh.e0);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld32(o_col + 32u * c, o);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * unit.x * inv * unit.y);
          if (!live) continue;
          if (splits == 1) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + b * p.os[0] + tok * p.os[1] +
                                                  hq * p.os[2] + 32 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dst[i] = make_uint4(pack_bf16x2(o[8 * i], o[8 * i + 1]), pack_bf16x2(o[8 * i + 2], o[8 * i + 3]),
                                  pack_bf16x2(o[8 * i + 4], o[8 * i + 5]), pack_bf16x2(o[8 * i + 6], o[8 * i + 7]));
          } else {
            float* dst = part_row(p, part, split, b, hk, r) + 32 * c;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              reinterpret_cast<uint4*>(dst)[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
        if (live) {
          if (splits > 1)
            *part_lse(p, part, splits, split, b, hk, r) = lse2;
          else if (p.lse)
            p.lse[(b * p.heads_q + hq) * p.n_q + tok] = lse2 * 0.6931471805599453f;
        }
        if (sh.redo) redo_rows<D>(p, splits, part, sh.q[warp], r0 + 32 * warp);
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------------ codes -> fp16 operands
    setmaxnreg_dec<kRegsConv>();
    constexpr int kPieces = D / 16;  // 16-byte pieces of a token, and of a thread's share of a tile
    const int tid = threadIdx.x & 127;
    const int64_t head0 = (b * p.c.heads + hk) * p.c.capacity;
    const uint8_t* kx = p.c.k_exp + head0 / 64;
    const uint8_t* vx = p.c.v_exp + head0 / 64;
    const int blocks = (sp.len + 63) >> 6;
    uint4 kreg[kPieces], vreg[kPieces];
    int ke[2], ve[2], e0 = 0, most = 0;  // exponent bytes of the next tile's blocks; V's first and largest so far
    auto fetch = [&](const uint8_t* codes, int j, uint4 (&u)[kPieces]) {
      const int j0 = kt.tile(i0 + j) * 128;
      const uint8_t* src = codes + (head0 + j0) * D;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int q = tid + 128 * i, tok = q / kPieces;
        u[i] = j0 + tok < sp.len ? ldg_v4(src + (int64_t)q * 16) : make_uint4(0, 0, 0, 0);
      }
    };
    auto fetch_exps = [&](int j) {  // a tile's first block is never past the end; a second one that is: the first's
      const int blk = kt.tile(i0 + j) * 2, next = blk + 1 < blocks ? blk + 1 : blk;
      ke[0] = (int)kx[blk], ke[1] = (int)kx[next];
      ve[0] = (int)vx[blk], ve[1] = (int)vx[next];
    };
    auto put = [&](uint32_t tile, const uint4 (&u)[kPieces]) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int q = tid + 128 * i, tok = q / kPieces, c = 2 * (q - tok * kPieces);
        const uint4 v = u[i];
        st_shared_v4(tile_addr(tile, tok, c), e4m3x2_f16x2(v.x), e4m3x2_f16x2(v.x >> 16), e4m3x2_f16x2(v.y),
                     e4m3x2_f16x2(v.y >> 16));
        st_shared_v4(tile_addr(tile, tok, c + 1), e4m3x2_f16x2(v.z), e4m3x2_f16x2(v.z >> 16), e4m3x2_f16x2(v.w),
                     e4m3x2_f16x2(v.w >> 16));
      }
    };
    bool ok = true;
    if (n > 0) {
      fetch(p.c.k_codes, 0, kreg);
      fetch_exps(0);
      e0 = ve[0];
      if (tid == 0) sh.e0 = e0;
      fetch(p.c.v_codes, 0, vreg);
    }
    for (int j = 0; ok && j < n; ++j) {
      const int s = j & 1;
      const uint32_t ph = (uint32_t)((j >> 1) & 1);
      if (!mbar_wait_bounded(&sh.k_empty[s], ph ^ 1u, abort, kWaitNs)) {
        ok = false;
        break;
      }
      // More than 2^64 below the largest so far, which no row's exponent passes: the block stands at 2^-64 with values
      // of zero, which is right if it holds zeros; if not, the rows are computed again.
      const int floor0 = max(most, ve[0]) - kFar, floor1 = max(most, max(ve[0], ve[1])) - kFar;
      const bool far[2] = {ve[0] < floor0, ve[1] < floor1};
      bool redo = max(ve[0], ve[1]) >= kNanExp;
      most = max(most, max(ve[0], ve[1]));
      if (tid < 2) {  // four tiles' worth: a softmax may still read those of tile j - 2 here
        TileExp& te = sh.exps[j & 3][tid];
        te.k = pow2_byte(tid ? ke[1] : ke[0]);
        te.e = (tid ? max(ve[1], floor1) : max(ve[0], floor0)) - e0;
        te.v = (float)te.e;
      }
      put(k_s + s * kOp, kreg);
      fence_proxy_async_smem();
      mbar_arrive(&sh.k_full[s]);
      if (j + 1 < n) {
        fetch(p.c.k_codes, j + 1, kreg);
        fetch_exps(j + 1);
      }
      if (!mbar_wait_bounded(&sh.v_empty[s], ph ^ 1u, abort, kWaitNs)) {
        ok = false;
        break;
      }
      if (far[0] || far[1]) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          if (!far[i >= kPieces / 2]) continue;
          redo |= ((vreg[i].x | vreg[i].y | vreg[i].z | vreg[i].w) & 0x7f7f7f7fu) != 0;
          vreg[i] = make_uint4(0, 0, 0, 0);
        }
      }
      if (redo) sh.redo = 1;
      put(v_s + s * kOp, vreg);
      fence_proxy_async_smem();
      mbar_arrive(&sh.v_full[s]);
      if (j + 1 < n) fetch(p.c.v_codes, j + 1, vreg);
    }
    if (!ok) {
      set_error(p.hdr, SB_ETIMEOUT);
      *abort = 1;
    }
  } else {
    // ------------------------------------------------------------------ MMA issue
    setmaxnreg_dec<kRegsMma>();
    if (warp == 12 && elect_one() && n > 0) {
      constexpr uint32_t kIdesc = (1u << 4) | (8u << 24);  // FP32 accumulators, fp16 operands, M = 128
      constexpr uint32_t kIdescS = kIdesc | (64u >> 3 << 17);
      constexpr uint32_t kIdescO = kIdesc | ((uint32_t)D >> 3 << 17) | (1u << 16);  // B: rows contracted
      const int tiles = two ? 2 : 1;
      auto qk = [&](int t, int u) {  // scores of step u
        const uint64_t bd = desc_sw128(k_s + ((u >> 1) & 1) * kOp) + (uint32_t)((u & 1) * (64 * 128 >> 4));
        const int buf = kBufs == 2 ? u & 1 : 0;
        const uint32_t d = tmem + kSCols * t + 64u * buf, a = tmem + kQCol + (uint32_t)(D / 2 * t);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (uint32_t)((k >> 2) * (kSlab >> 4) + (k & 3) * 2);
          mma_ts(d, a + 8u * k, bd + off, kIdescS, k ? 1u : 0u);
        }
        mma_commit(&sh.s_full[t][buf]);
      };
      auto run = [&]() {
        if (!mbar_wait_bounded(&sh.q_full, 0u, abort, kWaitNs)) return false;
        if (!mbar_wait_bounded(&sh.k_full[0], 0u, abort, kWaitNs)) return false;
        tc_fence_after();
        for (int u = 0; u < kBufs; ++u)
          for (int t = 0; t < tiles; ++t) qk(t, u);
        if (kBufs == 2) mma_commit(&sh.k_empty[0]);
        for (int u = 0; u < 2 * n; ++u) {
          const int j = u >> 1, s = j & 1, v = u + kBufs;  // v: the step whose scores take this one's place
          const bool more = v < 2 * n;
          if ((u & 1) == 0 && !mbar_wait_bounded(&sh.v_full[s], (uint32_t)((j >> 1) & 1), abort, kWaitNs)) return false;
          if ((v & 1) == 0 && more &&
              !mbar_wait_bounded(&sh.k_full[(v >> 1) & 1], (uint32_t)((v >> 2) & 1), abort, kWaitNs))
            return false;
          const int buf = kBufs == 2 ? u & 1 : 0;
          const uint64_t vd = desc_mn_sw128(v_s + s * kOp) + (uint32_t)((u & 1) * (64 * 128 >> 4));
          for (int t = 0; t < tiles; ++t) {
            if (!mbar_wait_bounded(&sh.p_full[t][buf], (uint32_t)((u / kBufs) & 1), abort, kWaitNs)) return false;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ts(tmem + kOCol + (uint32_t)(D * t), tmem + kSCols * t + 64u * buf + 8u * k, vd + 128u * k, kIdescO,
                     (u | k) ? 1u : 0u);
            mma_commit(&sh.o_done[t]);
            if (u + 1 == 2 * n) mma_commit(&sh.o_full[t]);
            if (more) qk(t, v);  // after the product before it, which reads the weights this overwrites
          }
          if (u & 1) mma_commit(&sh.v_empty[s]);
          if (more && (v & 1)) mma_commit(&sh.k_empty[(v >> 1) & 1]);
        }
        return true;
      };
      if (!run()) {
        set_error(p.hdr, SB_ETIMEOUT);
        *abort = 1;
      }
      mma_commit(&sh.drain);  // every MMA issued is done before TMEM is released
      mbar_wait_bounded(&sh.drain, 0u, nullptr, kWaitNs);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
static cudaError_t launch_tiles_d(const Kv8Attn& p, int splits, float* part, cudaStream_t s, const char** why) {
  static std::atomic<uint64_t> attr{0};
  constexpr int kBytes = tile_smem<D>();
  static_assert(kBytes <= 232448, "shared memory per CTA");
  *why = "sb_kv8_attention: cudaFuncSetAttribute(max dynamic shared memory)";
  cudaError_t e = smem_attr_once(k_kv8_tiles<D>, kBytes, attr);
  if (e != cudaSuccess) return e;
  static std::atomic<int> regs{-1};
  if (regs.load() < 0) {
    cudaFuncAttributes fa;
    *why = "sb_kv8_attention: cudaFuncGetAttributes";
    if ((e = cudaFuncGetAttributes(&fa, k_kv8_tiles<D>)) != cudaSuccess) return e;
    regs.store(fa.numRegs);
  }
  *why = "sb_kv8_attention: compiled with fewer registers per thread than the warpgroup split needs";
  if (regs.load() * kThreads < kRegsNeeded) return cudaErrorInvalidConfiguration;
  *why = "sb_kv8_attention";
  const int64_t row_tiles = ceil_div(p.n_q * (p.heads_q / p.c.heads), 256);
  if (row_tiles * splits > 0x7fffffff) return cudaErrorInvalidValue;
  k_kv8_tiles<D><<<dim3((unsigned)(row_tiles * splits), (unsigned)p.c.heads, (unsigned)p.c.batch), kThreads, kBytes,
                   s>>>(p, splits, part);
  return cudaGetLastError();
}

}  // namespace kv8

cudaError_t launch_kv8_tiles(const Kv8Attn& p, int splits, float* part, cudaStream_t s, const char** why) {
  return p.c.dim == 64 ? kv8::launch_tiles_d<64>(p, splits, part, s, why)
                       : kv8::launch_tiles_d<128>(p, splits, part, s, why);
}

}  // namespace sb
