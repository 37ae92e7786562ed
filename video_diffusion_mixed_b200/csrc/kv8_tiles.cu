// kv8_tiles.cu -- attention over the FP8 key/value cache for many query rows, on the tensor cores.
//
// A row is one query token of one query head; the rows of all query heads that share a key head stand
// together (row = token * group + head in the group), so a key tile serves all of them. A CTA takes 256
// rows (two tiles of 128, one warpgroup each) of one key head and a run of 128-token key tiles:
//
//   S = Q K^T       tcgen05 kind::f16, both operands in shared memory, FP32 in tensor memory
//   w = 2^(c S + ev - m), running maximum m and sum, one row a thread
//   O += w V        tcgen05 kind::f16, w (fp16) from tensor memory, O (FP32) in tensor memory
//
// Keys and values are E4M3 codes, which fp16 holds exactly, so a warpgroup turns each tile's codes into
// fp16 operands once for the 256 rows. The block scales are powers of two and never touch the tiles:
// the keys' enters c, the values' exponent ev (relative to the largest of the CTA's range) the exponent
// of w, and with it the running maximum, which is that of what w V sums; the row sum takes it out again
// by an exact factor. Blocks more than 2^64 below the largest count as zero in V. Queries are scaled by
// a power of two to [2^14, 2^15) and rounded to fp16, exact for every component within 2^-31 of the row's
// largest. The maximum moves only when it would rise by more than 2^8 (fp16 has the room), so the
// accumulator is rescaled rarely.
//
// Warps: 0-3 and 4-7 softmax of the two row tiles, 8-11 codes -> fp16, 12 MMA issue. While one tile's
// softmax runs, the tensor core works on the other's products. Every wait is bounded (SB_ETIMEOUT).
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

struct TileExp {  // a key tile's two blocks: 2^ek, ev and 2^-ev (relative)
  float k[2], v[2], iv[2];
  float pad[2];
};

struct TileShared {
  uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full[2], drain;
  uint32_t tmem;
  int abort;
  int evmax;  // largest exponent byte of V in the CTA's range
  TileExp exps[4];
};

template <int D>
constexpr int tile_smem() {
  return 6 * (D / 64) * kSlab + (int)sizeof(TileShared) + 1024;
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

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A row of a 128-row operand tile: 8 channels (16 bytes) at chunk c.
__device__ __forceinline__ uint32_t tile_addr(uint32_t base, int row, int c) {
  return base + (uint32_t)((c >> 3) * kSlab + row * 128 + (((c & 7) ^ (row & 7)) << 4));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) k_kv8_tiles(const Kv8Attn p, int splits, float* part) {
  extern __shared__ uint8_t smem_raw[];
  if (p.prec && *p.prec == SB_SKIP) return;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  constexpr int kOp = (D / 64) * kSlab;  // one operand tile
  TileShared& sh = *reinterpret_cast<TileShared*>(smem + 6 * kOp);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t q_s = sbase, k_s = sbase + 2 * kOp, v_s = sbase + 4 * kOp;
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
      mbar_init(&sh.s_full[s], 1);
      mbar_init(&sh.p_full[s], 128);
      mbar_init(&sh.o_full[s], 1);
    }
    mbar_init(&sh.drain, 1);
    sh.abort = 0;
    sh.evmax = 0;
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
        for (int c = 0; c < D / 8; ++c) {
          float v[8];
          unpack8(u[c], v);
          st_shared_v4(tile_addr(q_s + t * kOp, row, c), pack_f16(v[0] * f, v[1] * f), pack_f16(v[2] * f, v[3] * f),
                       pack_f16(v[4] * f, v[5] * f), pack_f16(v[6] * f, v[7] * f));
        }
        fence_proxy_async_smem();
        mbar_arrive(&sh.q_full);
      }
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t s_col = tmem + lanes + 128u * t, o_col = tmem + lanes + 256u + (uint32_t)(D * t);
      float m = -INFINITY, l = 0.0f;
      bool ok = true;
      for (int j = 0; j < n; ++j) {
        if (!mbar_wait_bounded(&sh.s_full[t], (uint32_t)(j & 1), abort, kWaitNs)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t x[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_col + 32u * c, x[c]);
        const TileExp& te = sh.exps[j & 3];
        const float c0 = fminf(fmaxf(qc * te.k[0], 0x1p-126f), 0x1p126f);
        const float c1 = fminf(fmaxf(qc * te.k[1], 0x1p-126f), 0x1p126f);
        tmem_ld_wait();
        const int j0 = kt.tile(i0 + j) * 128;
        if (tile_needs_mask(p, j0, 128, pmin, pmax)) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!key_visible(p, pos, j0 + 32 * c + i)) x[c][i] = 0xff800000u;
        }
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            mx[c >> 1] = max3(mx[c >> 1], __uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1]));
        const float mn = max3(m, fmaf(mx[0], c0, te.v[0]), fmaf(mx[1], c1, te.v[1]));
        if (__any_sync(0xffffffffu, mn > m + kRise)) {
          const float f = mn == m ? 1.0f : ex2(m - mn);
          m = mn;
          l *= f;
          if (j > 0) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(o_col + 32u * c, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st32(o_col + 32u * c, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.0f : m;
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float cc = h ? c1 : c0, dd = te.v[h] - base;
          uint32_t w[32];
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float a = ex2(fmaf(__uint_as_float(x[2 * h + c][i]), cc, dd));
              const float d = ex2(fmaf(__uint_as_float(x[2 * h + c][i + 1]), cc, dd));
              sum[h] += a + d;
              w[16 * c + i / 2] = pack_f16(a, d);
            }
          tmem_st32(s_col + 32u * h, w);
        }
        l = fmaf(sum[0], te.iv[0], fmaf(sum[1], te.iv[1], l));
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&sh.p_full[t]);
      }
      if (ok && n > 0) ok = mbar_wait_bounded(&sh.o_full[t], 0u, abort, kWaitNs);
      if (!ok) {
        set_error(p.hdr, SB_ETIMEOUT);
        *abort = 1;
      } else {
        tc_fence_after();
        // nothing visible: zeros and -inf; a NaN row has a NaN sum and stays NaN
        const float inv = l > 0.0f ? __uint_as_float((uint32_t)max(sh.evmax, 1) << 23) / l : l;
        const float lse2 = l > 0.0f ? m + log2f(l) : l == 0.0f ? -INFINITY : l;
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
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
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
    {  // the largest exponent of V over this CTA's tiles
      int e = 0;
      for (int i = tid; i < 2 * n; i += 128) {
        const int blk = kt.tile(i0 + (i >> 1)) * 2 + (i & 1);
        if (blk < blocks) e = max(e, (int)vx[blk]);
      }
#pragma unroll
      for (int s = 16; s >= 1; s >>= 1) e = max(e, __shfl_xor_sync(0xffffffffu, e, s));
      if (lane == 0) atomicMax(&sh.evmax, e);
      asm volatile("bar.sync 1, 128;" ::: "memory");
    }
    const int evmax = sh.evmax;
    uint4 kreg[kPieces], vreg[kPieces];
    int ke = 127, ve = 0;  // thread h < 2: exponent bytes of the next tile's block h
    auto fetch = [&](const uint8_t* codes, int j, uint4 (&u)[kPieces]) {
      const int j0 = kt.tile(i0 + j) * 128;
      const uint8_t* src = codes + (head0 + j0) * D;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int q = tid + 128 * i, tok = q / kPieces;
        u[i] = j0 + tok < sp.len ? ldg_v4(src + (int64_t)q * 16) : make_uint4(0, 0, 0, 0);
      }
    };
    auto fetch_exps = [&](int j) {  // a block past the end: any finite scale
      const int blk = kt.tile(i0 + j) * 2 + tid;
      if (tid < 2) ke = blk < blocks ? (int)kx[blk] : 127, ve = blk < blocks ? (int)vx[blk] : 0;
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
      fetch(p.c.v_codes, 0, vreg);
    }
    for (int j = 0; ok && j < n; ++j) {
      const int s = j & 1;
      const uint32_t ph = (uint32_t)((j >> 1) & 1);
      if (!mbar_wait_bounded(&sh.k_empty[s], ph ^ 1u, abort, kWaitNs)) {
        ok = false;
        break;
      }
      if (tid < 2) {  // four tiles' worth: a softmax reads tile j's until its weights are out, and K of
                      // tile j + 2 comes after that of j + 1 has been multiplied with both row tiles
        TileExp& te = sh.exps[j & 3];
        const int rel = max(ve - evmax, -64);
        te.k[tid] = pow2_byte(ke);
        te.v[tid] = (float)rel;
        te.iv[tid] = __uint_as_float((uint32_t)(127 - rel) << 23);
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
      {  // a block more than 2^64 below the largest counts as zero
        const int j0 = kt.tile(i0 + j) * 128;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int blk = (j0 + (tid + 128 * i) / kPieces) >> 6;
          if (blk < blocks && (int)__ldg(vx + blk) < evmax - 64) vreg[i] = make_uint4(0, 0, 0, 0);
        }
      }
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
      constexpr uint32_t kIdescS = kIdesc | (128u >> 3 << 17);
      constexpr uint32_t kIdescO = kIdesc | ((uint32_t)D >> 3 << 17) | (1u << 16);  // B: rows contracted
      const int tiles = two ? 2 : 1;
      auto qk = [&](int t, int s) {
        const uint64_t a = desc_sw128(q_s + t * kOp), bd = desc_sw128(k_s + s * kOp);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (uint32_t)((k >> 2) * (kSlab >> 4) + (k & 3) * 2);
          mma_ss(tmem + 128u * t, a + off, bd + off, kIdescS, k ? 1u : 0u);
        }
      };
      auto run = [&]() {
        if (!mbar_wait_bounded(&sh.q_full, 0u, abort, kWaitNs)) return false;
        if (!mbar_wait_bounded(&sh.k_full[0], 0u, abort, kWaitNs)) return false;
        tc_fence_after();
        for (int t = 0; t < tiles; ++t) {
          qk(t, 0);
          mma_commit(&sh.s_full[t]);
        }
        mma_commit(&sh.k_empty[0]);
        for (int j = 0; j < n; ++j) {
          const int s = j & 1, s1 = (j + 1) & 1;
          for (int t = 0; t < tiles; ++t) {
            if (t == 0 && !mbar_wait_bounded(&sh.v_full[s], (uint32_t)((j >> 1) & 1), abort, kWaitNs)) return false;
            if (!mbar_wait_bounded(&sh.p_full[t], (uint32_t)(j & 1), abort, kWaitNs)) return false;
            tc_fence_after();
            const uint64_t vd = desc_mn_sw128(v_s + s * kOp);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_ts(tmem + 256u + (uint32_t)(D * t), tmem + 128u * t + 8u * k, vd + 128u * k, kIdescO,
                     (j | k) ? 1u : 0u);
            if (j + 1 < n) {
              if (t == 0 && !mbar_wait_bounded(&sh.k_full[s1], (uint32_t)(((j + 1) >> 1) & 1), abort, kWaitNs))
                return false;
              tc_fence_after();
              qk(t, s1);  // after the product before it, which reads the weights this overwrites
              mma_commit(&sh.s_full[t]);
            } else {
              mma_commit(&sh.o_full[t]);
            }
          }
          mma_commit(&sh.v_empty[s]);
          if (j + 1 < n) mma_commit(&sh.k_empty[s1]);
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
