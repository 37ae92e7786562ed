// fp8_gemm.cu -- the FP8 linear layer's product on the tensor cores:
//
//   Y[m][n] = act(sum_b 2^(ex[m][b] + ew[n][b]) sum_{k in block b} x[m][k] w[n][k] + bias[n])
//
// with E4M3 codes x, w and one E8M0 scale per 128 channels of a row on both sides. The scale enters
// the product inside the tensor core (tcgen05.mma kind::mxf8f6f4, block scaled): an MMA consumes 32
// channels, and the four MMAs of a 128-channel K-block all read the same scale byte. One 32-bit word
// of a row holds the bytes of four consecutive K-blocks, the scale-factor id of the instruction
// descriptor picks the K-block's, so a 512-byte atom (128 rows x 4 K-blocks) is loaded and copied to
// tensor memory once per 512 channels. No accumulator ever leaves tensor memory to be scaled.
//
// Persistent kernel in two forms. Pair form (CG = 2): clusters of two CTAs on an SM pair, one 256 x BN
// output tile at a time, as in the quantized GEMM beside it. Single form (CG = 1) for few rows: one CTA
// per 128 x BN tile, so that a product bound by reading the weight once is spread over the whole chip;
// its ring is as deep as the rows of A that exist leave room for (the MMA's other rows read whatever
// lies behind them in shared memory, and their results are never looked at). Warp roles: warp 0 loads
// with TMA (no multicast), warp 1 (of the even CTA) issues the MMAs, warps 4-11 drain the accumulators.
#include <cudaTypedefs.h>

#include "gemm_epi.cuh"
#include "launch_util.h"
#include "sb_device.cuh"
#include "sb_kernels.h"
#include "tmap.h"

namespace sb {

namespace fp8 {

// A stage of the ring: A (up to 128 rows x 128 B), B (up to 128 rows x 128 B), 512 B of A's scales for
// four K-blocks, up to 3 x 512 B of B's; every part a multiple of 1024 (the 128B-swizzle atom).
constexpr int kSfBytes = 2048;
constexpr int kMaxStages = 12;
constexpr int kStageArea = 5 * (32768 + kSfBytes);
constexpr int kThreads = 384;
constexpr int kEpiWarp0 = 4, kEpiWarps = 8;
constexpr uint32_t kRegsCtl = 72, kRegsEpi = 216;
constexpr int kRegsNeeded = (int)(kRegsCtl * 128 + kRegsEpi * 256);
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSfCols = 16;                  // 4 columns for A's scales, up to 12 for B's
constexpr uint64_t kWaitNs = 2000000000ull;       // 2 s, far above any legitimate wait
constexpr uint64_t kDrainNs = 20000000ull;
constexpr int kOutOff = kStageArea + 1024;
constexpr int kOutBox = 2048;                     // 32 x 32 bf16, 64B swizzle; two per epilogue warp
constexpr int kSmemBytes = kOutOff + kEpiWarps * 2 * kOutBox + 1024;
constexpr int kStoreLane = 31;
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

struct Maps {
  CUtensorMap a, b, sfa, sfb, y;
};

struct Params {
  int M, N, K, BN;
  int a_rows;              // rows of A that a CTA loads: 128, or the multiple of 8 that holds all of M
  int off_b, off_sf, stage_bytes, stages;
  const int32_t* prec;
  const __nv_bfloat16* bias;
  void* Y;
  int out_f32, gelu, group_m;
  WsHeader* hdr;
};

// The instructions of the two forms.
template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                    uint32_t acc) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(sfa), "r"(sfb)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(sfa), "r"(sfb)
        : "memory");
}
template <int CG>
__device__ __forceinline__ void copy_sf(uint32_t taddr, uint64_t desc) {
  if constexpr (CG == 2)
    tmem_cp_sf_pair(taddr, desc);
  else
    tmem_cp_sf(taddr, desc);
}
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar, uint16_t mask) {
  if constexpr (CG == 2)
    mma_commit_pair(bar, mask);
  else
    mma_commit(bar);
}
template <int CG>
__device__ __forceinline__ void load_2d(void* dst, const void* map, uint64_t* own, uint32_t leader, int x, int y) {
  if constexpr (CG == 2)
    tma_load_2d_pair(dst, map, leader, x, y);
  else
    tma_load_2d(dst, map, own, x, y);
}
template <int CG>
__device__ __forceinline__ void load_3d(void* dst, const void* map, uint64_t* own, uint32_t leader, int x, int y,
                                        int z) {
  if constexpr (CG == 2)
    tma_load_3d_pair(dst, map, leader, x, y, z);
  else
    tma_load_3d(smem_u32(dst), map, smem_u32(own), x, y, z);
}
template <int CG>
__device__ __forceinline__ void sync_ctas() {
  if constexpr (CG == 2)
    cluster_sync();
  else
    __syncthreads();
}

struct Ring {
  uint64_t *full, *empty, *tfull, *tempty;
  volatile int* abort;
};

// MMA issue (one thread of the even CTA). Returns false when a wait gave up. The tensor core runs the
// copies of scales and the MMAs of one issuer in order, so the scale columns need no second buffer.
template <int CG>
__device__ __forceinline__ bool issue_all(const Params& p, const Ring r, uint32_t smem, uint32_t tmem, int unit,
                                          int nunits, int tiles, int m_tiles, int n_tiles, int nacc) {
  const int nkb = (p.K + 127) / 128, tail = (p.K - (nkb - 1) * 128) / 32;
  const int stages = p.stages;
  const uint32_t sfa = tmem + (uint32_t)(nacc * p.BN), sfb = sfa + 4u;
  // E4M3 x E4M3 (format 0), UE8M0 scales (bit 23), M = 128 CG, N = BN
  const uint32_t idesc = (1u << 23) | ((uint32_t)(p.BN >> 3) << 17) | (8u * CG << 24);
  const uint32_t off_b = (uint32_t)p.off_b >> 4, off_sf = (uint32_t)p.off_sf >> 4, stage16 = (uint32_t)p.stage_bytes >> 4;
  const uint64_t dsw = desc_sw128(smem), dsf = desc_sf(smem);
  int s = 0, it = 0;
  uint32_t ph = 0;
  for (int tile = unit; tile < tiles; tile += nunits, ++it) {
    const int b = nacc == 1 ? 0 : (it & 1);
    const uint32_t tph = (uint32_t)((nacc == 1 ? it : it >> 1) & 1);
    if (!mbar_wait_bounded(&r.tempty[b], tph ^ 1u, r.abort, kWaitNs)) return false;
    tc_fence_after();
    int mt, nt;
    tile_coords(tile, m_tiles, n_tiles, p.group_m, &mt, &nt);
    const int n0 = nt * p.BN;
    const uint32_t shift = (uint32_t)((n0 & 127) >> 5);
    const int sf_tiles = ((n0 & 127) + p.BN + 127) >> 7;
    const uint32_t d = tmem + (uint32_t)(b * p.BN);
    for (int kb = 0; kb < nkb; ++kb) {
      if (!mbar_wait_bounded(&r.full[s], ph, r.abort, kWaitNs)) return false;
      tc_fence_after();
      const uint32_t so = (uint32_t)s * stage16;
      if ((kb & 3) == 0) {
        copy_sf<CG>(sfa, dsf + so + off_sf);
        for (int t = 0; t < sf_tiles; ++t) copy_sf<CG>(sfb + 4u * t, dsf + so + off_sf + 32u * (t + 1));
      }
      const uint32_t id = (uint32_t)(kb & 3);
      const uint32_t desc = idesc | (id << 4) | (id << 29);
      const uint64_t ad = dsw + so, bd = ad + off_b;
      if (kb < nkb - 1 || tail == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) mma<CG>(d, ad + 2u * j, bd + 2u * j, desc, sfa, sfb + shift, (kb | j) ? 1u : 0u);
      } else {
        for (int j = 0; j < tail; ++j) mma<CG>(d, ad + 2u * j, bd + 2u * j, desc, sfa, sfb + shift, (kb | j) ? 1u : 0u);
      }
      commit<CG>(&r.empty[s], (uint16_t)3);
      if (++s == stages) s = 0, ph ^= 1u;
    }
    commit<CG>(&r.tfull[b], (uint16_t)3);
  }
  return true;
}

struct Bias32 {
  uint4 q[4];
};
__device__ __forceinline__ void load_bias(const Params& p, int n, Bias32& o) {
  if (p.bias && n < p.N) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o.q[i] = __ldg(reinterpret_cast<const uint4*>(p.bias + n) + i);
  }
}

// Bias, optional GELU of 32 accumulator columns of one row, in place.
__device__ __forceinline__ void finish32(const Params& p, const Bias32& o, uint32_t (&r)[32]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint4 q = o.q[j >> 2];
    const uint32_t w = (j & 3) == 0 ? q.x : (j & 3) == 1 ? q.y : (j & 3) == 2 ? q.z : q.w;
    const float2 bias =
        p.bias ? make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)) : make_float2(0.0f, 0.0f);
    float2 y = ep_add2(make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), bias);
    if (p.gelu) y = gelu_exp2(y);
    r[2 * j] = __float_as_uint(y.x);
    r[2 * j + 1] = __float_as_uint(y.y);
  }
}

// One row's 32 finished columns: bf16 through a staging box and a TMA store (rows past M are clipped
// there), FP32 directly.
__device__ __forceinline__ void store32(const Params& p, const CUtensorMap* ty, uint32_t boxes, int lane, int m,
                                        int m_warp, int n, const uint32_t (&r)[32], uint32_t& oc) {
  if (p.out_f32) {
    if (m < p.M) {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<float*>(p.Y) + (int64_t)m * p.N + n);
#pragma unroll
      for (int i = 0; i < 8; ++i) dst[i] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
    }
    return;
  }
  const uint32_t box = boxes + (oc & 1u) * (uint32_t)kOutBox;
  if (lane == kStoreLane) bulk_wait_read<1>();
  __syncwarp();
  stage_bf16_row(box, lane, r);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == kStoreLane) {
    tma_store_2d(ty, box, n, m_warp);
    bulk_commit();
  }
  ++oc;
}

template <int CG, bool ONE_ACC>  // one accumulator (BN = 256): drained whole before any arithmetic
__device__ __forceinline__ void epilogue(const Params& p, const Maps& tm, const Ring r, uint32_t tmem, uint32_t boxes,
                                         uint32_t tempty_leader, int warp, int lane, int row_off, int unit, int nunits,
                                         int tiles, int m_tiles, int n_tiles) {
  const int q = warp & 3, half = (warp - kEpiWarp0) >> 2;
  const int cols = p.BN / 2, nch = cols / 32;
  uint32_t oc = 0;
  int it = 0;
  for (int tile = unit; tile < tiles; tile += nunits, ++it) {
    int mt, nt;
    tile_coords(tile, m_tiles, n_tiles, p.group_m, &mt, &nt);
    const int m_warp = mt * 128 * CG + row_off + 32 * q, m = m_warp + lane;
    const int n0 = nt * p.BN + half * cols;
    const int b = ONE_ACC ? 0 : (it & 1);
    const uint32_t tph = (uint32_t)((ONE_ACC ? it : it >> 1) & 1);
    Bias32 bias;
    load_bias(p, n0, bias);  // before the wait; each chunk's next one is loaded while it is stored
    if (!mbar_wait_bounded(&r.tfull[b], tph, r.abort, kWaitNs)) {
      set_error(p.hdr, SB_ETIMEOUT);
      *r.abort = 1;
      break;
    }
    tc_fence_after();
    const uint32_t t0 = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(b * p.BN + half * cols);
    if constexpr (ONE_ACC) {
      uint32_t v[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(t0 + 32u * c, v[c]);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty_leader);  // this form is a pair's only
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int n = n0 + 32 * c;
        if (n < p.N && m_warp < p.M) {
          finish32(p, bias, v[c]);
          if (c < 3) load_bias(p, n + 32, bias);
          store32(p, &tm.y, boxes, lane, m, m_warp, n, v[c], oc);
        }
      }
    } else {
      for (int c = 0; c < nch; ++c) {
        uint32_t v[32];
        tmem_ld32(t0 + 32u * c, v);
        tmem_ld_wait();
        if (c == nch - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(tempty_leader + 8u * b);
        }
        const int n = n0 + 32 * c;
        if (n < p.N && m_warp < p.M) {
          finish32(p, bias, v);
          if (c + 1 < nch) load_bias(p, n + 32, bias);
          store32(p, &tm.y, boxes, lane, m, m_warp, n, v, oc);
        }
      }
    }
  }
  if (lane == kStoreLane) bulk_wait_read<0>();  // the boxes are read; the kernel's end completes the writes
  __syncwarp();
}

template <int CG>
__global__ void __cluster_dims__(CG, 1, 1) __launch_bounds__(kThreads, 1)
    k_fp8_gemm(const __grid_constant__ Maps tm, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Ring r;
  r.full = reinterpret_cast<uint64_t*>(smem + kStageArea);
  r.empty = r.full + kMaxStages;
  r.tfull = r.empty + kMaxStages;
  r.tempty = r.tfull + 2;
  uint64_t* drain = r.tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  r.abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  if (p.prec && *p.prec == SB_SKIP) {  // uniform over the grid
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int nkb = (p.K + 127) / 128;
  const int m_tiles = (p.M + 128 * CG - 1) / (128 * CG), n_tiles = (p.N + p.BN - 1) / p.BN, tiles = m_tiles * n_tiles;
  const int unit = (int)blockIdx.x / CG, nunits = (int)gridDim.x / CG;
  if (unit >= tiles) return;  // both CTAs of a pair leave together
  const int row_off = 128 * (int)rank;
  const int nacc = 2 * p.BN + (int)kSfCols <= (int)kTmemCols ? 2 : 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&r.full[s], 1);
      mbar_init(&r.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&r.tfull[b], 1);
      mbar_init(&r.tempty[b], CG * kEpiWarps);
    }
    mbar_init(drain, 1);
    *r.abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  sync_ctas<CG>();
  if (warp == 1) {
    if constexpr (CG == 2) {
      tmem_alloc_pair(tmem_slot, kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < kEpiWarp0) {
    setmaxnreg_dec<kRegsCtl>();
    if (warp == 0) {
      if (elect_one()) {
        prefetch_tmap(&tm.a);
        prefetch_tmap(&tm.b);
        prefetch_tmap(&tm.sfa);
        prefetch_tmap(&tm.sfb);
        const uint32_t full_leader = CG == 2 ? cluster_addr(&r.full[0], 0) : 0u;
        asm volatile("griddepcontrol.wait;" ::: "memory");  // A's codes come from the launch before
        int s = 0;
        uint32_t ph = 0;
        int64_t issued = 0;
        bool ok = true;
        for (int tile = unit; ok && tile < tiles; tile += nunits) {
          int mt, nt;
          tile_coords(tile, m_tiles, n_tiles, p.group_m, &mt, &nt);
          const int m0 = mt * 128 * CG + row_off, n0 = nt * p.BN;
          const int sf_tiles = ((n0 & 127) + p.BN + 127) >> 7;
          const uint32_t tx = (uint32_t)(CG * p.a_rows + p.BN) * 128u;  // all CTAs' operands
          for (int kb = 0; kb < nkb; ++kb) {
            if (!mbar_wait_bounded(&r.empty[s], ph ^ 1u, r.abort, kWaitNs)) {
              ok = false;
              break;
            }
            uint8_t* st = smem + s * p.stage_bytes;
            const uint32_t fb = full_leader + 8u * s;
            const bool sf = (kb & 3) == 0;
            if (leader) mbar_arrive_expect_tx(&r.full[s], tx + (sf ? CG * 512u * (1u + (uint32_t)sf_tiles) : 0u));
            load_2d<CG>(st, &tm.a, &r.full[s], fb, kb * 128, m0);
            load_2d<CG>(st + p.off_b, &tm.b, &r.full[s], fb, kb * 128, n0 + (p.BN / CG) * (int)rank);
            if (sf) {
              load_3d<CG>(st + p.off_sf, &tm.sfa, &r.full[s], fb, 0, kb >> 2, m0 >> 7);
              for (int t = 0; t < sf_tiles; ++t)
                load_3d<CG>(st + p.off_sf + 512 * (t + 1), &tm.sfb, &r.full[s], fb, 0, kb >> 2, (n0 >> 7) + t);
            }
            ++issued;
            if (++s == p.stages) s = 0, ph ^= 1u;
          }
        }
        if (!ok) {
          set_error(p.hdr, SB_ETIMEOUT);
          *r.abort = 1;
          if (leader) {  // both CTAs' copies complete on the leader's barriers: let them land
            const int64_t first = issued > p.stages ? issued - p.stages : 0;
            for (int64_t k = first; k < issued; ++k)
              mbar_wait_bounded(&r.full[k % p.stages], (uint32_t)((k / p.stages) & 1), nullptr, kDrainNs);
          }
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      if (leader && elect_one()) {
        if (!issue_all<CG>(p, r, smem_u32(smem), tmem, unit, nunits, tiles, m_tiles, n_tiles, nacc)) {
          set_error(p.hdr, SB_ETIMEOUT);
          *r.abort = 1;
        }
        commit<CG>(drain, (uint16_t)1);  // every MMA issued is done before TMEM is released
        mbar_wait_bounded(drain, 0u, nullptr, kWaitNs);
      }
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<kRegsEpi>();
    const uint32_t boxes = smem_u32(smem + kOutOff) + (uint32_t)(2 * (warp - kEpiWarp0) * kOutBox);
    const uint32_t te = CG == 2 ? cluster_addr(&r.tempty[0], 0) : smem_u32(&r.tempty[0]);
    if constexpr (CG == 2) {
      if (nacc == 1)
        epilogue<2, true>(p, tm, r, tmem, boxes, te, warp, lane, row_off, unit, nunits, tiles, m_tiles, n_tiles);
      else
        epilogue<2, false>(p, tm, r, tmem, boxes, te, warp, lane, row_off, unit, nunits, tiles, m_tiles, n_tiles);
    } else {
      epilogue<1, false>(p, tm, r, tmem, boxes, te, warp, lane, row_off, unit, nunits, tiles, m_tiles, n_tiles);
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CG == 2)
      tmem_dealloc_pair(tmem, kTmemCols);
    else
      tmem_dealloc(tmem, kTmemCols);
  }
}

static bool operand_map(CUtensorMap* m, const void* base, uint64_t K, uint64_t rows, uint32_t box_rows) {
  auto fn = tmap_encoder();
  cuuint64_t dims[2] = {K, rows};
  cuuint64_t strides[1] = {K};
  cuuint32_t box[2] = {128, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale atoms: 128 words x ceil(K / 512) atoms x 128-row tiles; box = one atom.
static bool scale_map(CUtensorMap* m, const void* base, uint64_t K, uint64_t rows) {
  auto fn = tmap_encoder();
  const uint64_t atoms = (K + 511) / 512;
  cuuint64_t dims[3] = {128, atoms, (rows + 127) / 128};
  cuuint64_t strides[2] = {512, atoms * 512};
  cuuint32_t box[3] = {128, 1, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace fp8

template <int CG>
static cudaError_t launch_form(const Fp8Linear& L, int BN, cudaStream_t s, const char** why) {
  using namespace fp8;
  static std::atomic<uint64_t> attr{0};
  *why = "sb_linear_fp8: cudaFuncSetAttribute(max dynamic shared memory)";
  cudaError_t e = smem_attr_once(k_fp8_gemm<CG>, kSmemBytes, attr);
  if (e != cudaSuccess) return e;
  // the register split must fit what a CTA is launched with, or setmaxnreg.inc would wait for good
  static std::atomic<int> regs{-1};
  if (regs.load() < 0) {
    cudaFuncAttributes fa;
    *why = "sb_linear_fp8: cudaFuncGetAttributes";
    if ((e = cudaFuncGetAttributes(&fa, k_fp8_gemm<CG>)) != cudaSuccess) return e;
    regs.store(fa.numRegs);
  }
  *why = "sb_linear_fp8: compiled with fewer registers per thread than the warpgroup split needs";
  if (regs.load() * kThreads < kRegsNeeded) return cudaErrorInvalidConfiguration;
  Params p{};
  p.M = (int)L.M;
  p.N = (int)L.N;
  p.K = (int)L.K;
  p.BN = BN;
  p.a_rows = CG == 1 && L.M < 128 ? (int)ceil_div(L.M, 8) * 8 : 128;
  p.off_b = p.a_rows * 128;  // 8 rows are a 1024-byte atom
  p.off_sf = p.off_b + BN / CG * 128;
  p.stage_bytes = p.off_sf + kSfBytes;
  // the last stage's A is read as 128 rows: those past a_rows must lie inside the ring
  const int room = CG == 1 ? kStageArea - (16384 - p.off_b) : kStageArea;
  p.stages = room / p.stage_bytes < kMaxStages ? room / p.stage_bytes : kMaxStages;
  p.prec = L.prec;
  p.bias = static_cast<const __nv_bfloat16*>(L.bias);
  p.Y = L.Y;
  p.out_f32 = L.out_dtype == SB_OUT_F32;
  p.gelu = L.epilogue == SB_EPI_GELU_TANH;
  p.group_m = 8;
  p.hdr = static_cast<WsHeader*>(L.hdr);
  Maps tm;
  memset(&tm, 0, sizeof(tm));
  *why = "sb_linear_fp8: cuTensorMapEncodeTiled";
  if (!operand_map(&tm.a, L.A, (uint64_t)L.K, (uint64_t)L.M, (uint32_t)p.a_rows) ||
      !operand_map(&tm.b, L.W, (uint64_t)L.K, (uint64_t)L.N, (uint32_t)BN / CG) ||
      !scale_map(&tm.sfa, L.sfA, (uint64_t)L.K, (uint64_t)L.M) ||
      !scale_map(&tm.sfb, L.sfW, (uint64_t)L.K, (uint64_t)L.N))
    return cudaErrorInvalidValue;
  if (!p.out_f32) {
    cuuint64_t dims[2] = {(cuuint64_t)L.N, (cuuint64_t)L.M};
    cuuint64_t strides[1] = {(cuuint64_t)L.N * 2};
    cuuint32_t box[2] = {32, 32};
    cuuint32_t estr[2] = {1, 1};
    if (tmap_encoder()(&tm.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, L.Y, dims, strides, box, estr,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  const int64_t want = CG * ceil_div(L.M, 128 * CG) * ceil_div(L.N, BN), sms = device_sm_count() & ~1;
  *why = "sb_linear_fp8";
  const LaunchAfter cfg((unsigned)(want < sms ? want : sms), kThreads, kSmemBytes, s, L.X != nullptr);
  return cudaLaunchKernelEx(&cfg.cfg, k_fp8_gemm<CG>, tm, p);
}

cudaError_t launch_fp8_gemm(const Fp8Linear& L, cudaStream_t s, const char** why) {
  const int sms = device_sm_count() & ~1;
  // Form and tile width: the ones with the shortest schedule. ns: a tile's time with K = 1920, measured on
  // full waves of the 74 CTA pairs or 148 CTAs (256 columns have one accumulator, so its drain is not
  // hidden). What it decides, measured in us (pair form with 64 / 128 columns, single form with 64 / 128 /
  // 192): 128 x 7680 14.1 / 11.6, 10.0 / 11.1 / 13.2; 226 x 1920 10.1 / 10.9, 9.5 / 10.6 / 12.7;
  // 300 x 7680 21.4 / 15.5, 17.4 / 15.4 / 13.7; 600 x 1920 13.8 / 11.1, 12.9 / 10.6 / 12.6; with 1350 x
  // 5760 the pair form's 64 / 128 / 192 / 256 columns take 41.0 / 28.7 / 26.6 / 24.6. The order holds at other
  // K: with K = 256 and 7680, thirteen sizes of 64 to 4096 rows, what it picks is the fastest of the seven or
  // within 1 us of it, but for 1350 x 1920 x 256 (12.4, single form with 192 columns 10.2) and 4096 x 7680 x 7680 (171, pair form with
  // 256 columns 160).
  static const struct { int cg, bn, ns; } kForms[] = {{2, 256, 6550}, {2, 192, 4980}, {2, 128, 4250}, {2, 64, 3680},
                                                      {1, 192, 7000}, {1, 128, 4500}, {1, 64, 3600}};
  int64_t best = INT64_MAX;
  int cg = 2, bn = 256;
  for (const auto& f : kForms) {
    const int64_t t = ceil_div(ceil_div(L.M, 128 * f.cg) * ceil_div(L.N, f.bn), sms / f.cg) * f.ns;
    if (t < best) best = t, cg = f.cg, bn = f.bn;
  }
  return cg == 2 ? launch_form<2>(L, bn, s, why) : launch_form<1>(L, bn, s, why);
}

}  // namespace sb
