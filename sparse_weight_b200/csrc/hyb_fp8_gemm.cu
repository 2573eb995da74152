// The 8-bit floating-point product for more than a few tokens, on the 5th-
// generation tensor cores:
//
//   Y[m][n] = sum_b sx[m][b] sw[n / 128][b] sum_{k in block b} xq[m][k] wq[n][k]
//
// tcgen05.mma multiplies a block of 128 columns exactly as the sum over k asks
// (e4m3 x e4m3 products are exact, accumulation in fp32), but the scales change
// from block to block, so a block's products go to a tensor-memory buffer of
// their own and the epilogue warps add them, scaled, to fp32 sums in registers
// while the tensor cores fill the other buffer.
//
//   * A CTA owns 128 tokens (the MMA's M, one tensor-memory lane each) and BN
//     rows of W (its N).  With the tokens in the lanes a thread's token scale is
//     one register and W's scale one per 128 columns: a block costs one FMA per
//     value and no other scale traffic.
//   * warp 0 moves operand blocks with TMA (128-byte rows in the 128-byte
//     swizzle: one block of k is one swizzle row), warp 1 issues the MMAs, the
//     last 8 (two per lane quarter, half of the columns each) scale and add.
//   * Where the tiles alone do not fill the GPU, a cluster of CTAs splits k; its
//     partial sums meet in distributed shared memory in a fixed order.
//
// Bound by the epilogue's reads of tensor memory and FMAs beside the MMAs.  2048
// tokens x 14336 x 4096: 180 us (1.34 PFLOP/s) with BN = 256, the quantiser
// included, of which a seventh round of 8 tiles takes a whole tile's time; 45 x 1000 x
// 4100 in e4m3: 7.5 us, latency of one launch whose 64 CTAs leave half of the SMs idle;
// 128 x 4096 x 4096 in bf16: 15.9 us.  With inputs in L2 these take 168, 6.8 and 14.9
// us, and so measured the first took 176 us with BN = 224 (6.9 rounds of CTAs), 171 with
// rows of W first (W read three times), and the last 33 us when the lanes that add up
// a cluster's sums read 32 bytes apart from one another.
//
// Registers: 12 bytes are spilled at BN = 128 (two CTAs per SM), 32 at BN = 256, whose
// 10 warps put three on a scheduler (168 registers).
#include "hyb_fp8.cuh"
#include "hyb_tcgen05.cuh"

#include <cooperative_groups.h>

namespace cg = cooperative_groups;

namespace hyb {
namespace {

constexpr int kTok = 128;       // tokens per CTA
constexpr int kMaxC = 8;        // CTAs of a cluster at most
constexpr int kGroup = 16;      // token tiles that pass along W together

template <int BN>
struct Shape {
  static constexpr int kStage = (kTok + BN) * kBlk;  // bytes of one block's operands
  static constexpr int kStages = BN == 256 ? 4 : 3;
  static constexpr int kRing = kStage * kStages;
  static constexpr int kCols = BN / 2;               // columns per epilogue thread
  static constexpr int kPitch = BN + 4;              // floats per row of the result in shared memory
  static constexpr int kTmem = 2 * BN;
  static constexpr int kLoad = BN == 256 ? 32 : 16;  // columns per tensor-memory read
  // producer, MMA, then 8 epilogue warps
  static constexpr int kCtl = 2;
  static constexpr int kThreads = 32 * (kCtl + 8);
  static_assert(kTok * kPitch * 4 <= kRing, "the result reuses the ring");
  static_assert(tmem_fits(kTmem, kRing), "tensor memory of the CTAs that fit an SM");
  static_assert(kStage % 1024 == 0, "swizzle alignment");
};

__device__ __forceinline__ void umma_f8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                        uint32_t accumulate, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %4, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(accumulate), "r"(idesc)
      : "memory");
}

// N (16 or 32) columns of this thread's lane; the values are there after
// tmem_wait
__device__ __forceinline__ void tmem_issue(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_issue(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]),
                 "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

// acc += d * s on pairs of fp32
__device__ __forceinline__ void fma2(uint64_t &acc, uint32_t lo, uint32_t hi, uint64_t s) {
  asm("{\n\t.reg .b64 d;\n\t"
      "mov.b64 d, {%1, %2};\n\t"
      "fma.rn.f32x2 %0, d, %3, %0;\n\t}"
      : "+l"(acc)
      : "r"(lo), "r"(hi), "l"(s));
}
__device__ __forceinline__ uint64_t twice(float s) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "r"(__float_as_uint(s)));
  return r;
}

// One block's products (COLS columns from taddr) times `scale` onto acc;
// `freed` gets the warp's arrival once they have been read.  The next N
// columns are on their way while N are added.
template <int COLS, int N>
__device__ __forceinline__ void scale_add(uint32_t taddr, float scale, uint64_t (&acc)[COLS / 2],
                                          uint64_t *freed) {
  const uint64_t s = twice(scale);
  uint32_t d[2][N];
  tmem_issue(taddr, d[0]);
#pragma unroll
  for (int c = 0; c < COLS / N; ++c) {
    tmem_wait(d[c & 1]);
    if (c + 1 < COLS / N) {
      tmem_issue(taddr + N * (c + 1), d[(c + 1) & 1]);
    } else {
      tc_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(freed);
    }
#pragma unroll
    for (int q = 0; q < N / 2; ++q)
      fma2(acc[N / 2 * c + q], d[c & 1][2 * q], d[c & 1][2 * q + 1], s);
  }
}

template <int BN>
__global__ void __launch_bounds__(Shape<BN>::kThreads)
    fp8_gemm_kernel(const Fp8Params p, const __grid_constant__ CUtensorMap xmap,
                    const __grid_constant__ CUtensorMap wmap) {
  using Sh = Shape<BN>;
  constexpr int NS = Sh::kStages;
  // D fp32, A and B e4m3 (format 0), K-major, N = BN, M = 128
  constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(kTok >> 4) << 24);
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[NS], empty[NS], tfull[2], tempty[2];
  __shared__ uint32_t s_tmem;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the tile: token tiles first, kGroup of them at a time, then along W, so that a
  // group's X stays in L2 while W passes once
  int64_t n0, m0;
  {
    const int64_t wt = gridDim.x / C, t = (int64_t)blockIdx.y * wt + blockIdx.x / C;
    const int64_t first = t / (kGroup * wt) * kGroup, in = t - first * wt;
    const int64_t toks = min((int64_t)kGroup, (int64_t)gridDim.y - first);
    m0 = (first + in % toks) * kTok;
    n0 = in / toks * BN;
  }
  const int kb = (int)((p.k + kBlk - 1) / kBlk);
  const int b0 = (int)((int64_t)kb * rank / C), nb = (int)((int64_t)kb * (rank + 1) / C) - b0;
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tfull[s], 1);
      mbar_init(&tempty[s], 8);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&s_tmem)),
                 "r"(Sh::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      bool waited = !p.early_w;
      if (waited) asm volatile("griddepcontrol.wait;" ::: "memory");
      for (int j = 0; j < nb && ok; ++j) {
        const int s = j % NS;
        ok = ring_wait(&empty[s], ((uint32_t)(j / NS) & 1u) ^ 1u);
        if (!ok) break;
        uint8_t *st = smem + (size_t)s * Sh::kStage;
        mbar_arrive_expect_tx(&full[s], Sh::kStage);
        // W is no output of the preceding kernel; X (or its scales) may be
        tma_load_2d(st + kTok * kBlk, &wmap, (b0 + j) * kBlk, (int)n0, &full[s]);
        if (!waited) {
          asm volatile("griddepcontrol.wait;" ::: "memory");
          waited = true;
        }
        tma_load_2d(st, &xmap, (b0 + j) * kBlk, (int)m0, &full[s]);
      }
      if (!ok) atomicOr(p.status, kStatusTimeout);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      bool ok = true;
      // X is not there before that; a bounded wait must not count the time of the
      // kernel before this one
      asm volatile("griddepcontrol.wait;" ::: "memory");
      for (int j = 0; j < nb && ok; ++j) {
        const int s = j % NS, buf = j & 1;
        ok = ring_wait(&full[s], (uint32_t)(j / NS) & 1u) &&
             ring_wait(&tempty[buf], ((uint32_t)(j >> 1) & 1u) ^ 1u);
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = smem_u32(smem + (size_t)s * Sh::kStage), b = a + kTok * kBlk;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)  // 32 columns (32 bytes of the swizzle row) at a time
          umma_f8(tmem + buf * BN, sw128_desc(a + kk * 32), sw128_desc(b + kk * 32), kk != 0,
                  kIdesc);
        umma_commit(&empty[s]);
        umma_commit(&tfull[buf]);
      }
      if (!ok) atomicOr(p.status, kStatusTimeout);
    }
    __syncwarp();
  } else if (warp >= Sh::kCtl) {
    const int half = (warp - Sh::kCtl) >> 2;
    const int row = 32 * (warp & 3) + lane;  // this thread's token, its tensor-memory lane
    const uint32_t tbase = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)(half * Sh::kCols);
    uint64_t acc[Sh::kCols / 2];  // pairs of fp32
#pragma unroll
    for (int c = 0; c < Sh::kCols / 2; ++c) acc[c] = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float *sxp = p.sx + min(m0 + row, p.m - 1) * p.ldsx + b0;
    // the scale of this thread's columns (they lie in one block of 128 rows of W)
    const float *swp = p.sw + min(n0 + half * Sh::kCols, p.n - 1) / kBlk * p.ldsw + b0;
    float sx = 0.0f, sw = 0.0f;
    if (nb > 0) {
      sx = ld_dep(sxp);
      sw = ld_dep(swp);
    }
    bool ok = true;
    for (int j = 0; j < nb; ++j) {
      const int buf = j & 1;
      const float s = sx * sw;
      if (j + 1 < nb) {
        sx = ld_dep(sxp + j + 1);
        sw = ld_dep(swp + j + 1);
      }
      ok = ring_wait(&tfull[buf], (uint32_t)(j >> 1) & 1u);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      tc_fence_after();
      scale_add<Sh::kCols, Sh::kLoad>(tbase + buf * BN, s, acc, &tempty[buf]);
    }
    if (!ok && lane == 0) atomicOr(p.status, kStatusTimeout);
    // every epilogue thread is past its last block: the MMAs have read the ring
    asm volatile("bar.sync 1, 256;" ::: "memory");
    float *out = reinterpret_cast<float *>(smem) + row * Sh::kPitch + half * Sh::kCols;
#pragma unroll
    for (int c = 0; c < Sh::kCols; c += 4)
      *reinterpret_cast<ulonglong2 *>(out + c) = make_ulonglong2(acc[c / 2], acc[c / 2 + 1]);
  }
  tc_fence_before();
  __syncthreads();  // warps that wait here do not poll, as they would in the cluster's barrier
  if (C > 1) cluster.sync();

  // the cluster's CTAs share the rows: a warp takes a row of BN sums at a time, four
  // neighbours per lane
  {
    const int rows = (int)min((int64_t)kTok, p.m - m0);
    const float *mine = reinterpret_cast<const float *>(smem);
    const int es = p.bf16_out ? 2 : 4;
    const bool vec = ((uintptr_t)p.Y % (4 * es) == 0) && (p.ldy % 4 == 0);
    for (int r = rank + C * warp; r < rows; r += C * (Sh::kThreads / 32)) {
#pragma unroll
      for (int c = lane * 4; c < BN; c += 128) {
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (C == 1) {
          v = *reinterpret_cast<const float4 *>(mine + r * Sh::kPitch + c);
        } else {
          float4 a[kMaxC];  // all on their way at once, then added in order
#pragma unroll
          for (int q = 0; q < kMaxC; ++q)
            if (q < C)
              a[q] = *reinterpret_cast<const float4 *>(cluster.map_shared_rank(mine, q) +
                                                       r * Sh::kPitch + c);
#pragma unroll
          for (int q = 0; q < kMaxC; ++q)
            if (q < C) {
              v.x += a[q].x;
              v.y += a[q].y;
              v.z += a[q].z;
              v.w += a[q].w;
            }
        }
        const int64_t n = n0 + c, at = (m0 + r) * p.ldy + n;
        const float o[4] = {v.x, v.y, v.z, v.w};
        if (p.bf16_out) {
          uint16_t *y = static_cast<uint16_t *>(p.Y) + at;
          if (vec && n + 4 <= p.n) {
            *reinterpret_cast<uint2 *>(y) =
                make_uint2(f32_to_bf16_rne(o[0]) | ((uint32_t)f32_to_bf16_rne(o[1]) << 16),
                           f32_to_bf16_rne(o[2]) | ((uint32_t)f32_to_bf16_rne(o[3]) << 16));
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (n + q < p.n) y[q] = f32_to_bf16_rne(o[q]);
          }
        } else {
          float *y = static_cast<float *>(p.Y) + at;
          if (vec && n + 4 <= p.n) {
            *reinterpret_cast<float4 *>(y) = v;
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (n + q < p.n) y[q] = o[q];
          }
        }
      }
    }
  }
  if (C > 1) cluster.sync();  // no CTA leaves while another reads its shared memory
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(Sh::kTmem)
                 : "memory");
  }
}

// [rows][k] bytes, boxes of 128 columns x box_rows rows in the 128-byte swizzle
int encode_bytes(const void *base, int64_t k, int64_t rows, int64_t ld, int box_rows,
                 CUtensorMap *map) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (!encode) return HYB_ERR_CUDA;
  const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld};
  const cuuint32_t box[2] = {(cuuint32_t)kBlk, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult res = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims,
                              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return res == CUDA_SUCCESS ? HYB_OK : HYB_ERR_CUDA;
}

template <int BN>
int launch_gemm(const Fp8Params &p, int C, cudaStream_t st) {
  using Sh = Shape<BN>;
  const int64_t tiles = (p.n + BN - 1) / BN, toks = (p.m + kTok - 1) / kTok;
  if (tiles * C > INT32_MAX || toks > 65535) return HYB_ERR_UNSUPPORTED;
  alignas(64) CUtensorMap xmap{}, wmap{};
  int rc = encode_bytes(p.X, p.k, p.m, p.ldx, kTok, &xmap);
  if (rc == HYB_OK) rc = encode_bytes(p.W, p.k, p.n, p.ldw, BN, &wmap);
  if (rc != HYB_OK) return rc;
  const int dyn = Sh::kRing + 1024;
  static std::atomic<uint64_t> done{0};
  if (allow_smem(reinterpret_cast<const void *>(fp8_gemm_kernel<BN>), dyn, done) != HYB_OK)
    return HYB_ERR_CUDA;
  return launch_dependent(fp8_gemm_kernel<BN>, dim3((unsigned)(tiles * C), (unsigned)toks), Sh::kThreads, dyn, C, st, p,
                          xmap, wmap);
}

// ---------------------------------------------------------------------------
// decode
// ---------------------------------------------------------------------------
//
// The same product for m <= 32 tokens, which is bound by W's bytes: the tokens
// fill one warp's lanes of the MMA's 128 rows and the other lanes' products are
// not looked at (the MMA unit has the time, and its operand rows 32 .. 127 are
// whatever lies behind X's 4 KB: W's tile, and behind a narrow one the next
// stage's).  Two warps, half of the columns each, scale and add.  16 x 4096 x
// 14336: 15.8 us with the quantiser's kernel, 13.8 us (4.3 TB/s) without (13.1 and 11.4
// where W is in L2); its 256 equal CTAs leave some SMs with two and some with one, and
// the clusters' start and last sums come on top.  Quantising a
// bf16 X in this kernel, by the warps that are idle, was slower than a kernel
// before it that this one overlaps (16 x 4096 x 14336: 27 us and 16 us): every
// row tile does that work again.

// warps 0 and 4 (whose tensor-memory lanes hold the tokens): epilogue; 1: MMA;
// 2: TMA
constexpr int kDecodeThreads = 160;

template <int BN>
struct DecodeShape {
  static constexpr int kStage = (kDecodeTokens + BN) * kBlk;
  static constexpr int kStages = BN == 128 ? 5 : 8;
  static constexpr int kTail = kTok * kBlk > kStage ? kTok * kBlk - kStage : 0;
  static constexpr int kBytes = kStage * kStages + kTail;
  static constexpr int kCols = BN / 2;
  static constexpr int kPitch = BN + 4;
  static constexpr int kTmem = 2 * BN;
  static constexpr int kLoad = 16;
  static_assert(kDecodeTokens * kPitch * 4 <= kStage * kStages, "the result reuses the ring");
  static_assert(tmem_fits(kTmem, kBytes), "tensor memory of the CTAs that fit an SM");
  static_assert(kStage % 1024 == 0, "swizzle alignment");
};

template <int BN>
__global__ void __launch_bounds__(kDecodeThreads, 2)
    fp8_decode_kernel(const Fp8Params p, const __grid_constant__ CUtensorMap xmap,
                      const __grid_constant__ CUtensorMap wmap) {
  using Sh = DecodeShape<BN>;
  constexpr int NS = Sh::kStages;
  constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(kTok >> 4) << 24);
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[NS], empty[NS], tfull[2], tempty[2];
  __shared__ uint32_t s_tmem;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t n0 = (int64_t)(blockIdx.x / C) * BN;
  const int kb = (int)((p.k + kBlk - 1) / kBlk);
  const int b0 = (int)((int64_t)kb * rank / C), nb = (int)((int64_t)kb * (rank + 1) / C) - b0;
  const int m = (int)p.m;
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  auto load_w = [&](int j) {
    const int s = j % NS;
    mbar_arrive_expect_tx(&full[s], Sh::kStage);
    tma_load_2d(smem + (size_t)s * Sh::kStage + kDecodeTokens * kBlk, &wmap, (b0 + j) * kBlk,
                (int)n0, &full[s]);
  };
  if (tid == 64) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tfull[s], 1);
      mbar_init(&tempty[s], 2);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    // W's first blocks set out before anything else is ready
    if (!p.early_w) asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int j = 0; j < min(nb, NS); ++j) load_w(j);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&s_tmem)),
                 "r"(Sh::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  if (warp == 2) {
    if (lane == 0) {
      bool ok = true;
      asm volatile("griddepcontrol.wait;" ::: "memory");
      for (int j = 0; j < nb && ok; ++j) {
        const int s = j % NS;
        if (j >= NS) {
          ok = ring_wait(&empty[s], ((uint32_t)(j / NS) & 1u) ^ 1u);
          if (!ok) break;
          load_w(j);
        }
        tma_load_2d(smem + (size_t)s * Sh::kStage, &xmap, (b0 + j) * kBlk, 0, &full[s]);
      }
      if (!ok) atomicOr(p.status, kStatusTimeout);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      bool ok = true;
      // X is not there before that; a bounded wait must not count the time of the
      // kernel before this one
      asm volatile("griddepcontrol.wait;" ::: "memory");
      for (int j = 0; j < nb && ok; ++j) {
        const int s = j % NS, buf = j & 1;
        ok = ring_wait(&full[s], (uint32_t)(j / NS) & 1u) &&
             ring_wait(&tempty[buf], ((uint32_t)(j >> 1) & 1u) ^ 1u);
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = smem_u32(smem + (size_t)s * Sh::kStage), b = a + kDecodeTokens * kBlk;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f8(tmem + buf * BN, sw128_desc(a + kk * 32), sw128_desc(b + kk * 32), kk != 0,
                  kIdesc);
        umma_commit(&empty[s]);
        umma_commit(&tfull[buf]);
      }
      if (!ok) atomicOr(p.status, kStatusTimeout);
    }
    __syncwarp();
  } else if (warp != 3) {
    // scale and add: lane = token (lanes 0 .. 31 of tensor memory), half of the columns
    const int half = warp >> 2;
    const uint32_t tbase = tmem + (uint32_t)(half * Sh::kCols);
    uint64_t acc[Sh::kCols / 2];  // pairs of fp32
#pragma unroll
    for (int c = 0; c < Sh::kCols / 2; ++c) acc[c] = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float *sxp = p.sx + min(lane, m - 1) * p.ldsx + b0;
    const float *swp = p.sw + min(n0 + half * Sh::kCols, p.n - 1) / kBlk * p.ldsw + b0;
    float sx = 0.0f, sw = 0.0f;
    if (nb > 0) {
      sx = ld_dep(sxp);
      sw = ld_dep(swp);
    }
    bool ok = true;
    for (int j = 0; j < nb; ++j) {
      const int buf = j & 1;
      const float s = sx * sw;
      if (j + 1 < nb) {
        sx = ld_dep(sxp + j + 1);
        sw = ld_dep(swp + j + 1);
      }
      ok = ring_wait(&tfull[buf], (uint32_t)(j >> 1) & 1u);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      tc_fence_after();
      scale_add<Sh::kCols, Sh::kLoad>(tbase + buf * BN, s, acc, &tempty[buf]);
    }
    if (!ok && lane == 0) atomicOr(p.status, kStatusTimeout);
    if (lane < m) {  // past the last block: the MMAs have read the ring
      float *out = reinterpret_cast<float *>(smem) + lane * Sh::kPitch + half * Sh::kCols;
#pragma unroll
      for (int c = 0; c < Sh::kCols; c += 4)
        *reinterpret_cast<ulonglong2 *>(out + c) = make_ulonglong2(acc[c / 2], acc[c / 2 + 1]);
    }
  }
  tc_fence_before();
  __syncthreads();  // warps that wait here do not poll, as they would in the cluster's barrier
  if (C > 1) cluster.sync();

  // the cluster's CTAs share the sums, four columns of a token at a time, each a
  // stretch of neighbours: a warp's reads of another CTA's memory are then whole
  // rows (with every C-th one 4096 x 14336 took 3 us more at 32 tokens)
  {
    const float *mine = reinterpret_cast<const float *>(smem);
    const int es = p.bf16_out ? 2 : 4;
    const bool vec = ((uintptr_t)p.Y % (4 * es) == 0) && (p.ldy % 4 == 0);
    const int share = (m * (BN / 4) + C - 1) / C, e1 = min((rank + 1) * share, m * (BN / 4));
    for (int e = rank * share + tid; e < e1; e += kDecodeThreads) {
      const int r = e / (BN / 4), c = e % (BN / 4) * 4;
      float4 a[kMaxC];  // all on their way at once, then added in order
#pragma unroll
      for (int q = 0; q < kMaxC; ++q)
        if (q < C)
          a[q] = *reinterpret_cast<const float4 *>(
              (C == 1 ? mine : cluster.map_shared_rank(mine, q)) + r * Sh::kPitch + c);
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int q = 0; q < kMaxC; ++q)
        if (q < C) {
          v.x += a[q].x;
          v.y += a[q].y;
          v.z += a[q].z;
          v.w += a[q].w;
        }
      const int64_t n = n0 + c, at = r * p.ldy + n;
      const float o[4] = {v.x, v.y, v.z, v.w};
      if (p.bf16_out) {
        uint16_t *y = static_cast<uint16_t *>(p.Y) + at;
        if (vec && n + 4 <= p.n) {
          *reinterpret_cast<uint2 *>(y) =
              make_uint2(f32_to_bf16_rne(o[0]) | ((uint32_t)f32_to_bf16_rne(o[1]) << 16),
                         f32_to_bf16_rne(o[2]) | ((uint32_t)f32_to_bf16_rne(o[3]) << 16));
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (n + q < p.n) y[q] = f32_to_bf16_rne(o[q]);
        }
      } else {
        float *y = static_cast<float *>(p.Y) + at;
        if (vec && n + 4 <= p.n) {
          *reinterpret_cast<float4 *>(y) = v;
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (n + q < p.n) y[q] = o[q];
        }
      }
    }
  }
  if (C > 1) cluster.sync();  // no CTA leaves while another reads its shared memory
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(Sh::kTmem)
                 : "memory");
  }
}

template <int BN>
int launch_decode(const Fp8Params &p, int C, cudaStream_t st) {
  using Sh = DecodeShape<BN>;
  const int64_t tiles = (p.n + BN - 1) / BN;
  if (tiles * C > INT32_MAX) return HYB_ERR_UNSUPPORTED;
  alignas(64) CUtensorMap xmap{}, wmap{};
  int rc = encode_bytes(p.W, p.k, p.n, p.ldw, BN, &wmap);
  if (rc == HYB_OK) rc = encode_bytes(p.X, p.k, p.m, p.ldx, kDecodeTokens, &xmap);
  if (rc != HYB_OK) return rc;
  const int dyn = Sh::kBytes + 1024;
  static std::atomic<uint64_t> done{0};
  if (allow_smem(reinterpret_cast<const void *>(fp8_decode_kernel<BN>), dyn, done) != HYB_OK)
    return HYB_ERR_CUDA;
  return launch_dependent(fp8_decode_kernel<BN>, dim3((unsigned)(tiles * C)), kDecodeThreads, dyn, C, st, p,
                          xmap, wmap);
}

}  // namespace

int fp8_decode(const Fp8Params &p, cudaStream_t st) {
  int sms;
  const int rc = device_sm_count(&sms);
  if (rc != HYB_OK) return rc;
  const int64_t kb = (p.k + kBlk - 1) / kBlk;
  // two CTAs fit an SM; a cluster has at most 8 and each CTA at least 2 blocks
  const bool narrow = (p.n + 127) / 128 * 8 < sms;
  const int64_t tiles = narrow ? (p.n + 63) / 64 : (p.n + 127) / 128;
  int64_t C = 2 * sms / tiles;
  if (C > kb / 2) C = kb / 2;
  C = C < 1 ? 1 : (C > kMaxC ? kMaxC : C);
  return narrow ? launch_decode<64>(p, (int)C, st)
                : launch_decode<128>(p, (int)C, st);
}

int fp8_gemm(const Fp8Params &p, cudaStream_t st) {
  int sms;
  const int rc = device_sm_count(&sms);
  if (rc != HYB_OK) return rc;
  const int64_t toks = (p.m + kTok - 1) / kTok;
  const int64_t kb = (p.k + kBlk - 1) / kBlk;
  const int64_t wide = (p.n + 255) / 256 * toks;
  // 256 columns where one CTA per SM fills more than half of the GPU (6144 x 4096, 700
  // tokens: 29 us, and 54 us with 128 columns when this was chosen); else 128, two
  // CTAs per SM, and k split while they fit (300 x 14336, 1000 tokens: 28 us, 41 us
  // with 256 columns); the border itself was not measured
  if (2 * wide > sms) return launch_gemm<256>(p, 1, st);
  const int64_t tiles = (p.n + 127) / 128 * toks;
  int C = 1;
  while (C < kMaxC && tiles * C * 2 <= 2 * sms && kb >= 4 * C) C *= 2;
  return launch_gemm<128>(p, C, st);
}

}  // namespace hyb
