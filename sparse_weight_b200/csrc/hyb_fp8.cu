// Products with an 8-bit floating-point weight (e4m3, one fp32 scale per
// 128 x 128 block) and activations in e4m3 with one fp32 scale per token and
// 128 columns:
//
//   Y[m][n] = sum_b sx[m][b] sw[n / 128][b] sum_{k in block b} xq[m][k] wq[n][k]
//
// and the quantiser that makes both operands (hyb_fp8_quant):
//
//   a = max(largest finite |x| of the block, 448 * 2^-64)
//   scale = a / 448,   q = e4m3(sat(x * (448 / a)))
//
// every operation rounded to fp32 once, the last one to e4m3 (round to nearest
// even, saturating at +-448; a NaN stays a NaN).
#include "hyb_fp8.cuh"

#include <cooperative_groups.h>
#include <cuda_fp8.h>

namespace cg = cooperative_groups;

namespace hyb {
namespace {

constexpr float kE4m3Max = 448.0f;
// blocks whose largest value is smaller quantise as if it were this (an all-
// zero block then needs no case of its own): 448 * 2^-64
constexpr float kMinAmax = 448.0f / 18446744073709551616.0f;

// largest finite |x| so far; flags a NaN or an infinity
__device__ __forceinline__ void amax_finite(float x, float &a, bool &bad) {
  const float v = fabsf(x);
  const bool fin = v <= 3.402823466e38f;  // false for NaN and infinity
  bad |= !fin;
  a = fmaxf(a, fin ? v : 0.0f);
}

// two fp32 -> two e4m3 bytes (lo in the low byte), round to nearest even,
// saturating; NaN -> 0x7F
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

// 8 consecutive values of a row as fp32; those at or past `left` read as zero.
// `vec`: the rows start on 16 bytes (else they are read value by value).
template <bool F32>
__device__ __forceinline__ void load8(const void *X, int64_t off, int left, bool vec,
                                      float (&v)[8]) {
  if (left >= 8 && vec) {
    if constexpr (F32) {
      const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(X) + off);
      const float4 a = __ldg(p), b = __ldg(p + 1);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      const uint4 r = ld_keep16(static_cast<const uint16_t *>(X) + off);
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = 0.0f;
      if (i < left) {
        if constexpr (F32)
          v[i] = static_cast<const float *>(X)[off + i];
        else
          v[i] = __uint_as_float((uint32_t) static_cast<const uint16_t *>(X)[off + i] << 16);
      }
    }
  }
}

// 8 bytes of a row; those at or past `left` are not written
__device__ __forceinline__ void store8(uint8_t *Q, int64_t off, int left, uint2 w) {
  if (left >= 8) {
    *reinterpret_cast<uint2 *>(Q + off) = w;
  } else {
    for (int i = 0; i < left; ++i)
      Q[off + i] = (uint8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
  }
}

// One scale per row and 128 columns.  A half-warp owns one block at a time (16
// lanes x 8 values: 16 bytes of bf16 per lane, 8 bytes written).
template <bool F32>
__global__ void __launch_bounds__(256) fp8_quant_rows_kernel(int64_t rows, int64_t cols,
                                                             const void *X, int64_t ldx,
                                                             uint8_t *Q, int64_t ldq,
                                                             float *scale, int64_t lds,
                                                             int64_t cb, bool vec, uint32_t *status) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 15;
  const int64_t unit = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const unsigned half = 0xFFFFu << (threadIdx.x & 16);
  if (unit >= rows * cb) return;
  const int64_t row = unit / cb, blk = unit - row * cb;
  const int64_t col = blk * kBlk + lane * 8;
  const int left = (int)max((int64_t)0, min((int64_t)8, cols - col));
  float v[8];
  load8<F32>(X, row * ldx + col, left, vec, v);
  float a = 0.0f;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax_finite(v[i], a, bad);
#pragma unroll
  for (int o = 8; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(half, a, o));
  a = fmaxf(a, kMinAmax);
  const float inv = __fdiv_rn(kE4m3Max, a);
  uint2 w;
  w.x = e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
  w.y = e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
  store8(Q, row * ldq + col, left, w);
  if (lane == 0) scale[row * lds + blk] = __fdiv_rn(a, kE4m3Max);
  if (bad) atomicOr(status, kStatusNaN);
}

// One scale per 128 x 128 block: one CTA per block, 64 values per thread kept
// in registers between the two passes.
template <bool F32>
__global__ void __launch_bounds__(256) fp8_quant_blocks_kernel(int64_t rows, int64_t cols,
                                                               const void *X, int64_t ldx,
                                                               uint8_t *Q, int64_t ldq,
                                                               float *scale, int64_t lds,
                                                               bool vec, uint32_t *status) {
  __shared__ float s_a[8];
  const int lane = threadIdx.x & 15, r16 = threadIdx.x >> 4;
  const int64_t col = (int64_t)blockIdx.x * kBlk + lane * 8;
  const int64_t row0 = (int64_t)blockIdx.y * kBlk + r16;
  const int left = (int)max((int64_t)0, min((int64_t)8, cols - col));
  float v[8][8];
  float a = 0.0f;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t row = row0 + 16 * j;
    load8<F32>(X, row * ldx + col, row < rows ? left : 0, vec, v[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) amax_finite(v[j][i], a, bad);
#pragma unroll
  for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
  if ((threadIdx.x & 31) == 0) s_a[threadIdx.x >> 5] = a;
  __syncthreads();
  a = kMinAmax;
#pragma unroll
  for (int w = 0; w < 8; ++w) a = fmaxf(a, s_a[w]);
  const float inv = __fdiv_rn(kE4m3Max, a);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t row = row0 + 16 * j;
    uint2 w;
    w.x = e4m3x4(v[j][0] * inv, v[j][1] * inv, v[j][2] * inv, v[j][3] * inv);
    w.y = e4m3x4(v[j][4] * inv, v[j][5] * inv, v[j][6] * inv, v[j][7] * inv);
    if (row < rows) store8(Q, row * ldq + col, left, w);
  }
  if (threadIdx.x == 0) scale[(int64_t)blockIdx.y * lds + blockIdx.x] = __fdiv_rn(a, kE4m3Max);
  if (bad) atomicOr(status, kStatusNaN);
}

template <typename... P, typename... A>
int launch(void (*kernel)(P...), dim3 grid, bool overlap, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = overlap ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, (P)args...) == cudaSuccess ? HYB_OK : HYB_ERR_CUDA;
}

int quant_launch(int64_t rows, int64_t cols, const void *X, int64_t ldx, hyb_dtype xdt,
                 int block_rows, uint8_t *Q, int64_t ldq, float *scale, int64_t lds,
                 uint32_t *status, bool overlap, cudaStream_t st) {
  const int64_t cb = (cols + kBlk - 1) / kBlk;
  const bool vec = (uintptr_t)X % 16 == 0 && ldx % (xdt == HYB_F32 ? 4 : 8) == 0;
  if (block_rows == 1) {
    const int64_t ctas = (rows * cb + 15) / 16;
    if (ctas > INT32_MAX) return HYB_ERR_UNSUPPORTED;
    return launch(xdt == HYB_F32 ? fp8_quant_rows_kernel<true> : fp8_quant_rows_kernel<false>,
                  dim3((unsigned)ctas), overlap, st, rows, cols, X, ldx, Q, ldq, scale, lds, cb,
                  vec, status);
  }
  const int64_t rb = (rows + kBlk - 1) / kBlk;
  if (rb > 65535 || cb > INT32_MAX) return HYB_ERR_UNSUPPORTED;
  return launch(xdt == HYB_F32 ? fp8_quant_blocks_kernel<true> : fp8_quant_blocks_kernel<false>,
                dim3((unsigned)cb, (unsigned)rb), overlap, st, rows, cols, X, ldx, Q, ldq, scale,
                lds, vec, status);
}

// ---------------------------------------------------------------------------
// skinny product
// ---------------------------------------------------------------------------

// D += A B, one m16n8k32 e4m3 product with fp32 accumulation
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the bytes of a 16-byte word below `left` (>= 0), zeros behind
__device__ __forceinline__ uint4 keep_bytes(uint4 v, int left) {
  if (left >= 16) return v;
  uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = left - 4 * i;
    w[i] = b >= 4 ? w[i] : (b <= 0 ? 0u : w[i] & ((1u << (8 * b)) - 1u));
  }
  return v;
}

// Y of 16 RT WR weight rows and 8 NT tokens per cluster.  The 8 warps are WR
// row groups x 8 / WR slices of K; the cluster's CTAs split K further, and its
// partial sums meet in distributed shared memory in a fixed order.
//
// A fragment register of m16n8k32 holds 4 bytes of K; the sum over a block
// does not care which of the block's columns sit in which register as long as
// both operands agree, so a lane takes 16 consecutive bytes of its row and
// feeds them to two products: every load of W is 16 bytes straight from
// global memory to the fragment registers, with no shared memory between.
template <int NT, int RT, int WR, bool XBF16>
__global__ void __launch_bounds__(256) fp8_skinny_kernel(const Fp8Params p) {
  constexpr int WK = 8 / WR;
  constexpr int ROWS = 16 * RT * WR;
  constexpr int TOK = 8 * NT;
  __shared__ float part[WK][TOK][ROWS + 4];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks();
  const int rank = (int)cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int wr = warp % WR, wk = warp / WR;
  const int64_t row0 = (int64_t)(blockIdx.x / C) * ROWS;
  const int64_t tok0 = (int64_t)blockIdx.y * TOK;
  const int kb = (int)((p.k + kBlk - 1) / kBlk);
  const int step = WK * C;
  const int64_t wrow = row0 + wr * 16 * RT;

  // this lane's rows of W (rows past the end read as zeros)
  const uint8_t *wp[RT][2];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t row = wrow + r * 16 + h * 8 + g;
      wp[r][h] = row < p.n ? p.W + row * p.ldw : nullptr;
    }
  float acc[RT][NT][4];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[r][i][c] = 0.0f;

  auto load_w = [&](int b, uint4 (&w)[RT][2][2]) {
    const int64_t c0 = (int64_t)b * kBlk + t * 16;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int64_t c = c0 + 64 * q;
          w[r][h][q] = make_uint4(0, 0, 0, 0);
          if (b < kb && wp[r][h] != nullptr && c < p.k) w[r][h][q] = ld_stream16(wp[r][h] + c);
        }
  };

  bool bad = false;
  uint4 nxt[RT][2][2];
  int b = rank * WK + wk;
  load_w(b, nxt);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (; b < kb; b += step) {
    uint4 w[RT][2][2];
    const bool tail = (int64_t)(b + 1) * kBlk > p.k;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 2; ++q) w[r][h][q] = nxt[r][h][q];
    load_w(b + step, nxt);
    if (tail) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int left = (int)max((int64_t)0, p.k - ((int64_t)b * kBlk + t * 16 + 64 * q));
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int h = 0; h < 2; ++h) w[r][h][q] = keep_bytes(w[r][h][q], left);
      }
    }
    float swv[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int64_t row = min(wrow + r * 16, p.n - 1);
      swv[r] = __ldg(p.sw + (row / kBlk) * p.ldsw + b);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      // B fragments: token g of this tile, 2 x 16 columns
      const int64_t tok = tok0 + i * 8 + g;
      const bool live = tok < p.m;
      uint4 x[2];
      float sx = 0.0f;
      if constexpr (XBF16) {
        float v[2][16];
        float a = 0.0f;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int64_t c = (int64_t)b * kBlk + t * 16 + 64 * q;
          const int left = live ? (int)max((int64_t)0, min((int64_t)16, p.k - c)) : 0;
          float lo[8], hi[8];
          load8<false>(p.X, tok * p.ldx + c, min(left, 8), true, lo);
          load8<false>(p.X, tok * p.ldx + c + 8, max(left - 8, 0), true, hi);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[q][e] = lo[e];
            v[q][8 + e] = hi[e];
          }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int e = 0; e < 16; ++e) amax_finite(v[q][e], a, bad);
        a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
        a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 2));
        a = fmaxf(a, kMinAmax);
        const float inv = __fdiv_rn(kE4m3Max, a);
        sx = __fdiv_rn(a, kE4m3Max);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          x[q].x = e4m3x4(v[q][0] * inv, v[q][1] * inv, v[q][2] * inv, v[q][3] * inv);
          x[q].y = e4m3x4(v[q][4] * inv, v[q][5] * inv, v[q][6] * inv, v[q][7] * inv);
          x[q].z = e4m3x4(v[q][8] * inv, v[q][9] * inv, v[q][10] * inv, v[q][11] * inv);
          x[q].w = e4m3x4(v[q][12] * inv, v[q][13] * inv, v[q][14] * inv, v[q][15] * inv);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int64_t c = (int64_t)b * kBlk + t * 16 + 64 * q;
          x[q] = make_uint4(0, 0, 0, 0);
          if (live && c < p.k)
            x[q] = keep_bytes(ld_keep16(static_cast<const uint8_t *>(p.X) + tok * p.ldx + c),
                              (int)min((int64_t)16, p.k - c));
        }
        if (live) sx = __ldg(p.sx + tok * p.ldsx + b);
      }
      // the scales of this lane's result columns, tokens 2 t and 2 t + 1
      const float s0 = __shfl_sync(0xFFFFFFFFu, sx, 8 * t);
      const float s1 = __shfl_sync(0xFFFFFFFFu, sx, 8 * t + 4);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          mma_e4m3(d, w[r][0][q].x, w[r][1][q].x, w[r][0][q].y, w[r][1][q].y, x[q].x, x[q].y);
          mma_e4m3(d, w[r][0][q].z, w[r][1][q].z, w[r][0][q].w, w[r][1][q].w, x[q].z, x[q].w);
        }
        acc[r][i][0] += d[0] * (s0 * swv[r]);
        acc[r][i][1] += d[1] * (s1 * swv[r]);
        acc[r][i][2] += d[2] * (s0 * swv[r]);
        acc[r][i][3] += d[3] * (s1 * swv[r]);
      }
    }
  }
  if (XBF16 && bad) atomicOr(p.status, kStatusNaN);

  // partial sums: this CTA's K slices, then the cluster's CTAs, in order
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        part[wk][i * 8 + 2 * t + (c & 1)][wr * 16 * RT + r * 16 + (c >> 1) * 8 + g] = acc[r][i][c];
  __syncthreads();
  for (int e = threadIdx.x; e < ROWS * TOK; e += 256) {
    const int row = e % ROWS, tok = e / ROWS;
    float s = part[0][tok][row];
#pragma unroll
    for (int j = 1; j < WK; ++j) s += part[j][tok][row];
    part[0][tok][row] = s;
  }
  cluster.sync();
  const int per = (ROWS * TOK + C - 1) / C;
  for (int e = rank * per + (int)threadIdx.x; e < min((rank + 1) * per, ROWS * TOK); e += 256) {
    const int row = e % ROWS, tok = e / ROWS;
    float s = 0.0f;
    for (int j = 0; j < C; ++j) s += *cluster.map_shared_rank(&part[0][tok][row], j);
    const int64_t yr = row0 + row, yt = tok0 + tok;
    if (yr < p.n && yt < p.m) {
      if (p.bf16_out)
        static_cast<uint16_t *>(p.Y)[yt * p.ldy + yr] = f32_to_bf16_rne(s);
      else
        static_cast<float *>(p.Y)[yt * p.ldy + yr] = s;
    }
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

template <int NT, int RT, int WR, bool XBF16>
int launch_skinny(const Fp8Params &p, int C, bool overlap, cudaStream_t st) {
  const int64_t tiles = (p.n + 16 * RT * WR - 1) / (16 * RT * WR);
  const int64_t toks = (p.m + 8 * NT - 1) / (8 * NT);
  if (tiles * C > INT32_MAX || toks > 65535) return HYB_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * C), (unsigned)toks);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = overlap ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fp8_skinny_kernel<NT, RT, WR, XBF16>, p) == cudaSuccess
             ? HYB_OK
             : HYB_ERR_CUDA;
}

// the most tokens that the skinny kernel takes
constexpr int kSkinnyTokens = 16;

// X's values in the workspace, behind its scales
size_t fp8_x_offset(int64_t m, int64_t k) {
  return align_up(kHeaderBytes + (size_t)m * (size_t)((k + kBlk - 1) / kBlk) * 4, 256);
}

int fp8_check(const hyb_fp8_matrix *A) {
  if (!A || !A->q || !A->scale) return HYB_ERR_INVALID_ARG;
  if (A->n < 1 || A->k < 1 || A->ldq < A->k || A->lds < (A->k + kBlk - 1) / kBlk)
    return HYB_ERR_INVALID_ARG;
  if (A->n > INT32_MAX || A->k > INT32_MAX - kBlk) return HYB_ERR_UNSUPPORTED;
  if ((uintptr_t)A->q % 16 != 0 || A->ldq % 16 != 0 || (uintptr_t)A->scale % 4 != 0)
    return HYB_ERR_ALIGNMENT;
  return HYB_OK;
}

}  // namespace
}  // namespace hyb

using namespace hyb;

size_t hyb_fp8_quant_workspace_bytes(void) { return kHeaderBytes; }

int hyb_fp8_quant(int64_t rows, int64_t cols, const void *X, int64_t ldx, hyb_dtype xdt,
                  int block_rows, uint8_t *Q, int64_t ldq, float *scale, int64_t lds, void *ws,
                  size_t ws_bytes, hyb_stream_t stream) {
  if (!X || !Q || !scale || rows < 1 || cols < 1) return HYB_ERR_INVALID_ARG;
  if (xdt != HYB_F32 && xdt != HYB_BF16) return HYB_ERR_INVALID_ARG;
  if (block_rows != 1 && block_rows != kBlk) return HYB_ERR_INVALID_ARG;
  if (rows > INT32_MAX || cols > INT32_MAX - kBlk) return HYB_ERR_UNSUPPORTED;
  if (ldx < cols || ldq < cols || lds < (cols + kBlk - 1) / kBlk) return HYB_ERR_INVALID_ARG;
  if ((uintptr_t)X % (xdt == HYB_F32 ? 4 : 2) != 0 || (uintptr_t)Q % 16 != 0 || ldq % 16 != 0 ||
      (uintptr_t)scale % 4 != 0)
    return HYB_ERR_ALIGNMENT;
  if (!ws || ws_bytes < kHeaderBytes) return HYB_ERR_WORKSPACE;
  if ((uintptr_t)ws % 256 != 0) return HYB_ERR_ALIGNMENT;
  return quant_launch(rows, cols, X, ldx, xdt, block_rows, Q, ldq, scale, lds,
                      static_cast<uint32_t *>(ws), false, (cudaStream_t)stream);
}

// workspace: header; for the tensor-core product also X's scales and values
size_t hyb_fp8_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  if (m < 1 || n < 1 || k < 1 || m > INT32_MAX || n > INT32_MAX || k > INT32_MAX - kBlk) return 0;
  if (m <= kSkinnyTokens) return kHeaderBytes;
  return fp8_x_offset(m, k) + (size_t)m * align_up((size_t)k, 16);
}

int hyb_fp8_matmul(const hyb_fp8_matrix *A, int64_t m, const void *X, int64_t ldx, hyb_dtype xdt,
                   const float *xs, int64_t ldxs, void *Y, int64_t ldy, hyb_dtype ydt,
                   uint32_t flags, void *ws, size_t ws_bytes, hyb_stream_t stream) {
  int rc = fp8_check(A);
  if (rc != HYB_OK) return rc;
  if (!X || !Y || m < 1) return HYB_ERR_INVALID_ARG;
  if (xdt != HYB_BF16 && xdt != HYB_E4M3) return HYB_ERR_INVALID_ARG;
  if ((xdt == HYB_E4M3) != (xs != nullptr)) return HYB_ERR_INVALID_ARG;
  if (ydt != HYB_F32 && ydt != HYB_BF16) return HYB_ERR_INVALID_ARG;
  if (flags & ~HYB_LAUNCH_OVERLAP_PREV) return HYB_ERR_INVALID_ARG;
  const int64_t kb = (A->k + kBlk - 1) / kBlk;
  if (ldx < A->k || ldy < A->n || (xs && ldxs < kb)) return HYB_ERR_INVALID_ARG;
  if (m > INT32_MAX) return HYB_ERR_UNSUPPORTED;
  if ((uintptr_t)X % 16 != 0 || ldx % (xdt == HYB_BF16 ? 8 : 16) != 0 ||
      (uintptr_t)Y % (ydt == HYB_F32 ? 4 : 2) != 0 || (uintptr_t)xs % 4 != 0)
    return HYB_ERR_ALIGNMENT;
  if (!ws || ws_bytes < hyb_fp8_workspace_bytes(m, A->n, A->k)) return HYB_ERR_WORKSPACE;
  if ((uintptr_t)ws % 256 != 0) return HYB_ERR_ALIGNMENT;
  Fp8Params p{};
  p.n = A->n;
  p.k = A->k;
  p.m = m;
  p.W = A->q;
  p.ldw = A->ldq;
  p.sw = A->scale;
  p.ldsw = A->lds;
  p.X = X;
  p.ldx = ldx;
  p.sx = xs;
  p.ldsx = ldxs;
  p.Y = Y;
  p.ldy = ldy;
  p.bf16_out = ydt == HYB_BF16;
  p.status = static_cast<uint32_t *>(ws);
  const bool overlap = (flags & HYB_LAUNCH_OVERLAP_PREV) != 0;
  cudaStream_t st = (cudaStream_t)stream;
  const bool bf = xdt == HYB_BF16;
  if (m > kSkinnyTokens) {
    if (bf) {
      uint8_t *base = static_cast<uint8_t *>(ws);
      float *sx = reinterpret_cast<float *>(base + kHeaderBytes);
      uint8_t *xq = base + fp8_x_offset(m, A->k);
      const int64_t ld = (int64_t)align_up((size_t)A->k, 16);
      rc = quant_launch(m, A->k, X, ldx, HYB_BF16, 1, xq, ld, sx, kb, p.status, overlap, st);
      if (rc != HYB_OK) return rc;
      p.X = xq;
      p.ldx = ld;
      p.sx = sx;
      p.ldsx = kb;
    }
    return fp8_gemm(p, bf || overlap, st);
  }
  if (m <= 8)
    return bf ? launch_skinny<1, 2, 1, true>(p, 4, overlap, st)
              : launch_skinny<1, 2, 1, false>(p, 4, overlap, st);
  return bf ? launch_skinny<2, 2, 4, true>(p, 8, overlap, st)
            : launch_skinny<2, 2, 4, false>(p, 8, overlap, st);
}
