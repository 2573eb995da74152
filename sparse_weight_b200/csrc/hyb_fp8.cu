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

namespace hyb {
namespace {

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
  // dependents start once the preceding kernel has ended: a product behind this
  // kernel may then read W at once
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
  asm volatile("griddepcontrol.wait;" ::: "memory");
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

int quant_launch(int64_t rows, int64_t cols, const void *X, int64_t ldx, hyb_dtype xdt,
                 int block_rows, uint8_t *Q, int64_t ldq, float *scale, int64_t lds,
                 uint32_t *status, cudaStream_t st) {
  const int64_t cb = (cols + kBlk - 1) / kBlk;
  const bool vec = (uintptr_t)X % 16 == 0 && ldx % (xdt == HYB_F32 ? 4 : 8) == 0;
  if (block_rows == 1) {
    const int64_t ctas = (rows * cb + 15) / 16;
    if (ctas > INT32_MAX) return HYB_ERR_UNSUPPORTED;
    return launch_dependent(
        xdt == HYB_F32 ? fp8_quant_rows_kernel<true> : fp8_quant_rows_kernel<false>,
        dim3((unsigned)ctas), 256, 0, 1, st, rows, cols, X, ldx, Q, ldq, scale, lds, cb, vec,
        status);
  }
  const int64_t rb = (rows + kBlk - 1) / kBlk;
  if (rb > 65535 || cb > INT32_MAX) return HYB_ERR_UNSUPPORTED;
  return launch_dependent(
      xdt == HYB_F32 ? fp8_quant_blocks_kernel<true> : fp8_quant_blocks_kernel<false>,
      dim3((unsigned)cb, (unsigned)rb), 256, 0, 1, st, rows, cols, X, ldx, Q, ldq, scale, lds, vec,
      status);
}

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
                      static_cast<uint32_t *>(ws), (cudaStream_t)stream);
}

// workspace: header; but for small products also X's scales and values
size_t hyb_fp8_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  if (m < 1 || n < 1 || k < 1 || m > INT32_MAX || n > INT32_MAX || k > INT32_MAX - kBlk) return 0;
  if (fp8_is_small(m, n, k)) return kHeaderBytes;
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
  p.early_w = (flags & HYB_LAUNCH_OVERLAP_PREV) != 0;
  cudaStream_t st = (cudaStream_t)stream;
  p.x_bf16 = xdt == HYB_BF16;
  if (fp8_is_small(m, A->n, A->k)) return fp8_small(p, st);
  if (p.x_bf16) {
    uint8_t *base = static_cast<uint8_t *>(ws);
    float *sx = reinterpret_cast<float *>(base + kHeaderBytes);
    uint8_t *xq = base + fp8_x_offset(m, A->k);
    const int64_t ld = (int64_t)align_up((size_t)A->k, 16);
    rc = quant_launch(m, A->k, X, ldx, HYB_BF16, 1, xq, ld, sx, kb, p.status, st);
    if (rc != HYB_OK) return rc;
    p.X = xq;
    p.ldx = ld;
    p.sx = sx;
    p.ldsx = kb;
    p.x_bf16 = 0;
    p.early_w = 1;  // the quantiser's CTAs let this kernel start after the one before them ended
  }
  return m <= kDecodeTokens ? fp8_decode(p, st) : fp8_gemm(p, st);
}
