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

// 8 consecutive values of a row as they lie in memory (no value is looked at, so
// that several loads are on their way at once); those at or past `left` are
// zeros.  `vec`: the rows start on 16 bytes (else they are read one by one).
template <bool F32>
struct Raw {
  uint4 w[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ Raw<F32> load_raw(const void *X, int64_t off, int left, bool vec) {
  Raw<F32> r;
  r.w[0] = make_uint4(0, 0, 0, 0);
  if constexpr (F32) r.w[1] = make_uint4(0, 0, 0, 0);
  const float *xf = static_cast<const float *>(X) + off;
  const uint16_t *xb = static_cast<const uint16_t *>(X) + off;
  if (left >= 8 && vec) {
    if constexpr (F32) {
      r.w[0] = ld_dep16(xf);
      r.w[1] = ld_dep16(xf + 4);
    } else {
      r.w[0] = ld_dep16(xb);
    }
  } else if (left > 0) {
    uint32_t e[F32 ? 8 : 4] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) {
        if constexpr (F32)
          e[i] = __float_as_uint(ld_dep(xf + i));
        else
          e[i >> 1] |= (uint32_t) * static_cast<const volatile uint16_t *>(xb + i) << (16 * (i & 1));
      }
    r.w[0] = make_uint4(e[0], e[1], e[2], e[3]);
    if constexpr (F32) r.w[1] = make_uint4(e[4], e[5], e[6], e[7]);
  }
  return r;
}
template <bool F32>
__device__ __forceinline__ void unpack(const Raw<F32> &r, float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < (F32 ? 2 : 1); ++h) {
    const uint32_t w[4] = {r.w[h].x, r.w[h].y, r.w[h].z, r.w[h].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F32) {
        v[4 * h + i] = __uint_as_float(w[i]);
      } else {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
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

// The largest |x| of 8 values as its bits: magnitudes order as integers, an
// infinity or a NaN above every finite value.
template <bool F32>
__device__ __forceinline__ uint32_t top_bits(const Raw<F32> &r) {
  if constexpr (F32) {
    uint32_t a = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      a = max(max(max(a, r.w[h].x & 0x7FFFFFFFu), max(r.w[h].y & 0x7FFFFFFFu, r.w[h].z & 0x7FFFFFFFu)),
              r.w[h].w & 0x7FFFFFFFu);
    return a;
  } else {  // two values at a time, joined by top_of
    return __vmaxu2(__vmaxu2(r.w[0].x & 0x7FFF7FFFu, r.w[0].y & 0x7FFF7FFFu),
                    __vmaxu2(r.w[0].z & 0x7FFF7FFFu, r.w[0].w & 0x7FFF7FFFu));
  }
}
template <bool F32>
__device__ __forceinline__ uint32_t top_max(uint32_t a, uint32_t b) {
  return F32 ? max(a, b) : __vmaxu2(a, b);
}
template <bool F32>
__device__ __forceinline__ uint32_t top_of(uint32_t a) {
  return F32 ? a : max(a << 16, a & 0xFFFF0000u);
}
constexpr uint32_t kInfBits = 0x7F800000u;

// 8 values times inv as e4m3
template <bool F32>
__device__ __forceinline__ uint2 to_e4m3(const Raw<F32> &r, float inv) {
  float v[8];
  unpack(r, v);
  return make_uint2(e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}

// One scale per row and 128 columns.  A warp owns 2 kSeg blocks of a row, a half-
// warp every other one of them (16 lanes x 8 values: 16 bytes of bf16 per lane,
// 8 bytes written), with all of them on their way at once.  The instructions
// count here as much as the bytes: the largest values are compared as bits, two
// at a time, and a lane makes one of its half-warp's 2 kSeg divisions.  2048 x 14336
// in bf16: 17.0 us a call with changing inputs, 0.80 of the measured copy rate (15.4 us
// in a graph; 14.6 where the inputs are in L2).
template <bool F32, int kSeg>
__global__ void __launch_bounds__(256) fp8_quant_rows_kernel(int64_t rows, int64_t cols64,
                                                             const void *X, int64_t ldx,
                                                             uint8_t *Q, int64_t ldq,
                                                             float *scale, int64_t lds,
                                                             int segs, bool vec, uint32_t *status) {
  static_assert(kSeg <= 8, "two divisions per block over 16 lanes");
  // dependents start once the preceding kernel has ended: a product behind this
  // kernel may then read W at once
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int cols = (int)cols64;
  const int l16 = threadIdx.x & 15, half = (threadIdx.x >> 4) & 1;
  const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int row = (int)(unit / segs);
  if (row >= rows) return;
  const int blk0 = (int)(unit - (int64_t)row * segs) * (2 * kSeg) + half;
  const int col0 = blk0 * kBlk + l16 * 8;
  const int64_t x0 = row * ldx, q0 = row * ldq;
  Raw<F32> raw[kSeg];
#pragma unroll
  for (int j = 0; j < kSeg; ++j)
    raw[j] = load_raw<F32>(X, x0 + col0 + 2 * kBlk * j, cols - (col0 + 2 * kBlk * j), vec);
  float a[kSeg];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < kSeg; ++j) {
    uint32_t m = top_bits(raw[j]);
#pragma unroll
    for (int o = 8; o; o >>= 1) m = top_max<F32>(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    m = top_of<F32>(m);
    a[j] = __uint_as_float(m);
    if (__any_sync(0xFFFFFFFFu, m >= kInfBits)) {  // only the finite values count
      float v[8];
      unpack(raw[j], v);
      a[j] = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) amax_finite(v[i], a[j], bad);
#pragma unroll
      for (int o = 8; o; o >>= 1) a[j] = fmaxf(a[j], __shfl_xor_sync(0xFFFFFFFFu, a[j], o));
    }
    a[j] = fmaxf(a[j], kMinAmax);
  }
  // lane i < kSeg: 448 / a of block i; lane kSeg + i: a / 448 of it
  float mine = a[0];
#pragma unroll
  for (int j = 1; j < kSeg; ++j)
    if (l16 % kSeg == j) mine = a[j];
  const bool is_scale = (l16 / kSeg) & 1;
  const float quot = __fdiv_rn(is_scale ? mine : kE4m3Max, is_scale ? kE4m3Max : mine);
  if (l16 >= kSeg && l16 < 2 * kSeg) {
    const int blk = blk0 + 2 * (l16 - kSeg);
    if (blk * kBlk < cols) scale[row * lds + blk] = quot;
  }
#pragma unroll
  for (int j = 0; j < kSeg; ++j) {
    const float inv = __shfl_sync(0xFFFFFFFFu, quot, j, 16);
    const int col = col0 + 2 * kBlk * j;
    store8(Q, q0 + col, cols - col, to_e4m3(raw[j], inv));
  }
  if (bad) atomicOr(status, kStatusNaN);
}

// One scale per 128 x 128 block: one CTA per block, 64 values per thread kept
// in registers between the two passes.  1000 x 4100 in fp32: 6.3 us in a graph (4.3 where
// the inputs are in L2); 14336 x 4096: 28.6 us in bf16, 45 in fp32 (0.94 and 0.99 of the
// measured copy rate).
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
  Raw<F32> raw[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t row = row0 + 16 * j;
    raw[j] = load_raw<F32>(X, row * ldx + col, row < rows ? left : 0, vec);
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = top_max<F32>(m, top_bits(raw[j]));
#pragma unroll
  for (int o = 16; o; o >>= 1) m = top_max<F32>(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  float a = __uint_as_float(top_of<F32>(m));
  bool bad = false;
  if (!(a <= 3.402823466e38f)) {  // only the finite values count
    a = 0.0f;
    for (int j = 0; j < 8; ++j) {
      float v[8];
      unpack(raw[j], v);
      for (int i = 0; i < 8; ++i) amax_finite(v[i], a, bad);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
  }
  if ((threadIdx.x & 31) == 0) s_a[threadIdx.x >> 5] = a;
  __syncthreads();
  a = kMinAmax;
#pragma unroll
  for (int w = 0; w < 8; ++w) a = fmaxf(a, s_a[w]);
  const float inv = __fdiv_rn(kE4m3Max, a);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t row = row0 + 16 * j;
    if (row < rows) store8(Q, row * ldq + col, left, to_e4m3(raw[j], inv));
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
    // Where one block per half-warp fits the GPU at a time, that is the shortest
    // way (16 x 4096 in bf16: 1.6 us, 2.4 us with four); else four hide the loads
    // and share the divisions.
    const bool small = rows * cb <= 2 * 32 * 148;
    const int per = 2 * (small ? 1 : 4);  // blocks per warp
    const int64_t segs = (cb + per - 1) / per;
    const int64_t ctas = (rows * segs + 7) / 8;
    if (ctas > INT32_MAX) return HYB_ERR_UNSUPPORTED;
    return launch_dependent(
        xdt == HYB_F32 ? (small ? fp8_quant_rows_kernel<true, 1> : fp8_quant_rows_kernel<true, 4>)
                       : (small ? fp8_quant_rows_kernel<false, 1> : fp8_quant_rows_kernel<false, 4>),
        dim3((unsigned)ctas), 256, 0, 1, st, rows, cols, X, ldx, Q, ldq, scale, lds, (int)segs, vec,
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
  if (A->n > INT32_MAX || A->k > kMaxCols) return HYB_ERR_UNSUPPORTED;
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
  if (rows > INT32_MAX || cols > kMaxCols) return HYB_ERR_UNSUPPORTED;
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
  if (m < 1 || n < 1 || k < 1 || m > INT32_MAX || n > INT32_MAX || k > kMaxCols) return 0;
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
