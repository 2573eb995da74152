// hyb_fp8.cuh -- what the kernels of the 8-bit floating-point product share.
#pragma once

#include "hyb_internal.cuh"

namespace hyb {

constexpr int kBlk = 128;  // columns (and rows of W) per scale
// The most tokens of the decode kernel: its rows are one warp's lanes.
constexpr int kDecodeTokens = 32;
// The largest weight of the small kernel.
constexpr int64_t kSmallBytes = 8 << 20;
// The most columns: those that the kernels count past the last one, a warp's
// 8 blocks at most, stay within 31 bits.
constexpr int64_t kMaxCols = INT32_MAX - 16 * kBlk;
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

// One product: W [n][k] and X [m][k] e4m3 (X bf16 where the small kernel
// quantises it itself), their scales, and Y.
struct Fp8Params {
  int64_t n, k, m;
  const uint8_t *W;
  int64_t ldw;
  const float *sw;
  int64_t ldsw;
  const void *X;
  int64_t ldx;
  const float *sx;
  int64_t ldsx;
  void *Y;
  int64_t ldy;
  int bf16_out, x_bf16;
  int early_w;  // W may be read before the preceding kernel has ended
  uint32_t *status;
};

// All of these kernels are programmatic dependents of whatever precedes them on
// the stream: their CTAs start while it ends, and each waits
// (griddepcontrol.wait) for its completion before it touches memory, but for
// reads of W where early_w allows them.  Every CTA waits, so that a kernel's end
// also means the end of all before it.
//
// The tensor-core kernels allocate tensor memory before that wait: see
// hyb_tcgen05.cuh.

// The tensor-core product (hyb_fp8_gemm.cu) of e4m3 operands.
int fp8_gemm(const Fp8Params &p, cudaStream_t st);
// The same for m <= kDecodeTokens.
int fp8_decode(const Fp8Params &p, cudaStream_t st);
// The same for few tokens and a small weight (hyb_fp8_small.cu), of X in bf16
// or e4m3.
bool fp8_is_small(int64_t m, int64_t n, int64_t k);
int fp8_small(const Fp8Params &p, cudaStream_t st);

}  // namespace hyb
