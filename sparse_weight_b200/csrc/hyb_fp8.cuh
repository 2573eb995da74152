// hyb_fp8.cuh -- what the kernels of the 8-bit floating-point product share.
#pragma once

#include "hyb_internal.cuh"

namespace hyb {

constexpr int kBlk = 128;  // columns (and rows of W) per scale

// One product: W [n][k] and X [m][k] e4m3 (X bf16 where the skinny kernel
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
  int bf16_out;
  uint32_t *status;
};

// The tensor-core product (hyb_fp8_gemm.cu) of e4m3 operands.  `after_quant`:
// X and its scales come from the kernel queued just before (programmatic
// dependent launch).
int fp8_gemm(const Fp8Params &p, bool after_quant, cudaStream_t st);

}  // namespace hyb
