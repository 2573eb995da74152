// hyb_cache.cuh -- what the kernels of the 8-bit key / value cache share.
#pragma once

#include "hyb_internal.cuh"

#include <cuda_fp16.h>

namespace hyb {

struct SeqParams {
  int batch, max_new;
  int64_t rows;
  const int32_t *lens, *off, *table;
  int max_pages;
  int64_t table_stride;
  int page_shift;  // log2 of the page size
};

// Sequence b: its first row, its new tokens and its length; false (flagged)
// where the caller's arrays contradict one another.
__device__ __forceinline__ bool sequence(const SeqParams &s, int b, uint32_t *status,
                                         int64_t &row0, int &fresh, int &len) {
  len = ld_dep(s.lens + b);
  bool ok = len >= 0 && (int64_t)len <= ((int64_t)s.max_pages << s.page_shift);
  if (s.off) {
    const int64_t o0 = ld_dep(s.off + b), o1 = ld_dep(s.off + b + 1);
    ok &= o0 >= 0 && o0 <= o1 && o1 <= s.rows && o1 - o0 <= s.max_new;
    row0 = o0;
    fresh = (int)(o1 - o0);
  } else {
    row0 = (int64_t)b * s.max_new;
    fresh = s.max_new;
  }
  ok &= len == 0 || len >= fresh;
  if (!ok) atomicOr(status, kStatusBadSeq);
  return ok;
}

struct AttnParams {
  SeqParams s;
  const uint16_t *Q;
  int64_t ldq, hsq;
  uint16_t *O;
  int64_t ldo, hso;
  float *lse;
  int64_t ldl;
  const float *k_scale, *v_scale;
  int num_pages, kv_heads, group;
  float qmul;  // softmax_scale * log2(e)
  int window, sinks;
  int qtiles;  // units per sequence and head
  int splits, chunk;  // CTAs per unit, steps of each
  float *part;        // [unit][split]: O [rows][D], reference [rows], sum [rows], rows of a unit
  uint32_t *tickets;  // [unit]
  uint32_t *status;
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// whether a unit that sees tokens [0, sinks) and [lo, hi), up to hi, sees one of
// tok .. tok + n - 1
__device__ __forceinline__ bool seen(int tok, int n, int lo, int hi, int sinks) {
  return tok < hi && (tok + n > lo || tok < sinks);
}

// A page's scales of head h.  The kernels work with the logarithm and the
// reciprocal of the value scale, so one below 2^-64 (a page of zeros may have 0)
// counts as 2^-64: its values are then below 2^-55.  Where no row sees the page
// (id -1) whatever its scales hold must not count.
__device__ __forceinline__ void page_scales(const AttnParams &p, int id, int h, float &ks,
                                            float &vs) {
  constexpr float kLeast = 1.0f / 18446744073709551616.0f;
  ks = 0.0f;
  vs = 1.0f;
  if (id >= 0) {
    ks = ld_dep(p.k_scale + (int64_t)id * p.kv_heads + h);
    vs = ld_dep(p.v_scale + (int64_t)id * p.kv_heads + h);
    if (vs >= 0.0f && vs < kLeast) vs = kLeast;
  }
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            int z, int w, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// (kernel parameters: open before the preceding kernel has ended)
__device__ __forceinline__ void prefetch_maps(const CUtensorMap &a, const CUtensorMap &b) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&a)) : "memory");
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&b)) : "memory");
}

// Whether this CTA is the last of its unit's `active` ones; the parts of all are
// then visible to its threads (read past L1).  One thread's fences between two
// barriers order the whole CTA's writes and reads.
__device__ __forceinline__ bool last_of_unit(const AttnParams &p, int unit, int active,
                                             uint32_t *s_last) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    const uint32_t n = atomicAdd(p.tickets + unit, 1u);
    *s_last = n == (uint32_t)active - 1u;
    if (*s_last) p.tickets[unit] = 0;  // ready for the next call
    __threadfence();
  }
  __syncthreads();
  return *s_last != 0;
}

// two 8-bit values (the low or high half of w) as a pair of fp16, exactly
template <bool I8, int HALF>
__device__ __forceinline__ uint32_t to_f16x2(uint32_t w) {
  uint32_t r;
  if constexpr (I8) {
    // 0x6400 | (q + 128) is 1024 + 128 + q in fp16
    const uint32_t u = __byte_perm(w ^ 0x80808080u, 0x64646464u, HALF ? 0x4342 : 0x4140);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&u), __float2half2_rn(1152.0f));
    r = *reinterpret_cast<const uint32_t *>(&x);
  } else {
    const uint16_t two = (uint16_t)(HALF ? w >> 16 : w);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(two));
  }
  return r;
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(a));
  return r;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
  return r;
}

// byte offset of 16-byte chunk c of row r in a box of D-byte rows, as the
// tensor map's swizzle (128 or 64 bytes) stores it
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  if constexpr (D == 128) return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
  return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// A unit's last CTA adds the parts of its `active` CTAs in their order: first all
// maxima and sums (kMergeRows of them at most, which bounds the splits) come to
// shared memory at once and become each part's weight, then the rows are summed
// with several loads on their way.  `lift`: what the stored maximum has to be
// lowered by to be P's reference.
constexpr int kMergeRows = 4096;
constexpr int kMergeBytes = 8 * kMergeRows;
template <int D, int ROWS, int THREADS>
__device__ __forceinline__ void merge_parts(const AttnParams &p, const float *up, int active,
                                            int urows, int64_t u0, int64_t row0, int h, float lift,
                                            float *sm) {
  constexpr int kPart = ROWS * D + 2 * ROWS;
  const int tid = threadIdx.x, G = p.group;
  float *sm_m = sm, *sm_l = sm + kMergeRows;  // [active][urows]
  for (int e = tid; e < active * urows; e += THREADS) {
    const int s = e / urows, row = e - s * urows;
    const float *q = up + (int64_t)s * kPart + ROWS * D + row;
    sm_m[e] = __ldcg(q);
    sm_l[e] = __ldcg(q + ROWS);
  }
  __syncthreads();
  for (int row = tid; row < urows; row += THREADS) {
    float mx = -INFINITY, den = 0.0f;
    for (int s = 0; s < active; ++s) mx = fmaxf(mx, sm_m[s * urows + row]);
    const float safe = mx == -INFINITY ? 0.0f : mx;
    for (int s = 0; s < active; ++s) {
      const float f = ex2(sm_m[s * urows + row] - safe);
      den = fmaf(f, sm_l[s * urows + row], den);
      sm_m[s * urows + row] = f;
    }
    const int64_t rr = u0 + row;
    if (p.lse)
      p.lse[(row0 + rr / G) * p.ldl + h * G + rr % G] =
          den != 0.0f ? (safe - lift + log2f(den)) * 0.693147180559945309f : -INFINITY;
    sm_l[row] = den != 0.0f ? 1.0f / den : 0.0f;  // (the row's own first sum is used up)
  }
  __syncthreads();
  for (int e = tid; e < urows * (D / 4); e += THREADS) {
    const int row = e / (D / 4), d = e % (D / 4) * 4;
    const float *q = up + row * D + d;
    float4 num = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s0 = 0; s0 < active; s0 += 8) {
      float4 x[8];
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (s0 + s < active) x[s] = __ldcg(reinterpret_cast<const float4 *>(q + (int64_t)(s0 + s) * kPart));
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        if (s0 + s >= active) break;
        const float f = sm_m[(s0 + s) * urows + row];
        num.x = fmaf(f, x[s].x, num.x);
        num.y = fmaf(f, x[s].y, num.y);
        num.z = fmaf(f, x[s].z, num.z);
        num.w = fmaf(f, x[s].w, num.w);
      }
    }
    const int64_t rr = u0 + row;
    const float r = sm_l[row];
    *reinterpret_cast<uint2 *>(p.O + (row0 + rr / G) * p.ldo + (h * G + rr % G) * p.hso + d) =
        make_uint2(f32_to_bf16_rne(num.x * r) | ((uint32_t)f32_to_bf16_rne(num.y * r) << 16),
                   f32_to_bf16_rne(num.z * r) | ((uint32_t)f32_to_bf16_rne(num.w * r) << 16));
  }
}

// Attention of units of 256 query rows on the tensor cores
// (hyb_cache_prefill.cu); p.chunk counts steps of 128 tokens there.
constexpr int kPrefillRows = 256, kPrefillStep = 128;
int cache_attention_prefill(const AttnParams &p, const CUtensorMap &km, const CUtensorMap &vm,
                            int64_t units, int dim, bool i8, cudaStream_t st);

}  // namespace hyb
