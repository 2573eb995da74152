// The 8-bit floating-point product of up to 8 tokens with a small weight: what
// such a call takes is latency, not bytes, so this kernel keeps its chain short.
// One launch (a bf16 X is quantised here), no tensor memory, no tensor maps;
// every warp asks for all the bytes it will multiply at once and waits once.
//
//   * A warp owns 16 rows of W and up to U blocks of 128 columns; a CTA's 4
//     warps and a cluster's CTAs split k.  The sums meet in shared, then
//     distributed shared memory in a fixed order.
//   * m16n8k32 on e4m3, W as the 16 rows and the tokens as the 8 columns.  A
//     fragment register holds 4 bytes of k; the sum over a block does not care
//     which of its columns sit in which register as long as both operands
//     agree, so a lane takes 16 consecutive bytes of its row and feeds them to
//     two products: W goes straight from global memory to the fragments.
//
// 1 x 1024 x 4096: 6.6 us with X in bf16, 5.3 us in e4m3 (one launch each; 6.0 and 4.9
// where W is in L2).
#include "hyb_fp8.cuh"

#include <cooperative_groups.h>

namespace cg = cooperative_groups;

namespace hyb {
namespace {

constexpr int kWarps = 4, kRows = 16, kToks = 8;
constexpr int kMaxC = 8;  // CTAs of a cluster at most

// D += A B, one m16n8k32 e4m3 product with fp32 accumulation
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the bytes of a 16-byte word below `left`, zeros behind
__device__ __forceinline__ uint4 keep_bytes(uint4 v, int64_t left) {
  if (left >= 16) return v;
  uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = (int)left - 4 * i;
    w[i] = b >= 4 ? w[i] : (b <= 0 ? 0u : w[i] & ((1u << (8 * b)) - 1u));
  }
  return v;
}

template <int U, bool XBF16>
__global__ void __launch_bounds__(32 * kWarps) fp8_small_kernel(const Fp8Params p) {
  constexpr int XW = XBF16 ? 4 : 2;  // 16-byte words of X per lane and block
  __shared__ float part[kWarps][kToks][kRows + 1];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t row0 = (int64_t)(blockIdx.x / C) * kRows;
  const int kb = (int)((p.k + kBlk - 1) / kBlk);
  const int b0 = (rank * kWarps + warp) * U;  // this warp's blocks: b0 .. b0 + U - 1
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!p.early_w) asm volatile("griddepcontrol.wait;" ::: "memory");

  // block u of this warp, 16 columns at t * 16 + 64 q of it
  auto col = [&](int u, int q) { return (int64_t)(b0 + u) * kBlk + t * 16 + 64 * q; };
  uint4 w[U][2][2];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int64_t row = row0 + 8 * h + g;
        w[u][h][q] = make_uint4(0, 0, 0, 0);
        if (row < p.n && col(u, q) < p.k)
          w[u][h][q] = ld_dep_stream16(p.W + row * p.ldw + col(u, q));
      }
  float sw[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    sw[u] = b0 + u < kb ? ld_dep(p.sw + row0 / kBlk * p.ldsw + b0 + u) : 0.0f;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const bool live = g < p.m;
  uint4 x[U][XW];
  float sx[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int q = 0; q < XW; ++q) {
      const int64_t c = XBF16 ? col(u, q >> 1) + 8 * (q & 1) : col(u, q);
      x[u][q] = make_uint4(0, 0, 0, 0);
      if (live && c < p.k)
        x[u][q] = XBF16 ? ld_dep16(static_cast<const uint16_t *>(p.X) + g * p.ldx + c)
                        : ld_dep16(static_cast<const uint8_t *>(p.X) + g * p.ldx + c);
    }
    sx[u] = 0.0f;
    if (!XBF16 && live && b0 + u < kb) sx[u] = ld_dep(p.sx + g * p.ldsx + b0 + u);
  }

  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  bool bad = false;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (b0 + u >= kb) break;
    uint4 xq[2];
    if constexpr (XBF16) {
      float v[2][16], a = 0.0f;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int64_t left = p.k - col(u, q);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 r = x[u][2 * q + (i >> 2)];
          const uint32_t two = (i & 3) == 0 ? r.x : (i & 3) == 1 ? r.y : (i & 3) == 2 ? r.z : r.w;
          v[q][2 * i] = 2 * i < left ? bf16_lo(two) : 0.0f;
          v[q][2 * i + 1] = 2 * i + 1 < left ? bf16_hi(two) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) amax_finite(v[q][i], a, bad);
      }
      a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
      a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 2));
      a = fmaxf(a, kMinAmax);
      const float inv = __fdiv_rn(kE4m3Max, a);
      sx[u] = __fdiv_rn(a, kE4m3Max);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          b[i] = e4m3x4(v[q][4 * i] * inv, v[q][4 * i + 1] * inv, v[q][4 * i + 2] * inv,
                        v[q][4 * i + 3] * inv);
        xq[q] = make_uint4(b[0], b[1], b[2], b[3]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 2; ++q) xq[q] = keep_bytes(x[u][q], p.k - col(u, q));
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < 2; ++q) w[u][h][q] = keep_bytes(w[u][h][q], p.k - col(u, q));
    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      mma_e4m3(d, w[u][0][q].x, w[u][1][q].x, w[u][0][q].y, w[u][1][q].y, xq[q].x, xq[q].y);
      mma_e4m3(d, w[u][0][q].z, w[u][1][q].z, w[u][0][q].w, w[u][1][q].w, xq[q].z, xq[q].w);
    }
    // the scales of this lane's result columns, tokens 2 t and 2 t + 1
    const float s0 = __shfl_sync(0xFFFFFFFFu, sx[u], 8 * t) * sw[u];
    const float s1 = __shfl_sync(0xFFFFFFFFu, sx[u], 8 * t + 4) * sw[u];
    acc[0] = fmaf(d[0], s0, acc[0]);
    acc[1] = fmaf(d[1], s1, acc[1]);
    acc[2] = fmaf(d[2], s0, acc[2]);
    acc[3] = fmaf(d[3], s1, acc[3]);
  }
  if (XBF16 && bad) atomicOr(p.status, kStatusNaN);
#pragma unroll
  for (int c = 0; c < 4; ++c) part[warp][2 * t + (c & 1)][8 * (c >> 1) + g] = acc[c];
  __syncthreads();
  if (C > 1) cluster.sync();
  // 128 sums at most, a stretch of them per CTA, one per thread; all parts on
  // their way at once, then added in order
  const int sums = kRows * (int)p.m, share = (sums + C - 1) / C;
  const int e = rank * share + (int)threadIdx.x;
  if ((int)threadIdx.x < share && e < sums) {
    const int row = e % kRows, tok = e / kRows;
    float a[kMaxC][kWarps];
#pragma unroll
    for (int j = 0; j < kMaxC; ++j)
      if (j < C)
#pragma unroll
        for (int q = 0; q < kWarps; ++q)
          a[j][q] = C == 1 ? part[q][tok][row] : *cluster.map_shared_rank(&part[q][tok][row], j);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < kMaxC; ++j)
      if (j < C)
#pragma unroll
        for (int q = 0; q < kWarps; ++q) s += a[j][q];
    if (row0 + row < p.n) {
      const int64_t at = tok * p.ldy + row0 + row;
      if (p.bf16_out)
        static_cast<uint16_t *>(p.Y)[at] = f32_to_bf16_rne(s);
      else
        static_cast<float *>(p.Y)[at] = s;
    }
  }
  if (C > 1) cluster.sync();  // no CTA leaves while another reads its shared memory
}

template <int U, bool XBF16>
int launch_small(const Fp8Params &p, int C, cudaStream_t st) {
  return launch_dependent(fp8_small_kernel<U, XBF16>,
                          dim3((unsigned)((p.n + kRows - 1) / kRows * C)), 32 * kWarps, 0, C, st, p);
}

}  // namespace

bool fp8_is_small(int64_t m, int64_t n, int64_t k) {
  return m <= kToks && k <= kMaxC * kWarps * 4 * kBlk && n * k <= kSmallBytes;
}

int fp8_small(const Fp8Params &p, cudaStream_t st) {
  const int64_t kb = (p.k + kBlk - 1) / kBlk;
  // two blocks per warp where a cluster of 8 covers k with them, else four
  const int u = kb <= kMaxC * kWarps * 2 ? 2 : 4;
  const int C = (int)((kb + u * kWarps - 1) / (u * kWarps));
  if (u == 2)
    return p.x_bf16 ? launch_small<2, true>(p, C, st)
                    : launch_small<2, false>(p, C, st);
  return p.x_bf16 ? launch_small<4, true>(p, C, st)
                  : launch_small<4, false>(p, C, st);
}

}  // namespace hyb
