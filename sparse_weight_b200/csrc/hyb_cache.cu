// The 8-bit key / value cache: hyb_cache_append stores new tokens' keys and
// values in pages with one scale per page and head, hyb_cache_attention lets
// the new tokens' queries attend over them,
//
//   S[i][t] = softmax_scale * q_i . (ks[page(t)] kq_t)
//   O[i]    = sum_t softmax_t(S[i]) (vs[page(t)] vq_t)
//
// causal, with an optional window and sinks.
#include "hyb_internal.cuh"

#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace hyb {
namespace {

constexpr int kMinExp = -40, kMaxExp = 60;  // exponents of a scale that the append writes

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
  len = __ldg(s.lens + b);
  bool ok = len >= 0 && (int64_t)len <= ((int64_t)s.max_pages << s.page_shift);
  if (s.off) {
    const int64_t o0 = __ldg(s.off + b), o1 = __ldg(s.off + b + 1);
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

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------

struct AppendParams {
  SeqParams s;
  uint8_t *q[2];          // k, v
  float *scale[2];
  const uint16_t *x[2];   // new keys, new values
  int64_t ldx[2], hsx[2];
  int num_pages, kv_heads;
  int64_t sp, sh, st;     // strides of the cache, bytes
  uint32_t *status;
};

__device__ __forceinline__ uint32_t e4m3x2_rn(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t i8x2_rn(float lo, float hi) {
  const int a = __float2int_rn(fminf(fmaxf(lo, -127.0f), 127.0f));
  const int b = __float2int_rn(fminf(fmaxf(hi, -127.0f), 127.0f));
  return (uint32_t)(a & 0xFF) | ((uint32_t)(b & 0xFF) << 8);
}
template <bool I8>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (I8) return i8x2_rn(lo, hi);
  return e4m3x2_rn(lo, hi);
}
template <bool I8>
__device__ __forceinline__ float2 unpack2(uint32_t two) {
  if constexpr (I8) return make_float2((float)(int8_t)(two & 0xFF), (float)(int8_t)(two >> 8 & 0xFF));
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return __half22float2(*reinterpret_cast<__half2 *>(&h));
}

// One CTA per (page of a sequence that new tokens touch, head, K or V).  A
// thread holds 8 values of up to 8 tokens in registers between the pass that
// finds the largest one and the pass that stores them.
template <int D, bool I8>
__global__ void __launch_bounds__(128) cache_append_kernel(const AppendParams p) {
  constexpr int LANES = D / 8;         // threads per token
  constexpr int TPP = 128 / LANES;     // tokens per pass
  constexpr int PASSES = 64 / TPP;     // for the largest page
  __shared__ float s_a[4];
  const int b = blockIdx.z, h = blockIdx.y;
  const int which = blockIdx.x & 1, nth = blockIdx.x >> 1;
  int64_t row0;
  int fresh, len;
  if (!sequence(p.s, b, p.status, row0, fresh, len) || len == 0 || fresh == 0) return;
  const int start = len - fresh;
  const int P = 1 << p.s.page_shift;
  const int slot = (start >> p.s.page_shift) + nth;
  if (((int64_t)slot << p.s.page_shift) >= len) return;
  const int page = __ldg(p.s.table + b * p.s.table_stride + slot);
  if (page < 0 || page >= p.num_pages) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusBadSeq);
    return;
  }
  const int t0 = slot << p.s.page_shift;              // first token of the page
  const int lo = max(start - t0, 0), hi = min(len - t0, P);  // its new tokens
  const int c = threadIdx.x % LANES, tok0 = threadIdx.x / LANES;
  float *sc = p.scale[which] + (int64_t)page * p.kv_heads + h;
  const float had = lo > 0 ? *sc : 0.0f;
  uint8_t *q = p.q[which] + page * p.sp + h * p.sh + c * 8;
  const uint16_t *x = p.x[which] + h * p.hsx[which] + c * 8;

  uint4 raw[PASSES];
  float a = 0.0f;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < PASSES; ++j) {
    const int tok = j * TPP + tok0;
    raw[j] = make_uint4(0, 0, 0, 0);
    if (tok >= lo && tok < hi)
      raw[j] = ld_keep16(x + (row0 + (t0 + tok - start)) * p.ldx[which]);
  }
#pragma unroll
  for (int j = 0; j < PASSES; ++j) {
    const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v0 = fabsf(bf16_lo(w[i])), v1 = fabsf(bf16_hi(w[i]));
      const bool f0 = v0 <= 3.402823466e38f, f1 = v1 <= 3.402823466e38f;
      bad |= !f0 || !f1;
      a = fmaxf(a, fmaxf(f0 ? v0 : 0.0f, f1 ? v1 : 0.0f));
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
  if ((threadIdx.x & 31) == 0) s_a[threadIdx.x >> 5] = a;
  __syncthreads();
  a = fmaxf(fmaxf(s_a[0], s_a[1]), fmaxf(s_a[2], s_a[3]));
  // the smallest 2^e with QMAX 2^e >= a, from a's exponent and fraction:
  // 448 = 1.75 * 2^8, 127 = 1.984375 * 2^6
  const uint32_t bits = __float_as_uint(a);
  const uint32_t frac = bits & 0x7FFFFFu;
  int e = (int)(bits >> 23) - 127 - (I8 ? 6 : 8) + (frac > (I8 ? 0x7E0000u : 0x600000u) ? 1 : 0);
  e = min(max(e, kMinExp), kMaxExp);
  const float scale = fmaxf(__uint_as_float((uint32_t)(e + 127) << 23), had);

  // earlier tokens of the page, where the scale grew
  if (lo > 0 && scale != had) {
    const float ratio = __fdiv_rn(had, scale);
    for (int tok = tok0; tok < lo; tok += TPP) {
      uint2 *at = reinterpret_cast<uint2 *>(q + tok * p.st);
      const uint2 o = *at;
      uint32_t w[2] = {o.x, o.y};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 f0 = unpack2<I8>(w[i] & 0xFFFFu), f1 = unpack2<I8>(w[i] >> 16);
        w[i] = pack2<I8>(f0.x * ratio, f0.y * ratio) | pack2<I8>(f1.x * ratio, f1.y * ratio) << 16;
      }
      *at = make_uint2(w[0], w[1]);
    }
  }
#pragma unroll
  for (int j = 0; j < PASSES; ++j) {
    const int tok = j * TPP + tok0;
    if (tok < lo || tok >= hi) continue;
    const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
    uint32_t o[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v0 = bf16_lo(w[i]), v1 = bf16_hi(w[i]);
      v0 = v0 != v0 ? 0.0f : __fdiv_rn(v0, scale);  // a NaN is stored as zero
      v1 = v1 != v1 ? 0.0f : __fdiv_rn(v1, scale);
      const uint32_t two = pack2<I8>(v0, v1);
      if (i & 1)
        o[i >> 1] |= two << 16;
      else
        o[i >> 1] = two;
    }
    *reinterpret_cast<uint2 *>(q + tok * p.st) = make_uint2(o[0], o[1]);
  }
  if (threadIdx.x == 0) *sc = scale;  // every thread read the old one before the barrier
  if (bad) atomicOr(p.status, kStatusNaN);
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------

constexpr int kStep = 32;   // tokens per step of a warp
constexpr int kRows = 16;   // query rows (new token x head of the group) per unit
constexpr int kWarps = 4;   // warps of a CTA, each with its own steps
constexpr int kStages = 3;  // steps in flight per warp
// probabilities are held times 2^15 (exp2 of t - max + 15): fp16's 11 bits then
// reach down to 2^-29 of the largest one and its steps to 2^-39
constexpr float kLift = 15.0f;

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
  float *part;        // [unit][split]: O [16][D], mref [16], l [16]
  uint32_t *tickets;  // [unit]
  uint32_t *status;
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            int z, int w, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// D += A B, fp16 operands, fp32 accumulation
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// A unit is 16 query rows (new token x head of the group) of one sequence and
// one key / value head; its visible tokens are cut into steps of 32, the steps
// into `splits` CTAs and there over 4 warps.  Each warp runs its own ring of
// TMA boxes and its own running maximum and sum; the CTA's warps, then the
// unit's CTAs, are merged in a fixed order.
//
// Both products run as m16n8k16 on fp16 fragments built from the 8-bit bytes
// in registers.  A product's sum over k does not care which column sits in
// which register as long as both operands agree:
//   S = Q K^T: lane (g, t) takes 16-byte chunks of key g (chunks 2 t, 2 t + 1),
//     4 bytes per k-step; Q's fragments use the same columns.
//   O = P V:  lane (g, t) takes chunk g of values 2 t, 2 t + 1, 2 t + 8,
//     2 t + 9; byte j of each is column 16 g + j, product n-tile j.
template <int D, bool I8>
__global__ void __launch_bounds__(kWarps * 32)
    cache_attention_kernel(const AttnParams p, const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap vmap) {
  constexpr int KST = D / 16;              // k-steps of S
  constexpr int NT = D / 8;                // n-tiles of O
  constexpr int CH = D / 64;               // 16-byte chunks of a key per lane
  constexpr int kBox = kStep * D;          // bytes of a step's keys (or values)
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kWarps][kStages];
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ uint32_t s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int split = (int)(blockIdx.x % (unsigned)p.splits);
  const int unit = (int)(blockIdx.x / (unsigned)p.splits);
  const int qt = unit % p.qtiles;
  const int h = unit / p.qtiles % p.kv_heads;
  const int b = unit / p.qtiles / p.kv_heads;
  int64_t row0;
  int fresh, len;
  if (!sequence(p.s, b, p.status, row0, fresh, len)) return;
  const int G = p.group;
  const int64_t total = (int64_t)fresh * G;  // query rows of the sequence and head
  const int64_t r0 = (int64_t)qt * kRows;
  if (r0 >= total) return;
  const int nrows = (int)min((int64_t)kRows, total - r0);
  const int i0 = (int)(r0 / G), i1 = (int)((r0 + nrows - 1) / G);  // first, last new token

  // visible tokens: [0, sink) and [lo, hi); a query at place q sees t <= q
  const int first = len - fresh;
  const int hi = len == 0 ? 0 : first + i1 + 1;
  const int hi_min = first + i0 + 1;
  const int lo = p.window ? max(0, first + i0 - p.window + 1) : 0;
  const int lo_max = p.window ? first + i1 - p.window + 1 : 0;
  int na = p.window ? (min(p.sinks, hi) + kStep - 1) / kStep : 0;  // steps of the sinks
  int nb0 = lo / kStep;
  if (nb0 <= na) na = nb0 = 0;
  const int nsteps = hi == 0 ? 0 : na + (hi + kStep - 1) / kStep - nb0;
  const int active = max(1, (nsteps + p.chunk - 1) / p.chunk);  // CTAs with work
  if (split >= active) return;
  const int s_begin = split * p.chunk + warp, s_end = min(nsteps, (split + 1) * p.chunk);
  const int mine = s_begin < s_end ? (s_end - s_begin + kWarps - 1) / kWarps : 0;
  auto base_of = [&](int j) {  // first token of this warp's step j
    const int s = s_begin + j * kWarps;
    return (s < na ? s : s - na + nb0) * kStep;
  };

  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *ring = smem + warp * (kStages * 2 * kBox);
  const uint32_t ring32 = smem_u32(ring);
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&full[warp][s], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();

  // pages and scales, 16 steps at a time: lane l holds step l / 2's page of
  // tokens 16 (l & 1) .. (the same page twice where pages hold a step)
  const int32_t *table = p.s.table + b * p.s.table_stride;
  auto load_ids = [&](int w0) {
    const int j = w0 + (lane >> 1);
    int id = 0;
    if (j < mine) {
      const int tok = base_of(j) + 16 * (lane & 1);
      if (tok < hi) {
        id = __ldg(table + (tok >> p.s.page_shift));
        if (id < 0 || id >= p.num_pages) {
          atomicOr(p.status, kStatusBadSeq);
          id = 0;
        }
      }
    }
    return id;
  };
  auto load_scales = [&](int id, float &ks, float &vs) {
    ks = __ldg(p.k_scale + (int64_t)id * p.kv_heads + h);
    vs = __ldg(p.v_scale + (int64_t)id * p.kv_heads + h);
  };
  int id_cur = load_ids(0), id_nxt = load_ids(16);
  float ks_cur, vs_cur, ks_nxt, vs_nxt;
  load_scales(id_cur, ks_cur, vs_cur);
  load_scales(id_nxt, ks_nxt, vs_nxt);

  const int P = 1 << p.s.page_shift;
  const int boxes = P >= kStep ? 1 : 2;
  auto issue = [&](int j, int id0, int id1) {  // lane 0: step j's boxes into its slot
    const int s = j % kStages;
    const uint32_t dst = ring32 + s * (2 * kBox);
    const int tok = base_of(j);
    const int place = tok & (P - 1);
    mbar_arrive_expect_tx(&full[warp][s], 2 * kBox);
    tma_load_4d(dst, &kmap, 0, place, h, id0, &full[warp][s]);
    tma_load_4d(dst + kBox, &vmap, 0, place, h, id0, &full[warp][s]);
    if (boxes == 2) {
      tma_load_4d(dst + kBox / 2, &kmap, 0, 0, h, id1, &full[warp][s]);
      tma_load_4d(dst + kBox + kBox / 2, &vmap, 0, 0, h, id1, &full[warp][s]);
    }
  };
#pragma unroll
  for (int j = 0; j < kStages; ++j) {
    const int a = __shfl_sync(0xFFFFFFFFu, id_cur, 2 * j);
    const int c = __shfl_sync(0xFFFFFFFFu, id_cur, 2 * j + 1);
    if (j < mine && lane == 0) issue(j, a, c);
  }

  // Q: rows g and g + 8, each times a power of two that brings its largest
  // value to [128, 256), so that bf16's 8 bits survive the change to fp16
  uint32_t qf[KST][4];
  float qm[2];
  int bound_hi[2], bound_lo[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int rr = g + 8 * r;
    const bool live = rr < nrows;
    const int64_t row = r0 + (live ? rr : 0);
    const int i = (int)(row / G), hd = h * G + (int)(row % G);
    bound_hi[r] = live && len > 0 ? first + i + 1 : 0;
    bound_lo[r] = p.window ? first + i - p.window + 1 : 0;
    const uint16_t *src = p.Q + (row0 + i) * p.ldq + hd * p.hsq;
    uint32_t w[CH][8];
    uint32_t a = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const uint4 x = ld_keep16(src + (CH * t + c) * 16), y = ld_keep16(src + (CH * t + c) * 16 + 8);
      w[c][0] = x.x; w[c][1] = x.y; w[c][2] = x.z; w[c][3] = x.w;
      w[c][4] = y.x; w[c][5] = y.y; w[c][6] = y.z; w[c][7] = y.w;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        a = max(a, max((w[c][e] & 0x7FFFu) >> 7, (w[c][e] >> 23) & 0xFFu));
    }
    a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
    a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, 2));
    a = max(a, 8u);  // exponent field of the row's largest value
    const float f = __uint_as_float((261u - a) << 23);
    qm[r] = p.qmul * __uint_as_float((a - 7u) << 23);  // 2^(a - 134)
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const __half2 v = live ? __floats2half2_rn(bf16_lo(w[c][e]) * f, bf16_hi(w[c][e]) * f)
                               : __float2half2_rn(0.0f);
        qf[c * 4 + e / 2][2 * (e & 1) + r] = *reinterpret_cast<const uint32_t *>(&v);
      }
  }

  float o[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 4; ++c) o[n][c] = 0.0f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

  for (int j = 0; j < mine; ++j) {
    if ((j & 15) == 0 && j) {
      id_cur = id_nxt;
      ks_cur = ks_nxt;
      vs_cur = vs_nxt;
      id_nxt = load_ids(j + 16);
      load_scales(id_nxt, ks_nxt, vs_nxt);
    }
    const int src = 2 * (j & 15);
    const float ks0 = __shfl_sync(0xFFFFFFFFu, ks_cur, src);
    const float ks1 = __shfl_sync(0xFFFFFFFFu, ks_cur, src + 1);
    const float vs0 = __shfl_sync(0xFFFFFFFFu, vs_cur, src);
    const float vs1 = __shfl_sync(0xFFFFFFFFu, vs_cur, src + 1);
    const int slot = j % kStages;
    const uint32_t kb = ring32 + slot * (2 * kBox), vb = kb + kBox;
    const int base = base_of(j);
    if (!mbar_wait(&full[warp][slot], (uint32_t)(j / kStages) & 1u)) {
      if (lane == 0) atomicOr(p.status, kStatusTimeout);
      // the copies behind it may still land
      for (int q = j + 1; q < min(j + kStages, mine); ++q)
        mbar_wait(&full[warp][q % kStages], (uint32_t)(q / kStages) & 1u);
      break;
    }

    float s[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
#pragma unroll
      for (int c = 0; c < 4; ++c) s[n][c] = 0.0f;
      const int tok = n * 8 + g;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const uint4 w = lds16(kb + swz<D>(tok, CH * t + c));
        const uint32_t wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mma_f16(s[n], qf[c * 4 + e], to_f16x2<I8, 0>(wv[e]), to_f16x2<I8, 1>(wv[e]));
      }
    }

    // t = s + log2(vs): P then carries the page's value scale, and the running
    // maximum keeps it within fp16
    const float lv0 = __log2f(vs0), lv1 = __log2f(vs1);
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        s[n][c] = fmaf(s[n][c], (n < 2 ? ks0 : ks1) * qm[c >> 1], n < 2 ? lv0 : lv1);
    // a step that some row does not see whole
    const bool edge = base + kStep > hi_min || base < lo_max;
    if (edge) {
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int tok = base + n * 8 + 2 * t + (c & 1);
          const bool see = tok < bound_hi[c >> 1] && (tok >= bound_lo[c >> 1] || tok < p.sinks);
          if (!see) s[n][c] = -INFINITY;
        }
    }
    float corr[2], ref[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float v = m[r];
#pragma unroll
      for (int n = 0; n < 4; ++n) v = fmaxf(v, fmaxf(s[n][2 * r], s[n][2 * r + 1]));
      v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
      v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
      const float safe = v == -INFINITY ? 0.0f : v;
      corr[r] = ex2(m[r] - safe);
      ref[r] = safe - kLift;
      m[r] = v;
    }
    const float iv0 = __fdividef(1.0f, vs0), iv1 = __fdividef(1.0f, vs1);
    uint32_t pf[2][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float a = ex2(s[n][2 * r] - ref[r]), c = ex2(s[n][2 * r + 1] - ref[r]);
        if (n < 2)
          sum0 += a + c;
        else
          sum1 += a + c;
        const __half2 hp = __floats2half2_rn(a, c);
        pf[n >> 1][2 * (n & 1) + r] = *reinterpret_cast<const uint32_t *>(&hp);
      }
      l[r] = fmaf(l[r], corr[r], fmaf(sum0, iv0, sum1 * iv1));
    }
    if (__any_sync(0xFFFFFFFFu, corr[0] != 1.0f || corr[1] != 1.0f)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        o[n][0] *= corr[0];
        o[n][1] *= corr[0];
        o[n][2] *= corr[1];
        o[n][3] *= corr[1];
      }
    }

#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      uint32_t w[4][D / 32];  // values 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int tok = kk * 16 + 2 * t + (e & 1) + 8 * (e >> 1);
        if constexpr (D == 128) {
          const uint4 x = lds16(vb + swz<D>(tok, g));
          w[e][0] = x.x; w[e][1] = x.y; w[e][2] = x.z; w[e][3] = x.w;
        } else {
          const uint2 x = lds8(vb + swz<D>(tok, g >> 1) + 8 * (g & 1));
          w[e][0] = x.x; w[e][1] = x.y;
        }
        if (edge) {  // what lies in tokens that no row sees must not count
          const int at = base + tok;
          if (!(at < hi && (at >= lo || at < p.sinks))) {
#pragma unroll
            for (int q = 0; q < D / 32; ++q) w[e][q] = 0;
          }
        }
      }
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        const uint32_t a01 = __byte_perm(w[0][q], w[1][q], 0x5140);
        const uint32_t a23 = __byte_perm(w[0][q], w[1][q], 0x7362);
        const uint32_t c01 = __byte_perm(w[2][q], w[3][q], 0x5140);
        const uint32_t c23 = __byte_perm(w[2][q], w[3][q], 0x7362);
        mma_f16(o[4 * q + 0], pf[kk], to_f16x2<I8, 0>(a01), to_f16x2<I8, 0>(c01));
        mma_f16(o[4 * q + 1], pf[kk], to_f16x2<I8, 1>(a01), to_f16x2<I8, 1>(c01));
        mma_f16(o[4 * q + 2], pf[kk], to_f16x2<I8, 0>(a23), to_f16x2<I8, 0>(c23));
        mma_f16(o[4 * q + 3], pf[kk], to_f16x2<I8, 1>(a23), to_f16x2<I8, 1>(c23));
      }
    }

    // every lane has read the slot: its next step may overwrite it
    __syncwarp();
    const int jn = j + kStages;
    if (jn < mine) {
      const int sl = 2 * (jn & 15);
      const bool same = (jn >> 4) == (j >> 4);
      const int a0 = __shfl_sync(0xFFFFFFFFu, id_cur, sl), a1 = __shfl_sync(0xFFFFFFFFu, id_cur, sl + 1);
      const int c0 = __shfl_sync(0xFFFFFFFFu, id_nxt, sl), c1 = __shfl_sync(0xFFFFFFFFu, id_nxt, sl + 1);
      if (lane == 0) issue(jn, same ? a0 : c0, same ? a1 : c1);
    }
  }

#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
    l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
  }
  // the warp's rows into its ring's first slots (all its copies have landed)
  float *wo = reinterpret_cast<float *>(ring);  // [16][D]
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 4; ++c)
      wo[(g + 8 * (c >> 1)) * D + (D / 8) * (2 * t + (c & 1)) + n] = o[n][c];
  if (t == 0) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      s_m[warp][g + 8 * r] = m[r];
      s_l[warp][g + 8 * r] = l[r];
    }
  }
  __syncthreads();

  constexpr int kPart = kRows * D + 2 * kRows;  // floats of one CTA's partial result
  const bool alone = active == 1;
  float *mypart = alone ? nullptr : p.part + ((int64_t)unit * p.splits + split) * kPart;
  auto write_out = [&](int row, int d, float num, float den, float mx) {
    const int64_t rr = r0 + row;
    const int i = (int)(rr / G), hd = h * G + (int)(rr % G);
    p.O[(row0 + i) * p.ldo + hd * p.hso + d] = f32_to_bf16_rne(den != 0.0f ? num / den : 0.0f);
    if (d == 0 && p.lse)
      p.lse[(row0 + i) * p.ldl + hd] =
          den != 0.0f ? (mx - kLift + log2f(den)) * 0.693147180559945309f : -INFINITY;
  };
  for (int e = tid; e < nrows * D; e += kWarps * 32) {
    const int row = e / D, d = e % D;
    float mx = s_m[0][row];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][row]);
    const float safe = mx == -INFINITY ? 0.0f : mx;
    float num = 0.0f, den = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2(s_m[w][row] - safe);
      num = fmaf(f, reinterpret_cast<const float *>(smem + w * (kStages * 2 * kBox))[row * D + d], num);
      den = fmaf(f, s_l[w][row], den);
    }
    if (alone) {
      write_out(row, d, num, den, safe);
    } else {
      mypart[row * D + d] = num;
      if (d == 0) {
        mypart[kRows * D + row] = mx;
        mypart[kRows * D + kRows + row] = den;
      }
    }
  }
  if (alone) return;
  __threadfence();
  __syncthreads();
  if (tid == 0) {
    const uint32_t n = atomicAdd(p.tickets + unit, 1u);
    s_last = n == (uint32_t)active - 1u;
    if (s_last) p.tickets[unit] = 0;  // ready for the next call
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  const float *up = p.part + (int64_t)unit * p.splits * kPart;
  for (int e = tid; e < nrows * D; e += kWarps * 32) {
    const int row = e / D, d = e % D;
    float mx = -INFINITY;
    for (int s = 0; s < active; ++s) mx = fmaxf(mx, __ldcg(up + (int64_t)s * kPart + kRows * D + row));
    const float safe = mx == -INFINITY ? 0.0f : mx;
    float num = 0.0f, den = 0.0f;
    for (int s = 0; s < active; ++s) {
      const float *q = up + (int64_t)s * kPart;
      const float f = ex2(__ldcg(q + kRows * D + row) - safe);
      num = fmaf(f, __ldcg(q + row * D + d), num);
      den = fmaf(f, __ldcg(q + kRows * D + kRows + row), den);
    }
    write_out(row, d, num, den, safe);
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

int page_shift(int size) { return size == 16 ? 4 : size == 32 ? 5 : size == 64 ? 6 : 0; }

int cache_check(const hyb_cache *C) {
  if (!C || !C->k || !C->v || !C->k_scale || !C->v_scale) return HYB_ERR_INVALID_ARG;
  if (C->type != HYB_E4M3 && C->type != HYB_I8) return HYB_ERR_INVALID_ARG;
  if (C->num_pages < 1 || C->kv_heads < 1) return HYB_ERR_INVALID_ARG;
  if (!page_shift(C->page_size) || (C->head_dim != 64 && C->head_dim != 128))
    return HYB_ERR_UNSUPPORTED;
  if (C->stride_page < C->head_dim || C->stride_head < C->head_dim ||
      C->stride_token < C->head_dim)
    return HYB_ERR_INVALID_ARG;
  if (C->kv_heads > 65535 || C->stride_page >= (1ll << 40) || C->stride_head >= (1ll << 40) ||
      C->stride_token >= (1ll << 40))
    return HYB_ERR_UNSUPPORTED;
  if ((uintptr_t)C->k % 16 != 0 || (uintptr_t)C->v % 16 != 0 || C->stride_page % 16 != 0 ||
      C->stride_head % 16 != 0 || C->stride_token % 16 != 0 || (uintptr_t)C->k_scale % 4 != 0 ||
      (uintptr_t)C->v_scale % 4 != 0)
    return HYB_ERR_ALIGNMENT;
  return HYB_OK;
}

int seq_check(const hyb_cache *C, const hyb_sequences *S, SeqParams *p) {
  if (!S || !S->lens || !S->page_table || S->batch < 1 || S->max_new < 1 || S->max_pages < 1 ||
      S->rows < 0 || S->table_stride < S->max_pages)
    return HYB_ERR_INVALID_ARG;
  if (S->batch > 65535 || S->max_new > (1 << 24) || S->rows > INT32_MAX ||
      (int64_t)S->max_pages * C->page_size > INT32_MAX / 2)
    return HYB_ERR_UNSUPPORTED;
  if (!S->off && S->rows != (int64_t)S->batch * S->max_new) return HYB_ERR_INVALID_ARG;
  if ((uintptr_t)S->lens % 4 != 0 || (uintptr_t)S->off % 4 != 0 ||
      (uintptr_t)S->page_table % 4 != 0)
    return HYB_ERR_ALIGNMENT;
  p->batch = S->batch;
  p->max_new = S->max_new;
  p->rows = S->rows;
  p->lens = S->lens;
  p->off = S->off;
  p->table = S->page_table;
  p->max_pages = S->max_pages;
  p->table_stride = S->table_stride;
  p->page_shift = page_shift(C->page_size);
  return HYB_OK;
}

// The split of a unit's steps: enough CTAs to fill the GPU a few times over,
// none below 4 steps (one per warp) nor, unless the units alone fill it, above
// 32 (1024 tokens: sequences of different lengths then end at about the same
// time).  Only units that are split have tickets, which lie at a fixed place
// whatever the call's shape, so that calls of different shapes can share a
// workspace.
constexpr int kMinChunk = 4, kMaxChunk = 32;
constexpr int kTickets = 2048;
void split_plan(int64_t units, int64_t tokens, int sms, int *splits, int *chunk) {
  const int64_t steps = (tokens + kStep - 1) / kStep + 1;  // a range may start inside a step
  const bool many = units >= 8ll * sms || units > kTickets;
  const int64_t want = many ? 1 : (4ll * sms + units - 1) / units;
  int64_t c = (steps + want - 1) / want;
  if (c < kMinChunk) c = kMinChunk;
  if (c > kMaxChunk && !many) c = kMaxChunk;
  c = (c + kWarps - 1) / kWarps * kWarps;
  *chunk = (int)c;
  *splits = (int)((steps + c - 1) / c);
}

int attn_units(const hyb_cache *C, int32_t batch, int32_t max_new, int32_t heads, int64_t *units,
               int *qtiles) {
  if (batch < 1 || max_new < 1 || heads < 1 || heads % C->kv_heads != 0) return HYB_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)max_new * (heads / C->kv_heads);
  const int64_t qt = (rows + kRows - 1) / kRows;
  *units = (int64_t)batch * C->kv_heads * qt;
  if (batch > 65535 || max_new > (1 << 24) || *units > (1 << 30)) return HYB_ERR_UNSUPPORTED;
  *qtiles = (int)qt;
  return HYB_OK;
}

// workspace: header, tickets, partial results
constexpr size_t kPartOffset = kHeaderBytes + 4 * kTickets;
size_t attn_bytes(const hyb_cache *C, int64_t units, int splits) {
  return kPartOffset + (splits > 1 ? (size_t)units * splits * (kRows * C->head_dim + 2 * kRows) * 4 : 0);
}

int encode_pages(const hyb_cache *C, const uint8_t *base, CUtensorMap *map) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (!encode) return HYB_ERR_CUDA;
  const cuuint64_t dims[4] = {(cuuint64_t)C->head_dim, (cuuint64_t)C->page_size,
                              (cuuint64_t)C->kv_heads, (cuuint64_t)C->num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)C->stride_token, (cuuint64_t)C->stride_head,
                                 (cuuint64_t)C->stride_page};
  const cuuint32_t box[4] = {(cuuint32_t)C->head_dim,
                             (cuuint32_t)(C->page_size < kStep ? C->page_size : kStep), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult res = encode(
      map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t *>(base), dims, strides, box, estr,
      CU_TENSOR_MAP_INTERLEAVE_NONE,
      C->head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
      CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return res == CUDA_SUCCESS ? HYB_OK : HYB_ERR_CUDA;
}

template <int D, bool I8>
int launch_attention(const AttnParams &p, const CUtensorMap &km, const CUtensorMap &vm,
                     int64_t units, cudaStream_t st) {
  const size_t dyn = (size_t)kWarps * kStages * 2 * kStep * D + 1024;
  if (cudaFuncSetAttribute(cache_attention_kernel<D, I8>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, (int)dyn) != cudaSuccess)
    return HYB_ERR_CUDA;
  if (units * p.splits > INT32_MAX) return HYB_ERR_UNSUPPORTED;
  cache_attention_kernel<D, I8><<<(unsigned)(units * p.splits), kWarps * 32, dyn, st>>>(p, km, vm);
  return cudaGetLastError() == cudaSuccess ? HYB_OK : HYB_ERR_CUDA;
}

}  // namespace
}  // namespace hyb

using namespace hyb;

size_t hyb_cache_append_workspace_bytes(void) { return kHeaderBytes; }

int hyb_cache_append(const hyb_cache *C, const hyb_sequences *S, const uint16_t *K, int64_t ldk,
                     int64_t hsk, const uint16_t *V, int64_t ldv, int64_t hsv, void *ws,
                     size_t ws_bytes, hyb_stream_t stream) {
  int rc = cache_check(C);
  if (rc != HYB_OK) return rc;
  AppendParams p{};
  rc = seq_check(C, S, &p.s);
  if (rc != HYB_OK) return rc;
  if (!K || !V || ldk < C->head_dim || ldv < C->head_dim || hsk < C->head_dim ||
      hsv < C->head_dim)
    return HYB_ERR_INVALID_ARG;
  if ((uintptr_t)K % 16 != 0 || (uintptr_t)V % 16 != 0 || ldk % 8 != 0 || ldv % 8 != 0 ||
      hsk % 8 != 0 || hsv % 8 != 0)
    return HYB_ERR_ALIGNMENT;
  if (!ws || ws_bytes < kHeaderBytes) return HYB_ERR_WORKSPACE;
  if ((uintptr_t)ws % 256 != 0) return HYB_ERR_ALIGNMENT;
  p.q[0] = C->k;
  p.q[1] = C->v;
  p.scale[0] = C->k_scale;
  p.scale[1] = C->v_scale;
  p.x[0] = K;
  p.x[1] = V;
  p.ldx[0] = ldk;
  p.ldx[1] = ldv;
  p.hsx[0] = hsk;
  p.hsx[1] = hsv;
  p.num_pages = C->num_pages;
  p.kv_heads = C->kv_heads;
  p.sp = C->stride_page;
  p.sh = C->stride_head;
  p.st = C->stride_token;
  p.status = static_cast<uint32_t *>(ws);
  // pages that max_new tokens touch at most
  const int64_t touched = ((int64_t)S->max_new + C->page_size - 2) / C->page_size + 1;
  const dim3 grid((unsigned)(2 * touched), (unsigned)C->kv_heads, (unsigned)S->batch);
  cudaStream_t st = (cudaStream_t)stream;
  if (C->head_dim == 128) {
    if (C->type == HYB_I8)
      cache_append_kernel<128, true><<<grid, 128, 0, st>>>(p);
    else
      cache_append_kernel<128, false><<<grid, 128, 0, st>>>(p);
  } else {
    if (C->type == HYB_I8)
      cache_append_kernel<64, true><<<grid, 128, 0, st>>>(p);
    else
      cache_append_kernel<64, false><<<grid, 128, 0, st>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? HYB_OK : HYB_ERR_CUDA;
}

size_t hyb_cache_attention_workspace_bytes(const hyb_cache *C, int32_t batch, int32_t max_new,
                                           int32_t max_pages, int32_t heads) {
  if (cache_check(C) != HYB_OK || max_pages < 1) return 0;
  int64_t units;
  int qtiles, sms, splits, chunk;
  if (attn_units(C, batch, max_new, heads, &units, &qtiles) != HYB_OK) return 0;
  if (device_sm_count(&sms) != HYB_OK) return 0;
  split_plan(units, (int64_t)max_pages * C->page_size, sms, &splits, &chunk);
  return attn_bytes(C, units, splits);
}

int hyb_cache_attention(const hyb_cache *C, const hyb_sequences *S, const uint16_t *Q, int64_t ldq,
                        int64_t hsq, uint16_t *O, int64_t ldo, int64_t hso, float *lse,
                        int64_t ldl, int32_t heads, float softmax_scale, int32_t window,
                        int32_t sinks, void *ws, size_t ws_bytes, hyb_stream_t stream) {
  int rc = cache_check(C);
  if (rc != HYB_OK) return rc;
  AttnParams p{};
  rc = seq_check(C, S, &p.s);
  if (rc != HYB_OK) return rc;
  if (!Q || !O || heads < 1 || heads % C->kv_heads != 0 || window < 0 || sinks < 0 ||
      !(softmax_scale == softmax_scale))
    return HYB_ERR_INVALID_ARG;
  if (ldq < C->head_dim || hsq < C->head_dim || ldo < C->head_dim || hso < C->head_dim ||
      (lse && ldl < heads))
    return HYB_ERR_INVALID_ARG;
  if ((uintptr_t)Q % 16 != 0 || (uintptr_t)O % 16 != 0 || ldq % 8 != 0 || hsq % 8 != 0 ||
      ldo % 8 != 0 || hso % 8 != 0 || (uintptr_t)lse % 4 != 0)
    return HYB_ERR_ALIGNMENT;
  int64_t units;
  int qtiles, sms, splits, chunk;
  rc = attn_units(C, S->batch, S->max_new, heads, &units, &qtiles);
  if (rc != HYB_OK) return rc;
  const size_t need = hyb_cache_attention_workspace_bytes(C, S->batch, S->max_new, S->max_pages,
                                                          heads);
  if (!ws || need == 0 || ws_bytes < need) return HYB_ERR_WORKSPACE;
  if ((uintptr_t)ws % 256 != 0) return HYB_ERR_ALIGNMENT;
  rc = device_sm_count(&sms);
  if (rc != HYB_OK) return rc;
  // tokens that one unit sees at most
  const int64_t all = (int64_t)S->max_pages * C->page_size;
  int64_t tokens = all;
  if (window) {
    const int64_t span = (int64_t)window + kRows + (int64_t)sinks + 2 * kStep;
    if (span < tokens) tokens = span;
  }
  int full_splits, full_chunk;
  split_plan(units, all, sms, &full_splits, &full_chunk);
  split_plan(units, tokens, sms, &splits, &chunk);
  if (splits > full_splits) {  // never more than the workspace holds
    splits = full_splits;
    chunk = full_chunk;
  }
  p.Q = Q;
  p.ldq = ldq;
  p.hsq = hsq;
  p.O = O;
  p.ldo = ldo;
  p.hso = hso;
  p.lse = lse;
  p.ldl = ldl;
  p.k_scale = C->k_scale;
  p.v_scale = C->v_scale;
  p.num_pages = C->num_pages;
  p.kv_heads = C->kv_heads;
  p.group = heads / C->kv_heads;
  p.qmul = softmax_scale * 1.44269504088896341f;
  p.window = window;
  p.sinks = sinks;
  p.qtiles = qtiles;
  p.splits = splits;
  p.chunk = chunk;
  p.tickets = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(ws) + kHeaderBytes);
  p.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kPartOffset);
  p.status = static_cast<uint32_t *>(ws);
  alignas(64) CUtensorMap km{}, vm{};
  rc = encode_pages(C, C->k, &km);
  if (rc == HYB_OK) rc = encode_pages(C, C->v, &vm);
  if (rc != HYB_OK) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  if (C->head_dim == 128)
    return C->type == HYB_I8 ? launch_attention<128, true>(p, km, vm, units, st)
                             : launch_attention<128, false>(p, km, vm, units, st);
  return C->type == HYB_I8 ? launch_attention<64, true>(p, km, vm, units, st)
                           : launch_attention<64, false>(p, km, vm, units, st);
}
