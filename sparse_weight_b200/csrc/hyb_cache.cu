// The 8-bit key / value cache: hyb_cache_append stores new tokens' keys and
// values in pages with one scale per page and head, hyb_cache_attention lets
// the new tokens' queries attend over them,
//
//   S[i][t] = softmax_scale * q_i . (ks[page(t)] kq_t)
//   O[i]    = sum_t softmax_t(S[i]) (vs[page(t)] vq_t)
//
// causal, with an optional window and sinks.
#include "hyb_cache.cuh"

namespace hyb {
namespace {

constexpr int kMinExp = -40, kMaxExp = 60;  // exponents of a scale that the append writes

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
// (adding 1.5 * 2^23 rounds to a whole number, nearest even, which then stands in
// the low bits; a conversion takes four times as long as an addition)
__device__ __forceinline__ uint32_t i8x2_rn(float lo, float hi) {
  const float a = __fadd_rn(fminf(fmaxf(lo, -127.0f), 127.0f), 12582912.0f);
  const float b = __fadd_rn(fminf(fmaxf(hi, -127.0f), 127.0f), 12582912.0f);
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7740) & 0xFFFFu;
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
// finds the largest one and the pass that stores them.  The loads of the new
// tokens do not wait for the page table; the largest value is found in the bits,
// two at a time; and where the scale is a power of two (always, unless the page
// brought another one) its reciprocal is exact and the divisions are products.
// 3 prompts of up to 2048 tokens (8 heads of 128, 8-bit integers): 5.8 us in a graph, 7.4
// with inputs that are not in L2 (floor 3.4); 64 x 1 token: 3.3 us, a chain of latencies.
template <int D, bool I8>
__global__ void __launch_bounds__(128) cache_append_kernel(const AppendParams p) {
  constexpr int LANES = D / 8;         // threads per token
  constexpr int TPP = 128 / LANES;     // tokens per pass
  constexpr int PASSES = 64 / TPP;     // for the largest page
  __shared__ float s_a[4];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.z, h = blockIdx.y;
  const int which = blockIdx.x & 1, nth = blockIdx.x >> 1;
  int64_t row0;
  int fresh, len;
  if (!sequence(p.s, b, p.status, row0, fresh, len) || len == 0 || fresh == 0) return;
  const int start = len - fresh;
  const int P = 1 << p.s.page_shift;
  const int slot = (start >> p.s.page_shift) + nth;
  if (((int64_t)slot << p.s.page_shift) >= len) return;
  const int t0 = slot << p.s.page_shift;              // first token of the page
  const int lo = max(start - t0, 0), hi = min(len - t0, P);  // its new tokens
  const int c = threadIdx.x % LANES, tok0 = threadIdx.x / LANES;
  const uint16_t *x = p.x[which] + h * p.hsx[which] + c * 8;
  uint4 raw[PASSES];
#pragma unroll
  for (int j = 0; j < PASSES; ++j) {
    const int tok = j * TPP + tok0;
    raw[j] = make_uint4(0, 0, 0, 0);
    if (tok >= lo && tok < hi)
      raw[j] = ld_dep16(x + (row0 + (t0 + tok - start)) * p.ldx[which]);
  }
  const int page = ld_dep(p.s.table + b * p.s.table_stride + slot);
  if (page < 0 || page >= p.num_pages) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusBadSeq);
    return;
  }
  float *sc = p.scale[which] + (int64_t)page * p.kv_heads + h;
  const float had = lo > 0 ? ld_dep(sc) : 0.0f;
  uint8_t *q = p.q[which] + page * p.sp + h * p.sh + c * 8;

  // magnitudes order as integers, an infinity or a NaN above every finite value
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < PASSES; ++j)
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(raw[j].x & 0x7FFF7FFFu, raw[j].y & 0x7FFF7FFFu),
                                 __vmaxu2(raw[j].z & 0x7FFF7FFFu, raw[j].w & 0x7FFF7FFFu)));
  float a = __uint_as_float(max(top << 16, top & 0xFFFF0000u));
  const bool bad = !(a <= 3.402823466e38f);
  if (bad) {  // only the finite values count
    a = 0.0f;
#pragma unroll
    for (int j = 0; j < PASSES; ++j) {
      const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v0 = fabsf(bf16_lo(w[i])), v1 = fabsf(bf16_hi(w[i]));
        a = fmaxf(a, fmaxf(v0 <= 3.402823466e38f ? v0 : 0.0f, v1 <= 3.402823466e38f ? v1 : 0.0f));
      }
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
      const uint2 o = __ldcg(at);
      uint32_t w[2] = {o.x, o.y};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 f0 = unpack2<I8>(w[i] & 0xFFFFu), f1 = unpack2<I8>(w[i] >> 16);
        w[i] = pack2<I8>(f0.x * ratio, f0.y * ratio) | pack2<I8>(f1.x * ratio, f1.y * ratio) << 16;
      }
      *at = make_uint2(w[0], w[1]);
    }
  }
  auto store = [&](auto &&scaled) {
#pragma unroll
    for (int j = 0; j < PASSES; ++j) {
      const int tok = j * TPP + tok0;
      if (tok < lo || tok >= hi) continue;
      const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = pack2<I8>(scaled(bf16_lo(w[i])), scaled(bf16_hi(w[i])));
      *reinterpret_cast<uint2 *>(q + tok * p.st) = make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
    }
  };
  // (2^e and 2^-e are both normal numbers between 2^-126 and 2^126)
  const uint32_t sb = __float_as_uint(scale), se = sb >> 23;
  if (!bad && (sb & 0x7FFFFFu) == 0 && se >= 1 && se <= 253) {
    const float inv = __uint_as_float((254u - se) << 23);
    store([&](float v) { return v * inv; });
  } else {
    store([&](float v) { return v != v ? 0.0f : __fdiv_rn(v, scale); });  // a NaN is stored as zero
  }
  if (threadIdx.x == 0) *sc = scale;  // every thread read the old one before the barrier
  if (bad) atomicOr(p.status, kStatusNaN);
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------

constexpr int kStep = 32;   // tokens per step
constexpr int kWarps = 4;   // warps that compute
// Probabilities are rounded to fp16 for the second product: the tensor cores take 16
// bits, V's 8-bit values are exact in fp16, and bf16 would keep 8 bits of P instead
// of 11.  (The sum of the softmax is of the fp32 ones.  The error against 64 bits is
// 0.0016 to 0.0017 of the output's size with it and without it: bf16's rounding of O.)
// They are held times 2^4 where the reference of the exponentials is the
// largest exponent, and times 2^15 at most: the reference moves only where it has
// been outgrown by more (a vote instead of a maximum over lanes in most steps).
// fp16's smallest step is then at most 2^-28 of the largest probability.
constexpr float kLift = 4.0f, kGrow = 11.0f;

// D += A B, fp16 operands, fp32 accumulation
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// transpose of an 8 x 8 matrix of fp16 held by the warp
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// What a CTA's shape is: NR tiles of 8 query rows (new token x head of the
// group) per warp.  Split tokens (SHARE false): the 4 warps take the unit's
// steps of 32 tokens in turn, each through a ring of its own, and are merged.
// Split rows (SHARE true): the warps have their own rows and share one ring,
// which a fifth warp fills.
template <int D, int NR, bool SHARE>
struct AttnShape {
  static constexpr int kRows = 8 * NR * (SHARE ? kWarps : 1);  // of a unit
  static constexpr int kBox = kStep * D;                       // a step's keys (or values), bytes
  static constexpr int kStages = SHARE ? 4 : 2;                // per ring
  static constexpr int kRing = kStages * 2 * kBox;
  static constexpr int kRings = SHARE ? 1 : kWarps;
  static constexpr int kThreads = 32 * (kWarps + (SHARE ? 1 : 0));
  static constexpr int kPitch = D + 4;                         // floats per row of a warp's result
  static constexpr int kOut = 8 * NR * kPitch * 4;             // bytes of it
  static constexpr int kWarpOut = SHARE ? kOut : kRing;        // from one warp's to the next's
  static constexpr int kUsed = kRing * kRings > kWarps * kWarpOut ? kRing * kRings : kWarps * kWarpOut;
  static constexpr int kBytes = kUsed > kMergeBytes ? kUsed : kMergeBytes;
  static constexpr int kPart = kRows * D + 2 * kRows;          // floats of a CTA's partial result
  static_assert(SHARE || kOut <= kRing, "a warp's result fits its ring");
};

// A unit is kRows query rows of one sequence and one key / value head; its
// visible tokens are cut into steps of 32 and the steps into `splits` CTAs,
// which are merged in a fixed order.
//
// Both products run as m16n8k16 on fp16 fragments built from the 8-bit bytes
// in registers, with the tokens (then the dimensions) as the 16 rows, so that a
// byte is converted once for all of a warp's query rows and 8 of them cost half
// of what 16 would.  A product's sum over k does not care which column sits in
// which register as long as both operands agree, nor does the order of rows:
//   S^T = K Q^T: lane (g, t) takes chunks 2 t, 2 t + 1 (16 bytes each) of keys g
//     and g + 8, 4 bytes per k-step; Q's fragments use the same columns.
//   O^T = V^T P^T: lane (g, t) takes chunk g of values 2 t, 2 t + 1, 2 t + 8,
//     2 t + 9; bytes 2 j and 2 j + 1 of each are rows g and g + 8 of tile j.
//     P^T's fragments are S^T's, transposed 8 x 8 by movmatrix.
//
// Bound by the latency of a warp's chain (a third of the issue slots are used, the
// tensor pipe a sixth): 32 sequences to 8192, 64 heads over 8: 44.7 us, 4.4 TB/s;
// 8 x 4 tokens in a window of 4096, 32 heads over 8: 25.4 us (2.8 times the floor).
// Split rows, 8 x 4 tokens over 8192, 64 heads over 8 (32 rows a unit): 150 us (0.9 TB/s),
// 100 us at 64 dimensions; a quarter of the issue slots are used.  At 128 dimensions 88 to
// 92 bytes are spilled: 10 warps on an SM put three on one scheduler (168 registers).
// Measured and not kept:
// 3 CTAs per SM for 16 rows (28 to 31 us for the latter), units' first parts before
// all second ones (48 us for the former).
template <int D, bool I8, int NR, bool SHARE>
__global__ void __launch_bounds__(AttnShape<D, NR, SHARE>::kThreads, NR == 1 ? 3 : 2)
    cache_attention_kernel(const AttnParams p, const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap vmap) {
  using Sh = AttnShape<D, NR, SHARE>;
  constexpr int KST = D / 16;      // k-steps of S^T
  constexpr int MT = D / 16;       // row tiles of O^T
  constexpr int CH = D / 64;       // 16-byte chunks of a key per lane
  constexpr int NS = Sh::kStages;
  constexpr int kBox = Sh::kBox;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[Sh::kRings][NS], empty[NS];
  __shared__ float s_m[kWarps][8 * NR], s_l[kWarps][8 * NR];
  __shared__ uint32_t s_last;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) prefetch_maps(kmap, vmap);
  asm volatile("griddepcontrol.wait;" ::: "memory");
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
  const int64_t u0 = (int64_t)qt * Sh::kRows;
  if (u0 >= total) return;
  const int urows = (int)min((int64_t)Sh::kRows, total - u0);
  const int first = len - fresh;

  // the unit's visible tokens: [0, sinks) and [lo, hi); a query at place q sees t <= q
  int na, nb0, nsteps, ulo, uhi;
  {
    const int i0 = (int)(u0 / G), i1 = (int)((u0 + urows - 1) / G);
    uhi = len == 0 ? 0 : first + i1 + 1;
    ulo = p.window ? max(0, first + i0 - p.window + 1) : 0;
    na = p.window ? (min(p.sinks, uhi) + kStep - 1) / kStep : 0;  // steps of the sinks
    nb0 = ulo / kStep;
    if (nb0 <= na) na = nb0 = 0;
    nsteps = uhi == 0 ? 0 : na + (uhi + kStep - 1) / kStep - nb0;
  }
  const int active = max(1, (nsteps + p.chunk - 1) / p.chunk);  // CTAs with work
  if (split >= active) return;
  const int stride = SHARE ? 1 : kWarps;
  const int s_begin = split * p.chunk + (SHARE ? 0 : warp);
  const int s_end = min(nsteps, (split + 1) * p.chunk);
  const int mine = s_begin < s_end ? (s_end - s_begin + stride - 1) / stride : 0;
  auto base_of = [&](int j) {  // first token of this warp's step j
    const int s = s_begin + j * stride;
    return (s < na ? s : s - na + nb0) * kStep;
  };

  // this warp's query rows and what they see
  const bool computes = !SHARE || warp < kWarps;
  const int64_t r0 = u0 + (SHARE ? 8 * NR * warp : 0);
  const int nrows = !computes ? 0 : (int)max((int64_t)0, min((int64_t)(8 * NR), total - r0));
  const int i0 = nrows ? (int)(r0 / G) : 0, i1 = nrows ? (int)((r0 + nrows - 1) / G) : 0;
  const int hi = len == 0 || !nrows ? 0 : first + i1 + 1;
  const int hi_min = first + i0 + 1;
  const int lo = p.window ? max(0, first + i0 - p.window + 1) : 0;
  const int lo_max = p.window ? first + i1 - p.window + 1 : 0;

  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int ring_no = SHARE ? 0 : warp;
  uint8_t *ring = smem + ring_no * Sh::kRing;
  const uint32_t ring32 = smem_u32(ring);
  if (SHARE ? tid == 0 : lane == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[ring_no][s], 1);
      if (SHARE) mbar_init(&empty[s], kWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (SHARE)
    __syncthreads();
  else
    __syncwarp();

  // pages, 16 steps at a time: lane l holds step l / 2's page of tokens
  // 16 (l & 1) .. (the same page twice where pages hold a step); -1 where no row
  // sees a token of that half (or step)
  const int P = 1 << p.s.page_shift;
  const int32_t *table = p.s.table + b * p.s.table_stride;
  auto load_ids = [&](int w0) {
    const int j = w0 + (lane >> 1);
    int id = -1;
    if (j < mine) {
      const int tok = base_of(j) + (P < kStep ? 16 * (lane & 1) : 0);
      if (seen(tok, min(P, kStep), ulo, uhi, p.sinks)) {
        id = ld_dep(table + (tok >> p.s.page_shift));
        if (id < 0 || id >= p.num_pages) {
          atomicOr(p.status, kStatusBadSeq);
          id = 0;
        }
      }
    }
    return id;
  };
  auto issue = [&](int j, int id0, int id1) {  // one lane: step j's boxes into its slot
    id0 = max(id0, 0);  // (what no row sees is masked, whatever lies there)
    id1 = max(id1, 0);
    const int s = j % NS;
    const uint32_t dst = ring32 + s * (2 * kBox);
    const int place = base_of(j) & (P - 1);
    uint64_t *bar = &full[ring_no][s];
    mbar_arrive_expect_tx(bar, 2 * kBox);
    tma_load_4d(dst, &kmap, 0, place, h, id0, bar);
    tma_load_4d(dst + kBox, &vmap, 0, place, h, id0, bar);
    if (P < kStep) {
      tma_load_4d(dst + kBox / 2, &kmap, 0, 0, h, id1, bar);
      tma_load_4d(dst + kBox + kBox / 2, &vmap, 0, 0, h, id1, bar);
    }
  };

  if (SHARE && warp == kWarps) {
    // the warp that fills the shared ring
    int ids = 0;
    bool ok = true;
    for (int j = 0; j < mine && ok; ++j) {
      if ((j & 15) == 0) ids = load_ids(j);
      const int id0 = __shfl_sync(0xFFFFFFFFu, ids, 2 * (j & 15));
      const int id1 = __shfl_sync(0xFFFFFFFFu, ids, 2 * (j & 15) + 1);
      if (j >= NS) ok = mbar_wait(&empty[j % NS], ((uint32_t)(j / NS) & 1u) ^ 1u);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (ok && lane == 0) issue(j, id0, id1);
    }
    if (!ok && lane == 0) atomicOr(p.status, kStatusTimeout);
  }

  float o[MT][NR][4];
  float m[NR][2], l[NR][2];  // of a row: the reference, and the sum of P / vs
  if (computes) {
    // (lane l also holds the scales of its page: K's, and V's logarithm and reciprocal)
    // (the first bytes set out as soon as their pages are known, what the steps
    // behind them need only after that)
    int id_cur = load_ids(0), id_nxt;
    float ks_cur, vs_cur, ks_nxt, vs_nxt, lv_cur, iv_cur;
    if constexpr (!SHARE) {
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        const int a = __shfl_sync(0xFFFFFFFFu, id_cur, 2 * j);
        const int c = __shfl_sync(0xFFFFFFFFu, id_cur, 2 * j + 1);
        if (j < mine && lane == 0) issue(j, a, c);
      }
    }
    page_scales(p, id_cur, h, ks_cur, vs_cur);

    // Q: row g of each tile, times a power of two that brings its largest value
    // to [128, 256), so that bf16's 8 bits survive the change to fp16
    uint32_t qf[NR][KST][2];
    float qm[NR][2];                      // of rows 2 t and 2 t + 1: softmax scale and that power
    int bound_hi[NR][2], bound_lo[NR][2];  // what those rows see
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const bool live = 8 * n + g < nrows;
      const int64_t row = live ? r0 + 8 * n + g : u0;
      const int i = (int)(row / G), hd = h * G + (int)(row % G);
      const uint16_t *src = p.Q + (row0 + i) * p.ldq + hd * p.hsq;
      uint32_t w[CH][8];
      uint32_t a = 0;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const uint4 x = ld_dep16(src + (CH * t + c) * 16), y = ld_dep16(src + (CH * t + c) * 16 + 8);
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
      const float back = p.qmul * __uint_as_float((a - 7u) << 23);  // 2^(a - 134)
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const __half2 v = live ? __floats2half2_rn(bf16_lo(w[c][e]) * f, bf16_hi(w[c][e]) * f)
                                 : __float2half2_rn(0.0f);
          qf[n][c * 4 + e / 2][e & 1] = *reinterpret_cast<const uint32_t *>(&v);
        }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        qm[n][c] = __shfl_sync(0xFFFFFFFFu, back, 4 * (2 * t + c));
        const int rr = 8 * n + 2 * t + c;
        const int ii = (int)((r0 + rr) / G);
        bound_hi[n][c] = rr < nrows && len > 0 ? first + ii + 1 : 0;
        bound_lo[n][c] = p.window ? first + ii - p.window + 1 : 0;
        m[n][c] = -INFINITY;
        l[n][c] = 0.0f;
      }
    }
#pragma unroll
    for (int k = 0; k < MT; ++k)
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[k][n][c] = 0.0f;

    lv_cur = __log2f(vs_cur);
    iv_cur = __fdividef(1.0f, vs_cur);
    id_nxt = load_ids(16);
    page_scales(p, id_nxt, h, ks_nxt, vs_nxt);

    for (int j = 0; j < mine; ++j) {
      if ((j & 15) == 0 && j) {
        id_cur = id_nxt;
        ks_cur = ks_nxt;
        lv_cur = __log2f(vs_nxt);
        iv_cur = __fdividef(1.0f, vs_nxt);
        id_nxt = load_ids(j + 16);
        page_scales(p, id_nxt, h, ks_nxt, vs_nxt);
      }
      const int src = 2 * (j & 15);
      float ks[2], lv[2], iv[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ks[i] = __shfl_sync(0xFFFFFFFFu, ks_cur, src + i);
        lv[i] = __shfl_sync(0xFFFFFFFFu, lv_cur, src + i);
        iv[i] = __shfl_sync(0xFFFFFFFFu, iv_cur, src + i);
      }
      const int slot = j % NS;
      const uint32_t kb = ring32 + slot * (2 * kBox), vb = kb + kBox;
      const int base = base_of(j);
      // (the vote makes the lanes one warp again for the collective instructions
      // below, and lets none go on where another's wait ran out)
      const bool here = mbar_wait(&full[ring_no][slot], (uint32_t)(j / NS) & 1u);
      if (!__all_sync(0xFFFFFFFFu, here)) {
        if (lane == 0) atomicOr(p.status, kStatusTimeout);
        // the copies behind it may still land
        for (int q = j + 1; q < min(j + NS, mine); ++q)
          mbar_wait(&full[ring_no][q % NS], (uint32_t)(q / NS) & 1u);
        break;
      }
      // (shared steps may lie outside what this warp's rows see)
      if (!SHARE || (base < hi && (base + kStep > lo || base < p.sinks))) {
        float s[2][NR][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[i][n][c] = 0.0f;
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            const uint4 x = lds16(kb + swz<D>(16 * i + g, CH * t + c));
            const uint4 y = lds16(kb + swz<D>(16 * i + 8 + g, CH * t + c));
            const uint32_t xv[4] = {x.x, x.y, x.z, x.w}, yv[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t a[4] = {to_f16x2<I8, 0>(xv[e]), to_f16x2<I8, 0>(yv[e]),
                                     to_f16x2<I8, 1>(xv[e]), to_f16x2<I8, 1>(yv[e])};
#pragma unroll
              for (int n = 0; n < NR; ++n)
                mma_f16(s[i][n], a, qf[n][c * 4 + e][0], qf[n][c * 4 + e][1]);
            }
          }
        }

        // t = s + log2(vs): P then carries the page's value scale, and the
        // reference keeps it within fp16
        const bool edge = base + kStep > hi_min || base < lo_max;  // some row does not see it whole
        uint32_t pf[2][NR][2];
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              s[i][n][e] = fmaf(s[i][n][e], ks[i] * qm[n][e & 1], lv[i]);
        if (edge) {  // (a branch of its own: few steps take it)
#pragma unroll
          for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) {  // tokens g and g + 8, rows 2 t and 2 t + 1
                const int tok = base + 16 * i + 8 * (e >> 1) + g, c = e & 1;
                if (!(tok < bound_hi[n][c] && (tok >= bound_lo[n][c] || tok < p.sinks)))
                  s[i][n][e] = -INFINITY;
              }
          asm volatile("" ::: "memory");
        }
        float top[NR][2];
        bool need = false;
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            top[n][c] = fmaxf(fmaxf(s[0][n][c], s[0][n][2 + c]), fmaxf(s[1][n][c], s[1][n][2 + c]));
            need |= top[n][c] > m[n][c] + kGrow;
          }
        if (__any_sync(0xFFFFFFFFu, need)) {
          // the largest exponents become the references; what is summed counts
          // against the old ones
          float corr[NR][2];
#pragma unroll
          for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float v = fmaxf(top[n][c], m[n][c]);
              v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
              v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
              v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
              corr[n][c] = ex2(m[n][c] - (v == -INFINITY ? 0.0f : v));
              m[n][c] = v;
              l[n][c] *= corr[n][c];
            }
#pragma unroll
          for (int k = 0; k < MT; ++k)
#pragma unroll
            for (int n = 0; n < NR; ++n) {
              o[k][n][0] *= corr[n][0];
              o[k][n][1] *= corr[n][1];
              o[k][n][2] *= corr[n][0];
              o[k][n][3] *= corr[n][1];
            }
          asm volatile("" ::: "memory");  // (a branch of its own: few steps take it)
        }
#pragma unroll
        for (int n = 0; n < NR; ++n) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float ref = (m[n][c] == -INFINITY ? 0.0f : m[n][c]) - kLift;
            float sum[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              s[i][n][c] = ex2(s[i][n][c] - ref);
              s[i][n][2 + c] = ex2(s[i][n][2 + c] - ref);
              sum[i] = s[i][n][c] + s[i][n][2 + c];
            }
            l[n][c] += fmaf(sum[0], iv[0], sum[1] * iv[1]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int d = 0; d < 2; ++d) {
              const __half2 hp = __floats2half2_rn(s[i][n][2 * d], s[i][n][2 * d + 1]);
              pf[i][n][d] = movmatrix(*reinterpret_cast<const uint32_t *>(&hp));
            }
        }

#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t w[4][D / 32];  // values 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tok = 16 * i + 2 * t + (e & 1) + 8 * (e >> 1);
            if constexpr (D == 128) {
              const uint4 x = lds16(vb + swz<D>(tok, g));
              w[e][0] = x.x; w[e][1] = x.y; w[e][2] = x.z; w[e][3] = x.w;
            } else {
              const uint2 x = lds8(vb + swz<D>(tok, g >> 1) + 8 * (g & 1));
              w[e][0] = x.x; w[e][1] = x.y;
            }
          }
          if (edge) {  // what lies in tokens that no row sees must not count
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int at = base + 16 * i + 2 * t + (e & 1) + 8 * (e >> 1);
              if (!(at < hi && (at >= lo || at < p.sinks))) {
#pragma unroll
                for (int q = 0; q < D / 32; ++q) w[e][q] = 0;
              }
            }
            __syncwarp();  // (the products below are the whole warp's)
          }
#pragma unroll
          for (int q = 0; q < D / 32; ++q)
#pragma unroll
            for (int z = 0; z < 2; ++z) {  // bytes 2 z, 2 z + 1 of word q: tile 2 q + z
              const uint32_t x = __byte_perm(w[0][q], w[1][q], z ? 0x7362 : 0x5140);
              const uint32_t y = __byte_perm(w[2][q], w[3][q], z ? 0x7362 : 0x5140);
              const uint32_t a[4] = {to_f16x2<I8, 0>(x), to_f16x2<I8, 1>(x), to_f16x2<I8, 0>(y),
                                     to_f16x2<I8, 1>(y)};
#pragma unroll
              for (int n = 0; n < NR; ++n) mma_f16(o[2 * q + z][n], a, pf[i][n][0], pf[i][n][1]);
            }
        }
      }

      // every lane has read the slot: its next step may overwrite it
      __syncwarp();
      if constexpr (SHARE) {
        if (lane == 0) mbar_arrive(&empty[slot]);
      } else {
        const int jn = j + NS;
        if (jn < mine) {
          const bool same = (jn >> 4) == (j >> 4);
          const int from = same ? id_cur : id_nxt;
          const int a = __shfl_sync(0xFFFFFFFFu, from, 2 * (jn & 15));
          const int c = __shfl_sync(0xFFFFFFFFu, from, 2 * (jn & 15) + 1);
          if (lane == 0) issue(jn, a, c);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int x = 4; x <= 16; x *= 2) l[n][c] += __shfl_xor_sync(0xFFFFFFFFu, l[n][c], x);
  }
  // a shared ring is free once every warp has left it; a warp's own is already
  if (SHARE) __syncthreads();
  if (computes) {
    float *wo = reinterpret_cast<float *>(smem + warp * Sh::kWarpOut);  // [8 NR][kPitch]
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        // dimensions (D / 8) g .. of row 2 t + c
        float *to = wo + (8 * n + 2 * t + c) * Sh::kPitch + (D / 8) * g;
#pragma unroll
        for (int k = 0; k < MT; k += 2)
          *reinterpret_cast<float4 *>(to + 2 * k) =
              make_float4(o[k][n][c], o[k][n][2 + c], o[k + 1][n][c], o[k + 1][n][2 + c]);
        if (g == 0) {
          s_m[warp][8 * n + 2 * t + c] = m[n][c];
          s_l[warp][8 * n + 2 * t + c] = l[n][c];
        }
      }
  }
  __syncthreads();

  const bool alone = active == 1;
  float *mypart = alone ? nullptr : p.part + ((int64_t)unit * p.splits + split) * Sh::kPart;
  // four dimensions of a row: the result, or this CTA's part of it
  auto write_out = [&](int row, int d, float4 num, float den, float mx) {
    const int64_t rr = u0 + row;
    const int i = (int)(rr / G), hd = h * G + (int)(rr % G);
    const float r = den != 0.0f ? 1.0f / den : 0.0f;
    *reinterpret_cast<uint2 *>(p.O + (row0 + i) * p.ldo + hd * p.hso + d) =
        make_uint2(f32_to_bf16_rne(num.x * r) | ((uint32_t)f32_to_bf16_rne(num.y * r) << 16),
                   f32_to_bf16_rne(num.z * r) | ((uint32_t)f32_to_bf16_rne(num.w * r) << 16));
    if (d == 0 && p.lse)
      p.lse[(row0 + i) * p.ldl + hd] =
          den != 0.0f ? (mx - kLift + log2f(den)) * 0.693147180559945309f : -INFINITY;
  };
  auto add = [](float4 &a, float f, const float4 &x) {
    a.x = fmaf(f, x.x, a.x);
    a.y = fmaf(f, x.y, a.y);
    a.z = fmaf(f, x.z, a.z);
    a.w = fmaf(f, x.w, a.w);
  };
  for (int e = tid; e < urows * (D / 4); e += Sh::kThreads) {
    const int row = e / (D / 4), d = e % (D / 4) * 4;
    float4 num = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float den = 0.0f, mx;
    if constexpr (SHARE) {
      const int w = row / (8 * NR), r = row % (8 * NR);
      mx = s_m[w][r];
      den = s_l[w][r];
      num = *reinterpret_cast<const float4 *>(smem + w * Sh::kWarpOut + (r * Sh::kPitch + d) * 4);
    } else {
      mx = s_m[0][row];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][row]);
      const float safe = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(s_m[w][row] - safe);
        add(num, f, *reinterpret_cast<const float4 *>(smem + w * Sh::kWarpOut + (row * Sh::kPitch + d) * 4));
        den = fmaf(f, s_l[w][row], den);
      }
    }
    if (alone) {
      write_out(row, d, num, den, mx);
    } else {
      *reinterpret_cast<float4 *>(mypart + row * D + d) = num;
      if (d == 0) {
        mypart[Sh::kRows * D + row] = mx;
        mypart[Sh::kRows * D + Sh::kRows + row] = den;
      }
    }
  }
  if (alone) return;
  if (!last_of_unit(p, unit, active, &s_last)) return;
  merge_parts<D, Sh::kRows, Sh::kThreads>(p, p.part + (int64_t)unit * p.splits * Sh::kPart, active,
                                          urows, u0, row0, h, kLift,
                                          reinterpret_cast<float *>(smem));
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

// The split of a unit's steps over CTAs: as many CTAs as fit the GPU at a time
// (3 per SM for units of 8 rows, 2 for 16 and 64, 1 for 256; a third more where
// all the work is small and the CTAs' start counts), none below 4 steps; units of 8
// or 16 rows and up to 12 steps are left whole.  Where
// units alone fill the GPU, and there for units of few rows only, a CTA has at
// most 40 steps (else 64), so that sequences of different lengths end at about
// the same time: 32 sequences of 1024 to 8192 tokens took 49.6 us with 48 steps
// and 46.9 us with 32, one of 65536 45 us with 32 and 36 us with 40.  (12, 40, and 3
// CTAs instead of 4 rest on those cases; sizes beside them were not measured.)
//
// The host has no lengths, so the steps are those of the table's width: 8192 tokens
// in a table of 131072 take 22 us instead of 19 (1 token, 32 heads over 8; 13 in one
// of 16384), 143 instead of 38 (4 tokens, 64 heads), 183 instead of 54 (64 tokens).
// `many` units stay whole whatever their lengths: 148 sequences of 1024, one of
// them of 65536, take 440 us, 147 take 191.
//
// Only units that are split have tickets, which lie at a fixed place whatever the
// call's shape, so that calls of different shapes can share a workspace.
constexpr int kMinChunk = 4, kUnsplit = 12;
constexpr int kShareRows = 64;  // most rows of mma.sync units
constexpr int kTickets = 2048;
constexpr int kLeastTop = 40;
int most_per_sm(int rows) { return rows == kPrefillRows ? 1 : rows > 8 ? 2 : 4; }
int step_of(int rows) { return rows == kPrefillRows ? kPrefillStep : kStep; }
void split_plan(int64_t units, int rows, int64_t tokens, int sms, int *splits, int *chunk) {
  const int step = step_of(rows);
  const int64_t steps = (tokens + step - 1) / step + 1;  // a range may start inside a step
  const int64_t fit = rows == 8 && units * steps >= 32ll * sms ? 3 : most_per_sm(rows);
  const int64_t fill = fit * sms;
  const bool many = units >= (rows <= 16 ? 8ll * sms : fill) || units > kTickets;
  // (a unit of 256 rows has its SM to itself: a CTA more than there are SMs would
  // wait for a whole one)
  const int64_t want = many ? 1 : (rows == kPrefillRows ? fill : fill + units - 1) / units;
  int64_t c = (steps + want - 1) / want;
  // (one short sequence of 300 tokens: 6.2 us in one part per unit, 7.8 in three)
  const int64_t least = rows <= 16 && steps <= kUnsplit ? kUnsplit : kMinChunk;
  if (c < least) c = least;
  const int64_t top = units >= sms ? kLeastTop : 64;
  if (c > top && !many && rows <= 16) c = top;
  const int64_t most = kMergeRows / rows;  // parts that the last CTA can add
  if ((steps + c - 1) / c > most) c = (steps + most - 1) / most;
  c = (c + kMinChunk - 1) / kMinChunk * kMinChunk;
  *chunk = (int)c;
  *splits = (int)((steps + c - 1) / c);
}

// Query rows (of one head and sequence) per unit: 8 or 16 in a CTA that splits
// the tokens over its warps, 64 in one whose warps have 16 each, 256 on the
// 5th-generation tensor cores.
int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }
int unit_rows(int64_t rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= kShareRows ? 64 : kPrefillRows; }

int attn_units(const hyb_cache *C, int32_t batch, int32_t max_new, int32_t heads, int64_t *units,
               int *qtiles) {
  if (batch < 1 || max_new < 1 || heads < 1 || heads % C->kv_heads != 0) return HYB_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)max_new * (heads / C->kv_heads);
  const int64_t qt = (rows + unit_rows(rows) - 1) / unit_rows(rows);
  *units = (int64_t)batch * C->kv_heads * qt;
  if (batch > 65535 || max_new > (1 << 24) || *units > (1 << 30)) return HYB_ERR_UNSUPPORTED;
  *qtiles = (int)qt;
  return HYB_OK;
}

// Workspace: header, tickets, partial results.  Enough for every call of at most
// these sizes, fewer tokens or units of fewer rows being split further: where
// units are split, units x splits is below 2 x `fill` (units < fill then, and
// splits <= fill / units + 1), or, for chunks of kLeastTop steps and more, at most
// that many splits of the units there can be.
constexpr size_t kPartOffset = kHeaderBytes + 4 * kTickets;
size_t attn_bytes(const hyb_cache *C, int32_t batch, int32_t max_new, int32_t max_pages,
                  int32_t heads, int sms) {
  const int64_t group = heads / C->kv_heads, all = max_new * group;
  const int64_t tokens = (int64_t)max_pages * C->page_size;
  int64_t floats = 0;
  for (int rows : {8, 16, kShareRows, kPrefillRows}) {
    if (rows < unit_rows(group) || rows > unit_rows(all)) continue;
    const int64_t qt = rows == kPrefillRows ? (all + rows - 1) / rows : 1;
    const int64_t units = (int64_t)batch * C->kv_heads * qt;
    const int64_t steps = (tokens + step_of(rows) - 1) / step_of(rows) + 1;
    auto splits = [&](int64_t c) { return min64((steps + c - 1) / c, kMergeRows / rows); };
    int64_t parts = 2ll * most_per_sm(rows) * sms;
    if (rows <= 16) {
      const int64_t top = min64(units, min64(8ll * sms, kTickets)) * splits(kLeastTop);
      if (top > parts) parts = top;
    }
    if (splits(kMinChunk) == 1) parts = 0;
    parts = min64(parts, units * splits(kMinChunk));
    const int64_t f = parts * (rows * C->head_dim + 2 * rows);
    if (f > floats) floats = f;
  }
  return kPartOffset + 4 * (size_t)floats;
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

template <int D, bool I8, int NR, bool SHARE>
int launch_shape(const AttnParams &p, const CUtensorMap &km, const CUtensorMap &vm, int64_t units,
                 cudaStream_t st) {
  using Sh = AttnShape<D, NR, SHARE>;
  const int dyn = Sh::kBytes + 1024;
  static std::atomic<uint64_t> done{0};
  if (allow_smem(reinterpret_cast<const void *>(cache_attention_kernel<D, I8, NR, SHARE>), dyn, done) != HYB_OK)
    return HYB_ERR_CUDA;
  if (units * p.splits > INT32_MAX) return HYB_ERR_UNSUPPORTED;
  return launch_dependent(cache_attention_kernel<D, I8, NR, SHARE>,
                          dim3((unsigned)(units * p.splits)), Sh::kThreads, dyn, 1, st, p, km, vm);
}

template <int D, bool I8>
int launch_attention(const AttnParams &p, const CUtensorMap &km, const CUtensorMap &vm,
                     int64_t units, int rows, cudaStream_t st) {
  return rows == 8    ? launch_shape<D, I8, 1, false>(p, km, vm, units, st)
         : rows == 16 ? launch_shape<D, I8, 2, false>(p, km, vm, units, st)
                      : launch_shape<D, I8, 2, true>(p, km, vm, units, st);
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
  const bool i8 = C->type == HYB_I8;
  return launch_dependent(C->head_dim == 128
                              ? (i8 ? cache_append_kernel<128, true> : cache_append_kernel<128, false>)
                              : (i8 ? cache_append_kernel<64, true> : cache_append_kernel<64, false>),
                          grid, 128, 0, 1, st, p);
}

size_t hyb_cache_attention_workspace_bytes(const hyb_cache *C, int32_t batch, int32_t max_new,
                                           int32_t max_pages, int32_t heads) {
  if (cache_check(C) != HYB_OK || max_pages < 1) return 0;
  int64_t units;
  int qtiles, sms;
  if (attn_units(C, batch, max_new, heads, &units, &qtiles) != HYB_OK) return 0;
  if (device_sm_count(&sms) != HYB_OK) return 0;
  return attn_bytes(C, batch, max_new, max_pages, heads, sms);
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
  if (!ws) return HYB_ERR_WORKSPACE;
  rc = device_sm_count(&sms);
  if (rc != HYB_OK) return rc;
  const int rows = unit_rows((int64_t)S->max_new * (heads / C->kv_heads));
  if (ws_bytes < attn_bytes(C, S->batch, S->max_new, S->max_pages, heads, sms))
    return HYB_ERR_WORKSPACE;
  if ((uintptr_t)ws % 256 != 0) return HYB_ERR_ALIGNMENT;
  // tokens that one unit sees at most
  int64_t tokens = (int64_t)S->max_pages * C->page_size;
  if (window) {
    const int64_t span = (int64_t)window + rows + (int64_t)sinks + 2 * step_of(rows);
    if (span < tokens) tokens = span;
  }
  split_plan(units, rows, tokens, sms, &splits, &chunk);
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
  if (rows == kPrefillRows)
    return cache_attention_prefill(p, km, vm, units, C->head_dim, C->type == HYB_I8, st);
  if (C->head_dim == 128)
    return C->type == HYB_I8 ? launch_attention<128, true>(p, km, vm, units, rows, st)
                             : launch_attention<128, false>(p, km, vm, units, rows, st);
  return C->type == HYB_I8 ? launch_attention<64, true>(p, km, vm, units, rows, st)
                           : launch_attention<64, false>(p, km, vm, units, rows, st);
}
