// Attention over the 8-bit cache for many query rows (prompts, chunks of them),
// on the 5th-generation tensor cores:
//
//   S = Q K^T,  P = exp2(S scaled - max),  O = P V
//
// A CTA owns 256 query rows (new token x head of the group) of one sequence and
// key / value head, as two tiles of 128 (the MMA's M, one tensor-memory lane
// per row), and walks their visible tokens in steps of 128:
//
//   * warp 0 brings the pages' bytes with TMA, a step's keys and values in turn.
//   * warps 4-7 turn them into fp16, once for all 256 rows: MMA operands of
//     64-column halves in the 128-byte swizzle (K by rows of its contraction,
//     V by rows of tokens, read transposed), in a ring of four.
//   * warp 1 issues S = Q K^T and O += P V with P from tensor memory, for one
//     tile while the other one's softmax is computed.
//   * warps 8-11 and 12-15, a row per thread, read S half a step at a time (64
//     values, which stay in registers from S to P), mask it, take the maximum, and
//     write P as fp16 over S.  O stays in tensor memory; it is rescaled only where
//     a row's maximum has grown by more than 2^11 since the last time (P then
//     stays within fp16).
//
// 2 x 1024 tokens over 5120, window 2048, 32 heads over 8 of 128: 113 us (0.40 PFLOP/s);
// without a window 208 us, and 190 at 64 dimensions.  256 units on 148 SMs: two rounds,
// of which the second fills three quarters.
//
// Tensor memory: per tile 128 columns of S and D of O.  A step takes about 5200
// clocks: 2700 of a tile's softmax, then its two products and their way to the
// next one, which the other tile's softmax hides in part.  The MMAs alone would
// take 3100 (96 each, from shared and tensor memory alike), the exponentials 2048.
// Measured and not kept: P handed over by halves, so that its product starts
// earlier (118 us instead of 112 at 2 x 1024 tokens over 5120, window 2048: the
// waits of the MMA warp cost more); S by halves too (129 us: MMAs of N = 64 take as
// long as those of 128); maxima and exponentials in one pass, repeated where the
// reference moves (134 us, spills).
#include "hyb_cache.cuh"
#include "hyb_tcgen05.cuh"

namespace hyb {
namespace {

constexpr int kT = kPrefillStep;
constexpr int kH = kT / 2;  // tokens of a half step
constexpr int kThreads = 512;
constexpr int kRaw = 2;  // keys or values of a step on their way
constexpr int kOps = 4;  // and as fp16 operands
constexpr int kSc = 3;   // steps whose scales are held
// P is rounded to fp16 for the second product (11 bits; V's 8-bit values are exact in
// fp16, and with P in bf16, 8 bits, both operands would have to be bf16); the sum of
// the softmax is of the fp32 ones.  P is held times 2^4 at the reference, 2^15 at
// most: fp16's smallest step is then 2^-28 of the largest P
constexpr float kLift = 4.0f, kGrow = 11.0f;

constexpr int kTmem = 512;

template <int D>
struct PShape {
  static constexpr int kQ = 128 * D * 2;    // a row tile's Q
  static constexpr int kOp = kT * D * 2;    // a step's K (or V) in fp16
  static constexpr int kBytes8 = kT * D;    // and in 8 bits
  static constexpr int kQOff = 0, kOpOff = 2 * kQ, kRawOff = kOpOff + kOps * kOp;
  // (at 64 dimensions more than is used: the SM's tensor memory is this CTA's alone)
  static constexpr int kUsed = kRawOff + kRaw * kBytes8;
  static constexpr int kBytes = kUsed > kSmemPerSm / 3 * 2 ? kUsed : kSmemPerSm / 3 * 2 + 1024;
  static constexpr int kTile = kT + D;      // tensor-memory columns of a row tile
  static constexpr int kPart = kPrefillRows * D + 2 * kPrefillRows;
  static_assert(2 * kTile <= kTmem, "tensor memory");
  static_assert(tmem_fits(kTmem, kBytes), "tensor memory of the CTAs that fit an SM");
};

// The MMA warp runs as a whole and only its leader's instructions take effect:
// operands then stay in uniform registers (from a branch of one lane they were
// moved there one by one, which took longer than the products).
__device__ __forceinline__ void umma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b,
                                        uint32_t acc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %4, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(acc), "r"(idesc), "r"(leader)
      : "memory");
}
// A from tensor memory: lane = row, two fp16 of the contraction per column
__device__ __forceinline__ void umma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b,
                                        uint32_t acc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %4, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(acc), "r"(idesc), "r"(leader)
      : "memory");
}
// Operand whose contraction runs along rows (V: rows of tokens), 128-byte
// swizzle: 64 of the other index per row, the next 64 `half` bytes on (leading
// byte offset), 8 rows 1024 bytes apart (stride byte offset).
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t saddr, uint32_t half) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(half >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

#define HYB_R32(r)                                                                             \
  "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),         \
      "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), \
      "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),           \
      "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),           \
      "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])

// 32 columns of this thread's lane (tcgen05.wait::ld before the values are used)
__device__ __forceinline__ void tmem_get(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31}, [%32];"
      : HYB_R32(r)
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_get(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
template <int N>
__device__ __forceinline__ void tmem_got(uint32_t (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));  // not read before the wait
}
#undef HYB_R32

__device__ __forceinline__ void tmem_put(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// on pairs of fp32: (a, b) = (a, b) * f + o, and sum += (a, b)
__device__ __forceinline__ uint64_t pair(float v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ void fma2(uint32_t &a, uint32_t &b, uint64_t f, uint64_t o) {
  asm("{\n\t.reg .b64 t;\n\t"
      "mov.b64 t, {%0, %1};\n\t"
      "fma.rn.f32x2 t, t, %2, %3;\n\t"
      "mov.b64 {%0, %1}, t;\n\t}"
      : "+r"(a), "+r"(b)
      : "l"(f), "l"(o));
}
__device__ __forceinline__ void add2(uint64_t &sum, float a, float b) {
  asm("{\n\t.reg .b64 t;\n\t"
      "mov.b64 t, {%1, %2};\n\t"
      "add.rn.f32x2 %0, %0, t;\n\t}"
      : "+l"(sum)
      : "f"(a), "f"(b));
}

__device__ __forceinline__ void sts16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

template <int D, bool I8>
__global__ void __launch_bounds__(kThreads, 1)
    cache_attention_prefill_kernel(const AttnParams p, const __grid_constant__ CUtensorMap kmap,
                                   const __grid_constant__ CUtensorMap vmap) {
  using Sh = PShape<D>;
  // D fp32, A and B fp16 (format 0); S: N = 128 tokens; O: N = D, B transposed
  constexpr uint32_t kM = (uint32_t)(128 >> 4) << 24;
  constexpr uint32_t kIdS = (1u << 4) | ((uint32_t)(kT >> 3) << 17) | kM;
  constexpr uint32_t kIdO = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | kM;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t raw_full[kRaw], raw_empty[kRaw], op_full[kOps], op_empty[kOps],
      sc_full[kSc], q_full, s_full[2], p_full[2], pv_done[2], o_full[2];
  __shared__ float s_sc[kSc][3][kT / 16];  // scale of K, log2 of V's, its reciprocal, per 16 tokens
  __shared__ uint32_t s_tmem, s_last;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) prefetch_maps(kmap, vmap);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = (int)(blockIdx.x % (unsigned)p.splits);
  const int unit = (int)(blockIdx.x / (unsigned)p.splits);
  const int qt = unit % p.qtiles;
  const int h = unit / p.qtiles % p.kv_heads;
  const int b = unit / p.qtiles / p.kv_heads;
  int64_t row0;
  int fresh, len;
  if (!sequence(p.s, b, p.status, row0, fresh, len)) return;
  const int G = p.group;
  const int64_t total = (int64_t)fresh * G;
  const int64_t u0 = (int64_t)qt * kPrefillRows;
  if (u0 >= total) return;
  const int urows = (int)min((int64_t)kPrefillRows, total - u0);
  const int tiles = urows > 128 ? 2 : 1;
  const int first = len - fresh;

  // the unit's visible tokens: [0, sinks) and [lo, hi); a query at place q sees t <= q
  const int i0 = (int)(u0 / G), i1 = (int)((u0 + urows - 1) / G);
  const int hi = len == 0 ? 0 : first + i1 + 1;
  const int lo = p.window ? max(0, first + i0 - p.window + 1) : 0;
  int na = p.window ? (min(p.sinks, hi) + kT - 1) / kT : 0;  // steps of the sinks
  int nb0 = lo / kT;
  if (nb0 <= na) na = nb0 = 0;
  const int nsteps = hi == 0 ? 0 : na + (hi + kT - 1) / kT - nb0;
  const int active = max(1, (nsteps + p.chunk - 1) / p.chunk);  // CTAs with work
  if (split >= active) return;
  const int s_begin = split * p.chunk, n = min(nsteps, s_begin + p.chunk) - s_begin;
  auto base_of = [&](int j) {
    const int s = s_begin + j;
    return (s < na ? s : s - na + nb0) * kT;
  };

  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sm = smem_u32(smem);
  if (tid == 0) {
    for (int s = 0; s < kRaw; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], 4);
    }
    for (int s = 0; s < kOps; ++s) {
      mbar_init(&op_full[s], 4);
      mbar_init(&op_empty[s], 1);
    }
    for (int s = 0; s < kSc; ++s) mbar_init(&sc_full[s], 1);
    for (int r = 0; r < 2; ++r) {
      mbar_init(&p_full[r], 4);
      mbar_init(&pv_done[r], 1);
      mbar_init(&s_full[r], 1);
      mbar_init(&o_full[r], 1);
    }
    mbar_init(&q_full, 128 * tiles);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&s_tmem)),
                 "r"(kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int32_t *table = p.s.table + b * p.s.table_stride;
  // page of a token's box; -1 where no row sees a token of the box
  const int per = min(1 << p.s.page_shift, 32);  // tokens of a box
  auto page_of = [&](int tok) {
    int id = -1;
    if (seen(tok & ~(per - 1), per, lo, hi, p.sinks)) {
      id = ld_dep(table + (tok >> p.s.page_shift));
      if (id < 0 || id >= p.num_pages) {
        atomicOr(p.status, kStatusBadSeq);
        id = 0;
      }
    }
    return id;
  };

  bool ok = true;
  // of a softmax thread's row: the sum of P / vs, the reference (P = exp2(t - ref)),
  // and whether nothing of it lies in O yet
  float l = 0.0f, ref = 0.0f;
  bool fresh_row = true;
  if (warp == 0) {
    // lane i < 8: tokens 16 i .. of the step
    const int P = 1 << p.s.page_shift;
    const int mine = 16 * (lane & 7);
    int id = n > 0 ? page_of(base_of(0) + mine) : 0, next = 0;
    for (int h2 = 0; h2 < 2 * n; ++h2) {  // keys, then values of each step
      const int s = h2 % kRaw, j = h2 >> 1;
      if (!(h2 & 1) && j + 1 < n) next = page_of(base_of(j + 1) + mine);
      ok = h2 < kRaw || ring_wait(&raw_empty[s], ((uint32_t)(h2 / kRaw) & 1u) ^ 1u);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&raw_full[s], Sh::kBytes8);
      __syncwarp();
      if (lane < 8 && mine % per == 0)
        tma_load_4d(sm + Sh::kRawOff + s * Sh::kBytes8 + mine * D, h2 & 1 ? &vmap : &kmap, 0,
                    (base_of(j) + mine) & (P - 1), h, max(id, 0), &raw_full[s]);  // (-1: masked)
      if (h2 & 1) id = next;
    }
  } else if (warp == 1) {
    if (n > 0) {
      const uint32_t leader = lane == 0;
      auto wait = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xFFFFFFFFu, ring_wait(bar, parity)) != 0;
      };
      const uint64_t qd = sw128_desc(sm + Sh::kQOff), kd = sw128_desc(sm + Sh::kOpOff);
      const uint64_t vd = sw128_desc_mn(sm + Sh::kOpOff, kT * 128);
      auto slot = [&](int h2) { return (uint64_t)((h2 % kOps) * Sh::kOp >> 4); };
      auto ready = [&](int h2) { return wait(&op_full[h2 % kOps], (uint32_t)(h2 / kOps) & 1u); };
      auto scores = [&](int j, int r) {
        tc_fence_after();
        const uint64_t q = qd + (uint64_t)(r * Sh::kQ >> 4), k = kd + slot(2 * j);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_ss(leader, tmem + r * Sh::kTile, q + (((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4),
                  k + (((kk >> 2) * (kT * 128) + (kk & 3) * 32) >> 4), kk != 0, kIdS);
        umma_commit_if(leader, &s_full[r]);
        if (r == tiles - 1) umma_commit_if(leader, &op_empty[2 * j % kOps]);
      };
      ok = wait(&q_full, 0u) && ready(0);
      for (int r = 0; r < tiles && ok; ++r) scores(0, r);
      for (int j = 0; j < n && ok; ++j) {
        const uint32_t parity = (uint32_t)j & 1u;
        ok = ready(2 * j + 1);
        for (int r = 0; r < tiles && ok; ++r) {
          const uint64_t v = vd + slot(2 * j + 1);
          ok = wait(&p_full[r], parity);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kT / 16; ++kk)  // (P of the second half lies 64 columns on)
            umma_ts(leader, tmem + r * Sh::kTile + kT,
                    tmem + r * Sh::kTile + (kk >> 2) * kH + 8 * (kk & 3), v + (kk * 2048 >> 4),
                    (j | kk) != 0, kIdO);
          if (r == tiles - 1) umma_commit_if(leader, &op_empty[(2 * j + 1) % kOps]);
          if (j + 1 == n) {
            umma_commit_if(leader, &o_full[r]);
          } else {
            // S goes where P lies: its product has to be done
            umma_commit_if(leader, &pv_done[r]);
            ok = (r > 0 || ready(2 * j + 2)) && wait(&pv_done[r], parity);
            if (ok) scores(j + 1, r);
          }
        }
      }
    }
  } else if (warp >= 4 && warp < 8) {
    // bytes to fp16.  A thread takes 16-byte chunk c of token tok; tokens that no
    // row sees become zeros, whatever lies there.
    const int e = tid - 128;
    constexpr int kItems = kT * (D / 16) / 128, kAtOnce = 4;
    // scales of the step's groups of 16 tokens: lane i < 8 of warp 4, the pages
    // two steps and the scales one step ahead
    auto scales = [&](int id, float &ks, float &vs) { page_scales(p, id, h, ks, vs); };
    const bool sc = warp == 4 && lane < kT / 16;
    float ks = 0.0f, vs = 1.0f;
    int id = -1;
    if (sc && n > 0) {
      scales(page_of(base_of(0) + 16 * lane), ks, vs);
      if (n > 1) id = page_of(base_of(1) + 16 * lane);
    }
    for (int h2 = 0; h2 < 2 * n; ++h2) {
      const int s = h2 % kRaw, j = h2 >> 1, base = base_of(j);
      ok = ring_wait(&raw_full[s], (uint32_t)(h2 / kRaw) & 1u) &&
           (h2 < kOps || ring_wait(&op_empty[h2 % kOps], ((uint32_t)(h2 / kOps) & 1u) ^ 1u));
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      if (warp == 4 && !(h2 & 1)) {
        // (a slot's last step has been through its softmax: the step after it
        // has had its S, of the keys whose operand slot is free now)
        if (sc) {
          s_sc[j % kSc][0][lane] = ks;
          s_sc[j % kSc][1][lane] = __log2f(vs);
          s_sc[j % kSc][2][lane] = __fdividef(1.0f, vs);
          if (j + 1 < n) scales(id, ks, vs);
          if (j + 2 < n) id = page_of(base_of(j + 2) + 16 * lane);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_full[j % kSc]);
      }
      const bool whole = base + kT <= hi && (base >= lo || base + kT <= p.sinks);
      const uint32_t raw = sm + Sh::kRawOff + s * Sh::kBytes8;
      const uint32_t op = sm + Sh::kOpOff + (h2 % kOps) * Sh::kOp;
#pragma unroll
      for (int i0 = 0; i0 < kItems; i0 += kAtOnce) {
        uint4 x[kAtOnce];
        int tok[kAtOnce], ch[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          if (D == 128) {
            // 8 neighbours: 4 chunks of a token and the other 4 of the next one,
            // so that neither the reads nor the writes meet in a bank
            tok[i] = (e >> 2) + 32 * ((i0 + i) >> 1);
            ch[i] = (e & 3) + 4 * (((e >> 2) ^ i) & 1);
          } else {
            tok[i] = (e >> 2) + 32 * (i0 + i);
            ch[i] = e & 3;
          }
          x[i] = lds16(raw + swz<D>(tok[i], ch[i]));
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          if (!whole) {
            const int at = base + tok[i];
            if (!(at < hi && (at >= lo || at < p.sinks))) x[i] = make_uint4(0, 0, 0, 0);
          }
          // fp16 chunks 2 c, 2 c + 1 of the row: half c / 4
          const uint32_t row = op + (ch[i] >> 2) * (kT * 128) + tok[i] * 128;
          const int c = (2 * ch[i]) & 7, r7 = tok[i] & 7;
          sts16(row + ((c ^ r7) << 4), to_f16x2<I8, 0>(x[i].x), to_f16x2<I8, 1>(x[i].x),
                to_f16x2<I8, 0>(x[i].y), to_f16x2<I8, 1>(x[i].y));
          sts16(row + (((c + 1) ^ r7) << 4), to_f16x2<I8, 0>(x[i].z), to_f16x2<I8, 1>(x[i].z),
                to_f16x2<I8, 0>(x[i].w), to_f16x2<I8, 1>(x[i].w));
        }
      }
      // generic-proxy writes, read next by tcgen05.mma (async proxy)
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&op_full[h2 % kOps]);
        mbar_arrive(&raw_empty[s]);
      }
    }
  } else if (warp >= 8 && ((warp - 8) >> 2) < tiles) {
    // softmax: a row per thread
    const int r = (warp - 8) >> 2;
    const int trow = 32 * (warp & 3) + lane;       // row of the tile, tensor-memory lane
    const int row = 128 * r + trow;                // row of the unit
    const bool live = row < urows;
    const int64_t rr = u0 + (live ? row : 0);
    const int i = (int)(rr / G), hd = h * G + (int)(rr % G);
    const int bhi = live && len > 0 ? first + i + 1 : 0;
    const int blo = p.window ? first + i - p.window + 1 : 0;
    // Q's row times a power of two that brings its largest value to [128, 256)
    float qm;
    {
      const uint16_t *src = p.Q + (row0 + i) * p.ldq + hd * p.hsq;
      uint4 w[D / 8];
      uint32_t a = 0;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        w[c] = ld_dep16(src + 8 * c);
        const uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) a = max(a, max((x[e] & 0x7FFFu) >> 7, (x[e] >> 23) & 0xFFu));
      }
      a = max(a, 8u);
      const float f = __uint_as_float((261u - a) << 23);
      qm = p.qmul * __uint_as_float((a - 7u) << 23);  // 2^(a - 134)
      const uint32_t q = sm + Sh::kQOff + r * Sh::kQ + trow * 128;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __half2 v = live ? __floats2half2_rn(bf16_lo(x[e]) * f, bf16_hi(x[e]) * f)
                                 : __float2half2_rn(0.0f);
          y[e] = *reinterpret_cast<const uint32_t *>(&v);
        }
        sts16(q + (c >> 3) * (128 * 128) + (((c & 7) ^ (trow & 7)) << 4), y[0], y[1], y[2], y[3]);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(&q_full);
    }
    const uint32_t tl = tmem + r * Sh::kTile + ((uint32_t)(32 * (warp & 3)) << 16);
    // the warp's narrowest and widest bounds: outside them a step needs no mask
    const int whi = __reduce_min_sync(0xFFFFFFFFu, live ? bhi : INT32_MAX);
    const int wlo = __reduce_max_sync(0xFFFFFFFFu, live ? blo : 0);
    for (int i2 = 0; i2 < 2 * n; ++i2) {
      const int j = i2 >> 1, half = i2 & 1, base = base_of(j) + half * kH;
      if (!half) {
        ok = ring_wait(&s_full[r], (uint32_t)j & 1u) &&
             ring_wait(&sc_full[j % kSc], (uint32_t)(j / kSc) & 1u);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tc_fence_after();
      }
      const bool edge = base + kH > whi || base < wlo;  // some row of the warp does not see it whole
      const uint32_t th = tl + half * kH;
      uint32_t x[2][32];
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      tmem_get(th, x[0]);
      tmem_get(th + 32, x[1]);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (c == 0) {
          tmem_got(x[0]);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) asm volatile("" : "+r"(x[1][e]));
        }
        // exponents against the reference: s * scale + log2(vs) - ref
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const uint64_t f = pair(s_sc[j % kSc][0][4 * half + 2 * c + g] * qm);
          const uint64_t o = pair(s_sc[j % kSc][1][4 * half + 2 * c + g] - ref);
#pragma unroll
          for (int e = 16 * g; e < 16 * g + 16; e += 2) fma2(x[c][e], x[c][e + 1], f, o);
        }
        if (edge) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int at = base + 32 * c + e;
            if (!(at < bhi && (at >= blo || at < p.sinks))) x[c][e] = 0xFF800000u;  // -infinity
          }
        }
#pragma unroll
        for (int e = 0; e < 32; e += 8)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            m4[q] = fmaxf(fmaxf(m4[q], __uint_as_float(x[c][e + q])),
                          __uint_as_float(x[c][e + q + 4]));
      }
      const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
      const bool need = mx > (fresh_row ? -INFINITY : kLift + kGrow);
      if (__any_sync(0xFFFFFFFFu, need)) {
        // a new reference: what lies in O, l and the first half's P counts against
        // the old one (a whole number of binades, so that none of it is rounded)
        const float by = need ? floorf(mx - kLift) : 0.0f;
        ref += by;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            x[c][e] = __float_as_uint(__uint_as_float(x[c][e]) - by);
        if (__any_sync(0xFFFFFFFFu, need && !fresh_row)) {
          // (the product of the step before is done: it was waited for before S
          // was computed)
          const float corr = need && !fresh_row ? ex2(-by) : 1.0f;
          l *= corr;
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t y[16];
            tmem_get(tl + kT + 16 * c, y);
            tmem_got(y);
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * corr);
            tmem_put(tl + kT + 16 * c, y);
          }
          if (half) {
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              uint32_t y[16];
              tmem_get(tl + 16 * c, y);
              tmem_got(y);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&y[e]));
                const __half2 hp = __floats2half2_rn(f.x * corr, f.y * corr);
                y[e] = *reinterpret_cast<const uint32_t *>(&hp);
              }
              tmem_put(tl + 16 * c, y);
            }
          }
        }
        fresh_row = fresh_row && !need;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t pk[16];  // P, pairs of fp16
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint64_t s2[2] = {0, 0};  // pairs of sums
#pragma unroll
          for (int e = 16 * g; e < 16 * g + 16; e += 2) {
            const float a = ex2(__uint_as_float(x[c][e])), d = ex2(__uint_as_float(x[c][e + 1]));
            add2(s2[e >> 1 & 1], a, d);
            const __half2 hp = __floats2half2_rn(a, d);
            pk[e / 2] = *reinterpret_cast<const uint32_t *>(&hp);
          }
          l = fmaf((__uint_as_float((uint32_t)s2[0]) + __uint_as_float((uint32_t)s2[1])) +
                       (__uint_as_float((uint32_t)(s2[0] >> 32)) + __uint_as_float((uint32_t)(s2[1] >> 32))),
                   s_sc[j % kSc][2][4 * half + 2 * c + g], l);
        }
        tmem_put(th + 16 * c, pk);  // over columns of S that have been read
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      tc_fence_before();
      __syncwarp();
      if (half && lane == 0) mbar_arrive(&p_full[r]);
    }
    // O: the last step's product is done
    if (n > 0 && ok) {
      ok = ring_wait(&o_full[r], 0u);
      ok = __all_sync(0xFFFFFFFFu, ok);
    }
    tc_fence_after();
    const bool alone = active == 1;
    float *mypart = alone ? nullptr : p.part + ((int64_t)unit * p.splits + split) * Sh::kPart;
    const bool some = l != 0.0f;  // NaN counts
    const float inv = some ? 1.0f / l : 0.0f;
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t y[32];
      if (n > 0 && ok) {
        tmem_get(tl + kT + 32 * c, y);
        tmem_got(y);
      }
      if (live) {
        // a row without a visible token: its products may be of anything
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (!some) y[e] = 0;
        if (alone) {
          uint16_t *to = p.O + (row0 + i) * p.ldo + hd * p.hso + 32 * c;
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t o[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              o[q] = f32_to_bf16_rne(__uint_as_float(y[e + 2 * q]) * inv) |
                     ((uint32_t)f32_to_bf16_rne(__uint_as_float(y[e + 2 * q + 1]) * inv) << 16);
            *reinterpret_cast<uint4 *>(to + e) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4 *>(mypart + row * D + 32 * c + e) =
                make_uint4(y[e], y[e + 1], y[e + 2], y[e + 3]);
        }
      }
      __syncwarp();  // the next read of tensor memory is the whole warp's
    }
    if (live) {
      if (!alone) {
        mypart[kPrefillRows * D + row] = fresh_row ? -INFINITY : ref;
        mypart[kPrefillRows * D + kPrefillRows + row] = l;
      } else if (p.lse) {
        p.lse[(row0 + i) * p.ldl + hd] =
            some ? (ref + log2f(l)) * 0.693147180559945309f : -INFINITY;
      }
    }
  }
  if (!ok && lane == 0) atomicOr(p.status, kStatusTimeout);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmem)
                 : "memory");
  }
  if (active == 1) return;

  // the unit's last CTA adds the parts in order
  if (!last_of_unit(p, unit, active, &s_last)) return;
  merge_parts<D, kPrefillRows, kThreads>(p, p.part + (int64_t)unit * p.splits * Sh::kPart, active,
                                         urows, u0, row0, h, 0.0f, reinterpret_cast<float *>(smem));
}

template <int D, bool I8>
int launch(const AttnParams &p, const CUtensorMap &km, const CUtensorMap &vm, int64_t units,
           cudaStream_t st) {
  const int dyn = PShape<D>::kBytes + 1024;
  static std::atomic<uint64_t> done{0};
  if (allow_smem(reinterpret_cast<const void *>(cache_attention_prefill_kernel<D, I8>), dyn, done) != HYB_OK)
    return HYB_ERR_CUDA;
  if (units * p.splits > INT32_MAX) return HYB_ERR_UNSUPPORTED;
  return launch_dependent(cache_attention_prefill_kernel<D, I8>,
                          dim3((unsigned)(units * p.splits)), kThreads, dyn, 1, st, p, km, vm);
}

}  // namespace

int cache_attention_prefill(const AttnParams &p, const CUtensorMap &km, const CUtensorMap &vm,
                            int64_t units, int dim, bool i8, cudaStream_t st) {
  if (dim == 128)
    return i8 ? launch<128, true>(p, km, vm, units, st) : launch<128, false>(p, km, vm, units, st);
  return i8 ? launch<64, true>(p, km, vm, units, st) : launch<64, false>(p, km, vm, units, st);
}

}  // namespace hyb
