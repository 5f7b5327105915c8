// Attention forward with shaped scores on the sm_100a tensor cores: bf16 in, fp32
// accumulate; at D = 128 two 128-row query tiles per CTA, at D = 64 one, with two CTAs a
// SM, so that one's start and end overlap the other's tiles.
//
//     x_ij = c2 q_i.k_j  or  A tanh(scale q_i.k_j / cap)      (base-2 units)
//     z_ij = x_ij - slope2 |i - j|,  hidden keys left out,
// and over key tiles the online softmax: a reference m >= about the row's
// maximum, l = sum 2^(z - m), O = sum 2^(z - m) V, O / l at the end, LSE =
// (m + log2 l) ln 2. The reference moves only when a tile's maximum exceeds it
// by more than 2^8.
//
// Which tiles. A query's visible keys are one range [lo, hi). The CTA reduces
// its rows' ranges to one key-tile range per query tile and walks the union;
// inside, a warp whose 32 rows see all 128 keys of a tile runs without masks,
// one that sees none writes zeros.
//
// Roles: eight softmax warps a query tile, two threads a row (half of a tile's 128 keys,
// TMEM lane quarter), then a TMA warp and an MMA warp (576 threads at D = 128, 320 at D =
// 64). With G query tiles S_g lies at TMEM columns [128 g, 128 g + 128), P_g as bf16 over
// the first 32 columns of either half of S_g, O_g from 128 G on; per step P_0 V, S_0 of
// the next, and with two tiles P_1 V, S_1 of the next. Two threads a row instead of one:
// the cap costs five products on packed pairs a score pair and the exponential one of 16
// lanes a clock, and four warps a scheduler keep both busy.
//
// What bounds it: the latency of a softmax warp's chain from scores to P (no unit is full:
// tensor core and special-function unit 48 % each, issue 45 %), and a start and end of
// about 10 us a CTA that nothing overlaps at D = 128. B2 H16 N8192 D128 causal, cap 50: 566
// us a call after a rest (971 TFLOP/s), 627 back to back under the power cap; the products
// alone would be 335 us, the unshaped forward is 466. B4 H16 N2048 D64 causal, bias: 82 us,
// where one exponential a score is 30 us. Every form with a running maximum spills 12 to 64
// bytes a thread at its 96 registers.
//
// One reading of S. The reference a tile's P are taken at is the maximum of the tiles
// before it (the halves' maxima meet in shared memory; the next step's S orders
// that); the tile's own maximum is found beside its exponentials. Only if a score
// exceeds the reference by 2^64, or a row's first visible tile lies below 2^-20 of
// reference 0, is the tile read again for its maximum first; the two warps of the
// same rows agree on that with one barrier. A bias can make that the rule where its
// favourites come last: see the order of the tiles below.
//
// The cap. Up to |s| <= 0.4 cap / scale a polynomial of four terms, up to 0.8 cap /
// scale one of six (score_cap.cuh), which leave the special-function unit to the one
// exponential a score; a warp with a larger score among 16 columns takes tanh by
// exponential and reciprocal there.
//
// The bias. Along a row |i - j| slope2 is linear on either side of the diagonal: one
// fused multiply-add a score; 16 columns that hold the diagonal take the distance
// per element.
#include <limits.h>
#include <math.h>

#include "score_cap.cuh"
#include "shaped.h"

namespace fa {
namespace {
namespace sfwd {

constexpr int BM = 128;
constexpr int BN = 128;
constexpr uint32_t TM_S = 0;
constexpr uint32_t SPAN = 128 * 128;
constexpr float RESCALE_LOG2 = 8.f;
constexpr float HIGH_LOG2 = 64.f;     // largest z - m that is taken as it is
constexpr float LOW_LOG2 = -20.f;     // least one of a row's first visible tile
constexpr unsigned FULL = 0xffffffffu;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.69314718055994531f;

template <int D>
struct Cfg {
  static constexpr int G = D == 128 ? 2 : 1;         // query tiles per CTA
  static constexpr int CTAS = D == 128 ? 1 : 2;      // CTAs per SM
  // Query tiles x two halves of 64 keys x four lane quarters.
  static constexpr int SOFTMAX_WARPS = 8 * G;
  static constexpr int THREADS = 32 * SOFTMAX_WARPS + 64;
  static constexpr int WARP_TMA = SOFTMAX_WARPS;
  static constexpr int WARP_MMA = SOFTMAX_WARPS + 1;
  static constexpr uint32_t TM_O = G * 128;
  static constexpr uint32_t TMEM_COLS = 256 * G;
  static_assert(TM_O + G * D <= TMEM_COLS && CTAS * TMEM_COLS <= 512, "TMEM budget");
  static constexpr uint32_t TILE = BM * D * 2;
  static constexpr int KS = 3;
  static constexpr int VS = 2;
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_K = OFF_Q + G * TILE;
  static constexpr uint32_t OFF_V = OFF_K + KS * TILE;
  static constexpr uint32_t OFF_BAR = OFF_V + VS * TILE;
  // q_full, k_full[KS], k_empty[KS], v_full[VS], v_empty[VS], s_full[2],
  // p_ready[2], o_full
  static constexpr int NBAR = 1 + 2 * KS + 2 * VS + 5;
  static constexpr uint32_t OFF_MISC = OFF_BAR + NBAR * 8;   // tmem slot, abort, lo[2], hi[2]
  static constexpr uint32_t OFF_ROW = OFF_MISC + 32;   // float [2 halves][G BM]: row maxima, sums
  static constexpr uint32_t SMEM = OFF_ROW + 2 * G * BM * 4;
  static_assert(CTAS == 1 ? SMEM <= 232448 : 2 * (SMEM + 1024) <= 233472, "shared memory budget");
};

template <int D>
struct Bars {
  using C = Cfg<D>;
  uint32_t b;
  __device__ uint32_t q_full() const { return b; }
  __device__ uint32_t k_full(int s) const { return b + 8u * (1 + s); }
  __device__ uint32_t k_empty(int s) const { return b + 8u * (1 + C::KS + s); }
  __device__ uint32_t v_full(int s) const { return b + 8u * (1 + 2 * C::KS + s); }
  __device__ uint32_t v_empty(int s) const { return b + 8u * (1 + 2 * C::KS + C::VS + s); }
  __device__ uint32_t s_full(int g) const { return b + 8u * (1 + 2 * C::KS + 2 * C::VS + g); }
  __device__ uint32_t p_ready(int g) const { return b + 8u * (3 + 2 * C::KS + 2 * C::VS + g); }
  __device__ uint32_t o_full() const { return b + 8u * (5 + 2 * C::KS + 2 * C::VS); }
};

enum : unsigned {
  W_Q = 0xC0100, W_KEMPTY = 0xC0200, W_VEMPTY = 0xC0300, W_KFULL = 0xC0400, W_VFULL = 0xC0500,
  W_SFULL = 0xC0600, W_PREADY = 0xC0700, W_OFULL = 0xC0800, BAD_ALIGN = 0xC0900
};

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const DevErr& e,
                                          volatile int* abort, unsigned where) {
  const bool ok = mbar_wait(bar, parity, e, abort, where);
  return __all_sync(FULL, ok);
}

// The two warps that hold the halves of the same 32 rows meet. The AND form tells both
// whether both are on track, so that a wait that ran out ends the loops of both at the
// same barrier; the OR form gathers a vote.
__device__ __forceinline__ bool rows_and(int id, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "bar.red.and.pred q, %1, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(id), "r"(ok ? 1u : 0u)
      : "memory");
  return all != 0;
}

__device__ __forceinline__ bool rows_or(int id, bool v) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "bar.red.or.pred q, %1, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(v ? 1u : 0u)
      : "memory");
  return any != 0;
}

// TMEM column of k-step kk of P: each 64-key half lies in the first 32 of its own
// 64 score columns.
__device__ __forceinline__ uint32_t packed_col(int kk) { return (kk >> 2) * 64 + (kk & 3) * 8; }

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// What a thread knows of its row and its 64 keys of one tile.
constexpr int HK = 64;
struct RowTile {
  int lo, hi;   // visible columns [lo, hi) of the half
  int dist0;    // first key - query
};

// 16 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// Under a cap and without a bias the scores lie in [-A, A], and while A <= 74 (a cap of
// 51) no maximum is needed: with the reference m = max(0, ceil(A) - 64), P = 2^(x - m) lies
// in [2^-84, 2^64] whatever the row holds. No half waits for the other and O is never
// rescaled: B2 H16 N8192 D128 causal 562 us under a cap just inside, 692 with the running
// maximum. The top is the one that a running maximum allows too (HIGH_LOG2), so that O
// overflows in no mode while the |v| of a query's keys add up to less than 2^63; at the
// other end P v keeps fp32's precision for |v| from 2^-42 on.
constexpr float FIXED_AMP = 74.f;

// MODE: which parts of the shape the scores have (key ranges always).
enum Mode : int { RANGES = 0, BIASED = 1, CAPPED = 2, CAPPED_BIASED = 3, CAPPED_FIXED = 4 };

constexpr bool has_bias(int mode) { return mode == BIASED || mode == CAPPED_BIASED; }
constexpr bool has_cap(int mode) { return mode >= CAPPED; }

// z - m of 16 scores, their maximum into mx; with EXP P = 2^(z - m) as packed bf16 and
// its sum, with PARTIAL what packing added to it too. FORM: 0 and 1 the polynomials of
// the cap, 2 its exponential form.
template <int MODE, bool PARTIAL, bool EXP, int FORM>
__device__ __forceinline__ void chunk(const uint32_t (&r)[16], int lo, int hi, int d0, float c2,
                                      const CapArgs& cap, float slope2, float m, float2 (&sum)[2],
                                      float2& drift, float (&mx)[2], uint32_t* pk) {
  constexpr bool BIAS = has_bias(MODE);
  const float sl = d0 >= 0 ? -slope2 : slope2;
  const bool mixed = PARTIAL && BIAS && __any_sync(FULL, d0 < 0 && d0 + 15 > 0);
  const float d0f = static_cast<float>(d0);
  const float base = BIAS ? fmaf(sl, d0f, -m) : -m;
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const float2 s = make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1]));
    float2 add = make_float2(base, base);
    if (BIAS) {
      if (mixed) {
        add.x = fmaf(-slope2, fabsf(d0f + static_cast<float>(i)), -m);
        add.y = fmaf(-slope2, fabsf(d0f + static_cast<float>(i + 1)), -m);
      } else {
        add = __ffma2_rn(make_float2(sl, sl),
                         make_float2(static_cast<float>(i), static_cast<float>(i + 1)), add);
      }
    }
    float2 x;
    if (!has_cap(MODE))
      x = __ffma2_rn(s, make_float2(c2, c2), add);
    else if (FORM < 2)
      x = __ffma2_rn(s, cap_poly2<FORM>(cap, s), add);
    else
      x = make_float2(fmaf(cap.amp, cap_tanh(cap, s.x), add.x), fmaf(cap.amp, cap_tanh(cap, s.y), add.y));
    if (PARTIAL) {
      x.x = (i >= lo && i < hi) ? x.x : -INFINITY;
      x.y = (i + 1 >= lo && i + 1 < hi) ? x.y : -INFINITY;
    }
    if (MODE != CAPPED_FIXED) mx[(i >> 1) & 1] = max3(mx[(i >> 1) & 1], x.x, x.y);
    if (EXP) {
      const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
      sum[(i >> 1) & 1] = __fadd2_rn(sum[(i >> 1) & 1], make_float2(p0, p1));
      pk[i >> 1] = pack_bf16x2(p0, p1);
      if (PARTIAL) {
        const float2 held = make_float2(__uint_as_float(pk[i >> 1] << 16),
                                        __uint_as_float(pk[i >> 1] & 0xffff0000u));
        drift = __fadd2_rn(drift, __fadd2_rn(held, make_float2(-p0, -p1)));
      }
    }
  }
}

// The thread's 64 scores of a tile, 16 at a time, the next 16 on their way. Returns the
// largest z - m; with EXP P's sum is added to l, with PARTIAL too the rounding of its P to
// drift, and P goes into pk or, in the fixed mode, straight to TMEM.
template <int MODE, bool PARTIAL, bool EXP>
__device__ __forceinline__ float half_tile(uint32_t s_col, const RowTile& t, float c2,
                                           const CapArgs& cap, float slope2, float m, float& l,
                                           float& drift, uint32_t* pk) {
  constexpr bool FIXED = MODE == CAPPED_FIXED;
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  float2 dr = make_float2(0.f, 0.f);
  float mx[2] = {-INFINITY, -INFINITY};
  uint32_t r[2][16];
  tmem_ld16(s_col, r[0]);
#pragma unroll
  for (int c = 0; c < HK / 16; ++c) {
    uint32_t(&q)[16] = r[c & 1];
    uint32_t here[8];
    uint32_t* to = FIXED ? here : pk + 8 * c;
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(q[i]));
    if (c + 1 < HK / 16) tmem_ld16(s_col + 16 * (c + 1), r[(c + 1) & 1]);
    const int lo = t.lo - 16 * c, hi = t.hi - 16 * c, d0 = t.dist0 + 16 * c;
    if (!has_cap(MODE)) {
      chunk<MODE, PARTIAL, EXP, 0>(q, lo, hi, d0, c2, cap, slope2, m, sum, dr, mx, to);
    } else {
      float ab[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 16; i += 2)
        ab[(i >> 1) & 1] = max3(ab[(i >> 1) & 1], fabsf(__uint_as_float(q[i])),
                                fabsf(__uint_as_float(q[i + 1])));
      const int form = cap_form(cap, fmaxf(ab[0], ab[1]));
      if (form == 0)
        chunk<MODE, PARTIAL, EXP, 0>(q, lo, hi, d0, c2, cap, slope2, m, sum, dr, mx, to);
      else if (form == 1)
        chunk<MODE, PARTIAL, EXP, 1>(q, lo, hi, d0, c2, cap, slope2, m, sum, dr, mx, to);
      else
        chunk<MODE, PARTIAL, EXP, 2>(q, lo, hi, d0, c2, cap, slope2, m, sum, dr, mx, to);
    }
    // Columns 8 c .. 8 c + 7: scores that have been read.
    if (FIXED) tmem_st8(s_col + 8 * c, here);
  }
  if (EXP) l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
  if (EXP && PARTIAL) drift += dr.x + dr.y;
  return fmaxf(mx[0], mx[1]);
}

// (m + log2 l) ln 2, the exponent of l apart: under the fixed reference it is a large
// part of log2 l, whose approximation has a relative error.
__device__ __forceinline__ float row_lse(float m, float l) {
  if (!(l > 0.f)) return -INFINITY;
  const int e = (__float_as_int(l) >> 23) - 127;
  const float f = __int_as_float((__float_as_int(l) & 0x007fffff) | 0x3f800000);
  return (m + static_cast<float>(e) + __log2f(f)) * LN2;
}

template <int D, int MODE>
__global__ void __launch_bounds__(Cfg<D>::THREADS, Cfg<D>::CTAS)
    shaped_fwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const AttnParams p,
                      const ShapeArgs sh, const CapArgs cap, int num_m, int group) {
  using C = Cfg<D>;
  constexpr bool BIAS = has_bias(MODE);
  constexpr bool FIXED = MODE == CAPPED_FIXED;
  constexpr int KS = C::KS, VS = C::VS, G = C::G;
  constexpr int SOFTMAX_WARPS = C::SOFTMAX_WARPS, WARP_TMA = C::WARP_TMA, WARP_MMA = C::WARP_MMA;
  constexpr uint32_t TM_O = C::TM_O, TMEM_COLS = C::TMEM_COLS;
  constexpr uint32_t TILE = C::TILE, OFF_Q = C::OFF_Q, OFF_K = C::OFF_K, OFF_V = C::OFF_V;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if ((sbase & 1023u) != 0) {
    if (threadIdx.x == 0) record_bounds(p.err, BAD_ALIGN);
    return;
  }
  // Groups of heads for L2 reuse of K / V; inside a group the last query tiles
  // (the longest under a causal mask) first.
  const TileSlot ts = grouped_slot(blockIdx.x, num_m, p.H * p.B, group);
  const int mt = (num_m - 1 - ts.t) * G;   // first query tile
  const int h = ts.unit % p.H;
  const int b = ts.unit / p.H;
  const SeqInfo sq = seq_info(p, b);
  if (!seq_ok(p, sq) || mt * BM >= sq.len) return;   // whole CTA, before any shared state
  const int hk = h / (p.H / p.H_kv);

  const Bars<D> bars{sbase + C::OFF_BAR};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* s_lo = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);    // per query tile
  int* s_hi = reinterpret_cast<int*>(smem + C::OFF_MISC + 16);
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;

  // This thread's row (softmax warps) and its keys: warps 0-7 query tile 0, 8-15
  // tile 1; of each the first four the keys [0, 64) of a tile, the others the rest.
  const int qpos = (mt + (warp >> 3)) * BM + (warp & 3) * 32 + lane;
  KeyRange kr = {0, 0};
  if (warp < SOFTMAX_WARPS && qpos < sq.len) kr = key_range(p, sh, sq, qpos);
  if (threadIdx.x == WARP_TMA * 32) {
    *abort = 0;
    s_lo[0] = s_lo[1] = INT_MAX;
    s_hi[0] = s_hi[1] = 0;
    mbar_init(bars.q_full(), 1);
    for (int s = 0; s < KS; ++s) {
      mbar_init(bars.k_full(s), 1);
      mbar_init(bars.k_empty(s), 1);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(bars.v_full(s), 1);
      mbar_init(bars.v_empty(s), 1);
    }
    for (int g = 0; g < G; ++g) {
      mbar_init(bars.s_full(g), 1);
      mbar_init(bars.p_ready(g), 256);
    }
    mbar_init(bars.o_full(), 1);
    fence_mbar_init();
    // Q does not wait for the ranges.
    mbar_arrive_expect_tx(bars.q_full(), G * TILE);
    for (int g = 0; g < G; ++g)
      for (int c = 0; c < D / 64; ++c)
        tma_load_2d(sbase + OFF_Q + g * TILE + c * SPAN, &tm_q, bars.q_full(), h * D + c * 64,
                    sq.start + (mt + g) * BM);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == WARP_MMA) {
    tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  __syncthreads();
  if (warp < SOFTMAX_WARPS && (warp & 4) == 0) {
    const int lo = __reduce_min_sync(FULL, kr.lo < kr.hi ? kr.lo : INT_MAX);
    const int hi = __reduce_max_sync(FULL, kr.hi);
    if (lane == 0 && hi > 0) {
      atomicMin(&s_lo[warp >> 3], lo);
      atomicMax(&s_hi[warp >> 3], hi);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Key tiles [t_g, e_g) of query tile g. The CTA walks their union [t0, t1); tile g
  // takes part in the steps [b_g, f_g). With a bias from the end: under a causal mask
  // the keys nearest to the queries, which the bias favours, then come first and set
  // the reference for good (91 against 127 us on B4 H16 N2048 D64); without one the
  // order makes no difference (571 us on B2 H16 N8192 D128 with a cap either way). Where
  // queries see keys behind them too, an early one starts with its farthest: each tile on
  // its way to the diagonal moves the reference, or is read again where the bias grows by
  // 2^64 within it (the same case not causal, slopes of 2^(-h/2): 257 us; of 0.6: 294; the
  // unshaped forward 120; negative slopes, causal, -0.6: 217).
  const bool any_0 = s_hi[0] > 0, any_1 = G > 1 && s_hi[1] > 0;
  const int t_0 = any_0 ? s_lo[0] / BN : INT_MAX, t_1 = any_1 ? s_lo[1] / BN : INT_MAX;
  const int e_0 = (s_hi[0] + BN - 1) / BN, e_1 = any_1 ? (s_hi[1] + BN - 1) / BN : 0;
  const int t0 = min(t_0, t_1), t1 = max(e_0, e_1);
  const int n_kv = t1 > 0 ? t1 - t0 : 0;
  const int b_0 = !any_0 ? 0 : BIAS ? t1 - e_0 : t_0 - t0;
  const int b_1 = !any_1 ? 0 : BIAS ? t1 - e_1 : t_1 - t0;
  const int f_0 = !any_0 ? 0 : b_0 + e_0 - t_0, f_1 = !any_1 ? 0 : b_1 + e_1 - t_1;
  auto key_tile = [&](int it) { return BIAS ? t1 - 1 - it : t0 + it; };

  if (warp == WARP_TMA) {
    // ------------------------------------------------------------ producer ---
    // The whole warp runs the loop; lane 0 issues the copies.
    int jk = 0, jv = 0;
    long long t_last = clock64();
    while (jk < n_kv || jv < n_kv) {
      bool progress = false;
      if (jk < n_kv &&
          __all_sync(FULL, mbar_try_wait(bars.k_empty(jk % KS), ((jk / KS) & 1) ^ 1))) {
        const int st = jk % KS;
        if (lane == 0) {
          mbar_arrive_expect_tx(bars.k_full(st), TILE);
          for (int c = 0; c < D / 64; ++c)
            tma_load_2d(sbase + OFF_K + st * TILE + c * SPAN, &tm_k, bars.k_full(st),
                        hk * D + c * 64, sq.start + key_tile(jk) * BN);
        }
        __syncwarp();
        ++jk;
        progress = true;
      }
      if (jv < jk &&
          __all_sync(FULL, mbar_try_wait(bars.v_empty(jv % VS), ((jv / VS) & 1) ^ 1))) {
        const int st = jv % VS;
        if (lane == 0) {
          mbar_arrive_expect_tx(bars.v_full(st), TILE);
          for (int c = 0; c < D / 64; ++c)
            tma_load_2d(sbase + OFF_V + st * TILE + c * SPAN, &tm_v, bars.v_full(st),
                        hk * D + c * 64, sq.start + key_tile(jv) * BN);
        }
        __syncwarp();
        ++jv;
        progress = true;
      }
      if (progress) {
        t_last = clock64();
        continue;
      }
      // Lane 0 decides, so the whole warp leaves the loop together.
      const int stop =
          __shfl_sync(FULL, *abort ? 1 : (clock64() - t_last > p.err.budget ? 2 : 0), 0);
      if (stop == 1) break;
      if (stop == 2) {
        if (lane == 0) {
          *abort = 1;
          atomicOr(p.err.word, ERR_TIMEOUT);
          atomicExch(p.err.word + 1, jk < n_kv ? W_KEMPTY : W_VEMPTY);
        }
        break;
      }
    }
    if (lane == 0) {
      // Q has landed even where no key is seen.
      if (n_kv == 0) mbar_wait(bars.q_full(), 0, p.err, abort, W_Q);
      // Drain: the tensor core's arrivals on the last stages' empty barriers
      // must land before the CTA's shared memory is released.
      for (int j = max(0, n_kv - KS); j < n_kv && !*abort; ++j)
        if (!mbar_wait(bars.k_empty(j % KS), (j / KS) & 1, p.err, abort, W_KEMPTY)) break;
      for (int j = max(0, n_kv - VS); j < n_kv && !*abort; ++j)
        if (!mbar_wait(bars.v_empty(j % VS), (j / VS) & 1, p.err, abort, W_VEMPTY)) break;
    }
  } else if (warp == WARP_MMA) {
    // ---------------------------------------------------------- MMA issuer ---
    // Per step: P_0 V, S_0 of the next, P_1 V, S_1 of the next, for the tiles
    // that take part. S_g of the next step overwrites P_g: it follows P_g V.
    const uint32_t leader = elect_one();
    constexpr uint32_t IDESC_QK = idesc_bf16(BM, BN, false, false);
    constexpr uint32_t IDESC_PV = idesc_bf16(BM, D, false, true);
    const uint64_t q_desc = sdesc_sw128(sbase + OFF_Q, 16, 1024);
    const uint64_t k_desc = sdesc_sw128(sbase + OFF_K, 16, 1024);
    const uint64_t v_desc = sdesc_sw128(sbase + OFF_V, SPAN, 1024);
    auto issue_s = [&](int g, int it) {
      const int st = it % KS;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t o = (kk >> 2) * SPAN + (kk & 3) * 32;
        mma_ss_if(leader, tmem + TM_S + g * BN, sdesc_add(q_desc, g * TILE + o),
                  sdesc_add(k_desc, st * TILE + o), IDESC_QK, kk > 0);
      }
      tc_commit_if(leader, bars.s_full(g));
    };
    auto issue_pv = [&](int g, int it, bool fresh) {
      const int st = it % VS;
#pragma unroll
      for (int kk = 0; kk < BN / 16; ++kk)
        mma_ts_if(leader, tmem + TM_O + g * D, tmem + TM_S + g * BN + packed_col(kk),
                  sdesc_add(v_desc, st * TILE + kk * 2048), IDESC_PV,
                  (!fresh || kk > 0) ? 1u : 0u);
    };
    bool ok = n_kv > 0;
    if (ok) {
      ok = warp_wait(bars.q_full(), 0, p.err, abort, W_Q) &&
           warp_wait(bars.k_full(0), 0, p.err, abort, W_KFULL);
      if (ok) {
        tc_fence_after();
        if (b_0 == 0 && f_0 > 0) issue_s(0, 0);
        if (G > 1 && b_1 == 0 && f_1 > 0) issue_s(1, 0);
        tc_commit_if(leader, bars.k_empty(0));
      }
    }
    for (int it = 0; ok && it < n_kv; ++it) {
      const bool next = it + 1 < n_kv;
      if (!(ok = warp_wait(bars.v_full(it % VS), (it / VS) & 1, p.err, abort, W_VFULL))) break;
      bool k_seen = false;
#pragma unroll
      for (int g = 0; g < G && ok; ++g) {
        const int bg = g ? b_1 : b_0, fg = g ? f_1 : f_0;
        if (it >= bg && it < fg) {
          if (!(ok = warp_wait(bars.p_ready(g), (it - bg) & 1, p.err, abort, W_PREADY))) break;
          tc_fence_after();
          issue_pv(g, it, it == bg);
        }
        if (it + 1 >= bg && it + 1 < fg) {
          if (!k_seen) {
            if (!(ok = warp_wait(bars.k_full((it + 1) % KS), ((it + 1) / KS) & 1, p.err, abort,
                                 W_KFULL)))
              break;
            tc_fence_after();
            k_seen = true;
          }
          issue_s(g, it + 1);
        }
      }
      if (!ok) break;
      tc_commit_if(leader, bars.v_empty(it % VS));
      if (next) {
        // A tile between the two ranges is read by neither: its stage is given
        // back once it has landed.
        if (!k_seen && !(ok = warp_wait(bars.k_full((it + 1) % KS), ((it + 1) / KS) & 1, p.err,
                                        abort, W_KFULL)))
          break;
        tc_commit_if(leader, bars.k_empty((it + 1) % KS));
      }
    }
    if (n_kv > 0) tc_commit_if(leader, bars.o_full());   // some softmax group waits for it
  } else {
    // ------------------------------------------------------------- softmax ---
    const int g = warp >> 3;            // query tile
    const int hf = (warp >> 2) & 1;     // half of a tile's keys; half of O's columns
    const int row = (warp & 3) * 32 + lane;
    const int bar_id = 1 + g * 4 + (warp & 3);
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_off + TM_S + g * BN + hf * HK;
    const uint32_t o_col = tmem + lane_off + TM_O + g * D + hf * (D / 2);
    float* s_row = reinterpret_cast<float*>(smem + C::OFF_ROW) + g * BM + row;
    const int bg = g ? b_1 : b_0, n = (g ? f_1 : f_0) - bg;
    const float c2 = p.scale_log2;
    const float slope2 = BIAS ? __ldg(sh.slopes + h) * LOG2E : 0.f;
    float m_ref = FIXED ? fmaxf(0.f, ceilf(cap.amp) - HIGH_LOG2) : -INFINITY;
    float last = -INFINITY;   // this half's maximum of the step before
    float l = 0.f;            // this half's part of the row's sum
    // What the rounding of P to bf16 added to that, in tiles with masks: O is divided by
    // l + drift, the sum of the P that it was made of, so that a row with one key is that
    // key's V, and one with a few loses less. (Over whole tiles the roundings average out.)
    float drift = 0.f;
    bool ok = true;
    for (int i = 0; i < n && ok; ++i) {
      const int key0 = key_tile(bg + i) * BN + hf * HK;
      RowTile t;
      t.lo = kr.lo - key0;
      t.hi = kr.hi - key0;
      t.dist0 = key0 - qpos;
      // A warp that sees all 64 keys on one side of the diagonal needs no
      // element-wise mask or distance.
      const bool whole = __all_sync(FULL, t.lo <= 0 && t.hi >= HK &&
                                              (!BIAS || t.dist0 >= 0 || t.dist0 + HK <= 1));
      const bool none = !whole && !__any_sync(FULL, t.lo < HK && t.hi > 0 && t.lo < t.hi);
      ok = warp_wait(bars.s_full(g), i & 1, p.err, abort, W_SFULL);
      tc_fence_after();
      if (FIXED && !ok) break;
      // O, which holds the tiles before the last step's (S_g of this step completing
      // means P_g V of the last one has), moves with the reference.
      auto rescale = [&](float alpha) {
        l *= alpha;
        drift *= alpha;
        if (i == 0 || !__any_sync(FULL, alpha != 1.f)) return;
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          uint32_t o[32];
          tmem_ld32(o_col + 32 * c, o);
          tmem_ld_wait();
          reg_fence(o);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
          tmem_st32(o_col + 32 * c, o);
        }
      };
      if (!FIXED && ok && i > 0) {
        const float m_cand = fmaxf(last, s_row[(hf ^ 1) * G * BM]);
        float alpha = 1.f;
        // The first tile with a visible key, of either half, was taken at reference 0.
        if (m_ref == -INFINITY && m_cand != -INFINITY) m_ref = 0.f;
        if (m_cand > m_ref + RESCALE_LOG2) {
          alpha = ex2_approx(m_ref - m_cand);
          m_ref = m_cand;
        }
        rescale(alpha);
      }
      if constexpr (FIXED) {
        if (none) {
          const uint32_t z[16] = {};
          tmem_st16(s_col, z);
          tmem_st16(s_col + 16, z);
        } else if (whole) {
          half_tile<MODE, false, true>(s_col, t, c2, cap, slope2, m_ref, l, drift, nullptr);
        } else {
          half_tile<MODE, true, true>(s_col, t, c2, cap, slope2, m_ref, l, drift, nullptr);
        }
      } else {
        uint32_t pk[32];
        float sum = 0.f, dr = 0.f, mx = -INFINITY;
        float m_use = m_ref == -INFINITY ? 0.f : m_ref;
        if (none || !ok) {
#pragma unroll
          for (int k = 0; k < 32; ++k) pk[k] = 0u;
        } else {
          mx = whole ? half_tile<MODE, false, true>(s_col, t, c2, cap, slope2, m_use, sum, dr, pk)
                     : half_tile<MODE, true, true>(s_col, t, c2, cap, slope2, m_use, sum, dr, pk);
        }
        bool again = rows_or(bar_id, mx > HIGH_LOG2 || !ok);
        if (!again && __any_sync(FULL, m_ref == -INFINITY)) {
          // A row's first visible tile: low if both halves are. The partner, which holds
          // the same rows and references, comes to the same answer.
          s_row[hf * G * BM] = m_use + mx;
          if (!(ok = rows_and(bar_id, ok))) break;
          const float top = fmaxf(m_use + mx, s_row[(hf ^ 1) * G * BM]);
          again = __any_sync(FULL, m_ref == -INFINITY && top < LOW_LOG2 && top != -INFINITY);
        }
        if (again) {
          if (!(ok = rows_and(bar_id, ok))) break;
          // The maximum first, of both halves, then P.
          sum = dr = 0.f;
          mx = -INFINITY;
          if (!none) mx = half_tile<MODE, true, false>(s_col, t, c2, cap, slope2, 0.f, sum, dr, pk);
          s_row[hf * G * BM] = mx;
          if (!(ok = rows_and(bar_id, ok))) break;
          const float m_cand = fmaxf(mx, s_row[(hf ^ 1) * G * BM]);
          if (!(ok = rows_and(bar_id, ok))) break;   // both have read
          float alpha = 1.f;
          if (m_cand > m_ref + RESCALE_LOG2) {
            if (m_ref != -INFINITY) alpha = ex2_approx(m_ref - m_cand);
            m_ref = m_cand;
          }
          rescale(alpha);
          m_use = m_ref == -INFINITY ? 0.f : m_ref;
          if (!none) mx = half_tile<MODE, true, true>(s_col, t, c2, cap, slope2, m_use, sum, dr, pk);
        }
        last = m_use + mx;
        s_row[hf * G * BM] = last;
        l += sum;
        drift += dr;
        uint32_t lo16[16], hi16[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          lo16[k] = pk[k];
          hi16[k] = pk[16 + k];
        }
        tmem_st16(s_col, lo16);
        tmem_st16(s_col + 16, hi16);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bars.p_ready(g));
    }
    // ------------------------------------------------------------ epilogue ---
    const bool row_ok = qpos < sq.len;
    const size_t out_row = static_cast<size_t>(sq.start + qpos) * p.H + h;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + out_row * D + hf * (D / 2));
    if (n > 0) ok = ok && warp_wait(bars.o_full(), 0, p.err, abort, W_OFULL);
    s_row[hf * G * BM] = l;   // o_full: the partner has read the last maximum
    ok = rows_and(bar_id, ok);
    l += s_row[(hf ^ 1) * G * BM];
    ok = rows_and(bar_id, ok);   // both have read
    s_row[hf * G * BM] = drift;
    ok = rows_and(bar_id, ok);
    drift += s_row[(hf ^ 1) * G * BM];
    if (ok) {
      tc_fence_after();
      const float inv_l = (l > 0.f) ? 1.f / (l + drift) : 0.f;
#pragma unroll 1
      for (int c = 0; c < D / 64; ++c) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32(o_col + 32 * c, o);
          tmem_ld_wait();
          reg_fence(o);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0u;
        }
        if (row_ok) {
#pragma unroll
          for (int v4 = 0; v4 < 4; ++v4) {
            uint4 w;
            w.x = pack_bf16x2(__uint_as_float(o[8 * v4 + 0]) * inv_l, __uint_as_float(o[8 * v4 + 1]) * inv_l);
            w.y = pack_bf16x2(__uint_as_float(o[8 * v4 + 2]) * inv_l, __uint_as_float(o[8 * v4 + 3]) * inv_l);
            w.z = pack_bf16x2(__uint_as_float(o[8 * v4 + 4]) * inv_l, __uint_as_float(o[8 * v4 + 5]) * inv_l);
            w.w = pack_bf16x2(__uint_as_float(o[8 * v4 + 6]) * inv_l, __uint_as_float(o[8 * v4 + 7]) * inv_l);
            dst[4 * c + v4] = w;
          }
        }
      }
      if (row_ok && hf == 0)
        p.lse[lse_index(p, b, h, sq.start, qpos)] =
            row_lse(m_ref == -INFINITY ? 0.f : m_ref, l);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

template <int D, int MODE>
cudaError_t launch(const AttnParams& p, const ShapeArgs& sh, cudaStream_t stream) {
  using C = Cfg<D>;
  const int num_m = (p.max_seqlen + C::G * BM - 1) / (C::G * BM);
  const long long tiles = static_cast<long long>(num_m) * p.H * p.B;
  if (tiles > INT_MAX) return cudaErrorInvalidConfiguration;
  CUtensorMap tq, tk, tv;
  if (!make_tmap_bf16_2d(&tq, p.q, p.total, static_cast<unsigned long long>(p.H) * D, 64, BM) ||
      !make_tmap_bf16_2d(&tk, p.k, p.total, static_cast<unsigned long long>(p.H_kv) * D, 64, BN) ||
      !make_tmap_bf16_2d(&tv, p.v, p.total, static_cast<unsigned long long>(p.H_kv) * D, 64, BN))
    return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem<shaped_fwd_kernel<D, MODE>>(C::SMEM);
  if (e != cudaSuccess) return e;
  const int group = l2_group(4ll * p.max_seqlen * D, p.H / p.H_kv, p.H * p.B);
  const CapArgs cap = MODE >= CAPPED ? cap_args(sh.cap, p.scale) : CapArgs{};
  shaped_fwd_kernel<D, MODE><<<static_cast<unsigned>(tiles), C::THREADS, C::SMEM, stream>>>(
      tq, tk, tv, p, sh, cap, num_m, group);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const AttnParams& p, const ShapeArgs& sh, cudaStream_t stream) {
  const bool bias = sh.slopes != nullptr;
  if (!(sh.cap > 0.f)) return bias ? launch<D, BIASED>(p, sh, stream) : launch<D, RANGES>(p, sh, stream);
  if (bias) return launch<D, CAPPED_BIASED>(p, sh, stream);
  return sh.cap * LOG2E <= FIXED_AMP ? launch<D, CAPPED_FIXED>(p, sh, stream)
                                     : launch<D, CAPPED>(p, sh, stream);
}

}  // namespace sfwd
}  // namespace

cudaError_t launch_shaped_fwd(const AttnParams& p, const ShapeArgs& sh, cudaStream_t stream) {
  return p.D == 64 ? sfwd::launch_d<64>(p, sh, stream) : sfwd::launch_d<128>(p, sh, stream);
}

}  // namespace fa
