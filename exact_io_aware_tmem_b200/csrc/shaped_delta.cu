// D_i of the backward with shaped scores, from the probabilities themselves:
//     D_i = sum_j P_ij dP_ij,  P = exp(z - LSE),  dP = dO V^T;
// the dQ accumulator's rows set to zero; and the range of keys that each query tile sees.
//
// Why not dO_i . O_i. Where a row's weight lies on a few keys, as under a window, a
// steep bias or large logits, dP_ij - D_i of those keys is a small difference, and D
// from an O that was formed from bf16 P and rounded to bf16 makes up most of dQ's and
// dK's error: relative (Frobenius) 0.0060 on H 1 N 512 D 64 with a cap of 50, logits of
// standard deviation 4 and a slope of 0.7, against 0.0024 with D as here, where only dX
// and the outputs are rounded.
//
// How, on B200. One CTA per (sequence, head, 128-row query tile): S = Q K^T and dP = dO
// V^T per key tile, two tensor-core products into TMEM, which the softmax warps read and
// reduce; nothing goes back to the tensor core, so that the two sides run apart: at D =
// 128 over two buffers of both products, at D = 64 over one, with two CTAs a SM. A thread
// has a row and 32 (D = 128) or 64 keys of a tile; the row's partial sums meet at the end.
// The references are the saved LSEs: no maximum, one reading, one exponential a score.
//
// B1 H16/4 N8192 D128 causal, cap 50: 254 us, where the two products are 168 us at the
// tensor core's measured rate (sm__pipe_tensor 47 % active at N 4096, the
// special-function unit 48 %): neither is full, because both wait through the start and
// end of each CTA and at D = 128 shared memory holds one CTA a SM.
#include <limits.h>
#include <math.h>

#include "score_cap.cuh"
#include "shaped.h"

namespace fa {
namespace {
namespace sdelta {

constexpr int BM = 128;
constexpr int BN = 128;
constexpr uint32_t SPAN = 128 * 128;
constexpr unsigned FULL = 0xffffffffu;
constexpr float LOG2E = 1.4426950408889634f;

template <int D>
struct Cfg {
  static constexpr int NB = D == 128 ? 2 : 1;       // buffers of S and dP
  static constexpr int CTAS = D == 128 ? 1 : 2;     // CTAs per SM
  static constexpr int CG = D == 128 ? 4 : 2;       // threads per row
  static constexpr int COLS = BN / CG;              // keys of a thread per tile
  static constexpr int SOFTMAX_WARPS = 4 * CG;
  static constexpr int THREADS = 32 * SOFTMAX_WARPS + 64;
  static constexpr int WARP_TMA = SOFTMAX_WARPS;
  static constexpr int WARP_MMA = SOFTMAX_WARPS + 1;
  static constexpr uint32_t TMEM_COLS = 256 * NB;   // S, dP per buffer
  static constexpr uint32_t TILE = BM * D * 2;
  static constexpr int ST = 2;                      // K and V stages
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_DO = OFF_Q + TILE;
  static constexpr uint32_t OFF_K = OFF_DO + TILE;
  static constexpr uint32_t OFF_V = OFF_K + ST * TILE;
  static constexpr uint32_t OFF_BAR = OFF_V + ST * TILE;
  // q_full, kv_full[ST], kv_empty[ST], full[NB], free[NB]
  static constexpr int NBAR = 1 + 2 * ST + 2 * NB;
  static constexpr uint32_t OFF_MISC = OFF_BAR + NBAR * 8;   // tmem slot, abort, lo, hi
  static constexpr uint32_t OFF_SUM = OFF_MISC + 16;         // float [CG][BM]
  static constexpr uint32_t SMEM = OFF_SUM + CG * BM * 4;
  static_assert(CTAS == 1 ? SMEM <= 232448 : 2 * (SMEM + 1024) <= 233472, "shared memory budget");
};

template <int D>
struct Bars {
  using C = Cfg<D>;
  uint32_t b;
  __device__ uint32_t q_full() const { return b; }
  __device__ uint32_t kv_full(int s) const { return b + 8u * (1 + s); }
  __device__ uint32_t kv_empty(int s) const { return b + 8u * (1 + C::ST + s); }
  __device__ uint32_t full(int i) const { return b + 8u * (1 + 2 * C::ST + i); }
  __device__ uint32_t free(int i) const { return b + 8u * (1 + 2 * C::ST + C::NB + i); }
};

enum : unsigned {
  W_Q = 0xF0100, W_KVEMPTY = 0xF0200, W_KVFULL = 0xF0300, W_FULL = 0xF0400, W_FREE = 0xF0500,
  BAD_ALIGN = 0xF0900
};

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const DevErr& e,
                                          volatile int* abort, unsigned where) {
  const bool ok = mbar_wait(bar, parity, e, abort, where);
  return __all_sync(FULL, ok);
}

// acc += sum over 32 columns of 2^(z - LSE) dP; d0 = first key - query.
template <bool CAP, bool BIAS, bool PARTIAL, int FORM>
__device__ __forceinline__ void chunk(const uint32_t (&s)[32], const uint32_t (&g)[32], int lo,
                                      int hi, int d0, float c2, const CapArgs& cap, float slope2,
                                      float lse2, float2 (&acc)[2]) {
  const float sl = d0 >= 0 ? -slope2 : slope2;
  const bool mixed = PARTIAL && BIAS && __any_sync(FULL, d0 < 0 && d0 + 31 > 0);
  const float d0f = static_cast<float>(d0);
  const float base = BIAS ? fmaf(sl, d0f, -lse2) : -lse2;
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float2 sc = make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1]));
    float2 add = make_float2(base, base);
    if (BIAS) {
      if (mixed) {
        add.x = fmaf(-slope2, fabsf(d0f + static_cast<float>(i)), -lse2);
        add.y = fmaf(-slope2, fabsf(d0f + static_cast<float>(i + 1)), -lse2);
      } else {
        add = __ffma2_rn(make_float2(sl, sl),
                         make_float2(static_cast<float>(i), static_cast<float>(i + 1)), add);
      }
    }
    float2 x;
    if (!CAP)
      x = __ffma2_rn(sc, make_float2(c2, c2), add);
    else if (FORM < 2)
      x = __ffma2_rn(sc, cap_poly2<FORM>(cap, sc), add);
    else
      x = make_float2(fmaf(cap.amp, cap_tanh(cap, sc.x), add.x), fmaf(cap.amp, cap_tanh(cap, sc.y), add.y));
    float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
    if (PARTIAL) {
      p0 = (i >= lo && i < hi) ? p0 : 0.f;
      p1 = (i + 1 >= lo && i + 1 < hi) ? p1 : 0.f;
    }
    acc[(i >> 1) & 1] =
        __ffma2_rn(make_float2(p0, p1),
                   make_float2(__uint_as_float(g[i]), __uint_as_float(g[i + 1])), acc[(i >> 1) & 1]);
  }
}

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(Cfg<D>::THREADS, Cfg<D>::CTAS)
    shaped_delta_kernel(const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ CUtensorMap tm_do, const AttnParams p,
                        const ShapeArgs sh, const CapArgs cap, int2* tile_range, int num_m,
                        int group) {
  using C = Cfg<D>;
  constexpr int ST = C::ST, NB = C::NB;
  constexpr uint32_t TILE = C::TILE;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if ((sbase & 1023u) != 0) {
    if (threadIdx.x == 0) record_bounds(p.err, BAD_ALIGN);
    return;
  }
  // Rows behind the last sequence, which total_tokens == cu_seqlens[B] rules out, get a dQ
  // of zero all the same, as from the unshaped backward: the conversion reads every row.
  if (blockIdx.x == 0 && p.cu_seqlens != nullptr) {
    const long long end = max(0, __ldg(p.cu_seqlens + p.B)), row = static_cast<long long>(p.H) * D;
    for (long long i = end * row + threadIdx.x; i < p.total * row; i += C::THREADS) p.dq_accum[i] = 0.f;
  }
  const TileSlot ts = grouped_slot(blockIdx.x, num_m, p.H * p.B, group);
  const int mt = num_m - 1 - ts.t;
  const int h = ts.unit % p.H;
  const int b = ts.unit / p.H;
  const SeqInfo sq = seq_info(p, b);
  if (!seq_ok(p, sq) || mt * BM >= sq.len) return;   // whole CTA, before any shared state
  const int hk = h / (p.H / p.H_kv);
  release_dependents();   // the next kernel's CTAs come as this grid's leave

  const Bars<D> bars{sbase + C::OFF_BAR};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* s_range = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const int row = (warp & 3) * 32 + lane;
  const int qpos = mt * BM + row;
  KeyRange kr = {0, 0};
  if (warp < C::SOFTMAX_WARPS && qpos < sq.len) kr = key_range(p, sh, sq, qpos);
  if (threadIdx.x == C::WARP_TMA * 32) {
    *abort = 0;
    s_range[0] = INT_MAX;
    s_range[1] = 0;
    mbar_init(bars.q_full(), 1);
    for (int s = 0; s < ST; ++s) {
      mbar_init(bars.kv_full(s), 1);
      mbar_init(bars.kv_empty(s), 1);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(bars.full(i), 1);
      mbar_init(bars.free(i), 32 * C::SOFTMAX_WARPS);
    }
    fence_mbar_init();
    // Q and dO do not wait for the ranges.
    mbar_arrive_expect_tx(bars.q_full(), 2 * TILE);
    for (int c = 0; c < D / 64; ++c) {
      tma_load_2d(sbase + C::OFF_Q + c * SPAN, &tm_q, bars.q_full(), h * D + c * 64, sq.start + mt * BM);
      tma_load_2d(sbase + C::OFF_DO + c * SPAN, &tm_do, bars.q_full(), h * D + c * 64, sq.start + mt * BM);
    }
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == C::WARP_MMA) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  __syncthreads();
  if (warp < 4) {
    const int lo = __reduce_min_sync(FULL, kr.lo < kr.hi ? kr.lo : INT_MAX);
    const int hi = __reduce_max_sync(FULL, kr.hi);
    if (lane == 0 && hi > 0) {
      atomicMin(&s_range[0], lo);
      atomicMax(&s_range[1], hi);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (tile_range != nullptr && h == 0 && threadIdx.x == 0)
    tile_range[tile_base(sq, b) + mt] = make_int2(s_range[0], s_range[1]);
  const int t0 = s_range[1] > 0 ? s_range[0] / BN : 0;
  const int n = (s_range[1] + BN - 1) / BN - t0;   // key tiles; 0 when no row sees a key

  if (warp == C::WARP_TMA) {
    // ------------------------------------------------------------ producer ---
    bool ok = true;
    for (int it = 0; it < n && ok; ++it) {
      const int st = it % ST;
      ok = warp_wait(bars.kv_empty(st), ((it / ST) & 1) ^ 1, p.err, abort, W_KVEMPTY);
      if (ok && lane == 0) {
        mbar_arrive_expect_tx(bars.kv_full(st), 2 * TILE);
        for (int c = 0; c < D / 64; ++c) {
          tma_load_2d(sbase + C::OFF_K + st * TILE + c * SPAN, &tm_k, bars.kv_full(st),
                      hk * D + c * 64, sq.start + (t0 + it) * BN);
          tma_load_2d(sbase + C::OFF_V + st * TILE + c * SPAN, &tm_v, bars.kv_full(st),
                      hk * D + c * 64, sq.start + (t0 + it) * BN);
        }
      }
      __syncwarp();
    }
    // Drain: Q and dO have landed and the tensor core's last arrivals come before the
    // CTA's shared memory is released.
    ok = ok && warp_wait(bars.q_full(), 0, p.err, abort, W_Q);
    for (int it = max(0, n - ST); it < n && ok; ++it)
      ok = warp_wait(bars.kv_empty(it % ST), (it / ST) & 1, p.err, abort, W_KVEMPTY);
  } else if (warp == C::WARP_MMA) {
    // ---------------------------------------------------------- MMA issuer ---
    const uint32_t leader = elect_one();
    constexpr uint32_t IDESC = idesc_bf16(BM, BN, false, false);
    const uint64_t q_desc = sdesc_sw128(sbase + C::OFF_Q, 16, 1024);
    const uint64_t g_desc = sdesc_sw128(sbase + C::OFF_DO, 16, 1024);
    const uint64_t k_desc = sdesc_sw128(sbase + C::OFF_K, 16, 1024);
    const uint64_t v_desc = sdesc_sw128(sbase + C::OFF_V, 16, 1024);
    bool ok = n > 0 && warp_wait(bars.q_full(), 0, p.err, abort, W_Q);
    for (int it = 0; it < n && ok; ++it) {
      const int st = it % ST, buf = it % NB;
      ok = warp_wait(bars.kv_full(st), (it / ST) & 1, p.err, abort, W_KVFULL) &&
           warp_wait(bars.free(buf), ((it / NB) & 1) ^ 1, p.err, abort, W_FREE);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t o = (kk >> 2) * SPAN + (kk & 3) * 32;
        mma_ss_if(leader, tmem + buf * 256, sdesc_add(q_desc, o), sdesc_add(k_desc, st * TILE + o),
                  IDESC, kk > 0);
      }
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t o = (kk >> 2) * SPAN + (kk & 3) * 32;
        mma_ss_if(leader, tmem + buf * 256 + BN, sdesc_add(g_desc, o),
                  sdesc_add(v_desc, st * TILE + o), IDESC, kk > 0);
      }
      tc_commit_if(leader, bars.full(buf));
      tc_commit_if(leader, bars.kv_empty(st));
    }
  } else {
    // ------------------------------------------------------------- softmax ---
    const int cgp = warp >> 2;   // column group
    const bool row_ok = qpos < sq.len;
    const uint32_t col = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + cgp * C::COLS;
    const float c2 = p.scale_log2;
    const float slope2 = BIAS ? __ldg(sh.slopes + h) * LOG2E : 0.f;
    // A row that sees nothing has an LSE of -inf; its keys are all masked.
    const float lse = (row_ok && kr.lo < kr.hi) ? __ldg(p.lse + lse_index(p, b, h, sq.start, qpos)) : 0.f;
    const float lse2 = lse == -INFINITY ? 0.f : lse * LOG2E;
    // dQ accumulator rows of this tile, a row per warp and turn.
    for (int r = warp; r < BM && mt * BM + r < sq.len; r += C::SOFTMAX_WARPS) {
      float* a = p.dq_accum + (static_cast<size_t>(sq.start + mt * BM + r) * p.H + h) * D;
      if (4 * lane < D) *reinterpret_cast<float4*>(a + 4 * lane) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    bool ok = true;
    for (int it = 0; it < n && ok; ++it) {
      const int buf = it % NB;
      const int key0 = (t0 + it) * BN + cgp * C::COLS;
      const int lo = kr.lo - key0, hi = kr.hi - key0, dist0 = key0 - qpos;
      const bool whole = __all_sync(FULL, lo <= 0 && hi >= C::COLS &&
                                              (!BIAS || dist0 >= 0 || dist0 + C::COLS <= 1));
      const bool none = !whole && !__any_sync(FULL, lo < C::COLS && hi > 0 && lo < hi);
      ok = warp_wait(bars.full(buf), (it / NB) & 1, p.err, abort, W_FULL);
      if (!ok) break;
      tc_fence_after();
      if (!none) {
#pragma unroll 1
        for (int c = 0; c < C::COLS / 32; ++c) {
          uint32_t s[32], g[32];
          tmem_ld32(col + buf * 256 + 32 * c, s);
          tmem_ld32(col + buf * 256 + BN + 32 * c, g);
          tmem_ld_wait();
          reg_fence(s);
          reg_fence(g);
          const int l = lo - 32 * c, hh = hi - 32 * c, d0 = dist0 + 32 * c;
          int form = 0;
          if (CAP) {
            float ab[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              ab[(i >> 1) & 1] = fmaxf(fmaxf(ab[(i >> 1) & 1], fabsf(__uint_as_float(s[i]))),
                                       fabsf(__uint_as_float(s[i + 1])));
            form = cap_form(cap, fmaxf(ab[0], ab[1]));
          }
          if (whole && form == 0)
            chunk<CAP, BIAS, false, 0>(s, g, l, hh, d0, c2, cap, slope2, lse2, acc);
          else if (!CAP || form == 0)
            chunk<CAP, BIAS, true, 0>(s, g, l, hh, d0, c2, cap, slope2, lse2, acc);
          else if (form == 1)
            chunk<CAP, BIAS, true, 1>(s, g, l, hh, d0, c2, cap, slope2, lse2, acc);
          else
            chunk<CAP, BIAS, true, 2>(s, g, l, hh, d0, c2, cap, slope2, lse2, acc);
        }
      }
      tc_fence_before();
      mbar_arrive(bars.free(buf));
    }
    reinterpret_cast<float*>(smem + C::OFF_SUM)[cgp * BM + row] =
        (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
  }

  tc_fence_before();
  __syncthreads();
  if (warp < 4 && qpos < sq.len) {
    const float* s = reinterpret_cast<const float*>(smem + C::OFF_SUM) + row;
    float d = 0.f;
#pragma unroll
    for (int g = 0; g < C::CG; ++g) d += s[g * BM];
    p.delta[static_cast<size_t>(h) * p.total + sq.start + qpos] = d;
  }
  if (warp == C::WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int D, bool CAP, bool BIAS>
cudaError_t launch(const AttnParams& p, const ShapeArgs& sh, int2* ranges, cudaStream_t stream) {
  using C = Cfg<D>;
  const int num_m = (p.max_seqlen + BM - 1) / BM;
  const long long tiles = static_cast<long long>(num_m) * p.H * p.B;
  if (tiles > INT_MAX) return cudaErrorInvalidConfiguration;
  CUtensorMap tq, tk, tv, tg;
  const unsigned long long cq = static_cast<unsigned long long>(p.H) * D, ck = static_cast<unsigned long long>(p.H_kv) * D;
  if (!make_tmap_bf16_2d(&tq, p.q, p.total, cq, 64, BM) ||
      !make_tmap_bf16_2d(&tg, p.dout, p.total, cq, 64, BM) ||
      !make_tmap_bf16_2d(&tk, p.k, p.total, ck, 64, BN) ||
      !make_tmap_bf16_2d(&tv, p.v, p.total, ck, 64, BN))
    return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem<shaped_delta_kernel<D, CAP, BIAS>>(C::SMEM);
  if (e != cudaSuccess) return e;
  const int group = l2_group(4ll * p.max_seqlen * D, p.H / p.H_kv, p.H * p.B);
  const CapArgs cap = CAP ? cap_args(sh.cap, p.scale) : CapArgs{};
  shaped_delta_kernel<D, CAP, BIAS><<<static_cast<unsigned>(tiles), C::THREADS, C::SMEM, stream>>>(
      tq, tk, tv, tg, p, sh, cap, ranges, num_m, group);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const AttnParams& p, const ShapeArgs& sh, int2* ranges, cudaStream_t stream) {
  const bool cap = sh.cap > 0.f, bias = sh.slopes != nullptr;
  if (cap)
    return bias ? launch<D, true, true>(p, sh, ranges, stream)
                : launch<D, true, false>(p, sh, ranges, stream);
  return bias ? launch<D, false, true>(p, sh, ranges, stream)
              : launch<D, false, false>(p, sh, ranges, stream);
}

}  // namespace sdelta
}  // namespace

cudaError_t launch_shaped_delta(const AttnParams& p, const ShapeArgs& sh, int2* ranges,
                                cudaStream_t stream) {
  return p.D == 64 ? sdelta::launch_d<64>(p, sh, ranges, stream)
                   : sdelta::launch_d<128>(p, sh, ranges, stream);
}

}  // namespace fa
