// Attention backward with shaped scores, every product once per (query tile, key
// tile) pair, bf16 in / fp32 accumulate, on the sm_100a tensor cores.
//
//     t = tanh(scale q.k / cap),  z = cap t - slope |i - j|,  P = exp(z - LSE),
//     dV = P^T dO,  dZ = P (dO V^T - D),  D from shaped_delta.cu,  dX = dZ (1 - t^2),
//     dQ = scale dX K,  dK = scale dX^T Q
// (no cap: z = scale q.k - slope |i - j|, dX = dZ). The plan is that of the
// unshaped fused backward (bwd_fused.cu): one CTA per (sequence, key/value head,
// 128-key tile), K and V resident, the 128-row query tiles of every query head
// of the group streaming past; keys on the TMEM lanes; per step
//     S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dQ_t = dX K, dK += dX^T Q
// with dQ_t added into an fp32 accumulator by TMA tensor reductions; warps 0-7
// form P and dX, 8-11 read dQ_t out, 12 is the TMA producer, 13 issues the
// tensor-core products in the order dV_t, S_{t+1}, dQ_t, dK_t, dP_{t+1}.
//
// What the shape adds:
// - Which query tiles. The kernel that makes D leaves the ranges of each query tile's
//   rows as one, [least begin, largest end); a CTA takes the query tiles from the
//   first to the last whose range meets its keys. A key tile that no query sees
//   gets zeros.
// - Masks. The producer stages, beside a step's LSE and D, each query's visible
//   rows [lo, hi) of the key tile as two bytes (all that shared memory has room
//   for) and whether all are visible; the others' P and dX words are cleared
//   after they are packed.
// - The factor of dP - D. P (1 - t^2) 2^14 waits as fp16 for dP: 11 bits down to
//   P = 4e-9, where bf16 would add a rounding of 2^-9 to that of dX. The 2^14
//   leaves again with the scale of dQ and dK.
// - The cap per 32 scores by the shortest polynomial that their largest allows, or by
//   exponential and reciprocal (score_cap.cuh).
//
// B1 H16/4 N8192 D128 causal, cap 50: 980 us of a step of 1541 us after a rest (1665 back
// to back, under the power cap), 700 TFLOP/s (the unshaped fused backward takes 859 with
// its D); bound by the chain of the warps that form P and dX, which the cap and 1 - t^2
// lengthen, as the unshaped one is by its own. At D = 128 the forms with a cap spill: 24
// bytes of stores and 144 of loads a thread without a bias, 8 and 28 with one; the others
// nothing.
#include <cuda_fp16.h>
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "ex2_fma.cuh"
#include "score_cap.cuh"
#include "shaped.h"

namespace fa {
namespace {

namespace sbwd {
constexpr int BT = 128;        // keys per CTA = query rows per step = TMEM lanes
constexpr int THREADS = 512;
constexpr int N_DS = 256;      // dS warps' threads (warpgroups 0 and 1)
constexpr int WARP_DQ0 = 8;    // dQ warps 8-11 (warpgroup 2): TMEM lane quarters 0-3
constexpr int N_DQ = 128;      // dQ warps' threads
constexpr int WARP_TMA = 12;   // warpgroup 3: producer, MMA warp, two idle warps
constexpr int WARP_MMA = 13;
// Registers per thread (setmaxnreg): the block launches at 128; 2 x 136 + 160 +
// 80 = 4 x 128 on every sub-partition and for the block.
constexpr uint32_t REG_DS = 136;
constexpr uint32_t REG_DQ = 160;
constexpr uint32_t REG_CTRL = 80;
static_assert(2 * REG_DS + REG_DQ + REG_CTRL == 4 * 128, "register split of the block");
constexpr uint32_t TMEM_COLS = 512;
constexpr unsigned FULL = 0xffffffffu;
constexpr uint32_t SPAN = BT * 128;   // 128 rows x 128 bytes: one 128-byte swizzle column block
constexpr float LOG2E = 1.4426950408889634f;
constexpr float UP = 16384.f;         // 2^14: scale of the factor of dP - D, and so of dX
constexpr float DOWN = 1.f / UP;

template <int D>
struct Cfg {
  static_assert(D == 64 || D == 128, "head dim");
  static constexpr uint32_t TILE = BT * D * 2;       // one 128-row bf16 tile of Q, K, V or dO
  static constexpr int QS = 2;                       // Q stages (with LSE, D_i)
  static constexpr int GS = 1;                       // dO stages (dO_{t+1} is read after dV_t)
  static constexpr bool ALIAS = D == 128;            // dQ_t formed over dP
  static constexpr uint32_t TM_S = 0, TM_DP = 128, TM_DV = 256, TM_DK = 256 + D;
  static constexpr uint32_t TM_DQ = ALIAS ? TM_DP : 256 + 2 * D;
  static constexpr uint32_t OFF_K = 0;
  static constexpr uint32_t OFF_V = OFF_K + TILE;
  static constexpr uint32_t OFF_Q = OFF_V + TILE;
  static constexpr uint32_t OFF_DO = OFF_Q + QS * TILE;
  static constexpr uint32_t OFF_DS = OFF_DO + GS * TILE;       // dS^T: 128 keys x 128 queries bf16
  static constexpr uint32_t OFF_STG = OFF_DS + 2 * SPAN;       // dQ staging: 8 KB per dQ warp
  static constexpr uint32_t OFF_LSE = OFF_STG + 8 * 4096;      // float [QS][BT]: -LSE * log2(e)
  static constexpr uint32_t OFF_DLT = OFF_LSE + QS * BT * 4;   // float [QS][BT]: -D_i
  static constexpr uint32_t OFF_VIS = OFF_DLT + QS * BT * 4;   // uint16 [QS][BT]: lo | hi << 8
  static constexpr uint32_t OFF_ALL = OFF_VIS + QS * BT * 2;   // int [QS][2]: halves seen in full
  static constexpr uint32_t OFF_BAR = OFF_ALL + QS * 8;
  // kv_full, q_full[QS], q_empty[QS], do_full[GS], do_empty[GS], s_full,
  // dp_full, p_ready, ds_ready, dq_full, dq_free, dkv_done
  static constexpr int NBAR = 1 + 2 * QS + 2 * GS + 7;
  static constexpr uint32_t OFF_MISC = OFF_BAR + NBAR * 8;
  // No alignment slack: the dynamic shared memory must start on a 1024-byte
  // boundary (128-byte swizzle atoms); the kernel checks and reports.
  static constexpr uint32_t SMEM = OFF_MISC + 16;   // tmem slot, abort, query tiles [i0, i1)
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(TM_DQ + D <= TMEM_COLS, "TMEM budget");
};

template <int D>
struct Bars {
  using C = Cfg<D>;
  uint32_t b;
  __device__ uint32_t kv_full() const { return b; }
  __device__ uint32_t q_full(int s) const { return b + 8u * (1 + s); }
  __device__ uint32_t q_empty(int s) const { return b + 8u * (1 + C::QS + s); }
  __device__ uint32_t do_full(int s) const { return b + 8u * (1 + 2 * C::QS + s); }
  __device__ uint32_t do_empty(int s) const { return b + 8u * (1 + 2 * C::QS + C::GS + s); }
  __device__ uint32_t s_full() const { return b + 8u * (1 + 2 * C::QS + 2 * C::GS); }
  __device__ uint32_t dp_full() const { return b + 8u * (2 + 2 * C::QS + 2 * C::GS); }
  __device__ uint32_t p_ready() const { return b + 8u * (3 + 2 * C::QS + 2 * C::GS); }
  __device__ uint32_t ds_ready() const { return b + 8u * (4 + 2 * C::QS + 2 * C::GS); }
  __device__ uint32_t dq_full() const { return b + 8u * (5 + 2 * C::QS + 2 * C::GS); }
  __device__ uint32_t dq_free() const { return b + 8u * (6 + 2 * C::QS + 2 * C::GS); }
  __device__ uint32_t dkv_done() const { return b + 8u * (7 + 2 * C::QS + 2 * C::GS); }
};

enum : unsigned {
  W_KV = 0xD0100, W_QEMPTY = 0xD0200, W_QFULL = 0xD0300, W_SFULL = 0xD0400, W_PREADY = 0xD0500,
  W_DPFULL = 0xD0600, W_DSREADY = 0xD0700, W_DKV = 0xD0800, W_DOFULL = 0xD0900,
  W_DOEMPTY = 0xD0A00, W_DQFULL = 0xD0B00, W_DQFREE = 0xD0C00, BAD_ALIGN = 0xD0D00
};

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const DevErr& e,
                                          volatile int* abort, unsigned where) {
  const bool ok = mbar_wait(bar, parity, e, abort, where);
  return __all_sync(FULL, ok);
}

template <uint32_t N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <uint32_t N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// One 128-row tile of a token-major tensor (its D / 64 column blocks).
template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                          int head, int row) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c) tma_load_3d(dst + c * SPAN, map, bar, 64 * c, head, row);
}

// Packed-bf16 TMEM column of k-step kk (16 elements) when each 64-wide half
// of a 128-wide operand was written by its own thread into the first 32 of
// its 64 columns: halves start 64 columns apart.
__device__ __forceinline__ uint32_t packed_col(int kk) { return (kk >> 2) * 64 + (kk & 3) * 8; }

__device__ __forceinline__ void store_row_bf16(__nv_bfloat16* dst, const uint32_t (&a)[32],
                                               float scale) {
#pragma unroll
  for (int v4 = 0; v4 < 4; ++v4) {
    uint4 w;
    w.x = pack_bf16x2(__uint_as_float(a[8 * v4 + 0]) * scale, __uint_as_float(a[8 * v4 + 1]) * scale);
    w.y = pack_bf16x2(__uint_as_float(a[8 * v4 + 2]) * scale, __uint_as_float(a[8 * v4 + 3]) * scale);
    w.z = pack_bf16x2(__uint_as_float(a[8 * v4 + 4]) * scale, __uint_as_float(a[8 * v4 + 5]) * scale);
    w.w = pack_bf16x2(__uint_as_float(a[8 * v4 + 6]) * scale, __uint_as_float(a[8 * v4 + 7]) * scale);
    reinterpret_cast<uint4*>(dst)[v4] = w;
  }
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

// Global [y .. y + 31, x .. x + 31] (fp32) += the 32 x 32 box at ``src``
// (128-byte swizzled), by the tensor-memory accelerator; completion is
// tracked per issuing thread in bulk groups.
__device__ __forceinline__ void tma_reduce_add_2d(const CUtensorMap* map, uint32_t src, int x,
                                                  int y) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::
          "l"(reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(src)
      : "memory");
}

__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// This thread's bulk groups have finished reading shared memory.
__device__ __forceinline__ void bulk_wait_read_all() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// This thread's bulk groups have completed.
__device__ __forceinline__ void bulk_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float2 unpack_half2(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// 32 scores of a key row (queries q0 .. q0 + 31 of the step): P as packed bf16
// and F = P (1 - t^2) 2^14 as packed fp16. d0 = first query - key; lse holds
// -LSE log2 e.
template <bool CAP, bool BIAS, int FORM>
__device__ __forceinline__ void probs(const uint32_t (&sr)[32], const float* lse, float c2,
                                      const CapArgs& cap, float slope2, int d0,
                                      uint32_t (&pk)[16], uint32_t* f) {
  // Bias: linear on either side of the diagonal; a chunk on both takes the
  // distance per element.
  const bool right = d0 < 0;
  const float sl = right ? slope2 : -slope2;
  const bool mixed = BIAS && __any_sync(FULL, d0 < 0 && d0 + 31 > 0);
  const float d0f = static_cast<float>(d0);
  const float base = BIAS ? sl * d0f : 0.f;
  const float4* lse4 = reinterpret_cast<const float4*>(lse);
#pragma unroll
  for (int q = 0; q < 32; q += 2) {
    const float4 l4 = lse4[q >> 2];
    float2 add = (q & 2) ? make_float2(l4.z, l4.w) : make_float2(l4.x, l4.y);
    const float2 s = make_float2(__uint_as_float(sr[q]), __uint_as_float(sr[q + 1]));
    if (BIAS) {
      float2 bias;
      if (mixed)
        bias = make_float2(-slope2 * fabsf(d0f + static_cast<float>(q)),
                           -slope2 * fabsf(d0f + static_cast<float>(q + 1)));
      else
        bias = __ffma2_rn(make_float2(sl, sl), make_float2(static_cast<float>(q), static_cast<float>(q + 1)),
                          make_float2(base, base));
      add = __fadd2_rn(add, bias);
    }
    float2 x, g = make_float2(UP, UP);
    if (!CAP) {
      x = __ffma2_rn(s, make_float2(c2, c2), add);
    } else if (FORM < 2) {
      const float2 y = __fmul2_rn(s, cap_poly2<FORM>(cap, s));   // A t
      const float k = -UP * cap.inv_amp2;
      x = __fadd2_rn(y, add);
      g = __ffma2_rn(__fmul2_rn(y, y), make_float2(k, k), g);
    } else {
      const float2 th = make_float2(cap_tanh(cap, s.x), cap_tanh(cap, s.y));
      x = __ffma2_rn(th, make_float2(cap.amp, cap.amp), add);
      g = __ffma2_rn(__fmul2_rn(th, th), make_float2(-UP, -UP), g);
    }
    // Without a cap an eighth of the exponentials run on the FMA pipe: two dS
    // warps share each sub-partition's special-function unit.
    const bool fma_pipe = !CAP && (q % 16) == 0;
    const float p0 = fma_pipe ? ex2_fma(x.x) : ex2_approx(x.x);
    const float p1 = fma_pipe ? ex2_fma(x.y) : ex2_approx(x.y);
    pk[q >> 1] = pack_bf16x2(p0, p1);
    const float2 v = __fmul2_rn(make_float2(p0, p1), g);
    f[q >> 1] = pack_half2(v.x, v.y);
  }
}

// Clears the words of the queries that do not see key row r.
__device__ __forceinline__ void mask_words(const uint16_t* vis, int r, uint32_t (&pk)[16],
                                           uint32_t* f) {
  const uint32_t* v2 = reinterpret_cast<const uint32_t*>(vis);   // two queries a word
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const uint32_t v = v2[q];
    const int lo0 = v & 255u, hi0 = (v >> 8) & 255u, lo1 = (v >> 16) & 255u, hi1 = v >> 24;
    const uint32_t m = ((r >= lo0 && r < hi0) ? 0xffffu : 0u) |
                       ((r >= lo1 && r < hi1) ? 0xffff0000u : 0u);
    pk[q] &= m;
    f[q] &= m;
  }
}

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(THREADS, 1)
    shaped_bwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ CUtensorMap tm_do,
                     const __grid_constant__ CUtensorMap tm_dqa, const AttnParams p,
                     const ShapeArgs sh, const CapArgs cap, const int2* tile_range, int num_j,
                     int group) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if ((sbase & 1023u) != 0) {
    if (threadIdx.x == 0) {
      atomicOr(p.err.word, ERR_BOUNDS);
      atomicExch(p.err.word + 1, BAD_ALIGN);
    }
    wait_for_primary();
    return;
  }

  // Tile order: groups of key/value heads for L2 reuse of Q, dO and the dQ
  // accumulator; inside a group the causal CTAs with the most query tiles
  // (small key tile j) first.
  const TileSlot ts = grouped_slot(blockIdx.x, num_j, p.H_kv * p.B, group);
  const int j = ts.t;
  const int hk = ts.unit % p.H_kv;
  const int b = ts.unit / p.H_kv;
  const SeqInfo sq = seq_info(p, b);
  if (!seq_ok(p, sq) || j * BT >= sq.len) {
    wait_for_primary();
    return;
  }
  const int g = p.H / p.H_kv;
  const int n_q = (sq.len + BT - 1) / BT;

  const Bars<D> bars{sbase + C::OFF_BAR};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  int* s_range = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);

  if (threadIdx.x == 0) {
    *abort = 0;
    s_range[0] = tile_range != nullptr ? INT_MAX : (p.causal ? j : 0);
    s_range[1] = tile_range != nullptr ? 0 : n_q;
    mbar_init(bars.kv_full(), 1);
    for (int s = 0; s < C::QS; ++s) {
      mbar_init(bars.q_full(s), 2);  // Q bytes + the staged LSE / D_i
      mbar_init(bars.q_empty(s), 1);
    }
    for (int s = 0; s < C::GS; ++s) {
      mbar_init(bars.do_full(s), 1);
      mbar_init(bars.do_empty(s), 1);
    }
    mbar_init(bars.s_full(), 1);
    mbar_init(bars.dp_full(), 1);
    mbar_init(bars.p_ready(), N_DS);
    mbar_init(bars.ds_ready(), N_DS);
    mbar_init(bars.dq_full(), 1);
    mbar_init(bars.dq_free(), N_DQ);
    mbar_init(bars.dkv_done(), 1);
    fence_mbar_init();
  }
  wait_for_primary();   // D, the dQ accumulator's zeros, the ranges
  __syncthreads();
  if (tile_range != nullptr) {
    const int2* tr = tile_range + tile_base(sq, b);
    int first = INT_MAX, last = 0;
    for (int i = (p.causal ? j : 0) + threadIdx.x; i < n_q; i += THREADS) {
      const int2 r = tr[i];
      if (r.x < min((j + 1) * BT, sq.len) && r.y > j * BT) {
        first = min(first, i);
        last = i + 1;
      }
    }
    first = __reduce_min_sync(FULL, first);
    last = __reduce_max_sync(FULL, last);
    if (lane == 0 && last > 0) {
      atomicMin(&s_range[0], first);
      atomicMax(&s_range[1], last);
    }
    __syncthreads();
  }
  // Query tiles [i0, i0 + n_qt) of each head.
  const int i0 = s_range[0];
  const int n_qt = s_range[1] > i0 ? s_range[1] - i0 : 0;
  const int n_steps = g * n_qt;
  if (n_steps == 0) {   // no query sees these keys
    const int rows = min(BT, sq.len - j * BT);
    for (int k = threadIdx.x; k < rows * (D / 8); k += THREADS) {
      const size_t off = (static_cast<size_t>(sq.start + j * BT + k / (D / 8)) * p.H_kv + hk) * D +
                         (k % (D / 8)) * 8;
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dk) + off) = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dv) + off) = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  if (warp == WARP_MMA) {
    tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Each warpgroup sets its register count at the head of its own branch,
  // so the compiler fits each branch's code to it.
  if (warp / 4 == WARP_TMA / 4) {
  regs_dec<REG_CTRL>();
  if (warp == WARP_TMA) {
    // ------------------------------------------------------------ producer ---
    float* s_lse = reinterpret_cast<float*>(smem + C::OFF_LSE);
    float* s_dlt = reinterpret_cast<float*>(smem + C::OFF_DLT);
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      tma_prefetch_desc(&tm_do);
      const int row_kv = sq.start + j * BT;
      mbar_arrive_expect_tx(bars.kv_full(), 2 * C::TILE);
      load_tile<D>(sbase + C::OFF_K, &tm_k, bars.kv_full(), hk, row_kv);
      load_tile<D>(sbase + C::OFF_V, &tm_v, bars.kv_full(), hk, row_kv);
    }
    // LSE and D_i of step t (four query rows per lane), fetched one step
    // ahead into registers so the global loads overlap the wait for a stage.
    uint16_t* s_vis = reinterpret_cast<uint16_t*>(smem + C::OFF_VIS);
    int* s_all = reinterpret_cast<int*>(smem + C::OFF_ALL);
    float pl[BT / 32], pd[BT / 32];
    int pv[BT / 32];   // visible rows of the key tile: lo | hi << 8
    auto fetch = [&](int t) {
      const int h = hk * g + t / n_qt;
      const int qbase = (i0 + t % n_qt) * BT;
#pragma unroll
      for (int k = 0; k < BT / 32; ++k) {
        const int qpos = qbase + lane + 32 * k;
        const bool qv = qpos < sq.len;
        pl[k] = qv ? __ldg(p.lse + lse_index(p, b, h, sq.start, qpos)) : 0.f;
        pd[k] = qv ? p.delta[static_cast<size_t>(h) * p.total + sq.start + qpos] : 0.f;
        KeyRange kr = {0, 0};
        if (qv) kr = key_range(p, sh, sq, qpos);
        const int lo = min(max(kr.lo - j * BT, 0), BT), hi = min(max(kr.hi - j * BT, 0), BT);
        pv[k] = lo | (hi << 8);
      }
    };
    if (n_steps > 0) fetch(0);
    for (int t = 0; t < n_steps; ++t) {
      const int st = t % C::QS;
      const int gt = t % C::GS;
      const int h = hk * g + t / n_qt;
      const int row_q = sq.start + (i0 + t % n_qt) * BT;
      if (!warp_wait(bars.q_empty(st), ((t / C::QS) & 1) ^ 1, p.err, abort, W_QEMPTY)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(bars.q_full(st), C::TILE);
        load_tile<D>(sbase + C::OFF_Q + st * C::TILE, &tm_q, bars.q_full(st), h, row_q);
      }
#pragma unroll
      for (int k = 0; k < BT / 32; ++k) {
        // Negated, so the dS warps add them in packed fp32 pairs.
        s_lse[st * BT + lane + 32 * k] = -(pl[k] * LOG2E);
        s_dlt[st * BT + lane + 32 * k] = -pd[k];
        s_vis[st * BT + lane + 32 * k] = static_cast<uint16_t>(pv[k]);
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const bool all = __all_sync(FULL, pv[2 * hf] == (BT << 8) && pv[2 * hf + 1] == (BT << 8));
        if (lane == 0) s_all[st * 2 + hf] = all;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bars.q_full(st));
      if (!warp_wait(bars.do_empty(gt), ((t / C::GS) & 1) ^ 1, p.err, abort, W_DOEMPTY)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(bars.do_full(gt), C::TILE);
        load_tile<D>(sbase + C::OFF_DO + gt * C::TILE, &tm_do, bars.do_full(gt), h, row_q);
      }
      if (t + 1 < n_steps) fetch(t + 1);
    }
    // Drain: the tensor core's last arrivals on the empty barriers land
    // before the CTA's shared memory is released.
    for (int t = max(0, n_steps - C::QS); t < n_steps && !*abort; ++t)
      if (!warp_wait(bars.q_empty(t % C::QS), (t / C::QS) & 1, p.err, abort, W_QEMPTY)) break;
    for (int t = max(0, n_steps - C::GS); t < n_steps && !*abort; ++t)
      if (!warp_wait(bars.do_empty(t % C::GS), (t / C::GS) & 1, p.err, abort, W_DOEMPTY)) break;
  } else if (warp == WARP_MMA) {
    // ---------------------------------------------------------- MMA issuer ---
    // The whole warp runs the loop (waits and operands stay warp-uniform);
    // one elected lane issues the tensor-core instructions and commits.
    const uint32_t leader = elect_one();
    constexpr uint32_t ID_SDP = idesc_bf16(BT, BT, false, false);  // S^T, dP^T
    constexpr uint32_t ID_KV = idesc_bf16(BT, D, false, true);     // dV, dK (A from TMEM)
    constexpr uint32_t ID_DQ = idesc_bf16(BT, D, true, true);      // dQ_t = dS K
    const uint64_t k_kmaj = sdesc_sw128(sbase + C::OFF_K, 16, 1024);
    const uint64_t v_kmaj = sdesc_sw128(sbase + C::OFF_V, 16, 1024);
    const uint64_t q_kmaj = sdesc_sw128(sbase + C::OFF_Q, 16, 1024);
    const uint64_t g_kmaj = sdesc_sw128(sbase + C::OFF_DO, 16, 1024);
    const uint64_t q_mn = sdesc_sw128(sbase + C::OFF_Q, SPAN, 1024);
    const uint64_t g_mn = sdesc_sw128(sbase + C::OFF_DO, SPAN, 1024);
    const uint64_t k_mn = sdesc_sw128(sbase + C::OFF_K, SPAN, 1024);
    // dS as the A operand of dQ_t: queries (M) run along the rows of the dS^T
    // tile, in two 64-query column blocks one span apart; keys (K) down them.
    const uint64_t ds_mn = sdesc_sw128(sbase + C::OFF_DS, SPAN, 1024);
    // dS^T as the A operand of dK: keys (M) down the rows, queries (K) along
    // them, K-major like the Q and K tiles.
    const uint64_t ds_kmaj = sdesc_sw128(sbase + C::OFF_DS, 16, 1024);
    auto issue_s = [&](int st) {     // S^T = K Q^T, K-dim = D
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t o = (kk >> 2) * SPAN + (kk & 3) * 32;
        mma_ss_if(leader, tmem + C::TM_S, sdesc_add(k_kmaj, o),
                  sdesc_add(q_kmaj, st * C::TILE + o), ID_SDP, kk > 0);
      }
      tc_commit_if(leader, bars.s_full());
    };
    auto issue_dp = [&](int gt) {    // dP^T = V dO^T, K-dim = D
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t o = (kk >> 2) * SPAN + (kk & 3) * 32;
        mma_ss_if(leader, tmem + C::TM_DP, sdesc_add(v_kmaj, o),
                  sdesc_add(g_kmaj, gt * C::TILE + o), ID_SDP, kk > 0);
      }
      tc_commit_if(leader, bars.dp_full());
    };
    bool ok = warp_wait(bars.kv_full(), 0, p.err, abort, W_KV);
    if (ok && n_steps > 0) {
      ok = warp_wait(bars.q_full(0), 0, p.err, abort, W_QFULL);
      if (ok) {
        tc_fence_after();
        issue_s(0);
      }
      ok = ok && warp_wait(bars.do_full(0), 0, p.err, abort, W_DOFULL);
      if (ok) {
        tc_fence_after();
        issue_dp(0);
      }
    }
    for (int t = 0; ok && t < n_steps; ++t) {
      const int st = t % C::QS;
      const int gt = t % C::GS;
      const bool more = t + 1 < n_steps;
      // dV += P^T_t dO_t (K-dim = 128 queries of the step).
      if (!(ok = warp_wait(bars.p_ready(), t & 1, p.err, abort, W_PREADY))) break;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < BT / 16; ++kk)
        mma_ts_if(leader, tmem + C::TM_DV, tmem + C::TM_S + packed_col(kk),
                  sdesc_add(g_mn, gt * C::TILE + kk * 2048), ID_KV, (t > 0 || kk > 0) ? 1u : 0u);
      tc_commit_if(leader, bars.do_empty(gt));
      // S^T_{t+1}: overwrites P^T_t, so it follows dV_t in the tensor pipe.
      if (more) {
        if (!(ok = warp_wait(bars.q_full((t + 1) % C::QS), ((t + 1) / C::QS) & 1, p.err, abort,
                             W_QFULL)))
          break;
        tc_fence_after();
        issue_s((t + 1) % C::QS);
      }
      // dQ_t = dS_t K (K-dim = 128 keys), then dK += dS^T_t Q_t (K-dim = 128
      // queries). Both read dS from the shared dS^T tile (MN-major for dQ,
      // K-major for dK), so dQ_t - whose read-out gates dP_{t+1} - goes first.
      if (!(ok = warp_wait(bars.ds_ready(), t & 1, p.err, abort, W_DSREADY))) break;
      tc_fence_after();
      if (!C::ALIAS && t > 0) {
        // dQ_{t-1} must have been read out of its columns.
        if (!(ok = warp_wait(bars.dq_free(), (t - 1) & 1, p.err, abort, W_DQFREE))) break;
        tc_fence_after();
      }
#pragma unroll
      for (int kk = 0; kk < BT / 16; ++kk)   // K-dim = 128 keys in steps of 16
        mma_ss_if(leader, tmem + C::TM_DQ, sdesc_add(ds_mn, kk * 2048), sdesc_add(k_mn, kk * 2048),
                  ID_DQ, kk > 0);
      tc_commit_if(leader, bars.dq_full());
#pragma unroll
      for (int kk = 0; kk < BT / 16; ++kk) {
        const uint32_t o = (kk >> 2) * SPAN + (kk & 3) * 32;   // queries 16 kk .. 16 kk + 15
        mma_ss_if(leader, tmem + C::TM_DK, sdesc_add(ds_kmaj, o),
                  sdesc_add(q_mn, st * C::TILE + kk * 2048), ID_KV, (t > 0 || kk > 0) ? 1u : 0u);
      }
      tc_commit_if(leader, bars.q_empty(st));
      if (more) {
        if (C::ALIAS) {
          // dP_{t+1} overwrites dQ_t: wait until it has been read out.
          if (!(ok = warp_wait(bars.dq_free(), t & 1, p.err, abort, W_DQFREE))) break;
        }
        if (!(ok = warp_wait(bars.do_full((t + 1) % C::GS), ((t + 1) / C::GS) & 1, p.err, abort,
                             W_DOFULL)))
          break;
        tc_fence_after();
        issue_dp((t + 1) % C::GS);
      }
    }
    tc_commit_if(leader, bars.dkv_done());
  }   // warps 14 and 15: no role
  } else if (warp / 4 == WARP_DQ0 / 4) {
    regs_inc<REG_DQ>();
    // ------------------------------------------------------------ dQ warps ---
    // Thread = query row (warp & 3) * 32 + lane of the step's tile. The
    // whole row block of dQ_t (D / 32 boxes of 32 x 32 fp32) comes out of
    // TMEM at once and dq_free goes out; then, two boxes a round, the boxes
    // are staged 128-byte swizzled in this warp's 8 KB of the staging area
    // and one lane adds them into dQacc with TMA tensor reductions, which run
    // on their own.
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t stg = sbase + C::OFF_STG + (warp - WARP_DQ0) * 8192u;
    for (int t = 0; t < n_steps; ++t) {
      if (!warp_wait(bars.dq_full(), t & 1, p.err, abort, W_DQFULL)) break;
      tc_fence_after();
      uint32_t a[D / 32][32];
#pragma unroll
      for (int c = 0; c < D / 32; ++c) tmem_ld32(tmem + lane_off + C::TM_DQ + 32 * c, a[c]);
      tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < D / 32; ++c) reg_fence(a[c]);
      tc_fence_before();
      mbar_arrive(bars.dq_free());
      const int h = hk * g + t / n_qt;
      const int row0 = sq.start + (i0 + t % n_qt) * BT + (warp & 3) * 32;
      // Rows past the sequence's end hold exact zeros (their dS rows are
      // zero), so adding them to the next sequence's rows changes nothing;
      // rows past the tensor are clipped by the copy. A box wholly past the
      // sequence is not added at all.
      const bool add = row0 < sq.start + sq.len;
#pragma unroll
      for (int rd = 0; rd < D / 64; ++rd) {
        // The slots' previous boxes must have been read.
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int m = 0; m < 8; ++m)
            st_shared_v4(stg + c * 4096u + lane * 128 + ((m ^ (lane & 7)) << 4),
                         a[2 * rd + c][4 * m], a[2 * rd + c][4 * m + 1], a[2 * rd + c][4 * m + 2],
                         a[2 * rd + c][4 * m + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && add &&
            FA_CHECK(p, row0 >= 0 && row0 < p.total && h < p.H, 0xDB0402u)) {
          tma_reduce_add_2d(&tm_dqa, stg, h * D + 64 * rd, row0);
          tma_reduce_add_2d(&tm_dqa, stg + 4096u, h * D + 64 * rd + 32, row0);
        }
        if (lane == 0) bulk_commit();
      }
    }
    // The reductions read this CTA's shared memory: all must be done before exit.
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  } else {
    regs_inc<REG_DS>();
    // ------------------------------------------------------------ dS warps ---
    // Key-side work: thread = key row r (TMEM lane); warps w and w+4 take the
    // query columns [64 hf, 64 hf + 64) of the step.
    const int r = threadIdx.x & (BT - 1);
    const int hf = threadIdx.x >> 7;
    const int kpos = j * BT + r;
    const bool key_ok = kpos < sq.len;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float* s_lse = reinterpret_cast<const float*>(smem + C::OFF_LSE);
    const float* s_dlt = reinterpret_cast<const float*>(smem + C::OFF_DLT);
    const uint16_t* s_vis = reinterpret_cast<const uint16_t*>(smem + C::OFF_VIS);
    const int* s_all = reinterpret_cast<const int*>(smem + C::OFF_ALL);
    const float c2 = p.scale_log2;
    // This thread's 128-byte row block of the dS^T tile (keys = rows, 64
    // queries per 128-byte block, 16-byte chunks XOR-swizzled by row & 7).
    uint8_t* ds_row = smem + C::OFF_DS + hf * SPAN + r * 128;

    bool ok = true;
    for (int t = 0; t < n_steps && ok; ++t) {
      const int st = t % C::QS;
      const int qbase = (i0 + t % n_qt) * BT + 64 * hf;   // first query of this half
      const float* lse_t = s_lse + st * BT + 64 * hf;
      const float* dlt_t = s_dlt + st * BT + 64 * hf;
      const uint16_t* vis_t = s_vis + st * BT + 64 * hf;
      if (!(ok = warp_wait(bars.q_full(st), (t / C::QS) & 1, p.err, abort, W_QFULL))) break;
      if (!(ok = warp_wait(bars.s_full(), t & 1, p.err, abort, W_SFULL))) break;
      tc_fence_after();
      const bool full = s_all[st * 2 + hf] != 0;
      const float slope2 = BIAS ? __ldg(sh.slopes + hk * g + t / n_qt) * LOG2E : 0.f;
      uint32_t f[32];   // F, packed fp16
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t sr[32], pk[16];
        tmem_ld32(tmem + lane_off + C::TM_S + 64 * hf + 32 * c, sr);
        tmem_ld_wait();
        reg_fence(sr);
        int form = 0;
        if (CAP) {
          float ab[2] = {0.f, 0.f};
#pragma unroll
          for (int q = 0; q < 32; q += 2)
            ab[(q >> 1) & 1] = fmaxf(fmaxf(ab[(q >> 1) & 1], fabsf(__uint_as_float(sr[q]))),
                                     fabsf(__uint_as_float(sr[q + 1])));
          form = cap_form(cap, fmaxf(ab[0], ab[1]));
        }
        const int d0 = qbase + 32 * c - kpos;
        if (!CAP || form == 0)
          probs<CAP, BIAS, 0>(sr, lse_t + 32 * c, c2, cap, slope2, d0, pk, f + 16 * c);
        else if (form == 1)
          probs<CAP, BIAS, 1>(sr, lse_t + 32 * c, c2, cap, slope2, d0, pk, f + 16 * c);
        else
          probs<CAP, BIAS, 2>(sr, lse_t + 32 * c, c2, cap, slope2, d0, pk, f + 16 * c);
        if (!full) mask_words(vis_t + 32 * c, r, pk, f + 16 * c);
        // P^T over the first 32 of this half's own 64 S^T columns.
        tmem_st16(tmem + lane_off + C::TM_S + 64 * hf + 16 * c, pk);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bars.p_ready());


      if (!(ok = warp_wait(bars.dp_full(), t & 1, p.err, abort, W_DPFULL))) break;
      tc_fence_after();
      uint32_t dsk[32];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t dr[32];
        tmem_ld32(tmem + lane_off + C::TM_DP + 64 * hf + 32 * c, dr);
        tmem_ld_wait();
        reg_fence(dr);
        const float4* dlt4 = reinterpret_cast<const float4*>(dlt_t + 32 * c);
#pragma unroll
        for (int q = 0; q < 32; q += 2) {
          const float4 d4 = dlt4[q >> 2];
          const float da = (q & 2) ? d4.z : d4.x;
          const float db = (q & 2) ? d4.w : d4.y;
          // dX 2^14 = F (dP - D) on packed pairs (da, db hold -D).
          const float2 v = __fmul2_rn(
              unpack_half2(f[16 * c + (q >> 1)]),
              __fadd2_rn(make_float2(__uint_as_float(dr[q]), __uint_as_float(dr[q + 1])),
                         make_float2(da, db)));
          dsk[16 * c + (q >> 1)] = pack_bf16x2(v.x, v.y);
        }
      }
      // dS^T into the shared dS^T tile: the A operand of dQ (read MN-major)
      // and of dK (read K-major). dP_t completing means dQ_{t-1} and dK_{t-1}
      // (issued before it) have read the tile.
#pragma unroll
      for (int m = 0; m < 8; ++m)
        *reinterpret_cast<uint4*>(ds_row + ((m ^ (r & 7)) << 4)) =
            make_uint4(dsk[4 * m + 0], dsk[4 * m + 1], dsk[4 * m + 2], dsk[4 * m + 3]);
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(bars.ds_ready());
    }
    // --------------------------------------------------- dK / dV epilogue ---
    if (ok && warp_wait(bars.dkv_done(), 0, p.err, abort, W_DKV)) {
      tc_fence_after();
      const size_t off = (static_cast<size_t>(sq.start + kpos) * p.H_kv + hk) * D;
#pragma unroll
      for (int cc = 0; cc < D / 64; ++cc) {
        const int c = (D / 64) * hf + cc;   // 32-column block of the head dim
        uint32_t a[32], v[32];
        tmem_ld32(tmem + lane_off + C::TM_DK + 32 * c, a);
        tmem_ld32(tmem + lane_off + C::TM_DV + 32 * c, v);
        tmem_ld_wait();
        reg_fence(a);
        reg_fence(v);
        if (key_ok && FA_CHECK(p, sq.start + kpos < p.total && hk < p.H_kv, 0xDB0401u)) {
          store_row_bf16(static_cast<__nv_bfloat16*>(p.dk) + off + 32 * c, a, p.scale * DOWN);
          store_row_bf16(static_cast<__nv_bfloat16*>(p.dv) + off + 32 * c, v, 1.f);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

template <int D, bool CAP, bool BIAS>
cudaError_t launch(const AttnParams& p, const ShapeArgs& sh, const int2* tiles, cudaStream_t stream) {
  using C = Cfg<D>;
  const int num_t = (p.max_seqlen + BT - 1) / BT;
  const long long ctas = static_cast<long long>(num_t) * p.H_kv * p.B;
  if (ctas > INT_MAX) return cudaErrorInvalidConfiguration;
  CUtensorMap tq, tk, tv, tg, ta;
  if (!make_tmap_bf16_3d(&tq, p.q, p.total, p.H, D, 1, BT) ||
      !make_tmap_bf16_3d(&tk, p.k, p.total, p.H_kv, D, 1, BT) ||
      !make_tmap_bf16_3d(&tv, p.v, p.total, p.H_kv, D, 1, BT) ||
      !make_tmap_bf16_3d(&tg, p.dout, p.total, p.H, D, 1, BT) ||
      !make_tmap_f32_2d(&ta, p.dq_accum, p.total, static_cast<unsigned long long>(p.H) * D, 32, 32))
    return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem<shaped_bwd_kernel<D, CAP, BIAS>>(C::SMEM);
  if (e != cudaSuccess) return e;
  // A group's streams: Q and dO (bf16) plus the dQ accumulator (fp32) of its
  // g query heads.
  const int group = l2_group(8ll * p.max_seqlen * D * (p.H / p.H_kv), 1, p.H_kv * p.B);
  const CapArgs cap = CAP ? cap_args(sh.cap, p.scale) : CapArgs{};
  // Launched while the kernel that makes D still runs; it waits for it before it reads.
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, shaped_bwd_kernel<D, CAP, BIAS>, tq, tk, tv, tg, ta, p, sh, cap,
                            tiles, num_t, group);
}

template <int D>
cudaError_t launch_d(const AttnParams& p, const ShapeArgs& sh, const int2* tiles, cudaStream_t stream) {
  const bool cap = sh.cap > 0.f, bias = sh.slopes != nullptr;
  if (cap)
    return bias ? launch<D, true, true>(p, sh, tiles, stream)
                : launch<D, true, false>(p, sh, tiles, stream);
  return bias ? launch<D, false, true>(p, sh, tiles, stream)
              : launch<D, false, false>(p, sh, tiles, stream);
}

}  // namespace sbwd
}  // namespace

size_t shaped_bwd_tiles_bytes(long long total, int B) {
  return (static_cast<size_t>(total) / sbwd::BT + B + 1) * sizeof(int2);
}

cudaError_t launch_shaped_bwd(const AttnParams& p, const ShapeArgs& sh, void* tiles,
                              cudaStream_t stream) {
  const bool ranged = sh.key_begin != nullptr || sh.key_end != nullptr;
  int2* t = ranged ? static_cast<int2*>(tiles) : nullptr;
  cudaError_t e = launch_shaped_delta(p, sh, t, stream);
  if (e != cudaSuccess) return e;
  e = p.D == 64 ? sbwd::launch_d<64>(p, sh, t, stream) : sbwd::launch_d<128>(p, sh, t, stream);
  if (e != cudaSuccess) return e;
  AttnParams c = p;
  c.scale = p.scale * sbwd::DOWN;   // the accumulator holds 2^14 dX K
  return launch_dq_convert(c, stream);
}

}  // namespace fa
