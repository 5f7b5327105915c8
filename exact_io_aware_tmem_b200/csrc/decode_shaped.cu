// Decode with shaped scores over a contiguous or paged cache, D = 64 or 128, at
// most 64 query rows per kv head; and the attention weight each slot receives.
//
// The plan is that of the balanced decode (decode_t.cu): the (sequence, kv head,
// 128-key tile) units are cut into one contiguous range of equal size per SM;
// keys on the TMEM lanes,
//     S^T = K_j Q^T  (M = 128 keys, N = NQ query columns, K = D)
//     O^T += V_j^T P^T  (M = 128, N = NQ, K = 128 keys);
// segments cut by a range boundary leave partials that a second kernel joins.
//
// What the shape adds. A thread owns one key and NH of the rows, so the cap (tanh by
// a polynomial, or exponential and reciprocal), the bias (slope x distance of two positions) and the
// window are a few instructions on a few scores. What a tile costs is then the latency
// of the chain from its scores to its P: four threads share a key, in groups of 128
// threads that own their rows and never wait for one another (16 sequences, 32 rows a kv
// head, 4096 keys each: 98 us with two threads a key and one barrier for all, 89 so; 64
// rows, 4096 keys, cap and bias: 227 and 145; D = 64, 16 rows: 62 and 58). A segment's
// tiles are walked from its end: with a bias the newest keys hold the maximum, and the
// reference of the softmax then hardly moves (each move is two barriers and a pass over
// O^T). With a window the units are the tiles from the first one a query sees: the
// others are never read.
//
// The weights. A slot's weight needs the row's final LSE, which no CTA has while
// it walks. Each walked tile's shaped scores (fp32, R x 128) go to the workspace, 4 R
// bytes a key beside the 4 D bytes of K and V (3 % at R = 4, D = 128; 25 % at R = 32),
// and the second kernel forms sum_r 2^(z_r - LSE_r) per slot from them: no second pass
// over K, no atomics, a fixed order. K and V are read once, so their tiles are loaded to
// leave L2 first, and the scores are still there when they are read back (the case above
// 89 -> 84 us; 16 sequences of up to 32768 keys in pages of 64, four rows, 205 -> 200 us,
// 1.14 GB: 5.7 TB/s).
//
// D = 64: the products keep M = 128 for V^T; its second 64 rows are whatever
// lies behind the tile in shared memory (the next V stage or the first K stage,
// which is why V comes first), and the O^T rows they give are never read.
#include <limits.h>
#include <math.h>

#include "decode_t.h"
#include "score_cap.cuh"
#include "shaped.h"

namespace fa {
namespace {
namespace sdec {

constexpr int BN = 128;                   // keys per tile
constexpr int STAGES = 3;
constexpr uint32_t KV_SPAN = BN * 128;    // one column block of a K / V tile
constexpr float LOG2E = 1.4426950408889634f;
constexpr float RESCALE_LOG2 = 8.f;
constexpr unsigned FULL = 0xffffffffu;

// NQ: query columns of the products (R <= NQ).
template <int D, int NQ>
struct Cfg {
  static_assert(D == 64 || D == 128, "head dim");
  static constexpr int CHUNKS = D / 64;             // 128-byte column blocks of a bf16 row
  static constexpr uint32_t TILE = BN * D * 2;      // K / V tile
  static_assert(NQ == 16 || NQ == 32 || NQ == 64, "query columns");
  // Threads a key, each with NH of the query columns.
  static constexpr int SPLIT = 4;
  static constexpr int NH = NQ / SPLIT;
  static constexpr int SOFTMAX_THREADS = SPLIT * BN;
  static constexpr int THREADS = SOFTMAX_THREADS + 64;
  static constexpr int WARP_TMA = SOFTMAX_THREADS / 32;
  static constexpr int WARP_MMA = WARP_TMA + 1;
  static constexpr int QBUF = NQ <= 32 ? 2 : 1;     // Q buffers
  static constexpr int PBUF = NQ <= 32 ? 2 : 1;     // P buffers
  static constexpr uint32_t SPAN = NQ * 128;        // one column block of a Q or P tile
  static constexpr uint32_t Q_BYTES = CHUNKS * SPAN;   // NQ rows x D
  static constexpr uint32_t P_BYTES = 2 * SPAN;        // NQ rows x 128 keys
  static constexpr uint32_t OFF_V = 0;
  static constexpr uint32_t OFF_K = STAGES * TILE;
  static constexpr uint32_t OFF_Q = 2 * STAGES * TILE;
  static constexpr uint32_t OFF_P = OFF_Q + QBUF * Q_BYTES;  // P: NQ rows x 128 keys, K-major
  static constexpr uint32_t OFF_MREF = OFF_P + PBUF * P_BYTES;  // float [NQ]: reference max
  static constexpr uint32_t OFF_ALPHA = OFF_MREF + NQ * 4;    // float [NQ]: its last move
  static constexpr uint32_t OFF_RED = OFF_ALPHA + NQ * 4;     // float [4][NQ]: per-warp max / sum
  static constexpr uint32_t OFF_SLOPE = OFF_RED + 4 * NQ * 4; // float2 [NQ]: -slope log2 e of a row,
                                                              // its position - row 0's
  static constexpr uint32_t OFF_QPOS = OFF_SLOPE + NQ * 8;    // int [NQ]: the same position
  static constexpr uint32_t OFF_ROWS = OFF_QPOS + NQ * 4;  // int [8][8]: paged rows per tile
  static constexpr uint32_t OFF_BAR = OFF_ROWS + 8 * 8 * 4;
  // k_full[S], k_empty[S], v_full[S], v_empty[S], q_full[QBUF], q_empty[QBUF],
  // s_full[2], s_free[2], p_ready[PBUF], pv_done[PBUF], v_land
  static constexpr int NBAR = 4 * STAGES + 2 * QBUF + 4 + 2 * PBUF + 1;
  // tmem slot, abort, first tile (b, hk, t), u0, u1
  static constexpr uint32_t OFF_MISC = OFF_BAR + NBAR * 8;
  // No alignment slack: the dynamic shared memory must start on a 1024-byte
  // boundary (128-byte swizzle atoms); the kernel checks and reports.
  static constexpr uint32_t SMEM = OFF_MISC + 48;
  static_assert(SMEM <= 232448, "shared memory budget");
  static constexpr uint32_t TMEM_COLS = NQ == 16 ? 64 : NQ == 32 ? 128 : 256;
  static constexpr uint32_t TM_S = 0;
  static constexpr uint32_t TM_O = 2 * NQ;
};

template <int D, int NQ>
struct Bars {
  using C = Cfg<D, NQ>;
  uint32_t b;
  __device__ uint32_t k_full(int s) const { return b + 8u * s; }
  __device__ uint32_t k_empty(int s) const { return b + 8u * (STAGES + s); }
  __device__ uint32_t v_full(int s) const { return b + 8u * (2 * STAGES + s); }
  __device__ uint32_t v_empty(int s) const { return b + 8u * (3 * STAGES + s); }
  __device__ uint32_t q_full(int i) const { return b + 8u * (4 * STAGES + i); }
  __device__ uint32_t q_empty(int i) const { return b + 8u * (4 * STAGES + C::QBUF + i); }
  __device__ uint32_t s_full(int i) const { return b + 8u * (4 * STAGES + 2 * C::QBUF + i); }
  __device__ uint32_t s_free(int i) const { return b + 8u * (4 * STAGES + 2 * C::QBUF + 2 + i); }
  __device__ uint32_t p_ready(int i) const { return b + 8u * (4 * STAGES + 2 * C::QBUF + 4 + i); }
  __device__ uint32_t pv_done(int i) const {
    return b + 8u * (4 * STAGES + 2 * C::QBUF + 4 + C::PBUF + i);
  }
  __device__ uint32_t v_land() const {
    return b + 8u * (4 * STAGES + 2 * C::QBUF + 4 + 2 * C::PBUF);
  }
};

// Codes recorded in the device error word.
enum : unsigned {
  W_QFULL = 0xE0100, W_QEMPTY = 0xE0200, W_KEMPTY = 0xE0300, W_VEMPTY = 0xE0400,
  W_KFULL = 0xE0500, W_VFULL = 0xE0600, W_SFULL = 0xE0700, W_SFREE = 0xE0800,
  W_PREADY = 0xE0900, W_PVDONE = 0xE0A00, W_VLAND = 0xE0B00, BAD_CACHE_LEN = 0xE0F01,
  BAD_PAGE = 0xE0F02, BAD_MERGE = 0xE0F03, BAD_ALIGN = 0xE0F04
};

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const DevErr& e,
                                          volatile int* abort, unsigned where) {
  const bool ok = mbar_wait(bar, parity, e, abort, where);
  return __all_sync(FULL, ok);
}

// For tiles of K and V, which are read once: they leave L2 before the scores.
__device__ __forceinline__ uint64_t read_once_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

__device__ __forceinline__ void tma_load_once(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                              int x, int y, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "l"(pol)
      : "memory");
}

// Non-blocking test of a phase, agreed by the whole warp.
__device__ __forceinline__ bool warp_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return __all_sync(FULL, done != 0);
}

// The four warps of a row group (128 threads: the keys of a tile) meet at named
// barrier `bar`; the groups share no row and do not wait for one another. The AND form
// also tells every thread whether all of them are still on track, so that a failed
// wait in one warp ends the loop of all four at the same barrier; the OR form
// gathers a vote.
__device__ __forceinline__ void group_sync(int bar) {
  asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool group_sync_and(int bar, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(ok ? 1u : 0u), "r"(bar)
      : "memory");
  return all != 0;
}

__device__ __forceinline__ bool group_sync_or(int bar, bool v) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(v ? 1u : 0u), "r"(bar)
      : "memory");
  return any != 0;
}

// 32 lanes x 16 consecutive 32-bit TMEM columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st16p(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}

__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

// N (4, 8, 16) consecutive columns of this thread's TMEM lane, valid on
// return.
template <int N>
__device__ __forceinline__ void tmem_row_ld(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 4) {
    tmem_ld4(taddr, r);
  } else if constexpr (N == 8) {
    tmem_ld8(taddr, r);
  } else {
#pragma unroll
    for (int c = 0; c < N / 16; ++c) tmem_ld16(taddr + 16 * c, r + 16 * c);
  }
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

template <int N>
__device__ __forceinline__ void tmem_row_st(uint32_t taddr, const uint32_t (&r)[N]) {
  if constexpr (N == 4) {
    tmem_st4(taddr, r);
  } else if constexpr (N == 8) {
    tmem_st8(taddr, r);
  } else {
#pragma unroll
    for (int c = 0; c < N / 16; ++c) tmem_st16p(taddr + 16 * c, r + 16 * c);
  }
  tmem_st_wait();
}

// What the walk over the tiles needs of the call.
struct Lens {
  const int* lens;
  int B, max_len;
  int reach;   // slots before the last token that some query may see (window), or INT_MAX
  int tiles;   // the most tiles of a sequence that are walked
};

// First slot some query of the sequence may see. Positions of a cache that lost
// slots are further apart than its slots, so the window in slots is a bound.
__device__ __forceinline__ int first_slot(const Lens& s, int len) { return max(0, len - s.reach); }

// Tiles [first, end) of sequence b; a length outside [0, max_len] counts as no
// key (the start scan reports it).
__device__ __forceinline__ int seq_tiles(const Lens& s, int b, int& first, int& len) {
  const int l = __ldg(s.lens + b);
  len = (l >= 0 && l <= s.max_len) ? l : 0;
  first = first_slot(s, len) / BN;
  return (len + BN - 1) / BN;
}

// Position of a role in the CTA's range of units: key tile t of kv head hk of
// sequence b, unit u. Every role walks the same sequence of tiles.
struct Walk {
  int b, t;
  int f, n, len;            // tiles [f, n) and keys of sequence b, walked from the last
  long long u, u0, u1;      // current unit, the CTA's range [u0, u1)
  __device__ bool done() const { return u >= u1; }
  // First / last tile of its piece (the part of a segment inside the range).
  __device__ bool first() const { return t + 1 == n || u == u0; }
  __device__ bool last() const { return t == f || u + 1 == u1; }
  __device__ bool tail() const { return t + 1 == n; }
  __device__ void next(const Lens& s) {
    ++u;
    --t;
    if (u >= u1 || t >= f) return;
    do {
      if (++b >= s.B) {
        u = u1;
        return;
      }
      n = seq_tiles(s, b, f, len);
    } while (n == 0);
    t = n - 1;
  }
  // To the first tile of the next piece.
  __device__ void next_piece(const Lens& s) {
    const long long step = (t - f + 1 < u1 - u) ? static_cast<long long>(t - f + 1) : u1 - u;
    u += step - 1;
    t -= static_cast<int>(step - 1);
    next(s);
  }
};

template <int D, int NQ>
__global__ void __launch_bounds__((Cfg<D, NQ>::THREADS), 1)
    decode_shaped_kernel(const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const AttnParams p,
                    const DecodeArgs dec, const DecodeTArgs dt, const DecodeShapeArgs sh,
                    const CapArgs cap, const Lens seqs, float* __restrict__ xs) {
  using C = Cfg<D, NQ>;
  constexpr int CHUNKS = C::CHUNKS;
  constexpr uint32_t TILE = C::TILE;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if ((sbase & 1023u) != 0) {
    if (threadIdx.x == 0) record_bounds(p.err, BAD_ALIGN);
    return;
  }
  const Bars<D, NQ> bars{sbase + C::OFF_BAR};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* start = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);
  long long* range = reinterpret_cast<long long*>(smem + C::OFF_MISC + 24);
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const int* lens = dec.cache_seqlens;
  const int R = dec.n_rows;

  if (threadIdx.x == 0) {
    *abort = 0;
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bars.k_full(s), 1);
      mbar_init(bars.k_empty(s), 1);
      mbar_init(bars.v_full(s), 1);
      mbar_init(bars.v_empty(s), 1);
    }
    for (int i = 0; i < C::QBUF; ++i) {
      mbar_init(bars.q_full(i), 1);
      mbar_init(bars.q_empty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars.s_full(i), 1);
      mbar_init(bars.s_free(i), C::SOFTMAX_THREADS);
    }
    for (int i = 0; i < C::PBUF; ++i) {
      mbar_init(bars.p_ready(i), C::SOFTMAX_THREADS);
      mbar_init(bars.pv_done(i), 1);
    }
    mbar_init(bars.v_land(), 1);
    fence_mbar_init();
  }
  // CTA c serves kv head c % H_kv over range c / H_kv of the groups.
  const int groups = dt.ctas / p.H_kv;
  const int grp = blockIdx.x / p.H_kv;
  const int hk = blockIdx.x % p.H_kv;
  if (warp == C::WARP_TMA) {
    // This CTA's range [u0, u1) of the U = sum_b n_b units, and the tile at
    // u0: a scan of the lengths, 32 sequences per step.
    long long tot = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int b = b0 + lane;
      if (b < p.B) {
        int len, f;
        const int l = __ldg(lens + b);
        if (l < 0 || l > p.max_seqlen) record_bounds(p.err, BAD_CACHE_LEN);
        const int n = seq_tiles(seqs, b, f, len);
        tot += n - f;
      }
    }
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) tot += __shfl_xor_sync(FULL, tot, sh);
    // No more ranges than units: an empty one inside a segment would be one more
    // partial for the merge to read.
    const long long used = min(tot, static_cast<long long>(groups));
    const long long u0 = grp < used ? tot * grp / used : tot;
    const long long u1 = grp < used ? tot * (grp + 1) / used : tot;
    int sb = 0, sl = 0;
    long long base = 0;
    if (u0 < tot) {
      long long acc = 0;
      for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        int len = 0, f = 0;
        const int n = (b < p.B) ? seq_tiles(seqs, b, f, len) : 0;
        const long long units = n - f;
        long long incl = units;
#pragma unroll
        for (int sh = 1; sh < 32; sh <<= 1) {
          const long long v = __shfl_up_sync(FULL, incl, sh);
          if (lane >= sh) incl += v;
        }
        incl += acc;
        const long long excl = incl - units;
        const unsigned hit = __ballot_sync(FULL, units > 0 && excl <= u0 && u0 < incl);
        if (hit != 0) {
          const int src = __ffs(hit) - 1;
          sb = b0 + src;
          base = __shfl_sync(FULL, excl, src);
          sl = __shfl_sync(FULL, n, src) - 1;
          break;
        }
        acc = __shfl_sync(FULL, incl, 31);
      }
    }
    const long long off = u0 - base;   // < n_sb when u0 < tot
    if (lane == 0) {
      start[0] = sb;
      start[1] = static_cast<int>(u0 < tot ? sl - off : 0);
      range[0] = u0;
      range[1] = u1;
    }
  }
  if (warp == C::WARP_MMA) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  // Q rows R .. NQ - 1 are never loaded: zero, so that the score columns of
  // the rows past R are exactly 0 and need no mask.
  for (int k = threadIdx.x; k < C::QBUF * CHUNKS * (NQ - R) * 8; k += C::THREADS) {
    const int unit = k % 8, row = R + (k / 8) % (NQ - R), blk = k / (8 * (NQ - R));
    *reinterpret_cast<uint4*>(smem + C::OFF_Q + blk * C::SPAN + row * 128 + unit * 16) =
        make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // finish_kernel may take its places now; it waits for this grid's end.
  release_dependents();
  Walk w0;
  w0.b = start[0];
  w0.t = start[1];
  w0.u0 = range[0];
  w0.u1 = range[1];
  w0.u = w0.u0;
  w0.f = 0;
  w0.n = 0;
  w0.len = 0;
  if (w0.u0 < w0.u1) w0.n = seq_tiles(seqs, w0.b, w0.f, w0.len);
  auto advance = [&](Walk& w) { w.next(seqs); };

  if (warp == C::WARP_TMA) {
    // ------------------------------------------------------------ producer ---
    // The whole warp runs the loop; lane 0 issues Q and contiguous tiles,
    // lane u box u of a paged tile. Three independent streams: Q per piece
    // (once the buffer's last score MMA is done), K and V per tile; K leads.
    // Paged cache: the K stream reads the page ids of its sequence 32 at a
    // time (lane L holding page base + L, the batch before it in flight), takes a
    // tile's ids by shuffle and leaves the tile's rows in a ring of 8 for the
    // V stream, which reads the same rows.
    const bool paged = dec.block_table != nullptr;
    const int box = paged ? min(dec.page, BN) : BN;   // rows per TMA box
    const int n_box = BN / box;                       // boxes (pages) per tile
    const int tpp = paged ? max(dec.page / BN, 1) : 1;   // tiles per page, pages >= 128 rows
    const uint64_t pol = read_once_policy();
    int* rows_s = reinterpret_cast<int*>(smem + C::OFF_ROWS);
    struct PageBatch {
      int base, cur, nxt;
    };
    auto page_id = [&](const Walk& w, int pg) -> int {
      const int n_pages = (w.len + dec.page - 1) / max(dec.page, 1);
      return (pg >= 0 && pg < n_pages && pg < dec.max_blocks)
                 ? __ldg(dec.block_table + static_cast<size_t>(w.b) * dec.max_blocks + pg)
                 : -1;
    };
    // Cache row of box `lane` (< n_box) of the K stream's tile: pages past the
    // sequence's end load from beyond the cache (zeros). A tile's n_box pages
    // start at a multiple of n_box, and n_box divides 32, so they lie in one
    // batch.
    PageBatch kpb{0, -1, -1};
    auto tile_row = [&](const Walk& w) -> int {
      const int pg0 = (box < BN) ? w.t * n_box : w.t / tpp;
      const int base = pg0 & ~31;
      if (w.first()) {
        kpb.base = base;
        kpb.cur = page_id(w, base + lane);
        kpb.nxt = page_id(w, base - 32 + lane);
      } else if (base != kpb.base) {
        kpb.base = base;
        kpb.cur = kpb.nxt;
        kpb.nxt = page_id(w, base - 32 + lane);
      }
      const int blk = __shfl_sync(FULL, kpb.cur, (pg0 + min(lane, n_box - 1) - kpb.base) & 31);
      int row = static_cast<int>(dec.cache_rows);
      // So do pages before the first slot that some query sees: they may have been
      // given back.
      if (lane < n_box && w.t * BN + lane * box < w.len &&
          w.t * BN + lane * box + box > first_slot(seqs, w.len)) {
        if (blk >= 0 && (static_cast<long long>(blk) + 1) * dec.page <= dec.cache_rows)
          row = blk * dec.page + (box < BN ? 0 : (w.t - pg0 * tpp) * BN);
        else
          record_bounds(p.err, BAD_PAGE);
      }
      return row;
    };
    // Tile w of K (j: the K stream's tile count) or V (its rows from the ring).
    auto load_kv = [&](uint32_t dst, const CUtensorMap* map, uint32_t bar, const Walk& w, int j,
                       bool is_k) {
      if (!paged) {
        if (lane == 0) {
          const int row = w.b * dec.page + w.t * BN;
#pragma unroll
          for (int c = 0; c < CHUNKS; ++c)
            tma_load_once(dst + c * KV_SPAN, map, bar, hk * D + c * 64, row, pol);
        }
      } else {
        int row;
        if (is_k) {
          row = tile_row(w);
          if (lane < 8) rows_s[(j & 7) * 8 + lane] = row;
        } else {
          row = (lane < 8) ? rows_s[(j & 7) * 8 + lane] : 0;
        }
        if (lane < n_box) {
#pragma unroll
          for (int c = 0; c < CHUNKS; ++c)
            tma_load_once(dst + c * KV_SPAN + lane * box * 128, map, bar, hk * D + c * 64, row, pol);
        }
      }
    };
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    Walk kw = w0, vw = w0, qw = w0;
    int jk = 0, jv = 0, pq = 0, nland = 0;
    bool ok = true;
    long long t_last = clock64();
    while (!kw.done() || !vw.done() || !qw.done()) {
      bool progress = false;
      if (!qw.done()) {
        const int qb = pq % C::QBUF;
        if (pq < C::QBUF || warp_test(bars.q_empty(qb), ((pq / C::QBUF) - 1) & 1)) {
          // The q_len tokens x g heads of this piece's sequence and kv head:
          // one (64, g, q_len) box per column block, rows token * g + head.
          if (lane == 0) {
            mbar_arrive_expect_tx(bars.q_full(qb), R * 128 * CHUNKS);
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c)
              tma_load_3d(sbase + C::OFF_Q + qb * C::Q_BYTES + c * C::SPAN, &tm_q,
                          bars.q_full(qb), c * 64, hk * dec.g, qw.b * dec.q_len);
          }
          ++pq;
          qw.next_piece(seqs);
          progress = true;
        }
      }
      // (K stays fewer than 8 tiles ahead of V: the rows ring.)
      if (!kw.done() && jk - jv < 8 &&
          warp_test(bars.k_empty(jk % STAGES), ((jk / STAGES) & 1) ^ 1)) {
        const int st = jk % STAGES;
        if (lane == 0) mbar_arrive_expect_tx(bars.k_full(st), TILE);
        __syncwarp();
        load_kv(sbase + C::OFF_K + st * TILE, &tm_k, bars.k_full(st), kw, jk, true);
        ++jk;
        advance(kw);
        progress = true;
      }
      if (!vw.done() && jv < jk &&
          warp_test(bars.v_empty(jv % STAGES), ((jv / STAGES) & 1) ^ 1)) {
        const int st = jv % STAGES;
        const uint32_t dst = sbase + C::OFF_V + st * TILE;
        if (!(vw.tail() && (vw.len % BN) != 0)) {
          if (lane == 0) mbar_arrive_expect_tx(bars.v_full(st), TILE);
          __syncwarp();
          load_kv(dst, &tm_v, bars.v_full(st), vw, jv, false);
        } else {
          // A sequence's last, partly filled tile: its rows past the end may
          // hold anything (0 * NaN in P V would not be 0). It lands on
          // v_land; the rows are zeroed here and published on v_full.
          if (lane == 0) mbar_arrive_expect_tx(bars.v_land(), TILE);
          __syncwarp();
          load_kv(dst, &tm_v, bars.v_land(), vw, jv, false);
          if (!warp_wait(bars.v_land(), nland & 1, p.err, abort, W_VLAND)) {
            ok = false;
            break;
          }
          ++nland;
          const int first = vw.len - vw.t * BN;   // rows [first, 128) are past the end
          uint8_t* tile = smem + C::OFF_V + st * TILE;
          for (int i = lane; i < (BN - first) * 8 * CHUNKS; i += 32) {
            const int c = i / ((BN - first) * 8);
            const int rr = first + (i / 8) % (BN - first);
            *reinterpret_cast<uint4*>(tile + c * KV_SPAN + rr * 128 + (i % 8) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars.v_full(st));
        }
        ++jv;
        advance(vw);
        progress = true;
      }
      if (progress) {
        t_last = clock64();
        continue;
      }
      // Lane 0 decides, so the whole warp leaves the loop together.
      const int stop =
          __shfl_sync(FULL, *abort ? 1 : (clock64() - t_last > p.err.budget ? 2 : 0), 0);
      if (stop == 1) {
        ok = false;
        break;
      }
      if (stop == 2) {
        if (lane == 0) {
          *abort = 1;
          atomicOr(p.err.word, ERR_TIMEOUT);
          atomicExch(p.err.word + 1, !qw.done() ? W_QEMPTY : !kw.done() ? W_KEMPTY : W_VEMPTY);
        }
        ok = false;
        break;
      }
          }
    if (ok && lane == 0) {
      // Drain: the tensor core's last arrivals on the empty barriers must
      // land before the CTA's shared memory is released.
      for (int j = max(0, jk - STAGES); j < jk; ++j)
        if (!mbar_wait(bars.k_empty(j % STAGES), (j / STAGES) & 1, p.err, abort, W_KEMPTY)) break;
      for (int j = max(0, jv - STAGES); j < jv; ++j)
        if (!mbar_wait(bars.v_empty(j % STAGES), (j / STAGES) & 1, p.err, abort, W_VEMPTY)) break;
      for (int j = max(0, pq - C::QBUF); j < pq; ++j)
        if (!mbar_wait(bars.q_empty(j % C::QBUF), (j / C::QBUF) & 1, p.err, abort, W_QEMPTY))
          break;
    }
  } else if (warp == C::WARP_MMA) {
    // ---------------------------------------------------------- MMA issuer ---
    // The whole warp runs the loop; one elected lane issues and commits.
    const uint32_t leader = elect_one();
    constexpr uint32_t IDESC_S = idesc_bf16(BN, NQ, false, false);   // S^T = K Q^T
    constexpr uint32_t IDESC_O = idesc_bf16(128, NQ, true, false);   // O^T += V^T P^T
    const uint64_t k_desc = sdesc_sw128(sbase + C::OFF_K, 16, 1024);   // keys x D, K-major
    const uint64_t q_desc = sdesc_sw128(sbase + C::OFF_Q, 16, 1024);   // queries x D, K-major
    // V^T as A: M = D runs along each V row (two 64-column blocks KV_SPAN
    // apart), K = keys down the rows: MN-major.
    const uint64_t v_desc = sdesc_sw128(sbase + C::OFF_V, KV_SPAN, 1024);
    const uint64_t p_desc = sdesc_sw128(sbase + C::OFF_P, 16, 1024);   // queries x keys, K-major
    // Polls its two streams and issues whichever is ready:
    //   S^T_is once K_is has landed, the softmax has loaded S^T_{is-2} from
    //   the buffer and (first tile of a piece) the piece's Q has landed;
    //   P_ip V_ip once V_ip has landed and P_ip is published.
    // Each barrier polled here completes its next phase only after this warp
    // has acted on the current one, so a parity test never sees two phases.
    Walk sw = w0, pw = w0;
    int is = 0, ip = 0, ps = 0;
    long long t_last = clock64();
    while (!pw.done()) {
      bool progress = false;
      if (!sw.done()) {
        const int st = is % STAGES;
        const bool first = sw.first();
        if ((!first || warp_test(bars.q_full(ps % C::QBUF), (ps / C::QBUF) & 1)) &&
            warp_test(bars.k_full(st), (is / STAGES) & 1) &&
            (is < 2 || warp_test(bars.s_free(is & 1), ((is - 2) >> 1) & 1))) {
          if (first) ++ps;
          const int qb = (ps - 1) % C::QBUF;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss_if(leader, tmem + C::TM_S + (is & 1) * NQ,
                      sdesc_add(k_desc, st * TILE + (kk >> 2) * KV_SPAN + (kk & 3) * 32),
                      sdesc_add(q_desc, qb * C::Q_BYTES + (kk >> 2) * C::SPAN + (kk & 3) * 32),
                      IDESC_S, kk > 0);
          tc_commit_if(leader, bars.s_full(is & 1));
          tc_commit_if(leader, bars.k_empty(st));
          if (sw.last()) tc_commit_if(leader, bars.q_empty(qb));
          ++is;
          advance(sw);
          progress = true;
        }
      }
      if (ip < is) {
        const int st = ip % STAGES;
        const int pb = ip % C::PBUF;
        if (warp_test(bars.v_full(st), (ip / STAGES) & 1) &&
            warp_test(bars.p_ready(pb), (ip / C::PBUF) & 1)) {
          tc_fence_after();
          const bool fresh = pw.first();   // a piece's first tile starts O^T afresh
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)   // K = 128 keys in steps of 16
            mma_ss_if(leader, tmem + C::TM_O, sdesc_add(v_desc, st * TILE + kk * 2048),
                      sdesc_add(p_desc, pb * C::P_BYTES + (kk >> 2) * C::SPAN + (kk & 3) * 32),
                      IDESC_O, (fresh && kk == 0) ? 0u : 1u);
          tc_commit_if(leader, bars.v_empty(st));
          tc_commit_if(leader, bars.pv_done(pb));
          ++ip;
          advance(pw);
          progress = true;
        }
      }
      if (progress) {
        t_last = clock64();
        continue;
      }
      const int stop =
          __shfl_sync(FULL, *abort ? 1 : (clock64() - t_last > p.err.budget ? 2 : 0), 0);
      if (stop == 1) break;
      if (stop == 2) {
        if (lane == 0) {
          *abort = 1;
          atomicOr(p.err.word, ERR_TIMEOUT);
          atomicExch(p.err.word + 1, (ip < is) ? W_PREADY : W_KFULL);
        }
        break;
      }
          }
  } else {
    // ------------------------------------------------------------- softmax ---
    // Warp w owns TMEM lanes 32 (w % 4) .. +31 (keys of a tile; rows of O^T
    // at the end of a piece) and query rows [NH (w / 4), NH (w / 4 + 1)).
    constexpr int NH = C::NH;
    const int bar = 1 + (warp >> 2);             // the group's barrier
    const int quarter = warp & 3;
    const int kt = quarter * 32 + lane;          // key of the tile / row d of O^T
    const int r0 = (warp >> 2) * NH;             // this thread's first query row
    const int own = r0 + kt;                     // the row that thread kt < NH keeps for its group
    const bool keeper = kt < NH && own < R;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    float* mref = reinterpret_cast<float*>(smem + C::OFF_MREF);
    float* alpha_s = reinterpret_cast<float*>(smem + C::OFF_ALPHA);
    float* red = reinterpret_cast<float*>(smem + C::OFF_RED);   // [quarter][row]
    float2* bias_s = reinterpret_cast<float2*>(smem + C::OFF_SLOPE);
    int* qpos_s = reinterpret_cast<int*>(smem + C::OFF_QPOS);
    const float c2 = p.scale_log2;
    const int g = dec.g;
    const bool capped = sh.cap > 0.f, biased = sh.slopes != nullptr;
    const bool placed = sh.key_positions != nullptr;
    // This thread's P word for a row pair holds keys (kt & ~1, kt | 1) of
    // row r (even thread) or r + 1 (odd thread): the pair's column block,
    // 16-byte unit (swizzled by the row below) and byte in the unit.
    const int kp = kt & ~1;
    const uint32_t p_chunk = C::OFF_P + (kp >> 6) * C::SPAN;
    const int p_unit = (kp & 63) >> 3;
    const int p_byte = (kp & 7) * 2;
    const bool odd = (lane & 1) != 0;
    // Rows past R: scores 0 (zero Q rows) or -inf (masked), reference +inf
    // and no move, so their P is 2^-inf = 0 and the per-row loops below run
    // over all of this thread's rows without a branch.
    if (kt < NH) {
      mref[own] = keeper ? 0.f : INFINITY;
      alpha_s[own] = 1.f;
      bias_s[own].x = (biased && keeper) ? -__ldg(sh.slopes + hk * g + own % g) * LOG2E : 0.f;
    }
    group_sync(bar);
    // This thread's rows' references: the move threshold m + 8 and the
    // exponent offset (0 while a row has seen no key, m = -inf), kept in
    // registers up to 8 rows a thread, read from shared memory beyond.
    constexpr bool REF_REGS = NH <= 8;
    float mt[REF_REGS ? NH : 1], mu[REF_REGS ? NH : 1];
    auto load_ref = [&]() {
      if constexpr (REF_REGS) {
#pragma unroll
        for (int r = 0; r < NH; ++r) {
          const float m = mref[r0 + r];
          mt[r] = m + RESCALE_LOG2;
          mu[r] = (m == -INFINITY) ? 0.f : m;
        }
      }
    };
    auto thr = [&](int r) -> float {
      if constexpr (REF_REGS) return mt[r];
      else return mref[r0 + r] + RESCALE_LOG2;
    };
    auto off = [&](int r) -> float {
      if constexpr (REF_REGS) {
        return mu[r];
      } else {
        const float m = mref[r0 + r];
        return (m == -INFINITY) ? 0.f : m;
      }
    };
    load_ref();
    Walk w = w0;
    float l[NH];   // this thread's part of its rows' sums, in the current reference
#pragma unroll
    for (int r = 0; r < NH; ++r) l[r] = 0.f;
    int i = 0;     // the CTA's tile counter
    int t0 = 0;    // first tile of the current piece
    int q0 = 0;    // position of the sequence's first query token
    bool ok = true;
    while (!w.done()) {
      const bool first = w.first();
      const bool last = w.last();
      if (first) {
        t0 = w.t;
#pragma unroll
        for (int r = 0; r < NH; ++r) l[r] = 0.f;
        // The rows' positions (a token before slot 0 has its slot number).
        if (kt < NH) {
          const int slot = w.len - dec.q_len + own / g;
          const int s0 = w.len - dec.q_len;
          const int* pos = placed ? sh.key_positions +
                                        (static_cast<size_t>(w.b) * p.H_kv + hk) * sh.slots
                                  : nullptr;
          const int here = (placed && keeper && slot >= 0) ? __ldg(pos + slot) : slot;
          qpos_s[own] = here - ((placed && s0 >= 0) ? __ldg(pos + s0) : s0);
          bias_s[own].y = static_cast<float>(qpos_s[own]);
        }
        q0 = w.len - dec.q_len;
        if (placed && q0 >= 0)
          q0 = __ldg(sh.key_positions + (static_cast<size_t>(w.b) * p.H_kv + hk) * sh.slots + q0);
        group_sync(bar);
      }
      const int key = w.t * BN + kt;
      const int kpos = (placed && key < w.len)
                           ? __ldg(sh.key_positions +
                                   (static_cast<size_t>(w.b) * p.H_kv + hk) * sh.slots + key)
                           : key;
      uint32_t s[NH];
      ok = ok && warp_wait(bars.s_full(i & 1), (i >> 1) & 1, p.err, abort, W_SFULL);
      if (ok) {
        tc_fence_after();
        tmem_row_ld<NH>(tmem + lane_off + C::TM_S + (i & 1) * NQ + r0, s);
        tc_fence_before();
        mbar_arrive(bars.s_free(i & 1));
      }
      float x[NH];
      if (capped) {
        // The polynomial while a warp's scores allow it: it keeps logits far below the cap
        // to the precision of fp32.
        float most = 0.f;
#pragma unroll
        for (int r = 0; r < NH; ++r) most = fmaxf(most, fabsf(__uint_as_float(s[r])));
        // What lies past the end, or before every query's window, must not choose the form.
        if (key >= w.len || key < first_slot(seqs, w.len)) most = 0.f;
        if (cap_form(cap, most) == 0) {
#pragma unroll
          for (int r = 0; r < NH; r += 2) {
            const float2 sc = make_float2(__uint_as_float(s[r]), __uint_as_float(s[r + 1]));
            const float2 z = __fmul2_rn(sc, cap_poly2<0>(cap, sc));
            x[r] = z.x;
            x[r + 1] = z.y;
          }
        } else {
#pragma unroll
          for (int r = 0; r < NH; ++r) x[r] = cap_exact(cap, __uint_as_float(s[r]));
        }
      } else {
#pragma unroll
        for (int r = 0; r < NH; ++r) x[r] = __uint_as_float(s[r]) * c2;
      }
      const int dist = q0 - kpos;   // of row 0; row r is qpos_s[r] further on
      if (biased) {
        const float d = static_cast<float>(dist);
#pragma unroll
        for (int r = 0; r < NH; ++r) {
          const float2 s2 = bias_s[r0 + r];
          x[r] = fmaf(s2.x, fabsf(d + s2.y), x[r]);
        }
      }
      // Query row r sees key `key` when key < len, causally key <= len - q_len +
      // r / g, i.e. r >= g (key - len + q_len), and within the window. A tile
      // that lies before len - q_len (causal) or len and inside every row's
      // window needs no mask; between positions the window is checked always.
      const bool late = (w.t + 1) * BN > (p.causal ? w.len - dec.q_len + 1 : w.len);
      const bool early = sh.window > 0 && (placed || w.t * BN < w.len - sh.window);
      if (late || early) {
        const int rmin = p.causal ? max(0, g * (key - (w.len - dec.q_len))) : 0;
        const int rlim = key < w.len ? R : 0;
#pragma unroll
        for (int r = 0; r < NH; ++r)
          if (!(r0 + r >= rmin && r0 + r < rlim &&
                (sh.window <= 0 || dist + qpos_s[r0 + r] < sh.window)))
            x[r] = -INFINITY;
      }
      if (xs != nullptr) {
        float* dst =
            xs + ((static_cast<size_t>(w.b) * p.H_kv + hk) * seqs.tiles + w.t - w.f) * R * BN + kt;
#pragma unroll
        for (int r = 0; r < NH; ++r)
          if (r0 + r < R) dst[(r0 + r) * BN] = x[r];
      }
      bool ex = false;
      if (!first) {
#pragma unroll
        for (int r = 0; r < NH; ++r) ex |= x[r] > thr(r);
      }
      // Does any score move its row's reference (or has a wait failed)? The
      // rare yes takes a second barrier that tells the two apart.
      const bool any = group_sync_or(bar, ex || !ok);
      if (any && !group_sync_and(bar, ok)) break;
      const bool move = first || any;
      bool rescale = false;
      if (move) {
        // Row maxima over the 128 keys: per warp by shuffles, then thread r
        // combines the four quarters and moves row r's reference.
#pragma unroll
        for (int r = 0; r < NH; ++r) {
          if (r0 + r < R) {
            float v = x[r];
#pragma unroll
            for (int sh = 16; sh > 0; sh >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, sh));
            if (lane == 0) red[quarter * NQ + r0 + r] = v;
          }
        }
        group_sync(bar);
        if (keeper) {
          const float tmax = fmaxf(fmaxf(red[own], red[NQ + own]),
                                   fmaxf(red[2 * NQ + own], red[3 * NQ + own]));
          const float mo = first ? -INFINITY : mref[own];
          float mn = mo, a = 1.f;
          if (tmax > mo + RESCALE_LOG2) {
            mn = tmax;
            a = (mo == -INFINITY) ? 0.f : ex2_approx(mo - tmax);
          }
          mref[own] = mn;
          alpha_s[own] = a;
        }
        group_sync(bar);
        load_ref();
        if (!first) {
#pragma unroll
          for (int r = 0; r < NH; ++r) {
            const float a = alpha_s[r0 + r];
            l[r] *= a;
            rescale |= a != 1.f;
          }
        }
      }
      // P = 2^(x - m) for this key and each of its rows; adjacent keys'
      // values are paired into one bf16x2 word per row by a shuffle.
      uint32_t pk[NH / 2];
#pragma unroll
      for (int r = 0; r < NH; r += 2) {
        const float p0 = ex2_approx(x[r] - off(r));
        const float p1 = ex2_approx(x[r + 1] - off(r + 1));
        l[r] += p0;
        l[r + 1] += p1;
        const float recv = __shfl_xor_sync(FULL, odd ? p0 : p1, 1);
        pk[r >> 1] = odd ? pack_bf16x2(recv, p1) : pack_bf16x2(p0, recv);
      }
      // P buffer i % PBUF is free once P_{i-PBUF} V_{i-PBUF} is done; O^T may
      // be rescaled once P_{i-1} V_{i-1} is (the same wait when PBUF = 1).
      const int pb = i % C::PBUF;
      if (i >= C::PBUF)
        ok = ok && warp_wait(bars.pv_done(pb), ((i - C::PBUF) / C::PBUF) & 1, p.err, abort,
                             W_PVDONE);
      if (rescale && C::PBUF > 1)
        ok = ok && warp_wait(bars.pv_done((i - 1) % C::PBUF), ((i - 1) / C::PBUF) & 1, p.err,
                             abort, W_PVDONE);
      if (ok) {
        tc_fence_after();
        uint8_t* pbase = smem + p_chunk + pb * C::P_BYTES;
#pragma unroll
        for (int r = 0; r < NH; r += 2) {
          const int row = r0 + (odd ? r + 1 : r);
          *reinterpret_cast<uint32_t*>(pbase + row * 128 + ((p_unit ^ (row & 7)) << 4) + p_byte) =
              pk[r >> 1];
        }
        if (rescale) {
          // Row kt of O^T, this thread's columns: column r moves to row r's
          // new reference.
          uint32_t o[NH];
          tmem_row_ld<NH>(tmem + lane_off + C::TM_O + r0, o);
#pragma unroll
          for (int r = 0; r < NH; ++r)
            o[r] = __float_as_uint(__uint_as_float(o[r]) * alpha_s[r0 + r]);
          tmem_row_st<NH>(tmem + lane_off + C::TM_O + r0, o);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(bars.p_ready(pb));
      }
      if (last) {
        // ------------------------------------------------ end of a piece ---
        // Row sums over the 128 keys, then O = O^T / l and the LSE, as the
        // final output when the piece is the whole segment, else as a
        // partial for the merge.
#pragma unroll
        for (int r = 0; r < NH; ++r) {
          if (r0 + r < R) {
            float v = l[r];
#pragma unroll
            for (int sh = 16; sh > 0; sh >>= 1) v += __shfl_xor_sync(FULL, v, sh);
            if (lane == 0) red[quarter * NQ + r0 + r] = v;
          }
        }
        if (!group_sync_and(bar, ok)) break;
        ok = warp_wait(bars.pv_done(i % C::PBUF), (i / C::PBUF) & 1, p.err, abort, W_PVDONE);
        if (ok) {
          tc_fence_after();
          uint32_t o[NH];
          tmem_row_ld<NH>(tmem + lane_off + C::TM_O + r0, o);
          tc_fence_before();
          const int seg = w.b * p.H_kv + hk;
          const bool whole = t0 + 1 == w.n && w.t == w.f;
          const size_t slot = static_cast<size_t>((w.b + grp) * p.H_kv + hk) * R;
#pragma unroll
          for (int rr = 0; rr < NH; ++rr) {
            const int r = r0 + rr;
            if (r < R && kt < D) {
              const float lt = (red[r] + red[NQ + r]) + (red[2 * NQ + r] + red[3 * NQ + r]);
              const float v = __uint_as_float(o[rr]) * (lt > 0.f ? 1.f / lt : 0.f);
              if (whole) {
                const size_t orow = static_cast<size_t>(w.b * dec.q_len + r / g) * p.H +
                                    hk * g + r % g;
                static_cast<__nv_bfloat16*>(p.o)[orow * D + kt] = __float2bfloat16_rn(v);
              } else {
                dt.o_part[(slot + r) * D + kt] = v;
              }
            }
          }
          if (keeper) {
            const float lt =
                (red[own] + red[NQ + own]) + (red[2 * NQ + own] + red[3 * NQ + own]);
            const float lse =
                (lt > 0.f) ? (mref[own] + __log2f(lt)) * 0.69314718055994531f : -INFINITY;
            if (whole) {
              const size_t orow = static_cast<size_t>(w.b * dec.q_len + own / g) * p.H +
                                  hk * g + own % g;
              p.lse[orow] = lse;
            } else {
              dt.lse_part[slot + own] = lse;
            }
          }
          if (threadIdx.x == 0) {
            if (t0 + 1 == w.n) dt.seg_first[seg] = grp;
            if (w.t == w.f) dt.seg_last[seg] = grp;
          }
        }
      }
      ++i;
      advance(w);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Range of group partials [c0, c1] of a segment with keys; c0 == c1 when its CTA wrote the
// rows (one piece).
struct Pieces {
  int c0, c1;
  // Whether the partials lie in the workspace. They do not where a wait of the first kernel
  // ran out: a CTA that gives up leaves the entries as it found them.
  __device__ bool sound(int groups) const { return c0 >= 0 && c1 < groups && c0 <= c1; }
};
__device__ __forceinline__ Pieces seg_pieces(const DecodeTArgs& dt, int seg, int len) {
  if (len <= 0) return {0, -1};
  return {dt.seg_first[seg], dt.seg_last[seg]};
}

// LSE of row r over the pieces (group c's sits in slot (b + c) H_kv + hk).
__device__ __forceinline__ float pieces_lse(const DecodeTArgs& dt, const Pieces& pc, int b, int hk,
                                            int H_kv, int R, int r) {
  float m = -INFINITY, tot = 0.f;
  for (int c = pc.c0; c <= pc.c1; ++c)
    m = fmaxf(m, dt.lse_part[static_cast<size_t>((b + c) * H_kv + hk) * R + r]);
  if (m == -INFINITY) return m;
  for (int c = pc.c0; c <= pc.c1; ++c)
    tot += expf(dt.lse_part[static_cast<size_t>((b + c) * H_kv + hk) * R + r] - m);
  return m + logf(tot);
}

// What follows the ranges, in one launch. Blocks [0, merge_blocks): the merge of the
// partials, one output row per warp: LSE = ln sum_c exp(LSE_c), O = sum_c exp(LSE_c -
// LSE) O_c. Segments inside one CTA's range were written by that CTA; empty sequences
// get O = 0 and LSE = -inf here. The others: key_weights[b, hk, j] += sum_r 2^(z_rj -
// LSE_r log2 e), FIN_TILES tiles of a segment per block, a warp a tile, four slots a lane.
// (xs has no __restrict__: the first kernel still writes it when this one starts.)
constexpr int FIN_THREADS = 128;
constexpr int FIN_TILES = FIN_THREADS / 32;
template <int D>
__global__ void __launch_bounds__(FIN_THREADS)
    finish_kernel(const AttnParams p, const DecodeArgs dec, const DecodeTArgs dt,
                  const DecodeShapeArgs sh, const Lens seqs, const float* xs, int merge_blocks) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int R = dec.n_rows;
  if (static_cast<int>(blockIdx.x) < merge_blocks) {
    const long long rid = static_cast<long long>(blockIdx.x) * (FIN_THREADS / 32) + warp;
    wait_for_primary();
    if (rid >= static_cast<long long>(p.B) * p.H_kv * R) return;
    const int seg = static_cast<int>(rid / R);
    const int r = static_cast<int>(rid % R);
    const int b = seg / p.H_kv;
    const int hk = seg % p.H_kv;
    const int len = __ldg(dec.cache_seqlens + b);
    if (len < 0 || len > p.max_seqlen) return;   // reported by the partials kernel
    const Pieces pc = seg_pieces(dt, seg, len);
    if (len > 0 && !pc.sound(dt.ctas / p.H_kv)) {
      if (lane == 0) record_bounds(p.err, BAD_MERGE);
      return;
    }
    if (len > 0 && pc.c0 == pc.c1) return;   // one piece: its CTA wrote the row
    const size_t orow = static_cast<size_t>(b * dec.q_len + r / dec.g) * p.H + hk * dec.g +
                        r % dec.g;
    constexpr int PER = D / 32;   // columns per lane
    float acc[PER] = {};
    float m = -INFINITY, tot = 0.f;
    for (int c = pc.c0 + lane; c <= pc.c1; c += 32)
      m = fmaxf(m, dt.lse_part[static_cast<size_t>((b + c) * p.H_kv + hk) * R + r]);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, s));
    if (m != -INFINITY) {
      for (int c0 = pc.c0; c0 <= pc.c1; c0 += 32) {
        // The 32 weights at once, a lane each; the rows then come without waiting.
        const int c = c0 + lane;
        const float mine =
            c <= pc.c1 ? expf(dt.lse_part[static_cast<size_t>((b + c) * p.H_kv + hk) * R + r] - m) : 0.f;
        const int cnt = min(32, pc.c1 - c0 + 1);
#pragma unroll 4
        for (int k = 0; k < cnt; ++k) {
          const float wgt = __shfl_sync(FULL, mine, k);
          const float* src =
              dt.o_part + (static_cast<size_t>((b + c0 + k) * p.H_kv + hk) * R + r) * D + lane * PER;
          tot += wgt;
#pragma unroll
          for (int e = 0; e < PER; e += 2) {
            const float2 v = *reinterpret_cast<const float2*>(src + e);
            acc[e] = fmaf(wgt, v.x, acc[e]);
            acc[e + 1] = fmaf(wgt, v.y, acc[e + 1]);
          }
        }
      }
    }
    const float inv = (tot > 0.f) ? 1.f / tot : 0.f;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + orow * D + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; e += 2)
      *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0) p.lse[orow] = (tot > 0.f) ? m + logf(tot) : -INFINITY;
    return;
  }
  __shared__ float lse2[64];
  const int per = (seqs.tiles + FIN_TILES - 1) / FIN_TILES;
  const int id = static_cast<int>(blockIdx.x) - merge_blocks;
  const int seg = id / per;
  const int b = seg / p.H_kv, hk = seg % p.H_kv;
  int f, len;
  const int n = seq_tiles(seqs, b, f, len);
  const int t0 = f + (id % per) * FIN_TILES;
  wait_for_primary();
  if (t0 >= n) return;
  // The first rows' scores and the slots' weights are on their way while the LSEs form.
  const int t = t0 + warp;
  const bool on = t < n;
  const float* x = xs + (static_cast<size_t>(seg) * seqs.tiles + t - f) * R * BN + 4 * lane;
  float* dst = sh.key_weights + static_cast<size_t>(seg) * sh.slots + t * BN + 4 * lane;
  constexpr int AHEAD = 8;
  float4 v[AHEAD];
  float w[4] = {};
#pragma unroll
  for (int r = 0; r < AHEAD; ++r)
    if (on && r < R) v[r] = *reinterpret_cast<const float4*>(x + static_cast<size_t>(r) * BN);
  float old[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) old[k] = (on && t * BN + 4 * lane + k < len) ? dst[k] : 0.f;
  const Pieces pc = seg_pieces(dt, seg, len);   // (len > 0: the segment has tiles)
  if (!pc.sound(dt.ctas / p.H_kv)) {   // the block's one segment: nothing is added to it
    if (threadIdx.x == 0) record_bounds(p.err, BAD_MERGE);
    return;
  }
  if (threadIdx.x < R) {
    const int r = threadIdx.x;
    const float s = pc.c0 == pc.c1 ? p.lse[static_cast<size_t>(b * dec.q_len + r / dec.g) * p.H +
                                           hk * dec.g + r % dec.g]
                                   : pieces_lse(dt, pc, b, hk, p.H_kv, R, r);
    lse2[r] = s == -INFINITY ? 0.f : s * LOG2E;   // a row that sees nothing: its z are -inf
  }
  __syncthreads();
  if (!on) return;
  auto add = [&](const float4& s, int r) {
    const float e = lse2[r];
    w[0] += ex2_approx(s.x - e);
    w[1] += ex2_approx(s.y - e);
    w[2] += ex2_approx(s.z - e);
    w[3] += ex2_approx(s.w - e);
  };
#pragma unroll
  for (int r = 0; r < AHEAD; ++r)
    if (r < R) add(v[r], r);
#pragma unroll 8
  for (int r = AHEAD; r < R; ++r)
    add(*reinterpret_cast<const float4*>(x + static_cast<size_t>(r) * BN), r);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (t * BN + 4 * lane + k < len) dst[k] = old[k] + w[k];
}

struct Workspace {
  DecodeTArgs t;
  float* xs;
  size_t bytes;
};

// Partials for (B H_kv + CTAs) slots, the segments' first and last group, and
// with weights the shaped scores of every tile that is walked.
Workspace carve(void* base, long long B, int H_kv, long long n_rows, int D, int tiles,
                bool weights) {
  auto r256 = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  Workspace w = {};
  w.t.ctas = decode_t_ctas(H_kv);
  const size_t segs = static_cast<size_t>(B) * H_kv;
  const size_t rows = (segs + static_cast<size_t>(w.t.ctas)) * static_cast<size_t>(n_rows);
  char* at = static_cast<char*>(base);
  auto take = [&](size_t n) {
    char* r = at + w.bytes;
    w.bytes += r256(n);
    return r;
  };
  w.t.o_part = reinterpret_cast<float*>(take(rows * D * 4));
  w.t.lse_part = reinterpret_cast<float*>(take(rows * 4));
  w.t.seg_first = reinterpret_cast<int*>(take(segs * 4));
  w.t.seg_last = reinterpret_cast<int*>(take(segs * 4));
  if (weights)
    w.xs = reinterpret_cast<float*>(take(segs * tiles * BN * n_rows * 4));
  return w;
}

template <int D, int NQ>
cudaError_t launch_nq(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                      const AttnParams& p, const DecodeArgs& d, const DecodeShapeArgs& sh,
                      const Workspace& w, const Lens& seqs, cudaStream_t stream) {
  using C = Cfg<D, NQ>;
  const cudaError_t e = allow_smem<decode_shaped_kernel<D, NQ>>(C::SMEM);
  if (e != cudaSuccess) return e;
  const CapArgs cap = sh.cap > 0.f ? cap_args(sh.cap, p.scale) : CapArgs{};
  decode_shaped_kernel<D, NQ><<<static_cast<unsigned>(w.t.ctas), C::THREADS, C::SMEM, stream>>>(
      tq, tk, tv, p, d, w.t, sh, cap, seqs, w.xs);
  return cudaGetLastError();
}

Lens lens_of(const AttnParams& p, const DecodeArgs& d, const DecodeShapeArgs& sh) {
  const long long reach = sh.window > 0 ? static_cast<long long>(sh.window) + d.q_len - 1 : INT_MAX;
  const long long most = (p.max_seqlen + BN - 1ll) / BN;
  return {d.cache_seqlens, p.B, p.max_seqlen,
          static_cast<int>(min(reach, static_cast<long long>(INT_MAX))),
          static_cast<int>(min(most, (reach + BN - 1) / BN + 1))};
}

Workspace workspace_of(const AttnParams& p, const DecodeArgs& d, const DecodeShapeArgs& sh,
                       void* base) {
  return carve(base, p.B, p.H_kv, d.n_rows, p.D, lens_of(p, d, sh).tiles, sh.key_weights != nullptr);
}

template <int D>
cudaError_t launch_walk(const AttnParams& p, const DecodeArgs& d, const DecodeShapeArgs& sh,
                        const Workspace& w, cudaStream_t stream) {
  CUtensorMap tq, tk, tv;
  const unsigned box_rows =
      (d.block_table != nullptr) ? static_cast<unsigned>(min(d.page, BN)) : BN;
  const unsigned long long cols = static_cast<unsigned long long>(p.H_kv) * D;
  if (!make_tmap_bf16_3d(&tq, p.q, p.total, p.H, D, static_cast<unsigned>(d.g),
                         static_cast<unsigned>(d.q_len)) ||
      !make_tmap_bf16_2d(&tk, p.k, d.cache_rows, cols, 64, box_rows) ||
      !make_tmap_bf16_2d(&tv, p.v, d.cache_rows, cols, 64, box_rows))
    return cudaErrorInvalidValue;
  const Lens seqs = lens_of(p, d, sh);
  if (d.n_rows <= 16) return launch_nq<D, 16>(tq, tk, tv, p, d, sh, w, seqs, stream);
  if (d.n_rows <= 32) return launch_nq<D, 32>(tq, tk, tv, p, d, sh, w, seqs, stream);
  return launch_nq<D, 64>(tq, tk, tv, p, d, sh, w, seqs, stream);
}

template <int D>
cudaError_t launch_finish(const AttnParams& p, const DecodeArgs& d, const DecodeShapeArgs& sh,
                          const Workspace& w, cudaStream_t stream) {
  const Lens seqs = lens_of(p, d, sh);
  const long long rows = static_cast<long long>(p.B) * p.H_kv * d.n_rows;
  const long long merge = (rows + FIN_THREADS / 32 - 1) / (FIN_THREADS / 32);
  const long long blocks =
      merge + (sh.key_weights ? static_cast<long long>(p.B) * p.H_kv *
                                   ((seqs.tiles + FIN_TILES - 1) / FIN_TILES)
                             : 0);
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  // Launched while the ranges still run; it waits for them before it reads.
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(FIN_THREADS);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, finish_kernel<D>, p, d, w.t, sh, seqs,
                            static_cast<const float*>(w.xs), static_cast<int>(merge));
}

}  // namespace sdec
}  // namespace

size_t decode_shaped_workspace(long long B, int H_kv, long long n_rows, int D, int max_len,
                               bool weights) {
  return sdec::carve(nullptr, B, H_kv, n_rows, D, static_cast<int>((max_len + sdec::BN - 1ll) / sdec::BN),
                     weights).bytes;
}

cudaError_t launch_decode_shaped(const AttnParams& p, const DecodeArgs& d,
                                 const DecodeShapeArgs& sh, void* workspace, cudaStream_t stream) {
  const sdec::Workspace w = sdec::workspace_of(p, d, sh, workspace);
  const cudaError_t e = p.D == 64 ? sdec::launch_walk<64>(p, d, sh, w, stream)
                                  : sdec::launch_walk<128>(p, d, sh, w, stream);
  return e == cudaSuccess ? launch_decode_finish(p, d, sh, workspace, stream) : e;
}

cudaError_t launch_decode_finish(const AttnParams& p, const DecodeArgs& d,
                                 const DecodeShapeArgs& sh, void* workspace, cudaStream_t stream) {
  const sdec::Workspace w = sdec::workspace_of(p, d, sh, workspace);
  return p.D == 64 ? sdec::launch_finish<64>(p, d, sh, w, stream)
                   : sdec::launch_finish<128>(p, d, sh, w, stream);
}

}  // namespace fa
