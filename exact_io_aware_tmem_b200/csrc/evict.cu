// Eviction from a key/value cache by accumulated attention weight.
//
// Of each (sequence, kv head) the last ``recent`` slots stay, and the heaviest of the
// others up to ``keep`` in all (equal weights: the lower slot). select_kernel, one CTA
// per (sequence, kv head), finds the weight of the last one taken and writes the kept
// slots in ascending order; move_kernel copies their K and V rows into the other cache.
//
// The selection. Weights map to unsigned keys of the same order. The key of the n-th
// heaviest is found digit by digit, 11 bits at a time, over key - least key: the
// digits then spread over the bins (accumulated weights share a few exponents, so that
// digits of the keys themselves put thousands of counts on one shared-memory address:
// 70 us against 19 on B16 H8, 4096 to 32768 slots). Each warp then walks its own stretch
// of slots with ballots, so that the order needs one scan over the warps' counts.
// The keys wait in shared memory, up to 48K of them; longer rows are read again.
//
// The move is bound by its bytes: 16 of a K and a V row per thread, grid-stride.
#include <math.h>

#include <algorithm>

#include "shaped.h"

namespace fa {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int SELECT_THREADS = 1024;
constexpr int WARPS = SELECT_THREADS / 32;
constexpr int DIGIT = 11;
constexpr int BINS = 1 << DIGIT;
constexpr int KEYS_MAX = 48 * 1024;   // keys held in shared memory
constexpr int MOVE_THREADS = 256;
enum : unsigned { BAD_CACHE_LEN = 0xA0F01, BAD_PAGE = 0xA0F02 };

// Order-preserving map of a weight to an unsigned key: larger weight, larger key; -0
// counts as 0 and NaN as less than everything.
__device__ __forceinline__ unsigned weight_key(float w) {
  if (w != w) return 0u;
  const unsigned u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Block-wide inclusive sum of ``v`` over the threads.
__device__ __forceinline__ int block_scan(int v, int* part) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(FULL, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) part[warp] = v;
  __syncthreads();
  int before = lane < warp ? part[lane] : 0;
  before = __reduce_add_sync(FULL, before);
  return v + before;
}

__global__ void __launch_bounds__(SELECT_THREADS) select_kernel(const EvictArgs a, int held) {
  extern __shared__ unsigned s_key[];   // ``held`` keys
  __shared__ int hist[BINS];
  __shared__ int part[WARPS], part2[WARPS];
  __shared__ unsigned s_lo[WARPS], s_hi[WARPS];
  __shared__ unsigned s_digit;
  __shared__ int s_need;
  const int hk = blockIdx.x % a.H_kv, b = blockIdx.x / a.H_kv, tid = threadIdx.x;
  const int warp = tid / 32, lane = tid % 32;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int len = a.cache_seqlens[b];
  if (len < 0 || len > a.max_len) {
    if (tid == 0) record_bounds(a.err, BAD_CACHE_LEN);
    return;
  }
  const size_t seg = static_cast<size_t>(b) * a.H_kv + hk;
  const float* w = a.key_weights + seg * a.slots;
  const int n = min(len, a.keep);          // slots kept
  const int old = len - min(a.recent, n);  // slots [old, len) stay in any case
  const int want = n - (len - old);        // to take of the first ``old``
  if (tid == 0 && hk == 0) a.seqlens_out[b] = n;
  auto key = [&](int j) { return j < held ? s_key[j] : weight_key(w[j]); };
  const bool choose = want > 0 && want < old;
  unsigned limit = 0;   // key of the last one taken
  int ties = 0;         // how many with that key are taken
  if (choose) {
    unsigned lo = 0xffffffffu, hi = 0u;
    for (int j = tid; j < old; j += SELECT_THREADS) {
      const unsigned k = weight_key(w[j]);
      if (j < held) s_key[j] = k;
      lo = min(lo, k);
      hi = max(hi, k);
    }
    lo = __reduce_min_sync(FULL, lo);
    hi = __reduce_max_sync(FULL, hi);
    if (lane == 0) {
      s_lo[warp] = lo;
      s_hi[warp] = hi;
    }
    __syncthreads();
    lo = __reduce_min_sync(FULL, s_lo[lane]);
    hi = __reduce_max_sync(FULL, s_hi[lane]);
    // Digits of key - lo from the highest bit that differs downwards.
    int need = want;
    unsigned prefix = 0;
    int bits = 32 - __clz(hi - lo);   // undecided low bits
    while (bits > 0) {
      const int shift = max(bits - DIGIT, 0);
      for (int i = tid; i < BINS; i += SELECT_THREADS) hist[i] = 0;
      __syncthreads();
      for (int j = tid; j < old; j += SELECT_THREADS) {
        const unsigned k = key(j) - lo;
        if (bits == 32 || (k >> bits) == prefix)
          atomicAdd(&hist[(k >> shift) & ((1u << (bits - shift)) - 1u)], 1);
      }
      __syncthreads();
      // Two bins a thread, from the top: the bin where the running count reaches
      // ``need``.
      const int d0 = BINS - 1 - 2 * tid;
      const int h0 = hist[d0], h1 = hist[d0 - 1];
      const int incl = block_scan(h0 + h1, part);
      const int excl = incl - h0 - h1;
      if (excl < need && need <= incl) {
        const bool second = need > excl + h0;
        s_digit = static_cast<unsigned>(second ? d0 - 1 : d0);
        s_need = need - excl - (second ? h0 : 0);
      }
      __syncthreads();
      prefix = (prefix << (bits - shift)) | s_digit;
      need = s_need;
      bits = shift;
    }
    limit = lo + prefix;
    ties = need;
  }
  // Each warp's stretch of slots: how many are above the limit or stay anyway, and how
  // many sit on it.
  const int per = ((len + WARPS - 1) / WARPS + 31) & ~31;
  const int j0 = warp * per, j1 = min(len, j0 + per);
  auto sort_of = [&](int j, bool& above, bool& tie) {
    above = tie = false;
    if (j >= j1) return;
    if (j >= old || want >= old) {
      above = true;
    } else if (choose) {
      const unsigned k = key(j);
      above = k > limit;
      tie = k == limit;
    }
  };
  int n_above = 0, n_tie = 0;
  for (int j = j0; j < j1; j += 32) {
    bool above, tie;
    sort_of(j + lane, above, tie);
    n_above += __popc(__ballot_sync(FULL, above));
    n_tie += __popc(__ballot_sync(FULL, tie));
  }
  __syncthreads();
  if (lane == 0) {
    part[warp] = n_above;
    part2[warp] = n_tie;
  }
  __syncthreads();
  // Ties before this warp, and places taken before it.
  const int tie_all = part2[lane], above_all = part[lane];
  const int tie_before = __reduce_add_sync(FULL, lane < warp ? tie_all : 0);
  int at = __reduce_add_sync(FULL, lane < warp ? above_all : 0) + min(tie_before, ties);
  int rank = tie_before;
  const unsigned below = (1u << lane) - 1u;
  for (int j = j0; j < j1; j += 32) {
    bool above, tie;
    sort_of(j + lane, above, tie);
    const unsigned t = __ballot_sync(FULL, tie);
    const bool keep = above || (tie && rank + __popc(t & below) < ties);
    const unsigned k = __ballot_sync(FULL, keep);
    if (keep) {
      const int to = at + __popc(k & below);
      const int s = j + lane;
      a.src[seg * a.keep + to] = s;
      a.weights_out[seg * a.out_slots + to] = w[s];
      a.positions_out[seg * a.out_slots + to] =
          a.key_positions ? a.key_positions[seg * a.slots + s] : s;
    }
    rank += __popc(t);
    at += __popc(k);
  }
  for (long long i = n + tid; i < a.out_slots; i += SELECT_THREADS) {
    a.weights_out[seg * a.out_slots + i] = 0.f;
    a.positions_out[seg * a.out_slots + i] = -1;
  }
}

__global__ void __launch_bounds__(MOVE_THREADS) move_kernel(const EvictArgs a) {
  const int units = a.D / 8;
  const long long n = static_cast<long long>(a.B) * a.keep * a.H_kv * units;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the selection
  for (long long t = static_cast<long long>(blockIdx.x) * MOVE_THREADS + threadIdx.x; t < n;
       t += static_cast<long long>(gridDim.x) * MOVE_THREADS) {
    const int u = static_cast<int>(t % units);
    const int hk = static_cast<int>(t / units % a.H_kv);
    const long long bi = t / units / a.H_kv;
    const int i = static_cast<int>(bi % a.keep), b = static_cast<int>(bi / a.keep);
    const int len = a.cache_seqlens[b];
    if (len > a.max_len || i >= len) continue;
    const int j = a.src[(static_cast<size_t>(b) * a.H_kv + hk) * a.keep + i];
    const long long from = cache_row(a.block_table, a.max_blocks, a.page, a.cache_rows, b, j);
    const long long to = cache_row(a.out_table, a.out_max_blocks, a.out_page, a.out_rows, b, i);
    if (from < 0 || to < 0) {
      record_bounds(a.err, BAD_PAGE);
      continue;
    }
    const size_t f = (from * a.H_kv + hk) * units + u, d = (to * a.H_kv + hk) * units + u;
    static_cast<uint4*>(a.k_out)[d] = static_cast<const uint4*>(a.k)[f];
    static_cast<uint4*>(a.v_out)[d] = static_cast<const uint4*>(a.v)[f];
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
  const int held = std::min(a.max_len, KEYS_MAX);
  const cudaError_t e = allow_smem<select_kernel>(KEYS_MAX * 4);
  if (e != cudaSuccess) return e;
  select_kernel<<<a.B * a.H_kv, SELECT_THREADS, held * sizeof(unsigned), stream>>>(a, held);
  const long long n = static_cast<long long>(a.B) * a.keep * a.H_kv * (a.D / 8);
  // Launched while the selection still runs; it waits for it before it reads.
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(
      std::min<long long>((n + MOVE_THREADS - 1) / MOVE_THREADS, 148ll * 16)));
  cfg.blockDim = dim3(MOVE_THREADS);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, move_kernel, a);
}

}  // namespace fa
