// Eviction from a key/value cache by accumulated attention weight.
//
// Of each (sequence, kv head) the last ``recent`` slots stay, and the heaviest of the
// others up to ``keep`` in all (equal weights: the lower slot). select_kernel, one CTA
// per (sequence, kv head), finds the weight of the last one taken and writes the kept
// slots in ascending order; move_kernel copies their K and V rows into the other cache.
//
// The selection. Weights map to unsigned keys of the same order. The key of the n-th
// heaviest is found digit by digit, 11 bits at a time, over key - least key: the digits
// then spread over the bins (accumulated weights share a few exponents, so that digits
// of the keys themselves put thousands of counts on one shared-memory address: 70 us on
// B16 H8, 4096 to 32768 slots). After the first digit the few keys that share it are
// gathered, and the rest of the search goes over them alone. What is left is bound by
// the instructions per slot, so the passes take four slots a lane: two per 128 slots and
// warp for the counts, and for the order one scan of packed (tie, taken) counts by
// shuffles. The keys wait in shared memory, up to 48K of them; longer rows are read again.
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
constexpr int LIST_MAX = 2048;        // keys gathered after a digit
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

// Key of a slot that stays in any case: above every weight's.
constexpr unsigned STAYS = 0xffffffffu;

template <bool HELD>
__global__ void __launch_bounds__(SELECT_THREADS) select_kernel(const EvictArgs a) {
  extern __shared__ __align__(16) unsigned s_key[];   // HELD: the keys, to a multiple of 128
  __shared__ int hist[BINS];
  __shared__ unsigned list[LIST_MAX];
  __shared__ int part[WARPS], part2[WARPS];
  __shared__ unsigned s_lo[WARPS], s_hi[WARPS];
  __shared__ unsigned s_digit;
  __shared__ int s_need, s_count, s_listed;
  const int hk = blockIdx.x % a.H_kv, b = blockIdx.x / a.H_kv, tid = threadIdx.x;
  const int warp = tid / 32, lane = tid % 32;
  release_dependents();
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
  const bool all = want >= old, choose = want > 0 && !all;
  // Keys of slots j .. j + 3 (j a multiple of four): STAYS in [old, len), 0 behind.
  auto key4 = [&](int j, unsigned (&k)[4]) {
    if (HELD) {
      const uint4 v = *reinterpret_cast<const uint4*>(s_key + j);
      k[0] = v.x;
      k[1] = v.y;
      k[2] = v.z;
      k[3] = v.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        k[e] = j + e < old ? weight_key(w[j + e]) : j + e < len ? STAYS : 0u;
    }
  };
  unsigned lo = STAYS, hi = 0u;
  if (HELD || choose) {
    const int end = (len + 127) & ~127;
    for (int base = 0; base < end; base += 8 * SELECT_THREADS) {
      float v[8];   // eight loads on their way
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = base + k * SELECT_THREADS + tid;
        v[k] = j < old ? w[j] : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = base + k * SELECT_THREADS + tid;
        if (j >= end) continue;
        const unsigned u = j < old ? weight_key(v[k]) : j < len ? STAYS : 0u;
        if (HELD) s_key[j] = u;
        if (j < old) {
          lo = min(lo, u);
          hi = max(hi, u);
        }
      }
    }
  }
  unsigned limit = STAYS - 1;   // key of the last one taken; nothing but STAYS above it
  int ties = 0;                 // how many with that key are taken
  if (choose) {
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
    int need = want, listed = -1;   // listed: how many keys the list holds, or -1
    unsigned prefix = 0;
    int bits = 32 - __clz(hi - lo);   // undecided low bits
    while (bits > 0) {
      const int shift = max(bits - DIGIT, 0);
      const unsigned mask = (1u << (bits - shift)) - 1u;
      for (int i = tid; i < BINS; i += SELECT_THREADS) hist[i] = 0;
      __syncthreads();
      if (listed >= 0) {
        for (int j = tid; j < listed; j += SELECT_THREADS) {
          const unsigned k = list[j];
          if ((k >> bits) == prefix) atomicAdd(&hist[(k >> shift) & mask], 1);
        }
      } else {
        for (int j = 4 * tid; j < old; j += 4 * SELECT_THREADS) {
          unsigned k[4];
          key4(j, k);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const unsigned d = k[e] - lo;
            if (j + e < old && (bits == 32 || (d >> bits) == prefix))
              atomicAdd(&hist[(d >> shift) & mask], 1);
          }
        }
      }
      __syncthreads();
      // Two bins a thread, from the top: the bin where the running count reaches ``need``.
      const int d0 = BINS - 1 - 2 * tid;
      const int h0 = hist[d0], h1 = hist[d0 - 1];
      const int incl = block_scan(h0 + h1, part);
      const int excl = incl - h0 - h1;
      if (excl < need && need <= incl) {
        const bool second = need > excl + h0;
        s_digit = static_cast<unsigned>(second ? d0 - 1 : d0);
        s_need = need - excl - (second ? h0 : 0);
        s_count = second ? h1 : h0;
        s_listed = 0;
      }
      __syncthreads();
      prefix = (prefix << (bits - shift)) | s_digit;
      need = s_need;
      bits = shift;
      if (bits > 0 && listed < 0 && s_count <= LIST_MAX) {
        for (int j = 4 * tid; j < old; j += 4 * SELECT_THREADS) {
          unsigned k[4];
          key4(j, k);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const unsigned d = k[e] - lo;
            if (j + e < old && (d >> bits) == prefix) list[atomicAdd(&s_listed, 1)] = d;
          }
        }
        __syncthreads();
        listed = s_listed;
      }
    }
    limit = lo + prefix;
    ties = need;
  } else {
    __syncthreads();   // the keys
  }
  // Each warp's stretch of slots, four a lane: how many are above the limit or stay
  // anyway, and how many sit on it, packed (ties above bit 16; a stretch of a warp holds
  // fewer than 2^16 slots at a time).
  const int per = ((len + WARPS - 1) / WARPS + 127) & ~127;
  const int j0 = min(len, warp * per), j1 = min(len, j0 + per);
  auto sorts = [&](int j, unsigned& above, unsigned& tie) {   // bit e: slot j + e
    above = tie = 0u;
    unsigned k[4];
    if (j < j1) {
      key4(j, k);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (j + e < j1 && (all || k[e] > limit)) above |= 1u << e;
        if (j + e < j1 && !all && k[e] == limit) tie |= 1u << e;
      }
    }
  };
  int n_above = 0, n_tie = 0;
  for (int j = j0; j < j1; j += 128) {
    unsigned above, tie;
    sorts(j + 4 * lane, above, tie);
    n_above += __popc(above);
    n_tie += __popc(tie);
  }
  n_above = __reduce_add_sync(FULL, n_above);
  n_tie = __reduce_add_sync(FULL, n_tie);
  __syncthreads();
  if (lane == 0) {
    part[warp] = n_above;
    part2[warp] = n_tie;
  }
  __syncthreads();
  // Ties and places before this warp.
  int rank = __reduce_add_sync(FULL, lane < warp ? part2[lane] : 0);
  int taken = __reduce_add_sync(FULL, lane < warp ? part[lane] : 0);
  for (int j = j0; j < j1; j += 128) {
    unsigned above, tie;
    const int s = j + 4 * lane;
    sorts(s, above, tie);
    // Inclusive counts over the lanes: ties in the high half, above in the low.
    const int mine = (__popc(tie) << 16) | __popc(above);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(FULL, incl, o);
      if (lane >= o) incl += u;
    }
    const int sum = __shfl_sync(FULL, incl, 31);
    int r = rank + ((incl - mine) >> 16), t = taken + ((incl - mine) & 0xffff);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool is_tie = (tie >> e) & 1u, is_above = (above >> e) & 1u;
      if (is_above || (is_tie && r < ties)) {
        const int to = t + min(r, ties);
        if (to >= n) break;
        a.src[seg * a.keep + to] = s + e;
        a.weights_out[seg * a.out_slots + to] = w[s + e];
        a.positions_out[seg * a.out_slots + to] =
            a.key_positions ? a.key_positions[seg * a.slots + s + e] : s + e;
      }
      r += is_tie;
      t += is_above;
    }
    rank += sum >> 16;
    taken += sum & 0xffff;
  }
  for (long long i = n + tid; i < a.out_slots; i += SELECT_THREADS) {
    a.weights_out[seg * a.out_slots + i] = 0.f;
    a.positions_out[seg * a.out_slots + i] = -1;
  }
}

__global__ void __launch_bounds__(MOVE_THREADS) move_kernel(const EvictArgs a) {
  const int units = a.D / 8;
  const long long n = static_cast<long long>(a.B) * a.keep * a.H_kv * units;
  wait_for_primary();   // the selection
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
  const int keys = (a.max_len + 127) & ~127;
  if (keys <= KEYS_MAX) {
    const cudaError_t e = allow_smem<select_kernel<true>>(KEYS_MAX * 4);
    if (e != cudaSuccess) return e;
    select_kernel<true><<<a.B * a.H_kv, SELECT_THREADS, keys * sizeof(unsigned), stream>>>(a);
  } else {
    select_kernel<false><<<a.B * a.H_kv, SELECT_THREADS, 0, stream>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
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
