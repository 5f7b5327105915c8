// Eviction from a key/value cache by accumulated attention weight.
//
// Of each (sequence, kv head) the last ``recent`` slots stay, and the
// heaviest of the others up to ``keep`` in all (equal weights: the lower
// slot). select_kernel finds the weight of the last one taken by four counts
// over 8-bit digits and writes the kept slots in ascending order; move_kernel
// copies their K and V rows into the other cache.
#include <math.h>

#include "shaped.h"

namespace fa {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int SELECT_THREADS = 1024;
constexpr int MOVE_THREADS = 256;
enum : unsigned { BAD_CACHE_LEN = 0xA0F01, BAD_PAGE = 0xA0F02 };

// Order-preserving map of a weight to an unsigned key: larger weight, larger
// key; -0 counts as 0 and NaN as less than everything.
__device__ __forceinline__ unsigned weight_key(float w) {
  if (w != w) return 0u;
  const unsigned u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Block-wide exclusive sum of ``v``; ``total`` receives the sum.
__device__ __forceinline__ int block_scan(int v, int* part, int& total) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(FULL, incl, o);
    if (lane >= o) incl += u;
  }
  __syncthreads();
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int w = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(FULL, w, o);
      if (lane >= o) w += u;
    }
    part[lane] = w;
  }
  __syncthreads();
  total = part[31];
  return incl - v + (warp > 0 ? part[warp - 1] : 0);
}

__global__ void __launch_bounds__(SELECT_THREADS) select_kernel(const EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int part[32];
  __shared__ unsigned s_prefix;
  __shared__ int s_want;
  const int hk = blockIdx.x % a.H_kv, b = blockIdx.x / a.H_kv, tid = threadIdx.x;
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
  // The key of the want-th heaviest, digit by digit from the top.
  unsigned prefix = 0, mask = 0;
  if (want > 0 && want < old) {
    if (tid == 0) s_want = want;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int j = tid; j < old; j += SELECT_THREADS) {
        const unsigned key = weight_key(w[j]);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int need = s_want, d = 255;
        while (hist[d] < need) need -= hist[d--];
        s_want = need;
        s_prefix = prefix | (static_cast<unsigned>(d) << shift);
      }
      __syncthreads();
      prefix = s_prefix;
      mask |= 255u << shift;
    }
  }
  const bool all = want >= old;
  const int ties = (want > 0 && !all) ? s_want : 0;   // of the slots whose key equals prefix
  int taken = 0, tied = 0, total;
  for (int c0 = 0; c0 < len; c0 += SELECT_THREADS) {
    const int j = c0 + tid;
    bool keep = j < len && (j >= old || all);
    bool tie = false;
    if (j < old && want > 0 && !all) {
      const unsigned key = weight_key(w[j]);
      keep = key > prefix;
      tie = key == prefix;
    }
    const int rank = tied + block_scan(tie, part, total);
    tied += total;
    keep |= tie && rank < ties;
    const int at = taken + block_scan(keep, part, total);
    taken += total;
    if (keep) {
      a.src[seg * a.keep + at] = j;
      a.weights_out[seg * a.out_slots + at] = w[j];
      a.positions_out[seg * a.out_slots + at] =
          a.key_positions ? a.key_positions[seg * a.slots + j] : j;
    }
  }
  for (long long i = n + tid; i < a.out_slots; i += SELECT_THREADS) {
    a.weights_out[seg * a.out_slots + i] = 0.f;
    a.positions_out[seg * a.out_slots + i] = -1;
  }
}

// 16 bytes of a K row and of a V row per thread.
__global__ void __launch_bounds__(MOVE_THREADS) move_kernel(const EvictArgs a) {
  const int units = a.D / 8;
  const long long n = static_cast<long long>(a.B) * a.keep * a.H_kv * units;
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
  select_kernel<<<a.B * a.H_kv, SELECT_THREADS, 0, stream>>>(a);
  const long long n = static_cast<long long>(a.B) * a.keep * a.H_kv * (a.D / 8);
  if (n > 0)
    move_kernel<<<static_cast<unsigned>(min((n + MOVE_THREADS - 1) / MOVE_THREADS, 148ll * 16)),
                  MOVE_THREADS, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
