// Key ranges of every query token from document ids, prefix lengths and a window
// (fa_key_ranges).
#include "shaped.h"

namespace fa {
namespace {

constexpr unsigned FULL = 0xffffffffu;

// One CTA per sequence: the runs of equal document ids by a running maximum
// of run starts (forwards) and a running minimum of run ends (backwards).
__global__ void __launch_bounds__(1024)
    key_ranges_kernel(const AttnParams p, const int* doc, const int* prefix, int window,
                      int* key_begin, int* key_end) {
  __shared__ int part[32];
  __shared__ int carry;
  const SeqInfo s = seq_info(p, blockIdx.x);
  if (!seq_ok(p, s)) return;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int pre = prefix ? prefix[blockIdx.x] : 0;
  // Block-wide inclusive scan by max of ``v``, after ``carry``.
  auto scan = [&](int v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(FULL, v, o);
      if (lane >= o) v = max(v, u);
    }
    if (lane == 31) part[warp] = v;
    __syncthreads();
    if (warp == 0) {
      int w = part[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(FULL, w, o);
        if (lane >= o) w = max(w, u);
      }
      part[lane] = w;
    }
    __syncthreads();
    v = max(v, carry);
    if (warp > 0) v = max(v, part[warp - 1]);
    __syncthreads();
    if (tid == 1023) carry = v;
    __syncthreads();
    return v;
  };
  if (tid == 0) carry = 0;
  __syncthreads();
  for (int c0 = 0; c0 < s.len; c0 += 1024) {
    const int i = c0 + tid;
    const bool first = i < s.len && doc && i > 0 && doc[s.start + i] != doc[s.start + i - 1];
    const int lo = scan(first ? i : 0);
    if (i < s.len)
      key_begin[s.start + i] = (window > 0) ? max(lo, i - window + 1) : lo;
  }
  if (tid == 0) carry = -s.len;
  __syncthreads();
  for (int c0 = 0; c0 < s.len; c0 += 1024) {
    const int i = s.len - 1 - (c0 + tid);   // walking down: the maximum of -end
    const bool last = i >= 0 && doc && i + 1 < s.len && doc[s.start + i] != doc[s.start + i + 1];
    const int hi = -scan(last ? -(i + 1) : -s.len);
    if (i >= 0) key_end[s.start + i] = p.causal ? min(hi, max(i + 1, pre)) : hi;
  }
}

}  // namespace

cudaError_t launch_key_ranges(const AttnParams& p, const int* doc_ids, const int* prefix_lens,
                              int window, int* key_begin, int* key_end, cudaStream_t stream) {
  key_ranges_kernel<<<p.B, 1024, 0, stream>>>(p, doc_ids, prefix_lens, window, key_begin, key_end);
  return cudaGetLastError();
}

}  // namespace fa
