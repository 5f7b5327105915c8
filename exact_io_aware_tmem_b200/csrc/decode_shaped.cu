// Decode with shaped scores over a contiguous or paged cache: one warp per
// query row walks the keys with the online-softmax recurrence; a second
// kernel adds each slot's attention weights, one warp per slot.
#include <math.h>

#include "shaped.h"

namespace fa {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int WARPS = 4;
constexpr int DMAX = 128;
constexpr int PER = DMAX / 32;
enum : unsigned { BAD_CACHE_LEN = 0x90F01, BAD_PAGE = 0x90F02 };

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(FULL, x, o));
  return x;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(FULL, x, o);
  return x;
}

// Position of slot j of (sequence b, kv head hk); a query token before slot 0
// (j < 0) counts from the first slot as if none had been lost.
__device__ __forceinline__ int slot_position(const DecodeShapeArgs& sh, size_t seg, int j) {
  return (sh.key_positions != nullptr && j >= 0) ? sh.key_positions[seg * sh.slots + j] : j;
}

// z of the key in slot j for the query in slot sq, or -inf where hidden.
__device__ __forceinline__ float shape(const AttnParams& p, const DecodeShapeArgs& sh, size_t seg,
                                       float raw, float slope, int j, int sq, int pq) {
  const int dist = pq - slot_position(sh, seg, j);
  if ((p.causal && j > sq) || (sh.window > 0 && dist >= sh.window)) return -INFINITY;
  const float z = sh.cap > 0.f ? sh.cap * tanhf(raw * sh.scale_over_cap) : raw * p.scale;
  return fmaf(-slope, fabsf(static_cast<float>(dist)), z);
}

__device__ __forceinline__ float dot_row(const float* a, const __nv_bfloat16* b, int D) {
  float acc = 0.f;
  for (int d = 0; d < D; ++d) acc = fmaf(a[d], __bfloat162float(b[d]), acc);
  return acc;
}

__global__ void __launch_bounds__(WARPS * 32)
    rows_kernel(AttnParams p, DecodeArgs dec, DecodeShapeArgs sh) {
  __shared__ float qs[WARPS][DMAX];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long long row = static_cast<long long>(blockIdx.x) * WARPS + warp;   // token * H + h
  if (row >= p.total * p.H) return;
  const int h = static_cast<int>(row % p.H), tok = static_cast<int>(row / p.H);
  const int b = tok / dec.q_len, hk = h / dec.g, D = p.D;
  const int len = dec.cache_seqlens[b];
  if (len < 0 || len > p.max_seqlen) {
    if (lane == 0) record_bounds(p.err, BAD_CACHE_LEN);
    return;
  }
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + row * D;
  for (int d = lane; d < D; d += 32) qs[warp][d] = __bfloat162float(q[d]);
  __syncwarp();
  const size_t seg = static_cast<size_t>(b) * p.H_kv + hk;
  const float slope = sh.slopes ? sh.slopes[h] : 0.f;
  const int sq = len - dec.q_len + tok % dec.q_len, pq = slot_position(sh, seg, sq);
  const size_t stride = static_cast<size_t>(p.H_kv) * D;
  const __nv_bfloat16* K = static_cast<const __nv_bfloat16*>(p.k) + static_cast<size_t>(hk) * D;
  const __nv_bfloat16* V = static_cast<const __nv_bfloat16*>(p.v) + static_cast<size_t>(hk) * D;
  float m = -INFINITY, l = 0.f, acc[PER] = {};
  for (int c0 = 0; c0 < len; c0 += 32) {
    const int j = c0 + lane;
    float z = -INFINITY;
    long long r = -1;
    if (j < len) {
      r = cache_row(dec.block_table, dec.max_blocks, dec.page, dec.cache_rows, b, j);
      if (r < 0)
        record_bounds(p.err, BAD_PAGE);
      else
        z = shape(p, sh, seg, dot_row(qs[warp], K + r * stride, D), slope, j, sq, pq);
    }
    const float m_new = fmaxf(m, warp_max(z));
    const float m_use = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = expf(m - m_use), pj = expf(z - m_use);
    l = l * alpha + warp_sum(pj);
#pragma unroll
    for (int t = 0; t < PER; ++t) acc[t] *= alpha;
    for (int jj = 0; jj < min(32, len - c0); ++jj) {
      const float pb = __shfl_sync(FULL, pj, jj);
      const long long rb = __shfl_sync(FULL, r, jj);
      if (pb == 0.f) continue;
#pragma unroll
      for (int t = 0; t < PER; ++t)
        if (lane + 32 * t < D)
          acc[t] = fmaf(pb, __bfloat162float(V[rb * stride + lane + 32 * t]), acc[t]);
    }
    m = m_new;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int t = 0; t < PER; ++t)
    if (lane + 32 * t < D)
      static_cast<__nv_bfloat16*>(p.o)[row * D + lane + 32 * t] = __float2bfloat16_rn(acc[t] * inv);
  if (lane == 0) p.lse[row] = l > 0.f ? m + logf(l) : -INFINITY;
}

// key_weights[b, hk, j] += sum over the rows of (b, hk) of exp(z - LSE).
__global__ void __launch_bounds__(WARPS * 32)
    weights_kernel(AttnParams p, DecodeArgs dec, DecodeShapeArgs sh) {
  __shared__ float ks[WARPS][DMAX];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int j = blockIdx.x * WARPS + warp, hk = blockIdx.y, D = p.D;
  for (int b = blockIdx.z; b < p.B; b += gridDim.z) {
    const int len = dec.cache_seqlens[b];
    if (len > p.max_seqlen || j >= len) continue;
    const size_t seg = static_cast<size_t>(b) * p.H_kv + hk;
    const long long r = cache_row(dec.block_table, dec.max_blocks, dec.page, dec.cache_rows, b, j);
    if (r < 0) continue;
    __syncwarp();
    const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.k) + (r * p.H_kv + hk) * D;
    for (int d = lane; d < D; d += 32) ks[warp][d] = __bfloat162float(k[d]);
    __syncwarp();
    float w = 0.f;
    for (int rr = lane; rr < dec.n_rows; rr += 32) {
      const int t = rr / dec.g, h = hk * dec.g + rr % dec.g;
      const size_t row = static_cast<size_t>(b * dec.q_len + t) * p.H + h;
      const int sq = len - dec.q_len + t;
      const float z = shape(p, sh, seg, dot_row(ks[warp], static_cast<const __nv_bfloat16*>(p.q) + row * D, D),
                            sh.slopes ? sh.slopes[h] : 0.f, j, sq, slot_position(sh, seg, sq));
      if (z != -INFINITY) w += expf(z - p.lse[row]);
    }
    w = warp_sum(w);
    if (lane == 0) sh.key_weights[seg * sh.slots + j] += w;
  }
}

}  // namespace

cudaError_t launch_decode_shaped(const AttnParams& p, const DecodeArgs& d,
                                 const DecodeShapeArgs& sh, cudaStream_t stream) {
  const long long rows = p.total * p.H;
  rows_kernel<<<static_cast<unsigned>((rows + WARPS - 1) / WARPS), WARPS * 32, 0, stream>>>(p, d, sh);
  if (sh.key_weights != nullptr && p.max_seqlen > 0)
    weights_kernel<<<dim3((p.max_seqlen + WARPS - 1) / WARPS, p.H_kv, min(p.B, 65535)), WARPS * 32,
                     0, stream>>>(p, d, sh);
  return cudaGetLastError();
}

}  // namespace fa
