// Attention with shaped scores on CUDA cores: one warp per query row (forward,
// dQ) or key row (dK, dV), 32 keys or queries scored one per lane.
//
//     z = cap tanh(scale q.k / cap) - slope |i - j|,  O = softmax(z) V,
//     P = exp(z - LSE), dV = P^T dO, dZ = P (dO V^T - D), D_i = dO_i . O_i,
//     dS = dZ (1 - tanh^2), dQ = scale dS K, dK = scale dS^T Q.
// Every product and sum is a 32-bit FMA; bf16 inputs are widened first.
#include <math.h>

#include "shaped.h"

namespace fa {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int WARPS = 4;
constexpr int DMAX = 128;
constexpr int PER = DMAX / 32;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

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

template <typename T>
__device__ __forceinline__ float dot_row(const float* a, const T* b, int D) {
  float acc = 0.f;
  for (int d = 0; d < D; ++d) acc = fmaf(a[d], to_f(b[d]), acc);
  return acc;
}

// z of one (query, key) pair from the raw product, and the cap's derivative.
__device__ __forceinline__ float shape(const AttnParams& p, const ShapeArgs& sh, float slope,
                                       float raw, int dist, float& grad) {
  float z = raw * p.scale;
  grad = 1.f;
  if (sh.cap > 0.f) {
    const float t = tanhf(raw * sh.scale_over_cap);
    z = sh.cap * t;
    grad = 1.f - t * t;
  }
  return fmaf(-slope, static_cast<float>(abs(dist)), z);
}

template <typename T>
__global__ void __launch_bounds__(WARPS * 32) fwd_kernel(AttnParams p, ShapeArgs sh) {
  __shared__ float qs[WARPS][DMAX];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int b = blockIdx.z, h = blockIdx.y;
  const SeqInfo s = seq_info(p, b);
  if (!seq_ok(p, s)) return;
  const int i = blockIdx.x * WARPS + warp;
  if (i >= s.len) return;
  const int D = p.D, hk = h / (p.H / p.H_kv);
  const size_t kv_stride = static_cast<size_t>(p.H_kv) * D;
  const size_t koff = (static_cast<size_t>(s.start) * p.H_kv + hk) * D;
  const T* K = static_cast<const T*>(p.k) + koff;
  const T* V = static_cast<const T*>(p.v) + koff;
  const size_t off = (static_cast<size_t>(s.start + i) * p.H + h) * D;
  for (int d = lane; d < D; d += 32) qs[warp][d] = to_f(static_cast<const T*>(p.q)[off + d]);
  __syncwarp();
  const float slope = sh.slopes ? sh.slopes[h] : 0.f;
  const KeyRange kr = key_range(p, sh, s, i);
  float m = -INFINITY, l = 0.f, acc[PER] = {};
  for (int c0 = kr.lo; c0 < kr.hi; c0 += 32) {
    const int j = c0 + lane;
    float z = -INFINITY, unused;
    if (j < kr.hi) z = shape(p, sh, slope, dot_row(qs[warp], K + j * kv_stride, D), i - j, unused);
    const float m_new = fmaxf(m, warp_max(z));
    const float m_use = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = expf(m - m_use);
    const float pj = j < kr.hi ? expf(z - m_use) : 0.f;
    l = l * alpha + warp_sum(pj);
#pragma unroll
    for (int t = 0; t < PER; ++t) acc[t] *= alpha;
    for (int jj = 0; jj < min(32, kr.hi - c0); ++jj) {
      const float pb = __shfl_sync(FULL, pj, jj);
#pragma unroll
      for (int t = 0; t < PER; ++t)
        if (lane + 32 * t < D) acc[t] = fmaf(pb, to_f(V[(c0 + jj) * kv_stride + lane + 32 * t]), acc[t]);
    }
    m = m_new;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int t = 0; t < PER; ++t)
    if (lane + 32 * t < D) put(static_cast<T*>(p.o) + off + lane + 32 * t, acc[t] * inv);
  if (lane == 0) p.lse[lse_index(p, b, h, s.start, i)] = l > 0.f ? m + logf(l) : -INFINITY;
}

// D_i = dO_i . O_i, [H, T].
template <typename T>
__global__ void __launch_bounds__(WARPS * 32) delta_kernel(AttnParams p) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int h = blockIdx.y;
  const SeqInfo s = seq_info(p, blockIdx.z);
  if (!seq_ok(p, s)) return;
  const int i = blockIdx.x * WARPS + warp;
  if (i >= s.len) return;
  const size_t off = (static_cast<size_t>(s.start + i) * p.H + h) * p.D;
  float acc = 0.f;
  for (int d = lane; d < p.D; d += 32)
    acc = fmaf(to_f(static_cast<const T*>(p.o)[off + d]), to_f(static_cast<const T*>(p.dout)[off + d]), acc);
  acc = warp_sum(acc);
  if (lane == 0) p.delta[static_cast<size_t>(h) * p.total + s.start + i] = acc;
}

template <typename T>
__global__ void __launch_bounds__(WARPS * 32) dq_kernel(AttnParams p, ShapeArgs sh) {
  __shared__ float qs[WARPS][DMAX], gs[WARPS][DMAX];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int b = blockIdx.z, h = blockIdx.y;
  const SeqInfo s = seq_info(p, b);
  if (!seq_ok(p, s)) return;
  const int i = blockIdx.x * WARPS + warp;
  if (i >= s.len) return;
  const int D = p.D, hk = h / (p.H / p.H_kv);
  const size_t kv_stride = static_cast<size_t>(p.H_kv) * D;
  const size_t koff = (static_cast<size_t>(s.start) * p.H_kv + hk) * D;
  const T* K = static_cast<const T*>(p.k) + koff;
  const T* V = static_cast<const T*>(p.v) + koff;
  const size_t off = (static_cast<size_t>(s.start + i) * p.H + h) * D;
  for (int d = lane; d < D; d += 32) {
    qs[warp][d] = to_f(static_cast<const T*>(p.q)[off + d]);
    gs[warp][d] = to_f(static_cast<const T*>(p.dout)[off + d]);
  }
  __syncwarp();
  const float slope = sh.slopes ? sh.slopes[h] : 0.f;
  const float lse = p.lse[lse_index(p, b, h, s.start, i)];
  const float dlt = p.delta[static_cast<size_t>(h) * p.total + s.start + i];
  const KeyRange kr = key_range(p, sh, s, i);
  float acc[PER] = {};
  for (int c0 = kr.lo; c0 < kr.hi; c0 += 32) {
    const int j = c0 + lane;
    float ds = 0.f;
    if (j < kr.hi) {
      float grad;
      const float z = shape(p, sh, slope, dot_row(qs[warp], K + j * kv_stride, D), i - j, grad);
      ds = expf(z - lse) * (dot_row(gs[warp], V + j * kv_stride, D) - dlt) * grad;
    }
    for (int jj = 0; jj < min(32, kr.hi - c0); ++jj) {
      const float dsb = __shfl_sync(FULL, ds, jj);
#pragma unroll
      for (int t = 0; t < PER; ++t)
        if (lane + 32 * t < D) acc[t] = fmaf(dsb, to_f(K[(c0 + jj) * kv_stride + lane + 32 * t]), acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < PER; ++t)
    if (lane + 32 * t < D) put(static_cast<T*>(p.dq) + off + lane + 32 * t, acc[t] * p.scale);
}

// Every query of the sequence is visited: a range tells which keys a query
// sees, not which queries see a key.
template <typename T>
__global__ void __launch_bounds__(WARPS * 32) dkdv_kernel(AttnParams p, ShapeArgs sh) {
  __shared__ float ks[WARPS][DMAX], vs[WARPS][DMAX];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int b = blockIdx.z, hk = blockIdx.y;
  const SeqInfo s = seq_info(p, b);
  if (!seq_ok(p, s)) return;
  const int j = blockIdx.x * WARPS + warp;
  if (j >= s.len) return;
  const int D = p.D, g = p.H / p.H_kv;
  const size_t q_stride = static_cast<size_t>(p.H) * D;
  const size_t koff = (static_cast<size_t>(s.start + j) * p.H_kv + hk) * D;
  for (int d = lane; d < D; d += 32) {
    ks[warp][d] = to_f(static_cast<const T*>(p.k)[koff + d]);
    vs[warp][d] = to_f(static_cast<const T*>(p.v)[koff + d]);
  }
  __syncwarp();
  float dk[PER] = {}, dv[PER] = {};
  for (int h = hk * g; h < (hk + 1) * g; ++h) {
    const float slope = sh.slopes ? sh.slopes[h] : 0.f;
    const T* Q = static_cast<const T*>(p.q) + (static_cast<size_t>(s.start) * p.H + h) * D;
    const T* G = static_cast<const T*>(p.dout) + (static_cast<size_t>(s.start) * p.H + h) * D;
    for (int c0 = p.causal ? j : 0; c0 < s.len; c0 += 32) {
      const int i = c0 + lane;
      float pij = 0.f, ds = 0.f;
      if (i < s.len) {
        const KeyRange kr = key_range(p, sh, s, i);
        if (j >= kr.lo && j < kr.hi) {
          float grad;
          const float z = shape(p, sh, slope, dot_row(ks[warp], Q + i * q_stride, D), i - j, grad);
          pij = expf(z - p.lse[lse_index(p, b, h, s.start, i)]);
          ds = pij * grad * (dot_row(vs[warp], G + i * q_stride, D) -
                             p.delta[static_cast<size_t>(h) * p.total + s.start + i]);
        }
      }
      if (!__any_sync(FULL, pij != 0.f)) continue;
      for (int ii = 0; ii < min(32, s.len - c0); ++ii) {
        const float pb = __shfl_sync(FULL, pij, ii);
        const float dsb = __shfl_sync(FULL, ds, ii);
#pragma unroll
        for (int t = 0; t < PER; ++t)
          if (lane + 32 * t < D) {
            dv[t] = fmaf(pb, to_f(G[(c0 + ii) * q_stride + lane + 32 * t]), dv[t]);
            dk[t] = fmaf(dsb, to_f(Q[(c0 + ii) * q_stride + lane + 32 * t]), dk[t]);
          }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < PER; ++t)
    if (lane + 32 * t < D) {
      put(static_cast<T*>(p.dk) + koff + lane + 32 * t, dk[t] * p.scale);
      put(static_cast<T*>(p.dv) + koff + lane + 32 * t, dv[t]);
    }
}

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

template <typename T>
cudaError_t fwd_t(const AttnParams& p, const ShapeArgs& sh, cudaStream_t stream) {
  fwd_kernel<T><<<dim3((p.max_seqlen + WARPS - 1) / WARPS, p.H, p.B), WARPS * 32, 0, stream>>>(p, sh);
  return cudaGetLastError();
}

template <typename T>
cudaError_t bwd_t(const AttnParams& p, const ShapeArgs& sh, cudaStream_t stream) {
  const int rows = (p.max_seqlen + WARPS - 1) / WARPS;
  delta_kernel<T><<<dim3(rows, p.H, p.B), WARPS * 32, 0, stream>>>(p);
  dq_kernel<T><<<dim3(rows, p.H, p.B), WARPS * 32, 0, stream>>>(p, sh);
  dkdv_kernel<T><<<dim3(rows, p.H_kv, p.B), WARPS * 32, 0, stream>>>(p, sh);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_shaped_fwd_simt(const AttnParams& p, const ShapeArgs& sh, bool f32,
                                   cudaStream_t stream) {
  return f32 ? fwd_t<float>(p, sh, stream) : fwd_t<__nv_bfloat16>(p, sh, stream);
}

cudaError_t launch_shaped_bwd_simt(const AttnParams& p, const ShapeArgs& sh, bool f32,
                                   cudaStream_t stream) {
  return f32 ? bwd_t<float>(p, sh, stream) : bwd_t<__nv_bfloat16>(p, sh, stream);
}

cudaError_t launch_key_ranges(const AttnParams& p, const int* doc_ids, const int* prefix_lens,
                              int window, int* key_begin, int* key_end, cudaStream_t stream) {
  key_ranges_kernel<<<p.B, 1024, 0, stream>>>(p, doc_ids, prefix_lens, window, key_begin, key_end);
  return cudaGetLastError();
}

}  // namespace fa
