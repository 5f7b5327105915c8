// Attention with shaped scores in float32 on CUDA cores (tensor-core operands would
// round to tf32): one warp per query row (forward, dQ) or key row (dK, dV), eight rows
// a CTA.
//
//     z = cap tanh(scale q.k / cap) - slope |i - j|,  O = softmax(z) V,
//     P = exp(z - LSE), dV = P^T dO, dZ = P (dO V^T - D), D_i = dO_i . O_i,
//     dX = dZ (1 - tanh^2), dQ = scale dX K, dK = scale dX^T Q.
//
// The other side's rows come through shared memory, 32 at a time, loaded once for the
// CTA's eight rows, in rows of D + 4 floats: a lane that owns a row reads it four floats
// at a time without bank conflicts, and the second product reads the same rows along D,
// four columns a lane, the keys split over the lanes that D leaves over. Two buffers: the
// next 32 rows are on their way while these are worked on. Small heads and
// short sequences are bound by latency: three launches in all for a step (dQ's kernel
// makes the D_i that dK's reads).
#include <math.h>

#include <algorithm>

#include "shaped.h"

namespace fa {
namespace {
namespace f32 {

constexpr unsigned FULL = 0xffffffffu;
constexpr int WARPS = 8;
constexpr int THREADS = WARPS * 32;
constexpr int TK = 32;              // rows of the other side per tile
constexpr int DMAX = 128;
constexpr int LD = DMAX + 4;        // floats of a row in shared memory

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

// Shared memory of a CTA: two buffers of two tiles, and its own rows' two operands.
struct Shared {
  float a[2][TK][LD], b[2][TK][LD];
  float own_a[WARPS][DMAX], own_b[WARPS][DMAX];
  int range[2];
};

// dkdv_kernel: PARTS steps at a time.
template <int PARTS>
struct SharedSteps {
  float a[2][PARTS][TK][LD], b[2][PARTS][TK][LD];   // [buffer][part]
  float own_a[WARPS][DMAX], own_b[WARPS][DMAX];
  unsigned seen;   // which of 32 query tiles see a key of the CTA
};

// n rows (row stride ``stride``) of D floats into shared rows, 16 bytes at a time without
// waiting where D allows; the rest of 32 rows and of D4 = D rounded up to four are zeros.
template <int NT = THREADS>
__device__ __forceinline__ void load_rows(float (*dst)[LD], const float* src, size_t stride, int n,
                                          int D, int D4) {
  if ((D & 3) == 0) {
    const int units = D4 / 4;
    for (int t = threadIdx.x; t < TK * units; t += NT) {
      const int r = t / units, u = t % units;
      const int bytes = r < n ? 16 : 0;   // 0: the 16 bytes become zeros
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(&dst[r][4 * u])),
                   "l"(src + (r < n ? r * stride + 4 * u : 0)), "r"(bytes)
                   : "memory");
    }
  } else {
    for (int t = threadIdx.x; t < TK * D4; t += NT) {
      const int r = t / D4, d = t % D4;
      dst[r][d] = (r < n && d < D) ? src[r * stride + d] : 0.f;
    }
  }
}

__device__ __forceinline__ void loads_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest group have landed.
__device__ __forceinline__ void loads_wait() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// A warp's own row, zeros up to D4.
__device__ __forceinline__ void load_own(float* dst, const float* src, int D, int D4) {
  for (int d = threadIdx.x % 32; d < D4; d += 32) dst[d] = d < D ? src[d] : 0.f;
}

__device__ __forceinline__ float dot(const float* a, const float* b, int D4) {
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int d = 0; d < D4; d += 4) {
    const float4 x = *reinterpret_cast<const float4*>(a + d);
    const float4 y = *reinterpret_cast<const float4*>(b + d);
    s.x = fmaf(x.x, y.x, s.x);
    s.y = fmaf(x.y, y.y, s.y);
    s.z = fmaf(x.z, y.z, s.z);
    s.w = fmaf(x.w, y.w, s.w);
  }
  return (s.x + s.y) + (s.z + s.w);
}

// Lanes of the second product: column unit u (four columns), rows sub, sub + G, ..
struct Lanes {
  int G, sub, u;
  bool on;
};
__device__ __forceinline__ Lanes lanes_of(int D4) {
  const int units = D4 / 4, lane = threadIdx.x % 32;
  const int G = units <= 8 ? 4 : units <= 16 ? 2 : 1;
  const int w = 32 / G;
  return {G, lane / w, lane % w, lane % w < units};
}

// acc += sum over the 32 rows r of p_r row_r (p_r in lane r).
template <int G>
__device__ __forceinline__ void add_rows_g(float4& acc, const Lanes& ln, float p, float (*rows)[LD]) {
#pragma unroll
  for (int r0 = 0; r0 < TK; r0 += G) {
    const int r = r0 + ln.sub;
    const float w = __shfl_sync(FULL, p, r);
    if (ln.on) {
      const float4 v = *reinterpret_cast<const float4*>(&rows[r][4 * ln.u]);
      acc.x = fmaf(w, v.x, acc.x);
      acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z);
      acc.w = fmaf(w, v.w, acc.w);
    }
  }
}

__device__ __forceinline__ void add_rows(float4& acc, const Lanes& ln, float p, float (*rows)[LD]) {
  if (ln.G == 1)
    add_rows_g<1>(acc, ln, p, rows);
  else if (ln.G == 2)
    add_rows_g<2>(acc, ln, p, rows);
  else
    add_rows_g<4>(acc, ln, p, rows);
}

// Adds the subs up and stores scale acc as D floats.
__device__ __forceinline__ void store_row(float* dst, float4 a, const Lanes& ln, int D, float scale) {
  for (int o = 32 / ln.G; o < 32; o <<= 1) {
    a.x += __shfl_xor_sync(FULL, a.x, o);
    a.y += __shfl_xor_sync(FULL, a.y, o);
    a.z += __shfl_xor_sync(FULL, a.z, o);
    a.w += __shfl_xor_sync(FULL, a.w, o);
  }
  if (ln.sub != 0 || !ln.on) return;
  const float v[4] = {a.x * scale, a.y * scale, a.z * scale, a.w * scale};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (4 * ln.u + e < D) dst[4 * ln.u + e] = v[e];
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

// [least lo, largest hi) over the CTA's rows; s_range is two ints of shared memory.
__device__ __forceinline__ KeyRange cta_range(const KeyRange& kr, int* s_range) {
  if (threadIdx.x == 0) {
    s_range[0] = 0x7fffffff;
    s_range[1] = 0;
  }
  __syncthreads();
  if (threadIdx.x % 32 == 0 && kr.lo < kr.hi) {
    atomicMin(&s_range[0], kr.lo);
    atomicMax(&s_range[1], kr.hi);
  }
  __syncthreads();
  return {s_range[0], s_range[1]};
}

__global__ void __launch_bounds__(THREADS) fwd_kernel(AttnParams p, ShapeArgs sh) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& sm = *reinterpret_cast<Shared*>(raw);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int b = blockIdx.z, h = blockIdx.y;
  const SeqInfo s = seq_info(p, b);
  if (!seq_ok(p, s) || static_cast<int>(blockIdx.x) * WARPS >= s.len) return;
  const int i = blockIdx.x * WARPS + warp;
  const bool row = i < s.len;
  const int D = p.D, D4 = (D + 3) & ~3, hk = h / (p.H / p.H_kv);
  const size_t kv_stride = static_cast<size_t>(p.H_kv) * D;
  const size_t koff = (static_cast<size_t>(s.start) * p.H_kv + hk) * D;
  const float* K = static_cast<const float*>(p.k) + koff;
  const float* V = static_cast<const float*>(p.v) + koff;
  const size_t off = (static_cast<size_t>(s.start + (row ? i : 0)) * p.H + h) * D;
  load_own(sm.own_a[warp], static_cast<const float*>(p.q) + off, D, D4);
  const float slope = sh.slopes ? sh.slopes[h] : 0.f;
  KeyRange kr = {0, 0};
  if (row) kr = key_range(p, sh, s, i);
  const KeyRange all = cta_range(kr, sm.range);
  const Lanes ln = lanes_of(D4);
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto fetch = [&](int c0, int buf) {
    if (c0 < all.hi) {
      const int n = min(TK, s.len - c0);
      load_rows(sm.a[buf], K + c0 * kv_stride, kv_stride, n, D, D4);
      load_rows(sm.b[buf], V + c0 * kv_stride, kv_stride, n, D, D4);
    }
    loads_commit();
  };
  fetch(all.lo, 0);
  for (int c0 = all.lo, buf = 0; c0 < all.hi; c0 += TK, buf ^= 1) {
    fetch(c0 + TK, buf ^ 1);
    loads_wait();
    __syncthreads();
    if (c0 < kr.hi && c0 + TK > kr.lo) {
      const int j = c0 + lane;
      const bool see = j >= kr.lo && j < kr.hi;
      float unused;
      const float z = see ? shape(p, sh, slope, dot(sm.own_a[warp], sm.a[buf][lane], D4), i - j, unused) : -INFINITY;
      const float m_new = fmaxf(m, warp_max(z));
      const float m_use = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = expf(m - m_use);
      const float pj = expf(z - m_use);
      l = l * alpha + warp_sum(pj);
      acc = make_float4(acc.x * alpha, acc.y * alpha, acc.z * alpha, acc.w * alpha);
      add_rows(acc, ln, pj, sm.b[buf]);
      m = m_new;
    }
    __syncthreads();
  }
  if (!row) return;
  store_row(static_cast<float*>(p.o) + off, acc, ln, D, l > 0.f ? 1.f / l : 0.f);
  if (lane == 0) p.lse[lse_index(p, b, h, s.start, i)] = l > 0.f ? m + logf(l) : -INFINITY;
}

// Also D_i, [H, T], for dkdv_kernel.
__global__ void __launch_bounds__(THREADS) dq_kernel(AttnParams p, ShapeArgs sh) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& sm = *reinterpret_cast<Shared*>(raw);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int b = blockIdx.z, h = blockIdx.y;
  const SeqInfo s = seq_info(p, b);
  if (!seq_ok(p, s) || static_cast<int>(blockIdx.x) * WARPS >= s.len) return;
  const int i = blockIdx.x * WARPS + warp;
  const bool row = i < s.len;
  const int D = p.D, D4 = (D + 3) & ~3, hk = h / (p.H / p.H_kv);
  const size_t kv_stride = static_cast<size_t>(p.H_kv) * D;
  const size_t koff = (static_cast<size_t>(s.start) * p.H_kv + hk) * D;
  const float* K = static_cast<const float*>(p.k) + koff;
  const float* V = static_cast<const float*>(p.v) + koff;
  const size_t off = (static_cast<size_t>(s.start + (row ? i : 0)) * p.H + h) * D;
  load_own(sm.own_a[warp], static_cast<const float*>(p.q) + off, D, D4);
  load_own(sm.own_b[warp], static_cast<const float*>(p.dout) + off, D, D4);
  float dlt = 0.f;
  for (int d = lane; d < D; d += 32)
    dlt = fmaf(static_cast<const float*>(p.o)[off + d], static_cast<const float*>(p.dout)[off + d], dlt);
  dlt = warp_sum(dlt);
  if (row && lane == 0) p.delta[static_cast<size_t>(h) * p.total + s.start + i] = dlt;
  const float slope = sh.slopes ? sh.slopes[h] : 0.f;
  const float lse = row ? p.lse[lse_index(p, b, h, s.start, i)] : 0.f;
  KeyRange kr = {0, 0};
  if (row) kr = key_range(p, sh, s, i);
  const KeyRange all = cta_range(kr, sm.range);
  const Lanes ln = lanes_of(D4);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto fetch = [&](int c0, int buf) {
    if (c0 < all.hi) {
      const int n = min(TK, s.len - c0);
      load_rows(sm.a[buf], K + c0 * kv_stride, kv_stride, n, D, D4);
      load_rows(sm.b[buf], V + c0 * kv_stride, kv_stride, n, D, D4);
    }
    loads_commit();
  };
  fetch(all.lo, 0);
  for (int c0 = all.lo, buf = 0; c0 < all.hi; c0 += TK, buf ^= 1) {
    fetch(c0 + TK, buf ^ 1);
    loads_wait();
    __syncthreads();
    if (c0 < kr.hi && c0 + TK > kr.lo) {
      const int j = c0 + lane;
      float dx = 0.f;
      if (j >= kr.lo && j < kr.hi) {
        float grad;
        const float z = shape(p, sh, slope, dot(sm.own_a[warp], sm.a[buf][lane], D4), i - j, grad);
        dx = expf(z - lse) * (dot(sm.own_b[warp], sm.b[buf][lane], D4) - dlt) * grad;
      }
      add_rows(acc, ln, dx, sm.a[buf]);
    }
    __syncthreads();
  }
  if (row) store_row(static_cast<float*>(p.dq) + off, acc, ln, D, p.scale);
}

// Every query of the sequence is looked at, 1024 at a time: a range tells which keys a
// query sees, not which queries see a key. Tiles of 32 queries that see none of the CTA's
// keys are not loaded. A key row's chain of (tile, head) steps is the longest of the three
// kernels', so with at most two CTAs a SM two warps share a row (PARTS 2), each with every
// other step, and add up at the end: backward of B1 H4/2 D64 N600 165 us against 187, N1100
// 327 against 423. With more CTAs the smaller shared memory of one warp a row lets more of
// them run (B4 H8/2 N512 D64: 826 against 951).
template <int PARTS>
__global__ void __launch_bounds__(PARTS* THREADS) dkdv_kernel(AttnParams p, ShapeArgs sh) {
  extern __shared__ __align__(16) uint8_t raw[];
  constexpr int NT = PARTS * THREADS;
  SharedSteps<PARTS>& sm = *reinterpret_cast<SharedSteps<PARTS>*>(raw);
  const int warp = threadIdx.x / 32 % WARPS, part = threadIdx.x / THREADS, lane = threadIdx.x % 32;
  const int b = blockIdx.z, hk = blockIdx.y;
  const SeqInfo s = seq_info(p, b);
  if (!seq_ok(p, s) || static_cast<int>(blockIdx.x) * WARPS >= s.len) return;
  const int j = blockIdx.x * WARPS + warp;
  const bool row = j < s.len;
  const int D = p.D, D4 = (D + 3) & ~3, g = p.H / p.H_kv;
  const size_t q_stride = static_cast<size_t>(p.H) * D;
  const size_t koff = (static_cast<size_t>(s.start + (row ? j : 0)) * p.H_kv + hk) * D;
  if (part == 0) load_own(sm.own_a[warp], static_cast<const float*>(p.k) + koff, D, D4);
  if (part == PARTS - 1) load_own(sm.own_b[warp], static_cast<const float*>(p.v) + koff, D, D4);
  const Lanes ln = lanes_of(D4);
  float4 dk = make_float4(0.f, 0.f, 0.f, 0.f), dv = dk;
  // Steps: the tiles of 32 queries that see a key of the CTA, and of each the g heads;
  // the next pair's rows load while this one's are worked on.
  const int base = p.causal ? static_cast<int>(blockIdx.x) * WARPS : 0;
  const bool ranged = sh.key_begin != nullptr || sh.key_end != nullptr;
  constexpr int GROUP = 32 * TK;
  unsigned bits = 0;
  int in_bits = -1;   // the group of 32 tiles that bits tells of
  struct Step {
    int t, h;     // tile (queries base + 32 t ..), head of the group
    bool on, see;
  };
  auto next = [&](Step st) {
    if (!st.on || (st.t >= 0 && ++st.h < g)) return st;
    st.h = 0;
    for (++st.t;;) {
      if (!ranged) {   // every tile from the first on sees them
        st.on = base + TK * st.t < s.len;
        if (!st.on) return st;
        break;
      }
      if (st.t / 32 != in_bits) {
        in_bits = st.t / 32;
        st.on = base + in_bits * GROUP < s.len;
        if (!st.on) return st;
        __syncthreads();
        if (threadIdx.x == 0) sm.seen = 0;
        __syncthreads();
        for (int x = threadIdx.x; x < GROUP; x += NT) {
          const int i = base + in_bits * GROUP + x;
          bool hit = false;
          if (i < s.len) {
            const KeyRange kr = key_range(p, sh, s, i);
            hit = kr.lo < kr.hi && kr.lo < (static_cast<int>(blockIdx.x) + 1) * WARPS &&
                  kr.hi > static_cast<int>(blockIdx.x) * WARPS;
          }
          if (__any_sync(FULL, hit) && lane == 0) atomicOr(&sm.seen, 1u << (x / TK));
        }
        __syncthreads();
        bits = sm.seen;
      }
      const unsigned rest = bits >> (st.t & 31);
      if (rest != 0) {
        st.t += __ffs(rest) - 1;
        break;
      }
      st.t = (in_bits + 1) * 32;
    }
    const int i = base + TK * st.t + lane;
    st.see = false;
    if (row && i < s.len) {
      const KeyRange kr = key_range(p, sh, s, i);
      st.see = j >= kr.lo && j < kr.hi;
    }
    return st;
  };
  auto fetch = [&](const Step& st, int buf, int k) {
    if (!st.on) return;
    const int c0 = base + TK * st.t;
    const size_t off = (static_cast<size_t>(s.start + c0) * p.H + hk * g + st.h) * D;
    const int n = min(TK, s.len - c0);
    load_rows<NT>(sm.a[buf][k], static_cast<const float*>(p.q) + off, q_stride, n, D, D4);
    load_rows<NT>(sm.b[buf][k], static_cast<const float*>(p.dout) + off, q_stride, n, D, D4);
  };
  Step st[PARTS];
#pragma unroll
  for (int k = 0; k < PARTS; ++k) {
    st[k] = next(k ? st[k - 1] : Step{-1, 0, true, false});
    fetch(st[k], 0, k);
  }
  loads_commit();
  for (int buf = 0; st[0].on; buf ^= 1) {
    Step nx[PARTS];
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
      nx[k] = next(k ? nx[k - 1] : st[PARTS - 1]);
      fetch(nx[k], buf ^ 1, k);
    }
    loads_commit();
    loads_wait();
    __syncthreads();
    const Step me = PARTS > 1 && part ? st[PARTS - 1] : st[0];
    if (me.on && __any_sync(FULL, me.see)) {
      float(*const qs)[LD] = sm.a[buf][part];
      float(*const gs)[LD] = sm.b[buf][part];
      const int i = base + TK * me.t + lane, h = hk * g + me.h;
      float pij = 0.f, dx = 0.f;
      if (me.see) {
        float grad;
        const float z = shape(p, sh, sh.slopes ? sh.slopes[h] : 0.f, dot(sm.own_a[warp], qs[lane], D4),
                              i - j, grad);
        pij = expf(z - p.lse[lse_index(p, b, h, s.start, i)]);
        dx = pij * grad * (dot(sm.own_b[warp], gs[lane], D4) -
                           p.delta[static_cast<size_t>(h) * p.total + s.start + i]);
      }
      add_rows(dv, ln, pij, gs);
      add_rows(dk, ln, dx, qs);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PARTS; ++k) st[k] = nx[k];
  }
  if constexpr (PARTS == 2) {
    float4* const other = reinterpret_cast<float4*>(&sm.a[0][0][0][0]) + warp * 64 + lane;
    if (part == 1) {
      other[0] = dk;
      other[32] = dv;
    }
    __syncthreads();
    if (part == 1) return;
    auto plus = [](float4& x, const float4& y) {
      x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
    };
    plus(dk, other[0]);
    plus(dv, other[32]);
  }
  if (!row) return;
  store_row(static_cast<float*>(p.dk) + koff, dk, ln, D, p.scale);
  store_row(static_cast<float*>(p.dv) + koff, dv, ln, D, 1.f);
}

template <int PARTS>
cudaError_t launch_dkdv(const AttnParams& p, const ShapeArgs& sh, int rows, cudaStream_t stream) {
  using S = SharedSteps<PARTS>;
  const cudaError_t e = allow_smem<dkdv_kernel<PARTS>>(sizeof(S));
  if (e != cudaSuccess) return e;
  dkdv_kernel<PARTS><<<dim3(rows, p.H_kv, p.B), PARTS * THREADS, sizeof(S), stream>>>(p, sh);
  return cudaGetLastError();
}

}  // namespace f32
}  // namespace

cudaError_t launch_shaped_fwd_f32(const AttnParams& p, const ShapeArgs& sh, cudaStream_t stream) {
  const int rows = (p.max_seqlen + f32::WARPS - 1) / f32::WARPS;
  const cudaError_t e = allow_smem<f32::fwd_kernel>(sizeof(f32::Shared));
  if (e != cudaSuccess) return e;
  f32::fwd_kernel<<<dim3(rows, p.H, p.B), f32::THREADS, sizeof(f32::Shared), stream>>>(p, sh);
  return cudaGetLastError();
}

cudaError_t launch_shaped_bwd_f32(const AttnParams& p, const ShapeArgs& sh, cudaStream_t stream) {
  const int rows = (p.max_seqlen + f32::WARPS - 1) / f32::WARPS;
  cudaError_t e = allow_smem<f32::dq_kernel>(sizeof(f32::Shared));
  if (e != cudaSuccess) return e;
  f32::dq_kernel<<<dim3(rows, p.H, p.B), f32::THREADS, sizeof(f32::Shared), stream>>>(p, sh);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // Two CTAs a SM: see dkdv_kernel.
  const bool few = static_cast<long long>(rows) * p.H_kv * p.B <= 2 * 148;
  return few ? f32::launch_dkdv<2>(p, sh, rows, stream) : f32::launch_dkdv<1>(p, sh, rows, stream);
}

}  // namespace fa
