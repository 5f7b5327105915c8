// Attention with shaped scores: what the kernels of fa_fwd_shaped,
// fa_bwd_shaped, fa_decode_shaped and fa_cache_evict share.
//
// The scores of include/fa.h, "Shaped scores":
//     z_ij = cap tanh(scale q_i.k_j / cap) - slope_h |i - j|,
// key j visible to query i iff begin_i <= j < end_i (and j <= i when causal).
#pragma once

#include <atomic>

#include "params.h"

namespace fa {

struct ShapeArgs {
  float cap;               // 0: no cap
  float scale_over_cap;    // scale / cap (cap > 0)
  const float* slopes;     // [H] or null
  const int* key_begin;    // [T] or null
  const int* key_end;      // [T] or null
};

// Visible keys [lo, hi) of the query at position i of a sequence; an empty
// range is returned as [0, 0). Ranges reaching outside the sequence are
// clipped to it.
struct KeyRange {
  int lo, hi;
};

__device__ __forceinline__ KeyRange key_range(const AttnParams& p, const ShapeArgs& sh,
                                              const SeqInfo& s, int i) {
  int lo = 0, hi = s.len;
  if (sh.key_begin != nullptr) lo = max(0, __ldg(sh.key_begin + s.start + i));
  if (sh.key_end != nullptr) hi = min(hi, __ldg(sh.key_end + s.start + i));
  if (p.causal) hi = min(hi, i + 1);
  if (lo >= hi) lo = hi = 0;
  return {lo, hi};
}

// First entry of sequence b in the array of its 128-row query tiles' ranges: sequences
// take ceil(len / 128) <= floor((start + len) / 128) - floor(start / 128) + 1 entries.
__device__ __forceinline__ long long tile_base(const SeqInfo& s, int b) { return s.start / 128 + b; }

// In a kernel launched before the one ahead of it in the stream has ended: until it has,
// and its writes are seen. (Every CTA of such a kernel waits: its end stands for both.)
__device__ __forceinline__ void wait_for_primary() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Lets the next kernel's CTAs take free places once every CTA of this grid has come here.
__device__ __forceinline__ void release_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Decode over a cache: what fa_decode_shape adds to a decode's arguments.
struct DecodeShapeArgs {
  float cap;
  float scale_over_cap;
  const float* slopes;         // [H] or null
  int window;                  // 0: none
  const int* key_positions;    // [B, H_kv, slots] or null: the slot is the position
  float* key_weights;          // [B, H_kv, slots] or null
  long long slots;
};

// Eviction: keep the last ``recent`` slots and the heaviest others.
struct EvictArgs {
  const void* k;
  const void* v;
  const int* cache_seqlens;
  const int* block_table;      // null: contiguous
  int B, H_kv, D;
  int page, max_blocks;
  long long cache_rows;
  int max_len;
  const float* key_weights;    // [B, H_kv, slots]
  const int* key_positions;    // [B, H_kv, slots] or null
  long long slots;
  int keep, recent;
  void* k_out;
  void* v_out;
  const int* out_table;        // null: contiguous
  int out_page, out_max_blocks;
  long long out_rows;
  int* seqlens_out;            // [B]
  float* weights_out;          // [B, H_kv, out_slots]
  int* positions_out;          // [B, H_kv, out_slots]
  long long out_slots;
  int* src;                    // workspace: [B, H_kv, keep] slots kept, ascending
  DevErr err;
};

// Cache row of slot j of sequence b (include/fa.h, fa_decode), or -1 for a
// block-table entry outside the cache.
__device__ __forceinline__ long long cache_row(const int* table, int max_blocks, int page,
                                               long long rows, int b, int j) {
  long long r;
  if (table == nullptr) {
    r = static_cast<long long>(b) * page + j;
  } else {
    const int pg = j / page;
    if (pg >= max_blocks) return -1;
    r = static_cast<long long>(__ldg(table + static_cast<size_t>(b) * max_blocks + pg)) * page +
        j % page;
  }
  return (r >= 0 && r < rows) ? r : -1;
}

__device__ __forceinline__ void record_bounds(const DevErr& e, unsigned where) {
  atomicOr(e.word, ERR_BOUNDS);
  atomicExch(e.word + 1, where);
}

// Host: lets ``Kernel`` have up to ``bytes`` of dynamic shared memory, once per device.
template <auto Kernel>
inline cudaError_t allow_smem(int bytes) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  const cudaError_t got = cudaGetDevice(&dev);
  if (got != cudaSuccess) return got;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// float32 (shaped_f32.cu).
cudaError_t launch_shaped_fwd_f32(const AttnParams& p, const ShapeArgs& sh, cudaStream_t stream);
cudaError_t launch_shaped_bwd_f32(const AttnParams& p, const ShapeArgs& sh, cudaStream_t stream);
// bf16, D = 64 or 128 (shaped_fwd.cu).
cudaError_t launch_shaped_fwd(const AttnParams& p, const ShapeArgs& sh, cudaStream_t stream);
// bf16: p.delta = D_i, zeroes in p.dq_accum, and unless null the query tiles' key ranges
// at tile_base (shaped_delta.cu).
cudaError_t launch_shaped_delta(const AttnParams& p, const ShapeArgs& sh, int2* tiles,
                                cudaStream_t stream);
// bf16, D = 64 or 128 (shaped_bwd.cu): p.delta and p.dq_accum as for the fused
// backward, ``tiles`` shaped_bwd_tiles_bytes() of scratch.
size_t shaped_bwd_tiles_bytes(long long total, int B);
cudaError_t launch_shaped_bwd(const AttnParams& p, const ShapeArgs& sh, void* tiles,
                              cudaStream_t stream);
cudaError_t launch_key_ranges(const AttnParams& p, const int* doc_ids, const int* prefix_lens,
                              int window, int* key_begin, int* key_end, cudaStream_t stream);
// n_rows = q_len H / H_kv <= 64, D = 64 or 128 (decode_shaped.cu). ``max_len``: under a
// window no more than DecodeShapeArgs::window + q_len + 127.
size_t decode_shaped_workspace(long long B, int H_kv, long long n_rows, int D, int max_len,
                               bool weights);
cudaError_t launch_decode_shaped(const AttnParams& p, const DecodeArgs& d,
                                 const DecodeShapeArgs& sh, void* workspace, cudaStream_t stream);
// Its second kernel alone: the merge, and the weights.
cudaError_t launch_decode_finish(const AttnParams& p, const DecodeArgs& d,
                                 const DecodeShapeArgs& sh, void* workspace, cudaStream_t stream);
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream);

}  // namespace fa
