// C ABI of the shaped-score entry points and the cache eviction (declared in
// include/fa.h): host-side argument checks and dispatch.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/fa.h"
#include "host.h"
#include "shaped.h"

namespace fa {
namespace {

bool plain(const fa_score_shape* s) {
  return s == nullptr || (s->softcap == 0.f && s->alibi_slopes == nullptr &&
                          s->key_begin == nullptr && s->key_end == nullptr);
}

// Bounds within which cap, scale / cap and their products stay in fp32's range.
bool cap_ok(float cap, float scale) {
  return cap == 0.f || (cap > 0.f && cap <= 0x1p100f && scale / cap <= 0x1p100f);
}

ShapeArgs shape_args(const fa_score_shape& s, float scale) {
  ShapeArgs a = {};
  a.cap = s.softcap;
  a.scale_over_cap = s.softcap > 0.f ? scale / s.softcap : 0.f;
  a.slopes = s.alibi_slopes;
  a.key_begin = s.key_begin;
  a.key_end = s.key_end;
  return a;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

}  // namespace
}  // namespace fa

using fa::AttnParams;

extern "C" {

fa_status fa_fwd_shaped(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                        int H, int H_kv, int N, int D, fa_dtype dtype, int causal, float scale,
                        const int* cu_seqlens, int max_seqlen, long long total_tokens,
                        const fa_score_shape* shape, fa_stream_t stream) {
  if (fa::plain(shape))
    return fa_fwd(q, k, v, o, lse, B, H, H_kv, N, D, dtype, causal, scale, cu_seqlens, max_seqlen,
                  total_tokens, stream);
  AttnParams p = {};
  const fa_status st = fa::check_common(p, B, H, H_kv, N, D, dtype, causal, scale, cu_seqlens,
                                        max_seqlen, total_tokens);
  if (st != FA_OK) return st;
  if (!fa::cap_ok(shape->softcap, p.scale)) return FA_ERR_INVALID_ARG;
  if (p.total == 0 || p.max_seqlen == 0 || B == 0) return FA_OK;
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!fa::aligned16(q) || !fa::aligned16(k) || !fa::aligned16(v) || !fa::aligned16(o))
    return FA_ERR_INVALID_ARG;
  p.q = q;
  p.k = k;
  p.v = v;
  p.o = o;
  p.lse = lse;
  p.err.word = fa::err_word();
  if (p.err.word == nullptr) return FA_ERR_CUDA;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const fa::ShapeArgs a = fa::shape_args(*shape, p.scale);
  return fa::record_cuda(dtype == FA_F32 ? fa::launch_shaped_fwd_f32(p, a, s)
                                         : fa::launch_shaped_fwd(p, a, s));
}

size_t fa_bwd_shaped_workspace_size(long long total_tokens, int B, int H, int D, fa_dtype dtype) {
  const size_t base = fa_bwd_workspace_size(total_tokens, H, D, dtype);
  if (B < 0 || base == 0) return 0;
  return base + (dtype == FA_BF16 ? fa::round256(fa::shaped_bwd_tiles_bytes(total_tokens, B)) : 0);
}

fa_status fa_bwd_shaped(const void* q, const void* k, const void* v, const void* o,
                        const float* lse, const void* dout, void* dq, void* dk, void* dv, int B,
                        int H, int H_kv, int N, int D, fa_dtype dtype, int causal, float scale,
                        const int* cu_seqlens, int max_seqlen, long long total_tokens,
                        const fa_score_shape* shape, void* workspace, size_t ws_bytes,
                        fa_stream_t stream) {
  if (fa::plain(shape))
    return fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, B, H, H_kv, N, D, dtype, causal, scale,
                  cu_seqlens, max_seqlen, total_tokens, workspace, ws_bytes, stream);
  AttnParams p = {};
  const fa_status st = fa::check_common(p, B, H, H_kv, N, D, dtype, causal, scale, cu_seqlens,
                                        max_seqlen, total_tokens);
  if (st != FA_OK) return st;
  if (!fa::cap_ok(shape->softcap, p.scale)) return FA_ERR_INVALID_ARG;
  if (p.total == 0 || p.max_seqlen == 0 || B == 0) return FA_OK;
  if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv || !workspace)
    return FA_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, v, o, dout, dq, dk, dv};
  for (const void* ptr : ptrs)
    if (!fa::aligned16(ptr)) return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return FA_ERR_INVALID_ARG;
  if (ws_bytes < fa_bwd_shaped_workspace_size(p.total, B, H, D, dtype)) return FA_ERR_INVALID_ARG;
  p.q = q;
  p.k = k;
  p.v = v;
  p.o = const_cast<void*>(o);
  p.lse = const_cast<float*>(lse);
  p.dout = dout;
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  char* ws = static_cast<char*>(workspace);
  p.delta = reinterpret_cast<float*>(ws);
  p.err.word = fa::err_word();
  if (p.err.word == nullptr) return FA_ERR_CUDA;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const fa::ShapeArgs a = fa::shape_args(*shape, p.scale);
  if (dtype == FA_F32) return fa::record_cuda(fa::launch_shaped_bwd_f32(p, a, s));
  // D_i, the dQ accumulator, the query tiles' ranges.
  const size_t rows = static_cast<size_t>(p.total) * H;
  ws += fa::round256(rows * sizeof(float));
  p.dq_accum = reinterpret_cast<float*>(ws);
  ws += fa::round256(rows * D * sizeof(float));
  return fa::record_cuda(fa::launch_shaped_bwd(p, a, ws, s));
}

fa_status fa_key_ranges(const int* doc_ids, const int* prefix_lens, int window, int causal, int B,
                        int N, const int* cu_seqlens, int max_seqlen, long long total_tokens,
                        int* key_begin, int* key_end, fa_stream_t stream) {
  AttnParams p = {};
  const fa_status st = fa::check_common(p, B, 1, 1, N, 1, FA_F32, causal, 1.f, cu_seqlens,
                                        max_seqlen, total_tokens);
  if (st != FA_OK) return st;
  if (window < 0 || (prefix_lens != nullptr && !causal)) return FA_ERR_INVALID_ARG;
  if (p.total == 0 || p.max_seqlen == 0 || B == 0) return FA_OK;
  if (!key_begin || !key_end) return FA_ERR_INVALID_ARG;
  p.err.word = fa::err_word();
  if (p.err.word == nullptr) return FA_ERR_CUDA;
  return fa::record_cuda(fa::launch_key_ranges(p, doc_ids, prefix_lens, window, key_begin, key_end,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

size_t fa_decode_shaped_workspace_size(int B, int q_len, int H, int H_kv, int D, int max_seqlen_k,
                                       int weights) {
  if (B <= 0 || q_len <= 0 || H <= 0 || H_kv <= 0 || D <= 0 || max_seqlen_k < 0) return 0;
  const long long rows = static_cast<long long>(q_len) * (H / H_kv);
  if (H % H_kv != 0 || rows > 64) return 0;
  return fa::decode_shaped_workspace(B, H_kv, rows, D, max_seqlen_k, weights != 0);
}

fa_status fa_decode_shaped(const void* q, const void* k_cache, const void* v_cache, void* o,
                           float* lse, const int* cache_seqlens, const int* block_table, int B,
                           int q_len, int H, int H_kv, int D, int page_size, int max_blocks,
                           long long cache_rows, int max_seqlen_k, int causal, float scale,
                           const fa_decode_shape* shape, void* workspace, size_t ws_bytes,
                           fa_stream_t stream) {
  if (shape == nullptr) return FA_ERR_INVALID_ARG;
  AttnParams p = {};
  fa::DecodeArgs d = {};
  bool empty = false;
  if (shape->window < 0) return FA_ERR_INVALID_ARG;
  const fa_status st = fa::check_decode(p, d, empty, q, k_cache, v_cache, o, lse, cache_seqlens,
                                        block_table, B, q_len, H, H_kv, D, page_size, max_blocks,
                                        cache_rows, max_seqlen_k, causal, scale);
  if (st != FA_OK) return st;
  // (An empty call's scale was not resolved; any positive one will do.)
  if (!fa::cap_ok(shape->softcap, empty ? 1.f : p.scale)) return FA_ERR_INVALID_ARG;
  if (empty) return st;
  if (d.n_rows > 64) return FA_ERR_UNSUPPORTED;
  if ((shape->key_positions || shape->key_weights) && shape->slots < max_seqlen_k)
    return FA_ERR_INVALID_ARG;
  // Under a window the tiles of its window + q_len - 1 slots, which may start inside one.
  const long long span = shape->window > 0 ? shape->window + q_len + 127ll : max_seqlen_k;
  const size_t need = fa_decode_shaped_workspace_size(
      B, q_len, H, H_kv, D, static_cast<int>(std::min<long long>(max_seqlen_k, span)),
      shape->key_weights != nullptr);
  if (need > 0 && (workspace == nullptr || ws_bytes < need || !fa::aligned16(workspace)))
    return FA_ERR_INVALID_ARG;
  p.err.word = fa::err_word();
  if (p.err.word == nullptr) return FA_ERR_CUDA;
  fa::DecodeShapeArgs a = {};
  a.cap = shape->softcap;
  a.scale_over_cap = a.cap > 0.f ? p.scale / a.cap : 0.f;
  a.slopes = shape->alibi_slopes;
  a.window = shape->window;
  a.key_positions = shape->key_positions;
  a.key_weights = shape->key_weights;
  a.slots = shape->slots;
  return fa::record_cuda(
      fa::launch_decode_shaped(p, d, a, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

fa_status fa_selftest_decode_finish(void* o, float* lse, const int* cache_seqlens, int B,
                                    int q_len, int H, int H_kv, int D, int max_seqlen_k,
                                    float* key_weights, long long slots, void* workspace,
                                    size_t ws_bytes, fa_stream_t stream) {
  AttnParams p = {};
  fa::DecodeArgs d = {};
  bool empty = false;
  const fa_status st = fa::check_decode(p, d, empty, o, o, o, o, lse, cache_seqlens, nullptr, B,
                                        q_len, H, H_kv, D, max_seqlen_k, 0,
                                        static_cast<long long>(B) * max_seqlen_k, max_seqlen_k, 1,
                                        0.f);
  if (st != FA_OK || empty) return st;
  if (d.n_rows > 64) return FA_ERR_UNSUPPORTED;
  if (!key_weights || slots < max_seqlen_k) return FA_ERR_INVALID_ARG;
  if (workspace == nullptr || !fa::aligned16(workspace) ||
      ws_bytes < fa_decode_shaped_workspace_size(B, q_len, H, H_kv, D, max_seqlen_k, 1))
    return FA_ERR_INVALID_ARG;
  p.err.word = fa::err_word();
  if (p.err.word == nullptr) return FA_ERR_CUDA;
  fa::DecodeShapeArgs a = {};
  a.key_weights = key_weights;
  a.slots = slots;
  return fa::record_cuda(
      fa::launch_decode_finish(p, d, a, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

size_t fa_cache_evict_workspace_size(int B, int H_kv, int keep) {
  if (B <= 0 || H_kv <= 0 || keep <= 0) return 0;
  return fa::round256(static_cast<size_t>(B) * H_kv * keep * 4);
}

fa_status fa_cache_evict(const void* k_cache, const void* v_cache, const int* cache_seqlens,
                         const int* block_table, int B, int H_kv, int D, int page_size,
                         int max_blocks, long long cache_rows, int max_seqlen_k,
                         const float* key_weights, const int* key_positions, long long slots,
                         int keep, int recent, void* k_out, void* v_out,
                         const int* out_block_table, int out_page_size, int out_max_blocks,
                         long long out_rows, int* seqlens_out, float* weights_out,
                         int* positions_out, long long out_slots, void* workspace,
                         size_t ws_bytes, fa_stream_t stream) {
  if (B < 0 || H_kv <= 0 || D <= 0 || max_seqlen_k < 0 || cache_rows < 0 || out_rows < 0 ||
      keep <= 0 || recent < 0 || recent > keep)
    return FA_ERR_INVALID_ARG;
  if (D % 8 != 0 || D > 256) return FA_ERR_UNSUPPORTED;
  if (cache_rows >= (1ll << 31) || out_rows >= (1ll << 31) ||
      static_cast<long long>(B) * H_kv > (1ll << 24))
    return FA_ERR_UNSUPPORTED;
  if (B == 0) return FA_OK;
  fa_status st = fa::check_cache(B, block_table, page_size, max_blocks, cache_rows, max_seqlen_k);
  if (st != FA_OK) return st;
  const int most = std::min(keep, max_seqlen_k);   // longest sequence afterwards
  st = fa::check_cache(B, out_block_table, out_page_size, out_max_blocks, out_rows, most);
  if (st != FA_OK) return st;
  if (slots < max_seqlen_k || out_slots < most) return FA_ERR_INVALID_ARG;
  if (!k_cache || !v_cache || !cache_seqlens || !key_weights || !k_out || !v_out ||
      !seqlens_out || !weights_out || !positions_out)
    return FA_ERR_INVALID_ARG;
  const void* ptrs[] = {k_cache, v_cache, k_out, v_out};
  for (const void* ptr : ptrs)
    if (!fa::aligned16(ptr)) return FA_ERR_INVALID_ARG;
  const size_t need = fa_cache_evict_workspace_size(B, H_kv, keep);
  if (workspace == nullptr || ws_bytes < need || !fa::aligned16(workspace))
    return FA_ERR_INVALID_ARG;
  // Rows move while others are read: the two caches may share memory only as
  // pages of one pool.
  const size_t row = static_cast<size_t>(H_kv) * D * 2;
  if (fa::overlap(k_out, out_rows * row, v_out, out_rows * row)) return FA_ERR_INVALID_ARG;
  if (block_table == nullptr || out_block_table == nullptr) {
    const void* from[] = {k_cache, v_cache};
    const void* to[] = {k_out, v_out};
    for (const void* f : from)
      for (const void* t : to)
        if (fa::overlap(f, cache_rows * row, t, out_rows * row)) return FA_ERR_INVALID_ARG;
  }
  fa::EvictArgs a = {};
  a.k = k_cache;
  a.v = v_cache;
  a.cache_seqlens = cache_seqlens;
  a.block_table = block_table;
  a.B = B;
  a.H_kv = H_kv;
  a.D = D;
  a.page = page_size;
  a.max_blocks = max_blocks;
  a.cache_rows = cache_rows;
  a.max_len = max_seqlen_k;
  a.key_weights = key_weights;
  a.key_positions = key_positions;
  a.slots = slots;
  a.keep = keep;
  a.recent = recent;
  a.k_out = k_out;
  a.v_out = v_out;
  a.out_table = out_block_table;
  a.out_page = out_page_size;
  a.out_max_blocks = out_max_blocks;
  a.out_rows = out_rows;
  a.seqlens_out = seqlens_out;
  a.weights_out = weights_out;
  a.positions_out = positions_out;
  a.out_slots = out_slots;
  a.src = static_cast<int*>(workspace);
  a.err.word = fa::err_word();
  if (a.err.word == nullptr) return FA_ERR_CUDA;
  return fa::record_cuda(fa::launch_evict(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
