// Host-side argument checks shared by the files of the C ABI (fa_api.cu,
// shaped_api.cu). Include after fa.h.
#pragma once

#include "params.h"

namespace fa {

bool aligned16(const void* p);
size_t round256(size_t x);

// Device address of the current device's error word (looked up once), or null.
unsigned* err_word();

// Checks of fa_fwd / fa_bwd; fills the size fields of ``p``.
fa_status check_common(AttnParams& p, int B, int H, int H_kv, int N, int D, fa_dtype dtype,
                       int causal, float scale, const int* cu_seqlens, int max_seqlen,
                       long long total_tokens);

// Checks of a cache's layout: FA_OK, or the status fa_decode returns.
fa_status check_cache(int B, const int* block_table, int page_size, int max_blocks,
                      long long cache_rows, int max_seqlen_k);

// Checks of fa_decode but for its workspace; fills ``p`` (without the error
// word) and ``d`` (without the split partials). ``empty``: nothing to do.
fa_status check_decode(AttnParams& p, DecodeArgs& d, bool& empty, const void* q,
                       const void* k_cache, const void* v_cache, void* o, float* lse,
                       const int* cache_seqlens, const int* block_table, int B, int q_len, int H,
                       int H_kv, int D, int page_size, int max_blocks, long long cache_rows,
                       int max_seqlen_k, int causal, float scale);

}  // namespace fa
