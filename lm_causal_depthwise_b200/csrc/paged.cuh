// paged.cuh -- what the two operators over a paged 8-bit key/value cache share.
//
// Cache: k_cache, v_cache [num_pages, Hkv, page_size, D] e4m3 codes, k_scale, v_scale
// [num_pages, Hkv] fp32, one power of two for each page and head (e4m3.cuh).  Batch: the
// rows cu_tokens[i] .. cu_tokens[i + 1] - 1 are the new tokens of sequence i, at positions
// ctx_len[i], ctx_len[i] + 1, ...; position p lives in slot p % page_size of page
// block_table[i, p / page_size].
#pragma once

#include "e4m3.cuh"
#include "internal.h"

namespace rglru {
namespace paged {

struct Batch {
    int rows, S, H, Hkv, D, page, num_pages, max_pages, max_new, max_total;
    const int32_t *cu, *ctx, *table;
    WsHeader *ws;
};

struct Seq {
    int row0, n, ctx;  // first row, new tokens, tokens before them
};

// The lengths live on the device, so the host cannot check them: a sequence whose lengths
// are not inside the bounds the call was given is skipped (n = 0) and recorded.
__device__ __forceinline__ void record_invalid(WsHeader *ws)
{
    if (ws->status == 0) atomicCAS(&ws->status, 0, (int)RGLRU_ERR_INVALID_ARG);
}
__device__ __forceinline__ bool seq_ok(const Batch &b, int row0, int row1, int ctx)
{
    const long long n = (long long)row1 - row0;
    return row0 >= 0 && row1 <= b.rows && n >= 0 && n <= b.max_new && ctx >= 0 && ctx + n <= b.max_total;
}
__device__ __forceinline__ Seq load_seq(const Batch &b, int i)
{
    const int row0 = b.cu[i], row1 = b.cu[i + 1], ctx = b.ctx[i];
    if (!seq_ok(b, row0, row1, ctx)) {
        record_invalid(b.ws);
        return {0, 0, 0};
    }
    return {row0, row1 - row0, ctx};
}
// The page of table entry j of sequence i, or -1 (recorded) when it names no page of the pool.
__device__ __forceinline__ int load_page(const Batch &b, int i, int j)
{
    const int p = b.table[(size_t)i * b.max_pages + j];
    if (p >= 0 && p < b.num_pages) return p;
    record_invalid(b.ws);
    return -1;
}

// Host checks of the arguments both calls take (paged_append.cu).
rglru_status check_batch(const Batch &b, const void *k, const float *ks, const void *v, const float *vs, size_t ws_bytes,
                         size_t ws_need);

}  // namespace paged
}  // namespace rglru
