// Internal interface between the C-ABI front end (tg_api.cu) and the kernels of
// rotary positions and the paged 8-bit cache. Not installed; not part of the
// public ABI.
#pragma once

#include "tg_internal.h"

namespace tg {

// Status code of a length, an offset or a page number out of range, after the wait sites.
constexpr int kSiteRange = 9;

constexpr int kKvE4M3 = 0, kKvInt8 = 1;      // tg_kv_format
constexpr int kRopeHalf = 0, kRopeInterleaved = 1;
constexpr int kFp16 = 0, kBf16 = 1;          // tg_dtype

// Rotated pairs: (j, j + rotary / 2) in the half layout, (2 j, 2 j + 1) in the interleaved one.
struct RopeArgs {
    const double* inv_freq;  // rotary / 2 radians per position; null: no rotation
    float amplitude;
    int rotary, layout;
    float sign;              // -1: the transposed rotation (backward)
};

// (tokens, heads, dim) 16-bit tensor, dim contiguous, strides in elements.
struct Strided {
    void* p;
    int64_t token, head;
};

struct KvCacheArgs {
    uint8_t* k;      // (pages, kv_heads, page, dim) codes
    uint8_t* v;
    float* k_scale;  // (pages, kv_heads)
    float* v_scale;
    int64_t pages;
    int kv_heads, page, dim, fmt;
};

struct KvBatch {
    const int32_t* table;  // (batch, table_width) page numbers
    int64_t table_width;
    const int32_t* lens;   // batch lengths (append: before the call; attention: with the new tokens)
    const int32_t* cu;     // batch + 1 offsets into the packed rows, or null: one row a sequence
    int batch, total, max_new;
};

struct RopeCall {
    Strided x, y;
    const int32_t* positions;
    int tokens, heads, dim, dtype;
    RopeArgs rope;
};

struct KvAppendCall {
    KvCacheArgs cache;
    KvBatch batch;
    Strided k, v;        // new keys and values
    Strided q, q_out;    // queries rotated beside the keys (heads > 0)
    int heads, dtype;
    RopeArgs rope;
    Watchdog wd;
};

struct KvReadCall {
    KvCacheArgs cache;
    KvBatch batch;       // lens: first position of each sequence's range
    void* k;             // (total, kv_heads, dim) out
    void* v;
    int dtype;
    Watchdog wd;
};

struct KvAttnCall {
    KvCacheArgs cache;
    KvBatch batch;
    Strided q;
    void* out;           // (total, heads, dim)
    float* lse;          // (total, heads) or null
    int heads, dtype, causal;
    int64_t max_len;
    int64_t window;      // 0: none
    float scale;
    Watchdog wd;
};

cudaError_t launch_rope(const RopeCall& c, int sm_count, cudaStream_t stream);
cudaError_t launch_kv_append(const KvAppendCall& c, int sm_count, cudaStream_t stream);
cudaError_t launch_kv_read(const KvReadCall& c, int sm_count, cudaStream_t stream);
int64_t kv_attn_workspace(const KvAttnCall& c, int sm_count);
int64_t kv_attn_tile_workspace(const KvAttnCall& c, int sm_count);
cudaError_t launch_kv_attn_tile(const KvAttnCall& c, const CUtensorMap& tmK, const CUtensorMap& tmV, void* workspace,
                                int sm_count, cudaStream_t stream);
// Maps of the cache's codes as lines of 128 bytes, swizzled, in boxes of kv_attn_box_rows lines.
int kv_attn_box_rows(const KvAttnCall& c);
cudaError_t launch_kv_attn(const KvAttnCall& c, const CUtensorMap& tmK, const CUtensorMap& tmV, void* workspace,
                           int sm_count, cudaStream_t stream);

}  // namespace tg
