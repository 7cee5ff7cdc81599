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
    const int32_t* rows;   // row of `table` of each sequence, or null: its own number
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
    // Rows in two parts. The first call leaves out keys before begin[i] (a multiple of 64; 0: none) of sequence i, and
    // where there are some leaves in `found`, for each row and head, the values times their weights, and the weights'
    // reference (base 2) and sum, instead of out and lse; of other rows it says that they are done (a sum of -1).
    // The second call adds what it finds there to its own, `seed`, and finishes the rows that are not done.
    const int32_t* begin;
    float* found;               // (total, heads, dim)
    float2* found_weight;       // (total, heads)
    const float* seed;
    const float2* seed_weight;
};

// Attention of sequences that begin with the same tokens: groups of sequences, and how many tokens each group shares.
struct KvSharedCall {
    KvAttnCall c;
    const int32_t* groups;
    const int32_t* shared;
    int group_count, max_rows;
    bool always;       // whatever it pays: tests
};

// A page's first tokens on their way to another page.
struct PageItem {
    int from, to, tokens;
};

// What the bookkeeping of pages leaves for the copying: a list, and its length.
struct PageWork {
    int* items_count;
    PageItem* items;
};

struct PageCopyCall {
    KvCacheArgs from, to;
    const int32_t* src;      // count pairs of pages, or
    const int32_t* dst;
    int count;
    const PageItem* items;   // a list that another kernel leaves
    const int* items_count;
    Watchdog wd;
};

// Between the steps of a fork: per old sequence its children, the first of them, its pages, its length and the entries
// that its first child takes over; per new one the pages it needs and their place in the list of those given.
struct ForkWork : PageWork {
    int *children, *first, *held, *lens, *kept, *need;
    int64_t* place;
    int* given;
};

struct KvForkCall {
    KvCacheArgs cache;
    const int32_t *refs, *table, *lens;
    const int32_t* parents;  // null: every sequence continues itself
    int64_t width, room;
    int batch, count, page_shift;
    int32_t *refs_out, *table_out, *lens_out, *spare;
    ForkWork w;
    Watchdog wd;
};

struct KvCompactCall {
    KvCacheArgs cache;
    const int32_t *refs, *table;
    int64_t width;
    int batch;
    int32_t *refs_out, *table_out, *moved, *used;
    PageWork w;
    Watchdog wd;
};

struct SampleCall {
    const void* x;       // (rows, vocab), vocab contiguous
    int64_t row_stride, rows;
    int vocab, dtype;    // tg_dtype, or kFp32
    const float* u;
    // a setting a row, or where null one for all
    const float *temperature, *top_p, *min_p;
    const int32_t* top_k;
    float temperature_all, top_p_all, min_p_all;
    int top_k_all;
    int32_t* tokens;
};
constexpr int kFp32 = 2;
cudaError_t launch_sample(const SampleCall& c, int sm_count, cudaStream_t stream);

// Bytes of a call's workspace; its parts, if it lies at `at`.
int64_t kv_fork_workspace(int64_t pages, int64_t batch, int64_t count, int64_t width, ForkWork* w, void* at);
int64_t kv_compact_workspace(int64_t pages, PageWork* w, void* at);
cudaError_t launch_kv_copy(const PageCopyCall& c, int sm_count, cudaStream_t stream);
cudaError_t launch_kv_fork(const KvForkCall& c, int sm_count, cudaStream_t stream);
cudaError_t launch_kv_compact(const KvCompactCall& c, int sm_count, cudaStream_t stream);

cudaError_t launch_rope(const RopeCall& c, int sm_count, cudaStream_t stream);
cudaError_t launch_kv_append(const KvAppendCall& c, int sm_count, cudaStream_t stream);
cudaError_t launch_kv_read(const KvReadCall& c, int sm_count, cudaStream_t stream);
int64_t kv_attn_workspace(const KvAttnCall& c, int sm_count);
int64_t kv_attn_shared_workspace(const KvSharedCall& s, int sm_count);
// tmK2, tmV2: of the groups' pass (boxes of kv_attn_groups_box_rows lines).
cudaError_t launch_kv_attn_shared(const KvSharedCall& s, const CUtensorMap& tmK, const CUtensorMap& tmV, const CUtensorMap& tmK2, const CUtensorMap& tmV2,
                                  void* workspace, int sm_count, cudaStream_t stream);
int kv_attn_groups_box_rows(const KvSharedCall& s);
bool kv_attn_few_rows(const KvAttnCall& c);  // whether a call runs in the kernel for few rows
int64_t kv_attn_tile_workspace(const KvAttnCall& c, int sm_count);
int kv_attn_tile_box(const KvAttnCall& c);   // tokens a box of its maps
cudaError_t launch_kv_attn_tile(const KvAttnCall& c, const CUtensorMap& tmK, const CUtensorMap& tmV, void* workspace,
                                int sm_count, cudaStream_t stream);
// Maps of the cache's codes as lines of 128 bytes, swizzled, in boxes of kv_attn_box_rows lines.
int kv_attn_box_rows(const KvAttnCall& c);
cudaError_t launch_kv_attn(const KvAttnCall& c, const CUtensorMap& tmK, const CUtensorMap& tmV, void* workspace,
                           int sm_count, cudaStream_t stream);

}  // namespace tg
