// Attention of sequences that begin with the same tokens. The shared keys are
// attended by all rows of a group at once, as one sequence's that every row sees
// whole (the tokens come before all new ones), and read once for the group. Each
// sequence's own keys come before, in a first pass, whose findings this one adds:
//
//     o = (v1 2^(m1 - m) + v2 2^(m2 - m)) / (l1 2^(m1 - m) + l2 2^(m2 - m)),  m = max(m1, m2),
//
// v the values times their weights, m the weights' reference and l their sum, in
// fp32 between the passes. Both passes are the cache attention's own kernels; the
// second one takes many rows on tcgen05 (k_kv_tile.cu) where a group has many, and it is the second because
// it takes long to begin (shares, queries, an empty pipeline: 11 us) and needs the other's findings only at its end: it is
// launched early, and CTAs of it begin as SMs have done with the first. This
// file holds what comes before: which sequences take part, and each group's rows.
//
// Where the rows of one sequence are many by themselves (more than few_rows allows)
// a cache is read once for 256 of them in any case, and products bound the
// call; and where there is little to save, two passes cost more than they save
// (pays()): then it is attended as without groups.
#include <algorithm>
#include <climits>

#include "tg_device.cuh"
#include "tg_kv_split.cuh"

namespace tg {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 64;  // a sequence's own keys begin where a chunk of the few-rows kernel does

struct SharedWork {
    int32_t* cu;      // groups' rows of the packed tensors
    int32_t* lens;    // groups' shared tokens, as far as whole chunks of the few-rows kernel go
    int32_t* rows;    // table row that a group's pages are read from
    int32_t* begin;   // of each sequence: its keys before it are the group's
    float* found;
    float2* found_weight;
    void* first;      // the passes' workspaces
    void* second;
    int64_t bytes;
};

__device__ __forceinline__ int offset_of(const KvBatch& b, int i) { return b.cu != nullptr ? __ldg(b.cu + i) : i; }

// Whether the groups lie one behind another in the batch, and their rows too. Whole block.
__device__ __forceinline__ bool in_order(const KvSharedCall& s) {
    const KvBatch& b = s.c.batch;
    bool good = true;
    for (int g = threadIdx.x; g < s.group_count; g += kThreads) {
        const int first = __ldg(s.groups + g), last = __ldg(s.groups + g + 1);
        if (first < 0 || last < first || last > b.batch) {
            good = false;
        } else {
            const int row0 = offset_of(b, first), row1 = offset_of(b, last);
            good &= row0 >= 0 && row1 >= row0 && row1 <= b.total;
        }
    }
    return __syncthreads_and(good);
}

// Tokens that a group shares, in whole chunks of the few-rows kernel; -1: out of range. The groups are in order.
__device__ __forceinline__ int tokens_of(const KvSharedCall& s, int g) {
    const KvBatch& b = s.c.batch;
    const int tokens = __ldg(s.shared + g), rows = offset_of(b, __ldg(s.groups + g + 1)) - offset_of(b, __ldg(s.groups + g));
    if (rows > s.max_rows || tokens < 0 || tokens > s.c.max_len || tokens > b.table_width * s.c.cache.page) return -1;
    return tokens / kChunk * kChunk;
}

// Whether sequence i of group g, whose shared tokens in whole chunks are so many, holds all that is shared, the rest behind the chunks too:
// the pages of one that does not are its own from the first token on.
__device__ __forceinline__ bool takes_part(const KvSharedCall& s, int i, int g, int tokens) {
    const KvBatch& b = s.c.batch;
    int n = 1;
    if (b.cu != nullptr) {
        const int lo = __ldg(b.cu + i), hi = __ldg(b.cu + i + 1);
        n = hi - lo;
        if (lo < 0 || hi < lo || hi > b.total || n > b.max_new) return false;
    }
    const int len = __ldg(b.lens + i);
    return tokens > 0 && len <= s.c.max_len && len <= b.table_width * s.c.cache.page && len - n >= __ldg(s.shared + g);
}

// Block g < group_count: that group. The blocks behind: the sequences.
__global__ void __launch_bounds__(kThreads) group_kernel(const KvSharedCall s, const SharedWork w) {
    __shared__ int lowest;
    const int g = blockIdx.x;
    const bool good = in_order(s);
    if (g >= s.group_count) {
        const int i = (g - s.group_count) * kThreads + threadIdx.x;
        if (i >= s.c.batch.batch) return;
        int tokens = 0, lo = 0;
        if (good) {
            int hi = s.group_count;  // the last group that begins at i or before
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (__ldg(s.groups + mid) <= i) lo = mid;
                else hi = mid;
            }
            if (i >= __ldg(s.groups + lo) && i < __ldg(s.groups + lo + 1)) tokens = tokens_of(s, lo);
        }
        w.begin[i] = takes_part(s, i, lo, tokens) ? tokens : 0;
        return;
    }
    const int tokens = good ? tokens_of(s, g) : -1;
    if (threadIdx.x == 0) {
        lowest = INT_MAX;
        if (tokens < 0) report_range(s.c.wd);
    }
    __syncthreads();
    const int first = good ? __ldg(s.groups + g) : 0, last = good ? __ldg(s.groups + g + 1) : 0;
    for (int i = first + threadIdx.x; i < last; i += kThreads)
        if (takes_part(s, i, g, tokens)) {
            atomicMin(&lowest, i);
            break;
        }
    __syncthreads();
    if (threadIdx.x != 0) return;
    w.cu[g] = good ? offset_of(s.c.batch, first) : 0;
    if (g == s.group_count - 1) w.cu[g + 1] = good ? offset_of(s.c.batch, last) : 0;
    w.lens[g] = lowest < INT_MAX ? tokens : 0;
    w.rows[g] = lowest < INT_MAX ? lowest : 0;
}

// The second pass: groups as sequences.
KvAttnCall group_call(const KvSharedCall& s, const SharedWork& w) {
    KvAttnCall c = s.c;
    c.batch.lens = w.lens;
    c.batch.cu = w.cu;
    c.batch.rows = w.rows;
    c.batch.batch = s.group_count;
    c.batch.max_new = s.max_rows;
    c.causal = 0;
    c.seed = w.found;
    c.seed_weight = w.found_weight;
    return c;
}

SharedWork layout(const KvSharedCall& s, int sm_count, void* at) {
    SharedWork w{};
    char* p = static_cast<char*>(at);
    auto take = [&](int64_t bytes) {
        char* x = p + w.bytes;
        w.bytes += (bytes + 255) / 256 * 256;
        return static_cast<void*>(x);
    };
    const int64_t rows = static_cast<int64_t>(s.c.batch.total) * s.c.heads;
    w.cu = static_cast<int32_t*>(take((s.group_count + 1) * 4ll));
    w.lens = static_cast<int32_t*>(take(s.group_count * 4ll));
    w.rows = static_cast<int32_t*>(take(s.group_count * 4ll));
    w.begin = static_cast<int32_t*>(take(s.c.batch.batch * 4ll));
    w.found = static_cast<float*>(take(rows * s.c.cache.dim * 4));
    w.found_weight = static_cast<float2*>(take(rows * 8));
    w.first = take(kv_attn_workspace(s.c, sm_count));
    w.second = take(kv_attn_workspace(group_call(s, w), sm_count));
    return w;
}

// Whether groups are worth their pass. What sharing can save at most is the reading of all sequences but one a group, as long as they may
// be; a member has a row at least, so a group's are no more than max_rows, and sequences in no group save nothing. The further pass, the kernel
// before both and the join take some 20 us. Measured on a GB300, in us with groups and without,
// 32 heads over 8 of 128: 8 sequences of 4000 (58 MB to save) 34 and 18, of 16000 (230 MB) 38 and 41; 32 of 4000 (256 MB) 42 and 43; 64 of 1000
// (133 MB) 39 and 29, of 4000 (520 MB) 45 and 75, of 16000 60 and 255; four groups of 16 of 1000 (117 MB) 36 and 28, of 4000 (418 MB) 48
// and 65; a group of two among 64 of 16000 (31 MB) 334 and 321, of 16 (469 MB) 295 and 305, 32 groups of two of 8000 (500 MB) 107 and 160. The
// bounds that the caller gives are all that is known here: loose ones are taken for long sequences.
bool pays(const KvSharedCall& s) {
    const KvAttnCall& c = s.c;
    const int64_t each = std::min(c.max_len, c.batch.table_width * c.cache.page) * c.cache.kv_heads * c.cache.dim * 2;
    const int64_t spared = std::min<int64_t>(c.batch.batch - s.group_count, static_cast<int64_t>(s.group_count) * std::max(s.max_rows - 1, 0));
    return s.always || each * spared >= (256ll << 20);
}

bool in_groups(const KvSharedCall& s) { return s.group_count > 0 && kv_attn_few_rows(s.c) && pays(s); }

}  // namespace

int64_t kv_attn_shared_workspace(const KvSharedCall& s, int sm_count) {
    return in_groups(s) ? layout(s, sm_count, nullptr).bytes : kv_attn_workspace(s.c, sm_count);
}

int kv_attn_groups_box_rows(const KvSharedCall& s) { return kv_attn_box_rows(group_call(s, SharedWork{})); }

cudaError_t launch_kv_attn_shared(const KvSharedCall& s, const CUtensorMap& tmK, const CUtensorMap& tmV, const CUtensorMap& tmK2, const CUtensorMap& tmV2,
                                  void* workspace, int sm_count, cudaStream_t stream) {
    if (!in_groups(s)) return launch_kv_attn(s.c, tmK, tmV, workspace, sm_count, stream);
    const SharedWork w = layout(s, sm_count, workspace);
    group_kernel<<<s.group_count + (s.c.batch.batch + kThreads - 1) / kThreads, kThreads, 0, stream>>>(s, w);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    KvAttnCall c = s.c;
    c.begin = w.begin;
    c.found = w.found;
    c.found_weight = w.found_weight;
    if ((e = launch_kv_attn(c, tmK, tmV, w.first, sm_count, stream)) != cudaSuccess) return e;
    return launch_kv_attn(group_call(s, w), tmK2, tmV2, w.second, sm_count, stream);
}

}  // namespace tg
