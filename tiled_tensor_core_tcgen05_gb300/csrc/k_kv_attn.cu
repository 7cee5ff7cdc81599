// Attention over the paged 8-bit cache: for each new token's query head,
//
//     o = sum_j softmax_j(scale * q . k_j) v_j,  k_j = kcode_j * k_scale(page of j), v_j likewise,
//
// over the keys that the token sees: positions up to its own (or all of the
// sequence's when not causal), and with a window only the last `window` of
// them. Query heads h * share .. (h + 1) * share - 1 read kv head h. A row that
// sees no key gives zeros, and -inf as its log of the sum.
#include "tg_kv.cuh"

namespace tg {
namespace {

constexpr int kWarps = 8;
constexpr float kLog2e = 1.4426950408889634f;

// One warp per (token, query head), one key at a time, the running maximum and sum in fp32.
template <typename E, int kFmt, int kDim>
__global__ void __launch_bounds__(kWarps * 32) attn_rows_kernel(const KvAttnCall c) {
    constexpr int kPer = kDim / 32;
    const KvBatch& b = c.batch;
    const int lane = threadIdx.x % 32;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
    if (row >= static_cast<int64_t>(b.total) * c.heads) return;
    const int token = static_cast<int>(row / c.heads), head = static_cast<int>(row % c.heads);
    int seq = token;
    if (b.cu != nullptr) {
        int lo = 0, hi = b.batch;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (__ldg(b.cu + mid) <= token) lo = mid; else hi = mid;
        }
        seq = lo;
    }
    const SeqSpan span = seq_span(b, seq, c.wd);
    int64_t len = __ldg(b.lens + seq);
    const int page = c.cache.page;
    if (len < 0 || len > b.table_width * page || len > c.max_len) {
        report_range(c.wd);
        len = 0;
    }
    const int64_t pos = len - span.count + token - span.first;
    const bool mine = token >= span.first && token < span.first + span.count;
    int64_t end = c.causal ? min(len, pos + 1) : len;
    int64_t begin = c.window > 0 ? max(int64_t(0), pos - c.window + 1) : 0;
    if (!mine) end = 0;
    const int kvh = head / (c.heads / c.cache.kv_heads);
    const E* q = static_cast<const E*>(c.q.p) + token * c.q.token + head * c.q.head;
    float qr[kPer], acc[kPer] = {};
    for (int i = 0; i < kPer; ++i) qr[i] = to_float(q[lane + 32 * i]) * (c.scale * kLog2e);
    float m = -INFINITY, l = 0.0f;
    for (int64_t j = begin; j < end;) {
        const int p = seq_page(b, c.cache, seq, static_cast<int>(j / page), c.wd);
        const int64_t stop = min(end, (j / page + 1) * page);
        if (p < 0) {
            j = stop;
            continue;
        }
        const int64_t ph = static_cast<int64_t>(p) * c.cache.kv_heads + kvh;
        const float ks = c.cache.k_scale[ph], vs = c.cache.v_scale[ph];
        for (; j < stop; ++j) {
            const int64_t at = (ph * page + j % page) * kDim + lane;
            float s = 0.0f;
            for (int i = 0; i < kPer; ++i) s = fmaf(qr[i], decode<kFmt>(c.cache.k[at + 32 * i]), s);
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
            s *= ks;
            const float m_new = fmaxf(m, s);
            const float keep = exp2f(m - m_new), e = exp2f(s - m_new);
            m = m_new;
            l = l * keep + e;
            for (int i = 0; i < kPer; ++i) acc[i] = acc[i] * keep + e * vs * decode<kFmt>(c.cache.v[at + 32 * i]);
        }
    }
    E* out = static_cast<E*>(c.out) + row * kDim;
    const float inv = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);
    for (int i = 0; i < kPer; ++i) out[lane + 32 * i] = from_float<E>(acc[i] * inv);
    if (c.lse != nullptr && lane == 0) c.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * (1.0f / kLog2e);
}

template <typename E, int kFmt>
cudaError_t launch(const KvAttnCall& c, cudaStream_t stream) {
    const int64_t rows = static_cast<int64_t>(c.batch.total) * c.heads;
    const unsigned grid = static_cast<unsigned>((rows + kWarps - 1) / kWarps);
    if (c.cache.dim == 128) attn_rows_kernel<E, kFmt, 128><<<grid, kWarps * 32, 0, stream>>>(c);
    else attn_rows_kernel<E, kFmt, 64><<<grid, kWarps * 32, 0, stream>>>(c);
    return cudaGetLastError();
}

}  // namespace

int64_t kv_attn_workspace(const KvAttnCall&, int) { return 0; }

cudaError_t launch_kv_attn(const KvAttnCall& c, void*, int, cudaStream_t stream) {
    const bool h = c.dtype == kFp16, e4 = c.cache.fmt == kKvE4M3;
    if (h && e4) return launch<__half, kKvE4M3>(c, stream);
    if (h) return launch<__half, kKvInt8>(c, stream);
    if (e4) return launch<__nv_bfloat16, kKvE4M3>(c, stream);
    return launch<__nv_bfloat16, kKvInt8>(c, stream);
}

}  // namespace tg
