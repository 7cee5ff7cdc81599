// The paged 8-bit cache: writing new keys and values into it, quantised as
// they are written, and reading it back.
//
// A page holds `page` consecutive tokens of one sequence; each (page, kv head)
// has one fp32 scale s for keys and one for values, and a code q stands for
// q * s. Writing tokens into a page:
//
//     s = max(s of the tokens it holds, max |x| of the new ones * (1 / qmax), 2^-60),
//     held codes -> round(q * (s_old * (1 / s))) where s grew,
//     new codes  =  round(x * (1 / s)),
//
// rounding to nearest even into e4m3 (qmax 448) or int8 (qmax 127). A page
// whose first token is written by the call takes nothing over from what it
// held before. Keys may be rotated on the way (in fp32, not rounded between).
#include "tg_kv.cuh"

namespace tg {
namespace {

constexpr int kThreads = 128;

// The rotated (or plain) value d of a row at `pos`.
template <typename E>
__device__ __forceinline__ float row_value(const E* row, int d, int pos, const RopeArgs& r) {
    const float x = to_float(row[d]);
    if (r.inv_freq == nullptr || d >= r.rotary) return x;
    const int half = r.rotary / 2;
    const bool first = r.layout == kRopeHalf ? d < half : (d & 1) == 0;
    const int j = r.layout == kRopeHalf ? (first ? d : d - half) : d / 2;
    const int other = r.layout == kRopeHalf ? (first ? d + half : d - half) : d ^ 1;
    const float2 cs = turn_cos_sin(turn_step(__ldg(r.inv_freq + j)), pos, r.amplitude, r.sign);
    const float o = to_float(row[other]);
    return first ? x * cs.x - o * cs.y : x * cs.x + o * cs.y;
}

// One CTA per (page that a sequence writes to, kv head, keys or values). Sequence i's pages
// are items base(i) .. base(i + 1) - 1 with base(i) = cu[i] / page + 2 i: n tokens touch at most
// n / page + 2 pages, so some items have none.
template <typename E, int kFmt>
__global__ void __launch_bounds__(kThreads) append_kernel(const KvAppendCall c) {
    __shared__ float red[kThreads / 32];
    const KvBatch& b = c.batch;
    const int page = c.cache.page, dim = c.cache.dim;
    const int item = blockIdx.x, head = blockIdx.y;
    const bool values = blockIdx.z != 0;
    int lo = 0, hi = b.batch;  // the last sequence with base <= item
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        const int base = (b.cu ? __ldg(b.cu + mid) : mid) / page + 2 * mid;
        if (base <= item) lo = mid; else hi = mid;
    }
    const int seq = lo;
    const SeqSpan span = seq_span(b, seq, c.wd);
    if (span.count == 0) return;
    const int k = item - ((b.cu ? __ldg(b.cu + seq) : seq) / page + 2 * seq);
    const int64_t len = __ldg(b.lens + seq);
    if (len < 0 || len + span.count > b.table_width * page) {
        report_range(c.wd);
        return;
    }
    const int64_t first_slot = len / page;
    const int64_t slot = first_slot + k;
    if (slot * page >= len + span.count) return;
    const int p = seq_page(b, c.cache, seq, static_cast<int>(slot), c.wd);
    if (p < 0) return;
    const int from = k == 0 ? static_cast<int>(len % page) : 0;                    // first new place in the page
    const int to = static_cast<int>(min(static_cast<int64_t>(page), len + span.count - slot * page));
    const int64_t row0 = span.first + (slot * page + from - len);                   // its packed row
    const Strided& src = values ? c.v : c.k;
    const E* x = static_cast<const E*>(src.p) + row0 * src.token + head * src.head;
    uint8_t* codes = (values ? c.cache.v : c.cache.k) + (static_cast<int64_t>(p) * c.cache.kv_heads + head) * page * dim;
    float* scale = (values ? c.cache.v_scale : c.cache.k_scale) + static_cast<int64_t>(p) * c.cache.kv_heads + head;
    RopeArgs rope = c.rope;
    if (values) rope.inv_freq = nullptr;

    float most = 0.0f;  // of the finite values
    for (int i = threadIdx.x; i < (to - from) * dim; i += kThreads) {
        const int t = i / dim, d = i - t * dim;
        const float a = fabsf(row_value(x + t * src.token, d, static_cast<int>(slot * page) + from + t, rope));
        if (a <= 3.402823466e38f) most = fmaxf(most, a);
    }
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = most;
    const float s_old = from > 0 ? *scale : 0.0f;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) most = fmaxf(most, red[w]);
    const float s = fmaxf(s_old, fmaxf(__fmul_rn(most, code_max_inverse<kFmt>()), kScaleFloor));
    const float per = __fdiv_rn(1.0f, s);
    if (from > 0 && s != s_old) {
        const float ratio = __fmul_rn(s_old, per);
        for (int i = threadIdx.x; i < from * dim; i += kThreads)
            codes[i] = encode<kFmt>(__fmul_rn(decode<kFmt>(codes[i]), ratio));
    }
    for (int i = threadIdx.x; i < (to - from) * dim; i += kThreads) {
        const int t = i / dim, d = i - t * dim;
        float v = row_value(x + t * src.token, d, static_cast<int>(slot * page) + from + t, rope);
        v = min_nan(max_nan(v, -most), most);  // an infinity becomes the largest finite value
        codes[(from + t) * dim + d] = encode<kFmt>(__fmul_rn(v, per));
    }
    if (threadIdx.x == 0) *scale = s;
}

// The rotated queries of an append: one CTA per token.
template <typename E>
__global__ void __launch_bounds__(kThreads) append_q_kernel(const KvAppendCall c) {
    const KvBatch& b = c.batch;
    const int token = blockIdx.x;
    int seq = token;
    if (b.cu != nullptr) {
        int lo = 0, hi = b.batch;  // the last sequence that starts at or before the token
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (__ldg(b.cu + mid) <= token) lo = mid; else hi = mid;
        }
        seq = lo;
    }
    const SeqSpan span = seq_span(b, seq, c.wd);
    if (token < span.first || token >= span.first + span.count) return;
    const int pos = __ldg(b.lens + seq) + token - span.first;
    const E* x = static_cast<const E*>(c.q.p) + token * c.q.token;
    E* y = static_cast<E*>(c.q_out.p) + token * c.q_out.token;
    const int half = c.rope.rotary / 2, dim = c.cache.dim, per_head = half + dim - c.rope.rotary;
    for (int i = threadIdx.x; i < c.heads * per_head; i += kThreads) {
        const int h = i / per_head, j = i - h * per_head;
        const E* xh = x + h * c.q.head;
        E* yh = y + h * c.q_out.head;
        if (j < half) {
            const int ia = c.rope.layout == kRopeHalf ? j : 2 * j, ib = c.rope.layout == kRopeHalf ? j + half : 2 * j + 1;
            const float2 cs = turn_cos_sin(turn_step(__ldg(c.rope.inv_freq + j)), pos, c.rope.amplitude, c.rope.sign);
            const float u = to_float(xh[ia]), w = to_float(xh[ib]);
            yh[ia] = from_float<E>(u * cs.x - w * cs.y);
            yh[ib] = from_float<E>(w * cs.x + u * cs.y);
        } else {
            yh[half + j] = xh[half + j];
        }
    }
}

// One CTA per packed row: its sequence, page and place, then every kv head.
template <typename E, int kFmt>
__global__ void __launch_bounds__(kThreads) read_kernel(const KvReadCall c) {
    const KvBatch& b = c.batch;
    const int row = blockIdx.x, page = c.cache.page, dim = c.cache.dim, heads = c.cache.kv_heads;
    int seq = row;
    if (b.cu != nullptr) {
        int lo = 0, hi = b.batch;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (__ldg(b.cu + mid) <= row) lo = mid; else hi = mid;
        }
        seq = lo;
    }
    const SeqSpan span = seq_span(b, seq, c.wd);
    if (row < span.first || row >= span.first + span.count) return;
    const int64_t pos = static_cast<int64_t>(__ldg(b.lens + seq)) + row - span.first;
    if (pos < 0 || pos >= b.table_width * page) {
        report_range(c.wd);
        return;
    }
    const int p = seq_page(b, c.cache, seq, static_cast<int>(pos / page), c.wd);
    if (p < 0) return;
    const int place = static_cast<int>(pos % page);
    for (int i = threadIdx.x; i < heads * dim; i += kThreads) {
        const int h = i / dim, d = i - h * dim;
        const int64_t ph = static_cast<int64_t>(p) * heads + h;
        const int64_t at = (ph * page + place) * dim + d;
        const int64_t to = static_cast<int64_t>(row) * heads * dim + i;
        static_cast<E*>(c.k)[to] = from_float<E>(decode<kFmt>(c.cache.k[at]) * c.cache.k_scale[ph]);
        static_cast<E*>(c.v)[to] = from_float<E>(decode<kFmt>(c.cache.v[at]) * c.cache.v_scale[ph]);
    }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendCall& c, int, cudaStream_t stream) {
    const dim3 grid(c.batch.total / c.cache.page + 2 * c.batch.batch, c.cache.kv_heads, 2);
    const bool h = c.dtype == kFp16, e4 = c.cache.fmt == kKvE4M3;
    if (h && e4) append_kernel<__half, kKvE4M3><<<grid, kThreads, 0, stream>>>(c);
    else if (h) append_kernel<__half, kKvInt8><<<grid, kThreads, 0, stream>>>(c);
    else if (e4) append_kernel<__nv_bfloat16, kKvE4M3><<<grid, kThreads, 0, stream>>>(c);
    else append_kernel<__nv_bfloat16, kKvInt8><<<grid, kThreads, 0, stream>>>(c);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || c.heads == 0) return e;
    if (h) append_q_kernel<__half><<<c.batch.total, kThreads, 0, stream>>>(c);
    else append_q_kernel<__nv_bfloat16><<<c.batch.total, kThreads, 0, stream>>>(c);
    return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvReadCall& c, int, cudaStream_t stream) {
    const bool h = c.dtype == kFp16, e4 = c.cache.fmt == kKvE4M3;
    const int grid = c.batch.total;
    if (h && e4) read_kernel<__half, kKvE4M3><<<grid, kThreads, 0, stream>>>(c);
    else if (h) read_kernel<__half, kKvInt8><<<grid, kThreads, 0, stream>>>(c);
    else if (e4) read_kernel<__nv_bfloat16, kKvE4M3><<<grid, kThreads, 0, stream>>>(c);
    else read_kernel<__nv_bfloat16, kKvInt8><<<grid, kThreads, 0, stream>>>(c);
    return cudaGetLastError();
}

}  // namespace tg
