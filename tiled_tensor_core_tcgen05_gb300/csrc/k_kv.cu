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
//
// Memory bounds all of it. Prompts go page by page: the threads of a (page,
// head) hold its values in registers between the maximum and the rounding, so
// each is read once. Single tokens go sequence by sequence: a CTA rotates and
// writes all heads of one token (and rotates its queries), a head a warp, and
// only where a scale grows are the page's held codes touched at all.
//
// Measured: 17 410 tokens of 7 prompts, 8 heads of 128, to int8 in pages of 32: 23.5 us
// where its bytes take 15.7: conversion, rounding and addresses fill the issue slots.
// With rotation, and 32 heads of queries, e4m3, pages of 64: 87 us where the bytes take
// 58: keys 30, values 17 and queries 44 by themselves.
// One token each of 256 sequences, rotated: 7.5 us where no page's scale grows, 11.9 where
// every one does; 1024 sequences 23 and 47. A CTA's five dependent reads are paid for every
// wave of CTAs, and 512 threads of 115 to 128 registers let one CTA on an SM. Reading back
// 890 MB: 134 us, 6.6 TB/s or 0.98 of the copy rate.
#include "tg_rope.cuh"

#include <type_traits>

namespace tg {
namespace {

// The last i in [0, n) with start(i) <= x, start being non-decreasing: whole block, three barriers' worth.
template <typename F>
__device__ __forceinline__ int block_find(int n, F start, int64_t x) {
    int found = 0;
    for (int base = 0; base < n; base += blockDim.x) {
        const int i = base + threadIdx.x;
        const int here = __syncthreads_count(i < n && start(i) <= x);
        found += here;
        if (here < static_cast<int>(blockDim.x)) break;
    }
    return found > 0 ? found - 1 : 0;
}

__device__ __forceinline__ float max_finite(float most, float x) {
    const float a = fabsf(x);
    return a <= 3.402823466e38f ? fmaxf(most, a) : most;
}

// The largest |x| of eight values as they are stored; NaN where one of them is.
__device__ __forceinline__ float piece_most(const uint4& u, __half) {
    const __half2* x = reinterpret_cast<const __half2*>(&u);
    const __half2 m = __hmax2_nan(__hmax2_nan(__habs2(x[0]), __habs2(x[1])), __hmax2_nan(__habs2(x[2]), __habs2(x[3])));
    return __half2float(__hmax_nan(__low2half(m), __high2half(m)));
}
__device__ __forceinline__ float piece_most(const uint4& u, __nv_bfloat16) {
    const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&u);
    const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(__habs2(x[0]), __habs2(x[1])), __hmax2_nan(__habs2(x[2]), __habs2(x[3])));
    return __bfloat162float(__hmax_nan(__low2bfloat16(m), __high2bfloat16(m)));
}

// Codes of kN values of a row whose block has the largest finite value `most` and 1 / scale `per`.
template <int kFmt, int kN>
__device__ __forceinline__ void encode_values(const float (&x)[kN], float most, float per, uint32_t (&w)[kN / 4]) {
    float y[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i)  // an infinity becomes the largest finite value
        y[i] = __fmul_rn(min_nan(max_nan(x[i], -most), most), per);
#pragma unroll
    for (int i = 0; i < kN; i += 4) w[i / 4] = encode4<kFmt>(y[i], y[i + 1], y[i + 2], y[i + 3]);
}

template <int kFmt>
__device__ __forceinline__ uint32_t again4(uint32_t w, float ratio) {
    float x[4];
    decode4<kFmt>(w, x);
    return encode4<kFmt>(__fmul_rn(x[0], ratio), __fmul_rn(x[1], ratio), __fmul_rn(x[2], ratio), __fmul_rn(x[3], ratio));
}

// Eight values as they are stored.
template <typename E>
__device__ __forceinline__ uint4 load_piece(const E* p, bool vec) {
    if (vec) return *reinterpret_cast<const uint4*>(p);
    uint4 u;
    E* e = reinterpret_cast<E*>(&u);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = p[i];
    return u;
}

// The partners of values d .. d + 7 of a row in the half layout (zeros elsewhere).
template <typename E>
__device__ __forceinline__ uint4 load_partner_piece(const E* row, int d, bool vec, const RopeArgs& r) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (r.layout != kRopeHalf || d >= r.rotary) return u;
    const int half = r.rotary / 2;
    if (half % 8 == 0) return load_piece(row + (d < half ? d + half : d - half), vec);
    E* e = reinterpret_cast<E*>(&u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int at = d + i;
        if (at < r.rotary) e[i] = row[at < half ? at + half : at - half];
    }
    return u;
}

template <typename E>
__device__ __forceinline__ void piece_values(const uint4& u, float (&x)[8]) {
    const E* e = reinterpret_cast<const E*>(&u);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_float(e[i]);
}

// How rows may be read: 16-byte pieces (then 8-byte ones too) or single values.
struct Wide {
    bool k, v, q, q_out;
};

// ---------------------------------------------------------------- prompts: page by page

struct PageArgs {
    KvAppendCall c;
    Wide wide;
    int heads_a_cta;   // kv heads that a CTA's groups take one after another
    int values_only;   // without rotation: 1 values, 0 keys and values (blockIdx.z)
};

constexpr int kVecs = 4;  // 16-byte pieces a thread holds

// A group of page * dim / 32 threads takes one (page, head): piece i of thread t is piece
// t + i * group of the page's page * dim / 8. blockIdx: x pages that sequences write to (sequence i's
// are items base(i) .. base(i + 1) - 1 with base(i) = cu[i] / page + 2 i: n tokens touch at most
// n / page + 2 pages, so some items have none), y heads, z keys or values (keys that are rotated are a
// launch of their own).
template <typename E, int kFmt, int kDim, bool kRope>
__device__ __forceinline__ void append_pages(const PageArgs& a) {
    extern __shared__ float turns[];  // cos, then sin: (page, rotary / 2) each
    __shared__ float red[2][16];
    const KvAppendCall& c = a.c;
    const KvBatch& b = c.batch;
    const int page = c.cache.page, shift = 31 - __clz(page), item = blockIdx.x;  // a power of two
    const bool values = kRope ? false : a.values_only || blockIdx.z != 0;
    constexpr int kPieces = kDim / 8;  // of a row
    auto base_of = [&](int i) { return static_cast<int64_t>((b.cu ? __ldg(b.cu + i) : i) >> shift) + 2 * i; };
    const int seq = block_find(b.batch, base_of, item);
    const SeqSpan span = seq_span(b, seq, c.wd);
    if (span.count == 0) return;
    const int k = static_cast<int>(item - base_of(seq));
    const int64_t len = __ldg(b.lens + seq);
    if (len < 0 || len + span.count > b.table_width * page) {
        report_range(c.wd);
        return;
    }
    const int64_t slot = (len >> shift) + k;
    if (k < 0 || slot * page >= len + span.count) return;
    const int p = seq_page(b, c.cache, seq, static_cast<int>(slot), c.wd);
    if (p < 0) return;
    const int from = k == 0 ? static_cast<int>(len & (page - 1)) : 0;                     // first new place in the page
    const int to = static_cast<int>(min(static_cast<int64_t>(page), len + span.count - slot * page));
    const int64_t row0 = span.first + (slot * page - len);                          // packed row of place 0
    const RopeArgs& rope = c.rope;
    const int half = rope.rotary / 2;
    float *cs = turns, *sn = turns + page * half;
    const int group = page * kPieces / kVecs, groups = blockDim.x / group;
    const int g = threadIdx.x / group, t = threadIdx.x - g * group;
    // a group is page / kVecs whole rows: a thread's pieces are at one place of a row, `rows` rows apart
    const int place0 = t / kPieces, d = (t - place0 * kPieces) * 8, rows = page / kVecs;
    const Strided& src = values ? c.v : c.k;
    const bool vec = values ? a.wide.v : a.wide.k;
    const int head_end = min(c.cache.kv_heads, static_cast<int>(blockIdx.y + 1) * a.heads_a_cta);
    const E* x0 = static_cast<const E*>(src.p) + (row0 + place0) * src.token;
    const int64_t apart = rows * src.token;
    uint8_t* all_codes = values ? c.cache.v : c.cache.k;
    float* all_scales = values ? c.cache.v_scale : c.cache.k_scale;
    // one head's pieces (and, rotated, their partners) and old scale, fetched while the head before is worked on
    uint4 own[kVecs], other[kVecs];
    float s_old = 0.0f;
    auto fetch = [&](int head) {
        if (head >= head_end) return;
        s_old = from > 0 ? all_scales[static_cast<int64_t>(p) * c.cache.kv_heads + head] : 0.0f;
        auto pieces = [&](bool wide) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int place = place0 + i * rows;
                if (place >= from && place < to) {
                    const E* row = x0 + i * apart + head * src.head;
                    own[i] = load_piece(row + d, wide);
                    if constexpr (kRope) other[i] = load_partner_piece(row, d, wide, rope);
                }
            }
        };
        if (vec) pieces(true);
        else pieces(false);
    };
    fetch(blockIdx.y * a.heads_a_cta + g);
    if constexpr (kRope) {
        // a thread keeps to one pair, whose step is settled once; a block has twice a row's pairs or more
        const int j = threadIdx.x % half, many = blockDim.x / half;
        const auto step = turn_step(__ldg(rope.inv_freq + j));
        for (int i = from + threadIdx.x / half; i < to && threadIdx.x < many * half; i += many) {
            const float2 x = turn_cos_sin(step, static_cast<int>(slot << shift) + i, rope.amplitude, rope.sign);
            cs[i * half + j] = x.x;
            sn[i * half + j] = x.y;
        }
        __syncthreads();
    }
    int round = 0;
    // every group makes every round, so that all meet at the barriers
    for (int head0 = blockIdx.y * a.heads_a_cta; head0 < head_end; head0 += groups, ++round) {
        const int head = head0 + g;
        const bool real = head < head_end;
        const float s_held = s_old;
        // rotated values are kept in fp32, others as they were read: they are half the registers
        std::conditional_t<kRope, float[kVecs][8], uint4[kVecs]> x;
        float most = 0.0f;  // NaN or infinite where a value is
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int place = place0 + i * rows;
            if (real && place >= from && place < to) {
                if constexpr (kRope) {
                    float v[8], o[8];
                    piece_values<E>(own[i], v);
                    piece_values<E>(other[i], o);
                    rotate_values<8>(v, o, d, cs + place * half, sn + place * half, rope);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x[i][e] = v[e];
                        most = max_nan(most, fabsf(v[e]));
                    }
                } else {
                    x[i] = own[i];
                    most = max_nan(most, piece_most(own[i], E()));
                }
            }
        }
        // where the warp's values are all finite, they need no second look (a branch of the whole warp: taken
        // thread by thread, the instructions of the other way were issued too)
        const bool plain = __all_sync(0xFFFFFFFFu, most <= 3.402823466e38f);
        if (!plain) {
            most = 0.0f;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int place = place0 + i * rows;
                if (real && place >= from && place < to) {
                    float v[8];
                    if constexpr (kRope) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = x[i][e];
                    } else {
                        piece_values<E>(x[i], v);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) most = max_finite(most, v[e]);
                }
            }
        }
        fetch(head + groups);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
        if (group > 32) {
            float* r = red[round & 1];  // the other half is still being read
            if (threadIdx.x % 32 == 0) r[threadIdx.x / 32] = most;
            __syncthreads();
            for (int w = g * group / 32; w < (g + 1) * group / 32; ++w) most = fmaxf(most, r[w]);
        }
        if (real) {
            const int64_t ph = static_cast<int64_t>(p) * c.cache.kv_heads + head;
            uint8_t* codes = all_codes + ph * page * kDim + t * 8;
            const float s = fmaxf(s_held, fmaxf(__fmul_rn(most, code_max_inverse<kFmt>()), kScaleFloor));
            const float per = __fdiv_rn(1.0f, s);
            const float ratio = __fmul_rn(s_held, per);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int place = place0 + i * rows;
                uint2* q = reinterpret_cast<uint2*>(codes + i * group * 8);
                if (place >= from && place < to) {
                    uint32_t w[2];
                    float v[8];
                    if constexpr (kRope) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = x[i][e];
                    } else {
                        piece_values<E>(x[i], v);
                    }
                    if (plain) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(v[e], per);
                        w[0] = encode4_in_range<kFmt>(v[0], v[1], v[2], v[3]);
                        w[1] = encode4_in_range<kFmt>(v[4], v[5], v[6], v[7]);
                    } else {
                        encode_values<kFmt, 8>(v, most, per, w);
                    }
                    *q = make_uint2(w[0], w[1]);
                } else if (place < from && s != s_held) {
                    const uint2 w = *q;
                    *q = make_uint2(again4<kFmt>(w.x, ratio), again4<kFmt>(w.y, ratio));
                }
            }
            if (t == 0) all_scales[ph] = s;
        }
    }
}

// With rotation, keys, values and queries are three launches that neither read nor write one another's rows:
// each lets the next one start beside it, and ends after the one before it, so that the last one's end is
// the end of all.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void end_after_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename E, int kFmt, int kDim, bool kRope>
__global__ void __launch_bounds__(512, kRope ? 1 : 2) append_pages_kernel(const PageArgs a) {
    let_next_start();
    append_pages<E, kFmt, kDim, kRope>(a);
    end_after_last();
}

template <typename... Args>
cudaError_t launch_beside(void (*kernel)(Args...), dim3 grid, int threads, int smem, cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---------------------------------------------------------------- single tokens: sequence by sequence

constexpr int kTokenThreads = 512;
constexpr int kTokenWarps = kTokenThreads / 32;
constexpr int kRowsAtOnce = 4;

struct TokenArgs {
    KvAppendCall c;
    Wide wide;
};

// Queries first, first + step, .. before `last`, of no sequence or of no place, as they are: whole block.
template <typename E, int kDim>
__device__ __forceinline__ void copy_queries(const KvAppendCall& c, int first, int last, int step) {
    for (int64_t r = first; r < last; r += step) {
        const E* x = static_cast<const E*>(c.q.p) + r * c.q.token;
        E* y = static_cast<E*>(c.q_out.p) + r * c.q_out.token;
        for (int i = threadIdx.x; i < c.heads * kDim; i += blockDim.x) y[i / kDim * c.q_out.head + i % kDim] = x[i / kDim * c.q.head + i % kDim];
    }
}

// Rows of the token, a warp each: keys of every kv head, values of every kv head, queries.
template <typename E, int kFmt, int kDim>
__global__ void __launch_bounds__(kTokenThreads) append_token_kernel(const TokenArgs a) {
    constexpr int kN = 4;   // values a lane; a head of 64 takes half a warp
    __shared__ alignas(16) float cs[kDim / 2], sn[kDim / 2];
    const KvAppendCall& c = a.c;
    const KvBatch& b = c.batch;
    const int seq = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x % 32, d = lane * kN;
    if (seq >= b.batch) {  // queries of no sequence
        const Uncovered none = uncovered(b);
        copy_queries<E, kDim>(c, seq - b.batch, none.before, gridDim.x - b.batch);
        copy_queries<E, kDim>(c, none.after + seq - b.batch, b.total, gridDim.x - b.batch);
        return;
    }
    const SeqSpan span = seq_span(b, seq, c.wd);
    if (span.count == 0) {
        if (span.bad) copy_queries<E, kDim>(c, packed_row(b, seq), packed_row(b, seq + 1), 1);
        return;
    }
    const int64_t len = __ldg(b.lens + seq);
    const int page = c.cache.page, kv = c.cache.kv_heads;
    // rows are read before anything about pages is known
    const int rows = 2 * kv + c.heads;
    float x[kRowsAtOnce][kN], o[kRowsAtOnce][kN];
    auto source = [&](int r, bool& vec) {
        const Strided& s = r < kv ? c.k : r < 2 * kv ? c.v : c.q;
        vec = r < kv ? a.wide.k : r < 2 * kv ? a.wide.v : a.wide.q;
        const int h = r < kv ? r : r < 2 * kv ? r - kv : r - 2 * kv;
        return static_cast<const E*>(s.p) + static_cast<int64_t>(span.first) * s.token + h * s.head;
    };
    auto load = [&](int first) {
#pragma unroll
        for (int i = 0; i < kRowsAtOnce; ++i) {
            const int r = first + i * kTokenWarps;
            if (r >= rows) continue;
            bool vec;
            const E* row = source(r, vec);
#pragma unroll
            for (int e = 0; e < kN; ++e) x[i][e] = o[i][e] = 0.0f;
            if (d >= kDim) continue;
            load_values<E, kN>(row, d, vec, x[i]);
            if (c.rope.inv_freq != nullptr && (r < kv || r >= 2 * kv)) load_partners<E, kN>(row, d, vec, c.rope, o[i]);
        }
    };
    load(warp);
    bool in_range = len >= 0 && len < b.table_width * page;
    if (!in_range) report_range(c.wd);
    const int p = in_range ? seq_page(b, c.cache, seq, static_cast<int>(len >> (31 - __clz(page))), c.wd) : -1;  // a power of two
    const int place = in_range ? static_cast<int>(len & (page - 1)) : 0;
    // the old scales are on their way while cos and sin are computed
    float held_scale[kRowsAtOnce];
    auto block_of = [&](int r) { return static_cast<int64_t>(p) * kv + (r < kv ? r : r - kv); };
    auto load_scales = [&](int first) {
#pragma unroll
        for (int i = 0; i < kRowsAtOnce; ++i) {
            const int r = first + i * kTokenWarps;
            held_scale[i] = 0.0f;
            if (p >= 0 && place > 0 && r < 2 * kv) held_scale[i] = (r < kv ? c.cache.k_scale : c.cache.v_scale)[block_of(r)];
        }
    };
    load_scales(warp);
    if (c.rope.inv_freq != nullptr) {
        for (int j = threadIdx.x; j < c.rope.rotary / 2; j += kTokenThreads) {
            const float2 y = turn_cos_sin(turn_step(__ldg(c.rope.inv_freq + j)), static_cast<int>(len), c.rope.amplitude, c.rope.sign);
            cs[j] = y.x;
            sn[j] = y.y;
        }
        __syncthreads();
    }
    for (int first = warp; first < rows; first += kRowsAtOnce * kTokenWarps) {
        if (first != warp) {
            load(first);
            load_scales(first);
        }
#pragma unroll
        for (int i = 0; i < kRowsAtOnce; ++i) {
            const int r = first + i * kTokenWarps;
            if (r >= rows) continue;
            if (in_range && c.rope.inv_freq != nullptr && d < kDim && (r < kv || r >= 2 * kv)) rotate_values<kN>(x[i], o[i], d, cs, sn, c.rope);
            if (r >= 2 * kv) {
                E* y = static_cast<E*>(c.q_out.p) + static_cast<int64_t>(span.first) * c.q_out.token + (r - 2 * kv) * c.q_out.head;
                __syncwarp();  // in place, other lanes read their partners first
                if (d < kDim) store_values<E, kN>(y, d, a.wide.q_out, x[i]);
                continue;
            }
            if (p < 0) continue;
            const bool values = r >= kv;
            const int64_t ph = block_of(r);
            uint8_t* codes = (values ? c.cache.v : c.cache.k) + ph * page * kDim;
            float* scale = (values ? c.cache.v_scale : c.cache.k_scale) + ph;
            const float s_old = held_scale[i];
            float most = 0.0f;
#pragma unroll
            for (int e = 0; e < kN; ++e) most = max_finite(most, x[i][e]);
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, m));
            const float s = fmaxf(s_old, fmaxf(__fmul_rn(most, code_max_inverse<kFmt>()), kScaleFloor));
            const float per = __fdiv_rn(1.0f, s);
            if (place > 0 && s != s_old) {  // the held codes in the grown scale
                const float ratio = __fmul_rn(s_old, per);
                const int n = place * kDim / 16;
                uint4* held = reinterpret_cast<uint4*>(codes);
                for (int at = lane; at < n; at += 4 * 32) {
                    uint4 w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (at + 32 * j < n) w[j] = held[at + 32 * j];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (at + 32 * j < n)
                            held[at + 32 * j] = make_uint4(again4<kFmt>(w[j].x, ratio), again4<kFmt>(w[j].y, ratio), again4<kFmt>(w[j].z, ratio),
                                                           again4<kFmt>(w[j].w, ratio));
                }
            }
            uint32_t w[1];
            encode_values<kFmt, kN>(x[i], most, per, w);
            if (d < kDim) *reinterpret_cast<uint32_t*>(codes + place * kDim + d) = w[0];
            __syncwarp();  // every lane has read the old scale
            if (lane == 0 && s != s_old) *scale = s;
        }
    }
}

// ---------------------------------------------------------------- queries beside a prompt's keys

constexpr int kQTokens = 4;  // per CTA, where rows are not whole 16-byte pieces

// The positions of tokens token0 .. token0 + n - 1; -1 for one of no sequence, or of one that does not fit.
__device__ __forceinline__ void q_positions(const KvAppendCall& c, int32_t* where, int token0, int n) {
    const KvBatch& b = c.batch;
    const int first = block_find(b.batch, [&](int i) { return static_cast<int64_t>(b.cu ? __ldg(b.cu + i) : i); }, token0);
    if (threadIdx.x < n) {
        const int token = token0 + threadIdx.x;
        int seq = first, at = -1;
        while (seq + 1 < b.batch && (b.cu ? __ldg(b.cu + seq + 1) : seq + 1) <= token) ++seq;
        const SeqSpan span = seq_span(b, seq, c.wd);
        if (token >= span.first && token < span.first + span.count) {
            const int64_t len = __ldg(b.lens + seq);
            if (len >= 0 && len + span.count <= b.table_width * c.cache.page) at = static_cast<int>(len) + token - span.first;  // or the keys' kernel reports it
        }
        where[threadIdx.x] = at;
    }
}

template <typename E, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads, 4) append_q_kernel(const KvAppendCall c, const RopeRows r) {
    extern __shared__ float smem[];
    rope_rows<E, kHalf, true>(r, smem, [&](int32_t* where, int token0, int n) { q_positions(c, where, token0, n); });
    end_after_last();
}

// Any alignment and rotary width: pair by pair.
template <typename E>
__global__ void __launch_bounds__(kRopeThreads) append_q_any_kernel(const KvAppendCall c) {
    extern __shared__ float turns[];
    __shared__ int32_t where[kQTokens];
    const int token0 = blockIdx.x * kQTokens, n = min(kQTokens, c.batch.total - token0);
    q_positions(c, where, token0, n);
    __syncthreads();
    const int half = c.rope.rotary / 2, dim = c.cache.dim;
    float *cs = turns, *sn = turns + n * half;
    for (int i = threadIdx.x; i < n * half; i += kRopeThreads) {
        const int t = i / half;
        const float2 x = turn_cos_sin(turn_step(__ldg(c.rope.inv_freq + (i - t * half))), where[t], c.rope.amplitude, c.rope.sign);
        cs[i] = x.x;
        sn[i] = x.y;
    }
    __syncthreads();
    const int per_head = half + dim - c.rope.rotary;
    for (int i = threadIdx.x; i < n * c.heads * per_head; i += kRopeThreads) {
        const int row = i / per_head, j = i - row * per_head, t = row / c.heads, h = row - t * c.heads;
        const bool turns = where[t] >= 0;
        const E* x = static_cast<const E*>(c.q.p) + static_cast<int64_t>(token0 + t) * c.q.token + h * c.q.head;
        E* y = static_cast<E*>(c.q_out.p) + static_cast<int64_t>(token0 + t) * c.q_out.token + h * c.q_out.head;
        if (j < half) {
            const int ia = c.rope.layout == kRopeHalf ? j : 2 * j, ib = c.rope.layout == kRopeHalf ? j + half : 2 * j + 1;
            const float cc = cs[t * half + j], ss = sn[t * half + j];
            const E xa = x[ia], xb = x[ib];
            const float u = to_float(xa), w = to_float(xb);
            y[ia] = turns ? from_float<E>(u * cc - w * ss) : xa;
            y[ib] = turns ? from_float<E>(w * cc + u * ss) : xb;
        } else {
            y[half + j] = x[half + j];
        }
    }
    end_after_last();
}

// ---------------------------------------------------------------- reading back

constexpr int kReadThreads = 256;
constexpr int kReadRows = 16;  // packed rows a CTA
constexpr int kNoSequence = -2;  // in the place of a row's page: the row comes back as zeros (-1: it is left as it is)

// Eight codes in, eight values out, a thread: consecutive threads take consecutive pieces of a row of
// all heads, so the output is written in whole lines and the codes are read in lines of a head.
template <typename E, int kFmt, int kDim>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const KvReadCall c) {
    __shared__ int32_t page_of[kReadRows], place_of[kReadRows];
    const KvBatch& b = c.batch;
    const int row0 = blockIdx.x * kReadRows, n = min(kReadRows, b.total - row0), page = c.cache.page, heads = c.cache.kv_heads;
    constexpr int kPieces = kDim / 8;
    const int first = block_find(b.batch, [&](int i) { return static_cast<int64_t>(b.cu ? __ldg(b.cu + i) : i); }, row0);
    if (threadIdx.x < n) {
        const int row = row0 + threadIdx.x;
        int seq = first, p = kNoSequence, place = 0;
        while (seq + 1 < b.batch && (b.cu ? __ldg(b.cu + seq + 1) : seq + 1) <= row) ++seq;
        const SeqSpan span = b.batch > 0 ? seq_span(b, seq, c.wd) : SeqSpan{0, 0, false};
        if (row >= span.first && row < span.first + span.count) {
            const int64_t pos = static_cast<int64_t>(__ldg(b.lens + seq)) + row - span.first;
            p = -1;
            if (pos < 0 || pos >= b.table_width * page) report_range(c.wd);
            else {
                p = seq_page(b, c.cache, seq, static_cast<int>(pos / page), c.wd);
                place = static_cast<int>(pos % page);
            }
        }
        page_of[threadIdx.x] = p;
        place_of[threadIdx.x] = place;
    }
    __syncthreads();
    const int per_row = heads * kPieces, items = n * per_row;
    constexpr int kAtOnce = 4;
    for (int i0 = threadIdx.x; i0 < items; i0 += kAtOnce * kReadThreads) {
        uint2 kc[kAtOnce], vc[kAtOnce];
        float ks[kAtOnce], vs[kAtOnce];
        int64_t to[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int i = i0 + j * kReadThreads;
            to[j] = -1;
            if (i >= items) continue;
            const int row = i / per_row, in = i - row * per_row, h = in / kPieces, d = (in - h * kPieces) * 8;
            const int p = page_of[row];
            if (p == -1) continue;
            to[j] = static_cast<int64_t>(row0) * per_row * 8 + static_cast<int64_t>(i) * 8;
            if (p == kNoSequence) {
                kc[j] = vc[j] = make_uint2(0, 0);
                ks[j] = vs[j] = 0.0f;
                continue;
            }
            const int64_t ph = static_cast<int64_t>(p) * heads + h, at = (ph * page + place_of[row]) * kDim + d;
            kc[j] = __ldg(reinterpret_cast<const uint2*>(c.cache.k + at));
            vc[j] = __ldg(reinterpret_cast<const uint2*>(c.cache.v + at));
            ks[j] = __ldg(c.cache.k_scale + ph);
            vs[j] = __ldg(c.cache.v_scale + ph);
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            if (to[j] < 0) continue;
            float lo[4], hi[4], x[8];
            decode4<kFmt>(kc[j].x, lo);
            decode4<kFmt>(kc[j].y, hi);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = lo[e] * ks[j];
                x[4 + e] = hi[e] * ks[j];
            }
            store_values<E, 8>(static_cast<E*>(c.k) + to[j], 0, true, x);
            decode4<kFmt>(vc[j].x, lo);
            decode4<kFmt>(vc[j].y, hi);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = lo[e] * vs[j];
                x[4 + e] = hi[e] * vs[j];
            }
            store_values<E, 8>(static_cast<E*>(c.v) + to[j], 0, true, x);
        }
    }
}

bool is_wide(const Strided& s) { return reinterpret_cast<uintptr_t>(s.p) % 16 == 0 && s.token % 8 == 0 && s.head % 8 == 0; }

template <typename E, int kFmt, int kDim>
cudaError_t launch_append(const KvAppendCall& c, int sm_count, cudaStream_t stream) {
    const Wide wide{is_wide(c.k), is_wide(c.v), is_wide(c.q), is_wide(c.q_out)};
    if (c.batch.max_new == 1 || c.batch.batch == 0) {
        // queries of no sequence are copied by CTAs of their own, which look whether there are any (those of the sequences
        // would wait for the offsets: 256 tokens in 10.5 us a call, not 10.0)
        int copies = 0;
        if (c.heads > 0 && c.batch.cu != nullptr && c.q.p != c.q_out.p) {
            copies = c.batch.total - c.batch.batch;
            copies = copies < 1 ? 1 : copies > sm_count ? sm_count : copies;
        }
        if (c.batch.batch + copies == 0) return cudaSuccess;
        append_token_kernel<E, kFmt, kDim><<<c.batch.batch + copies, kTokenThreads, 0, stream>>>(TokenArgs{c, wide});
        return cudaGetLastError();
    }
    const int group = c.cache.page * kDim / 8 / kVecs;
    const int threads = group > 128 ? group : 128, groups = threads / group;
    const int half = c.rope.inv_freq != nullptr ? c.rope.rotary / 2 : 0;
    const int smem = c.cache.page * half * 2 * static_cast<int>(sizeof(float));
    const int items = c.batch.total / c.cache.page + 2 * c.batch.batch;
    // a CTA takes the heads of a page one after another, as many as leave a number of CTAs an SM: what comes
    // before the first head (five dependent reads, and for keys cos and sin of the page) is paid once,
    // and the next head's values are on their way while one is written
    auto heads_for = [&](int64_t ctas_a_round, int ctas_a_sm) {
        int heads = groups;
        while (heads < c.cache.kv_heads && ctas_a_round * ((c.cache.kv_heads + 2 * heads - 1) / (2 * heads)) >= ctas_a_sm * sm_count) heads *= 2;
        return heads;
    };
    auto rounds_of = [&](const PageArgs& p) { return static_cast<unsigned>((c.cache.kv_heads + p.heads_a_cta - 1) / p.heads_a_cta); };
    if (half == 0) {
        const PageArgs both{c, wide, heads_for(2 * items, 8), 0};
        append_pages_kernel<E, kFmt, kDim, false><<<dim3(items, rounds_of(both), 2), threads, 0, stream>>>(both);
        return cudaGetLastError();
    }
    static int attr_gen[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    auto* turning = append_pages_kernel<E, kFmt, kDim, true>;
    if (dev < 64 && attr_gen[dev] != g_generation) {
        if ((e = cudaFuncSetAttribute(turning, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * kDim * 4)) != cudaSuccess) return e;
        attr_gen[dev] = g_generation;
    }
    // Turned keys: as few CTAs as still fill one wave, two of 256 threads or the like an SM by their registers, since
    // each pays for cos and sin of its page. 17 410 tokens, the whole call with four or eight CTAs an SM
    // instead: 113 and 134 us with pages of 64, not 102 (before later steps took all of them down).
    const PageArgs of_keys{c, wide, heads_for(items, 512 / threads), 0}, of_values{c, wide, heads_for(items, 8), 1};
    turning<<<dim3(items, rounds_of(of_keys)), threads, smem, stream>>>(of_keys);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    e = launch_beside(append_pages_kernel<E, kFmt, kDim, false>, dim3(items, rounds_of(of_values)), threads, 0, stream, of_values);
    if (e != cudaSuccess || c.heads == 0) return e;
    if (!rope_whole(c.q, c.q_out, kDim, c.rope))
        return launch_beside(append_q_any_kernel<E>, (c.batch.total + kQTokens - 1) / kQTokens, kRopeThreads,
                             kQTokens * half * 2 * static_cast<int>(sizeof(float)), stream, c);
    const RopeRows r = rope_rows_of(c.q, c.q_out, c.batch.total, c.heads, kDim, c.rope, sm_count);
    auto* kernel = c.rope.layout == kRopeHalf ? append_q_kernel<E, true> : append_q_kernel<E, false>;
    return launch_beside(kernel, rope_grid(r), kRopeThreads, rope_smem(r), stream, c, r);
}

template <typename E, int kFmt, int kDim>
cudaError_t launch_read(const KvReadCall& c, int, cudaStream_t stream) {
    read_kernel<E, kFmt, kDim><<<(c.batch.total + kReadRows - 1) / kReadRows, kReadThreads, 0, stream>>>(c);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendCall& c, int sm_count, cudaStream_t stream) {
    const bool h = c.dtype == kFp16, e4 = c.cache.fmt == kKvE4M3, d128 = c.cache.dim == 128;
    auto go = [&](auto* f) { return f(c, sm_count, stream); };
    if (h && e4) return d128 ? go(launch_append<__half, kKvE4M3, 128>) : go(launch_append<__half, kKvE4M3, 64>);
    if (h) return d128 ? go(launch_append<__half, kKvInt8, 128>) : go(launch_append<__half, kKvInt8, 64>);
    if (e4) return d128 ? go(launch_append<__nv_bfloat16, kKvE4M3, 128>) : go(launch_append<__nv_bfloat16, kKvE4M3, 64>);
    return d128 ? go(launch_append<__nv_bfloat16, kKvInt8, 128>) : go(launch_append<__nv_bfloat16, kKvInt8, 64>);
}

cudaError_t launch_kv_read(const KvReadCall& c, int sm_count, cudaStream_t stream) {
    const bool h = c.dtype == kFp16, e4 = c.cache.fmt == kKvE4M3, d128 = c.cache.dim == 128;
    auto go = [&](auto* f) { return f(c, sm_count, stream); };
    if (h && e4) return d128 ? go(launch_read<__half, kKvE4M3, 128>) : go(launch_read<__half, kKvE4M3, 64>);
    if (h) return d128 ? go(launch_read<__half, kKvInt8, 128>) : go(launch_read<__half, kKvInt8, 64>);
    if (e4) return d128 ? go(launch_read<__nv_bfloat16, kKvE4M3, 128>) : go(launch_read<__nv_bfloat16, kKvE4M3, 64>);
    return d128 ? go(launch_read<__nv_bfloat16, kKvInt8, 128>) : go(launch_read<__nv_bfloat16, kKvInt8, 64>);
}

}  // namespace tg
