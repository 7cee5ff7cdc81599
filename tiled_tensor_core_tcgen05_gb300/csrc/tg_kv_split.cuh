// What the two kernels of the cache attention share: the even split of a batch's
// work and the joining of units that cross shares, and the codes' way to fp16.
#pragma once

#include "tg_device.cuh"
#include "tg_kv.cuh"

namespace tg {

// wait_phase for warps that share their scheduler with others' arithmetic: the hardware suspends the
// warp for up to 20 us a try, where shorter tries in a loop took half of the issue slots from the
// exponentials beside them. Same bound and abort rules.
__device__ __forceinline__ bool wait_suspended(uint32_t bar, uint32_t parity, const WaitCtx& w, int site) {
    uint64_t t0 = 0;
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(20000u)
            : "memory");
        if (ok) return true;
        if (*w.abort) return false;
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) {
            t0 = now;
        } else if (now - t0 > w.limit_ns) {
            *w.abort = 1;
            atomicCAS(w.status, 0, site);
            return false;
        }
    }
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNoMax = -1e30f;        // a row's reference before any visible key

// A row's weights are 2^(t - m) for a reference m that follows the row's maximum from kHeadroomLog2 below, and that
// moves only when a weight would pass 2^kMostLog2, near fp16's largest value. The sums carry the same factor, so the
// quotient and m + log2 of the sum do not know where m lies: it is chosen for fp16, in which the weights go into
// their product. Its ordinary values end at 2^-14 and its last one is 2^-24, so a key keeps 11 bits down to
// 2^-23 of the largest weight and counts for something down to 2^-34 of it, however many such keys there are under one
// that dominates. More headroom means that m moves more often (the chunks of k_kv_tile.cu take 675 us with 7,
// 676 with 9, 680 with 10).
constexpr float kHeadroomLog2 = 9.0f;
constexpr float kMostLog2 = 15.99f;

// Where CTA k of `ctas` begins in a list of `total` chunks: equal shares, the first ones one longer.
struct Shares {
    int64_t each;
    int rest;
    int ctas;
    __device__ Shares(int64_t total, int grid, int least) {
        const int64_t most = (total + least - 1) / least;
        ctas = static_cast<int>(min(static_cast<int64_t>(grid), most));
        each = ctas > 0 ? total / ctas : 0;
        rest = ctas > 0 ? static_cast<int>(total - each * ctas) : 0;
    }
    __device__ int64_t start(int k) const { return k * each + min(k, rest); }
    __device__ int owner(int64_t chunk) const {
        const int64_t longer = (each + 1) * rest;
        return static_cast<int>(chunk < longer ? chunk / (each + 1) : rest + (chunk - longer) / each);
    }
};

// What CTA k leaves for the joining kernel: the unit of which its share begins past the first chunk
// (chunks 0: none), and where that unit's entries begin in the list.
struct Meta {
    int64_t unit_start, total;
    int chunks, head, block;
    int first, count;   // the sequence's rows of the packed tensors
    int part;           // whether keys of the sequence are left to another call
};

// A split call: what both kernels and the join need.
struct SplitWork {
    KvAttnCall c;
    int share;          // query heads per kv head
    int least;          // fewest list entries worth a CTA
    int extra;          // entries before a unit's first chunk, for what every unit costs whatever its length
    int grid;
    int joined;         // whether the joining kernel runs
    int box;            // tokens a copy of codes, in the kernel for many rows
    int q_vec;          // Q aligned, and strides whole, for the kernel's wide loads
    int page_shift;
    Meta* meta;         // grid entries
    float* parts;       // grid x 2 parts: rows x (dim + 2) floats each (values, then references, then sums)
};

// Byte offset of piece `at` (bytes) of token t among tokens that TMA left as lines of 128 bytes, swizzled.
template <int kDim>
__device__ __forceinline__ int ring_offset(int t, int at) {
    const int line = kDim == 128 ? t : t >> 1;
    const int in = kDim == 128 ? at : (t & 1) * 64 + at;
    return line * 128 + (in ^ ((line & 7) << 4));
}

// Four codes to two fp16 pairs (codes 0 1, codes 2 3).
template <int kFmt>
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (kFmt == kKvE4M3) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        // code + 128 as the low byte of 1024 + (code + 128) in fp16, whose steps are 1 there
        const uint32_t u = w ^ 0x80808080u;
        const __half2 bias = __half2half2(__ushort_as_half(static_cast<unsigned short>(0x6480)));  // 1152
        uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), bias), y = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
        lo = *reinterpret_cast<const uint32_t*>(&x);
        hi = *reinterpret_cast<const uint32_t*>(&y);
    }
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr int kStep = 16;  // tokens a box of the cache's tensor maps

// 1 / a row's sum; 0 for a row that sees nothing.
__device__ __forceinline__ float row_inverse(float l) { return l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l); }

// The natural log of a row's sum l at the reference m (base 2). The sum's exponent goes to m first: the two are of
// about the same size and opposite signs where scores are small, and log2f(l) would be rounded at that size.
__device__ __forceinline__ float row_lse(float m, float l) {
    if (l == 0.0f) return -INFINITY;
    const int bits = __float_as_int(l), e = (bits >> 23) - 127;
    if (e <= -127 || e >= 128) return (m + log2f(l)) * (1.0f / kLog2e);  // not an ordinary positive number
    return (m + static_cast<float>(e) + log2f(__int_as_float((bits & 0x7FFFFF) | 0x3F800000))) * (1.0f / kLog2e);
}

// What the first of two calls says of a row that it has finished.
constexpr float2 kDone{0.0f, -1.0f};

// In the second of two calls: waits for the first, whose last kernel lets this one begin early.
__device__ __forceinline__ void wait_for_first() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Row r of the outputs as that of a token that sees nothing: whole block.
template <typename E, int kDim>
__device__ __forceinline__ void clear_row(const KvAttnCall& c, int64_t r) {
    uint4* y = reinterpret_cast<uint4*>(static_cast<E*>(c.out) + r * c.heads * kDim);
    for (int x = threadIdx.x; x < c.heads * (kDim / 8); x += blockDim.x) y[x] = make_uint4(0, 0, 0, 0);
    for (int h = threadIdx.x; c.lse != nullptr && h < c.heads; h += blockDim.x) c.lse[r * c.heads + h] = -INFINITY;
    for (int h = threadIdx.x; c.found != nullptr && h < c.heads; h += blockDim.x) c.found_weight[r * c.heads + h] = kDone;
}

// Clears the rows that no sequence has, and those of spans out of range, the grid's CTAs together. The joining kernel
// does it while the parts are being computed; where there is none, the kernel itself.
template <typename E, int kDim>
__device__ __forceinline__ void clear_uncovered(const KvAttnCall& c) {
    if (c.batch.cu == nullptr || c.seed != nullptr) return;  // the first of two calls has done it
    const Uncovered none = uncovered(c.batch);
    const int many = none.before + c.batch.total - none.after;
    for (int i = blockIdx.x; i < many; i += gridDim.x) clear_row<E, kDim>(c, i < none.before ? i : none.after + i - none.before);
    for (int i = blockIdx.x; i < c.batch.batch; i += gridDim.x)
        if (seq_span(c.batch, i, c.wd).bad)
            for (int r = packed_row(c.batch, i); r < packed_row(c.batch, i + 1); ++r) clear_row<E, kDim>(c, r);
}

// kN values from d on of row and head `to`, all of whose units are joined: their sum v of values times weights, the
// weights' reference and sum. Writes what the call leaves. kParts: it is one of two; `part`: keys of the sequence are left to the
// second.
template <typename E, int kDim, int kN, bool kParts>
__device__ __forceinline__ void finish_row(const KvAttnCall& c, int64_t to, int d, float (&v)[kN], float top, float sum, bool part) {
    if (kParts && c.found != nullptr) {
        if (d == 0) c.found_weight[to] = part ? make_float2(top, sum) : kDone;
        if (part) {
#pragma unroll
            for (int i = 0; i < kN; i += 2) *reinterpret_cast<float2*>(c.found + to * kDim + d + i) = make_float2(v[i], v[i + 1]);
            return;
        }
    }
    if (kParts && c.seed != nullptr) {
        const float2 w = c.seed_weight[to];
        if (w.y < 0.0f) return;
        const float all = fmaxf(top, w.x), a = ex2_approx(top - all), b = ex2_approx(w.x - all);
        top = all;
        sum = fmaf(sum, a, w.y * b);
#pragma unroll
        for (int i = 0; i < kN; i += 2) {
            const float2 x = *reinterpret_cast<const float2*>(c.seed + to * kDim + d + i);
            v[i] = fmaf(v[i], a, x.x * b);
            v[i + 1] = fmaf(v[i + 1], a, x.y * b);
        }
    }
    const float inv = row_inverse(sum);
    E out[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) out[i] = from_float<E>(v[i] * inv);
    E* y = static_cast<E*>(c.out) + to * kDim + d;
    if constexpr (kN == 4) *reinterpret_cast<uint2*>(y) = *reinterpret_cast<const uint2*>(out);
    else *reinterpret_cast<uint32_t*>(y) = *reinterpret_cast<const uint32_t*>(out);
    if (d == 0 && c.lse != nullptr) c.lse[to] = row_lse(top, sum);
}

// Whether share k begins inside a unit whose first border that is.
__device__ __forceinline__ bool first_border(const SplitWork& a, const Meta& m, int k) {
    return m.chunks != 0 && Shares(m.total, a.grid, a.least).start(k - 1) <= m.unit_start + a.extra;
}

// Joins the parts of row r of the unit inside which share k begins, if k's is its first border: a warp, kDim / 32 values a lane.
// The order of the parts is that of their keys. What a part counts for is computed once, a part a lane.
template <typename E, int kDim, int kRows, bool kParts>
__device__ __forceinline__ void join_row(const SplitWork& a, int k, int r) {
    constexpr int kN = kDim / 32;
    const KvAttnCall& c = a.c;
    const int lane = threadIdx.x % 32;
    const Meta m = a.meta[k];
    if (m.chunks == 0) return;
    const Shares shares(m.total, a.grid, a.least);
    const int64_t before = shares.start(k - 1), first_chunk = m.unit_start + a.extra;
    if (before > first_chunk) return;  // an earlier border lies in the unit's chunks
    const int row = m.block * kRows + r;
    if (row >= m.count * a.share) return;
    const int last = shares.owner(first_chunk + m.chunks - 1);
    auto part_of = [&](int x) {
        const int slot = x == k - 1 && before < m.unit_start ? 1 : 0;
        return a.parts + (static_cast<int64_t>(2 * x) + slot) * kRows * (kDim + 2);
    };
    struct alignas(4 * kN) Values {
        float v[kN];
    };
    auto values_of = [&](int x) { return *reinterpret_cast<const Values*>(part_of(x) + r * kDim + lane * kN); };
    // the first parts' values are on their way while the maxima and sums are read and compared
    constexpr int kAhead = 8;
    Values ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (k - 1 + i <= last) ahead[i] = values_of(k - 1 + i);
    float top = kNoMax, own_m = kNoMax, own_l = 0.0f;
    for (int x = k - 1 + lane; x <= last; x += 32) {
        const float y = part_of(x)[kRows * kDim + r];
        if (x < k - 1 + 32) {
            own_m = y;
            own_l = part_of(x)[kRows * (kDim + 1) + r];
        }
        top = fmaxf(top, y);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    float v[kN] = {}, sum = 0.0f;
    for (int x0 = k - 1; x0 <= last; x0 += 32) {
        if (x0 > k - 1) {
            const int x = x0 + lane;
            own_m = x <= last ? part_of(x)[kRows * kDim + r] : kNoMax;
            own_l = x <= last ? part_of(x)[kRows * (kDim + 1) + r] : 0.0f;
        }
        const float keep = ex2_approx(own_m - top), l = own_l * keep;
        const int many = min(32, last + 1 - x0);
        auto add = [&](int i, const Values& y) {
            const float w = __shfl_sync(0xFFFFFFFFu, keep, i);
            sum += __shfl_sync(0xFFFFFFFFu, l, i);
#pragma unroll
            for (int e = 0; e < kN; ++e) v[e] = fmaf(y.v[e], w, v[e]);
        };
        for (int i = 0; i < many; i += kAhead) {  // a group's reads together
            if (x0 > k - 1 || i > 0) {
#pragma unroll
                for (int j = 0; j < kAhead; ++j)
                    if (i + j < many) ahead[j] = values_of(x0 + i + j);
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (i + j < many) add(i + j, ahead[j]);
        }
    }
    const int t = row / a.share;
    const int64_t to = static_cast<int64_t>(m.first + t) * c.heads + m.head * a.share + row - t * a.share;
    finish_row<E, kDim, kN, kParts>(c, to, lane * kN, v, top, sum, m.part != 0);
}

// The same for units of many rows, whose parts hold their values in pieces of four, of eight rows one behind another (part_offset): a lane of the kernel
// that writes them has a row, so a warp's store is whole lines (rows one behind another: 32 quarters of lines, and 3 us more at a share's end). Here a
// warp reads 16 values of eight rows, whole lines too.
template <int kDim>
__device__ __forceinline__ int part_offset(int r, int d) { return ((r / 8 * (kDim / 4) + d / 4) * 8 + r % 8) * 4; }

template <typename E, int kDim, int kRows, bool kParts>
__device__ __forceinline__ void join_eight(const SplitWork& a, int k, int eight, int d) {
    const KvAttnCall& c = a.c;
    const Meta m = a.meta[k];
    if (m.chunks == 0) return;
    const Shares shares(m.total, a.grid, a.least);
    const int64_t before = shares.start(k - 1), first_chunk = m.unit_start + a.extra;
    if (before > first_chunk) return;  // an earlier border lies in the unit's chunks
    const int r = eight * 8 + threadIdx.x % 8, row = m.block * kRows + r;
    if (row >= m.count * a.share) return;
    const int last = shares.owner(first_chunk + m.chunks - 1);
    auto part_of = [&](int x) {
        const int slot = x == k - 1 && before < m.unit_start ? 1 : 0;
        return a.parts + (static_cast<int64_t>(2 * x) + slot) * kRows * (kDim + 2);
    };
    constexpr int kAhead = 8;  // parts whose reads are together; those of the first are on their way while the references are compared
    float4 y[kAhead];
    float ref[kAhead], l[kAhead];
    auto read = [&](int x0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (x0 + i <= last) y[i] = *reinterpret_cast<const float4*>(part_of(x0 + i) + part_offset<kDim>(r, d));
    };
    auto read_rest = [&](int x0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            ref[i] = x0 + i <= last ? part_of(x0 + i)[kRows * kDim + r] : kNoMax;
            l[i] = x0 + i <= last ? part_of(x0 + i)[kRows * (kDim + 1) + r] : 0.0f;
        }
    };
    read(k - 1);
    read_rest(k - 1);
    float top = kNoMax, sum = 0.0f, v[4] = {};
#pragma unroll
    for (int i = 0; i < kAhead; ++i) top = fmaxf(top, ref[i]);
    for (int x0 = k - 1 + kAhead; x0 <= last; x0 += kAhead)
#pragma unroll
        for (int i = 0; i < kAhead; ++i) top = fmaxf(top, x0 + i <= last ? part_of(x0 + i)[kRows * kDim + r] : kNoMax);
    for (int x0 = k - 1; x0 <= last; x0 += kAhead) {
        if (x0 > k - 1) {
            read(x0);
            read_rest(x0);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (x0 + i <= last) {
                const float w = ex2_approx(ref[i] - top);
                sum = fmaf(l[i], w, sum);
                v[0] = fmaf(y[i].x, w, v[0]);
                v[1] = fmaf(y[i].y, w, v[1]);
                v[2] = fmaf(y[i].z, w, v[2]);
                v[3] = fmaf(y[i].w, w, v[3]);
            }
    }
    const int t = row / a.share;
    const int64_t to = static_cast<int64_t>(m.first + t) * c.heads + m.head * a.share + row - t * a.share;
    finish_row<E, kDim, 4, kParts>(c, to, d, v, top, sum, m.part != 0);
}

// Block (k - 1, a piece of the rows). Where groups of many rows share keys, units are few, and so are the borders that are a unit's
// first: a grid of about what the GPU holds looks for them (a thread a border) and shares their rows out (64 sequences on 8192 shared tokens 89 -> 84 us;
// prompt chunks, where nearly every border is one, take 677 us that way and 667 with a block a border and piece).
constexpr int kJoinWarps = 8;
constexpr int kMostBorders = 1024;
template <int kDim, int kRows>
constexpr int kJoinPieces = kRows <= 64 ? kRows / kJoinWarps : kRows * kDim / (kJoinWarps * 128);  // a warp has a row, or 128 values of eight

template <typename E, int kDim, int kRows, bool kParts>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_join_kernel(const SplitWork a) {
    if constexpr (kParts) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.y == 0) clear_uncovered<E, kDim>(a.c);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    constexpr int kPieces = kJoinPieces<kDim, kRows>;
    auto join = [&](int k, int piece) {
        if constexpr (kRows <= 64) {
            join_row<E, kDim, kRows, kParts>(a, k, piece * kJoinWarps + warp);
        } else {
            const int at = piece * kJoinWarps + warp;  // of all 16 values of eight rows
            join_eight<E, kDim, kRows, kParts>(a, k, at / (kDim / 16), at % (kDim / 16) * 16 + lane / 8 * 4);
        }
    };
    if constexpr (!kParts || kRows <= 64) {
        join(blockIdx.x + 1, blockIdx.y);
    } else {
        __shared__ int borders[kMostBorders], found[kJoinWarps];
        int n = 0;
        for (int base = 1; base < a.grid; base += 32 * kJoinWarps) {
            const int k = base + threadIdx.x;
            const bool yes = k < a.grid && first_border(a, a.meta[k], k);
            const uint32_t all = __ballot_sync(0xFFFFFFFFu, yes);
            if (lane == 0) found[warp] = __popc(all);
            __syncthreads();
            for (int w = 0; w < kJoinWarps; ++w) {
                if (w == warp && yes) borders[n + __popc(all & ((1u << lane) - 1))] = k;
                n += found[w];
            }
            __syncthreads();
        }
        for (int i = blockIdx.x; i < n * kPieces; i += gridDim.x) join(borders[i / kPieces], i % kPieces);
    }
}

// Launches a call's first kernel; that of the second of two calls so that it begins while the first one's last does.
template <typename K>
cudaError_t launch_attn(K* kernel, const SplitWork& a, const CUtensorMap& tmK, const CUtensorMap& tmV, int grid, int threads, int smem, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = a.c.seed != nullptr ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, tmK, tmV, a);
}

// Launches the join so that its blocks are in place when the parts are.
template <typename E, int kDim, int kRows, bool kParts>
cudaError_t launch_join(const SplitWork& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = !kParts || kRows <= 64 ? dim3(a.grid - 1, kJoinPieces<kDim, kRows>) : dim3(8 * a.grid);
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<E, kDim, kRows, kParts>, a);
}

}  // namespace tg
