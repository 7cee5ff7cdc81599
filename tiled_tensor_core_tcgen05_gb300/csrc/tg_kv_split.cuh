// What the two kernels of the cache attention share: the even split of a batch's
// work and the joining of units that cross shares, and the codes' way to fp16.
#pragma once

#include "tg_kv.cuh"

namespace tg {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNoMax = -1e30f;        // running maximum before any visible key
constexpr float kRescaleLog2 = 8.0f;    // the maximum moves only when a weight would pass 2^8

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

// What CTA k leaves for the joining kernel: the unit that its share begins inside of (chunks 0: none).
struct Meta {
    int64_t unit_start, total;
    int chunks, seq, head, block;
};

// A split call: what both kernels and the join need.
struct SplitWork {
    KvAttnCall c;
    int share;          // query heads per kv head
    int least;          // fewest list entries worth a CTA
    int grid;
    int q_vec;          // Q aligned, and strides whole, for the kernel's wide loads
    int page_shift;
    Meta* meta;         // grid entries
    float* parts;       // grid x 2 parts: rows x (dim + 2) floats each (values, then maxima, then sums)
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

// The natural log of a row's sum l at the running maximum m (base 2).
__device__ __forceinline__ float row_lse(float m, float l) { return l == 0.0f ? -INFINITY : (m + log2f(l)) * (1.0f / kLog2e); }

// Joins the parts of the unit inside which share k begins, if k's is its first border: block
// (k - 1, rows blockIdx.y, blockIdx.y + gridDim.y, ..), a thread a value. The order of the parts is
// that of their keys.
template <typename E, int kDim, int kRows>
__global__ void __launch_bounds__(kDim) attn_join_kernel(const SplitWork a) {
    const KvAttnCall& c = a.c;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int k = blockIdx.x + 1, d = threadIdx.x;
    const Meta m = a.meta[k];
    if (m.chunks == 0) return;
    const Shares shares(m.total, a.grid, a.least);
    const int64_t before = shares.start(k - 1);
    if (before > m.unit_start) return;  // an earlier border lies in the unit
    const SeqSpan span = seq_span(c.batch, m.seq, c.wd);
    const int last = shares.owner(m.unit_start + m.chunks - 1);
    auto part_of = [&](int x) {
        const int slot = x == k - 1 && before < m.unit_start ? 1 : 0;
        return a.parts + (static_cast<int64_t>(2 * x) + slot) * kRows * (kDim + 2);
    };
    for (int r = blockIdx.y; r < kRows; r += gridDim.y) {
        const int row = m.block * kRows + r;
        if (row >= span.count * a.share) return;
        float top = kNoMax;
#pragma unroll 4
        for (int x = k - 1; x <= last; ++x) top = fmaxf(top, part_of(x)[kRows * kDim + r]);
        float v = 0.0f, sum = 0.0f;
#pragma unroll 4
        for (int x = k - 1; x <= last; ++x) {
            const float* p = part_of(x);
            const float keep = ex2_approx(p[kRows * kDim + r] - top);
            sum += p[kRows * (kDim + 1) + r] * keep;
            v += p[r * kDim + d] * keep;
        }
        const int t = row / a.share;
        const int64_t to = static_cast<int64_t>(span.first + t) * c.heads + m.head * a.share + row - t * a.share;
        static_cast<E*>(c.out)[to * kDim + d] = from_float<E>(v * row_inverse(sum));
        if (d == 0 && c.lse != nullptr) c.lse[to] = row_lse(top, sum);
    }
}

// Launches the join so that its blocks are in place when the parts are: `rows_y` of them a border.
template <typename E, int kDim, int kRows>
cudaError_t launch_join(const SplitWork& a, int rows_y, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.grid - 1, rows_y);
    cfg.blockDim = dim3(kDim);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<E, kDim, kRows>, a);
}

}  // namespace tg
