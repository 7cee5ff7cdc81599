// Rotary positions: pairs of values of each head turned by position times a
// frequency of the pair,
//
//     y_a = amplitude (x_a cos t - x_b sin t),  y_b = amplitude (x_b cos t + x_a sin t),
//     t = position * inv_freq[pair],
//
// for the first `rotary` values of a head; the rest pass through. The gradient
// is the transposed map, the same kernel with the sign of sin turned round.
// Angles are exact fractions of a turn (tg_kv.cuh), products and sums are fp32,
// and each value is rounded once to its 16-bit type.
//
// Memory bounds it: every value is read and written once. A CTA takes a few
// tokens, so that cos and sin, about forty instructions a pair, are computed
// once for all heads of a token (in shared memory, two arrays so that a
// thread's eight of each are two 16-byte reads), and each thread's loads are
// under way before it computes them.
#include "tg_kv.cuh"

namespace tg {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;  // per CTA

// ---- any alignment and any rotary width: one pair, or one value that passes, at a time
template <typename E>
__global__ void __launch_bounds__(kThreads) rope_any_kernel(const RopeCall c) {
    extern __shared__ float smem[];
    const int token = blockIdx.x;
    const int half = c.rope.rotary / 2;
    float *cs = smem, *sn = smem + half;
    const int pos = __ldg(c.positions + token);
    for (int j = threadIdx.x; j < half; j += kThreads) {
        const float2 x = turn_cos_sin(turn_step(__ldg(c.rope.inv_freq + j)), pos, c.rope.amplitude, c.rope.sign);
        cs[j] = x.x;
        sn[j] = x.y;
    }
    __syncthreads();
    const E* x = static_cast<const E*>(c.x.p) + token * c.x.token;
    E* y = static_cast<E*>(c.y.p) + token * c.y.token;
    const int per_head = half + (c.dim - c.rope.rotary);  // pairs, then values that pass
    for (int i = threadIdx.x; i < c.heads * per_head; i += kThreads) {
        const int h = i / per_head, j = i - h * per_head;
        const E* xh = x + h * c.x.head;
        E* yh = y + h * c.y.head;
        if (j < half) {
            const int ia = c.rope.layout == kRopeHalf ? j : 2 * j;
            const int ib = c.rope.layout == kRopeHalf ? j + half : 2 * j + 1;
            const float a = to_float(xh[ia]), b = to_float(xh[ib]);
            yh[ia] = from_float<E>(a * cs[j] - b * sn[j]);
            yh[ib] = from_float<E>(b * cs[j] + a * sn[j]);
        } else {
            yh[half + j] = xh[half + j];
        }
    }
}

// ---- rows on 16-byte boundaries, rotary / 2 (half layout) or rotary (interleaved) a multiple of 8
//
// An item is eight values of one head of one token, in the half layout with their eight partners. A
// thread keeps its place in the head (so what it does, and with which pairs, is settled once) and
// steps through the (token, head) rows of the CTA, four rows' loads at a time.
constexpr int kAtOnce = 4;

template <typename E, bool kHalf>
__global__ void __launch_bounds__(kThreads, 4) rope_kernel(const RopeCall c, int tokens_a_cta, int per_head, int rows_at_once) {
    extern __shared__ float smem[];
    __shared__ int32_t where[kMaxTokens];
    const int half = c.rope.rotary / 2;
    const int token0 = blockIdx.x * tokens_a_cta, n = min(tokens_a_cta, c.tokens - token0);
    float *cs = smem, *sn = smem + tokens_a_cta * half;
    const int v = threadIdx.x % per_head;
    const int turned = kHalf ? half / 8 : c.rope.rotary / 8;  // items of a head that turn
    const bool turns = v < turned;
    const int d = turns ? 8 * v : c.rope.rotary + 8 * (v - turned);
    int tok = 0, h = threadIdx.x / per_head;  // this thread's next row
    if (h >= rows_at_once) tok = n;           // beyond the whole rows of threads
    auto settle = [&] {
        while (h >= c.heads && tok < n) {
            h -= c.heads;
            ++tok;
        }
    };
    settle();
    uint4 a[kAtOnce], b[kAtOnce];
    int at[kAtOnce];
    E* to[kAtOnce];
    auto load = [&] {
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            at[i] = tok < n ? tok : -1;
            if (tok < n) {
                const E* x = static_cast<const E*>(c.x.p) + static_cast<int64_t>(token0 + tok) * c.x.token + h * c.x.head + d;
                to[i] = static_cast<E*>(c.y.p) + static_cast<int64_t>(token0 + tok) * c.y.token + h * c.y.head + d;
                a[i] = *reinterpret_cast<const uint4*>(x);
                if (kHalf && turns) b[i] = *reinterpret_cast<const uint4*>(x + half);
                h += rows_at_once;
                settle();
            }
        }
    };
    load();
    if (threadIdx.x < n) where[threadIdx.x] = __ldg(c.positions + token0 + threadIdx.x);
    __syncthreads();
    for (int i = threadIdx.x; i < n * half; i += kThreads) {
        const int slot = i / half, j = i - slot * half;
        const float2 x = turn_cos_sin(turn_step(__ldg(c.rope.inv_freq + j)), where[slot], c.rope.amplitude, c.rope.sign);
        cs[i] = x.x;
        sn[i] = x.y;
    }
    __syncthreads();
    constexpr int kPairs = kHalf ? 8 : 4;
    while (at[0] >= 0) {
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            if (at[i] < 0) continue;
            if (turns) {
                float cv[kPairs], sv[kPairs];
                const int j = at[i] * half + (kHalf ? d : d / 2);
#pragma unroll
                for (int e = 0; e < kPairs; e += 4) {
                    *reinterpret_cast<float4*>(cv + e) = *reinterpret_cast<const float4*>(cs + j + e);
                    *reinterpret_cast<float4*>(sv + e) = *reinterpret_cast<const float4*>(sn + j + e);
                }
                E* p = reinterpret_cast<E*>(&a[i]);
                E* q = reinterpret_cast<E*>(&b[i]);
#pragma unroll
                for (int e = 0; e < kPairs; ++e) {
                    E& first = kHalf ? p[e] : p[2 * e];
                    E& second = kHalf ? q[e] : p[2 * e + 1];
                    const float u = to_float(first), w = to_float(second);
                    first = from_float<E>(u * cv[e] - w * sv[e]);
                    second = from_float<E>(w * cv[e] + u * sv[e]);
                }
            }
            *reinterpret_cast<uint4*>(to[i]) = a[i];
            if (kHalf && turns) *reinterpret_cast<uint4*>(to[i] + half) = b[i];
        }
        load();
    }
}

template <typename E>
cudaError_t launch(const RopeCall& c, int sm_count, cudaStream_t stream) {
    const int half = c.rope.rotary / 2;
    auto wide = [](const Strided& s) {
        return reinterpret_cast<uintptr_t>(s.p) % 16 == 0 && s.token % 8 == 0 && s.head % 8 == 0;
    };
    const bool split = c.rope.layout == kRopeHalf;
    const bool whole = split ? half % 8 == 0 : c.rope.rotary % 8 == 0;
    const int per_head = (split ? half : c.rope.rotary) / 8 + (c.dim - c.rope.rotary) / 8;
    if (wide(c.x) && wide(c.y) && c.dim % 8 == 0 && whole) {
        const int rows_at_once = kThreads / per_head;  // dim is at most 1024: per_head at most 128
        // four rows a thread where there are tokens enough for eight CTAs an SM, and no more tokens than
        // keep cos and sin of all of them in 32 KB
        int tokens = kAtOnce * rows_at_once / c.heads;
        const int many = c.tokens / (8 * sm_count), fit = half > 0 ? 4096 / half : kMaxTokens;
        tokens = tokens < many ? tokens : many;
        tokens = tokens < fit ? tokens : fit;
        tokens = tokens < 1 ? 1 : tokens > kMaxTokens ? kMaxTokens : tokens;
        const int smem = tokens * half * 2 * static_cast<int>(sizeof(float));
        const int grid = (c.tokens + tokens - 1) / tokens;
        if (split) rope_kernel<E, true><<<grid, kThreads, smem, stream>>>(c, tokens, per_head, rows_at_once);
        else rope_kernel<E, false><<<grid, kThreads, smem, stream>>>(c, tokens, per_head, rows_at_once);
    } else {
        rope_any_kernel<E><<<c.tokens, kThreads, c.rope.rotary * static_cast<int>(sizeof(float)), stream>>>(c);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeCall& c, int sm_count, cudaStream_t stream) {
    return c.dtype == kFp16 ? launch<__half>(c, sm_count, stream) : launch<__nv_bfloat16>(c, sm_count, stream);
}

}  // namespace tg
