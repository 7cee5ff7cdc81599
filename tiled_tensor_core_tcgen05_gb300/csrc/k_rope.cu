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
// An item is eight values of one head of one token, in the half layout with their eight partners.
template <typename E>
struct Item {
    const E* x;
    E* y;
    int d;       // first value
    int kind;    // 0 none, 1 passes, 2 rotated with partners at d + half, 3 rotated in itself
    uint4 a, b;
};

template <typename E>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeCall c, int tokens_a_cta, int per_head) {
    extern __shared__ float smem[];
    __shared__ int32_t where[kMaxTokens];
    const int half = c.rope.rotary / 2;
    const int token0 = blockIdx.x * tokens_a_cta, n = min(tokens_a_cta, c.tokens - token0);
    float *cs = smem, *sn = smem + tokens_a_cta * half;
    const int items = n * c.heads * per_head;
    const int rotated = c.rope.layout == kRopeHalf ? half / 8 : c.rope.rotary / 8;  // items of a head that turn
    auto load = [&](int i, Item<E>& t, int& slot) {
        t.kind = 0;
        if (i >= items) return;
        const int row = i / per_head, v = i - row * per_head;
        slot = row / c.heads;
        const int h = row - slot * c.heads;
        t.x = static_cast<const E*>(c.x.p) + (token0 + slot) * c.x.token + h * c.x.head;
        t.y = static_cast<E*>(c.y.p) + (token0 + slot) * c.y.token + h * c.y.head;
        if (v < rotated) {
            t.kind = c.rope.layout == kRopeHalf ? 2 : 3;
            t.d = 8 * v;
        } else {
            t.kind = 1;
            t.d = c.rope.rotary + 8 * (v - rotated);
        }
        t.a = *reinterpret_cast<const uint4*>(t.x + t.d);
        if (t.kind == 2) t.b = *reinterpret_cast<const uint4*>(t.x + t.d + half);
    };
    auto finish = [&](Item<E>& t, int slot) {
        if (t.kind == 0) return;
        if (t.kind > 1) {
            const float *cj = cs + slot * half, *sj = sn + slot * half;
            E* a = reinterpret_cast<E*>(&t.a);
            if (t.kind == 2) {
                E* b = reinterpret_cast<E*>(&t.b);
                float cv[8], sv[8];
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    *reinterpret_cast<float4*>(cv + i) = *reinterpret_cast<const float4*>(cj + t.d + i);
                    *reinterpret_cast<float4*>(sv + i) = *reinterpret_cast<const float4*>(sj + t.d + i);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float u = to_float(a[i]), w = to_float(b[i]);
                    a[i] = from_float<E>(u * cv[i] - w * sv[i]);
                    b[i] = from_float<E>(w * cv[i] + u * sv[i]);
                }
            } else {
                float cv[4], sv[4];
                *reinterpret_cast<float4*>(cv) = *reinterpret_cast<const float4*>(cj + t.d / 2);
                *reinterpret_cast<float4*>(sv) = *reinterpret_cast<const float4*>(sj + t.d / 2);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float u = to_float(a[2 * i]), w = to_float(a[2 * i + 1]);
                    a[2 * i] = from_float<E>(u * cv[i] - w * sv[i]);
                    a[2 * i + 1] = from_float<E>(w * cv[i] + u * sv[i]);
                }
            }
        }
        *reinterpret_cast<uint4*>(t.y + t.d) = t.a;
        if (t.kind == 2) *reinterpret_cast<uint4*>(t.y + t.d + half) = t.b;
    };
    Item<E> t0, t1;
    int s0 = 0, s1 = 0;
    load(threadIdx.x, t0, s0);
    load(threadIdx.x + kThreads, t1, s1);
    if (threadIdx.x < n) where[threadIdx.x] = __ldg(c.positions + token0 + threadIdx.x);
    __syncthreads();
    for (int i = threadIdx.x; i < n * half; i += kThreads) {
        const int slot = i / half, j = i - slot * half;
        const float2 x = turn_cos_sin(turn_step(__ldg(c.rope.inv_freq + j)), where[slot], c.rope.amplitude, c.rope.sign);
        cs[i] = x.x;
        sn[i] = x.y;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < items; i += 2 * kThreads) {
        finish(t0, s0);
        finish(t1, s1);
        load(i + 2 * kThreads, t0, s0);
        load(i + 3 * kThreads, t1, s1);
    }
}

template <typename E>
cudaError_t launch(const RopeCall& c, cudaStream_t stream) {
    const int half = c.rope.rotary / 2;
    auto wide = [](const Strided& s) {
        return reinterpret_cast<uintptr_t>(s.p) % 16 == 0 && s.token % 8 == 0 && s.head % 8 == 0;
    };
    const bool whole = c.rope.layout == kRopeHalf ? half % 8 == 0 : c.rope.rotary % 8 == 0;
    if (wide(c.x) && wide(c.y) && c.dim % 8 == 0 && whole) {
        const int per_head = (c.rope.layout == kRopeHalf ? half : c.rope.rotary) / 8 + (c.dim - c.rope.rotary) / 8;
        // two items a thread in a CTA, or a few more where heads are few
        int tokens = 2 * kThreads / (c.heads * per_head);
        tokens = tokens < 1 ? 1 : tokens > kMaxTokens ? kMaxTokens : tokens;
        const int smem = tokens * half * 2 * static_cast<int>(sizeof(float));
        rope_kernel<E><<<(c.tokens + tokens - 1) / tokens, kThreads, smem, stream>>>(c, tokens, per_head);
    } else {
        rope_any_kernel<E><<<c.tokens, kThreads, c.rope.rotary * static_cast<int>(sizeof(float)), stream>>>(c);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeCall& c, int, cudaStream_t stream) {
    return c.dtype == kFp16 ? launch<__half>(c, stream) : launch<__nv_bfloat16>(c, stream);
}

}  // namespace tg
