#pragma once

#include "tg_kv.cuh"

namespace tg {
namespace {

// Rotary positions over whole 16-byte pieces: rows on 16-byte boundaries, rotary / 2 (half layout) or rotary
// (interleaved) a multiple of 8. Used for packed rows with given positions (k_rope.cu) and for the queries beside
// a prompt's keys, whose positions follow from the sequences (k_kv.cu).
//
// An item is eight values of one head of one token, in the half layout with their eight partners. A
// thread keeps its place in the head (so what it does, and with which pairs, is settled once) and
// steps through the (token, head) rows of the CTA, four rows' loads at a time.
constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 16;  // most tokens a CTA
constexpr int kAtOnce = 4;

// `fill(where, token0, n)` gives each token's position; with kSkips a token at a negative one has none and is copied.
struct RopeRows {
    Strided x, y;
    int tokens, heads, dim;
    RopeArgs rope;
    int tokens_a_cta, per_head, rows_at_once;  // items a head, (token, head) rows that the threads take at once
};

template <typename E, bool kHalf, bool kSkips, typename Fill>
__device__ __forceinline__ void rope_rows(const RopeRows& c, float* smem, Fill fill) {
    __shared__ int32_t where[kRopeTokens];
    const int half = c.rope.rotary / 2, per_head = c.per_head, rows_at_once = c.rows_at_once;
    const int token0 = blockIdx.x * c.tokens_a_cta, n = min(c.tokens_a_cta, c.tokens - token0);
    float *cs = smem, *sn = smem + c.tokens_a_cta * half;
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
    fill(where, token0, n);
    __syncthreads();
    for (int i = threadIdx.x; i < n * half; i += kRopeThreads) {
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
            if (turns && !(kSkips && where[at[i]] < 0)) {
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

// Whether rope_rows can take a call.
inline bool rope_whole(const Strided& x, const Strided& y, int dim, const RopeArgs& rope) {
    auto wide = [](const Strided& s) {
        return reinterpret_cast<uintptr_t>(s.p) % 16 == 0 && s.token % 8 == 0 && s.head % 8 == 0;
    };
    return wide(x) && wide(y) && dim % 8 == 0 && (rope.layout == kRopeHalf ? rope.rotary / 2 % 8 == 0 : rope.rotary % 8 == 0);
}

// Four rows a thread where there are tokens enough for eight CTAs an SM, and no more tokens a CTA than keep cos
// and sin of all of them in 32 KB.
inline RopeRows rope_rows_of(const Strided& x, const Strided& y, int tokens, int heads, int dim, const RopeArgs& rope, int sm_count) {
    RopeRows r{x, y, tokens, heads, dim, rope, 0, 0, 0};
    const int half = rope.rotary / 2;
    r.per_head = (rope.layout == kRopeHalf ? half : rope.rotary) / 8 + (dim - rope.rotary) / 8;
    r.rows_at_once = kRopeThreads / r.per_head;  // dim is at most 1024: per_head at most 128
    int take = kAtOnce * r.rows_at_once / heads;
    const int many = tokens / (8 * sm_count), fit = half > 0 ? 4096 / half : kRopeTokens;
    take = take < many ? take : many;
    take = take < fit ? take : fit;
    r.tokens_a_cta = take < 1 ? 1 : take > kRopeTokens ? kRopeTokens : take;
    return r;
}

inline int rope_grid(const RopeRows& r) { return (r.tokens + r.tokens_a_cta - 1) / r.tokens_a_cta; }
inline int rope_smem(const RopeRows& r) { return r.tokens_a_cta * r.rope.rotary * static_cast<int>(sizeof(float)); }

}  // namespace
}  // namespace tg
