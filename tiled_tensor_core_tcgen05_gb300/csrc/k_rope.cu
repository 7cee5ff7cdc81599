// Rotary positions: pairs of values of each head turned by position times a
// frequency of the pair,
//
//     y_a = amplitude (x_a cos t - x_b sin t),  y_b = amplitude (x_b cos t + x_a sin t),
//     t = position * inv_freq[pair],
//
// for the first `rotary` values of a head; the rest pass through. The gradient
// is the transposed map, the same kernel with the sign of sin turned round.
// Angles are computed as 64-bit fractions of a turn and off by at most 1e-7
// radians (tg_kv.cuh), products and sums are fp32, and each value is rounded
// once to its 16-bit type.
//
// Memory bounds it: every value is read and written once. A CTA takes a few
// tokens, so that cos and sin, about forty instructions a pair, are computed
// once for all heads of a token (in shared memory, two arrays so that a
// thread's eight of each are two 16-byte reads), and each thread's loads are
// under way before it computes them. Measured: 8192 tokens of 40 heads of 128,
// 28.3 us, 5.9 TB/s or 0.87 of the copy rate; 4099 of 32 heads, 64 of 128
// values turned, interleaved, 14.2 us, 0.70; one token 2.3 us. A CTA a token
// (cos and sin in waits of their own): 36 and 18.5 us.
#include "tg_rope.cuh"

namespace tg {
namespace {

constexpr int kThreads = 256;

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

// ---- whole 16-byte pieces
template <typename E, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const RopeRows c, const int32_t* positions) {
    extern __shared__ float smem[];
    rope_rows<E, kHalf, false>(c, smem, [&](int32_t* where, int token0, int n) {
        if (threadIdx.x < n) where[threadIdx.x] = __ldg(positions + token0 + threadIdx.x);
    });
}

template <typename E>
cudaError_t launch(const RopeCall& c, int sm_count, cudaStream_t stream) {
    if (rope_whole(c.x, c.y, c.dim, c.rope)) {
        const RopeRows r = rope_rows_of(c.x, c.y, c.tokens, c.heads, c.dim, c.rope, sm_count);
        auto* kernel = c.rope.layout == kRopeHalf ? rope_kernel<E, true> : rope_kernel<E, false>;
        kernel<<<rope_grid(r), kRopeThreads, rope_smem(r), stream>>>(r, c.positions);
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
