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
#include "tg_kv.cuh"

namespace tg {
namespace {

constexpr int kThreads = 256;

// One CTA per token: cos and sin of its pairs once, in shared memory, then every head.
template <typename E>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeCall c) {
    extern __shared__ float2 cs[];
    const int token = blockIdx.x;
    const int half = c.rope.rotary / 2;
    const int pos = __ldg(c.positions + token);
    for (int j = threadIdx.x; j < half; j += kThreads)
        cs[j] = turn_cos_sin(turn_step(__ldg(c.rope.inv_freq + j)), pos, c.rope.amplitude, c.rope.sign);
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
            yh[ia] = from_float<E>(a * cs[j].x - b * cs[j].y);
            yh[ib] = from_float<E>(b * cs[j].x + a * cs[j].y);
        } else {
            yh[half + j] = xh[half + j];
        }
    }
}

}  // namespace

cudaError_t launch_rope(const RopeCall& c, int, cudaStream_t stream) {
    const int smem = c.rope.rotary / 2 * static_cast<int>(sizeof(float2));
    if (c.dtype == kFp16)
        rope_kernel<__half><<<c.tokens, kThreads, smem, stream>>>(c);
    else
        rope_kernel<__nv_bfloat16><<<c.tokens, kThreads, smem, stream>>>(c);
    return cudaGetLastError();
}

}  // namespace tg
