// Device helpers of the 8-bit cache kernels: 16-bit element types, rotation
// angles, the two 8-bit code formats, and the lookup of a batch's sequences
// and pages with its range checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tg_internal.h"
#include "tg_ptx.cuh"

namespace tg {

// ---- 16-bit elements

template <typename E>
__device__ __forceinline__ float to_float(E x);
template <>
__device__ __forceinline__ float to_float<__half>(__half x) {
    return __half2float(x);
}
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) {
    return __bfloat162float(x);
}
template <typename E>
__device__ __forceinline__ E from_float(float x);
template <>
__device__ __forceinline__ __half from_float<__half>(float x) {
    return __float2half_rn(x);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

// ---- rotation angles

// Turns per position as a 64-bit fraction of a turn. position * step modulo
// 2^64 is then the exact fraction of a turn after that many steps, whatever the
// position: the angle's error is the position times 2^-65 turns (the rounding
// of the step; the frequency itself carries 2^-53 of its own value from the
// caller), where position * frequency in 32 bits would be off by radians.
__device__ __forceinline__ uint64_t turn_step(double radians_per_position) {
    double turns = radians_per_position * 0.15915494309189533577;  // 1 / (2 pi)
    turns -= floor(turns);
    return static_cast<uint64_t>(__double2ull_rn(turns * 18446744073709551616.0));
}

// amplitude * (cos, sin) of the angle at `position`, sin negated for the backward rotation.
__device__ __forceinline__ float2 turn_cos_sin(uint64_t step, int32_t position, float amplitude, float sign) {
    const uint64_t frac = step * static_cast<uint64_t>(static_cast<int64_t>(position));
    // the top 32 bits, signed: [-1/2, 1/2) turn, to half turns for sincospi
    const float half_turns = static_cast<float>(static_cast<int32_t>(frac >> 32)) * 4.656612873077393e-10f;  // 2^-31
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c * amplitude, s * (amplitude * sign));
}

// ---- 8-bit codes

constexpr float kScaleFloor = 8.673617379884035e-19f;  // 2^-60

// 1 / the largest code, rounded to fp32
template <int kFmt>
__device__ __forceinline__ constexpr float code_max_inverse() {
    return kFmt == kKvE4M3 ? 1.0f / 448.0f : 1.0f / 127.0f;
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// x (in units of the scale) to the nearest code, ties to even; beyond the
// largest code it saturates. A NaN stays one in e4m3 and becomes 0 in int8.
template <int kFmt>
__device__ __forceinline__ uint8_t encode(float x) {
    if constexpr (kFmt == kKvE4M3) {
        uint16_t two;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.0f), "f"(x));
        return static_cast<uint8_t>(two);
    } else {
        const float c = fminf(fmaxf(rintf(x), -127.0f), 127.0f);
        return static_cast<uint8_t>(x == x ? static_cast<int>(c) : 0);
    }
}

template <int kFmt>
__device__ __forceinline__ float decode(uint8_t code) {
    if constexpr (kFmt == kKvE4M3) {
        uint32_t h2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(code)));
        return __half2float(__ushort_as_half(static_cast<unsigned short>(h2 & 0xFFFFu)));
    } else {
        return static_cast<float>(static_cast<int8_t>(code));
    }
}

// ---- sequences and pages

// Records that a length, an offset or a page number of the call is out of range.
__device__ __forceinline__ void report_range(const Watchdog& wd) { atomicCAS(wd.status, 0, kSiteRange); }

struct SeqSpan {
    int first;  // first packed row of the sequence's new tokens
    int count;  // how many
};

// Sequence i's rows of the packed tensors: cu[i] .. cu[i + 1], or row i where cu is NULL.
// A span outside [0, total] or longer than max_new is reported and comes back empty.
__device__ __forceinline__ SeqSpan seq_span(const KvBatch& b, int i, const Watchdog& wd) {
    SeqSpan s{i, 1};
    if (b.cu != nullptr) {
        const int lo = __ldg(b.cu + i), hi = __ldg(b.cu + i + 1);
        s.first = lo;
        s.count = hi - lo;
        if (lo < 0 || hi < lo || hi > b.total || s.count > b.max_new) {
            report_range(wd);
            s.first = 0;
            s.count = 0;
        }
    }
    return s;
}

// Page `slot` of sequence i, or -1 (reported) where the table holds no page of the cache.
__device__ __forceinline__ int seq_page(const KvBatch& b, const KvCacheArgs& c, int i, int slot, const Watchdog& wd) {
    const int p = __ldg(b.table + static_cast<int64_t>(i) * b.table_width + slot);
    if (p < 0 || p >= c.pages) {
        report_range(wd);
        return -1;
    }
    return p;
}

}  // namespace tg
