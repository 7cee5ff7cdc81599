// Device helpers of the 8-bit cache kernels: 16-bit element types, rotation
// angles, the two 8-bit code formats, and the lookup of a batch's sequences
// and pages with its range checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tg_kv_internal.h"
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
// position: the angle's error is the position times 2^-63 turns (the step's
// own; the frequency carries 2^-53 of its value from the caller), where
// position * frequency in 32 bits would be off by radians. In integers, since
// the 64-bit floating point unit is narrow.
__device__ __forceinline__ uint64_t turn_step(double radians_per_position) {
    const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(radians_per_position));
    const int e = static_cast<int>(bits >> 52 & 0x7FF) - 1023;
    const uint64_t m = (bits << 11) | 0x8000000000000000ull;  // value = m 2^(e - 63)
    const uint64_t kInv2Pi = 0xA2F9836E4E44152Aull;           // 2^66 / (2 pi)
    const uint64_t hi = __umul64hi(m, kInv2Pi), lo = m * kInv2Pi;
    // turns 2^64 = (hi 2^64 + lo) 2^(e - 65)
    uint64_t step;
    if (e <= 0) {
        const int down = 1 - e;  // at least 1
        step = down <= 64 ? (down == 64 ? 0 : hi >> down) + (hi >> (down - 1) & 1) : 0;
    } else {
        const int up = e - 1;
        step = up == 0 ? hi : up < 64 ? hi << up | lo >> (64 - up) : up < 128 ? lo << (up - 64) : 0;
    }
    return bits >> 63 ? 0 - step : step;
}

// amplitude * (cos, sin) of the angle at `position`, sin negated for the backward rotation.
__device__ __forceinline__ float2 turn_cos_sin(uint64_t step, int32_t position, float amplitude, float sign) {
    const uint64_t frac = step * static_cast<uint64_t>(static_cast<int64_t>(position));
    // the top 32 bits, signed: [-1/2, 1/2) turn, to half turns for sincospi, in 24 bits: off by 2^-25 and
    // the 2^-31 that the lower bits are worth, 1e-7 radians in all
    const float half_turns = static_cast<float>(static_cast<int32_t>(frac >> 32)) * 4.656612873077393e-10f;  // 2^-31
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c * amplitude, s * (amplitude * sign));
}

// ---- values of a row, rotated or not

// kN (4 or 8) values of a row from d on, in one load where `vec` says that rows begin on the boundary for it.
template <typename E, int kN>
__device__ __forceinline__ void load_values(const E* row, int d, bool vec, float (&x)[kN]) {
    if (vec) {
        uint32_t w[kN / 2];
        if constexpr (kN == 8) {
            const uint4 u = *reinterpret_cast<const uint4*>(row + d);
            w[0] = u.x;
            w[1] = u.y;
            w[2] = u.z;
            w[3] = u.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(row + d);
            w[0] = u.x;
            w[1] = u.y;
        }
        const E* e = reinterpret_cast<const E*>(w);
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] = to_float(e[i]);
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] = to_float(row[d + i]);
    }
}

template <typename E, int kN>
__device__ __forceinline__ void store_values(E* row, int d, bool vec, const float (&x)[kN]) {
    if (vec) {
        uint32_t w[kN / 2];
        E* e = reinterpret_cast<E*>(w);
#pragma unroll
        for (int i = 0; i < kN; ++i) e[i] = from_float<E>(x[i]);
        if constexpr (kN == 8) *reinterpret_cast<uint4*>(row + d) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2*>(row + d) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) row[d + i] = from_float<E>(x[i]);
    }
}

// What rotates d .. d + kN - 1 of a row besides themselves: in the half layout their partners (zeros elsewhere).
template <typename E, int kN>
__device__ __forceinline__ void load_partners(const E* row, int d, bool vec, const RopeArgs& r, float (&o)[kN]) {
    const int half = r.rotary / 2;
    if (r.layout == kRopeHalf && d < r.rotary) {
        if (half % kN == 0) {
            load_values<E, kN>(row, d < half ? d + half : d - half, vec, o);
            return;
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int at = d + i;
            o[i] = at < r.rotary ? to_float(row[at < half ? at + half : at - half]) : 0.0f;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) o[i] = 0.0f;
}

// Rotates x (values d .. d + kN - 1) given their partners: cs[j], sn[j] are cos and sin of pair j.
template <int kN>
__device__ __forceinline__ void rotate_values(float (&x)[kN], const float (&o)[kN], int d, const float* cs, const float* sn,
                                              const RopeArgs& r) {
    const int half = r.rotary / 2;
    if (d >= r.rotary) return;
    if (r.layout == kRopeHalf) {
        if (half % kN == 0) {
            const bool first = d < half;
            const int j = first ? d : d - half;
#pragma unroll
            for (int i = 0; i < kN; i += 4) {
                const float4 c = *reinterpret_cast<const float4*>(cs + j + i), s = *reinterpret_cast<const float4*>(sn + j + i);
                const float c4[4] = {c.x, c.y, c.z, c.w}, s4[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) x[i + k] = x[i + k] * c4[k] + o[i + k] * (first ? -s4[k] : s4[k]);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int at = d + i;
            if (at < half) x[i] = x[i] * cs[at] - o[i] * sn[at];
            else if (at < r.rotary) x[i] = x[i] * cs[at - half] + o[i] * sn[at - half];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kN; i += 2) {
        if (d + i < r.rotary) {
            const float c = cs[(d + i) / 2], s = sn[(d + i) / 2], a = x[i], b = x[i + 1];
            x[i] = a * c - b * s;
            x[i + 1] = b * c + a * s;
        }
    }
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

// Four codes, the first in the low byte: x (in units of the scale) to the nearest code, ties to even; beyond the
// largest code it saturates. A NaN stays one in e4m3 and becomes 0 in int8.
template <int kFmt>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    if constexpr (kFmt == kKvE4M3) {
        uint32_t w;
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
            "mov.b32 %0, {lo, hi};\n\t}"
            : "=r"(w)
            : "f"(a), "f"(b), "f"(c), "f"(d));
        return w;
    } else {
        // to nearest even, a NaN to 0; |x| is at most the largest code and a rounding error more
        const float x[4] = {a, b, c, d};
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            int v;
            asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(v) : "f"(x[i]));
            w |= (static_cast<uint32_t>(max(v, -127)) & 0xFFu) << (8 * i);
        }
        return w;
    }
}

// encode4 for values known to be finite and at most the largest code (and a rounding error): int8 codes
// are the low bytes of x + 1.5 * 2^23, whose steps are 1 and whose rounding is to nearest even.
template <int kFmt>
__device__ __forceinline__ uint32_t encode4_in_range(float a, float b, float c, float d) {
    if constexpr (kFmt == kKvE4M3) {
        return encode4<kFmt>(a, b, c, d);
    } else {
        const float k = 12582912.0f;
        const uint32_t lo = __byte_perm(__float_as_uint(__fadd_rn(a, k)), __float_as_uint(__fadd_rn(b, k)), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(__fadd_rn(c, k)), __float_as_uint(__fadd_rn(d, k)), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    }
}

template <int kFmt>
__device__ __forceinline__ void decode4(uint32_t w, float (&x)[4]) {
    if constexpr (kFmt == kKvE4M3) {
        uint32_t lo, hi;
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        x[0] = a.x;
        x[1] = a.y;
        x[2] = b.x;
        x[3] = b.y;
    } else {
        // code + 128 as the low byte of 2^23 + (code + 128), whose steps are 1: no integer conversion
        const uint32_t u = w ^ 0x80808080u;
        x[0] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440)) - 8388736.0f;
        x[1] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441)) - 8388736.0f;
        x[2] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7442)) - 8388736.0f;
        x[3] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7443)) - 8388736.0f;
    }
}

// ---- sequences and pages

// Records that a length, an offset or a page number of the call is out of range.
__device__ __forceinline__ void report_range(const Watchdog& wd) { atomicCAS(wd.status, 0, kSiteRange); }

struct SeqSpan {
    int first;  // first packed row of the sequence's new tokens
    int count;  // how many
    bool bad;   // out of range
};

// Sequence i's rows of the packed tensors: cu[i] .. cu[i + 1], or row i where cu is NULL.
// A span outside [0, total] or longer than max_new is reported and comes back empty.
__device__ __forceinline__ SeqSpan seq_span(const KvBatch& b, int i, const Watchdog& wd) {
    SeqSpan s{i, 1, false};
    if (b.cu != nullptr) {
        const int lo = __ldg(b.cu + i), hi = __ldg(b.cu + i + 1);
        s.first = lo;
        s.count = hi - lo;
        if (lo < 0 || hi < lo || hi > b.total || s.count > b.max_new) {
            report_range(wd);
            s.first = 0;
            s.count = 0;
            s.bad = true;
        }
    }
    return s;
}

// An offset as a row of the packed tensors, whatever it is.
__device__ __forceinline__ int packed_row(const KvBatch& b, int i) { return min(max(__ldg(b.cu + i), 0), b.total); }

// Rows that no sequence has: 0 .. before - 1 and after .. total - 1 (a batch padded to a fixed size, say).
struct Uncovered {
    int before, after;
};
__device__ __forceinline__ Uncovered uncovered(const KvBatch& b) {
    return b.cu == nullptr ? Uncovered{0, b.total} : Uncovered{packed_row(b, 0), packed_row(b, b.batch)};
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
