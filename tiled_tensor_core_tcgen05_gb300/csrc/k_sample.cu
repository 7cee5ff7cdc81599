// Drawing a token from each row of logits: temperature, the top_k largest, a
// least weight min_p, the top_p of the mass, and one given number u a row.
//
//     w_i = exp((x_i - max) / T) = 2^t_i,  token = first kept i with sum_{j <= i, kept} w_j > u sum_{kept} w_j
//
// The answer is a whole number, and a border (of the mass, or of u) lies between
// two tokens of a vocabulary of 10^5, whose shares are about 10^-5 of the sum or
// less: sums in 32 bits, off by 10^-7 and by how the row was split, would give
// another token in one row of some hundreds. So weights are integers, of 2^-42 of the
// row's largest, from a 2^t good to 2^-40 (weigh), and sums of them are exact
// in 64 bits: the same whatever the order, the split and the rest of the batch.
//
// Order: a token's rank is that of its 64-bit `place`: the logit's bits as an
// ordered 32-bit integer, then the index inverted, so equal logits rank by index
// and what a row keeps is every place >= one cut.
//
// A cluster of CTAs takes a row, each CTA a stretch of it, which the first pass leaves in
// shared memory: the logits are read from HBM once. The passes, of which a row makes
// those its settings ask for:
//   1  the largest logit (a greedy row ends here);
//   2  a count in each of kBins bins of t, 1/32 wide, and where top_p needs it the exact
//      mass: the bin with the k-th, and a guess at the bin in which the mass reaches top_p;
//   3  the tokens down to that bin, brought together where they are at most kList: the first
//      CTA sorts them, cuts, and draws.
// Otherwise:
//   4  the exact mass above, and in each bin near the guess; the border's bin, its
//      tokens brought together and sorted: the cut;
//   5  the mass of what is kept, group by group of 32 lanes' pieces; the group,
//      lane and token in which u of it is passed.
#include "tg_device.cuh"
#include "tg_kv.cuh"

#include <climits>
#include <cstring>
#include <type_traits>

namespace tg {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;
constexpr int kUnit = 42;                    // weights are multiples of 2^-42
constexpr int kSteps = 256;                  // of the table of powers: 2^(j / 256)
constexpr int kBinSteps = 8;                 // of a bin
constexpr int kBins = (kUnit + 3) * kSteps / kBinSteps;
constexpr int kWindow = 16;                  // bins whose mass is taken exactly at a time
constexpr int kList = 2048;                  // tokens that are sorted at a time
constexpr int kSub = 1024;                   // parts of a bin that holds more
constexpr int kMostGroups = (1 << 18) / 128 / kMaxCtas + 2;  // of a CTA
constexpr float kNone = -INFINITY;
using u64 = unsigned long long;

// 2^(j / 256) as the sum of two floats, by repeated square roots and products in integers.
struct Powers {
    float2 v[kSteps];
};
constexpr uint64_t product_2_62(uint64_t a, uint64_t b) { return static_cast<uint64_t>((static_cast<unsigned __int128>(a) * b + (1ull << 61)) >> 62); }
constexpr uint64_t root_2_62(uint64_t a) {  // the largest r with r^2 <= a, in units of 2^-62
    uint64_t r = 0;
    for (int b = 63; b >= 0; --b) {
        const uint64_t x = r | 1ull << b;
        if (static_cast<unsigned __int128>(x) * x <= static_cast<unsigned __int128>(a) << 62) r = x;
    }
    return r;
}
constexpr Powers make_powers() {
    Powers p{};
    uint64_t step = 1ull << 63;  // 2
    for (int i = 1; i < kSteps; i *= 2) step = root_2_62(step);
    uint64_t x = 1ull << 62;
    for (int j = 0; j < kSteps; ++j) {
        const uint64_t hi = (x + (1ull << 38)) >> 39 << 39;  // 24 bits
        p.v[j].x = static_cast<float>(hi >> 39) / static_cast<float>(1 << 23);
        p.v[j].y = static_cast<float>(static_cast<int64_t>(x - hi)) / static_cast<float>(1ull << 62);
        x = product_2_62(x, step);
    }
    return p;
}
__device__ const Powers kPowers = make_powers();

// What a row's logits are weighed with.
struct Scale {
    float top;       // the largest logit
    float hi, lo;    // 2 * 256 log2(e) / T
    bool flat;       // the largest is infinite: what is kept weighs the same
};

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 minus(float2 a, float2 b) { return __ffma2_rn(b, both(-1.0f), a); }

// Weights of two logits as multiples of 2^-20 and 2^-42: w = hi + lo, each such that eight of them add up exactly in a float.
// bits: 256 t to the nearest integer, above 0x4B400000. The logits are at most c.top and not so far below it that 2^t is no ordinary
// float; t off by 2^-8 of 2^-40, and so the weight, before its rounding to 2^-42, by 2^-40 of itself: with the difference of halves of
// the logits (which stays finite) as d + e exactly and the factor as hi + lo, 256 t = p + q; n = round(p); 2^(n / 256) is a power of two
// times a table's entry th + tl; with f = p - n + q, at most 1/2 and a little, 2^(f / 256) = 1 + y + y^2 / 2 + y^3 / 6, y = f ln(2) / 256 <= 2^-9.5:
// y^4 / 24 is 2^-42.6. All pairs of operations, two logits an instruction.
__device__ __forceinline__ void weigh(float2 x, const Scale& c, const float2* powers, float2& hi, float2& lo, int& bits0, int& bits1) {
    constexpr double kLn = 0.693147180559945309417 / kSteps;
    constexpr float kLnHi = static_cast<float>(kLn), kLnLo = static_cast<float>(kLn - static_cast<double>(kLnHi));
    constexpr float kRound = 12582912.0f;                    // 1.5 * 2^23: a sum with it is a whole number
    constexpr float kHigh = 12.0f, kLow = 1.5f / 524288.0f;  // sums with them are multiples of 2^-20 and 2^-42
    const float2 a = __fmul2_rn(x, both(0.5f)), b = both(-0.5f * c.top);
    const float2 d = __fadd2_rn(a, b), bb = minus(d, a), e = __fadd2_rn(minus(a, minus(d, bb)), minus(b, bb));
    const float2 p = __fmul2_rn(d, both(c.hi));
    const float2 m = __fadd2_rn(p, both(kRound));
    bits0 = __float_as_int(m.x);
    bits1 = __float_as_int(m.y);
    const float2 t0 = powers[bits0 & (kSteps - 1)], t1 = powers[bits1 & (kSteps - 1)];
    const float2 th = make_float2(t0.x, t1.x), tl = make_float2(t0.y, t1.y);
    const float2 q = __ffma2_rn(d, both(c.lo), __ffma2_rn(e, both(c.hi), __ffma2_rn(d, both(c.hi), __fmul2_rn(p, both(-1.0f)))));
    const float2 f = minus(p, __fadd2_rn(m, both(-kRound)));
    // y as u + v, with its square and cube in v
    const float2 u = __fmul2_rn(f, both(kLnHi));
    float2 v = __ffma2_rn(f, both(kLnHi), __fmul2_rn(u, both(-1.0f)));
    v = __ffma2_rn(f, both(kLnLo), v);
    v = __ffma2_rn(q, both(kLnHi), v);
    v = __ffma2_rn(__fmul2_rn(u, u), __ffma2_rn(u, both(1.0f / 6.0f), both(0.5f)), v);
    // (th + tl) (1 + u + v) = s + r
    float2 s = __ffma2_rn(th, u, th);
    float2 r = __ffma2_rn(th, u, minus(th, s));
    r = __fadd2_rn(r, __ffma2_rn(th, v, __ffma2_rn(tl, u, tl)));
    const float2 by = make_float2(__int_as_float((bits0 >> 8 << 23) + 0x3F800000), __int_as_float((bits1 >> 8 << 23) + 0x3F800000));
    s = __fmul2_rn(s, by);
    r = __fmul2_rn(r, by);
    hi = __fadd2_rn(__fadd2_rn(s, both(kHigh)), both(-kHigh));
    lo = __fadd2_rn(__fadd2_rn(__fadd2_rn(minus(s, hi), r), both(kLow)), both(-kLow));
}

// Sums of at most eight hi and lo, in units of 2^-42.
__device__ __forceinline__ u64 units(float hi, float lo) {
    return static_cast<u64>((static_cast<int64_t>(__float2int_rn(hi * 1048576.0f)) << 22) + __float2int_rn(lo * 4398046511104.0f));
}

__device__ __forceinline__ u64 weight_of(float x, const Scale& c, const float2* powers) {
    if (c.flat) return 1ull << kUnit;
    float2 hi, lo;
    int n0, n1;
    weigh(make_float2(x, c.top), c, powers, hi, lo, n0, n1);
    return units(hi.x, lo.x);
}

// 256 t of a logit as weigh() has it, as a bin's number: falls as the logit does, so bins are in order.
__device__ __forceinline__ int bin_of_bits(int bits) { return min((0x4B400000 - bits) / kBinSteps, kBins - 1); }
__device__ __forceinline__ int bin_of(float x, const Scale& c) {
    const float d = __fadd_rn(0.5f * x, -0.5f * c.top);
    return c.flat ? 0 : bin_of_bits(__float_as_int(__fadd_rn(__fmul_rn(d, c.hi), 12582912.0f)));
}

// A logit's rank among all: larger ones higher, of equal ones the lower index (-0 and 0 are equal).
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ u64 place_of(float x, int i) { return static_cast<u64>(key_of(x)) << 32 | static_cast<uint32_t>(~i); }
__device__ __forceinline__ int index_of(u64 place) { return static_cast<int>(~static_cast<uint32_t>(place)); }
__device__ __forceinline__ float logit_of(u64 place) {
    const uint32_t k = static_cast<uint32_t>(place >> 32);
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// This CTA's stretch of a row: pieces of 16 bytes, kV logits each, on 16-byte boundaries of memory (the first and the last may reach beyond
// the row); 32 pieces are a group, which one warp takes, always the same.
template <typename E>
struct Row {
    static constexpr int kV = 16 / sizeof(E);
    const E* x;
    uint4* held;          // shared memory
    int vocab, shift;     // index of piece q's first logit: q * kV - shift
    int group0, groups;   // of this CTA
    __device__ Row(const E* row, uint4* smem, int n, uint32_t rank, uint32_t ctas) : x(row), held(smem), vocab(n) {
        shift = static_cast<int>(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(E));
        const int all = ((n + shift + kV - 1) / kV + 31) / 32, each = (all + ctas - 1) / ctas;
        group0 = min(all, static_cast<int>(rank) * each);
        groups = min(all, group0 + each) - group0;
    }
    __device__ int index(int group) const { return ((group0 + group) * 32 + (threadIdx.x & 31)) * kV - shift; }
    __device__ uint4 read(int group) const {
        const int i = index(group);
        uint4 u;
        if (i >= 0 && i + kV <= vocab) return __ldg(reinterpret_cast<const uint4*>(x + i));
        E v[kV];
#pragma unroll
        for (int e = 0; e < kV; ++e) {
            if (i + e >= 0 && i + e < vocab) v[e] = x[i + e];
            else if constexpr (std::is_same<E, float>::value) v[e] = kNone;
            else v[e] = from_float<E>(kNone);
        }
        memcpy(&u, v, 16);
        return u;
    }
    __device__ __forceinline__ static void open(const uint4& u, float (&v)[kV]) {
        const E* e = reinterpret_cast<const E*>(&u);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            if constexpr (std::is_same<E, float>::value) v[i] = e[i];
            else v[i] = to_float(e[i]);
        }
    }
    // The first pass: reads, keeps, f(index of the first, the kV logits).
    template <typename F>
    __device__ __forceinline__ void load(F f) {
        constexpr int kAhead = 4;
        for (int g = threadIdx.x / 32; g < groups; g += kWarps * kAhead) {
            uint4 u[kAhead];
#pragma unroll
            for (int a = 0; a < kAhead; ++a)
                if (g + a * kWarps < groups) u[a] = read(g + a * kWarps);
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                if (g + a * kWarps >= groups) break;
                held[(g + a * kWarps) * 32 + (threadIdx.x & 31)] = u[a];
                float v[kV];
                open(u[a], v);
                f(index(g + a * kWarps), v);
            }
        }
    }
    // Further passes, over groups in which some logit is at least `least`: f(group, index of the first, the kV logits), whole warps.
    template <typename F>
    __device__ __forceinline__ void each(float least, F f) const {
        for (int g = threadIdx.x / 32; g < groups; g += kWarps) {
            const uint4 u = held[g * 32 + (threadIdx.x & 31)];
            float v[kV];
            open(u, v);
            float most = v[0];
#pragma unroll
            for (int e = 1; e < kV; ++e) most = fmaxf(most, v[e]);
            if (!__any_sync(0xFFFFFFFFu, !(most < least))) continue;
            f(g, index(g), v);
        }
    }
};

struct Shared {
    float2 powers[kSteps];
    u64 list[kList];           // of the first CTA; parts' masses
    u64 groups[kMostGroups];
    uint32_t bins[kBins], all[kBins];
    u64 window[kWindow];
    uint32_t window_count[kWindow];
    u64 box[2][2][kMaxCtas];   // what the CTAs tell each other
    u64 sums[kWarps];
    u64 answer;
    int found[2];
    uint32_t listed[2];
    double log_min_p;
};
constexpr int kHeld = (sizeof(Shared) + 15) / 16 * 16;  // where the row's stretch begins
static_assert(kSub <= kBins && kSub <= kList && kSub == 2 * kThreads, "parts' counts and masses");

__device__ __forceinline__ u64 add_across(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sum over lower threads of the CTA, and over all of it (`total`).
template <typename V>
__device__ __forceinline__ V scan_block(V v, V* sums, V& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    V x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    V low = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) low += sums[w];
        total += sums[w];
    }
    return low + x - v;
}

// floor or ceiling of a whole number times a fraction in [0, 1).
__device__ __forceinline__ u64 part_of(u64 whole, float fraction, bool up) {
    // the fraction in units of 2^-64: exact from 2^-40 on
    const float high = ldexpf(fraction, 32), low = ldexpf(high - truncf(high), 32);
    const u64 f = fraction > 0.0f ? static_cast<u64>(high) << 32 | static_cast<u64>(low) : 0;
    return __umul64hi(whole, f) + (up && whole * f != 0 ? 1 : 0);
}

template <typename E>
struct Sampler {
    static constexpr int kV = Row<E>::kV;
    const SampleCall& c;
    Shared& s;
    Row<E> row;
    const uint32_t rank, ctas;
    Scale scale;
    int turn = 0;      // of the boxes
    u64 cut = 0;       // least place kept: that of logit cut_x at index cut_i
    float cut_x;
    uint32_t cut_i;

    __device__ Sampler(const SampleCall& call, Shared& shared, const E* x, uint4* held, uint32_t r, uint32_t n)
        : c(call), s(shared), row(x, held, call.vocab, r, n), rank(r), ctas(n) {}

    __device__ __forceinline__ void keep_from(u64 place) {
        cut = place;
        cut_x = logit_of(place);
        cut_i = ~static_cast<uint32_t>(place);
    }
    // NaN and -inf are not kept
    __device__ __forceinline__ bool kept(float x, int i) const { return x > cut_x || (x == cut_x && static_cast<uint32_t>(i) <= cut_i); }
    // A logit that no one of bin b or before is below.
    __device__ __forceinline__ float lowest_of(int b) const {
        return scale.flat ? scale.top : scale.top - (2.0f * (b + 2) * kBinSteps / scale.hi) * 1.0001f - 1e-5f * fabsf(scale.top);
    }

    // Two numbers of this CTA's to every CTA; afterwards all of them are in the box that comes back. Threads of the CTA
    // agree on the numbers at thread 0 .. kMaxCtas - 1.
    __device__ __forceinline__ u64 (*tell(u64 a, u64 b))[kMaxCtas] {
        u64 (*box)[kMaxCtas] = s.box[turn];
        turn ^= 1;
        if (threadIdx.x < ctas) {
            asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(mapa_shared(smem_u32(&box[0][rank]), threadIdx.x)), "l"(a) : "memory");
            asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(mapa_shared(smem_u32(&box[1][rank]), threadIdx.x)), "l"(b) : "memory");
        }
        cluster_sync();
        return box;
    }
    // A sum over the CTA, at every thread.
    __device__ __forceinline__ u64 sum_block(u64 v) {
        v = add_across(v);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) s.sums[threadIdx.x >> 5] = v;
        __syncthreads();
        u64 t = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) t += s.sums[w];
        return t;
    }
    __device__ __forceinline__ u64 sum_cluster(u64 v) {
        u64 (*box)[kMaxCtas] = tell(sum_block(v), 0);
        u64 t = 0;
        for (uint32_t r = 0; r < ctas; ++r) t += box[0][r];
        return t;
    }

    // The place of the largest logit; 0: there is none above -inf. `ready`: run once every CTA of the cluster runs.
    __device__ u64 largest() {
        float best = kNone;
        int at = INT_MAX;
        row.load([&](int i, const float (&v)[kV]) {
#pragma unroll
            for (int e = 0; e < kV; ++e)
                if (v[e] > best) {
                    best = v[e];
                    at = i + e;
                }
        });
        u64 p = best > kNone ? place_of(best, at) : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) p = max(p, __shfl_xor_sync(0xFFFFFFFFu, p, o));
        if ((threadIdx.x & 31) == 0) s.sums[threadIdx.x >> 5] = p;
        __syncthreads();
        p = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) p = max(p, s.sums[w]);
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");  // the arrival is at the kernel's start: every CTA runs
        u64 (*box)[kMaxCtas] = tell(p, 0);
        for (uint32_t r = 0; r < ctas; ++r) p = max(p, box[0][r]);
        return p;
    }

    // Weights of a piece's kept logits, added up. f(e, bits): each kept one's step, as weigh() has it.
    template <typename F>
    __device__ __forceinline__ u64 weigh_piece(int i, const float (&v)[kV], F f) {
        if (scale.flat) {
            u64 n = 0;
#pragma unroll
            for (int e = 0; e < kV; ++e)
                if (kept(v[e], i + e)) {
                    ++n;
                    f(e, 0x4B400000);
                }
            return n << kUnit;
        }
        float2 hi = both(0.0f), lo = both(0.0f);
#pragma unroll
        for (int e = 0; e < kV; e += 2) {
            const bool k0 = kept(v[e], i + e), k1 = kept(v[e + 1], i + e + 1);
            float2 h, l;
            int n0, n1;
            weigh(make_float2(k0 ? v[e] : scale.top, k1 ? v[e + 1] : scale.top), scale, s.powers, h, l, n0, n1);
            hi = __fadd2_rn(hi, make_float2(k0 ? h.x : 0.0f, k1 ? h.y : 0.0f));
            lo = __fadd2_rn(lo, make_float2(k0 ? l.x : 0.0f, k1 ? l.y : 0.0f));
            if (k0) f(e, n0);
            if (k1) f(e + 1, n1);
        }
        return units(hi.x + hi.y, lo.x + lo.y);
    }

    // Counts of what is kept a bin, of all CTAs, in s.all; with kMass also its weight.
    template <bool kMass>
    __device__ u64 count() {
        for (int b = threadIdx.x; b < kBins; b += kThreads) s.bins[b] = 0;
        __syncthreads();
        u64 mass = 0;
        row.each(cut_x, [&](int, int i, const float (&v)[kV]) {
            // many equal logits: one addition a warp
            bool same = true;
#pragma unroll
            for (int e = 1; e < kV; ++e) same &= v[e] == v[0];
            const float first = __shfl_sync(0xFFFFFFFFu, v[0], 0);
            if (__all_sync(0xFFFFFFFFu, same && v[0] == first && v[0] > cut_x)) {
                if ((threadIdx.x & 31) == 0) atomicAdd(&s.bins[bin_of(first, scale)], 32u * kV);
                if (kMass) mass += weight_of(first, scale, s.powers) * kV;
                return;
            }
            auto add = [&](int, int bits) { atomicAdd(&s.bins[bin_of_bits(bits)], 1u); };
            if constexpr (kMass) {
                mass += weigh_piece(i, v, add);
            } else {
#pragma unroll
                for (int e = 0; e < kV; ++e)
                    if (kept(v[e], i + e)) atomicAdd(&s.bins[bin_of(v[e], scale)], 1u);
            }
        });
        const u64 total = kMass ? sum_cluster(mass) : (cluster_sync(), 0);
        for (int b = threadIdx.x; b < kBins; b += kThreads) {
            uint32_t n = 0;
            for (uint32_t r = 0; r < ctas; ++r) {
                uint32_t x;
                asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(mapa_shared(smem_u32(&s.bins[b]), r)));
                n += x;
            }
            s.all[b] = n;
        }
        __syncthreads();
        return total;
    }

    // The weight of what is kept.
    __device__ u64 mass() {
        u64 sum = 0;
        row.each(cut_x, [&](int, int i, const float (&v)[kV]) { sum += weigh_piece(i, v, [](int, int) {}); });
        return sum_cluster(sum);
    }

    // Among counts v(b): the first bin up to which they reach `want`, and the sum before it; kBins where they do not.
    template <typename V, typename F>
    __device__ void reach(F v, V want, V* sums, int& bin, V& before) {
        constexpr int kEach = (kBins + kThreads - 1) / kThreads;
        V mine = 0, total;
        const int b0 = threadIdx.x * kEach;
        for (int b = b0; b < min(kBins, b0 + kEach); ++b) mine += v(b);
        V at = scan_block(mine, sums, total);
        if (threadIdx.x == 0) s.found[0] = kBins;
        __syncthreads();
        V past = at;
        for (int b = b0; b < min(kBins, b0 + kEach); ++b) {
            const V next = past + v(b);
            if (past < want && next >= want) {
                s.found[0] = b;
                s.answer = 0;
                memcpy(&s.answer, &past, sizeof(V));
            }
            past = next;
        }
        __syncthreads();
        bin = s.found[0];
        before = total;
        if (bin < kBins) memcpy(&before, &s.answer, sizeof(V));
        __syncthreads();
    }

    // Brings the kept places of logits of at least `least` for which f holds together in the first CTA's list, at most kList. The cluster
    // meets afterwards.
    template <typename F>
    __device__ void gather(int which, float least, F f) {
        const uint32_t counter = mapa_shared(smem_u32(&s.listed[which]), 0), list = mapa_shared(smem_u32(s.list), 0);
        const int lane = threadIdx.x & 31;
        row.each(fmaxf(least, cut_x), [&](int, int i, const float (&v)[kV]) {
            uint32_t mine = 0;
#pragma unroll
            for (int e = 0; e < kV; ++e)
                if (kept(v[e], i + e) && f(v[e], i + e)) mine |= 1u << e;
            int x = __popc(mine);
            const int own = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
                if (lane >= o) x += y;
            }
            uint32_t at = 0;
            if (lane == 31 && x > 0) asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(at) : "r"(counter), "r"(x) : "memory");
            at = __shfl_sync(0xFFFFFFFFu, at, 31) + x - own;
#pragma unroll
            for (int e = 0; e < kV; ++e)
                if (mine >> e & 1) {
                    if (at < kList) asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(list + 8 * at), "l"(place_of(v[e], i + e)) : "memory");
                    ++at;
                }
        });
        cluster_sync();
    }

    // Sorts n numbers of the list, the largest first (first CTA).
    __device__ void sort(int n) {
        int size = 1;
        while (size < n) size *= 2;
        for (int i = n + threadIdx.x; i < size; i += kThreads) s.list[i] = 0;
        for (int k = 2; k <= size; k *= 2)
            for (int j = k / 2; j > 0; j /= 2) {
                __syncthreads();
                for (int t = threadIdx.x; t < size / 2; t += kThreads) {
                    const int lo = 2 * t - (t & (j - 1)), hi = lo + j;
                    const u64 a = s.list[lo], b = s.list[hi];
                    if ((a < b) == ((lo & k) == 0)) {
                        s.list[lo] = b;
                        s.list[hi] = a;
                    }
                }
            }
        __syncthreads();
    }

    // In the first CTA's sorted list of n places: how many come first that have less than `target` of weight before them (at least one).
    // total: the weight of all n.
    __device__ int within(int n, u64 target, u64& total) {
        constexpr int kEach = kList / kThreads;
        const int i0 = threadIdx.x * kEach;
        u64 w[kEach], mine = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            w[i] = i0 + i < n ? weight_of(logit_of(s.list[i0 + i]), scale, s.powers) : 0;
            mine += w[i];
        }
        u64 before = scan_block(mine, s.sums, total);
        if (threadIdx.x == 0) s.found[1] = 1;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (i0 + i < n && before < target) atomicMax(&s.found[1], i0 + i + 1);
            before += w[i];
        }
        __syncthreads();
        return s.found[1];
    }

    // The cut inside bin b, which holds n places >= cut: the target-th of them, or with kMass the last one that has less than
    // `target` of the bin's weight before it.
    template <bool kMass>
    __device__ u64 inside(int which, int b, uint32_t n, u64 target) {
        u64 low = 0, high = ~0ull;
        const float from = fmaxf(lowest_of(b), cut_x);
        if (n > kList) {  // first the bin's own range
            u64 least = ~0ull, most = 0;
            row.each(from, [&](int, int i, const float (&v)[kV]) {
#pragma unroll
                for (int e = 0; e < kV; ++e)
                    if (kept(v[e], i + e) && bin_of(v[e], scale) == b) {
                        least = min(least, place_of(v[e], i + e));
                        most = max(most, place_of(v[e], i + e));
                    }
            });
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                least = min(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
                most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
            }
            if (threadIdx.x == 0) {
                s.groups[0] = ~0ull;
                s.groups[1] = 0;
            }
            __syncthreads();
            if ((threadIdx.x & 31) == 0) {
                atomicMin(&s.groups[0], least);
                atomicMax(&s.groups[1], most);
            }
            __syncthreads();
            u64 (*box)[kMaxCtas] = tell(s.groups[0], s.groups[1]);
            low = ~0ull;
            high = 0;
            for (uint32_t r = 0; r < ctas; ++r) {
                low = min(low, box[0][r]);
                high = max(high, box[1][r]);
            }
        }
        while (n > kList) {  // parts of the range, down to one that the list can hold
            const int bits = 64 - __clzll(high - low), shift = max(0, bits - 10);
            u64* mass = s.list;
            for (int i = threadIdx.x; i < kSub; i += kThreads) {
                s.bins[i] = 0;
                mass[i] = 0;
            }
            __syncthreads();
            row.each(from, [&](int, int i, const float (&v)[kV]) {
#pragma unroll
                for (int e = 0; e < kV; ++e) {
                    if (!kept(v[e], i + e) || bin_of(v[e], scale) != b) continue;
                    const u64 p = place_of(v[e], i + e);
                    if (p < low || p > high) continue;
                    const int at = static_cast<int>((high - p) >> shift);
                    atomicAdd(&s.bins[at], 1u);
                    if (kMass) atomicAdd(&mass[at], weight_of(v[e], scale, s.powers));
                }
            });
            cluster_sync();
            // a part a thread, twice: the sums of all CTAs
            auto sum = [&](int i, u64& m) {
                uint32_t k = 0;
                m = 0;
                for (uint32_t r = 0; r < ctas; ++r) {
                    uint32_t x;
                    u64 y;
                    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(mapa_shared(smem_u32(&s.bins[i]), r)));
                    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(y) : "r"(mapa_shared(smem_u32(&mass[i]), r)));
                    k += x;
                    m += y;
                }
                return k;
            };
            u64 m0, m1, total;
            const uint32_t k0 = sum(2 * threadIdx.x, m0), k1 = sum(2 * threadIdx.x + 1, m1);
            const u64 a0 = kMass ? m0 : k0, a1 = kMass ? m1 : k1;
            const u64 before = scan_block(a0 + a1, s.sums, total);
            if (before < target && before + a0 + a1 >= target) {
                const bool second = before + a0 < target;
                s.found[0] = 2 * threadIdx.x + second;
                s.found[1] = static_cast<int>(second ? k1 : k0);
                s.answer = before + (second ? a0 : 0);
            }
            cluster_sync();  // nobody reads the others' parts any more
            const u64 at = static_cast<u64>(s.found[0]) << shift;
            n = static_cast<uint32_t>(s.found[1]);
            target -= s.answer;
            const u64 top = high - at, span = (1ull << shift) - 1;
            low = top - low > span ? top - span : low;
            high = top;
            __syncthreads();
        }
        gather(which, from, [&](float x, int i) { return bin_of(x, scale) == b && place_of(x, i) >= low && place_of(x, i) <= high; });
        u64 found = 0;
        if (rank == 0) {
            sort(static_cast<int>(n));
            u64 all;
            const int i = kMass ? within(static_cast<int>(n), target, all) - 1 : static_cast<int>(target) - 1;
            found = s.list[i];
            __syncthreads();
        }
        return tell(found, 0)[0][0];
    }

    // The token in which u of the weight of the first n places of the first CTA's sorted list is passed, by index.
    __device__ void draw_list(int n, float u, int32_t* token) {
        // by index, with the logit in the low half: the lowest index is the largest number
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const u64 p = s.list[i];
            s.list[i] = p << 32 | p >> 32;
        }
        sort(n);
        constexpr int kEach = kList / kThreads;
        const int i0 = threadIdx.x * kEach;
        u64 w[kEach], mine = 0, total;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            w[i] = i0 + i < n ? weight_of(logit_of(s.list[i0 + i] << 32), scale, s.powers) : 0;
            mine += w[i];
        }
        u64 before = scan_block(mine, s.sums, total);
        const u64 want = part_of(total, u, false);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (before <= want && want < before + w[i]) *token = index_of(s.list[i0 + i] >> 32);
            before += w[i];
        }
    }

    // The token in which u of the weight of what is kept is passed.
    __device__ void draw(float u, int32_t* token) {
        u64 mine = 0;
        for (int g = threadIdx.x / 32 + (threadIdx.x & 31) * kWarps; g < row.groups; g += kThreads) s.groups[g] = 0;
        __syncwarp();
        row.each(cut_x, [&](int g, int i, const float (&v)[kV]) {
            const u64 sum = add_across(weigh_piece(i, v, [](int, int) {}));
            if ((threadIdx.x & 31) == 0) {
                s.groups[g] = sum;
                mine += sum;
            }
        });
        const u64 all = sum_block(mine);
        u64 (*box)[kMaxCtas] = tell(all, 0);
        u64 total = 0, before = 0;
        for (uint32_t r = 0; r < ctas; ++r) {
            if (r < rank) before += box[0][r];
            total += box[0][r];
        }
        const u64 want = part_of(total, u, false);
        if (want < before || want >= before + all) return;  // another CTA's
        static_assert(kMostGroups <= kThreads, "a group a thread");
        const u64 sum = threadIdx.x < row.groups ? s.groups[threadIdx.x] : 0;
        u64 whole;
        const u64 at = before + scan_block(sum, s.sums, whole);
        if (at <= want && want < at + sum) {
            s.found[0] = threadIdx.x;
            s.answer = at;
        }
        __syncthreads();
        if (threadIdx.x >= 32) return;
        const int g = s.found[0], i = row.index(g);
        float v[kV];
        Row<E>::open(row.held[g * 32 + threadIdx.x], v);
        u64 w[kV], lane_sum = 0;
#pragma unroll
        for (int e = 0; e < kV; ++e) {
            w[e] = kept(v[e], i + e) ? weight_of(v[e], scale, s.powers) : 0;
            lane_sum += w[e];
        }
        u64 x = lane_sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (threadIdx.x >= o) x += y;
        }
        u64 past = s.answer + x - lane_sum;
#pragma unroll
        for (int e = 0; e < kV; ++e) {
            if (past <= want && want < past + w[e]) *token = i + e;
            past += w[e];
        }
    }

    // About the weight in bin b, from its count.
    __device__ __forceinline__ u64 guess(int b) const {
        const int n = -(b * kBinSteps + kBinSteps / 2 - 1);
        const float w = s.powers[n & (kSteps - 1)].x * __int_as_float(((kUnit + (n >> 8)) + 127) << 23);
        return s.all[b] * max(static_cast<u64>(w), 1ull);
    }

    // Whether what reaches `target` of the weight, by the counts a bin, fits the list, and then the token, drawn from it.
    __device__ bool draw_nucleus(u64 target, float u, int32_t* token) {
        int bin;
        u64 before;
        reach<u64>([&](int b) { return guess(b); }, target, s.sums, bin, before);
        bin = min(bin + 1, kBins - 1);  // the guess may be a little high
        u64 n = 0;
        for (int b = threadIdx.x; b <= bin; b += kThreads) n += s.all[b];
        n = sum_block(n);
        if (n > kList) return false;
        gather(0, lowest_of(bin), [&](float x, int) { return bin_of(x, scale) <= bin; });
        u64 enough = 0;
        if (rank == 0) {
            sort(static_cast<int>(n));
            const int k = within(static_cast<int>(n), target, enough);
            enough = enough >= target;
            if (enough) draw_list(k, u, token);
        }
        return tell(enough, 0)[0][0] != 0;
    }

    // The last place that has less than `target` of the weight of what is kept before it, given the counts a bin. Guesses where the
    // border is from the counts, and takes the exact weight above, and in the kWindow bins there; where the guess missed,
    // the next one starts from what is known exactly, on the border's side of the window: the search ends.
    __device__ u64 nucleus(u64 target) {
        int64_t known = 0;           // exact less guessed weight before a window
        int least = 0, most = kBins; // the border's bin is one of least .. most - 1
        while (true) {
            int bin;
            u64 skipped;
            reach<u64>([&](int b) { return guess(b); }, static_cast<u64>(max(static_cast<int64_t>(target) - known, static_cast<int64_t>(1))), s.sums, bin, skipped);
            const int from = max(least, min(bin - kWindow / 2, most - kWindow));
            for (int i = threadIdx.x; i < kWindow; i += kThreads) {
                s.window[i] = 0;
                s.window_count[i] = 0;
            }
            __syncthreads();
            u64 above = 0;
            row.each(fmaxf(cut_x, lowest_of(from + kWindow - 1)), [&](int, int i, const float (&v)[kV]) {
#pragma unroll
                for (int e = 0; e < kV; ++e) {
                    if (!kept(v[e], i + e)) continue;
                    const int b = bin_of(v[e], scale);
                    if (b >= from + kWindow) continue;
                    const u64 w = weight_of(v[e], scale, s.powers);
                    if (b < from) {
                        above += w;
                    } else {
                        atomicAdd(&s.window[b - from], w);
                        atomicAdd(&s.window_count[b - from], 1u);
                    }
                }
            });
            above = sum_cluster(above);
            u64 in = 0;
            uint32_t many = 0;
            if (threadIdx.x < kWindow)
                for (uint32_t r = 0; r < ctas; ++r) {
                    u64 x;
                    uint32_t y;
                    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(x) : "r"(mapa_shared(smem_u32(&s.window[threadIdx.x]), r)));
                    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(y) : "r"(mapa_shared(smem_u32(&s.window_count[threadIdx.x]), r)));
                    in += x;
                    many += y;
                }
            u64 inside_all;
            const u64 before = above + scan_block(in, s.sums, inside_all);
            if (threadIdx.x < kWindow && before < target && before + in >= target) {
                s.found[0] = from + threadIdx.x;
                s.found[1] = static_cast<int>(many);
                s.answer = before;
            }
            cluster_sync();  // nobody reads the others' windows any more
            if (above < target && target <= above + inside_all) {
                const int b = s.found[0], n = s.found[1];
                const u64 left = target - s.answer;
                __syncthreads();
                return inside<true>(1, b, static_cast<uint32_t>(n), left);
            }
            if (target <= above) most = from;
            else least = from + kWindow;
            u64 part = 0, guessed;
            for (int b = threadIdx.x; b < from; b += kThreads) part += guess(b);
            scan_block(part, s.sums, guessed);
            known = static_cast<int64_t>(above - guessed);
        }
    }
};

__device__ __forceinline__ float setting(const float* p, float all, int64_t r) { return p != nullptr ? __ldg(p + r) : all; }

template <typename E>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleCall c) {
    extern __shared__ uint4 smem[];
    Shared& s = *reinterpret_cast<Shared*>(smem);
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    const uint32_t rank = cluster_ctarank();
    uint32_t ctas;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    const int64_t r = blockIdx.x / ctas;
    Sampler<E> w(c, s, static_cast<const E*>(c.x) + r * c.row_stride, smem + kHeld / 16, rank, ctas);
    const float temperature = setting(c.temperature, c.temperature_all, r), min_p = setting(c.min_p, c.min_p_all, r);
    const float top_p = setting(c.top_p, c.top_p_all, r), u_given = __ldg(c.u + r);
    const int top_k = c.top_k != nullptr ? __ldg(c.top_k + r) : c.top_k_all;
    const float u = u_given > 0.0f ? fminf(u_given, 0.99999994f) : 0.0f;
    const bool greedy = !(temperature > 0.0f);
    for (int i = threadIdx.x; i < kSteps; i += kThreads) s.powers[i] = kPowers.v[i];
    if (threadIdx.x == 0) s.listed[0] = s.listed[1] = 0;
    if (threadIdx.x == kThreads - 32 && !greedy && min_p > 0.0f && min_p < 1.0f)  // in 64 bits, once, while the others read
        s.log_min_p = static_cast<double>(temperature) * log(static_cast<double>(min_p));
    const u64 top = w.largest();
    if (top == 0) {
        if (rank == 0 && threadIdx.x == 0) c.tokens[r] = -1;
        return;
    }
    if (greedy) {
        if (rank == 0 && threadIdx.x == 0) c.tokens[r] = index_of(top);
        return;
    }
    {
        // 512 log2(e) / T as hi + lo: 1 / T = y + y (1 - y T), good to 2^-46
        constexpr double kFactor = 512.0 * 1.4426950408889634074;
        constexpr float kHi = static_cast<float>(kFactor), kLo = static_cast<float>(kFactor - static_cast<double>(kHi));
        const float y = 1.0f / temperature, yl = y * fmaf(-y, temperature, 1.0f), hi = fminf(y * kHi, 3e38f);
        const float lo = fmaf(y, kHi, -hi) + fmaf(y, kLo, yl * kHi), x = logit_of(top);
        w.scale = Scale{x, hi, fabsf(lo) <= 1e-6f * hi ? lo : 0.0f, isinf(x)};  // 0 where T or 1 / T is infinite
        // what is kept at all: above -inf, and not so small that a weight is nothing (2^-45 and below)
        const float none = x - 45.0f * 0.6931472f * temperature;
        const u64 finite = static_cast<u64>(key_of(kNone) + 1) << 32;
        u64 cut = w.scale.flat ? top >> 32 << 32 : none > kNone ? max(finite, static_cast<u64>(key_of(none)) << 32) : finite;
        if (min_p >= 1.0f) {
            cut = top >> 32 << 32;
        } else if (min_p > 0.0f) {
            const double least = static_cast<double>(x) + s.log_min_p;
            float z = static_cast<float>(least);
            if (static_cast<double>(z) < least) z = nextafterf(z, INFINITY);  // the least float that is not below
            cut = max(cut, static_cast<u64>(key_of(z)) << 32);
        }
        w.keep_from(cut);
    }
    const bool by_count = top_k > 0 && top_k < c.vocab, by_mass = top_p < 1.0f;
    auto target_of = [&](u64 total) { return max(part_of(total, fmaxf(top_p, 0.0f), true), 1ull); };
    if (by_count) {
        w.template count<false>();
        int bin;
        uint32_t before;
        w.template reach<uint32_t>([&](int b) { return s.all[b]; }, static_cast<uint32_t>(top_k), reinterpret_cast<uint32_t*>(s.sums), bin, before);
        const uint32_t to = bin < kBins ? before + s.all[bin] : before;  // places to the end of that bin
        if (to <= kList) {
            const int last = min(bin, kBins - 1);
            w.gather(0, w.lowest_of(last), [&](float x, int) { return bin_of(x, w.scale) <= last; });
            if (rank == 0) {
                w.sort(static_cast<int>(to));
                int n = min(static_cast<int>(to), top_k);
                if (by_mass) {
                    u64 total;
                    w.within(n, 1, total);
                    n = w.within(n, target_of(total), total);
                }
                w.draw_list(n, u, c.tokens + r);
            }
            return;
        }
        if (bin < kBins) {
            const uint32_t n = s.all[bin];
            w.keep_from(w.template inside<false>(0, bin, n, top_k - before));
            if (by_mass) {  // the counts without what has been cut off
                __syncthreads();
                for (int b = bin + threadIdx.x; b < kBins; b += kThreads) s.all[b] = b == bin ? top_k - before : 0;
                __syncthreads();
            }
        }
        if (by_mass) w.keep_from(w.nucleus(target_of(w.mass())));
    } else if (by_mass) {
        const u64 target = target_of(w.template count<true>());
        if (w.draw_nucleus(target, u, c.tokens + r)) return;
        w.keep_from(w.nucleus(target));
    }
    w.draw(u, c.tokens + r);
}

template <typename E>
cudaError_t launch(const SampleCall& c, int sm_count, cudaStream_t stream) {
    static int attr_gen[64] = {};
    auto* kernel = sample_kernel<E>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && attr_gen[dev] != g_generation) {
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeld + (kMostGroups - 1) * 512)) != cudaSuccess) return e;
        attr_gen[dev] = g_generation;
    }
    // CTAs of a row: as many as give the GPU two CTAs an SM, with at least 2048 logits each, and at least so many that two stretches
    // fit an SM's shared memory
    const int64_t pieces = (c.vocab + Row<E>::kV - 1) / Row<E>::kV + 1, groups = (pieces + 31) / 32;
    int ctas = 1;
    while (ctas < kMaxCtas && ((c.rows * ctas * 2 <= 2 * sm_count && c.vocab > 2048 * ctas) || groups > kMostGroups / 2 * ctas)) ctas *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(c.rows * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kHeld + (groups + ctas - 1) / ctas * 512;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {static_cast<unsigned>(ctas), 1, 1};
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, c);
}

}  // namespace

cudaError_t launch_sample(const SampleCall& c, int sm_count, cudaStream_t stream) {
    if (c.dtype == kFp16) return launch<__half>(c, sm_count, stream);
    if (c.dtype == kBf16) return launch<__nv_bfloat16>(c, sm_count, stream);
    return launch<float>(c, sm_count, stream);
}

}  // namespace tg
