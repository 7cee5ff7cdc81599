// Drawing a token from each row of logits: temperature, the top_k largest, a
// least weight min_p, the top_p of the mass, and one given number u a row.
//
//     w_i = exp((x_i - max) / T) = 2^t_i,  token = first kept i with sum_{j <= i, kept} w_j > u sum_{kept} w_j
//
// The answer is a whole number, and a border (of the mass, or of u) lies between
// two tokens of a vocabulary of 10^5, whose shares are about 10^-5 of the sum or
// less: sums in 32 bits, off by 10^-7 and by how the row was split, would give
// another token in one row of some hundreds. So weights are integers, of 2^-44 of the
// row's largest, from a 2^t good to 2^-40 (fixed_weight), and sums of them are exact
// in 64 bits: the same whatever the order, the split and the rest of the batch.
//
// Order: a token's rank is that of its 64-bit `place`: the logit's bits as an
// ordered 32-bit integer, then the index inverted, so equal logits rank by index
// and what a row keeps is every place >= one cut.
//
// A cluster of CTAs takes a row, each CTA a stretch of it; passes after the first
// find the row in L2. The passes, of which a row makes those its settings ask for:
//   1  the largest logit (a greedy row ends here);
//   2  a count in each of kBins bins of t, 1/32 wide: the bin with the k-th, and a
//      guess at the bin in which the mass reaches top_p;
//   3  the exact mass above, in each bin near the guess, and below;
//   4  the tokens of a border's bin, brought together and sorted: the cut;
//   5  the mass of what is kept, group by group of 32 lanes' pieces; the group,
//      lane and token in which u of it is passed.
// With few tokens to the k-th's bin they are brought together at once, and the first
// CTA does the rest in its shared memory.
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
constexpr int kUnit = 44;                    // weights are multiples of 2^-44
constexpr int kSteps = 256;                  // of the table of powers: 2^(j / 256)
constexpr int kBinSteps = 8;                 // of a bin
constexpr int kBins = (kUnit + 1) * kSteps / kBinSteps;
constexpr int kWindow = 16;                  // bins whose mass is taken exactly at a time
constexpr int kList = 2048;                  // tokens that are sorted at a time
constexpr int kSub = 1024;                   // parts of a bin that holds more
constexpr int kMaxGroups = (1 << 18) / 128 + 2;
constexpr float kNone = -INFINITY;
constexpr float kLeast = 1 - (kUnit + 1) * kSteps;  // of 256 t: below 2^-45 nothing is left of a weight
using u64 = unsigned long long;

// 2^(j / 256) in units of 2^-44, by repeated square roots and products in integers.
struct Powers {
    uint64_t v[kSteps];
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
        p.v[j] = (x + (1ull << 17)) >> 18;
        x = product_2_62(x, step);
    }
    return p;
}
__device__ const Powers kPowers = make_powers();

// What a row's logits are weighed with.
struct Scale {
    float top;       // the largest logit
    float hi, lo;    // 2 * 256 log2(e) / T
};

// 256 t of a logit as the nearest integer (at most 0), or 1 where the weight is none. Falls as x falls, so bins of it are in order.
__device__ __forceinline__ int step_of(float x, const Scale& c) {
    const float p = __fmul_rn(__fmaf_rn(0.5f, x, -0.5f * c.top), c.hi);  // halves: the difference of two finite logits stays finite
    if (x == c.top) return 0;
    if (!(p > kLeast)) return 1;
    return __float_as_int(__fadd_rn(p, 12582912.0f)) - 0x4B400000;
}

// 2^t in units of 2^-44, off by at most 2^-40 of itself and a half. With the difference of the logits as d + e exactly and
// the factor as hi + lo, 256 t = p + q; n = round(p), 2^(n / 256) is a power of two and a table's entry, and what
// is left, f = p - n + q, at most 1/2 and a little, gives 2^(f / 256) = 1 + y + y^2 / 2 + y^3 / 6, y = f ln(2) / 256 <= 2^-9.5: y^4 / 24 is
// 2^-42. y is a sum of two floats, and 1 + y .. goes into the product with the entry in steps of 2^-40.
__device__ __forceinline__ u64 fixed_weight(float x, const Scale& c, const u64* powers) {
    if (x == c.top) return 1ull << kUnit;
    const float a = 0.5f * x, b = -0.5f * c.top, d = __fadd_rn(a, b);
    const float p = __fmul_rn(d, c.hi);
    if (!(p > kLeast)) return 0;
    const float bb = __fsub_rn(d, a), e = __fadd_rn(__fsub_rn(a, __fsub_rn(d, bb)), __fsub_rn(b, bb));
    const float q = __fadd_rn(__fmaf_rn(d, c.hi, -p), __fmaf_rn(d, c.lo, __fmul_rn(e, c.hi)));
    const float m = __fadd_rn(p, 12582912.0f);
    const int n = __float_as_int(m) - 0x4B400000;
    const float f = __fsub_rn(p, __fsub_rn(m, 12582912.0f));
    // ln(2) / 256 as two floats
    constexpr double kLn = 0.693147180559945309417 / 256;
    constexpr float kLnHi = static_cast<float>(kLn), kLnLo = static_cast<float>(kLn - static_cast<double>(kLnHi));
    const float y = __fmul_rn(f, kLnHi);
    const float yl = __fadd_rn(__fmaf_rn(f, kLnHi, -y), __fmaf_rn(f, kLnLo, __fmul_rn(q, kLnHi)));
    const float z = __fmaf_rn(__fmul_rn(y, y), __fmaf_rn(y, 1.0f / 6.0f, 0.5f), __fmaf_rn(y, yl, yl));
    const int w = __float2int_rn(y * 1099511627776.0f) + __float2int_rn(z * 1099511627776.0f);
    const u64 t = powers[n & (kSteps - 1)];
    const int64_t v = static_cast<int64_t>(t) + ((static_cast<int64_t>(w) * static_cast<uint32_t>(t >> 14)) >> 26);
    const int down = -(n >> 8);
    return down == 0 ? v : (static_cast<u64>(v) + (1ull << (down - 1))) >> down;
}

// A logit's rank among all: larger ones higher, of equal ones the lower index. -inf and NaN are brought to -inf, -0 to 0.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ u64 place_of(float x, int i) { return static_cast<u64>(key_of(x)) << 32 | static_cast<uint32_t>(~i); }
__device__ __forceinline__ int index_of(u64 place) { return static_cast<int>(~static_cast<uint32_t>(place)); }
__device__ __forceinline__ float logit_of(u64 place) {
    const uint32_t k = static_cast<uint32_t>(place >> 32);
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

template <typename E>
__device__ __forceinline__ float logit(E v) {
    float x;
    if constexpr (std::is_same<E, float>::value) x = v;
    else x = to_float(v);
    return x == x ? x + 0.0f : kNone;
}

// This CTA's stretch of a row: pieces of 16 bytes, kV logits each, on 16-byte boundaries (the first and the last may reach beyond the row);
// 32 pieces are a group.
template <typename E>
struct Row {
    static constexpr int kV = 16 / sizeof(E);
    const E* x;
    int vocab, shift;     // index of piece q's first logit: q * kV - shift
    int group0, groups;   // of this CTA
    __device__ Row(const E* row, int n, uint32_t rank, uint32_t ctas) : x(row), vocab(n) {
        shift = static_cast<int>(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(E));
        const int all = ((n + shift + kV - 1) / kV + 31) / 32, each = (all + ctas - 1) / ctas;
        group0 = min(all, static_cast<int>(rank) * each);
        groups = min(all, group0 + each) - group0;
    }
    __device__ uint4 raw(int group) const {
        const int i = ((group0 + group) * 32 + (threadIdx.x & 31)) * kV - shift;
        uint4 u;
        if (i >= 0 && i + kV <= vocab) return *reinterpret_cast<const uint4*>(x + i);
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
    __device__ int index(int group) const { return ((group0 + group) * 32 + (threadIdx.x & 31)) * kV - shift; }
    // f(group, index of the first, its kV logits), whole warps
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        constexpr int kAhead = 4;
        for (int g = threadIdx.x / 32; g < groups; g += kWarps * kAhead) {
            uint4 u[kAhead];
#pragma unroll
            for (int a = 0; a < kAhead; ++a)
                if (g + a * kWarps < groups) u[a] = raw(g + a * kWarps);
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                if (g + a * kWarps >= groups) break;
                const E* e = reinterpret_cast<const E*>(&u[a]);
                float v[kV];
#pragma unroll
                for (int i = 0; i < kV; ++i) v[i] = logit(e[i]);
                f(g + a * kWarps, index(g + a * kWarps), v);
            }
        }
    }
};

struct Shared {
    u64 powers[kSteps];
    u64 list[kList];           // of the first CTA; parts' masses
    u64 groups[kMaxGroups];
    uint32_t bins[kBins], all[kBins];
    u64 window[kWindow];
    uint32_t window_count[kWindow];
    u64 box[2][2][kMaxCtas];   // what the CTAs tell each other
    u64 sums[kWarps];
    u64 answer;
    int found[2];
    uint32_t listed[2];
    double log_min_p;
    float hi, lo;
};

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
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) low += sums[w];
        total += sums[w];
    }
    return low + x - v;
}

// floor and ceiling of a whole number times a fraction in [0, 1).
__device__ __forceinline__ u64 part_of(u64 whole, float fraction, bool up) {
    // the fraction in units of 2^-64: exact from 2^-40 on
    const u64 f = fraction > 0.0f ? static_cast<u64>(ldexpf(fraction, 32)) << 32 | static_cast<u64>(ldexpf(ldexpf(fraction, 32) - truncf(ldexpf(fraction, 32)), 32)) : 0;
    const u64 hi = __umul64hi(whole, f);
    return hi + (up && whole * f != 0 ? 1 : 0);
}

template <typename E>
struct Sampler {
    const SampleCall& c;
    Shared& s;
    const Row<E> row;
    const uint32_t rank, ctas;
    Scale scale;
    int turn = 0;   // of the boxes
    u64 cut = 0;    // least place kept

    __device__ Sampler(const SampleCall& call, Shared& shared, const E* x, uint32_t r, uint32_t n) : c(call), s(shared), row(x, call.vocab, r, n), rank(r), ctas(n) {}

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
        for (int w = 0; w < kWarps; ++w) t += s.sums[w];
        return t;
    }
    __device__ __forceinline__ int bin_of(float x) const {
        const int n = step_of(x, scale);
        return n > 0 ? kBins : -n / kBinSteps;
    }

    // The place of the largest logit.
    __device__ u64 largest() {
        float best = kNone;
        int at = INT_MAX;
        row.each([&](int, int i, const float (&v)[Row<E>::kV]) {
#pragma unroll
            for (int e = 0; e < Row<E>::kV; ++e)
                if (v[e] > best) {
                    best = v[e];
                    at = i + e;
                }
        });
        u64 p = best > kNone ? place_of(best, at) : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) p = max(p, __shfl_xor_sync(0xFFFFFFFFu, p, o));
        __syncthreads();
        if ((threadIdx.x & 31) == 0) s.sums[threadIdx.x >> 5] = p;
        __syncthreads();
        p = 0;
        for (int w = 0; w < kWarps; ++w) p = max(p, s.sums[w]);
        u64 (*box)[kMaxCtas] = tell(p, 0);
        for (uint32_t r = 0; r < ctas; ++r) p = max(p, box[0][r]);
        return p;
    }

    // Counts of the row's places >= cut a bin, of all CTAs, in s.all.
    __device__ void count() {
        for (int b = threadIdx.x; b < kBins; b += kThreads) s.bins[b] = 0;
        __syncthreads();
        row.each([&](int, int i, const float (&v)[Row<E>::kV]) {
#pragma unroll
            for (int e = 0; e < Row<E>::kV; ++e) {
                const int b = place_of(v[e], i + e) >= cut ? bin_of(v[e]) : kBins, first = __shfl_sync(0xFFFFFFFFu, b, 0);
                if (__all_sync(0xFFFFFFFFu, b == first)) {  // many equal logits: one addition
                    if (b < kBins && (threadIdx.x & 31) == 0) atomicAdd(&s.bins[b], 32u);
                } else if (b < kBins) {
                    atomicAdd(&s.bins[b], 1u);
                }
            }
        });
        cluster_sync();
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

    // Brings the places for which f holds together in the first CTA's list, at most kList.
    template <typename F>
    __device__ void gather(int which, F f) {
        const uint32_t counter = mapa_shared(smem_u32(&s.listed[which]), 0), list = mapa_shared(smem_u32(s.list), 0);
        const int lane = threadIdx.x & 31;
        row.each([&](int, int i, const float (&v)[Row<E>::kV]) {
#pragma unroll
            for (int e = 0; e < Row<E>::kV; ++e) {
                const u64 p = place_of(v[e], i + e);
                const bool in = p >= cut && f(v[e], p);
                const uint32_t who = __ballot_sync(0xFFFFFFFFu, in);
                if (who == 0) continue;
                uint32_t at = 0;
                if (lane == 0) asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(at) : "r"(counter), "r"(__popc(who)) : "memory");
                at = __shfl_sync(0xFFFFFFFFu, at, 0) + __popc(who & ((1u << lane) - 1));
                if (in && at < kList) asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(list + 8 * at), "l"(p) : "memory");
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
    __device__ int within(int n, u64 target) {
        constexpr int kEach = kList / kThreads;
        const int i0 = threadIdx.x * kEach;
        u64 mine = 0, total;
        for (int i = i0; i < min(n, i0 + kEach); ++i) mine += fixed_weight(logit_of(s.list[i]), scale, s.powers);
        u64 before = scan_block(mine, s.sums, total);
        if (threadIdx.x == 0) s.found[1] = 1;
        __syncthreads();
        for (int i = i0; i < min(n, i0 + kEach); ++i) {
            if (before < target) atomicMax(&s.found[1], i + 1);
            before += fixed_weight(logit_of(s.list[i]), scale, s.powers);
        }
        __syncthreads();
        return s.found[1];
    }

    // The cut inside bin b, which holds n places >= cut: the target-th of them, or with kMass the last one that has less than
    // `target` of the bin's weight before it.
    template <bool kMass>
    __device__ u64 inside(int which, int b, uint32_t n, u64 target) {
        u64 low = 0, high = ~0ull;
        if (n > kList) {  // first the bin's own range
            u64 least = ~0ull, most = 0;
            row.each([&](int, int i, const float (&v)[Row<E>::kV]) {
#pragma unroll
                for (int e = 0; e < Row<E>::kV; ++e) {
                    const u64 p = place_of(v[e], i + e);
                    if (p >= cut && bin_of(v[e]) == b) {
                        least = min(least, p);
                        most = max(most, p);
                    }
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
            row.each([&](int, int i, const float (&v)[Row<E>::kV]) {
#pragma unroll
                for (int e = 0; e < Row<E>::kV; ++e) {
                    const u64 p = place_of(v[e], i + e);
                    if (p < max(low, cut) || p > high || bin_of(v[e]) != b) continue;
                    const int at = static_cast<int>((high - p) >> shift);
                    atomicAdd(&s.bins[at], 1u);
                    if (kMass) atomicAdd(&mass[at], fixed_weight(v[e], scale, s.powers));
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
        gather(which, [&](float x, u64 p) { return p >= low && p <= high && bin_of(x) == b; });
        u64 found = 0;
        if (rank == 0) {
            sort(static_cast<int>(n));
            const int i = kMass ? within(static_cast<int>(n), target) - 1 : static_cast<int>(target) - 1;
            found = s.list[i];
            __syncthreads();
        }
        return tell(found, 0)[0][0];
    }

    // The token of rank-0 lists: n places, sorted, of which what top_p keeps is drawn from.
    __device__ void draw_list(int n, float top_p, float u, int32_t* token) {
        u64 total = 0;
        if (top_p < 1.0f) {
            u64 mine = 0;
            for (int i = threadIdx.x; i < n; i += kThreads) mine += fixed_weight(logit_of(s.list[i]), scale, s.powers);
            n = within(n, part_of(sum_block(mine), top_p, true));
        }
        // by index, with the logit in the low half: the lowest index is the largest number
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const u64 p = s.list[i];
            s.list[i] = p << 32 | p >> 32;
        }
        sort(n);
        constexpr int kEach = kList / kThreads;
        const int i0 = threadIdx.x * kEach;
        auto weight = [&](int i) { return fixed_weight(logit_of(s.list[i] << 32), scale, s.powers); };
        u64 mine = 0;
        for (int i = i0; i < min(n, i0 + kEach); ++i) mine += weight(i);
        u64 before = scan_block(mine, s.sums, total);
        const u64 want = part_of(total, u, false);
        for (int i = i0; i < min(n, i0 + kEach); ++i) {
            const u64 w = weight(i);
            if (before <= want && want < before + w) *token = static_cast<int>(~static_cast<uint32_t>(s.list[i] >> 32));
            before += w;
        }
    }

    // The token in which u of the weight of the places >= cut is passed.
    __device__ void draw(float u, int32_t* token) {
        u64 mine = 0;
        row.each([&](int g, int i, const float (&v)[Row<E>::kV]) {
            u64 sum = 0;
            bool some = false;
#pragma unroll
            for (int e = 0; e < Row<E>::kV; ++e) some |= place_of(v[e], i + e) >= cut;
            if (__any_sync(0xFFFFFFFFu, some)) {
#pragma unroll
                for (int e = 0; e < Row<E>::kV; ++e)
                    if (place_of(v[e], i + e) >= cut) sum += fixed_weight(v[e], scale, s.powers);
                sum = add_across(sum);
            }
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
        const int each = (row.groups + kThreads - 1) / kThreads, g0 = threadIdx.x * each;
        u64 sum = 0, whole;
        for (int g = g0; g < min(row.groups, g0 + each); ++g) sum += s.groups[g];
        u64 at = before + scan_block(sum, s.sums, whole);
        for (int g = g0; g < min(row.groups, g0 + each); ++g) {
            if (at <= want && want < at + s.groups[g]) {
                s.found[0] = g;
                s.answer = at;
            }
            at += s.groups[g];
        }
        __syncthreads();
        if (threadIdx.x >= 32) return;
        const int g = s.found[0], i = row.index(g);
        const uint4 raw = row.raw(g);
        const E* v = reinterpret_cast<const E*>(&raw);
        u64 w[Row<E>::kV], lane_sum = 0;
#pragma unroll
        for (int e = 0; e < Row<E>::kV; ++e) {
            const float x = logit(v[e]);
            w[e] = place_of(x, i + e) >= cut ? fixed_weight(x, scale, s.powers) : 0;
            lane_sum += w[e];
        }
        u64 x = lane_sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if ((threadIdx.x & 31) >= o) x += y;
        }
        u64 past = s.answer + x - lane_sum;
#pragma unroll
        for (int e = 0; e < Row<E>::kV; ++e) {
            if (past <= want && want < past + w[e]) *token = i + e;
            past += w[e];
        }
    }

    // The cut at top_p of the weight of the places >= cut, given their counts a bin. Guesses where the border is from the
    // counts, and takes the exact weight above, in the kWindow bins there, and below; where the guess missed, the next
    // one starts from what is known exactly.
    __device__ u64 nucleus(float top_p) {
        auto guess = [&](int b) {
            const int n = -(b * kBinSteps + kBinSteps / 2), down = -(n >> 8);
            return s.all[b] * max((s.powers[n & (kSteps - 1)] + (1ull << (down - 1))) >> down, 1ull);
        };
        u64 sum = 0, whole;
        for (int b = threadIdx.x; b < kBins; b += kThreads) sum += guess(b);
        scan_block(sum, s.sums, whole);
        int64_t want = static_cast<int64_t>(part_of(whole, top_p, true)), known = 0;  // known: exact less guessed weight before a window
        int least = 0, most = kBins;                                                  // the border's bin is one of least .. most - 1
        while (true) {
            int bin;
            u64 skipped;
            reach<u64>(guess, static_cast<u64>(max(want - known, static_cast<int64_t>(1))), s.sums, bin, skipped);
            const int from = max(least, min(bin - kWindow / 2, most - kWindow));
            for (int i = threadIdx.x; i < kWindow; i += kThreads) {
                s.window[i] = 0;
                s.window_count[i] = 0;
            }
            __syncthreads();
            u64 above = 0, below = 0;
            row.each([&](int, int i, const float (&v)[Row<E>::kV]) {
#pragma unroll
                for (int e = 0; e < Row<E>::kV; ++e) {
                    if (place_of(v[e], i + e) < cut) continue;
                    const int b = bin_of(v[e]);
                    if (b >= kBins) continue;
                    const u64 w = fixed_weight(v[e], scale, s.powers);
                    if (b < from) {
                        above += w;
                    } else if (b >= from + kWindow) {
                        below += w;
                    } else {
                        atomicAdd(&s.window[b - from], w);
                        atomicAdd(&s.window_count[b - from], 1u);
                    }
                }
            });
            above = sum_block(above);
            below = sum_block(below);
            u64 (*box)[kMaxCtas] = tell(above, below);
            above = below = 0;
            for (uint32_t r = 0; r < ctas; ++r) {
                above += box[0][r];
                below += box[1][r];
            }
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
            const u64 total = above + inside_all + below, target = max(part_of(total, top_p, true), 1ull);
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
            want = static_cast<int64_t>(target);
        }
    }
};

__device__ __forceinline__ float setting(const float* p, float all, int64_t r) { return p != nullptr ? __ldg(p + r) : all; }

template <typename E>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleCall c) {
    extern __shared__ uint8_t smem[];
    Shared& s = *reinterpret_cast<Shared*>(smem);
    const uint32_t rank = cluster_ctarank();
    uint32_t ctas;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    const int64_t r = blockIdx.x / ctas;
    Sampler<E> w(c, s, static_cast<const E*>(c.x) + r * c.row_stride, rank, ctas);
    const float temperature = setting(c.temperature, c.temperature_all, r), min_p = setting(c.min_p, c.min_p_all, r);
    const float top_p = setting(c.top_p, c.top_p_all, r), u_given = __ldg(c.u + r);
    const int top_k = c.top_k != nullptr ? __ldg(c.top_k + r) : c.top_k_all;
    const float u = u_given > 0.0f ? fminf(u_given, 0.99999994f) : 0.0f;
    const bool greedy = !(temperature > 0.0f);
    for (int i = threadIdx.x; i < kSteps; i += kThreads) s.powers[i] = kPowers.v[i];
    if (threadIdx.x == 0) s.listed[0] = s.listed[1] = 0;
    if (threadIdx.x == 32 && !greedy) {  // in 64 bits, once, while the others read
        const double f = 512.0 * 1.4426950408889634074 / static_cast<double>(temperature);
        s.hi = static_cast<float>(f);
        s.lo = isinf(s.hi) ? 0.0f : static_cast<float>(f - static_cast<double>(s.hi));
    }
    if (threadIdx.x == 64 && !greedy && min_p > 0.0f && min_p < 1.0f) s.log_min_p = static_cast<double>(temperature) * log(static_cast<double>(min_p));
    cluster_sync();
    const u64 top = w.largest();
    if (top == 0) {
        if (rank == 0 && threadIdx.x == 0) c.tokens[r] = -1;
        return;
    }
    if (greedy) {
        if (rank == 0 && threadIdx.x == 0) c.tokens[r] = index_of(top);
        return;
    }
    w.scale = Scale{logit_of(top), s.hi, s.lo};
    w.cut = static_cast<u64>(key_of(kNone) + 1) << 32;  // anything above -inf
    if (min_p >= 1.0f) {
        w.cut = top >> 32 << 32;
    } else if (min_p > 0.0f) {
        const double least = static_cast<double>(w.scale.top) + s.log_min_p;
        float x = static_cast<float>(least);
        if (static_cast<double>(x) < least) x = nextafterf(x, INFINITY);  // the least float that is not below
        w.cut = max(w.cut, static_cast<u64>(key_of(x + 0.0f)) << 32);
    }
    const bool by_count = top_k > 0 && top_k < c.vocab, by_mass = top_p < 1.0f;
    if (by_count || by_mass) w.count();
    if (by_count) {
        int bin;
        uint32_t before;
        w.template reach<uint32_t>([&](int b) { return s.all[b]; }, static_cast<uint32_t>(top_k), reinterpret_cast<uint32_t*>(s.sums), bin, before);
        const uint32_t to = bin < kBins ? before + s.all[bin] : before;  // places to the end of that bin
        if (to <= kList) {
            w.gather(0, [&](float x, u64) { return w.bin_of(x) <= min(bin, kBins - 1); });
            if (rank == 0) {
                w.sort(static_cast<int>(to));
                w.draw_list(min(static_cast<int>(to), top_k), top_p, u, c.tokens + r);
            }
            return;
        }
        if (bin < kBins) {
            const uint32_t n = s.all[bin];
            w.cut = w.template inside<false>(0, bin, n, top_k - before);
            if (by_mass) {  // the counts without what has been cut off
                __syncthreads();
                for (int b = bin + threadIdx.x; b < kBins; b += kThreads) s.all[b] = b == bin ? top_k - before : 0;
                __syncthreads();
            }
        }
    }
    if (by_mass) w.cut = w.nucleus(fmaxf(top_p, 0.0f));
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
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(Shared)))) != cudaSuccess) return e;
        attr_gen[dev] = g_generation;
    }
    // CTAs of a row: as many as give the GPU two CTAs an SM, with at least 2048 logits each
    int ctas = 1;
    while (ctas < kMaxCtas && c.rows * ctas * 2 <= 2 * sm_count && c.vocab > 2048 * ctas) ctas *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(c.rows * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
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
