// Drawing a token from each row of logits: temperature, the top_k largest, a
// least weight min_p, the top_p of the mass, and one given number u a row.
//
//     w_i = exp((x_i - max) / T) = 2^t_i,  token = first kept i with sum_{j <= i, kept} w_j > u sum_{kept} w_j
//
// The answer is a whole number, and a border (of the mass, or of u) lies between
// two tokens of a vocabulary of 10^5, whose shares are about 10^-5 of the sum or
// less: sums in 32 bits, off by 10^-7 and by how the row was split, would give
// another token in one row of some hundreds. So weights are integers, of 2^-42 of the
// row's largest, good to 2^-37 (weigh), and sums of them are exact
// in 64 bits: the same whatever the order, the split and the rest of the batch.
//
// Order: a token's rank is that of its 64-bit `place`: the logit's bits as an
// ordered 32-bit integer, then the index inverted, so equal logits rank by index
// and what a row keeps is every place >= one cut.
//
// A cluster of CTAs takes a row, each CTA a stretch of it, which the first pass leaves in
// shared memory: the logits are read from HBM once. The passes, of which a row makes
// those its settings ask for:
//   1  the largest logit (a greedy row ends here), and each thread's largest;
//   2  where top_p needs it, the exact weight of all;
//   3  a threshold from the threads' largest: as many of them are above it as top_k wants, or as much
//      weight as top_p does, so what the row keeps is above it, and not much else;
//   4  the tokens above it, brought together in order where they are at most kList: the first
//      CTA cuts and draws. Few rows go on:
//   5  a count in each of kBins bins of t, 1/32 wide: the bin with the k-th, and a guess at the bin in which
//      the weight reaches top_p; the exact weight above a window of bins around the guess, group by group of
//      32 lanes' pieces;
//   6  the tokens of the border's bins, brought together: the cut, and their kept weight to their groups;
//   7  the group, lane and token in which u of the kept weight is passed.
//
// What bounds it is the chain of these steps, between which the CTAs meet, and in rows without a cut the 23 operations that a
// weight takes, not the bytes: of 256 rows, warps issue in half of the cycles. Measured on a GB300, in a graph: one row of 32000 fp16 logits, top_p 0.9:
// 12.8 us; 64 rows of 131071 bf16: greedy 6.3, no cut 21, top_k 50 17, top_p 0.9 78, settings mixed 42; 256 rows of 131072 fp32,
// top_p 0.9: 220 (the bytes take 20).
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
constexpr int kList = 2047;                  // tokens in a list, at most: that many weights' upper halves add up in 32 bits
constexpr int kSub = 1024;                   // parts of a bin that holds more
constexpr int kSome = kThreads;              // tokens of a bin that are ranked by comparing each with each
constexpr int kGuess = 1280;                 // tokens around a guessed bin that are brought together with its own, half on either side
constexpr int kMostGroups = (1 << 18) / 128 / kMaxCtas + 2;  // of a CTA
constexpr float kNone = -INFINITY;
constexpr float kTiny = 0x1p-147f;            // a few of the least floats
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
        p.v[j].y = j > 0 ? static_cast<float>(static_cast<int64_t>(x - hi)) / static_cast<float>(1ull << 62) : 0x1p-45f;  // not 0: its exponent is moved
        x = product_2_62(x, step);
    }
    return p;
}
__device__ const Powers kPowers = make_powers();

// What a row's logits are weighed with.
struct Scale {
    float top;          // the largest logit
    float half, minus;  // where not near: a half, times a power of two where 2 / T is no good float, and as much of -top
    float hi, lo;       // 1 / T; where not near 1 / (half T)
    float round;        // kRound; near: less the steps of the largest, so that no logit is above kRound
    float none;         // a logit whose weight is none, and so are those below it; kNone: not known
    float t;            // T
    bool near;          // logits are at most some hundred T: they are weighed without the largest's being taken off first
    bool flat;          // the largest is infinite: what is kept weighs the same
};

constexpr double kLn = 0.693147180559945309417 / kSteps;
constexpr float kLnHi = static_cast<float>(kLn), kLnLo = static_cast<float>(kLn - static_cast<double>(kLnHi));
constexpr float kPerLn = static_cast<float>(1.0 / kLn);
constexpr float kRound = 12582912.0f;                    // 1.5 * 2^23: a sum with it is a whole number
constexpr int kRoundBits = 0x4B400000;
constexpr float kHigh = 12.0f, kLow = 1.5f / 524288.0f;  // sums with them are multiples of 2^-20 and 2^-42; with kLow of what is below 2^-20
constexpr int kHighBits = 0x41400000, kLowBits = 0x36400000;

// ln w of a logit, or what is taken off it in the end, as p + q and some, and 256 log2 w to the nearest integer, above kRoundBits.
__device__ __forceinline__ float differ(float x, const Scale& c) { return __fmaf_rn(c.half, x, c.minus); }
__device__ __forceinline__ int step_bits(float p, const Scale& c) { return __float_as_int(__fmaf_rn(p, kPerLn, c.round)); }

// The weight of a logit, in two parts added to `high` and `low` (units(), below): w = (high part) 2^-20 + (low part) 2^-42. A logit whose step is below
// `least` has none. The logit is at most c.top and not so far below it that w is no ordinary float. w is right to 2^-37 of itself, before its rounding to 2^-42. x / T = p + q
// with 1 / T as hi + lo, good to 2^-46 (an error that grows as x does is the same power of every weight: of their ratios, 2^-46 of the difference's);
// m = round(256 / ln(2) p); what is left after m ln(2) / 256 is u (exactly: it has 24 bits) and some more, f, at most 2^-15; and with U = u + f,
// at most 2^-9.4,
//     exp(x / T) = 2^(m / 256) (1 + u + (f + U^2 / 2 + U^3 / 6)),
// U^4 / 24 being 2^-42; 2^(m / 256) is a table's entry th + tl, whose exponents are moved: by m less the largest's, rounded up, so weights are
// relative to something up to 2^(1 / 256) larger than the largest's, for all alike. The weight is s + r, r up to 2^-15 of s: the high part is taken of their sum, so
// that the low one is within 2^-20. That takes 23 operations on the floating point pipe, which bound
// the passes that weigh all logits (two at a time, in packed form, they take as long): 256 rows of 131072 fp32, no cut, 106 us. With the largest taken
// off first it is 31 (with one operation less each: 105 and 120 us). Where logits are far from zero by T (`near` is not set) it is taken off: the difference of their halves, which stays finite,
// as d + e exactly.
template <bool kNear>
__device__ __forceinline__ void weigh(float x, const Scale& c, const float2* powers, int& high, int& low, int least = INT_MIN) {
    float d = x, e = 0.0f;
    if (!kNear && !c.near) {
        d = differ(x, c);
        const float a = c.half * x, bb = __fsub_rn(d, a);
        e = __fadd_rn(__fsub_rn(a, __fsub_rn(d, bb)), __fsub_rn(c.minus, bb));
    }
    const float p = __fmul_rn(d, c.hi);
    float q = __fmaf_rn(d, c.lo, __fmaf_rn(d, c.hi, -p));
    if (!kNear) q = __fmaf_rn(e, c.hi, q);
    const int bits = step_bits(p, c);
    const float m = __fsub_rn(__int_as_float(bits), c.round);
    const int moved = bits >= least ? bits : kRoundBits - 60 * kSteps;  // 2^-60
    const float2 t = powers[moved & (kSteps - 1)];
    const int by = (moved & ~(kSteps - 1)) << 15;
    const float th = __int_as_float(__float_as_int(t.x) + by), tl = __int_as_float(__float_as_int(t.y) + by);
    const float u = __fmaf_rn(m, -kLnHi, p), f = __fmaf_rn(m, -kLnLo, q), g = __fadd_rn(u, f);
    const float v = __fmaf_rn(__fmul_rn(g, g), __fmaf_rn(g, 1.0f / 6.0f, 0.5f), f);
    const float s = __fmaf_rn(th, u, th);
    const float r = __fadd_rn(__fmaf_rn(th, u, __fsub_rn(th, s)), __fmaf_rn(th, v, __fmaf_rn(tl, u, tl)));
    const float h = __fadd_rn(__fadd_rn(s, r), kHigh);
    const float l = __fadd_rn(__fadd_rn(__fsub_rn(s, __fsub_rn(h, kHigh)), r), kLow);
    high += __float_as_int(h) - kHighBits;
    low += __float_as_int(l) - kLowBits;
}

// Sums of weights' parts, in units of 2^-42.
__device__ __forceinline__ u64 units(int high, int low) { return static_cast<u64>((static_cast<int64_t>(high) << 22) + low); }

__device__ __forceinline__ u64 weight_of(float x, const Scale& c, const float2* powers) {
    if (c.flat) return 1ull << kUnit;
    if (c.near) x = fmaxf(x, c.none);
    else if (!(__fmul_rn(differ(x, c), c.hi) > -32.0f)) return 0;  // and where c.none says nothing
    int high = 0, low = 0;
    weigh<false>(x, c, powers, high, low);
    return units(high, low);
}

// A step's bin, and a logit's: it falls as the logit does, so bins are in order.
__device__ __forceinline__ int bin_of_bits(int bits) { return min(static_cast<int>(static_cast<uint32_t>(kRoundBits - bits) / kBinSteps), kBins - 1); }
__device__ __forceinline__ int bin_of(float x, const Scale& c) {
    return c.flat ? 0 : bin_of_bits(step_bits(__fmul_rn(differ(x, c), c.hi), c));
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
    int each_cta;         // of a CTA
    __device__ Row(const E* row, uint4* smem, int n, uint32_t rank, uint32_t ctas) : x(row), held(smem), vocab(n) {
        shift = static_cast<int>(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(E));
        const int all = ((n + shift + kV - 1) / kV + 31) / 32;
        each_cta = (all + ctas - 1) / ctas;
        group0 = min(all, static_cast<int>(rank) * each_cta);
        groups = min(all, group0 + each_cta) - group0;
    }
    __device__ int index(int group) const { return ((group0 + group) * 32 + (threadIdx.x & 31)) * kV - shift; }
    __device__ __forceinline__ static void open(const uint4& u, float (&v)[kV]) {
        const E* e = reinterpret_cast<const E*>(&u);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            if constexpr (std::is_same<E, float>::value) v[i] = e[i];
            else v[i] = to_float(e[i]);
        }
    }
    // The largest of a piece.
    __device__ __forceinline__ static float most(const uint4& u) {
        if constexpr (std::is_same<E, float>::value) {
            return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
        } else {
            using E2 = std::conditional_t<std::is_same<E, __half>::value, __half2, __nv_bfloat162>;
            E2 p[4];
            memcpy(p, &u, 16);
            const E2 x = __hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3]));
            return to_float(__hmax(x.x, x.y));
        }
    }
    // The first pass: reads, keeps, f(the piece).
    template <typename F>
    __device__ __forceinline__ void load(F f) {
        constexpr int kAhead = 4;
        constexpr uint32_t kNones = std::is_same<E, float>::value ? 0xFF800000u : std::is_same<E, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
        for (int g = threadIdx.x / 32; g < groups; g += kWarps * kAhead) {
            uint4 u[kAhead];
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const int i = index(g + a * kWarps);
                u[a] = make_uint4(kNones, kNones, kNones, kNones);
                if (g + a * kWarps < groups && i >= 0 && i + kV <= vocab) u[a] = __ldg(reinterpret_cast<const uint4*>(x + i));
            }
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                if (g + a * kWarps >= groups) break;
                held[(g + a * kWarps) * 32 + (threadIdx.x & 31)] = u[a];
                f(u[a]);
            }
        }
        edge(0, f);
        edge((vocab - 1 + shift) / kV, f);
    }
    // Piece q, where it reaches beyond the row.
    template <typename F>
    __device__ __forceinline__ void edge(int q, F f) {
        const int g = q / 32 - group0, i = q * kV - shift;
        if (g < 0 || g >= groups || static_cast<int>(threadIdx.x) != g % kWarps * 32 + q % 32 || (i >= 0 && i + kV <= vocab)) return;
        E v[kV];
        uint4 u = held[g * 32 + (threadIdx.x & 31)];
        memcpy(v, &u, 16);
#pragma unroll
        for (int e = 0; e < kV; ++e)
            if (i + e >= 0 && i + e < vocab) v[e] = x[i + e];
        memcpy(&u, v, 16);
        held[g * 32 + (threadIdx.x & 31)] = u;
        f(u);
    }
    // Further passes, over groups in which some logit is at least `least`: f(group, index of the first, the kV logits), whole warps.
    template <typename F>
    __device__ __forceinline__ void each(float least, F f) const {
        for (int g = threadIdx.x / 32; g < groups; g += kWarps) {
            const uint4 u = held[g * 32 + (threadIdx.x & 31)];
            if (!__any_sync(0xFFFFFFFFu, !(most(u) < least))) continue;
            float v[kV];
            open(u, v);
            f(g, index(g), v);
        }
    }
};

struct Shared {
    float2 powers[kSteps];
    u64 list[kList + 1];           // of the first CTA; parts' masses
    u64 groups[kMostGroups];   // weights
    int2 places[kMostGroups];  // how many go to the list, and where
    union {
        struct {
            uint32_t bins[kBins], all[kBins];
        };
        struct {
            uint32_t low[kSub], high[kSub];  // weights of a list's parts
        };
    };
    u64 some[kSome], some_weight[kSome];
    u64 box[2][2][kMaxCtas];   // what the CTAs tell each other
    u64 sums[kWarps];
    u64 answer;
    int found[2], window[2];
    uint32_t listed;
    float2 log_min_p;          // T ln(min_p), where T is large half of it, in two parts
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

// The weight that what comes before a token must not reach.
__device__ __forceinline__ u64 target_of(u64 total, float top_p) { return max(part_of(total, fmaxf(top_p, 0.0f), true), 1ull); }

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
    float best = kNone;  // the thread's largest
    bool easy = false;   // all that has a weight is kept

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
        return scale.flat ? scale.top : scale.top - (b + 2) * (kBinSteps * kLnHi * 1.0001f) * scale.t - 1e-5f * fabsf(scale.top) - kTiny;
    }
    // A logit above which there is none of bin b.
    __device__ __forceinline__ float highest_of(int b) const {
        const float half = (b - 1) * (0.5f * kBinSteps * kLnHi * 0.9999f) * scale.t;  // by halves: the whole way may pass what a float holds
        return scale.flat ? scale.top : scale.top - half - half + 1e-5f * fabsf(scale.top) + kTiny;
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

    // The place of the largest logit, -inf's where there is none above: of the first one if `first`, else of any index.
    __device__ u64 largest(bool first) {
        row.load([&](const uint4& u) { best = fmaxf(best, Row<E>::most(u)); });
        const uint32_t own = key_of(best);
        uint32_t k = __reduce_max_sync(0xFFFFFFFFu, own);
        u64 p = static_cast<u64>(k) << 32;
        if (first) {
            int at = INT_MAX;
            row.each(logit_of(p), [&](int, int i, const float (&v)[kV]) {
#pragma unroll
                for (int e = kV - 1; e >= 0; --e)
                    if (v[e] == logit_of(p)) at = min(at, i + e);
            });
            p |= static_cast<uint32_t>(~__reduce_min_sync(0xFFFFFFFFu, at));
        }
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

    // Weights of a piece's kept logits, added up (with kGroup over the warp); with kPart, of those in bins before `first`.
    template <bool kPart, bool kGroup>
    __device__ __forceinline__ u64 weigh_piece(int i, const float (&v)[kV], int first = 0) {
        if (!scale.near) {
            u64 sum = 0;
#pragma unroll 1
            for (int e = 0; e < kV; ++e) {
                float y = v[0];
#pragma unroll
                for (int k = 1; k < kV; ++k) y = k == e ? v[k] : y;
                if (kept(y, i + e) && (!kPart || bin_of(y, scale) < first)) sum += weight_of(y, scale, s.powers);
            }
            return kGroup ? add_across(sum) : sum;
        }
        float x[kV];
        if (easy) {  // below the cut there is no weight
#pragma unroll
            for (int e = 0; e < kV; ++e) x[e] = fmaxf(v[e], scale.none);
        } else {
#pragma unroll
            for (int e = 0; e < kV; ++e) x[e] = kept(v[e], i + e) ? v[e] : scale.none;
        }
        int high = 0, low = 0;
#pragma unroll
        for (int e = 0; e < kV; ++e) {
            weigh<true>(x[e], scale, s.powers, high, low, kPart ? kRoundBits - first * kBinSteps + 1 : INT_MIN);
        }
        if (kGroup) {  // a group's parts fit 32 bits: at most 2^8 of 2^20
            high = __reduce_add_sync(0xFFFFFFFFu, high);
            low = __reduce_add_sync(0xFFFFFFFFu, low);
        }
        return units(high, low);
    }

    // Counts of what is kept a bin, of all CTAs, in the first CTA's s.all.
    __device__ void count() {
        for (int b = threadIdx.x; b < kBins; b += kThreads) s.bins[b] = s.all[b] = 0;
        cluster_sync();
        row.each(cut_x, [&](int, int i, const float (&v)[kV]) {
            // many equal logits: one addition a warp
            const float first = __shfl_sync(0xFFFFFFFFu, v[0], 0);
            if (__all_sync(0xFFFFFFFFu, v[0] == first && v[0] > cut_x)) {
                bool same = true;
#pragma unroll
                for (int e = 1; e < kV; ++e) same &= v[e] == first;
                if (__all_sync(0xFFFFFFFFu, same)) {
                    if ((threadIdx.x & 31) == 0) atomicAdd(&s.bins[bin_of(first, scale)], 32u * kV);
                    return;
                }
            }
            if (cut_i == ~0u) {  // of logits as large as the cut's all are kept
#pragma unroll
                for (int e = 0; e < kV; ++e)
                    if (v[e] >= cut_x) atomicAdd(&s.bins[bin_of(v[e], scale)], 1u);
                return;
            }
#pragma unroll
            for (int e = 0; e < kV; ++e)
                if (kept(v[e], i + e)) atomicAdd(&s.bins[bin_of(v[e], scale)], 1u);
        });
        __syncthreads();
        const uint32_t to = mapa_shared(smem_u32(s.all), 0);
#pragma unroll
        for (int b = threadIdx.x; b < kBins; b += kThreads)
            if (s.bins[b] != 0) asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(to + 4 * b), "r"(s.bins[b]) : "memory");
        cluster_sync();
    }
    // Counts of the threads' largest a bin, of all CTAs, in the first CTA's s.all, which is clear.
    __device__ void count_best() {
        if (best >= cut_x)
            asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(&s.all[bin_of(best, scale)]), 0)), "r"(1u) : "memory");
        cluster_sync();
    }
    // Among numbers v(b): the first bin up to which they reach `want`, and the sum before it; kBins and the sum of all where they do not.
    template <typename V, typename F>
    __device__ void reach(F v, V want, V* sums, int& bin, V& before) {
        constexpr int kEach = (kBins + kThreads - 1) / kThreads;
        V x[kEach], mine = 0, total;
        const int b0 = threadIdx.x * kEach;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            x[i] = b0 + i < kBins ? v(b0 + i) : 0;
            mine += x[i];
        }
        V past = scan_block(mine, sums, total);
        if (past < want && past + mine >= want) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                if (past < want && past + x[i] >= want) {
                    s.found[0] = b0 + i;
                    s.answer = past;
                }
                past += x[i];
            }
        }
        __syncthreads();
        const bool reached = total >= want;
        bin = reached ? s.found[0] : kBins;
        before = reached ? static_cast<V>(s.answer) : total;
    }

    // Brings the kept places of logits of at least `least` for which f holds together in the first CTA's list, in the order of the row, if they are
    // at most kList. Afterwards the cluster has met. Returns how many they are.
    template <typename F>
    __device__ int gather(float least, F f) {
        const float from = fmaxf(least, cut_x);
        const int lane = threadIdx.x & 31;
        for (int g = threadIdx.x / 32 + lane * kWarps; g < row.groups; g += kThreads) s.places[g] = make_int2(0, 0);
        __syncwarp();
        row.each(from, [&](int g, int i, const float (&v)[kV]) {
            int mine = 0;
#pragma unroll
            for (int e = 0; e < kV; ++e) mine += f(v[e], i + e) && kept(v[e], i + e);
            mine = __reduce_add_sync(0xFFFFFFFFu, mine);
            if (lane == 0) s.places[g].x = mine;
        });
        __syncthreads();
        static_assert(kMostGroups <= kThreads, "a group a thread");
        const int mine = threadIdx.x < row.groups ? s.places[threadIdx.x].x : 0;
        int all, before = scan_block(mine, reinterpret_cast<int*>(s.sums), all), total = 0;
        u64 (*box)[kMaxCtas] = tell(all, 0);
        for (uint32_t r = 0; r < ctas; ++r) {
            if (r < rank) before += static_cast<int>(box[0][r]);
            total += static_cast<int>(box[0][r]);
        }
        if (total > kList) return total;
        if (threadIdx.x < row.groups) s.places[threadIdx.x].y = before;
        __syncthreads();
        const uint32_t list = mapa_shared(smem_u32(s.list), 0);
        for (int g = threadIdx.x / 32; g < row.groups; g += kWarps) {
            if (s.places[g].x == 0) continue;
            float v[kV];
            Row<E>::open(row.held[g * 32 + lane], v);
            const int i = row.index(g);
            uint32_t in = 0;
#pragma unroll
            for (int e = 0; e < kV; ++e)
                if (f(v[e], i + e) && kept(v[e], i + e)) in |= 1u << e;
            int x = __popc(in);
            const int own = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
                if (lane >= o) x += y;
            }
            int at = s.places[g].y + x - own;
#pragma unroll
            for (int e = 0; e < kV; ++e)
                if (in >> e & 1) {
                    asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(list + 8 * at), "l"(place_of(v[e], i + e)) : "memory");
                    ++at;
                }
        }
        cluster_sync();
        return total;
    }

    // Sorts n numbers of the list, the largest first (first CTA): in registers, kEach a lane, one after another, and through shared memory
    // only between warps.
    template <int kEach>
    __device__ void sort_by(int n) {
        int size = 32 * kEach;
        while (size < n) size *= 2;
        const int i0 = threadIdx.x * kEach;
        u64 x[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) x[e] = i0 + e < n ? s.list[i0 + e] : 0;
        const bool some = threadIdx.x / 32 * 32 * kEach < size;  // the warp takes part
        for (int k = 2; k <= size; k *= 2)
            for (int j = k / 2; j > 0; j /= 2) {
                if (j >= 32 * kEach) {
                    __syncthreads();
                    if (some) {
#pragma unroll
                        for (int e = 0; e < kEach; ++e) s.list[i0 + e] = x[e];
                    }
                    __syncthreads();
                    if (some) {
#pragma unroll
                        for (int e = 0; e < kEach; ++e) {
                            const u64 y = s.list[(i0 + e) ^ j];
                            const bool larger = ((i0 & j) == 0) == ((i0 & k) == 0);  // the larger one stays here
                            x[e] = larger == (x[e] > y) ? x[e] : y;
                        }
                    }
                } else if (j >= kEach) {
                    if (some) {
#pragma unroll
                        for (int e = 0; e < kEach; ++e) {
                            const u64 y = __shfl_xor_sync(0xFFFFFFFFu, x[e], j / kEach);
                            const bool larger = ((i0 & j) == 0) == ((i0 & k) == 0);
                            x[e] = larger == (x[e] > y) ? x[e] : y;
                        }
                    }
                } else if (some) {
#pragma unroll
                    for (int e = 0; e < kEach; ++e)
#pragma unroll
                        for (int d = 1; d < kEach; d *= 2)
                            if (d == j && (e & d) == 0) {
                                const bool down = ((i0 + e) & k) == 0;
                                const u64 a = x[e], b = x[e + d];
                                if (down == (a < b)) {
                                    x[e] = b;
                                    x[e + d] = a;
                                }
                            }
                }
            }
        __syncthreads();
        if (some) {
#pragma unroll
            for (int e = 0; e < kEach; ++e) s.list[i0 + e] = x[e];
        }
        __syncthreads();
    }
    __device__ void sort(int n) {
        if (n <= 32) sort_by<1>(n);
        else if (n <= 64) sort_by<2>(n);
        else sort_by<4>(n);
    }

    // The weights of n places of the first CTA's list, one thread's after another's: f(i, weight, weight before) for each. Returns the weight of
    // all n.
    template <typename G, typename F>
    __device__ __forceinline__ u64 weigh_list(int n, G logit, F f) {
        constexpr int kEach = (kList + 1) / kThreads;
        const int each = (n + kThreads - 1) / kThreads, i0 = threadIdx.x * each;
        u64 w[kEach], mine = 0, total;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            w[i] = i < each && i0 + i < n ? weight_of(logit(s.list[i0 + i]), scale, s.powers) : 0;
            mine += w[i];
        }
        u64 before = scan_block(mine, s.sums, total);
        f(total);  // whole block
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (i < each && i0 + i < n) f(i0 + i, w[i], before);
            before += w[i];
        }
        return total;
    }
    // Of the first CTA's sorted list of n places: how many come first that have less than target(weight of all) before them, at
    // least one; 0 where all have less than that.
    template <typename T>
    __device__ int within(int n, T target) {
        struct Find {
            Shared& s;
            T target;
            u64 want;
            __device__ void operator()(u64 total) {
                want = target(total);
                if (threadIdx.x == 0) s.found[1] = 1;
                __syncthreads();
            }
            __device__ void operator()(int i, u64, u64 before) {
                if (before < want) atomicMax(&s.found[1], i + 1);
            }
        } find{s, target, 0};
        const u64 total = weigh_list(n, [](u64 p) { return logit_of(p); }, [&](auto... x) { find(x...); });
        __syncthreads();
        return total < find.want ? 0 : s.found[1];
    }

    // The cut inside bin b, which holds n places >= cut: the target-th of them, or with kMass the last one that has less than
    // `target` of the bin's weight before it.
    template <bool kMass>
    __device__ u64 inside(int b, uint32_t n, u64 target) {
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
                s.some[0] = ~0ull;
                s.some[1] = 0;
            }
            __syncthreads();
            if ((threadIdx.x & 31) == 0) {
                atomicMin(&s.some[0], least);
                atomicMax(&s.some[1], most);
            }
            __syncthreads();
            u64 (*box)[kMaxCtas] = tell(s.some[0], s.some[1]);
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
        gather(from, [&](float x, int i) { return bin_of(x, scale) == b && place_of(x, i) >= low && place_of(x, i) <= high; });
        u64 found = 0;
        if (rank == 0) {
            u64 p[kOwn], w[kOwn];
            read_list(static_cast<int>(n), p, w);
            if (!kMass) {
#pragma unroll
                for (int i = 0; i < kOwn; ++i) w[i] = p[i] != 0;
            }
            found = cut_of<kMass>(static_cast<int>(n), p, w, target);
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
        __syncthreads();
        sort(n);
        struct Find {
            Shared& s;
            float u;
            int32_t* token;
            u64 want;
            __device__ void operator()(u64 total) { want = part_of(total, u, false); }
            __device__ void operator()(int i, u64 w, u64 before) {
                if (before <= want && want < before + w) *token = index_of(s.list[i] >> 32);
            }
        } find{s, u, token, 0};
        weigh_list(n, [](u64 p) { return logit_of(p << 32); }, [&](auto... x) { find(x...); });
    }

    // The cut of the first CTA's list: the target-th largest place, or with kMass the last one that has less than `target` of weight before it.
    // p, w: this thread's places and weights, 0 for those that do not count. By their part of the range of all, then each with each
    // in the border's part. 0: more than kSome are there; 1: there is less than the target.
    template <bool kMass, int kEach>
    __device__ u64 cut_list(const u64 (&p)[kEach], const u64 (&w)[kEach], u64 target) {
        u64 least = ~0ull, most = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (w[i] != 0) {
                least = min(least, p[i]);
                most = max(most, p[i]);
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            least = min(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
            most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
        }
        for (int b = threadIdx.x; b < kSub; b += kThreads) s.low[b] = s.high[b] = 0;
        __syncthreads();
        if ((threadIdx.x & 31) == 0) {
            s.sums[threadIdx.x >> 5] = least;
            s.some[threadIdx.x >> 5] = most;
        }
        if (threadIdx.x == 0) s.listed = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            least = min(least, s.sums[i]);
            most = max(most, s.some[i]);
        }
        if (least > most) return 1;
        const int shift = max(0, 64 - __clzll(most - least) - 10);
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (w[i] != 0) {
                const int part = static_cast<int>((most - p[i]) >> shift);
                if (kMass) {  // in two parts, whose sums fit 32 bits: additions in 64 bits are loops, which equal logits meet in
                    atomicAdd(&s.low[part], static_cast<uint32_t>(w[i]) & 0x1FFFFFu);
                    atomicAdd(&s.high[part], static_cast<uint32_t>(w[i] >> 21));
                } else {
                    atomicAdd(&s.low[part], 1u);
                }
            }
        __syncthreads();
        int part;
        u64 before;
        reach<u64>([&](int b) { return b < kSub ? (static_cast<u64>(s.high[b]) << 21) + s.low[b] : 0; }, target, s.sums, part, before);
        if (part == kBins) return 1;
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (w[i] != 0 && static_cast<int>((most - p[i]) >> shift) == part) {
                const uint32_t at = atomicAdd(&s.listed, 1u);
                if (at < kSome) {
                    s.some[at] = p[i];
                    s.some_weight[at] = kMass ? w[i] : 1;
                }
            }
        __syncthreads();
        const int n = static_cast<int>(s.listed);
        if (n > kSome) return 0;
        if (threadIdx.x < n) {
            const u64 own = s.some[threadIdx.x];
            u64 above = before;
            for (int j = 0; j < n; ++j)
                if (s.some[j] > own) above += s.some_weight[j];
            if (above < target && above + s.some_weight[threadIdx.x] >= target) s.answer = own;
        }
        __syncthreads();
        const u64 found = s.answer;
        __syncthreads();
        return found;
    }
    // The first CTA's list of n: a thread's places and weights, one thread's after another's.
    static constexpr int kOwn = (kList + 1) / kThreads;
    __device__ __forceinline__ void read_list(int n, u64 (&p)[kOwn], u64 (&w)[kOwn]) {
        const int each = (n + kThreads - 1) / kThreads, i0 = threadIdx.x * each;
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            const bool some = i < each && i0 + i < n;
            p[i] = some ? s.list[i0 + i] : 0;
            w[i] = some ? weight_of(logit_of(p[i]), scale, s.powers) : 0;
        }
    }
    // The cut of the first CTA's list of n, read as p and w, as cut_list says; the list is sorted where it has to be.
    template <bool kMass>
    __device__ u64 cut_of(int n, const u64 (&p)[kOwn], const u64 (&w)[kOwn], u64 target) {
        u64 found = cut_list<kMass>(p, w, target);
        if (found == 0) {
            sort(n);
            found = s.list[kMass ? within(n, [&](u64) { return target; }) - 1 : static_cast<int>(target) - 1];
            __syncthreads();
        }
        return found;
    }

    // draw_from of at most 128, by the first warp alone.
    __device__ void draw_from_warp(int n, int top_k, float top_p, u64 target, float u, int32_t* token) {
        constexpr int kEach = 4;
        const int lane = threadIdx.x, i0 = lane * kEach;
        auto before_lane = [&](u64 v, u64& total) {
            u64 x = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 y = __shfl_up_sync(0xFFFFFFFFu, x, o);
                if (lane >= o) x += y;
            }
            total = __shfl_sync(0xFFFFFFFFu, x, 31);
            return x - v;
        };
        u64 p[kEach], least = 1, total;
#pragma unroll
        for (int e = 0; e < kEach; ++e) p[e] = i0 + e < n ? s.list[i0 + e] : 0;
        if (n > top_k || top_p < 1.0f) {
            u64 q[kEach];
#pragma unroll
            for (int e = 0; e < kEach; ++e) q[e] = p[e];
            int size = kEach;
            while (size < n) size *= 2;
#pragma unroll 1
            for (int k = 2; k <= size; k *= 2) {
#pragma unroll 1
                for (int j = k / 2; j >= kEach; j /= 2)
#pragma unroll
                    for (int e = 0; e < kEach; ++e) {
                        const u64 y = __shfl_xor_sync(0xFFFFFFFFu, q[e], j / kEach);
                        const bool larger = ((i0 & j) == 0) == ((i0 & k) == 0);
                        q[e] = larger == (q[e] > y) ? q[e] : y;
                    }
#pragma unroll
                for (int j = kEach / 2; j > 0; j /= 2)
                    if (j < k)
#pragma unroll
                        for (int e = 0; e < kEach; ++e)
                            if ((e & j) == 0) {
                                const u64 a = q[e], b = q[e + j];
                                const bool swap = (((i0 + e) & k) == 0) == (a < b);
                                q[e] = swap ? b : a;
                                q[e + j] = swap ? a : b;
                            }
            }
            u64 w[kEach], mine = 0;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                w[e] = i0 + e < min(n, top_k) ? weight_of(logit_of(q[e]), scale, s.powers) : 0;
                mine += w[e];
            }
            u64 before = before_lane(mine, total);
            const u64 want = top_p >= 1.0f ? ~0ull : target != 0 ? target : target_of(total, top_p);
            u64 lowest = ~0ull;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                if (i0 + e < min(n, top_k) && before < want) lowest = q[e];
                before += w[e];
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) lowest = min(lowest, __shfl_xor_sync(0xFFFFFFFFu, lowest, o));
            least = lowest;
        }
        u64 w[kEach], mine = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            w[e] = p[e] >= least ? weight_of(logit_of(p[e]), scale, s.powers) : 0;
            mine += w[e];
        }
        u64 before = before_lane(mine, total);
        const u64 want = part_of(total, u, false);
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            if (before <= want && want < before + w[e]) *token = index_of(p[e]);
            before += w[e];
        }
    }

    // The token from the first CTA's list of n places, in the order of the row: of the top_k of it, and of the likeliest that reach `target` of
    // weight (0: top_p of the weight of what is kept), which the list does.
    __device__ void draw_from(int n, int top_k, float top_p, u64 target, float u, int32_t* token) {
        if (n <= 128) {
            if (threadIdx.x < 32) draw_from_warp(n, top_k, top_p, target, u, token);
            return;
        }
        u64 p[kOwn], w[kOwn], mine = 0, total;
        read_list(n, p, w);
        auto keep = [&](u64 least) {
            mine = 0;
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                w[i] = p[i] >= least ? w[i] : 0;
                mine += w[i];
            }
        };
        u64 least = n > top_k ? cut_list<false>(p, w, top_k) : 1;
        keep(least);
        u64 before = scan_block(mine, s.sums, total);
        if (least != 0 && top_p < 1.0f) {
            least = cut_list<true>(p, w, target != 0 ? target : target_of(total, top_p));
            keep(least);
            before = scan_block(mine, s.sums, total);
        }
        if (least == 0) {  // many alike at a border
            sort(n);
            n = min(n, top_k);
            if (top_p < 1.0f) n = within(n, [&](u64 all) { return target != 0 ? target : target_of(all, top_p); });
            draw_list(n, u, token);
            return;
        }
        const u64 want = part_of(total, u, false);
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            if (before <= want && want < before + w[i]) *token = index_of(p[i]);
            before += w[i];
        }
    }

    // Weights of what is kept of the CTA's stretch, a group.
    __device__ void weigh_groups() {
        for (int g = threadIdx.x / 32 + (threadIdx.x & 31) * kWarps; g < row.groups; g += kThreads) s.groups[g] = 0;
        __syncwarp();
        row.each(cut_x, [&](int g, int i, const float (&v)[kV]) {
            const u64 sum = weigh_piece<false, true>(i, v);
            if ((threadIdx.x & 31) == 0) s.groups[g] = sum;
        });
        __syncthreads();
    }

    // The token in which u of the weight of what is kept is passed, given its weight a group.
    __device__ void draw(float u, int32_t* token) {
        static_assert(kMostGroups <= kThreads, "a group a thread");
        const u64 sum = threadIdx.x < row.groups ? s.groups[threadIdx.x] : 0;
        u64 all, at = scan_block(sum, s.sums, all), total = 0;
        u64 (*box)[kMaxCtas] = tell(all, 0);
        for (uint32_t r = 0; r < ctas; ++r) {
            if (r < rank) at += box[0][r];
            total += box[0][r];
        }
        const u64 want = part_of(total, u, false);
        if (!__syncthreads_or(at <= want && want < at + sum)) return;  // another CTA's
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

    // About the weight in bin b, from its count: 2^t in the bin's middle, 8 b + 3.5 steps down; with kLow no more than it is.
    template <bool kLow>
    __device__ __forceinline__ u64 guess(int b) const {
        const int n = -(b * kBinSteps + (kLow ? kBinSteps : kBinSteps / 2));
        const float w = s.powers[n & (kSteps - 1)].x * (kLow ? 1.0f : 1.0013547f) * __int_as_float(((kUnit + (n >> 8)) + 127) << 23);
        return s.all[b] * max(static_cast<u64>(w), kLow ? 0ull : 1ull);
    }

    // Whether the token could be drawn from a list of few tokens: the top_k of the row among them, or (target not 0) the likeliest that have
    // `target` of weight.
    __device__ bool draw_few(int top_k, float top_p, u64 target, float u, int32_t* token) {
        count_best();
        int bin = 0;
        if (rank == 0) {
            u64 before;
            if (target == 0) reach<u64>([&](int b) { return s.all[b]; }, static_cast<u64>(top_k), s.sums, bin, before);
            else reach<u64>([&](int b) { return guess<true>(b); }, target, s.sums, bin, before);
        }
        bin = static_cast<int>(tell(bin, 0)[0][0]);
        if (bin == kBins) {  // fewer threads than top_k, or less weight: everything, if it is little
            if (c.vocab > kList) return false;
            bin = kBins - 1;
        }
        const int n = gather(lowest_of(bin), [&](float x, int) { return bin_of(x, scale) <= bin; });
        if (n > kList) return false;
        if (rank == 0) draw_from(n, target == 0 ? top_k : INT_MAX, top_p, target, u, token);
        return true;
    }

    // The first CTA, given the counts a bin: the bin in which a guessed weight of `want` is reached, and bins around it, of least .. most - 1, that
    // the list can be expected to hold. In s.found.
    __device__ void window(u64 want, int least, int most, int& first, int& last, uint32_t& many) {
        int bin;
        u64 before;
        reach<u64>([&](int b) { return guess<false>(b); }, want, s.sums, bin, before);
        bin = max(least, min(bin, most - 1));
        constexpr int kEach = (kBins + kThreads - 1) / kThreads;
        const int b0 = threadIdx.x * kEach;
        int mine = 0, all;
#pragma unroll
        for (int i = 0; i < kEach; ++i) mine += b0 + i < kBins ? static_cast<int>(s.all[b0 + i]) : 0;
        int up = scan_block(mine, reinterpret_cast<int*>(s.sums), all);  // counts before a bin
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (b0 + i < kBins) {
                if (b0 + i == bin) {
                    s.found[0] = up;
                    s.found[1] = up + static_cast<int>(s.all[bin]);
                }
                s.bins[b0 + i] = up;
                up += static_cast<int>(s.all[b0 + i]);
            }
        }
        __syncthreads();
        const int from = s.found[0], to = s.found[1];
        if (threadIdx.x == 0) s.window[0] = s.window[1] = bin;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kEach && to - from <= kList - kGuess; ++i) {  // a bin with more stays alone
            const int b = b0 + i;
            if (b < kBins && b >= least && b < bin && from - static_cast<int>(s.bins[b]) <= kGuess / 2) atomicMin(&s.window[0], b);
            if (b < most && b > bin && static_cast<int>(s.bins[b] + s.all[b]) - to <= kGuess / 2) atomicMax(&s.window[1], b);
        }
        __syncthreads();
        first = s.window[0];
        last = s.window[1];
        many = s.bins[last] + s.all[last] - s.bins[first];
    }

    // Cuts what is kept at the likeliest that have `target` of its weight. true: the token was drawn; false: the weight of each group is left.
    // A guess from the counts gives a few bins around the border; one pass takes the exact weight of what is above them, and they are brought
    // together. Where the guess missed, the next one starts from what is known exactly, on the border's side of the window: the search ends.
    __device__ bool nucleus(u64 total, u64 target, float u, int32_t* token) {
        count();
        int64_t known = 0;            // exact less guessed weight before a window
        if (rank == 0) {              // at first that of all: it is the few largest that a bin's middle misses most
            u64 part = 0, guessed;
            for (int b = threadIdx.x; b < kBins; b += kThreads) part += guess<false>(b);
            scan_block(part, s.sums, guessed);
            known = static_cast<int64_t>(total - guessed);
        }
        int least = 0, most = kBins;  // the border's bin is one of least .. most - 1: fewer each time, so the search ends
        while (least < most) {
            int first = 0, last = 0;
            uint32_t n = 0;
            if (rank == 0) window(static_cast<u64>(max(static_cast<int64_t>(target) - known, static_cast<int64_t>(1))), least, most, first, last, n);
            u64 (*box)[kMaxCtas] = tell(static_cast<u64>(first) << 32 | last, n);
            first = static_cast<int>(box[0][0] >> 32);
            last = static_cast<int>(static_cast<uint32_t>(box[0][0]));
            n = static_cast<uint32_t>(box[1][0]);
            u64 above = 0;
            if (first > 0) {
                for (int g = threadIdx.x / 32 + (threadIdx.x & 31) * kWarps; g < row.groups; g += kThreads) s.groups[g] = 0;
                __syncwarp();
                row.each(fmaxf(cut_x, lowest_of(first - 1)), [&](int g, int i, const float (&v)[kV]) {
                    const u64 part = weigh_piece<true, true>(i, v, first);
                    if ((threadIdx.x & 31) == 0) {
                        s.groups[g] = part;
                        above += part;
                    }
                });
                above = sum_cluster(above);
            }
            // 2: the border is after the window; 0: before
            u64 found = 0;
            if (n > kList) {  // one bin, with many
                u64 sum = 0;
                row.each(fmaxf(cut_x, lowest_of(first)), [&](int, int i, const float (&v)[kV]) {
#pragma unroll
                    for (int e = 0; e < kV; ++e)
                        if (kept(v[e], i + e) && bin_of(v[e], scale) == first) sum += weight_of(v[e], scale, s.powers);
                });
                sum = sum_cluster(sum);
                found = target <= above ? 0 : target > above + sum ? 2 : inside<true>(first, n, target - above);
            } else {
                const float low = lowest_of(last), high = highest_of(first);
                n = gather(low, [&](float x, int) {
                    if (x < low || x > high) return false;  // nearly all
                    const int b = bin_of(x, scale);
                    return b >= first && b <= last;
                });
                if (rank == 0 && above < target) {
                    u64 p[kOwn], w[kOwn], sum = 0;
                    read_list(n, p, w);
#pragma unroll
                    for (int i = 0; i < kOwn; ++i) sum += w[i];
                    found = above + sum_block(sum) < target ? 2 : first == 0 ? 3 : cut_of<true>(n, p, w, target - above);
                    if (found == 3) draw_from(n, INT_MAX, 0.5f, target, u, token);  // all that is kept is in the list
                    if (found > 3) {  // the window's kept tokens come to their groups
#pragma unroll
                        for (int i = 0; i < kOwn; ++i)
                            if (w[i] != 0 && p[i] >= found) {
                                const int g = (index_of(p[i]) + row.shift) / kV / 32, owner = g / row.each_cta;
                                asm volatile("red.relaxed.cluster.shared::cluster.add.u64 [%0], %1;" ::"r"(mapa_shared(smem_u32(&s.groups[g - owner * row.each_cta]), owner)), "l"(w[i]) : "memory");
                            }
                    }
                }
                found = tell(found, 0)[0][0];
                if (found == 3) return true;
                if (found > 3) {
                    keep_from(found);
                    return false;
                }
            }
            if (found > 2) {  // the bin's kept tokens come to their groups
                if (first == 0) {
                    for (int g = threadIdx.x / 32 + (threadIdx.x & 31) * kWarps; g < row.groups; g += kThreads) s.groups[g] = 0;
                    __syncwarp();
                }
                keep_from(found);
                row.each(cut_x, [&](int g, int i, const float (&v)[kV]) {
                    u64 sum = 0;
#pragma unroll
                    for (int e = 0; e < kV; ++e)
                        if (kept(v[e], i + e) && bin_of(v[e], scale) >= first) sum += weight_of(v[e], scale, s.powers);
                    if (__any_sync(0xFFFFFFFFu, sum != 0)) {
                        sum = add_across(sum);
                        if ((threadIdx.x & 31) == 0) s.groups[g] += sum;
                    }
                });
                __syncthreads();
                return false;
            }
            if (found == 0) most = first;
            else least = last + 1;
            if (rank == 0) {
                u64 part = 0, guessed;
                for (int b = threadIdx.x; b < first; b += kThreads) part += guess<false>(b);
                scan_block(part, s.sums, guessed);
                known = static_cast<int64_t>(above - guessed);
            }
        }
        weigh_groups();  // not reached: what is kept weighs at least the target
        return false;
    }

    // The weight of what is kept, and of the threads' largest of it.
    __device__ u64 mass(u64& largest) {
        u64 sum = 0;
        row.each(cut_x, [&](int, int i, const float (&v)[kV]) { sum += weigh_piece<false, false>(i, v); });
        sum = sum_block(sum);
        u64 (*box)[kMaxCtas] = tell(sum, sum_block(best >= cut_x ? weight_of(best, scale, s.powers) : 0));
        sum = largest = 0;
        for (uint32_t r = 0; r < ctas; ++r) {
            sum += box[0][r];
            largest += box[1][r];
        }
        return sum;
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
    if (!greedy) {
        for (int i = threadIdx.x; i < kSteps; i += kThreads) s.powers[i] = kPowers.v[i];
        for (int b = threadIdx.x; b < kBins; b += kThreads) s.all[b] = 0;
    }
    if (threadIdx.x == kThreads - 32 && !greedy && min_p > 0.0f && min_p < 1.0f) {  // in 64 bits, once, while the others read
        const double below = (temperature < 1e30f ? 1.0 : 0.5) * static_cast<double>(temperature) * log(static_cast<double>(min_p));
        s.log_min_p.x = static_cast<float>(below);
        s.log_min_p.y = isinf(s.log_min_p.x) ? 0.0f : __double2float_ru(below - static_cast<double>(s.log_min_p.x));
    }
    const u64 largest = w.largest(greedy);
    const float x = logit_of(largest);
    if (!(x > kNone)) {
        if (rank == 0 && threadIdx.x == 0) c.tokens[r] = -1;
        return;
    }
    if (greedy) {
        if (rank == 0 && threadIdx.x == 0) c.tokens[r] = index_of(largest);
        return;
    }
    {
        const float y = 1.0f / temperature;
        const u64 top = static_cast<u64>(key_of(x)) << 32;
        // what is kept at all: above -inf, and not so small that a weight is nothing (2^-45 and below)
        const float none = x - 45.0f * 0.6931472f * temperature, far = (0.5f * x - 0.5f * none) * y;
        const u64 finite = static_cast<u64>(key_of(kNone) + 1) << 32;
        u64 cut = isinf(x) ? top : none > kNone ? max(finite, static_cast<u64>(key_of(none)) << 32) : finite;
        Scale& a = w.scale;
        a.top = x;
        a.flat = isinf(x);
        a.none = none > kNone && far > 15.2f && far < 25.0f ? none : kNone;  // where logits are as coarse as T it may have a weight, or be too far off
        a.t = temperature;
        a.near = a.none > kNone && fabsf(x) * y <= 200.0f && temperature < 1e18f && temperature > 1e-18f;
        // 1 / t, with t = T, or as much of it as of the logits: 1 / t = z + z (1 - z t), good to 2^-46; lo is 0 where T or 1 / T is infinite. With T small and
        // |x| not, nothing beside x has a weight
        const float by = a.near || (temperature >= 1e-18f && temperature < 1e18f) ? 1.0f : temperature >= 1e18f ? 0x1p-100f : fabsf(x) < 0x1p20f ? 0x1p100f : 1.0f;
        const float t = temperature * by, z = 1.0f / t, times = a.near ? 1.0f : 2.0f;
        a.half = a.near ? 1.0f : 0.5f * by;
        a.minus = a.near ? 0.0f : -a.half * x;
        a.hi = fminf(times * z, 3e38f);
        const float lo = times * z * fmaf(-z, t, 1.0f);
        a.lo = fabsf(lo) <= 1e-6f * a.hi ? lo : 0.0f;
        a.round = a.near ? kRound - ceilf(__fmul_rn(__fmul_rn(x, a.hi), kPerLn)) : kRound;
        w.easy = a.near && !(min_p > 0.0f);
        if (min_p >= 1.0f) {
            cut = top;
        } else if (min_p > 0.0f) {
            // the least float that is not below x + T ln(min_p), or half of it, as s0 + t0 and less (64-bit arithmetic would take all threads 1000 cycles)
            const float part = temperature < 1e30f ? 1.0f : 0.5f, h = part * x, b = s.log_min_p.x, s0 = __fadd_rn(h, b), bb = __fsub_rn(s0, h);
            if (fabsf(s0) < INFINITY) {
                const float t0 = __fadd_rn(__fadd_rn(__fsub_rn(h, __fsub_rn(s0, bb)), __fsub_rn(b, bb)), s.log_min_p.y);
                float z = __fadd_rn(s0, t0);
                if (__fsub_rn(t0, __fsub_rn(z, s0)) > 0.0f) z = nextafterf(z, INFINITY);
                cut = max(cut, static_cast<u64>(key_of(z / part)) << 32);
            }
        }
        w.keep_from(cut);
    }
    const bool by_count = top_k > 0 && top_k < c.vocab, by_mass = top_p < 1.0f;
    if (by_count) {
        if (top_k <= kList && w.draw_few(top_k, top_p, 0, u, c.tokens + r)) return;
        w.count();
        int bin = 0;
        uint32_t before = 0, many = 0;
        if (rank == 0) {
            w.template reach<uint32_t>([&](int b) { return s.all[b]; }, static_cast<uint32_t>(top_k), reinterpret_cast<uint32_t*>(s.sums), bin, before);
            many = bin < kBins ? s.all[bin] : 0;
        }
        u64 (*box)[kMaxCtas] = w.tell(static_cast<u64>(bin) << 32 | many, before);
        bin = static_cast<int>(box[0][0] >> 32);
        many = static_cast<uint32_t>(box[0][0]);
        before = static_cast<uint32_t>(box[1][0]);
        if (bin < kBins) {
            w.keep_from(w.template inside<false>(bin, many, top_k - before));
            w.easy = false;
        }
    }
    if (by_mass) {
        u64 of_best;
        const u64 total = w.mass(of_best), target = target_of(total, top_p);
        if (!by_count && (of_best >= target || c.vocab <= kList) && w.draw_few(0, top_p, target, u, c.tokens + r)) return;
        if (w.nucleus(total, target, u, c.tokens + r)) return;
    } else {
        w.weigh_groups();
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
    // CTAs of a row: at least so many that two stretches fit an SM's shared memory; more where rows are few, with at least 2048 logits each: as
    // long as all run at once, two an SM, or, where rows have settings of their own, twice as many: the few that take several times as long as
    // the others end sooner. Measured, us, 64 rows of 131071 bf16 with four and eight each: top_k 50 17.2 and 31.1, top_p 0.9 at T = 2
    // 77 and 99, settings mixed 58.2 and 41.6.
    const int64_t pieces = (c.vocab + Row<E>::kV - 1) / Row<E>::kV + 1, groups = (pieces + 31) / 32;
    const int64_t most = (c.temperature != nullptr || c.top_k != nullptr || c.top_p != nullptr ? 4ll : 2ll) * sm_count;
    int ctas = 1;
    while (ctas < kMaxCtas && ((c.rows * ctas * 2 <= most && c.vocab > 2048 * ctas) || groups > kMostGroups / 2 * ctas)) ctas *= 2;
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
