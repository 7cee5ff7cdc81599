// Attention over the paged 8-bit cache: for each new token's query head,
//
//     o = sum_j softmax_j(scale * q . k_j) v_j,  k_j = kcode_j * k_scale(page of j), v_j likewise,
//
// over the keys that the token sees: positions up to its own (or all of the
// sequence's when not causal), and with a window only the last `window` of
// them. Query heads g * share .. (g + 1) * share - 1 read kv head g. A row that
// sees no key gives zeros, and -inf as its log of the sum.
//
// This file: few rows a kv head (single tokens, drafts). There the cache's
// bytes bound the work, so each code is read once, by the copy engine, and the
// products are arranged so that nothing has to be moved between lanes.
//
// Scales stay out of the products. With t_j = log2(e) scale k_scale (q . kcode_j)
// + log2(v_scale), the weights w_j = 2^(t_j - m) carry the value scale of their
// page, so o = sum w_j vcode_j / sum (w_j / v_scale): the codes enter both
// products exactly (e4m3 and int8 are exact in fp16), and w_j < 2^16 whatever
// the scales. w is rounded to fp16 for its product, so that it can meet the codes
// in one tensor-core instruction: by 2^-11 of itself down to 2^-23 of the largest
// w of the row, below that in steps of 2^-33 of it (tg_kv_split.cuh). Its sum is
// kept in fp32 from the unrounded value.
//
// Splitting. The batch's work is a list of 64-token chunks, unit by unit (a unit
// is a sequence, a kv head and a block of 8 * kTiles rows); every CTA takes the
// same share of that list, so ragged lengths balance and few long sequences
// spread over the GPU. A unit that lies inside one CTA's share is finished
// there; parts of a unit that crosses shares go to the workspace and a second
// kernel, launched early, joins them in order.
//
// Inside a CTA four warps take every fourth 16-token step of a chunk, each with
// a ring of its own that TMA fills (16 tokens of one head are contiguous in a
// page). Per step a warp computes, with m16n8k16:
//   S^T (16 tokens x 8 rows) = K (16 x dim) Q^T, K the A operand,
//   O^T (dim x 8 rows) += V^T (dim x 16) W^T, V the A operand,
// so up to 8 rows cost one MMA column block, both operands are read from shared
// memory as whole 16-byte pieces (which dim a lane's piece holds does not
// matter as long as Q or O agrees), and W^T is S^T's registers through one
// 8 x 8 transposition. The 128-byte swizzle and the order in which a step's
// tokens are given to MMA rows (mma_token) keep those reads free of bank
// conflicts.
//
// Measured (one GB300, in a graph): 64 ragged sequences of up to 8192, 32 heads over 8 of 128, 630 MB of cache, 110 us,
// 5.7 TB/s or 0.84 of the copy rate; four sequences of up to 131071, 104 us, 0.84. What is missing is the
// start (lengths, shares, first pages: three dependent reads) and the join. One token over 1023: 8.6 us,
// all of it latency of the two kernels.
#include "tg_device.cuh"
#include "tg_kv_split.cuh"

#include <type_traits>

namespace tg {
namespace {

// ---------------------------------------------------------------- few rows

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kChunk = kWarps * kStep;       // tokens per unit of the work list
constexpr int kCtasPerSm = 3;

template <int kDim>
struct Ring {
    static constexpr int kStages = 4;                // steps in flight per warp
    static constexpr int kHalf = kStep * kDim;       // bytes of one step's keys (or values)
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kWarp = kStages * kStage;
    static constexpr int kBytes = kWarps * kWarp;
};

// A sequence's share of the list.
struct SeqWork {
    int first, count;      // its rows of the packed tensors
    int len;
    int chunk0, chunks;    // 64-token chunks that any of its rows sees (at least one, perhaps empty)
    int blocks;            // row blocks per kv head
    int64_t total;         // chunks over its units
};

template <int kTiles>
__device__ __forceinline__ SeqWork seq_work(const SplitWork& a, int i) {
    const KvAttnCall& c = a.c;
    SeqWork w;
    const SeqSpan span = seq_span(c.batch, i, c.wd);
    w.first = span.first;
    w.count = span.count;
    w.len = __ldg(c.batch.lens + i);
    if (w.len < 0 || w.len > c.max_len || w.len > c.batch.table_width << a.page_shift) {
        report_range(c.wd);
        w.len = 0;
    }
    const int64_t begin = c.window > 0 ? static_cast<int64_t>(w.len) - w.count - c.window + 1 : 0;
    w.chunk0 = begin > 0 ? static_cast<int>(begin / kChunk) : 0;
    w.chunks = max(1, (w.len + kChunk - 1) / kChunk - w.chunk0);
    w.blocks = static_cast<int>((static_cast<int64_t>(w.count) * a.share + 8 * kTiles - 1) / (8 * kTiles));
    w.total = static_cast<int64_t>(w.blocks) * c.cache.kv_heads * (w.chunks + a.extra);
    return w;
}

// Token of a step that MMA row i stands for. A quarter-warp's 16-byte reads touch the rows 2 i and
// 2 i + 1 (keys) or the even or odd ones of eight (values); with 128-byte lines swizzled by their
// line number these orders send the eight reads to eight different 16-byte banks.
template <int kDim>
__device__ __forceinline__ int mma_token(int i) {
    if constexpr (kDim == 128) {
        const int r = i & 7;
        return (i & 8) | ((r & 1) ? (r ^ 4) : r);  // 0 5 2 7 4 1 6 3
    } else {
        const int r = i & 7;                          // lines of two tokens: 0 1 4 5 8 9 12 13, then two further
        return ((r >> 1) * 4 + (r & 1)) + ((i & 8) ? 2 : 0);
    }
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Four values of a query row as they are stored.
template <typename E>
__device__ __forceinline__ uint2 load_four(const E* p, bool vec) {
    if (vec) return __ldg(reinterpret_cast<const uint2*>(p));
    uint2 u;
    E* e = reinterpret_cast<E*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = p[i];
    return u;
}

template <typename E, int kFmt, int kDim, int kTiles>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    attn_few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const SplitWork a) {
    constexpr int kRows = 8 * kTiles;
    constexpr int kK = kDim / 16;            // MMA steps along dim (scores) and m16 tiles along dim (values)
    constexpr int kStages = Ring<kDim>::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ alignas(8) uint64_t bars[kWarps * kStages];
    __shared__ float red_m[kWarps][kRows], red_l[kWarps][kRows];
    __shared__ int64_t scan[kWarps], found_off;
    __shared__ int found_seq;
    __shared__ int abort_flag;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const KvAttnCall& c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * Ring<kDim>::kWarp;
    const uint32_t bar0 = smem_u32(bars + warp * kStages);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(bar0 + 8 * s, 1);
        fence_barrier_init();
    }
    if (threadIdx.x == 0) {
        abort_flag = 0;
        found_seq = -1;
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    const WaitCtx wc{&abort_flag, c.wd.status, c.wd.limit_ns};

    // ---- this CTA's share of the list: the total, then the sequence in which the share begins
    const int batch = c.batch.batch;
    int64_t total = 0;
    auto block_scan = [&](int64_t v, int64_t& before) {  // sum over the block; `before`: over lower threads
        int64_t x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) scan[warp] = x;
        __syncthreads();
        int64_t sum = 0, low = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) low += scan[w];
            sum += scan[w];
        }
        before = low + x - v;
        return sum;
    };
    int64_t mine = 0, before = 0;
    for (int base = 0; base < batch; base += kThreads) {
        const int i = base + threadIdx.x;
        mine = i < batch ? seq_work<kTiles>(a, i).total : 0;
        total += block_scan(mine, before);
    }
    if (!a.joined) clear_uncovered<E, kDim>(c);
    const Shares shares(total, a.grid, a.least);
    const int k = blockIdx.x;
    if (k >= shares.ctas) {
        if (threadIdx.x == 0) a.meta[k].chunks = 0;
        return;
    }
    int64_t pos = shares.start(k);
    const int64_t stop = shares.start(k + 1);
    int64_t carry = 0;
    for (int base = 0; base < batch; base += kThreads) {
        if (batch > kThreads) {
            const int i = base + threadIdx.x;
            mine = i < batch ? seq_work<kTiles>(a, i).total : 0;
            const int64_t sum = block_scan(mine, before);
            before += carry;
            carry += sum;
        }
        if (before <= pos && pos < before + mine) {
            found_seq = base + threadIdx.x;
            found_off = pos - before;
        }
    }
    __syncthreads();
    int seq = found_seq;
    int64_t off = found_off;
    SeqWork w = seq_work<kTiles>(a, seq);

    int step_no = 0;  // steps issued to this warp's ring so far: stage and phase
    bool first_segment = true;
    bool ok = true;
    while (pos < stop) {
        if (off >= w.total) {  // the next sequence that has rows
            do {
                if (++seq >= batch) return;
                w = seq_work<kTiles>(a, seq);
            } while (w.total == 0);
            off = 0;
        }
        const int entries = w.chunks + a.extra;
        const int unit = static_cast<int>(off / entries);
        const int e0 = static_cast<int>(off - static_cast<int64_t>(unit) * entries);
        const int e1 = static_cast<int>(min(static_cast<int64_t>(entries), e0 + (stop - pos)));
        const int c0 = max(0, e0 - a.extra), c1 = max(0, e1 - a.extra);
        const int head = unit / w.blocks, block = unit - head * w.blocks;
        if (first_segment && threadIdx.x == 0) {
            Meta m{pos - e0, total, c0 > 0 ? w.chunks : 0, head, block, w.first, w.count};
            a.meta[k] = m;
        }
        pos += e1 - e0;
        off += e1 - e0;
        if (c1 == 0) continue;  // the share ends before the unit's first chunk
        const int row0 = block * kRows, rows = min(kRows, w.count * a.share - row0);

        // ---- the steps of this warp: chunks i0 .. i1 - 1, its 16 tokens of each
        const int tok0 = (w.chunk0 + c0) * kChunk + warp * kStep;
        const int64_t see0 = c.window > 0 ? static_cast<int64_t>(w.len) - w.count + row0 / a.share - c.window + 1 : 0;
        int i0 = 0, i1 = c1 - c0;
        if (tok0 >= w.len) i1 = 0;
        else i1 = min(i1, (w.len - tok0 + kChunk - 1) / kChunk);
        if (see0 > tok0) i0 = static_cast<int>(min(static_cast<int64_t>(i1), (see0 - tok0) / kChunk));
        const int n_steps = i1 - i0;
        const int32_t* table = c.batch.table + static_cast<int64_t>(seq) * c.batch.table_width;

        // page and scales of 32 steps at a time, a step a lane; those of the next 32 in advance
        auto page_of = [&](int s) {
            if (s >= n_steps) return -1;
            const int p = __ldg(table + ((tok0 + (i0 + s) * kChunk) >> a.page_shift));
            if (p < 0 || p >= c.cache.pages) {
                report_range(c.wd);
                return -1;
            }
            return p;
        };
        auto scales_of = [&](int p, float& ks, float& lv, float& iv) {
            const int64_t ph = static_cast<int64_t>(max(p, 0)) * c.cache.kv_heads + head;
            ks = p >= 0 ? __ldg(c.cache.k_scale + ph) : 0.0f;
            const float vs = p >= 0 ? max_nan(__ldg(c.cache.v_scale + ph), kScaleFloor) : 1.0f;
            lv = lg2_approx(vs);  // both are off by 2^-22, far below the rounding of the weights
            iv = rcp_approx(vs);
        };
        // the watchdog's test hook: the first step of a CTA never arrives
        auto withheld = [&](int s) { return c.wd.skip_first_arrive != 0 && warp == 0 && step_no + s == 0; };
        auto issue = [&](int s, int p, int slot) {  // lane 0: the copies of step s into stage slot
            const uint32_t bar = bar0 + 8 * slot;
            if (withheld(s)) return;
            if (p >= 0) {
                const int64_t place = (static_cast<int64_t>(p) * c.cache.kv_heads + head) * c.cache.page +
                                      ((tok0 + (i0 + s) * kChunk) & (c.cache.page - 1));
                const int line = static_cast<int>(kDim == 128 ? place : place >> 1);
                mbar_arrive_expect_tx(bar, Ring<kDim>::kStage);
                tma_load_2d(ring + slot * Ring<kDim>::kStage, &tmK, bar, 0, line);
                tma_load_2d(ring + slot * Ring<kDim>::kStage + Ring<kDim>::kHalf, &tmV, bar, 0, line);
            } else {
                mbar_arrive(bar);
            }
        };
        int pg = page_of(lane), pg_next = -1;
        for (int s = 0; s < min(kStages, n_steps); ++s) {
            const int p = __shfl_sync(0xFFFFFFFFu, pg, s);
            if (lane == 0) issue(s, p, (step_no + s) % kStages);
        }
        float ks, lv, iv, ks_next = 0.0f, lv_next = 0.0f, iv_next = 0.0f;
        scales_of(pg, ks, lv, iv);

        // ---- the queries: lane (gid, tig) holds of row gid (of each tile) the values that meet its
        // pieces of the keys. bf16 rows are moved by a power of two so that their largest value lies
        // in [2^14, 2^15): fp16 then holds every value down to 2^-28 of it without loss.
        uint32_t q[kTiles][kK][2];
        float factor[kTiles][2];     // of rows 2 tig, 2 tig + 1: scale * log2(e) / that power
        int see_from[kTiles][2], see_to[kTiles][2];
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {  // all tiles' reads first, so that they wait once
            const int r = row0 + min(8 * n + gid, rows - 1), t = r / a.share;
            const E* x = static_cast<const E*>(c.q.p) + static_cast<int64_t>(w.first + t) * c.q.token + (head * a.share + r - t * a.share) * c.q.head;
#pragma unroll
            for (int s = 0; s < kK; ++s) {
                const uint2 u = load_four(x + (s >> 2) * 64 + tig * 16 + (s & 3) * 4, a.q_vec != 0);
                q[n][s][0] = u.x;
                q[n][s][1] = u.y;
            }
        }
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
            const bool real = 8 * n + gid < rows;
            float f = c.scale * kLog2e;
            if constexpr (!std::is_same<E, __half>::value) {
                float most = 0.0f;
#pragma unroll
                for (int s = 0; s < kK; ++s)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const __nv_bfloat162 y = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&q[n][s][e]));
                        most = fmaxf(most, fmaxf(__low2float(y), __high2float(y)));
                    }
                most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
                most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
                // the exponent of the largest value, kept where 2^(14 - e) is an ordinary number
                const int e = most > 0.0f && most <= 3.3895314e38f ? max(-100, (__float_as_int(most) >> 23) - 127) : 14;
                const float up = __int_as_float((14 - e + 127) << 23);
                f *= __int_as_float((e - 14 + 127) << 23);
#pragma unroll
                for (int s = 0; s < kK; ++s)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&q[n][s][j]));
                        q[n][s][j] = half2_bits(y.x * up, y.y * up);
                    }
            }
            if (!real) {
#pragma unroll
                for (int s = 0; s < kK; ++s) q[n][s][0] = q[n][s][1] = 0;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                factor[n][e] = __shfl_sync(0xFFFFFFFFu, f, (2 * tig + e) * 4);
                const int rr = row0 + min(8 * n + 2 * tig + e, rows - 1);
                const int p = w.len - w.count + rr / a.share;
                see_to[n][e] = c.causal ? min(w.len, p + 1) : w.len;
                see_from[n][e] = c.window > 0 && p - c.window + 1 > 0 ? static_cast<int>(p - c.window + 1) : 0;
            }
        }
        // keys that every row sees: no mask there
        const int p_first = w.len - w.count + row0 / a.share, p_last = w.len - w.count + (row0 + rows - 1) / a.share;
        const int all_to = c.causal ? min(w.len, p_first + 1) : w.len;
        const int all_from = c.window > 0 && p_last - c.window + 1 > 0 ? static_cast<int>(p_last - c.window + 1) : 0;

        float m[kTiles][2], l[kTiles][2], o[kTiles][kK][4];
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
            m[n][0] = m[n][1] = kNoMax;
            l[n][0] = l[n][1] = 0.0f;
#pragma unroll
            for (int j = 0; j < kK; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.0f;
        }

        const int kt0 = mma_token<kDim>(gid), kt1 = mma_token<kDim>(gid + 8);
        int s = 0;
        for (; s < n_steps; ++s) {
            const int in = s & 31;
            if (s > 0 && in == 0) {
                pg = pg_next;
                ks = ks_next;
                lv = lv_next;
                iv = iv_next;
            }
            if (in == 0) pg_next = page_of(s + 32 + lane);
            if (in == 8) scales_of(pg_next, ks_next, lv_next, iv_next);
            const int slot = (step_no + s) % kStages;
            const uint32_t phase = static_cast<uint32_t>((step_no + s) / kStages) & 1u;
            if (!__all_sync(0xFFFFFFFFu, wait_phase(bar0 + 8 * slot, phase, wc, kSiteConvFull))) {
                ok = false;
                break;
            }
            const int p = __shfl_sync(0xFFFFFFFFu, pg, in);
            if (p >= 0) {
                const float ksc = __shfl_sync(0xFFFFFFFFu, ks, in), lvs = __shfl_sync(0xFFFFFFFFu, lv, in);
                const float ivs = __shfl_sync(0xFFFFFFFFu, iv, in);
                const uint32_t kbase = ring + slot * Ring<kDim>::kStage, vbase = kbase + Ring<kDim>::kHalf;
                const int token = tok0 + (i0 + s) * kChunk;

                // S^T = K Q^T
                float sc[kTiles][4];
#pragma unroll
                for (int n = 0; n < kTiles; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
#pragma unroll
                for (int j = 0; j < kDim / 64; ++j) {
                    const uint4 x = lds_v4(kbase + ring_offset<kDim>(kt0, j * 64 + tig * 16));
                    const uint4 y = lds_v4(kbase + ring_offset<kDim>(kt1, j * 64 + tig * 16));
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t a0, a1, a2, a3;
                        codes_to_half<kFmt>(xs[e], a0, a2);
                        codes_to_half<kFmt>(ys[e], a1, a3);
#pragma unroll
                        for (int n = 0; n < kTiles; ++n) mma16816(sc[n], a0, a1, a2, a3, q[n][j * 4 + e][0], q[n][j * 4 + e][1]);
                    }
                }
                // t = scaled score + log2(value scale); masked keys -inf
                bool above = false;
#pragma unroll
                for (int n = 0; n < kTiles; ++n) {
                    const float f0 = factor[n][0] * ksc, f1 = factor[n][1] * ksc;
                    sc[n][0] = fmaf(sc[n][0], f0, lvs);
                    sc[n][1] = fmaf(sc[n][1], f1, lvs);
                    sc[n][2] = fmaf(sc[n][2], f0, lvs);
                    sc[n][3] = fmaf(sc[n][3], f1, lvs);
                }
                const bool edge = token < all_from || token + kStep > all_to;
                if (edge) {
#pragma unroll
                    for (int n = 0; n < kTiles; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int t0 = token + kt0, t1 = token + kt1;
                            if (t0 < see_from[n][e] || t0 >= see_to[n][e]) sc[n][e] = -INFINITY;
                            if (t1 < see_from[n][e] || t1 >= see_to[n][e]) sc[n][2 + e] = -INFINITY;
                        }
                }
#pragma unroll
                for (int n = 0; n < kTiles; ++n)
                    above |= fmaxf(sc[n][0], sc[n][2]) > m[n][0] + kMostLog2 || fmaxf(sc[n][1], sc[n][3]) > m[n][1] + kMostLog2;
                if (__any_sync(0xFFFFFFFFu, above)) {
#pragma unroll
                    for (int n = 0; n < kTiles; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float t = fmaxf(sc[n][e], sc[n][2 + e]);
                            t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 4));
                            t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 8));
                            t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 16));
                            const float m_new = fmaxf(m[n][e], t - kHeadroomLog2);
                            const float keep = ex2_approx(m[n][e] - m_new);
                            m[n][e] = m_new;
                            l[n][e] *= keep;
#pragma unroll
                            for (int j = 0; j < kK; ++j) {
                                o[n][j][e] *= keep;
                                o[n][j][2 + e] *= keep;
                            }
                        }
                }
                uint32_t wt[kTiles][2];
#pragma unroll
                for (int n = 0; n < kTiles; ++n) {
                    const float w0 = ex2_approx(sc[n][0] - m[n][0]), w1 = ex2_approx(sc[n][1] - m[n][1]);
                    const float w2 = ex2_approx(sc[n][2] - m[n][0]), w3 = ex2_approx(sc[n][3] - m[n][1]);
                    l[n][0] = fmaf(w0 + w2, ivs, l[n][0]);
                    l[n][1] = fmaf(w1 + w3, ivs, l[n][1]);
                    wt[n][0] = transpose8x8(half2_bits(w0, w1));
                    wt[n][1] = transpose8x8(half2_bits(w2, w3));
                }
                // O^T += V^T W^T
                uint32_t v[4][kDim / 32];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = mma_token<kDim>(2 * tig + (e & 1) + (e >> 1) * 8);
                    if constexpr (kDim == 128) {
                        const uint4 x = lds_v4(vbase + ring_offset<kDim>(t, gid * 16));
                        v[e][0] = x.x;
                        v[e][1] = x.y;
                        v[e][2] = x.z;
                        v[e][3] = x.w;
                    } else {
                        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                                     : "=r"(v[e][0]), "=r"(v[e][1])
                                     : "r"(vbase + ring_offset<kDim>(t, gid * 8))
                                     : "memory");
                    }
                    // what lies past the sequence's end may be anything, and 0 times a NaN is one
                    if (edge && token + t >= w.len) {
#pragma unroll
                        for (int j = 0; j < kDim / 32; ++j) v[e][j] = 0;
                    }
                }
#pragma unroll
                for (int j = 0; j < kDim / 32; ++j) {
                    uint32_t a0, a1, a2, a3;
                    codes_to_half<kFmt>(__byte_perm(v[0][j], v[1][j], 0x5140), a0, a1);
                    codes_to_half<kFmt>(__byte_perm(v[2][j], v[3][j], 0x5140), a2, a3);
#pragma unroll
                    for (int n = 0; n < kTiles; ++n) mma16816(o[n][2 * j], a0, a1, a2, a3, wt[n][0], wt[n][1]);
                    codes_to_half<kFmt>(__byte_perm(v[0][j], v[1][j], 0x7362), a0, a1);
                    codes_to_half<kFmt>(__byte_perm(v[2][j], v[3][j], 0x7362), a2, a3);
#pragma unroll
                    for (int n = 0; n < kTiles; ++n) mma16816(o[n][2 * j + 1], a0, a1, a2, a3, wt[n][0], wt[n][1]);
                }
            }
            // every lane has read the stage: it may be filled again. The copy that fills it writes through another
            // proxy than these reads, and without the fence could land before them
            fence_proxy_async_smem();
            __syncwarp();
            if (s + kStages < n_steps) {
                const int ahead = (s + kStages) & 31;
                const int p_ahead = __shfl_sync(0xFFFFFFFFu, ahead < in ? pg_next : pg, ahead);
                if (lane == 0) issue(s + kStages, p_ahead, slot);
            }
        }
        if (!ok) {  // let every copy in flight land, then stop with the others
            for (const int issued = min(n_steps, s + kStages); s < issued; ++s)
                if (!withheld(s)) wait_phase_drain(bar0 + 8 * ((step_no + s) % kStages), static_cast<uint32_t>((step_no + s) / kStages) & 1u, wc);
        }
        step_no += n_steps;

        // ---- join the four warps: each brings its values to the common maximum, in its own ring
        // (its copies have all been read), then all threads add them up
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], 4);
                l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], 8);
                l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], 16);
                if (gid == 0) {
                    red_m[warp][8 * n + 2 * tig + e] = m[n][e];
                    red_l[warp][8 * n + 2 * tig + e] = l[n][e];
                }
            }
        if (__syncthreads_or(!ok)) break;
        float* mine_o = reinterpret_cast<float*>(smem + warp * Ring<kDim>::kWarp);
        static_assert(kRows * kDim * 4 <= Ring<kDim>::kWarp, "a warp's values fit its ring");
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * n + 2 * tig + e;
                const float top = fmaxf(fmaxf(red_m[0][r], red_m[1][r]), fmaxf(red_m[2][r], red_m[3][r]));
                const float keep = ex2_approx(m[n][e] - top);
#pragma unroll
                for (int j = 0; j < kK; ++j) {
                    // (tile j, gid) holds value gid * dim / 8 + 2 j, (tile j, gid + 8) the next one
                    float2 x = make_float2(o[n][j][e] * keep, o[n][j][2 + e] * keep);
                    *reinterpret_cast<float2*>(mine_o + r * kDim + gid * (kDim / 8) + 2 * j) = x;
                }
            }
        __syncthreads();
        const bool whole = c0 == 0 && c1 == w.chunks;
        float* part = a.parts + (static_cast<int64_t>(2 * k) + (first_segment ? 0 : 1)) * kRows * (kDim + 2);
        for (int i = threadIdx.x; i < rows * (kDim / 4); i += kThreads) {
            const int r = i / (kDim / 4), d = (i % (kDim / 4)) * 4;
            float top = kNoMax, sum = 0.0f;
#pragma unroll
            for (int x = 0; x < kWarps; ++x) top = fmaxf(top, red_m[x][r]);
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int x = 0; x < kWarps; ++x) {
                sum += red_l[x][r] * ex2_approx(red_m[x][r] - top);
                const float4 y = *reinterpret_cast<const float4*>(smem + x * Ring<kDim>::kWarp + (r * kDim + d) * 4);
                v.x += y.x;
                v.y += y.y;
                v.z += y.z;
                v.w += y.w;
            }
            if (whole) {
                const int t = (row0 + r) / a.share;
                const int64_t to = static_cast<int64_t>(w.first + t) * c.heads + head * a.share + (row0 + r) - t * a.share;
                const float inv = row_inverse(sum);
                E h[4] = {from_float<E>(v.x * inv), from_float<E>(v.y * inv), from_float<E>(v.z * inv), from_float<E>(v.w * inv)};
                *reinterpret_cast<uint2*>(static_cast<E*>(c.out) + to * kDim + d) = *reinterpret_cast<const uint2*>(h);
                if (d == 0 && c.lse != nullptr) c.lse[to] = row_lse(top, sum);
            } else {
                *reinterpret_cast<float4*>(part + r * kDim + d) = v;
                if (d == 0) {
                    part[kRows * kDim + r] = top;
                    part[kRows * (kDim + 1) + r] = sum;
                }
            }
        }
        fence_proxy_async_smem();  // these reads and writes come before the next copies into the rings
        __syncthreads();
        first_segment = false;
    }
}

// Row tiles of a block. Wider blocks read the cache less often, but their queries and outputs take the
// registers of a third CTA on the SM, and there are fewer of them: 33 sequences of 35 rows, dim 64, window 2048, run in
// 32.5 us with blocks of 40 rows, 28.7 with 24, 25.8 with 16; 120 of them without a window, 368 MB of cache,
// in 119, 107 and 106 us (a unit's blocks are neighbours in the list, so the later ones read L2).
constexpr int kMaxTiles = 2;

// How the few-rows kernel runs a call: row tiles, CTAs, workspace.
struct FewPlan {
    int tiles, grid, rows;
    bool split;            // a unit may cross shares
    int least, extra;
    int64_t meta_bytes, bytes;
};

FewPlan few_plan(const KvAttnCall& c, int sm_count) {
    FewPlan p{};
    const int64_t most = static_cast<int64_t>(c.batch.max_new) * (c.heads / c.cache.kv_heads);
    // the fewest row blocks, then the fewest tiles that hold a block's rows
    const int64_t least_blocks = (most + 8 * kMaxTiles - 1) / (8 * kMaxTiles);
    p.tiles = static_cast<int>((most + 8 * least_blocks - 1) / (8 * least_blocks));
    p.rows = 8 * p.tiles;
    p.grid = sm_count * kCtasPerSm;
    p.split = c.max_len > kChunk;
    // Every unit costs a share about as much as four chunks, whatever its length (its queries, an empty
    // pipeline, the join of four warps), and a CTA is worth starting for eight. 64 ragged sequences, three of
    // them idle: 130 us without that charge (one share held all the idle units), 110 with it, 110 with
    // twice it; one sequence of 16000: 23.4 us with any CTA, 20.5 with eight. Where the whole list is less
    // than two chunks a CTA, every chunk pair has a CTA to itself (one sequence of 1023: 9.6 us, not 11.2),
    // and every unit of a single chunk.
    const int64_t blocks = (most + p.rows - 1) / p.rows, chunks = (c.max_len + kChunk - 1) / kChunk;
    const bool small = blocks * c.cache.kv_heads * c.batch.batch * chunks <= 2 * p.grid;
    p.least = !small ? 8 : chunks >= 2 ? 2 : 1;
    p.extra = small ? 0 : 4;
    p.meta_bytes = (static_cast<int64_t>(p.grid) * sizeof(Meta) + 255) / 256 * 256;
    p.bytes = p.meta_bytes + static_cast<int64_t>(p.grid) * 2 * p.rows * (c.cache.dim + 2) * 4;
    return p;
}

// Rows of one kv head up to which a call runs here; above, k_kv_tile.cu takes it. Measured in us, here and there,
// with 32 heads over 8: 32 sequences of 2000, 36 rows 44 and 85, 64 rows 56 and 91, 96 rows 81 and 91, 128 rows 94
// and 99, 192 rows 140 and 103; four of 30000, 64 rows 88 and 105, 96 rows 129 and 108. Up to 64 rows this kernel is
// the quicker one throughout. From there to 128 it depends on the lengths, by up to a fifth either way, and
// calls too small to fill the GPU stay quicker here further on (two of 2000, 128 rows 21 and 27, 256 rows 27 and
// 34): the rule does not look at either.
bool few_rows(const KvAttnCall& c) { return static_cast<int64_t>(c.batch.max_new) * (c.heads / c.cache.kv_heads) <= 64; }

template <typename E, int kFmt, int kDim, int kTiles>
cudaError_t launch_few(const KvAttnCall& c, const CUtensorMap& tmK, const CUtensorMap& tmV, void* workspace, const FewPlan& p,
                       cudaStream_t stream) {
    static int attr_gen[64] = {};
    constexpr int smem = Ring<kDim>::kBytes + 1024;
    auto* kernel = attn_few_kernel<E, kFmt, kDim, kTiles>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && attr_gen[dev] != g_generation) {
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
        attr_gen[dev] = g_generation;
    }
    SplitWork a{};
    a.c = c;
    a.share = c.heads / c.cache.kv_heads;
    a.least = p.least;
    a.extra = p.extra;
    a.grid = p.grid;
    a.joined = p.split;
    a.q_vec = reinterpret_cast<uintptr_t>(c.q.p) % 8 == 0 && c.q.token % 4 == 0 && c.q.head % 4 == 0;
    a.meta = static_cast<Meta*>(workspace);
    a.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.meta_bytes);
    while (c.cache.page >> (a.page_shift + 1)) ++a.page_shift;
    kernel<<<p.grid, kThreads, smem, stream>>>(tmK, tmV, a);
    if ((e = cudaGetLastError()) != cudaSuccess || !p.split) return e;
    return launch_join<E, kDim, 8 * kTiles>(a, stream);
}

template <typename E, int kFmt, int kDim>
cudaError_t launch(const KvAttnCall& c, const CUtensorMap& tmK, const CUtensorMap& tmV, void* workspace, int sm_count,
                   cudaStream_t stream) {
    const FewPlan p = few_plan(c, sm_count);
    if (p.tiles == 1) return launch_few<E, kFmt, kDim, 1>(c, tmK, tmV, workspace, p, stream);
    return launch_few<E, kFmt, kDim, 2>(c, tmK, tmV, workspace, p, stream);
}

}  // namespace

int kv_attn_box_rows(const KvAttnCall& c) { return kStep * c.cache.dim / 128; }

int64_t kv_attn_workspace(const KvAttnCall& c, int sm_count) {
    return few_rows(c) ? few_plan(c, sm_count).bytes : kv_attn_tile_workspace(c, sm_count);
}

cudaError_t launch_kv_attn(const KvAttnCall& c, const CUtensorMap& tmK, const CUtensorMap& tmV, void* workspace, int sm_count,
                           cudaStream_t stream) {
    if (!few_rows(c)) return launch_kv_attn_tile(c, tmK, tmV, workspace, sm_count, stream);
    const bool h = c.dtype == kFp16, e4 = c.cache.fmt == kKvE4M3, d128 = c.cache.dim == 128;
    auto go = [&](auto* f) { return f(c, tmK, tmV, workspace, sm_count, stream); };
    if (h && e4) return d128 ? go(launch<__half, kKvE4M3, 128>) : go(launch<__half, kKvE4M3, 64>);
    if (h) return d128 ? go(launch<__half, kKvInt8, 128>) : go(launch<__half, kKvInt8, 64>);
    if (e4) return d128 ? go(launch<__nv_bfloat16, kKvE4M3, 128>) : go(launch<__nv_bfloat16, kKvE4M3, 64>);
    return d128 ? go(launch<__nv_bfloat16, kKvInt8, 128>) : go(launch<__nv_bfloat16, kKvInt8, 64>);
}

}  // namespace tg
