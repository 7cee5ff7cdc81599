// Attention over the paged 8-bit cache, many rows a kv head (prompt chunks):
// the operation, the way the scales are kept out of the products and the even
// split of the work are those of k_kv_attn.cu. Here the products bound it, and
// they run on tcgen05.
//
// A unit is a sequence, a kv head and a block of 256 rows (query heads of one
// kv head, token by token); its list entries are tiles of 128 keys, from the
// first that any row sees to the last. One CTA per SM walks its share:
//   warps 0-7, 8-15 softmax of rows 0-127 and 128-255, two threads a row (its TMEM
//                   lane), 64 scores of a tile each, in registers. They also
//                   bring the rows of Q to shared memory and write the result;
//   warps 16-19     turn codes, 8 KB at a time, into fp16 (exact) tiles with the
//                   128-byte swizzle, two of keys and two of values: once for both
//                   halves of the rows, which is what the 256 rows are for;
//   warps 20, 21    one thread each issues the MMAs of a half;
//   warp 22         walks the share and hands the segments (the part of a unit that
//                   this CTA computes) to the others through a ring in shared memory;
//   warp 23         looks up pages and scales of four tiles at a time, the next four's while it has
//                   TMA bring these' codes into a ring of three slots of 8 KB.
// TMEM: scores of either half 128 columns, outputs dim columns each; the weights (fp16)
// overwrite the scores they come from at dim 128, where a half's chain is scores, softmax,
// product, and only then the next scores. The second half's scores of a tile are issued when the first
// half's weights begin to arrive, so that one half's MMAs lie beside the other's
// exponentials. At dim 64 the weights have columns of their own, and a half's next scores are computed
// as soon as its softmax has read these.
//
// Measured (one GB300): chunks of up to 4096 new tokens on 8192, 32 heads over 8 of 128, causal: 661 us, 770 TFLOP/s or
// 0.40 of the dense rate (with heads of 64: 465 us, 547 TFLOP/s); the tensor pipe is active 36 % of the cycles. MMAs of M = 128, N = 128 and fp16 operands take
// 104 (scores) and 93 (product) cycles where the dense rate has 64, which alone would leave 65 %: the attention
// over 16-bit keys (k_attn.cu) has the same MMAs and reaches 1118 TFLOP/s. What is different here: every tile of
// codes is turned into fp16 again for each block of 256 rows that sees it, by four warps and through a ring of its
// own, which leaves shared memory for two stages of keys and values and 80 to 96 registers for the softmax (160 to 176
// bytes spilled, the two-part form 138 to 176; with 88 to 104, before the look-ahead, heads of 128 took the same time); and some 600 cycles of a half's chain are hand-overs that the other half does not fill.
#include "tg_device.cuh"
#include "tg_kv_split.cuh"

#include <algorithm>
#include <type_traits>

namespace tg {
namespace {

constexpr int kHalfRows = 128;
constexpr int kRows = 2 * kHalfRows;
constexpr int kKeys = 128;               // keys a tile
constexpr int kBlocks = kKeys / kStep;   // blocks of 16 keys with one scale each (a page has at least 16)
constexpr int kSoftmaxThreads = 512;
constexpr int kConvThreads = 128;
constexpr int kThreads = kSoftmaxThreads + kConvThreads + 128;
// Registers a thread: all start with kRegs; the softmax threads, which hold 64 scores, take what the
// others give up, within the launch's kThreads x kRegs.
constexpr int kRegs = 80, kRegsSoftmax = 96, kRegsConv = 56, kRegsIssue = 40;
static_assert(kSoftmaxThreads * kRegsSoftmax + kConvThreads * kRegsConv + 128 * kRegsIssue <= kThreads * kRegs, "register split");
static_assert(kRegsSoftmax >= kRegs && kRegsConv <= kRegs && kRegsIssue <= kRegs, "who takes and who gives");
constexpr int kInfoSlots = 16;           // tiles whose scales are in shared memory (ten can be in use)
constexpr int kSegSlots = 4;             // segments handed out ahead
constexpr int kSegReaders = 16 + 2 + 1;  // warps that read a segment: softmax, issuers, loader
constexpr int kTurns = 4;                // tiles whose turns are told apart (the halves are two apart at most)
// Codes come in pieces of 8 KB: a tile is two of keys and two of values, or one each.
// (At dim 64 pieces of 4 KB take the warps that bring and convert them too long: four groups of 2 to 17 sequences on 30011 shared
// tokens 108 us, with these 94; and 105 where a half's scores wait for its product.)
template <int kDim>
constexpr int kPiece = 8192 / kDim;                 // tokens
template <int kDim>
constexpr int kPieces = kKeys / kPiece<kDim>;       // of a tile's keys
constexpr int kRawSlots = 3;                        // pieces in flight
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;            // + 128 half; the weights of keys 64 g .. are the first 32 of their 64 columns
constexpr uint32_t kColO = 256;          // + dim half
constexpr uint32_t kColP = 384;          // + 64 half: the weights of all keys, at dim 64
// Whether the weights have columns of their own, so that a half's next scores are computed while it weighs these.
template <int kDim>
constexpr bool kScoresAhead = kDim == 64;

// What a CTA holds back while the watchdog's test hook is on, one CTA after another: its first piece of codes, word
// of its products, or its first segment.
constexpr int kNoCodes = 1, kNoProduct = 2, kNoSegment = 3;

// What the softmax and the converters know of a tile: per block of 16 keys the key scale, log2 and
// inverse of the value scale, and how many tokens are there.
struct TileInfo {
    float ks[kBlocks], lv[kBlocks], iv[kBlocks];
    int there[kBlocks];
    int state;   // 1: every token is there, 0: not every one, -1: no tile, the share is done
    int pad[3];
};

template <int kDim>
struct Smem {
    static constexpr int kBox = 128 * 128;                 // 128 rows of 64 fp16
    static constexpr int kTile = kBox * (kDim / 64);
    static constexpr int kRaw = kPiece<kDim> * kDim;       // bytes of a piece
    static constexpr int kQ = 0;                           // 2 halves
    static constexpr int kK = 2 * kTile;                   // 2 stages
    static constexpr int kV = 4 * kTile;                   // 2 stages
    static constexpr int kRawAt = 6 * kTile;
    static constexpr int kRed = kRawAt + kRawSlots * kRaw; // [parity][half][key half][row] floats
    static constexpr int kInfo = kRed + 2 * 2 * 2 * kHalfRows * 4;
    static constexpr int kSegments = kInfo + kInfoSlots * static_cast<int>(sizeof(TileInfo));
    static constexpr int kBars = kSegments + kSegSlots * 64;
    static constexpr int kNumBars = 2 + 2 + 2 + 2 + 2 + 2 + 2 + 4 + 2 + kInfoSlots + 2 + kTurns + 2 * kSegSlots + 2 * kRawSlots + 1;
    static constexpr int kScan = kBars + 8 * kNumBars;      // a sum a warp, then found offset and sequence
    static constexpr int kFoundOff = kScan + kThreads / 32 * 8;
    static constexpr int kFoundSeq = kFoundOff + 8;
    static constexpr int kTmemSlot = kFoundSeq + 4;
    static constexpr int kAbort = kTmemSlot + 4;
    static constexpr int kUsed = kAbort + 4;
    static constexpr int kAlloc = kUsed + 1024;
    static_assert(kRed % 16 == 0 && kInfo % 16 == 0 && kSegments % 16 == 0 && kBars % 8 == 0 && kScan % 8 == 0 && kFoundOff % 8 == 0, "alignment");
    static_assert(kRawAt % 1024 == 0 && kRaw % 1024 == 0, "swizzle atoms");
    static_assert(kAlloc <= 227 * 1024, "shared memory of one CTA");
};

// A sequence and the tiles of its row blocks.
struct TileWork {
    int first, count, len;
    int blocks;       // row blocks per kv head
    int64_t total;    // tiles over all of them and all kv heads
};

// Tiles of row block `block`: first, and how many (at least one, perhaps of no key).
__device__ __forceinline__ void tiles_of(const SplitWork& a, int count, int len, int block, int& tile0, int& tiles) {
    const KvAttnCall& c = a.c;
    const int rows = count * a.share, row0 = block * kRows, row1 = min(rows, row0 + kRows) - 1;
    const int64_t p0 = static_cast<int64_t>(len) - count + row0 / a.share, p1 = static_cast<int64_t>(len) - count + row1 / a.share;
    const int64_t from = c.window > 0 ? p0 - c.window + 1 : 0;
    const int64_t to = c.causal ? min(static_cast<int64_t>(len), p1 + 1) : len;
    tile0 = from > 0 ? static_cast<int>(from / kKeys) : 0;
    tiles = max(1, (max(0, static_cast<int>(to)) + kKeys - 1) / kKeys - tile0);
}

__device__ __forceinline__ TileWork tile_work(const SplitWork& a, int i) {
    const KvAttnCall& c = a.c;
    TileWork w;
    const SeqSpan span = seq_span(c.batch, i, c.wd);
    w.first = span.first;
    w.count = span.count;
    w.len = __ldg(c.batch.lens + i);
    if (w.len < 0 || w.len > c.max_len || w.len > c.batch.table_width << a.page_shift) {
        report_range(c.wd);
        w.len = 0;
    }
    w.blocks = (w.count * a.share + kRows - 1) / kRows;
    int64_t per_head = 0;
    for (int b = 0; b < w.blocks; ++b) {
        int t0, n;
        tiles_of(a, w.count, w.len, b, t0, n);
        per_head += n;
    }
    w.total = per_head * c.cache.kv_heads;
    return w;
}

// One piece of a CTA's share: tiles t0 .. t1 - 1 of a unit (none: the share is done).
struct Segment {
    int seq, head, block, first, count, len;
    int tile0, tiles;   // of the unit
    int t0, t1;         // the segment's among them
};
static_assert(sizeof(Segment) <= 64, "a slot of the ring");

// The segments of a CTA's share, one after another.

struct Walk {
    const SplitWork& a;
    int64_t left;
    int seq, head, block, at;
    TileWork w;
    __device__ Walk(const SplitWork& args, int seq0, int64_t off, int64_t n) : a(args), left(n), seq(seq0), w(tile_work(args, seq0)) {
        const int64_t per_head = w.total / a.c.cache.kv_heads;
        head = static_cast<int>(off / per_head);
        int64_t in = off - head * per_head;
        block = 0;
        int t0, k;
        tiles_of(a, w.count, w.len, 0, t0, k);
        while (in >= k && block + 1 < w.blocks) {
            in -= k;
            tiles_of(a, w.count, w.len, ++block, t0, k);
        }
        at = static_cast<int>(in);
    }
    __device__ bool next(Segment& s) {
        if (left <= 0) return false;
        while (block >= w.blocks) {  // the next kv head, or the next sequence that has rows
            block = 0;
            if (++head >= a.c.cache.kv_heads || w.blocks == 0) {
                head = 0;
                if (++seq >= a.c.batch.batch) return false;
                w = tile_work(a, seq);
            }
        }
        s.seq = seq;
        s.head = head;
        s.block = block;
        s.first = w.first;
        s.count = w.count;
        s.len = w.len;
        tiles_of(a, w.count, w.len, block, s.tile0, s.tiles);
        s.t0 = at;
        s.t1 = static_cast<int>(min(static_cast<int64_t>(s.tiles), at + left));
        left -= s.t1 - s.t0;
        at = 0;
        ++block;
        return true;
    }
};

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
        "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

template <typename E, int kFmt, int kDim, bool kParts>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tile_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const SplitWork a) {
    using L = Smem<kDim>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const KvAttnCall& c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t bar = sbase + L::kBars;
    auto bars = [&](int n) {
        const uint32_t b = bar;
        bar += 8 * n;
        return b;
    };
    const uint32_t q_full = bars(2), k_full = bars(2), k_empty = bars(2), v_full = bars(2), v_empty = bars(2), s_full = bars(2), s_read = bars(2);
    const uint32_t p_full = bars(4), o_done = bars(2), info_full = bars(kInfoSlots), drain = bars(2), turn = bars(kTurns);
    const uint32_t seg_full = bars(kSegSlots), seg_empty = bars(kSegSlots), raw_full = bars(kRawSlots), raw_empty = bars(kRawSlots), nowhere = bars(1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kTmemSlot);
    int64_t* scan = reinterpret_cast<int64_t*>(smem + L::kScan);
    int* found_seq = reinterpret_cast<int*>(smem + L::kFoundSeq);
    int64_t* found_off = reinterpret_cast<int64_t*>(smem + L::kFoundOff);
    TileInfo* infos = reinterpret_cast<TileInfo*>(smem + L::kInfo);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + 8 * i, 8);           // a warp's share of one half's rows
            mbar_init(k_full + 8 * i, kConvThreads / 32);
            mbar_init(k_empty + 8 * i, 2);          // either half's products
            mbar_init(v_full + 8 * i, kConvThreads / 32);
            mbar_init(v_empty + 8 * i, 2);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(s_read + 8 * i, 8);           // the warps of the half (with kScoresAhead)
            mbar_init(o_done + 8 * i, 1);
            mbar_init(drain + 8 * i, 1);
        }
        mbar_init(nowhere, 2);  // that nothing waits for
        for (int i = 0; i < 4; ++i) mbar_init(p_full + 8 * i, 8);
        for (int i = 0; i < kTurns; ++i) mbar_init(turn + 8 * i, 1);
        for (int i = 0; i < kInfoSlots; ++i) mbar_init(info_full + 8 * i, 1);
        for (int i = 0; i < kSegSlots; ++i) {
            mbar_init(seg_full + 8 * i, 1);
            mbar_init(seg_empty + 8 * i, kSegReaders);
        }
        for (int i = 0; i < kRawSlots; ++i) {
            mbar_init(raw_full + 8 * i, 1);
            mbar_init(raw_empty + 8 * i, kConvThreads / 32);
        }
        fence_barrier_init();
        *abort_flag = 0;
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }

    // ---- this CTA's share of the list
    const int batch = c.batch.batch;
    int64_t total = 0;
    constexpr int kWarps = kThreads / 32;
    auto block_scan = [&](int64_t v, int64_t& before) {
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
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) low += scan[w];
            sum += scan[w];
        }
        before = low + x - v;
        return sum;
    };
    int64_t mine = 0, before = 0;
    const bool by_warp = kParts && batch <= 32;  // every warp by itself, without a barrier: 2 us sooner
    if (by_warp) {
        mine = lane < batch ? tile_work(a, lane).total : 0;
        int64_t x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        before = x - mine;
        total = __shfl_sync(0xFFFFFFFFu, x, 31);
    } else {
        for (int base = 0; base < batch; base += kThreads) {
            const int i = base + threadIdx.x;
            mine = i < batch ? tile_work(a, i).total : 0;
            total += block_scan(mine, before);
        }
    }
    if (!a.joined) clear_uncovered<E, kDim>(c);
    const Shares shares(total, a.grid, a.least);
    const int k = blockIdx.x;
    // the joining kernel runs whatever becomes of this one: until the first segment is known there is nothing to join
    if (threadIdx.x == 0) a.meta[k].chunks = 0;
    if (k >= shares.ctas) {
        if constexpr (kParts) wait_for_first();
        return;
    }
    const int64_t start = shares.start(k), stop = shares.start(k + 1);
    int64_t carry = 0;
    for (int base = 0; base < batch; base += kThreads) {
        if (batch > kThreads) {
            const int i = base + threadIdx.x;
            mine = i < batch ? tile_work(a, i).total : 0;
            const int64_t sum = block_scan(mine, before);
            before += carry;
            carry += sum;
        }
        if ((!by_warp || warp == 0) && before <= start && start < before + mine) {
            *found_seq = base + threadIdx.x;
            *found_off = start - before;
        }
    }
    if (warp == 20) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const WaitCtx wc{abort_flag, c.wd.status, c.wd.limit_ns};
    const int withheld = c.wd.skip_first_arrive ? 1 + static_cast<int>(blockIdx.x % 3) : 0;
    // the next segment for this warp; false when there is none, or a wait gave up
    uint32_t seg_no = 0;
    auto next_segment = [&](Segment& s) {
        const uint32_t slot = seg_no % kSegSlots;
        if (!__all_sync(0xFFFFFFFFu, wait_suspended(seg_full + 8 * slot, (seg_no / kSegSlots) & 1u, wc, kSiteMmaFull))) return false;
        s = *reinterpret_cast<const Segment*>(smem + L::kSegments + slot * 64);
        __syncwarp();
        if (lane == 0) mbar_arrive(seg_empty + 8 * slot);
        ++seg_no;
        return s.t1 > s.t0;
    };
    Segment sg;
    uint32_t tile_no = 0;  // tiles so far: stages and phases

    if (warp >= 20) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
        if (warp == 22) {
            // -------------------------------------------------------- segments
            if (lane == 0) {
                Walk walk(a, *found_seq, *found_off, stop - start);
                for (bool more = true; more; ++seg_no) {
                    const uint32_t slot = seg_no % kSegSlots;
                    if (!wait_phase_sleep(seg_empty + 8 * slot, ((seg_no / kSegSlots) & 1u) ^ 1u, wc, kSiteProducerEmpty, 64)) break;
                    more = walk.next(sg);
                    if (!more) sg.t0 = sg.t1 = 0;
                    *reinterpret_cast<Segment*>(smem + L::kSegments + slot * 64) = sg;
                    if (withheld != kNoSegment || seg_no != 0) mbar_arrive(seg_full + 8 * slot);
                }
            }
            __syncwarp();
        } else if (warp < 22) {
            // -------------------------------------------------------- MMA issue of half h
            const int h = warp - 20;
            constexpr uint32_t idesc_s = idesc_f16_f32(128, 128, false, false);
            constexpr uint32_t idesc_o = idesc_f16_f32(128, kDim, false, true);
            const uint64_t qd = smem_desc_sw128(sbase + L::kQ + h * L::kTile, 16, 1024);
            const uint64_t kd = smem_desc_sw128(sbase + L::kK, 16, 1024);
            const uint64_t vd = smem_desc_sw128(sbase + L::kV, L::kBox, 1024);
            const uint32_t col_s = tmem + kColS + 128 * h, col_o = tmem + kColO + kDim * h, col_p = kScoresAhead<kDim> ? tmem + kColP + 64 * h : col_s;
            const uint32_t product_done = withheld == kNoProduct ? nowhere : o_done + 8 * h;
            // 16 keys of the product; their weights are 8 columns
            auto product = [&](int kk, uint32_t st, bool add) {
                mma_f16_tmem_a(col_o, col_p + (kk >> 2) * (kScoresAhead<kDim> ? 32 : 64) + (kk & 3) * 8, vd + st * (L::kTile >> 4) + kk * (2048 >> 4), idesc_o, add);
            };
            auto scores = [&](uint32_t st) {
                tc_fence_after_sync();
#pragma unroll
                for (int kk = 0; kk < kDim / 16; ++kk) {
                    const uint32_t in = ((kk >> 2) * L::kBox + (kk & 3) * 32) >> 4;
                    mma_f16(col_s, qd + in, kd + st * (L::kTile >> 4) + in, idesc_s, kk != 0);
                }
                mma_commit(s_full + 8 * h);
                mma_commit(k_empty + 8 * st);
            };
            bool ok = true;
            while (ok && next_segment(sg)) {
                if (lane == 0) {
                    const int n = sg.t1 - sg.t0;
                    ok = wait_suspended(q_full + 8 * h, (seg_no - 1) & 1u, wc, kSiteMmaFull);
                    for (int j = 0; ok && j < n; ++j) {
                        const uint32_t g = tile_no + j, st = g & 1u, kph = (g >> 1) & 1u;
                        if (!kScoresAhead<kDim> || j == 0) {
                            // the scores overwrite the weights of tile j - 1
                            ok = wait_suspended(k_full + 8 * st, kph, wc, kSiteMmaFull) &&
                                 (j == 0 || wait_suspended(o_done + 8 * h, (g - 1) & 1u, wc, kSiteMmaAccEmpty)) &&
                                 (h == 0 || wait_suspended(turn + 8 * (g % kTurns), (g / kTurns) & 1u, wc, kSiteMmaFull));
                            if (!ok) break;
                            scores(st);
                        }
                        if (kScoresAhead<kDim> && j + 1 < n) {  // once these are read
                            ok = wait_suspended(k_full + 8 * (st ^ 1u), ((g + 1) >> 1) & 1u, wc, kSiteMmaFull) &&
                                 wait_suspended(s_read + 8 * h, g & 1u, wc, kSiteMmaAccEmpty);
                            if (!ok) break;
                            scores(st ^ 1u);
                        }
                        ok = wait_suspended(v_full + 8 * st, kph, wc, kSiteMmaFull) && wait_suspended(p_full + 16 * h, g & 1u, wc, kSiteMmaFull);
                        if (!ok) break;
                        if (h == 0) mbar_arrive(turn + 8 * (g % kTurns));
                        tc_fence_after_sync();
                        product(0, st, j != 0);  // keys 0-31 and 64-95 are handed over first
                        product(1, st, true);
                        product(4, st, true);
                        product(5, st, true);
                        ok = wait_suspended(p_full + 16 * h + 8, g & 1u, wc, kSiteMmaFull);
                        if (!ok) break;
                        tc_fence_after_sync();
                        product(2, st, true);
                        product(3, st, true);
                        product(6, st, true);
                        product(7, st, true);
                        mma_commit(product_done);
                        mma_commit(v_empty + 8 * st);
                    }
                    tile_no += n;
                }
                ok = __all_sync(0xFFFFFFFFu, ok);
            }
            if (lane == 0) {
                mma_commit(drain + 8 * h);
                wait_phase_drain(drain + 8 * h, 0, wc);
            }
            __syncwarp();
        } else {
            // -------------------------------------------------------- pages, scales and the copies of the codes
            // A lane per block of 16 keys, and four tiles at a time, their pages read while the four before are brought: what a
            // tile's lookups wait for (the page, then its scales) takes longer than its products.
            constexpr int kBatch = 32 / kBlocks;
            uint32_t piece = 0, slot = 0, turned = 1;  // pieces so far, the next one's slot, and what its emptiness is waited for by
            const int nth = lane / kBlocks, block = lane % kBlocks;
            const int step = a.box / kStep;            // blocks a copy
            constexpr int kInPiece = kPiece<kDim> / kStep;
            const int32_t* row = nullptr;
            int tile = 0, entry = 0;
            bool have, asked = false;
            auto look_up = [&] {  // the batch that begins at sg's `tile`
                const int token = (sg.tile0 + tile + nth) * kKeys + block * kStep;
                asked = tile + nth < sg.t1 && token < sg.len;
                entry = asked ? __ldg(row + (token >> a.page_shift)) : -1;
            };
            auto next = [&] {
                have = next_segment(sg);
                tile = sg.t0;
                if (have) row = table_row<kParts>(c.batch, sg.seq);
            };
            auto free_slot = [&] { return __all_sync(0xFFFFFFFFu, wait_suspended(raw_empty + 8 * slot, turned, wc, kSiteConvEmpty)); };
            next();
            if (have) look_up();
            bool ok = true;
            while (have) {
                const int token = (sg.tile0 + tile + nth) * kKeys + block * kStep, tiles = min(kBatch, sg.t1 - tile);
                int cur = entry;
                if (asked && (cur < 0 || cur >= c.cache.pages)) {
                    report_range(c.wd);
                    cur = -1;
                }
                const int there = cur >= 0 ? min(kStep, sg.len - token) : 0;
                const int64_t ph = static_cast<int64_t>(max(cur, 0)) * c.cache.kv_heads + sg.head;
                float ks = 0.0f, vs = 1.0f;
                if (cur >= 0) {
                    ks = __ldg(c.cache.k_scale + ph);
                    vs = __ldg(c.cache.v_scale + ph);
                }
                const int64_t place = ph * c.cache.page + (token & (c.cache.page - 1));
                const int line = static_cast<int>(kDim == 128 ? place : place >> 1);
                const bool first = cur >= 0 && block % step == 0;  // a copy begins here
                tile += tiles;
                if (tile >= sg.t1) next();
                if (have) look_up();
                for (int i = 0; i < tiles; ++i) {
#pragma unroll 1
                    for (int part = 0; part < 2 * kPieces<kDim>; ++part) {  // keys, then values
                        if (!(ok = free_slot())) break;
                        const bool mine = first && lane / kInPiece == kPieces<kDim> * i + part % kPieces<kDim>;
                        const uint32_t many = __popc(__ballot_sync(0xFFFFFFFFu, mine)) * step;
                        const uint32_t bar_at = raw_full + 8 * slot;
                        if (withheld != kNoCodes || piece != 0) {
                            if (lane == 0) {
                                if (many > 0) mbar_arrive_expect_tx(bar_at, many * kStep * kDim);
                                else mbar_arrive(bar_at);
                            }
                            __syncwarp();
                            if (mine) tma_load_2d(sbase + L::kRawAt + slot * L::kRaw + lane % kInPiece * kStep * kDim, part < kPieces<kDim> ? &tmK : &tmV, bar_at, 0, line);
                        }
                        ++piece;
                        if (++slot == kRawSlots) {
                            slot = 0;
                            turned ^= 1;
                        }
                        if (i == 0 && part == 0) {  // what is said of the four tiles
                            const uint32_t whole = __ballot_sync(0xFFFFFFFFu, there == kStep);
                            TileInfo& info = infos[(tile_no + nth) % kInfoSlots];
                            if (nth < tiles) {
                                const float v = max_nan(vs, kScaleFloor);
                                info.ks[block] = ks;
                                info.lv[block] = cur >= 0 ? log2f(v) : -INFINITY;  // no page: no weight
                                info.iv[block] = 1.0f / v;
                                info.there[block] = there;
                                if (block == 0) info.state = (whole >> (nth * kBlocks) & ((1u << kBlocks) - 1)) == (1u << kBlocks) - 1;
                            }
                            __syncwarp();
                            if (nth < tiles && block == 0) mbar_arrive(info_full + 8 * ((tile_no + nth) % kInfoSlots));
                        }
                    }
                    if (!ok) break;
                    ++tile_no;
                }
                if (!ok) break;
            }
            // the converters stop at a tile of which nothing is said but that it is the end
            if (ok && free_slot() && lane == 0) {
                infos[tile_no % kInfoSlots].state = -1;
                mbar_arrive(info_full + 8 * (tile_no % kInfoSlots));
            }
            // let every copy in flight land before the CTA ends
            for (uint32_t i = piece > kRawSlots ? piece - kRawSlots : withheld == kNoCodes; lane == 0 && i < piece; ++i)
                wait_phase_drain(raw_full + 8 * (i % kRawSlots), (i / kRawSlots) & 1u, wc);
            __syncwarp();
        }
    } else if (warp >= 16) {
        // ------------------------------------------------------------ codes to fp16 tiles
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConv));
        // A thread takes 16 codes (two 16-byte pieces of fp16) of a token: 64 of a row's codes, one box of the fp16
        // tile, are four lanes; a quarter-warp is two tokens whose numbers differ so that its reads of the
        // swizzled codes and its writes of the swizzled fp16 both go to eight different 16-byte banks. A warp is
        // 8 tokens of one box; the four warps take boxes and groups of 8 tokens in turn.
        const int at = lane & 3, r = lane >> 3, b = lane >> 2 & 1;
        const int t8 = kDim == 128 ? r ^ (b ? 5 : 0) : 2 * r + b;       // token of eight
        constexpr int kRounds = kPiece<kDim> / 8 * (kDim / 64) / 4;     // of the four warps in a piece
        const int box = kDim == 128 ? warp & 1 : 0;
        const int group0 = kDim == 128 ? (warp - 16) >> 1 : warp - 16;  // first group of 8 tokens, then every 2nd or 4th
        constexpr int kGroupStep = kDim == 128 ? 2 : 4;
        // groups of a warp are an even number apart, so a thread's place in the swizzle is the same in all
        const uint32_t get = ring_offset<kDim>(group0 * 8 + t8, (kDim == 128 ? box * 64 : 0) + at * 16);
        const uint32_t put = box * L::kBox + (group0 * 8 + t8) * 128, put0 = ((2 * at) ^ t8) << 4, put1 = ((2 * at + 1) ^ t8) << 4;
        uint32_t piece = 0;
        bool ok = true;
        while (ok) {
            const uint32_t st = tile_no & 1u, eph = ((tile_no >> 1) & 1u) ^ 1u;
            ok = __all_sync(0xFFFFFFFFu, wait_suspended(info_full + 8 * (tile_no % kInfoSlots), (tile_no / kInfoSlots) & 1u, wc, kSiteConvFull));
            if (!ok) break;
            const TileInfo& info = infos[tile_no % kInfoSlots];
            const int state = info.state;
            if (state < 0) break;
            for (int part = 0; part < 2 * kPieces<kDim>; ++part, ++piece) {
                const int nth = part % kPieces<kDim>;
                const uint32_t slot = piece % kRawSlots, raw = sbase + L::kRawAt + slot * L::kRaw + get;
                ok = __all_sync(0xFFFFFFFFu, wait_suspended(raw_full + 8 * slot, (piece / kRawSlots) & 1u, wc, kSiteConvFull));
                if (!ok) break;
                uint4 x[kRounds];
#pragma unroll
                for (int i = 0; i < kRounds; ++i) x[i] = lds_v4(raw + i * kGroupStep * 8 * kDim);
                // the next copy into this slot writes through another proxy than these reads: without the fence it
                // could land before them
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(raw_empty + 8 * slot);
                if (state == 0) {  // tokens past the end, or without a page, are zeros
#pragma unroll
                    for (int i = 0; i < kRounds; ++i) {
                        const int t = nth * kPiece<kDim> + (group0 + i * kGroupStep) * 8 + t8;
                        if ((t & 15) >= info.there[t >> 4]) x[i] = make_uint4(0, 0, 0, 0);
                    }
                }
                if (nth == 0) {
                    ok = __all_sync(0xFFFFFFFFu, wait_suspended((part == 0 ? k_empty : v_empty) + 8 * st, eph, wc, kSiteConvEmpty));
                    if (!ok) break;
                }
                const uint32_t base = sbase + (part < kPieces<kDim> ? L::kK : L::kV) + st * L::kTile + nth * kPiece<kDim> * 128 + put;
#pragma unroll
                for (int i = 0; i < kRounds; ++i) {
                    uint32_t h[8];
                    codes_to_half<kFmt>(x[i].x, h[0], h[1]);
                    codes_to_half<kFmt>(x[i].y, h[2], h[3]);
                    codes_to_half<kFmt>(x[i].z, h[4], h[5]);
                    codes_to_half<kFmt>(x[i].w, h[6], h[7]);
                    sts_v4(base + put0 + i * kGroupStep * 8 * 128, make_uint4(h[0], h[1], h[2], h[3]));
                    sts_v4(base + put1 + i * kGroupStep * 8 * 128, make_uint4(h[4], h[5], h[6], h[7]));
                }
                if (nth == kPieces<kDim> - 1) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive((part < kPieces<kDim> ? k_full : v_full) + 8 * st);
                }
            }
            ++tile_no;
        }
    } else {
        // ------------------------------------------------------------ softmax, Q and the result
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        const int h = warp >> 3, kh = (warp >> 2) & 1;                // rows' half, keys' half
        const int row = (warp & 3) * 32 + lane;                       // of the half: its TMEM lane
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t col_s = lanes + kColS + 128 * h + 64 * kh, col_o = lanes + kColO + kDim * h + kh * (kDim / 2);
        const uint32_t col_p = kScoresAhead<kDim> ? lanes + kColP + 64 * h + 32 * kh : col_s;
        const int pair = h * 4 + (warp & 3);                          // the two warps of the same 32 rows
        float* red = reinterpret_cast<float*>(smem + L::kRed) + (h * 2) * kHalfRows + row;  // + parity 4 * 128, + key half 128
        bool ok = true;
        bool first_segment = true;
        while (true) {
            // all of the half go on, or none: no warp waits at a barrier for one that has left
            if (named_barrier_or(1 + h, 256, !next_segment(sg))) break;
            if (first_segment && threadIdx.x == 0) a.meta[k] = Meta{start - sg.t0, total, sg.t0 > 0 ? sg.tiles : 0, sg.head, sg.block, sg.first, sg.count, 0};
            const int r = sg.block * kRows + h * kHalfRows + row;      // row of the (sequence, kv head)
            const bool real = r < sg.count * a.share;
            const int t = r / a.share;
            // Q: fp16 as it is; bf16 moved by a power of two so that the row's largest value lies in
            // [2^14, 2^15). A negative scale goes into Q, so that larger products mean larger weights.
            float f = fabsf(c.scale) * kLog2e;
            {
                const E* x = static_cast<const E*>(c.q.p) + static_cast<int64_t>(sg.first + t) * c.q.token + (sg.head * a.share + r - t * a.share) * c.q.head;
                float up = c.scale < 0.0f ? -1.0f : 1.0f;
                if constexpr (!std::is_same<E, __half>::value) {
                    float most = 0.0f;
                    if (real) {
#pragma unroll 4
                        for (int d = 0; d < kDim; d += 8) {
                            float v[8];
                            load_values<E, 8>(x, d, a.q_vec != 0, v);
#pragma unroll
                            for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(v[e]));
                        }
                    }
                    const int e = most > 0.0f && most <= 3.3895314e38f ? max(-100, (__float_as_int(most) >> 23) - 127) : 14;
                    up *= __int_as_float((14 - e + 127) << 23);
                    f *= __int_as_float((e - 14 + 127) << 23);
                }
                if (kParts && std::is_same<E, __half>::value && c.scale >= 0.0f && a.q_vec != 0) {
                    // no arithmetic: the warp's 32 half rows, several lanes a row, all reads at once (a row a lane takes half of each
                    // sector at a time, and twice as long)
                    constexpr int kPieces = kDim / 16, kRowsAtOnce = 32 / kPieces;
                    const int piece = lane % kPieces, row0 = (warp & 3) * 32 + lane / kPieces;
                    uint4 w[kPieces];
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        const int rr = sg.block * kRows + h * kHalfRows + row0 + i * kRowsAtOnce, tt = rr / a.share;
                        w[i] = make_uint4(0, 0, 0, 0);
                        if (rr < sg.count * a.share)
                            w[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const E*>(c.q.p) + static_cast<int64_t>(sg.first + tt) * c.q.token +
                                                                       (sg.head * a.share + rr - tt * a.share) * c.q.head + kh * (kDim / 2)) + piece);
                    }
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        const int d = kh * (kDim / 2) + piece * 8, to = row0 + i * kRowsAtOnce;
                        sts_v4(sbase + L::kQ + h * L::kTile + to * 128 + (d >> 6) * L::kBox + ((((d & 63) >> 3) ^ (to & 7)) << 4), w[i]);
                    }
                } else
#pragma unroll 4
                for (int i = 0; i < kDim / 2; i += 8) {
                    const int d = kh * (kDim / 2) + i;
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
                    if (real) load_values<E, 8>(x, d, a.q_vec != 0, v);
                    const uint4 w = make_uint4(half2_bits(v[0] * up, v[1] * up), half2_bits(v[2] * up, v[3] * up),
                                               half2_bits(v[4] * up, v[5] * up), half2_bits(v[6] * up, v[7] * up));
                    sts_v4(sbase + L::kQ + h * L::kTile + (d >> 6) * L::kBox + row * 128 + ((((d & 63) >> 3) ^ (row & 7)) << 4), w);
                }
            }
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full + 8 * h);
            int to = sg.len, from = 0;
            {
                const int64_t p = static_cast<int64_t>(sg.len) - sg.count + min(t, sg.count - 1);
                if (c.causal) to = static_cast<int>(min(static_cast<int64_t>(sg.len), p + 1));
                if (c.window > 0 && p - c.window + 1 > 0) from = static_cast<int>(p - c.window + 1);
            }
            float m = kNoMax, l = 0.0f;
            const int n = sg.t1 - sg.t0;
            for (int j = 0; j < n; ++j) {
                const uint32_t g = tile_no + j, ph = g & 1u;
                // a wait that gave up still reaches the barrier of the maxima, where both warps learn of it
                ok = wait_suspended(info_full + 8 * (g % kInfoSlots), (g / kInfoSlots) & 1u, wc, kSiteEpilogueAccFull) &&
                     wait_suspended(s_full + 8 * h, ph, wc, kSiteEpilogueAccFull);
                __syncwarp();
                tc_fence_after_sync();
                const TileInfo& info = infos[g % kInfoSlots];
                // keys key0 .. key0 + 63; a tile that some row of the warp does not see whole is masked
                const int key0 = (sg.tile0 + sg.t0 + j) * kKeys + 64 * kh, lo = from - key0, hi = to - key0;
                const bool edge = __any_sync(0xFFFFFFFFu, lo > 0 || hi < 64);
                // this half's maximum, block by block, then the row's. The scores are read twice, 32 at a
                // time, in loops: the code stays small and the registers few
                float top = kNoMax;
                float xs[2][32];
                tmem_ld_32x32b_x32(col_s, reinterpret_cast<uint32_t(&)[32]>(xs[0]));
                tmem_ld_32x32b_x32(col_s + 32, reinterpret_cast<uint32_t(&)[32]>(xs[1]));
                tmem_ld_wait();
                if constexpr (kScoresAhead<kDim>) {
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_read + 8 * h);
                }
                if (edge) {
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i < lo - 32 * q || i >= hi - 32 * q) xs[q][i] = -INFINITY;
                }
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float (&x)[32] = xs[q];
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const float* y = x + 16 * b;
                        const float u = max3(max3(y[0], y[1], y[2]), max3(y[3], y[4], y[5]), max3(y[6], y[7], y[8]));
                        const float v = max3(max3(y[9], y[10], y[11]), max3(y[12], y[13], y[14]), y[15]);
                        top = fmaxf(top, fmaf(fmaxf(u, v), max_nan(f * info.ks[4 * kh + 2 * q + b], 1e-38f), info.lv[4 * kh + 2 * q + b]));
                    }
                }
                red[ph * 4 * kHalfRows + kh * kHalfRows] = top;
                if (named_barrier_or(3 + pair, 64, !ok)) {
                    ok = false;
                    break;
                }
                top = fmaxf(top, red[ph * 4 * kHalfRows + (kh ^ 1) * kHalfRows]);
                float keep = 1.0f;
                bool grew = false;
                if (top > m + kMostLog2) {
                    keep = ex2_approx(m - (top - kHeadroomLog2));
                    m = top - kHeadroomLog2;
                    grew = true;
                }
                float sum = 0.0f;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float2 (&x)[16] = reinterpret_cast<float2(&)[16]>(xs[q]);
                    // pair by pair, in place: while the exponential unit takes a pair, the next one is scaled
                    // and the one before the last is summed and rounded
                    uint32_t w[16];
                    float2 part[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                    float2 cb[2], ob[2];
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const float cc = max_nan(f * info.ks[4 * kh + 2 * q + b], 1e-38f), oo = info.lv[4 * kh + 2 * q + b] - m;
                        cb[b] = make_float2(cc, cc);
                        ob[b] = make_float2(oo, oo);
                    }
#pragma unroll
                    for (int e = 0; e < 20; ++e) {
                        if (e < 16) x[e] = __ffma2_rn(x[e], cb[e >> 3], ob[e >> 3]);
                        if (e >= 2 && e < 18) {
                            x[e - 2].x = ex2_approx(x[e - 2].x);
                            x[e - 2].y = ex2_approx(x[e - 2].y);
                        }
                        if (e >= 4) {
                            w[e - 4] = half2_bits(x[e - 4].x, x[e - 4].y);
                            part[(e - 4) >> 3] = __fadd2_rn(part[(e - 4) >> 3], x[e - 4]);
                        }
                    }
#pragma unroll
                    for (int b = 0; b < 2; ++b) sum = fmaf(part[b].x + part[b].y, info.iv[4 * kh + 2 * q + b], sum);
                    // the product of the tile before has completed (its weights lie here, and its outputs are there) where this tile's
                    // scores were issued after it; where they were computed ahead it is waited for (a wait that gives up is
                    // told by the next one, at the latest at the segment's end)
                    if (kScoresAhead<kDim> && q == 0 && j > 0) {
                        wait_suspended(o_done + 8 * h, (g - 1) & 1u, wc, kSiteEpilogueAccFull);
                        __syncwarp();
                        tc_fence_after_sync();
                    }
                    tmem_st_x16(col_p + 16 * q, w);
                    // the outputs so far come to the new maximum before the first weights are handed over
                    if (q == 0 && j > 0 && __any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll 1
                        for (int d = 0; d < kDim / 2; d += 32) {
                            uint32_t o[32];
                            tmem_ld_32x32b_x32(col_o + d, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                            tmem_st_32x32b_x32(col_o + d, o);
                        }
                    }
                    tmem_st_wait();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full + 16 * h + 8 * q);
                }
                l = l * keep + sum;
            }
            // Every warp of the half comes to the barrier at the segment's end once, whatever became of its waits, and
            // all leave together: the others may have taken their last tile before this one saw the abort flag,
            // and the barrier has no limit of its own.
            if (!ok) {
                named_barrier_or(1 + h, 256, true);
                break;
            }
            tile_no += n;
            ok = wait_suspended(o_done + 8 * h, (tile_no - 1) & 1u, wc, kSiteEpilogueAccFull);
            // both key halves' sums; the maxima of the last tile were in the other parity
            red[(tile_no & 1u) * 4 * kHalfRows + kh * kHalfRows] = l;
            if (named_barrier_or(1 + h, 256, !ok)) break;
            l += red[(tile_no & 1u) * 4 * kHalfRows + (kh ^ 1) * kHalfRows];
            tc_fence_after_sync();
            const bool whole = sg.t0 == 0 && sg.t1 == sg.tiles;
            const int64_t out_row = static_cast<int64_t>(sg.first + t) * c.heads + sg.head * a.share + r - t * a.share;
            float* part = a.parts + (static_cast<int64_t>(2 * k) + (first_segment ? 0 : 1)) * kRows * (kDim + 2);
            const int pr = h * kHalfRows + row;
            // the first call's share of the row: what it counts for, and this one's
            float keep = 1.0f, more = 0.0f;
            bool write = real;
            if (kParts && whole) {
                wait_for_first();
                if (real) {
                    const float2 w = c.seed_weight[out_row];
                    const float top = fmaxf(m, w.x);
                    write = !(w.y < 0.0f);
                    keep = ex2_approx(m - top);
                    more = ex2_approx(w.x - top);
                    l = fmaf(l, keep, w.y * more);
                    m = top;
                }
            }
            const float inv = row_inverse(l);
#pragma unroll 1
            for (int i = 0; i < kDim / 2; i += 32) {
                const int d = kh * (kDim / 2) + i;
                uint32_t o[32];
                __syncwarp();
                tmem_ld_32x32b_x32(col_o + i, o);
                tmem_ld_wait();
                if (write && whole) {
                    E* y = static_cast<E*>(c.out) + out_row * kDim + d;
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float v[8];
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            v[x] = __uint_as_float(o[e + x]);
                            if constexpr (kParts) v[x] = fmaf(v[x], keep, c.seed[out_row * kDim + d + e + x] * more);
                            v[x] *= inv;
                        }
                        store_values<E, 8>(y, e, true, v);
                    }
                } else if (real && !whole) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<uint4*>(part + part_offset<kDim>(pr, d + e)) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
            }
            if (write && whole && kh == 0 && c.lse != nullptr) c.lse[out_row] = row_lse(m, l);
            if (real && !whole && kh == 0) {
                part[kRows * kDim + pr] = m;
                part[kRows * (kDim + 1) + pr] = l;
            }
            first_segment = false;
        }
    }
    if constexpr (kParts) wait_for_first();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 20) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

int64_t meta_bytes(int grid) { return (static_cast<int64_t>(grid) * sizeof(Meta) + 255) / 256 * 256; }

// kParts: the second of two calls.
template <typename E, int kFmt, int kDim, bool kParts>
cudaError_t launch(const KvAttnCall& c, const CUtensorMap& tmK, const CUtensorMap& tmV, void* workspace, int sm_count, cudaStream_t stream) {
    static int attr_gen[64] = {};
    auto* kernel = attn_tile_kernel<E, kFmt, kDim, kParts>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && attr_gen[dev] != g_generation) {
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<kDim>::kAlloc)) != cudaSuccess) return e;
        // the register split draws on what the launch reserves: never more than that
        cudaFuncAttributes fa{};
        if ((e = cudaFuncGetAttributes(&fa, kernel)) != cudaSuccess) return e;
        if (fa.numRegs < kRegs) return cudaErrorInvalidConfiguration;
        attr_gen[dev] = g_generation;
    }
    SplitWork a{};
    a.c = c;
    a.share = c.heads / c.cache.kv_heads;
    a.least = 2;
    a.grid = sm_count;
    a.joined = c.max_len > kKeys;
    a.box = kv_attn_tile_box(c);
    a.q_vec = reinterpret_cast<uintptr_t>(c.q.p) % 16 == 0 && c.q.token % 8 == 0 && c.q.head % 8 == 0;
    a.meta = static_cast<Meta*>(workspace);
    a.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + meta_bytes(a.grid));
    while (c.cache.page >> (a.page_shift + 1)) ++a.page_shift;
    if ((e = launch_attn(kernel, a, tmK, tmV, a.grid, kThreads, Smem<kDim>::kAlloc, stream)) != cudaSuccess || !a.joined) return e;
    return launch_join<E, kDim, kRows, kParts>(a, stream);
}

}  // namespace

// As many as lie together, up to a piece: a warp issues a copy in 130 cycles, and 16 of them a tile take longer than its products.
int kv_attn_tile_box(const KvAttnCall& c) { return std::min<int>(c.cache.page, 8192 / c.cache.dim); }

int64_t kv_attn_tile_workspace(const KvAttnCall& c, int sm_count) {
    return meta_bytes(sm_count) + static_cast<int64_t>(sm_count) * 2 * kRows * (c.cache.dim + 2) * 4;
}

cudaError_t launch_kv_attn_tile(const KvAttnCall& c, const CUtensorMap& tmK, const CUtensorMap& tmV, void* workspace, int sm_count,
                                cudaStream_t stream) {
    const bool h = c.dtype == kFp16, e4 = c.cache.fmt == kKvE4M3, d128 = c.cache.dim == 128;
    auto go = [&](auto* f) { return f(c, tmK, tmV, workspace, sm_count, stream); };
    auto one = [&](auto parts) {
        constexpr bool kParts = decltype(parts)::value;
        if (h && e4) return d128 ? go(launch<__half, kKvE4M3, 128, kParts>) : go(launch<__half, kKvE4M3, 64, kParts>);
        if (h) return d128 ? go(launch<__half, kKvInt8, 128, kParts>) : go(launch<__half, kKvInt8, 64, kParts>);
        if (e4) return d128 ? go(launch<__nv_bfloat16, kKvE4M3, 128, kParts>) : go(launch<__nv_bfloat16, kKvE4M3, 64, kParts>);
        return d128 ? go(launch<__nv_bfloat16, kKvInt8, 128, kParts>) : go(launch<__nv_bfloat16, kKvInt8, 64, kParts>);
    };
    return c.seed != nullptr ? one(std::true_type{}) : one(std::false_type{});
}

}  // namespace tg
