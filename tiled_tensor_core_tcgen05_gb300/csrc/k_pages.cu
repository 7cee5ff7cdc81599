// Pages of the 8-bit cache: copied, shared among sequences that continue the
// same one (forked), given and freed, and moved together (compacted).
//
// The bookkeeping (which entries a page is held by, which pages are free, the
// tables) is up to a few hundred kilobytes of integers in several steps that each
// need the whole of the one before. One CTA, or a cluster of kMostCtas where there is
// much (kLittleFork), does all of them, with its barrier between the steps: no launch and
// no host in between, and no CTA waits for one that might not run. Then a grid that
// fills the GPU copies the pages that were listed; it is launched early and
// waits for the list. Free pages are taken in rising order and given in the
// order of sequences and places, by prefix sums, so results do not depend on
// timing.
//
// Measured on a GB300, kernels alone: four beams of one prompt forked 11.2 us and 256 of 32 prompts of up to 8192 tokens 24.9
// (steps that wait for one another: table rows, counts, prefix sums; the bytes take 3); compacting a pool of 301 pages 7.3, one of
// 16384 pages of 128 KB that is 55 % full 177 (157 at the rate of a plain copy); copying 5003 such pages 202 (193).
#include <algorithm>
#include <climits>
#include <type_traits>

#include "tg_device.cuh"
#include "tg_kv.cuh"

namespace tg {
namespace {

constexpr int kMostCtas = 8;      // of the cluster (the portable most)
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kSeg = 256;         // entries of a table's row that a warp takes at a time

// All threads of the cluster: a block's barrier where it is a single CTA.
template <int kCtas>
__device__ __forceinline__ void meet() {
    if constexpr (kCtas == 1) __syncthreads();
    else cluster_sync();
}

// What other CTAs of the cluster have written: past the first-level cache.
__device__ __forceinline__ int fresh(const int* p) { return __ldcg(p); }

// Sum of a number a thread: over the threads before this one (ranks, warps, lanes), and over the whole cluster.
struct Order {
    int64_t before, total;
};

// All threads. Every CTA writes its sum into the others' `box` (a call's own; every CTA must be known to run); the
// cluster's barrier is inside.
template <int kCtas>
__device__ __forceinline__ Order cluster_order(int mine, int64_t* box, int* warps, uint32_t rank) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = x;
    __syncthreads();
    int low = 0, sum = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) low += warps[w];
        sum += warps[w];
    }
    if (threadIdx.x < kCtas) {  // this CTA's sum into every CTA's box
        const uint32_t to = mapa_shared(smem_u32(box + rank), threadIdx.x);
        asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(to), "l"(static_cast<int64_t>(sum)) : "memory");
    }
    meet<kCtas>();
    Order o{low + x - mine, 0};
    for (uint32_t r = 0; r < kCtas; ++r) {
        if (r < rank) o.before += box[r];
        o.total += box[r];
    }
    return o;
}

// A thread's `pages` are places first .. last - 1: contiguous, thread after thread in the order of Order.
struct Range {
    int first, last;
    __device__ Range(int64_t n, int t, int all) {
        const int64_t each = (n + all - 1) / all;
        first = static_cast<int>(min(n, each * t));
        last = static_cast<int>(min(n, each * (t + 1)));
    }
};

// Entries of a table's rows, a warp at a time kSeg of one row: f(row, place, what `of` says of the row).
template <int kAll, typename G, typename F>
__device__ __forceinline__ void for_entries(int rows, int64_t width, int t, G of, F f) {
    const int64_t segs = (width + kSeg - 1) / kSeg;
    for (int64_t s = t / 32; s < rows * segs; s += kAll / 32) {
        const int row = static_cast<int>(s / segs);
        const int64_t base = (s - row * segs) * kSeg;
        const auto x = of(row);
#pragma unroll
        for (int i = 0; i < kSeg / 32; ++i) {
            const int64_t at = base + i * 32 + (t & 31);
            if (at < width) f(row, static_cast<int>(at), x);
        }
    }
}

// ---------------------------------------------------------------- forking

// A parent that is there, or -1 (reported where it is no sequence of the call).
__device__ __forceinline__ int parent_of(const KvForkCall& c, int i) {
    const int p = c.parents != nullptr ? __ldg(c.parents + i) : i;
    if (p < 0) return -1;
    if (p >= c.batch) {
        report_range(c.wd);
        return -1;
    }
    return p;
}

// What the steps of a fork leave for one another: in the workspace, or for a single CTA in its shared memory.
template <int kCtas>
__device__ __forceinline__ int left(const int* p) {
    if constexpr (kCtas == 1) return *p;
    else return fresh(p);
}

// A child's pages: entries below `start` come from its parent, those up to `end` are new.
struct Child {
    int parent, len, start, end;
    int source;  // page whose tokens go to the first new one, or -1
};

template <int kCtas>
__device__ __forceinline__ Child child_of(const KvForkCall& c, const ForkWork& w, int i, bool tell) {
    Child x{parent_of(c, i), 0, 0, 0, -1};
    if (x.parent >= 0) {
        x.len = left<kCtas>(w.lens + x.parent);
        const int full = x.len >> c.page_shift;
        x.start = left<kCtas>(w.first + x.parent) == i ? left<kCtas>(w.kept + x.parent) : full;
        if ((x.len & (c.cache.page - 1)) && x.start == full) x.source = __ldg(c.table + x.parent * c.width + full);
    }
    const int64_t want = (x.len + c.room + c.cache.page - 1) >> c.page_shift;
    if (want > c.width && tell) report_range(c.wd);
    x.end = max(x.start, static_cast<int>(min(want, c.width)));
    return x;
}

template <int kCtas>
__global__ void __launch_bounds__(kThreads, 1) fork_kernel(const KvForkCall c) {
    constexpr int kAll = kCtas * kThreads;
    __shared__ int64_t box[2][kCtas];
    __shared__ int warps[kWarps];
    __shared__ int64_t carry, needs[kWarps];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t rank = cluster_ctarank();
    const int t = rank * kThreads + threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int page = c.cache.page;
    const int64_t pages = c.cache.pages;
    ForkWork w = c.w;
    int32_t* refs = c.refs_out;
    if constexpr (kCtas == 1) {
        extern __shared__ int64_t held_here[];
        w.place = held_here;
        w.children = reinterpret_cast<int*>(held_here + c.count);
        w.first = w.children + c.batch;
        w.held = w.first + c.batch;
        w.lens = w.held + c.batch;
        w.kept = w.lens + c.batch;
        w.need = w.kept + c.batch;
        refs = w.need + c.count;
        w.given = refs + pages;
    }

    for (int64_t p = t; p < pages; p += kAll) refs[p] = __ldg(c.refs + p);
    for (int j = t; j < c.batch; j += kAll) {
        w.children[j] = 0;
        w.first[j] = INT_MAX;
        w.held[j] = static_cast<int>(c.width);
    }
    meet<kCtas>();
    // children of each sequence, and the first of them; its pages are the entries before the first that is none
    for (int i = t; i < c.count; i += kAll) {
        const int p = parent_of(c, i);
        if (p < 0) continue;
        atomicAdd(w.children + p, 1);
        atomicMin(w.first + p, i);
    }
    for_entries<kAll>(c.batch, c.width, t, [](int) { return 0; }, [&](int j, int at, int) {
        const int p = __ldg(c.table + j * c.width + at);
        if (p >= 0 && p < pages) return;
        if (p >= 0) report_range(c.wd);
        atomicMin(w.held + j, at);
    });
    meet<kCtas>();
    // the entries that the first child takes over: the full pages, and open ones that no other sequence holds
    for (int j = t; j < c.batch; j += kAll) {
        const int held = left<kCtas>(w.held + j);
        int len = __ldg(c.lens + j);
        if (len < 0 || len > static_cast<int64_t>(held) * page) {
            report_range(c.wd);
            len = 0;
        }
        int kept = len >> c.page_shift;
        while (kept < held && __ldg(c.refs + __ldg(c.table + j * c.width + kept)) == 1) ++kept;
        w.lens[j] = len;
        w.kept[j] = kept;
    }
    meet<kCtas>();
    // entries that come and go; a page that tokens are copied from is let go of after the free ones have been
    // counted, so that it is not given away in the same call
    struct Old {
        int held, children, len, kept;
    };
    for_entries<kAll>(
        c.batch, c.width, t, [&](int j) { return Old{left<kCtas>(w.held + j), left<kCtas>(w.children + j), left<kCtas>(w.lens + j), left<kCtas>(w.kept + j)}; },
        [&](int j, int at, const Old& x) {
            if (at >= x.held) return;
            const int full = x.len >> c.page_shift, d = at < full ? x.children - 1 : at < x.kept && x.children > 0 ? 0 : -1;
            if (d == 0 || (at == full && at >= x.kept && x.children > 0 && (x.len & (page - 1)))) return;
            atomicAdd(refs + __ldg(c.table + j * c.width + at), d);
        });
    for_entries<kAll>(c.count, c.width, t, [&](int i) { return child_of<kCtas>(c, w, i, false); }, [&](int i, int at, const Child& x) {
        c.table_out[i * c.width + at] = at < x.start ? __ldg(c.table + x.parent * c.width + at) : -1;
    });
    for (int i = t; i < c.count; i += kAll) {
        const Child x = child_of<kCtas>(c, w, i, true);
        c.lens_out[i] = x.len;
        w.need[i] = x.end - x.start;
    }
    meet<kCtas>();
    // where each child's new pages begin in the list of all of them: every CTA by itself. In 64 bits: a child may ask for 2^27 pages,
    // whatever there are
    if (threadIdx.x == 0) carry = 0;
    for (int base = 0; base < c.count; base += kThreads) {
        const int i = base + threadIdx.x;
        const int64_t n = i < c.count ? left<kCtas>(w.need + i) : 0;
        int64_t x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) needs[warp] = x;
        __syncthreads();
        int64_t before = carry, sum = 0;
        for (int k = 0; k < kWarps; ++k) {
            if (k < warp) before += needs[k];
            sum += needs[k];
        }
        if (rank == 0 && i < c.count) w.place[i] = before + x - n;
        __syncthreads();
        if (threadIdx.x == 0) carry += sum;
    }
    __syncthreads();
    const int64_t wanted = carry;
    // the free pages, in rising order
    const Range r(pages, t, kAll);
    int mine = 0;
    for (int p = r.first; p < r.last; ++p) mine += left<kCtas>(refs + p) == 0;
    const Order o = cluster_order<kCtas>(mine, box[0], warps, rank);
    int64_t k = o.before;
    for (int p = r.first; p < r.last && k < wanted; ++p)
        if (left<kCtas>(refs + p) == 0) {
            w.given[k++] = p;
            refs[p] = 1;
        }
    if (t == 0) *c.spare = static_cast<int>(max(o.total - wanted, static_cast<int64_t>(INT_MIN)));
    meet<kCtas>();
    for (int i = t / 32; i < c.count; i += kAll / 32) {
        const Child x = child_of<kCtas>(c, w, i, false);
        const int64_t place = kCtas == 1 ? w.place[i] : __ldcg(w.place + i);
        for (int at = x.start + lane; at < x.end; at += 32) {
            const int64_t g = place + at - x.start;
            c.table_out[i * c.width + at] = g < o.total ? left<kCtas>(w.given + g) : -1;
        }
        if (lane == 0) {
            const bool copied = x.source >= 0 && x.end > x.start && place < o.total;
            w.items[i] = PageItem{x.source, copied ? left<kCtas>(w.given + place) : 0, copied ? x.len & (page - 1) : 0};
        }
    }
    for (int j = t; j < c.batch; j += kAll) {
        const int len = left<kCtas>(w.lens + j), full = len >> c.page_shift;
        if ((len & (page - 1)) && left<kCtas>(w.kept + j) == full && left<kCtas>(w.children + j) > 0) atomicAdd(refs + __ldg(c.table + j * c.width + full), -1);
    }
    if (t == 0) *w.items_count = c.count;
    if constexpr (kCtas == 1) {
        __syncthreads();
        for (int64_t p = t; p < pages; p += kAll) c.refs_out[p] = refs[p];
    }
}

// Shared memory that a single CTA's fork needs.
int64_t fork_smem(const KvForkCall& c) {
    return c.count * 8 + (c.batch * 5ll + c.count + c.cache.pages + std::min(c.cache.pages, c.count * c.width)) * 4;
}

// ---------------------------------------------------------------- compacting

template <int kCtas>
__global__ void __launch_bounds__(kThreads, 1) compact_kernel(const KvCompactCall c) {
    constexpr int kAll = kCtas * kThreads;
    __shared__ int64_t box[3][kCtas];
    __shared__ int warps[kWarps];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t rank = cluster_ctarank();
    const int t = rank * kThreads + threadIdx.x;
    const int64_t pages = c.cache.pages;
    const Range r(pages, t, kAll);
    int mine = 0;
    for (int p = r.first; p < r.last; ++p) mine += __ldg(c.refs + p) > 0;
    meet<kCtas>();  // every CTA runs: its shared memory may be written
    const int64_t used = cluster_order<kCtas>(mine, box[0], warps, rank).total;
    int holes = 0, movers = 0;
    for (int p = r.first; p < r.last; ++p) {
        const bool held = __ldg(c.refs + p) > 0;
        holes += !held && p < used;
        movers += held && p >= used;
    }
    const Order hole = cluster_order<kCtas>(holes, box[1], warps, rank);
    const Order mover = cluster_order<kCtas>(movers, box[2], warps, rank);
    int64_t h = hole.before, m = mover.before;
    for (int p = r.first; p < r.last; ++p) {
        const int n = __ldg(c.refs + p);
        c.moved[p] = n > 0 ? p : -1;
        c.refs_out[p] = n > 0 && p < used ? n : 0;
        if (n <= 0 && p < used) c.w.items[h++].to = p;
        if (n > 0 && p >= used) c.w.items[m++].from = p;
    }
    meet<kCtas>();
    for (int64_t i = t; i < mover.total; i += kAll) {
        PageItem* x = c.w.items + i;
        const int from = fresh(&x->from), to = fresh(&x->to);
        x->tokens = c.cache.page;
        c.moved[from] = to;
        c.refs_out[to] = __ldg(c.refs + from);
    }
    if (t == 0) {
        *c.used = static_cast<int>(used);
        *c.w.items_count = static_cast<int>(mover.total);
    }
    meet<kCtas>();
    for_entries<kAll>(c.batch, c.width, t, [](int) { return 0; }, [&](int j, int at, int) {
        int p = __ldg(c.table + j * c.width + at);
        if (p >= pages) report_range(c.wd);
        c.table_out[j * c.width + at] = p >= 0 && p < pages ? fresh(c.moved + p) : -1;
    });
}

// ---------------------------------------------------------------- copying

constexpr int kCopyThreads = 256;
constexpr int kAhead = 8;  // 16-byte pieces a lane has in flight

// Items of a list: the first `tokens` tokens of page `from`, codes and scales, to page `to`. A warp takes one head
// of the keys or of the values at a time (up to 16 KB, contiguous).
template <bool kListed>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const PageCopyCall c) {
    if constexpr (kListed) asm volatile("griddepcontrol.wait;" ::: "memory");
    const int count = kListed ? *c.items_count : c.count;
    const int heads = c.from.kv_heads, page = c.from.page, lane = threadIdx.x & 31;
    const int64_t line = static_cast<int64_t>(page) * c.from.dim, parts = static_cast<int64_t>(count) * 2 * heads;
    for (int64_t s = blockIdx.x * (kCopyThreads / 32) + threadIdx.x / 32; s < parts; s += gridDim.x * (kCopyThreads / 32)) {
        const int i = static_cast<int>(s / (2 * heads)), h = static_cast<int>(s - static_cast<int64_t>(i) * 2 * heads) >> 1;
        const bool keys = (s & 1) == 0;
        PageItem x;
        if constexpr (kListed) {
            x = c.items[i];
            if (x.tokens == 0) continue;
        } else {
            x = PageItem{__ldg(c.src + i), __ldg(c.dst + i), page};
            if (x.from < 0 || x.from >= c.from.pages || x.to < 0 || x.to >= c.to.pages) {
                if (lane == 0) report_range(c.wd);
                continue;
            }
        }
        const int64_t a = static_cast<int64_t>(x.from) * heads + h, b = static_cast<int64_t>(x.to) * heads + h;
        const uint4* get = reinterpret_cast<const uint4*>((keys ? c.from.k : c.from.v) + a * line);
        uint4* put = reinterpret_cast<uint4*>((keys ? c.to.k : c.to.v) + b * line);
        const int n = x.tokens * c.from.dim / 16;
        float scale = 0.0f;
        if (lane == 0) scale = (keys ? c.from.k_scale : c.from.v_scale)[a];
        for (int base = 0; base < n; base += 32 * kAhead) {
            uint4 v[kAhead];
#pragma unroll
            for (int e = 0; e < kAhead; ++e)
                if (base + e * 32 + lane < n) v[e] = get[base + e * 32 + lane];
#pragma unroll
            for (int e = 0; e < kAhead; ++e)
                if (base + e * 32 + lane < n) put[base + e * 32 + lane] = v[e];
        }
        if (lane == 0) (keys ? c.to.k_scale : c.to.v_scale)[b] = scale;
    }
}

int copy_grid(int64_t parts, int sm_count) {
    const int64_t want = (parts + kCopyThreads / 32 - 1) / (kCopyThreads / 32), most = static_cast<int64_t>(sm_count) * 8;
    return static_cast<int>(want < most ? want : most);
}

// The copies that a cluster's kernel has listed: in place when the list is.
cudaError_t launch_listed(const KvCacheArgs& cache, const PageWork& w, int64_t most, int sm_count, cudaStream_t stream) {
    PageCopyCall c{};
    c.from = c.to = cache;
    c.items = w.items;
    c.items_count = w.items_count;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(copy_grid(most * 2 * cache.kv_heads, sm_count));
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, copy_pages_kernel<true>, c);
}

// Pages and entries up to which one CTA keeps the books: its barrier takes a fraction of the cluster's, and what the steps of a fork leave
// for one another stays in its shared memory. Measured on a GB300, in us with one CTA and with eight: forks with 200 pages and entries 11.0 and 15.6,
// 10400 15.3 and 18.0, 40000 26.9 and 22.7, 125000 51.9 and 22.0; compacting 500 7.4 and 11.7, 6200 12.3 and 14.0, 12400 23.1 and 15.9, 25000 48.7 and 18.2.
constexpr int64_t kLittleFork = 16384, kLittleCompact = 8192;
constexpr int kMostSmem = 128 * 1024;

template <typename C>
cudaError_t launch_books(void (*kernel)(const C), const C& c, int ctas, int64_t smem, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {static_cast<unsigned>(ctas), 1, 1};
    cfg.attrs = &attr;
    cfg.numAttrs = ctas > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, c);
}

int64_t up(int64_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace

int64_t kv_fork_workspace(int64_t pages, int64_t batch, int64_t count, int64_t width, ForkWork* w, void* at) {
    char* p = static_cast<char*>(at);
    int64_t n = 0;
    auto take = [&](auto*& x, int64_t many) {
        x = reinterpret_cast<std::remove_reference_t<decltype(x)>>(p + n);
        n += up(many * static_cast<int64_t>(sizeof(*x)));
    };
    take(w->items_count, 1);
    take(w->items, count);
    take(w->children, batch);
    take(w->first, batch);
    take(w->held, batch);
    take(w->lens, batch);
    take(w->kept, batch);
    take(w->need, count);
    take(w->place, count);
    take(w->given, std::min(pages, count * width));
    return n;
}

int64_t kv_compact_workspace(int64_t pages, PageWork* w, void* at) {
    w->items_count = static_cast<int*>(at);
    w->items = reinterpret_cast<PageItem*>(static_cast<char*>(at) + up(sizeof(int)));
    return up(sizeof(int)) + up((pages / 2 + 1) * static_cast<int64_t>(sizeof(PageItem)));  // as many pages move as there are holes
}

cudaError_t launch_kv_copy(const PageCopyCall& c, int sm_count, cudaStream_t stream) {
    copy_pages_kernel<false><<<copy_grid(static_cast<int64_t>(c.count) * 2 * c.from.kv_heads, sm_count), kCopyThreads, 0, stream>>>(c);
    return cudaGetLastError();
}

cudaError_t launch_kv_fork(const KvForkCall& c, int sm_count, cudaStream_t stream) {
    const int64_t smem = fork_smem(c);
    cudaError_t e;
    if (c.cache.pages + (c.batch + c.count) * c.width <= kLittleFork && smem <= kMostSmem) {
        static int attr_gen[64] = {};
        int dev = 0;
        if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
        if (dev < 64 && attr_gen[dev] != g_generation) {
            if ((e = cudaFuncSetAttribute(fork_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem)) != cudaSuccess) return e;
            attr_gen[dev] = g_generation;
        }
        e = launch_books(fork_kernel<1>, c, 1, smem, stream);
    } else {
        e = launch_books(fork_kernel<kMostCtas>, c, kMostCtas, 0, stream);
    }
    return e != cudaSuccess || c.count == 0 || c.cache.pages == 0 ? e : launch_listed(c.cache, c.w, c.count, sm_count, stream);
}

cudaError_t launch_kv_compact(const KvCompactCall& c, int sm_count, cudaStream_t stream) {
    const cudaError_t e = c.cache.pages + c.batch * c.width <= kLittleCompact ? launch_books(compact_kernel<1>, c, 1, 0, stream) : launch_books(compact_kernel<kMostCtas>, c, kMostCtas, 0, stream);
    return e != cudaSuccess || c.cache.pages < 2 ? e : launch_listed(c.cache, c.w, c.cache.pages / 2, sm_count, stream);
}

}  // namespace tg
