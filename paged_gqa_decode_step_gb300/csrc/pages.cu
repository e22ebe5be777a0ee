// Bookkeeping of a paged cache on the device: rows that continue, fork, start
// anew, grow or give room back (update), and the pages in use moved to the
// lowest ids (compact).  The table part runs as one cluster, so that its
// phases are separated by cluster barriers (about a microsecond) and not by
// launches; the page data is copied by a second launch that works through a
// job list.
//
// update.  refs[x] counts the holders of page x: the rows whose first
// ceil(length / 64) entries name it, and holders outside the table (pins).
// Row r keeps the first keep = min(lengths[parent], new length) positions of
// its parent.  Full pages are shared.  A partly filled last page ("tail") is
// shared by rows that write no further, and needs one owner where a row will
// write into it: if every holder wants to write, the lowest such row keeps the
// page and the others copy its first keep % 64 positions, else all writers
// copy.  Fresh pages are the lowest free ids in order of (row, page); a page
// that no row holds any more is free at once.  A copy's source always stays
// in use, so a fresh page is never a source, and the copies need no order.
//
// compact.  With n pages in use, the k-th page in use of those >= n goes to
// the k-th free id below n: sources lie above n, targets below it.
//
// Everything is checked before anything is written: an error leaves table,
// counts and pools as they were.
#include <climits>

#include "internal.h"

namespace pdattn {
namespace {

constexpr int kPageCtas = 8;         // one cluster of the portable size
constexpr int kPageThreads = 1024;
constexpr int kAllThreads = kPageCtas * kPageThreads;

// Counters at PagesArgs::L.info: the phases' totals.
struct PagesInfo {
    int jobs;                  // page copies listed
    int bad;                   // an error was found: nothing is written
    int live_below;            // compact: pages in use below the n-th id
    int pad;
    int count[kPageCtas];      // per CTA: free (update) or used (compact) pages of its range
};

__device__ __forceinline__ int cluster_rank() {
    int r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Every thread of the cluster; writes before it are visible after it (to loads
// that pass L1 by: __ldcg).
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ int pages_of(int positions) { return (positions + kPageSize - 1) / kPageSize; }

// Exclusive sum over the block (1024 threads); *total gets the sum.
__device__ __forceinline__ int block_excl(int v, int* s_warp, int* total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int x = v;
    #pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += o;
    }
    if (lane == 31) s_warp[w] = x;
    __syncthreads();
    if (w == 0) {
        int t = s_warp[lane];
        #pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, t, d);
            if (lane >= d) t += o;
        }
        s_warp[lane] = t;
    }
    __syncthreads();
    const int before = (w > 0 ? s_warp[w - 1] : 0) + x - v;
    *total = s_warp[31];
    __syncthreads();
    return before;
}

// CTA c's pages [page_from(c), page_from(c + 1)).
__device__ __forceinline__ int page_from(int n, int c) { return (int)((long long)n * c / kPageCtas); }

// What row r keeps: its parent, positions, and whether its tail will be
// written into.  A bad row keeps nothing (the error stops the call).
struct Kept {
    int parent, keep, full, pages;
    bool part, writes;
};

__device__ __forceinline__ bool row_kept(const PagesArgs& a, int r, Kept& k) {
    const int cap = a.pages_per_row * kPageSize;
    const int p = __ldg(a.parents + r), want = __ldg(a.new_lengths + r);
    k = {-1, 0, 0, 0, false, false};
    if (p < -1 || p >= a.rows || want < 0 || want > cap) return false;
    const int held = p >= 0 ? __ldg(a.lengths + p) : 0;
    if (held < 0 || held > cap) return false;
    k.parent = p;
    k.keep = min(held, want);
    k.full = k.keep / kPageSize;
    k.part = k.keep % kPageSize > 0;
    k.writes = want > k.keep;
    k.pages = pages_of(want);
    return true;
}

__global__ void __cluster_dims__(kPageCtas, 1, 1) __launch_bounds__(kPageThreads, 1)
    pages_update_kernel(const __grid_constant__ PagesArgs a) {
    __shared__ int s_warp[32];
    griddep_launch_dependents();
    const int cta = cluster_rank(), tid = threadIdx.x, at = cta * kPageThreads + tid;
    const int R = a.rows, W = a.pages_per_row, N = a.num_pages, cap = W * kPageSize;
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(a.ws);
    PagesInfo* info = reinterpret_cast<PagesInfo*>(a.ws + a.L.info);
    int* old = reinterpret_cast<int*>(a.ws + a.L.table);
    int2* row_at = reinterpret_cast<int2*>(a.ws + a.L.rows);
    int4* jobs = reinterpret_cast<int4*>(a.ws + a.L.jobs);
    int* held = reinterpret_cast<int*>(a.ws + a.L.a);       // rows that held the page; then its rank among free ones
    int* others = reinterpret_cast<int*>(a.ws + a.L.b);     // holders that do not write into it
    int* first = reinterpret_cast<int*>(a.ws + a.L.c);      // lowest row that does; then the list of free pages

    for (int x = at; x < N; x += kAllThreads) {
        held[x] = 0;
        others[x] = 0;
        first[x] = INT_MAX;
    }
    if (at == 0) *info = PagesInfo{};
    cluster_sync();

    // Holders, old and new.  The table is copied because a row may take over
    // the entries of one that is being written.
    auto bad = [&](int bits) {
        set_error(ctrl, bits);
        info->bad = 1;
    };
    for (long long i = at; i < (long long)R * W; i += kAllThreads) {
        const int r = (int)(i / W), c = (int)(i - (long long)r * W);
        const int len = __ldg(a.lengths + r);
        if (len < 0 || len > cap) {
            if (c == 0) bad(kErrBadPos);
        } else if (c < pages_of(len)) {
            const int x = __ldcg(a.table + i);
            old[i] = x;
            if (x < 0 || x >= N) bad(kErrBadPage);
            else atomicAdd(held + x, 1);
        }
        Kept k;
        if (!row_kept(a, r, k)) {
            if (c == 0) bad(kErrBadPos);
        } else if (k.parent >= 0 && (c < k.full || (c == k.full && k.part))) {
            const int x = __ldcg(a.table + (size_t)k.parent * W + c);
            if (x < 0 || x >= N) bad(kErrBadPage);
            else if (c == k.full && k.writes) atomicMin(first + x, r);
            else atomicAdd(others + x, 1);
        }
    }
    cluster_sync();

    // Pages: pins counted in, the free ones ranked within the CTA's range.
    const int x0 = page_from(N, cta), x1 = page_from(N, cta + 1);
    int n_free = 0;
    for (int b = x0; b < x1; b += kPageThreads) {
        const int x = b + tid;
        bool free = false;
        if (x < x1) {
            const int refs = __ldcg(a.refs + x), h = __ldcg(held + x), o = __ldcg(others + x);
            if (refs < h || refs < 0) bad(kErrBadPage);
            const int o2 = o + refs - h;
            const bool owned = o2 == 0 && __ldcg(first + x) < INT_MAX;
            free = o2 == 0 && !owned;
            others[x] = o2;
        }
        int total;
        const int rank = n_free + block_excl(free ? 1 : 0, s_warp, &total);
        if (x < x1) held[x] = free ? rank : -1;
        n_free += total;
    }
    if (tid == 0) info->count[cta] = n_free;
    cluster_sync();

    // Rows: which tails are copied, and where each row's fresh pages start.
    // Every CTA scans all rows and keeps the ones it will write.
    int need = 0;
    for (int b = 0; b < R; b += kPageThreads) {
        const int r = b + tid;
        int mine = 0, kept = 0;
        if (r < R) {
            Kept k;
            row_kept(a, r, k);
            kept = k.full + (k.part ? 1 : 0);
            if (k.part && k.writes) {
                const int x = __ldcg(a.table + (size_t)k.parent * W + k.full);
                const bool alone = x >= 0 && x < N && __ldcg(others + x) == 0 && __ldcg(first + x) == r;
                if (!alone) kept = k.full;
            }
            mine = k.pages - kept;
        }
        int total;
        const int start = need + block_excl(mine, s_warp, &total);
        if (r < R && r % kPageCtas == cta) row_at[r] = make_int2(kept, start);
        need += total;
    }
    int have[kPageCtas + 1];
    have[0] = 0;
    #pragma unroll
    for (int c = 0; c < kPageCtas; ++c) have[c + 1] = have[c] + __ldcg(&info->count[c]);
    const bool stop = __ldcg(&info->bad) != 0;
    if (stop || need > have[kPageCtas]) {
        // info->jobs is 0: nothing is copied either
        if (!stop && at == 0) set_error(ctrl, kErrNoPages);
        return;
    }
    // No CTA reads first[] after this barrier, which then lists the free
    // pages by rank; none has left, as all took the same branch.
    cluster_sync();
    for (int x = x0 + tid; x < x1; x += kPageThreads) {
        const int rank = held[x];                       // this CTA's own
        if (rank < 0) {
            const int o = others[x];
            a.refs_out[x] = o == 0 ? 1 : o;             // not free at 0: one writer keeps it
        } else {
            first[have[cta] + rank] = x;
            a.refs_out[x] = have[cta] + rank < need ? 1 : 0;
        }
    }
    cluster_sync();
    const int rows_here = (R - cta + kPageCtas - 1) / kPageCtas;
    for (long long i = tid; i < (long long)rows_here * W; i += kPageThreads) {
        const int q = (int)(i / W), c = (int)(i - (long long)q * W), r = q * kPageCtas + cta;
        Kept k;
        row_kept(a, r, k);
        const int2 ra = row_at[r];
        int x = -1;
        if (c < ra.x) x = __ldcg(old + (size_t)k.parent * W + c);
        else if (c < k.pages) x = __ldcg(first + ra.y + c - ra.x);
        a.table_out[(size_t)r * W + c] = x;
        if (k.part && c == k.full && c == ra.x)         // a copied tail
            jobs[atomicAdd(&info->jobs, 1)] =
                make_int4(__ldcg(old + (size_t)k.parent * W + c), x, k.keep % kPageSize, 0);
    }
}

__global__ void __cluster_dims__(kPageCtas, 1, 1) __launch_bounds__(kPageThreads, 1)
    pages_compact_kernel(const __grid_constant__ PagesArgs a) {
    __shared__ int s_warp[32];
    griddep_launch_dependents();
    const int cta = cluster_rank(), tid = threadIdx.x, at = cta * kPageThreads + tid;
    const int R = a.rows, W = a.pages_per_row, N = a.num_pages, cap = W * kPageSize;
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(a.ws);
    PagesInfo* info = reinterpret_cast<PagesInfo*>(a.ws + a.L.info);
    int4* jobs = reinterpret_cast<int4*>(a.ws + a.L.jobs);
    int* rank = reinterpret_cast<int*>(a.ws + a.L.a);       // of a page in use among its CTA's; ~rank of a free one
    int* holes = reinterpret_cast<int*>(a.ws + a.L.b);      // free ids below n, in order

    if (at == 0) *info = PagesInfo{};
    cluster_sync();
    auto bad = [&](int bits) {
        set_error(ctrl, bits);
        info->bad = 1;
    };
    const int x0 = page_from(N, cta), x1 = page_from(N, cta + 1);
    int n_live = 0;
    for (int b = x0; b < x1; b += kPageThreads) {
        const int x = b + tid, refs = x < x1 ? __ldcg(a.refs + x) : 0;
        if (refs < 0) bad(kErrBadPage);
        int total;
        const int q = n_live + block_excl(refs > 0 ? 1 : 0, s_warp, &total);
        if (x < x1) rank[x] = refs > 0 ? q : ~q;
        n_live += total;
    }
    if (tid == 0) info->count[cta] = n_live;
    for (long long i = at; i < (long long)R * W; i += kAllThreads) {
        const int r = (int)(i / W), c = (int)(i - (long long)r * W);
        const int len = __ldg(a.lengths + r);
        if (len < 0 || len > cap) {
            if (c == 0) bad(kErrBadPos);
        } else if (c < pages_of(len)) {
            const int x = __ldcg(a.table + i);
            if (x < 0 || x >= N || __ldcg(a.refs + x) <= 0) bad(kErrBadPage);
        }
    }
    cluster_sync();
    if (__ldcg(&info->bad) != 0) return;                // the same for every CTA: no barrier is left waiting
    int before = 0, n = 0;
    #pragma unroll
    for (int c = 0; c < kPageCtas; ++c) {
        const int k = __ldcg(&info->count[c]);
        before += c < cta ? k : 0;
        n += k;
    }
    for (int x = x0 + tid; x < x1; x += kPageThreads) {
        const int q = rank[x], up = before + (q < 0 ? ~q : q);      // pages in use below x
        if (x == n) info->live_below = up;
        if (q < 0 && x < n) holes[x - up] = x;
    }
    cluster_sync();
    const int below = n < N ? __ldcg(&info->live_below) : n;
    for (int x = x0 + tid; x < x1; x += kPageThreads) {
        const int q = rank[x], up = before + (q < 0 ? ~q : q);
        int to = q < 0 ? -1 : x;
        if (q >= 0 && x >= n) {
            to = __ldcg(holes + up - below);
            jobs[up - below] = make_int4(x, to, kPageSize, 0);
            a.refs_out[to] = __ldcg(a.refs + x);
            a.refs_out[x] = 0;
        } else if (q >= 0) {
            if (a.refs_out != a.refs) a.refs_out[x] = __ldcg(a.refs + x);
        } else if (x >= n) {
            a.refs_out[x] = 0;
        }
        a.map[x] = to;
    }
    if (at == 0) info->jobs = n - below;
    cluster_sync();
    for (long long i = at; i < (long long)R * W; i += kAllThreads) {
        const int r = (int)(i / W), c = (int)(i - (long long)r * W);
        const int x = __ldcg(a.table + i);
        a.table_out[i] = c < pages_of(__ldg(a.lengths + r)) ? __ldcg(a.map + x) : x;
    }
}

// Copies the first `tokens` positions of page src to page dst in every pool:
// one block per (job, pool, head), a slab of at most 64 rows.
constexpr int kCopyThreads = 256;
constexpr int kCopyAhead = 4;

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ PoolList pools,
                                                                  const PagesInfo* info, const int4* jobs) {
    griddep_wait();
    const long long items = (long long)__ldcg(&info->jobs) * pools.slabs;
    for (long long item = blockIdx.x; item < items; item += gridDim.x) {
        const int4 job = __ldcg(jobs + item / pools.slabs);
        int slab = (int)(item % pools.slabs), lo = 0, hi = pools.n - 1;
        while (lo < hi) {                               // the pool that holds this slab
            const int mid = (lo + hi + 1) / 2;
            if (pools.first[mid] <= slab) lo = mid;
            else hi = mid - 1;
        }
        const int heads = (lo + 1 < pools.n ? pools.first[lo + 1] : pools.slabs) - pools.first[lo];
        const int row = pools.row_bytes[lo];
        slab -= pools.first[lo];
        char* base = static_cast<char*>(pools.data[lo]);
        const char* src = base + ((size_t)job.x * heads + slab) * kPageSize * row;
        char* dst = base + ((size_t)job.y * heads + slab) * kPageSize * row;
        const int bytes = job.z * row, vecs = bytes / 16;
        int v = threadIdx.x;
        for (; v + (kCopyAhead - 1) * kCopyThreads < vecs; v += kCopyAhead * kCopyThreads) {
            uint4 x[kCopyAhead];
            #pragma unroll
            for (int k = 0; k < kCopyAhead; ++k) x[k] = __ldcs(reinterpret_cast<const uint4*>(src) + v + k * kCopyThreads);
            #pragma unroll
            for (int k = 0; k < kCopyAhead; ++k) reinterpret_cast<uint4*>(dst)[v + k * kCopyThreads] = x[k];
        }
        for (; v < vecs; v += kCopyThreads) reinterpret_cast<uint4*>(dst)[v] = reinterpret_cast<const uint4*>(src)[v];
        for (int t = vecs * 16 + threadIdx.x; t < bytes; t += kCopyThreads) dst[t] = src[t];
    }
}

}  // namespace

cudaError_t launch_pages(const PagesArgs& a, bool compact, cudaStream_t stream) {
    if (compact) pages_compact_kernel<<<kPageCtas, kPageThreads, 0, stream>>>(a);
    else pages_update_kernel<<<kPageCtas, kPageThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_pages_copy(const PagesArgs& a, const PoolList& pools, int grid, bool after_plan, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = after_plan ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, pages_copy_kernel, pools, reinterpret_cast<const PagesInfo*>(a.ws + a.L.info),
                              reinterpret_cast<const int4*>(a.ws + a.L.jobs));
}

}  // namespace pdattn
