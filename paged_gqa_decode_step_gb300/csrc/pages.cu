// Bookkeeping of a paged cache on the device: rows that continue, fork, start
// anew, grow or give room back (update), and the pages in use moved to the
// lowest ids (compact).  The table's part runs as one CTA that counts in shared
// memory or, for larger tables and pools, as one cluster that counts in global
// memory, so that its phases are separated by barriers and not by launches.
// What it costs is half latency, a global round trip (0.6 us) or a cluster
// barrier (0.7 us) after another, and half issue (256 beams of 13 entries: slots
// 50 % busy; part of that is lanes without an entry).  The page data is copied
// by a second launch that works through a job list.
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
constexpr int kRowsKept = 1024;      // rows whose numbers a CTA keeps in shared memory
constexpr int kCountersPerPage = 4;  // ints of shared memory per page in one CTA
constexpr int kAhead = 4;            // entries whose loads a thread has in flight
constexpr int kTwo = 2;              // the same as rows x columns
constexpr int kPagesAhead = 8;

// Counters at PagesArgs::L.info: the phases' totals.
struct PagesInfo {
    int jobs;                  // page copies listed
    int live_below;            // compact: pages in use below the n-th id
    int pad[2];
    int tally[kPageCtas];      // per CTA: free (update) or used (compact) pages of its range, kBad if it found an error
};
constexpr int kBad = INT_MIN;  // nothing is written then

// A CTA's place, its barrier and its view of what other CTAs write.
template <int kCtas>
struct Team {
    static constexpr int kAll = kCtas * kPageThreads;
    int cta, at;
    __device__ Team() {
        cta = 0;
        if constexpr (kCtas > 1) asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(cta));
        at = cta * kPageThreads + (int)threadIdx.x;
    }
    // Every thread; writes before it are visible after it, to load().
    __device__ static void sync() {
        if constexpr (kCtas > 1)
            asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
        else
            __syncthreads();
    }
    // A counter: in shared memory for one CTA, else past L1.
    __device__ static int load(const int* p) {
        if constexpr (kCtas > 1) return __ldcg(p);
        else return *p;
    }
    // CTA c's pages are [from(c), from(c + 1)).
    __device__ static int from(int n, int c) { return kCtas > 1 ? (int)((long long)n * c / kCtas) : c * n; }
};

// Lanes that take a row of an update: the power of two that its entries fill, at
// most a warp.
__host__ __device__ __forceinline__ int row_lanes(int pages_per_row) {
    return pages_per_row > 16 ? 32 : pages_per_row > 8 ? 16 : 8;
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

// A row's parent, the positions it keeps, gets and held; parent -2: bad
// numbers (the row then counts for nothing, and the error stops the call).
struct __align__(16) Row {
    int parent, keep, want, held;
    __device__ int full() const { return keep / kPageSize; }
    __device__ bool part() const { return keep % kPageSize > 0; }
    __device__ bool writes() const { return want > keep; }
};

__device__ __forceinline__ Row read_row(const PagesArgs& a, int r) {
    const int cap = a.pages_per_row * kPageSize;
    const int p = __ldg(a.parents + r), want = __ldg(a.new_lengths + r), held = __ldg(a.lengths + r);
    const int given = p >= 0 && p < a.rows ? __ldg(a.lengths + p) : 0;
    if (p < -1 || p >= a.rows || want < 0 || want > cap || held < 0 || held > cap || given < 0 || given > cap)
        return {-2, 0, 0, 0};
    return {p, min(given, want), want, held};
}

template <int kCtas>
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kPageThreads, 1)
    pages_update_kernel(const __grid_constant__ PagesArgs a) {
    using T = Team<kCtas>;
    extern __shared__ int s_counters[];
    __shared__ Row s_row[kRowsKept];
    __shared__ int2 s_at[kRowsKept];            // entries a row keeps, and the rank of its first fresh page
    __shared__ int s_warp[32], s_bad, s_tally;
    griddep_launch_dependents();
    const T team;
    const int cta = team.cta, at = team.at, tid = threadIdx.x;
    const int R = a.rows, W = a.pages_per_row, N = a.num_pages;
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(a.ws);
    PagesInfo* info = reinterpret_cast<PagesInfo*>(a.ws + a.L.info);
    int2* row_at = reinterpret_cast<int2*>(a.ws + a.L.rows);
    int4* jobs = reinterpret_cast<int4*>(a.ws + a.L.jobs);
    // rows that held the page less its count (then its rank among its CTA's free
    // ones), rows that do not write into it (then with holders outside), the
    // lowest row that does, each CTA's free pages at its range's start, and
    // [row][page] the parent's entry
    int* held = kCtas > 1 ? reinterpret_cast<int*>(a.ws + a.L.a) : s_counters;
    int* others = kCtas > 1 ? reinterpret_cast<int*>(a.ws + a.L.b) : s_counters + N;
    int* first = kCtas > 1 ? reinterpret_cast<int*>(a.ws + a.L.c) : s_counters + 2 * N;
    int* list = kCtas > 1 ? reinterpret_cast<int*>(a.ws + a.L.d) : s_counters + 3 * N;
    int* kept = kCtas > 1 ? reinterpret_cast<int*>(a.ws + a.L.table) : s_counters + kCountersPerPage * N;

    bool negative = false;
    #pragma unroll 4
    for (int x = at; x < N; x += T::kAll) {
        const int refs = __ldcg(a.refs + x);
        negative = negative || refs < 0;
        held[x] = -refs;
        others[x] = 0;
        first[x] = INT_MAX;
    }
    if (at == 0) info->jobs = 0;
    if (tid == 0) s_bad = 0;
    if (tid < min(R, kRowsKept)) s_row[tid] = read_row(a, tid);
    auto row = [&](int r) { return r < kRowsKept ? s_row[r] : read_row(a, r); };
    auto bad = [&](int bits) {
        set_error(ctrl, bits);
        s_bad = 1;
    };
    T::sync();
    if (negative) bad(kErrBadPage);

    const int lanes = row_lanes(W), teams = T::kAll / lanes, l = at % lanes;

    // Holders, old and new.  What a row keeps is copied, because its parent's
    // entries may be overwritten before they are taken over.
    for (int r0 = at / lanes; r0 < R; r0 += kTwo * teams) {
        int full[kTwo], n_old[kTwo], n_takes[kTwo], parent[kTwo], most = 0;
        bool writes[kTwo];
        #pragma unroll
        for (int q = 0; q < kTwo; ++q) {
            const int r = r0 + q * teams;
            const Row w = r < R ? row(r) : Row{-1, 0, 0, 0};
            if (w.parent == -2 && l == 0) bad(kErrBadPos);
            parent[q] = w.parent;
            full[q] = w.full();
            writes[q] = w.writes();
            n_old[q] = pages_of(w.held);
            n_takes[q] = full[q] + (w.part() ? 1 : 0);
            most = max(most, max(n_old[q], n_takes[q]));
        }
        for (int c0 = l; c0 < most; c0 += kTwo * lanes) {
            int x[kTwo][kTwo], y[kTwo][kTwo];
            #pragma unroll
            for (int q = 0; q < kTwo; ++q) {
                #pragma unroll
                for (int k = 0; k < kTwo; ++k) {
                    const int c = c0 + k * lanes;
                    x[q][k] = c < n_old[q] ? __ldcg(a.table + (size_t)(r0 + q * teams) * W + c) : 0;
                    y[q][k] = c < n_takes[q] ? __ldcg(a.table + (size_t)parent[q] * W + c) : 0;
                }
            }
            #pragma unroll
            for (int q = 0; q < kTwo; ++q) {
                #pragma unroll
                for (int k = 0; k < kTwo; ++k) {
                    const int r = r0 + q * teams, c = c0 + k * lanes, xx = x[q][k], yy = y[q][k];
                    if (xx < 0 || xx >= N || yy < 0 || yy >= N) {
                        bad(kErrBadPage);
                        continue;
                    }
                    if (c < n_old[q]) atomicAdd(held + xx, 1);
                    if (c < n_takes[q]) {
                        kept[(size_t)r * W + c] = yy;
                        if (c == full[q] && writes[q]) atomicMin(first + yy, r);
                        else atomicAdd(others + yy, 1);
                    }
                }
            }
        }
    }
    T::sync();

    // Pages: pins counted in, the free ones ranked within the CTA's range, a
    // few pages in a row per thread.
    const int x0 = T::from(N, cta), x1 = T::from(N, cta + 1);
    int n_free = 0;
    for (int b = x0; b < x1;) {
        const int P = min(kPagesAhead, (x1 - b + kPageThreads - 1) / kPageThreads), x = b + tid * P;
        uint32_t free = 0;
        #pragma unroll
        for (int k = 0; k < kPagesAhead; ++k) {
            if (k >= P || x + k >= x1) continue;
            const int h = T::load(held + x + k), o = T::load(others + x + k) - h;
            if (h > 0) bad(kErrBadPage);
            others[x + k] = o;
            if (o == 0 && T::load(first + x + k) == INT_MAX) free |= 1u << k;
        }
        int total;
        int rank = n_free + block_excl(__popc(free), s_warp, &total);
        #pragma unroll
        for (int k = 0; k < kPagesAhead; ++k) {
            if (k >= P || x + k >= x1) continue;
            const bool f = free >> k & 1;
            held[x + k] = f ? rank : -1;
            if (f) list[x0 + rank++] = x + k;
        }
        n_free += total;
        b += P * kPageThreads;
    }
    // (the last barrier of a scan, or of the phase before, orders s_bad)
    __syncthreads();
    if (tid == 0) {
        s_tally = s_bad ? kBad : n_free;
        if (kCtas > 1) info->tally[cta] = s_tally;
    }
    T::sync();

    int have[kCtas + 1];
    bool stop = false;
    have[0] = 0;
    #pragma unroll
    for (int c = 0; c < kCtas; ++c) {
        const int n = kCtas > 1 ? __ldcg(&info->tally[c]) : s_tally;
        stop = stop || n == kBad;
        have[c + 1] = have[c] + n;
    }
    if (stop) return;                           // the same for every CTA; info->jobs is 0: nothing is copied either
    // Rows: which tails are copied, and where each row's fresh pages start.
    // Every CTA scans all rows.
    int need = 0;
    for (int b = 0; b < R; b += kPageThreads) {
        const int r = b + tid;
        int mine = 0, keeps = 0;
        if (r < R) {
            const Row k = row(r);
            keeps = k.full() + (k.part() ? 1 : 0);
            if (k.part() && k.writes()) {
                const int x = T::load(kept + (size_t)r * W + k.full());
                if (T::load(others + x) != 0 || T::load(first + x) != r) keeps = k.full();
            }
            mine = pages_of(k.want) - keeps;
        }
        int total;
        const int start = need + block_excl(mine, s_warp, &total);
        // (rows past the first: all CTAs write the same)
        if (r < kRowsKept) s_at[tid] = make_int2(keeps, start);
        else if (r < R) row_at[r] = make_int2(keeps, start);
        need += total;
    }
    if (need > have[kCtas]) {
        if (at == 0) set_error(ctrl, kErrNoPages);
        return;
    }
    __syncthreads();
    int base = 0;
    #pragma unroll
    for (int c = 0; c < kCtas; ++c) base = cta == c ? have[c] : base;
    #pragma unroll 4
    for (int x = x0 + tid; x < x1; x += kPageThreads) {
        const int rank = T::load(held + x), o = T::load(others + x);
        a.refs_out[x] = rank < 0 ? max(o, 1) : base + rank < need ? 1 : 0;      // not free at 0: one writer keeps it
    }
    for (int r0 = at / lanes; r0 < R; r0 += kTwo * teams) {
        int2 ra[kTwo];
        int n[kTwo], tail[kTwo], tokens[kTwo];
        #pragma unroll
        for (int q = 0; q < kTwo; ++q) {
            const int r = r0 + q * teams;
            ra[q] = make_int2(0, 0);
            n[q] = 0;
            tail[q] = -1;
            if (r >= R) continue;
            const Row w = row(r);
            ra[q] = r < kRowsKept ? s_at[r] : __ldcg(row_at + r);
            n[q] = pages_of(w.want);
            tokens[q] = w.keep % kPageSize;
            // a tail that is not kept is copied to the first fresh page
            if (w.part() && w.full() == ra[q].x) tail[q] = ra[q].x;
        }
        for (int c0 = l; c0 < W; c0 += kTwo * lanes) {
            int x[kTwo][kTwo], y[kTwo][kTwo];
            #pragma unroll
            for (int q = 0; q < kTwo; ++q) {
                #pragma unroll
                for (int k = 0; k < kTwo; ++k) {
                    const int c = c0 + k * lanes;
                    x[q][k] = -1;
                    if (c < ra[q].x || c == tail[q]) y[q][k] = T::load(kept + (size_t)(r0 + q * teams) * W + c);
                    if (c >= ra[q].x && c < n[q]) {
                        const int rank = ra[q].y + c - ra[q].x;
                        int at0 = 0, skip = 0;
                        #pragma unroll
                        for (int h = 1; h < kCtas; ++h)
                            if (rank >= have[h]) {
                                at0 = T::from(N, h);
                                skip = have[h];
                            }
                        x[q][k] = T::load(list + at0 + rank - skip);
                    }
                }
            }
            #pragma unroll
            for (int q = 0; q < kTwo; ++q) {
                #pragma unroll
                for (int k = 0; k < kTwo; ++k) {
                    const int r = r0 + q * teams, c = c0 + k * lanes;
                    if (r >= R || c >= W) continue;
                    a.table_out[(size_t)r * W + c] = c < ra[q].x ? y[q][k] : x[q][k];
                    if (c == tail[q]) jobs[atomicAdd(&info->jobs, 1)] = make_int4(y[q][k], x[q][k], tokens[q], 0);
                }
            }
        }
    }
}

template <int kCtas>
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kPageThreads, 1)
    pages_compact_kernel(const __grid_constant__ PagesArgs a) {
    using T = Team<kCtas>;
    extern __shared__ int s_counters[];
    __shared__ int s_warp[32], s_bad, s_tally, s_below;
    griddep_launch_dependents();
    const T team;
    const int cta = team.cta, at = team.at, tid = threadIdx.x;
    const int R = a.rows, W = a.pages_per_row, N = a.num_pages, cap = W * kPageSize;
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(a.ws);
    PagesInfo* info = reinterpret_cast<PagesInfo*>(a.ws + a.L.info);
    int4* jobs = reinterpret_cast<int4*>(a.ws + a.L.jobs);
    // a page in use: its rank among its CTA's; a free one: ~rank
    int* rank = kCtas > 1 ? reinterpret_cast<int*>(a.ws + a.L.a) : s_counters;
    int* holes = kCtas > 1 ? reinterpret_cast<int*>(a.ws + a.L.b) : s_counters + N;      // free ids below n, in order
    int* moved = kCtas > 1 ? reinterpret_cast<int*>(a.ws + a.L.c) : s_counters + 2 * N;  // new ids

    if (at == 0) info->jobs = 0;
    if (tid == 0) s_bad = 0;
    __syncthreads();
    auto bad = [&](int bits) {
        set_error(ctrl, bits);
        s_bad = 1;
    };
    // Held entries have to be in use.
    const unsigned entries = (unsigned)R * W;
    for (unsigned i0 = at; i0 < entries; i0 += kAhead * T::kAll) {
        int x[kAhead], len[kAhead];
        #pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const unsigned i = i0 + k * T::kAll;
            x[k] = len[k] = 0;
            if (i >= entries) continue;
            len[k] = __ldg(a.lengths + i / W);
            x[k] = __ldcg(a.table + i);
        }
        #pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const unsigned i = i0 + k * T::kAll;
            const int c = i % W;
            if (len[k] < 0 || len[k] > cap) {
                if (c == 0) bad(kErrBadPos);
            } else if (i < entries && c < pages_of(len[k])) {
                if (x[k] < 0 || x[k] >= N || __ldcg(a.refs + x[k]) <= 0) bad(kErrBadPage);
            }
        }
    }
    const int x0 = T::from(N, cta), x1 = T::from(N, cta + 1);
    int n_live = 0;
    for (int b = x0; b < x1;) {
        const int P = min(kPagesAhead, (x1 - b + kPageThreads - 1) / kPageThreads), x = b + tid * P;
        int refs[kPagesAhead];
        #pragma unroll
        for (int k = 0; k < kPagesAhead; ++k) refs[k] = k < P && x + k < x1 ? __ldcg(a.refs + x + k) : 0;
        int live = 0;
        #pragma unroll
        for (int k = 0; k < kPagesAhead; ++k) {
            if (refs[k] < 0) bad(kErrBadPage);
            live += refs[k] > 0;
        }
        int total;
        int q = n_live + block_excl(live, s_warp, &total);
        #pragma unroll
        for (int k = 0; k < kPagesAhead; ++k) {
            if (k >= P || x + k >= x1) continue;
            rank[x + k] = refs[k] > 0 ? q++ : ~q;
        }
        n_live += total;
        b += P * kPageThreads;
    }
    __syncthreads();
    if (tid == 0) {
        s_tally = s_bad ? kBad : n_live;
        if (kCtas > 1) info->tally[cta] = s_tally;
    }
    T::sync();
    int before = 0, n = 0;
    bool stop = false;
    #pragma unroll
    for (int c = 0; c < kCtas; ++c) {
        const int k = kCtas > 1 ? __ldcg(&info->tally[c]) : s_tally;
        stop = stop || k == kBad;
        before += c < cta ? k : 0;
        n += k;
    }
    if (stop) return;                           // the same for every CTA: no barrier is left waiting
    for (int x = x0 + tid; x < x1; x += kPageThreads) {
        const int q = T::load(rank + x), up = before + (q < 0 ? ~q : q);        // pages in use below x
        if (x == n) {
            if (kCtas > 1) info->live_below = up;
            else s_below = up;
        }
        if (q < 0 && x < n) holes[x - up] = x;
    }
    T::sync();
    const int below = n == N ? n : kCtas > 1 ? __ldcg(&info->live_below) : s_below;
    for (int x = x0 + tid; x < x1; x += kPageThreads) {
        const int q = T::load(rank + x), up = before + (q < 0 ? ~q : q);
        int to = q < 0 ? -1 : x;
        if (q >= 0 && x >= n) {
            to = T::load(holes + up - below);
            jobs[up - below] = make_int4(x, to, kPageSize, 0);
            a.refs_out[to] = __ldcg(a.refs + x);
            a.refs_out[x] = 0;
        } else if (q >= 0) {
            if (a.refs_out != a.refs) a.refs_out[x] = __ldcg(a.refs + x);
        } else if (x >= n) {
            a.refs_out[x] = 0;
        }
        moved[x] = to;
        a.map[x] = to;
    }
    if (at == 0) info->jobs = n - below;
    T::sync();
    for (unsigned i0 = at; i0 < entries; i0 += kAhead * T::kAll) {
        int x[kAhead], held[kAhead];
        #pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const unsigned i = i0 + k * T::kAll;
            x[k] = held[k] = 0;
            if (i >= entries) continue;
            held[k] = pages_of(__ldg(a.lengths + i / W));
            x[k] = __ldcg(a.table + i);
        }
        #pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const unsigned i = i0 + k * T::kAll;
            if (i < entries) a.table_out[i] = (int)(i % W) < held[k] ? T::load(moved + x[k]) : x[k];
        }
    }
}

// Copies the first `tokens` positions of page src to page dst in every pool:
// one block per (job, pool, head), a slab of at most 64 rows.
constexpr int kCopyThreads = 256;
constexpr int kCopyAhead = 4;

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ PoolList pools,
                                                                  const PagesInfo* info, const int4* jobs, int most) {
    griddep_wait();
    // the first job comes with the number of jobs (`most` places are there)
    int4 job = __ldcg(jobs + min((int)blockIdx.x / pools.slabs, most - 1));
    const long long items = (long long)__ldcg(&info->jobs) * pools.slabs;
    for (long long item = blockIdx.x; item < items; item += gridDim.x) {
        if (item >= gridDim.x) job = __ldcg(jobs + item / pools.slabs);
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
        for (int v0 = threadIdx.x; v0 < vecs; v0 += kCopyAhead * kCopyThreads) {
            uint4 x[kCopyAhead];
            #pragma unroll
            for (int k = 0; k < kCopyAhead; ++k)
                if (v0 + k * kCopyThreads < vecs) x[k] = __ldcs(reinterpret_cast<const uint4*>(src) + v0 + k * kCopyThreads);
            #pragma unroll
            for (int k = 0; k < kCopyAhead; ++k)
                if (v0 + k * kCopyThreads < vecs) reinterpret_cast<uint4*>(dst)[v0 + k * kCopyThreads] = x[k];
        }
        for (int t = vecs * 16 + threadIdx.x; t < bytes; t += kCopyThreads) dst[t] = src[t];
    }
}

}  // namespace

// One CTA for small tables and pools, else the cluster.  An update's rows are
// taken by teams of lanes (row_lanes), a compaction's entries one per thread; up
// to kOneCtaPages its threads count and rank all pages in one pass.  One CTA
// against the cluster, us of a graph replay, by num_pages:
//   rows x pages_per_row     4360         6000         8000        10000
//   update   16 x 64      8.9, 13.4    9.8, 13.4   13.7, 13.6   15.5, 14.8
//            64 x 65     11.1, 15.9   11.7, 15.9   15.4, 15.5   17.4, 17.0
//            64 x 128    11.2, 15.8   12.2, 16.5   15.8, 17.3   17.6, 18.4
//           128 x 64     12.4, 13.9   13.2, 14.5   16.9, 15.6   18.6, 16.1
//            24 x 340    12.6, 19.1   13.8, 19.9   18.3, 22.7   20.6, 24.7
//   compact  16 x 64      9.6, 12.3   10.6, 12.6   12.5, 12.9   14.6, 13.7
//            64 x 65     13.3, 12.8   14.2, 13.2   16.7, 13.3   18.8, 14.8
//           128 x 64     15.2, 12.0   16.1, 12.9   18.8, 13.4   21.8, 14.7
// An update of 256 x 32 in 4000 pages 17.6, 13.7; compact 256 x 13 in 2100 10.8,
// 11.9, 64 x 65 in 1000 10.5, 10.8: an entry of it counts as two pages.  The
// cluster in 32768 and 131072 pages: update of 64 x 65 21.6, 53.8, compact 18.0,
// 35.8.
constexpr int kOneCtaPages = kPagesAhead * kPageThreads;
constexpr int kOneCtaEntries = 8192;         // of an update: in shared memory
constexpr int kOneCtaLanes = 4096;           // of an update
constexpr int kOneCtaCompact = 10240;        // pages and twice the entries

template <typename K>
static cudaError_t launch_team(K one, K many, const PagesArgs& a, bool small, size_t smem, size_t most, int* configured_mask,
                               cudaStream_t stream) {
    if (!small) {
        many<<<kPageCtas, kPageThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 31 || !(__atomic_load_n(configured_mask, __ATOMIC_ACQUIRE) & (1 << dev))) {
        e = cudaFuncSetAttribute(one, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (e != cudaSuccess) return e;
        if (dev < 31) __atomic_fetch_or(configured_mask, 1 << dev, __ATOMIC_ACQ_REL);
    }
    one<<<1, kPageThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_pages(const PagesArgs& a, bool compact, cudaStream_t stream) {
    static int update_mask = 0, compact_mask = 0;   // bit per device id < 31
    const long long entries = (long long)a.rows * a.pages_per_row;
    const size_t counters = (size_t)a.num_pages * kCountersPerPage * sizeof(int);
    const size_t most = (size_t)kOneCtaPages * kCountersPerPage * sizeof(int);
    if (compact)
        return launch_team(pages_compact_kernel<1>, pages_compact_kernel<kPageCtas>, a,
                           a.num_pages <= kOneCtaPages && a.num_pages + 2 * entries <= kOneCtaCompact, counters, most,
                           &compact_mask, stream);
    const bool small = a.num_pages <= kOneCtaPages && entries <= kOneCtaEntries &&
                       (long long)a.rows * row_lanes(a.pages_per_row) <= kOneCtaLanes;
    return launch_team(pages_update_kernel<1>, pages_update_kernel<kPageCtas>, a, small, counters + entries * sizeof(int),
                       most + kOneCtaEntries * sizeof(int), &update_mask, stream);
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
                              reinterpret_cast<const int4*>(a.ws + a.L.jobs), max(a.rows, a.num_pages));
}

}  // namespace pdattn
