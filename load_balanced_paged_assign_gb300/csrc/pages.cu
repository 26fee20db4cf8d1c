// The pages of a paged cache as a pool: rows of a block table take pages, share
// them (a fork), give them back and are brought together (compaction), all on the
// device, so that a captured step may do it.
//
// A pool is three arrays: refs[p], the table entries that name page p; a stack of
// the pages with no holder, the next one handed out at its top; and the state
// {pages on the stack, flags}.  What a call does does not depend on the order in
// which threads run: pages are handed out and given back in the order of the
// call's list of rows (and within a row by position), by prefix sums.
//
// Each call's bookkeeping is one launch of one CTA, or of one cluster: its phases (look,
// count, write) follow one another at barriers, the warps' totals pass through
// distributed shared memory.  A thread holds its entries of the list in registers, so
// each phase is one round of reads in flight together; a longer list goes round by
// round.  A warp's entries are consecutive, so a prefix sum is a ballot per 32 entries
// and one sum over the warps.
//
// All of it is latency: a call is a chain of four to six dependent reads (the list, the
// table, the count, the mark) of 0.6 us each and a launch.  The copies that a fork or a
// compaction lists (pages moved in every layer's cache) are a kernel of their own, which
// HBM bounds.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>
#include <climits>

#include "internal.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace hpc {
namespace {

constexpr int kPoolThreads = 1024;
constexpr int kPoolWarps = kPoolThreads / 32;
constexpr int kPoolCtas = 16;  // of a cluster, at most
// List entries of a thread in a round: one where the cluster then holds the list, else eight.
// Code that runs once is fetched once: two calls over 4 rows 6.3 us with one entry, 12.0
// with eight; over 102,400 entries 60 us with two, 30 with eight.  And no more CTAs than
// hold the list: two calls over 4 rows 11.9 us on 16, 6.9 on one; over 102,400 entries 30 us
// on 16, 58 on eight, 265 on one.
constexpr int kFew = 1, kMany = 8;
constexpr int kUnroll = 2;  // of the other loops
constexpr int kForkPages = 128;  // of a child, for one warp at a time
constexpr int kIdle = INT_MAX;        // marks[p] between calls
constexpr int kUnheld = -1;           // marks[p] in a compaction, of a page that none holds
// Numbers below -2^30 in the table are the calls' own, and gone when they end: the list's
// place that claims an empty entry (the smaller wins).
constexpr int kCodes = 1 << 30;
constexpr unsigned kAll = 0xffffffffu;

struct Pool {
    int32_t *refs, *stack, *state, *marks;
    int num_pages;
};

// What the bookkeeping calls share: rows of a table, row i of the list being
// rows[i] (rows null: i), and the entries (i, j) of the list's rows.
struct Rows {
    int32_t *table;
    const int32_t *rows;
    int B, max_pages, n;
};

// The row of entry e of a list (its quotient by max_pages, below 2^14: off by one at most
// before the correction).
__device__ __forceinline__ int row_in_list(const Rows &t, int e, float inv) {
    const int q = (int)((float)e * inv), r = e - q * t.max_pages;
    return q + (r >= t.max_pages) - (r < 0);
}

__device__ __forceinline__ int row_of(const Rows &t, int i) { return t.rows ? __ldg(t.rows + i) : i; }

// A barrier of all the call's threads: what they wrote before it, all see after it.
__device__ __forceinline__ void sync_all() {
    if (gridDim.x == 1) __syncthreads();
    else cg::this_cluster().sync();
}

__device__ __forceinline__ int warp_index() {
    return (int)blockIdx.x * kPoolWarps + (int)(threadIdx.x >> 5);
}

struct Totals {
    int warp[kPoolWarps];
    int cta;
};

// The entries counted by the warps before this one, and by all: `count` is the warp's.
// A barrier as sync_all(); one has to follow before the next, or the kernel's end.
__device__ __forceinline__ int counts_before(int count, Totals &t, int &total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    if (lane == 0) t.warp[w] = count;
    __syncthreads();
    const int mine = t.warp[lane];
    const int cta = __reduce_add_sync(kAll, mine);
    int before = __reduce_add_sync(kAll, lane < w ? mine : 0);
    total = cta;
    if (gridDim.x == 1) return before;
    cg::cluster_group cluster = cg::this_cluster();
    if (threadIdx.x == 0) t.cta = cta;
    cluster.sync();
    const int n = lane < (int)gridDim.x ? cluster.map_shared_rank(&t, lane)->cta : 0;
    before += __reduce_add_sync(kAll, lane < (int)blockIdx.x ? n : 0);
    total = __reduce_add_sync(kAll, n);
    return before;
}

// Ranks a warp's flagged entries, in the order of k and then of the lanes, from `base`
// on; returns how many there are.
template <int OWN, class Emit>
__device__ __forceinline__ int ranked(const bool (&flag)[OWN], int base, Emit emit) {
    const unsigned below = (1u << (threadIdx.x & 31)) - 1u;
    int n = 0;
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
        const unsigned vote = __ballot_sync(kAll, flag[k]);
        if (flag[k]) emit(k, base + n + __popc(vote & below));
        n += __popc(vote);
    }
    return n;
}

struct Nothing {
    __device__ void operator()(int, int) const {}
};

__device__ __forceinline__ int code_of(int x) { return INT_MIN + x; }
// How many pages the stack can hold or hand out, whatever its count says.
__device__ __forceinline__ int stack_top(const Pool &pool) {
    return min(max(__ldcg(pool.state), 0), pool.num_pages);
}

// ------------------------------------------------------------------ give back
// Entries from ceil(keep / 64) on: each is exchanged for -1 (a row that is named twice
// gives its pages back once), its page loses a holder, and one that has none left goes
// on the stack, placed by the first entry of the list that named it (marks).  Rounds go
// from the list's end to its beginning, so the first page listed comes to lie on top;
// a page whose holders are in several rounds loses its last one in the first of the list.
template <int OWN>
__global__ void __launch_bounds__(kPoolThreads) free_kernel(const Pool pool, const Rows t,
                                                            const int32_t *keep, int rounds) {
    __shared__ Totals totals;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, entries = t.n * t.max_pages;
    const float inv = 1.f / (float)t.max_pages;
    unsigned flags = 0;
    int top = stack_top(pool);
    for (int round = rounds - 1; round >= 0; --round) {
        const long long e0 =
            ((long long)round * gridDim.x * kPoolWarps + warp_index()) * (32 * OWN) + lane;
        int32_t *at[OWN];
        int p[OWN];
#pragma unroll
        for (int k = 0; k < OWN; ++k) {
            const long long e = e0 + 32 * k;
            at[k] = nullptr;
            p[k] = -1;
            if (e >= entries) continue;
            const int i = row_in_list(t, (int)e, inv), j = (int)e - i * t.max_pages;
            const int r = row_of(t, i);
            const int n = keep ? __ldg(keep + i) : 0;
            if (r < 0 || r >= t.B || n < 0 || n > t.max_pages * kTile)
                flags |= HPC_FLAG_BAD_SEQLEN;
            else if (j >= (n + kTile - 1) / kTile)
                at[k] = t.table + (size_t)r * t.max_pages + j;
        }
#pragma unroll
        for (int k = 0; k < OWN; ++k)
            if (at[k]) p[k] = __ldcg(at[k]);
#pragma unroll
        for (int k = 0; k < OWN; ++k)
            if (p[k] >= 0) p[k] = atomicExch(at[k], -1);
#pragma unroll
        for (int k = 0; k < OWN; ++k)
            if (p[k] >= pool.num_pages) {
                flags |= HPC_FLAG_BAD_PAGE;
                p[k] = -1;
            }
        int held[OWN];
#pragma unroll
        for (int k = 0; k < OWN; ++k) held[k] = p[k] >= 0 ? atomicSub(pool.refs + p[k], 1) : 1;
#pragma unroll
        for (int k = 0; k < OWN; ++k) {
            if (held[k] <= 0) {  // held by none
                atomicAdd(pool.refs + p[k], 1);
                flags |= HPC_FLAG_BAD_PAGE;
                p[k] = -1;
            }
            if (p[k] >= 0) atomicMin(pool.marks + p[k], (int)(e0 + 32 * k));
        }
        sync_all();
        int mark[OWN];
        bool back[OWN];
#pragma unroll
        for (int k = 0; k < OWN; ++k) {
            mark[k] = p[k] >= 0 ? __ldcg(pool.marks + p[k]) : 0;
            held[k] = p[k] >= 0 ? __ldcg(pool.refs + p[k]) : 1;
        }
#pragma unroll
        for (int k = 0; k < OWN; ++k) back[k] = held[k] == 0 && mark[k] == (int)(e0 + 32 * k);
        int total;
        const int mine = ranked(back, 0, Nothing());
        const int base = counts_before(mine, totals, total);
        ranked(back, base, [&](int k, int rank) {
            const int to = top + total - 1 - rank;
            if (to < pool.num_pages) pool.stack[to] = p[k];
        });
#pragma unroll
        for (int k = 0; k < OWN; ++k)
            if (p[k] >= 0) pool.marks[p[k]] = kIdle;
        top += total;
        sync_all();
    }
    if (top > pool.num_pages) flags |= HPC_FLAG_BAD_PAGE;
    flags = __reduce_or_sync(kAll, flags);
    if (flags && lane == 0) atomicOr(pool.state + 1, (int)flags);
    if (blockIdx.x == 0 && threadIdx.x == 0) pool.state[0] = min(top, pool.num_pages);
}

// ------------------------------------------------------------------ take
// Negative entries below ceil(lens / 64) take a page each, or, where the stack has
// not enough for all, none does.  An entry is claimed first, and the first of the list
// wins, so a row that is named twice is served once.
template <int OWN>
__global__ void __launch_bounds__(kPoolThreads) extend_kernel(const Pool pool, const Rows t,
                                                              const int32_t *lens, int rounds) {
    __shared__ Totals totals;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, entries = t.n * t.max_pages;
    const float inv = 1.f / (float)t.max_pages;
    const int top = stack_top(pool);
    unsigned flags = 0;
    int32_t *at[OWN];
    int e0 = 0;
    auto look = [&](int round) {  // the entries of this thread that take pages
        const long long first =
            ((long long)round * gridDim.x * kPoolWarps + warp_index()) * (32 * OWN) + lane;
        e0 = (int)min(first, (long long)entries);
#pragma unroll
        for (int k = 0; k < OWN; ++k) {
            at[k] = nullptr;
            if (first + 32 * k >= entries) continue;
            const int e = e0 + 32 * k, i = row_in_list(t, e, inv), j = e - i * t.max_pages;
            const int r = row_of(t, i), L = __ldg(lens + i);
            if (r < 0 || r >= t.B || L < 0 || L > t.max_pages * kTile)
                flags |= HPC_FLAG_BAD_SEQLEN;
            else if (j < (L + kTile - 1) / kTile)
                at[k] = t.table + (size_t)r * t.max_pages + j;
        }
    };
    bool own[OWN];
    auto won = [&]() {
        int v[OWN];
#pragma unroll
        for (int k = 0; k < OWN; ++k) v[k] = at[k] ? __ldcg(at[k]) : 0;
#pragma unroll
        for (int k = 0; k < OWN; ++k) own[k] = at[k] && v[k] == code_of(e0 + 32 * k);
    };
    for (int round = 0; round < rounds; ++round) {
        look(round);
        int v[OWN];
#pragma unroll
        for (int k = 0; k < OWN; ++k) v[k] = at[k] ? __ldcg(at[k]) : 0;
#pragma unroll
        for (int k = 0; k < OWN; ++k)
            if (v[k] < 0) atomicMin(at[k], code_of(e0 + 32 * k));
    }
    sync_all();
    int need = 0;  // of this warp
    for (int round = 0; round < rounds; ++round) {
        if (rounds > 1) look(round);
        won();
        need += ranked(own, 0, Nothing());
    }
    int total, taken = 0;
    int base = counts_before(need, totals, total);
    const bool enough = total <= top;
    for (int round = 0; round < rounds; ++round) {
        int n = total;
        if (rounds > 1) {
            look(round);
            won();
            sync_all();
            base = counts_before(ranked(own, 0, Nothing()), totals, n);
        }
        ranked(own, base, [&](int k, int rank) {
            const int p = enough ? __ldcg(pool.stack + (top - 1 - taken - rank)) : -1;
            if (enough && (p < 0 || p >= pool.num_pages)) {
                flags |= HPC_FLAG_BAD_PAGE;
                *at[k] = -1;
                return;
            }
            *at[k] = p;
            if (enough) pool.refs[p] = 1;
        });
        taken += n;
    }
    if (!enough) flags |= HPC_FLAG_NO_PAGES;
    flags = __reduce_or_sync(kAll, flags);
    if (flags && lane == 0) atomicOr(pool.state + 1, (int)flags);
    if (enough && blockIdx.x == 0 && threadIdx.x == 0) pool.state[0] = top - total;
    sync_all();  // no CTA leaves while another may read its shared memory
}

// ------------------------------------------------------------------ fork
struct Fork {
    const int32_t *src, *lens;
    int32_t *copies;  // [1 + cap][2]
};

// Child i shares the whole pages of the first lens[i] tokens of row src[i], and
// gets a page of its own for the rest of them, with a copy listed.  Phases: claim
// the empty rows (the first of the list wins), look at every child's pages, place
// the new ones, write.
__global__ void __launch_bounds__(kPoolThreads) fork_kernel(const Pool pool, const Rows t,
                                                            const Fork f) {
    __shared__ Totals totals;
    __shared__ unsigned bad[HPC_MAX_BATCH / 32];  // a bit for each child that is refused
    cg::cluster_group cluster = cg::this_cluster();
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, first = (int)blockIdx.x * kPoolThreads + threadIdx.x;
    const int threads = (int)gridDim.x * kPoolThreads, warps = (int)gridDim.x * kPoolWarps;
    for (int i = threadIdx.x; i < (t.n + 31) / 32; i += kPoolThreads) bad[i] = 0;
    unsigned flags = 0;
    unsigned *bad0 = gridDim.x == 1 ? bad : cluster.map_shared_rank(bad, 0);
    auto refuse = [&](int i) { atomicOr(bad0 + (i >> 5), 1u << (i & 31)); };
    const int cap = t.max_pages * kTile, top = stack_top(pool);
    auto in_range = [&](int s, int d, int L) {
        return s >= 0 && s < t.B && d >= 0 && d < t.B && s != d && L >= 0 && L <= cap;
    };
    for (int i = first; i < t.n; i += threads) {
        const int s = __ldg(f.src + i), d = row_of(t, i), L = __ldg(f.lens + i);
        if (in_range(s, d, L) && L > 0) {
            int32_t *at = t.table + (size_t)d * t.max_pages;
            if (__ldcg(at) < 0) atomicMin(at, code_of(i));
        }
    }
    sync_all();
    // a warp takes a run of kForkPages pages of a child at a time
    const int runs = (t.max_pages + kForkPages - 1) / kForkPages;
    const long long items = (long long)t.n * runs;
    for (long long it = warp_index(); it < items; it += warps) {
        const int i = (int)(it / runs), j0 = (int)(it - (long long)i * runs) * kForkPages;
        const int s = __ldg(f.src + i), d = row_of(t, i), L = __ldg(f.lens + i);
        if (!in_range(s, d, L)) {
            if (lane == 0 && j0 == 0) {
                flags |= HPC_FLAG_BAD_SEQLEN;
                refuse(i);
            }
            continue;
        }
        const int n = (L + kTile - 1) / kTile;
        int p[kForkPages / 32], q[kForkPages / 32], held[kForkPages / 32];
        unsigned bits = 0;
#pragma unroll
        for (int k = 0; k < kForkPages / 32; ++k) {
            const int j = j0 + 32 * k + lane;
            p[k] = j < n ? __ldcg(t.table + (size_t)s * t.max_pages + j) : 0;
            q[k] = j < n ? __ldcg(t.table + (size_t)d * t.max_pages + j) : -1;
        }
#pragma unroll
        for (int k = 0; k < kForkPages / 32; ++k) {
            const int j = j0 + 32 * k + lane;
            held[k] = j < n && p[k] >= 0 && p[k] < pool.num_pages ? __ldcg(pool.refs + p[k]) : 1;
        }
#pragma unroll
        for (int k = 0; k < kForkPages / 32; ++k) {
            const int j = j0 + 32 * k + lane;
            if (j >= n) continue;
            if (p[k] < 0 || p[k] >= pool.num_pages || held[k] <= 0)
                bits |= HPC_FLAG_BAD_PAGE;
            else if (j == 0 ? q[k] != code_of(i) : q[k] >= 0)
                bits |= HPC_FLAG_BAD_SEQLEN;  // the row is not empty, or another child's
        }
        flags |= bits;
        if (__any_sync(kAll, bits != 0) && lane == 0) refuse(i);
    }
    sync_all();
    if (blockIdx.x > 0)
        for (int w = threadIdx.x; w < (t.n + 31) / 32; w += kPoolThreads) bad[w] = bad0[w];
    __syncthreads();
    auto refused = [&](int i) { return (bad[i >> 5] >> (i & 31) & 1u) != 0; };
    // The children that need a page of their own: all CTAs count them, the first one
    // (whose warps hold consecutive ones) places them.
    int mine = 0, total;
    const int per = ((t.n + kPoolWarps - 1) / kPoolWarps + 31) & ~31;
    const int lo = (int)(threadIdx.x >> 5) * per, hi = min(lo + per, t.n);
    auto partial = [&](int i) { return i < hi && !refused(i) && __ldg(f.lens + i) % kTile != 0; };
    for (int i0 = lo; i0 < hi; i0 += 32) mine += __popc(__ballot_sync(kAll, partial(i0 + lane)));
    if (lane == 0) totals.warp[threadIdx.x >> 5] = mine;
    __syncthreads();
    const int of = totals.warp[lane];
    total = __reduce_add_sync(kAll, of);
    const int base = __reduce_add_sync(kAll, lane < (int)(threadIdx.x >> 5) ? of : 0);
    const bool enough = total <= top;
    if (enough && blockIdx.x == 0) {
        int n = base;
        for (int i0 = lo; i0 < hi; i0 += 32) {
            const int i = i0 + lane;
            const bool yes = partial(i);
            const unsigned vote = __ballot_sync(kAll, yes);
            if (yes) {
                const int rank = n + __popc(vote & ((1u << lane) - 1u));
                const int whole = __ldg(f.lens + i) / kTile;
                const int p = __ldcg(pool.stack + (top - 1 - rank));
                int32_t *at = t.table + (size_t)row_of(t, i) * t.max_pages + whole;
                int from = __ldcg(t.table + (size_t)__ldg(f.src + i) * t.max_pages + whole);
                if (p < 0 || p >= pool.num_pages) {
                    flags |= HPC_FLAG_BAD_PAGE;
                    *at = -1;
                    from = -1;  // (not copied)
                } else {
                    *at = p;
                    pool.refs[p] = 1;
                }
                f.copies[2 * (rank + 1)] = from;
                f.copies[2 * (rank + 1) + 1] = p;
            }
            n += __popc(vote);
        }
    }
    for (long long it = warp_index(); it < items; it += warps) {
        const int i = (int)(it / runs), j0 = (int)(it - (long long)i * runs) * kForkPages;
        const int d = row_of(t, i);
        if (refused(i) || !enough) {  // the claim, where it is this child's, is withdrawn
            if (lane == 0 && j0 == 0 && d >= 0 && d < t.B)
                atomicCAS(t.table + (size_t)d * t.max_pages, code_of(i), -1);
            continue;
        }
        const int n = __ldg(f.lens + i) / kTile;
        const int32_t *from = t.table + (size_t)__ldg(f.src + i) * t.max_pages;
        int p[kForkPages / 32];
#pragma unroll
        for (int k = 0; k < kForkPages / 32; ++k) {
            const int j = j0 + 32 * k + lane;
            p[k] = j < n ? __ldcg(from + j) : -1;
        }
#pragma unroll
        for (int k = 0; k < kForkPages / 32; ++k) {
            if (p[k] < 0) continue;
            t.table[(size_t)d * t.max_pages + j0 + 32 * k + lane] = p[k];
            atomicAdd(pool.refs + p[k], 1);
        }
    }
    if (!enough) flags |= HPC_FLAG_NO_PAGES;
    flags = __reduce_or_sync(kAll, flags);
    if (flags && lane == 0) atomicOr(pool.state + 1, (int)flags);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        f.copies[0] = enough ? total : 0;
        f.copies[1] = 0;
        if (enough) pool.state[0] = top - total;
    }
    sync_all();  // no CTA leaves while another may read its shared memory
}

// ------------------------------------------------------------------ compact
// The live pages behind the first L places (L live ones in all) move, in order,
// into the holes among those; marks[p] holds a moved page's new place meanwhile, and
// kUnheld for a page that none holds: an entry that names one all the same becomes -1, as
// the page will be another's.  A page's number and the live ones before it say both its
// ranks, so one sum over the pages (and the live ones below L) places everything.
__global__ void __launch_bounds__(kPoolThreads)
    compact_kernel(const Pool in, const Pool out, const int32_t *table, int32_t *table_out,
                   int64_t entries, int32_t *copies) {
    __shared__ Totals totals, below;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, first = (int)blockIdx.x * kPoolThreads + threadIdx.x;
    const int threads = (int)gridDim.x * kPoolThreads, warps = (int)gridDim.x * kPoolWarps;
    const int per = ((in.num_pages + warps - 1) / warps + 31) & ~31;  // pages of a warp
    const int lo = (int)min((long long)warp_index() * per, (long long)in.num_pages);
    const int hi = min(lo + per, in.num_pages);
    // goes over the warp's pages up to `end`: fn(page, refs, live pages of the warp before)
    auto over = [&](int end, auto fn) {
        int n = 0;
        for (int p0 = lo; p0 < end; p0 += 32 * kUnroll) {
            int refs[kUnroll];
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                const int p = p0 + 32 * k + lane;
                refs[k] = p < end ? __ldcg(in.refs + p) : 0;
            }
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                const int p = p0 + 32 * k + lane;
                const unsigned vote = __ballot_sync(kAll, refs[k] > 0);
                if (p < end) fn(p, refs[k], n + __popc(vote & ((1u << lane) - 1u)));
                n += __popc(vote);
            }
        }
        return n;
    };
    auto nothing = [](int, int, int) {};
    int L, kept;
    const int live = over(hi, nothing);
    const int base = counts_before(live, totals, L);
    // live ones that stay: a warp's all, none, or (about place L) those that it counts
    const int stay = hi <= L ? live : lo >= L ? 0 : over(L, nothing);
    counts_before(stay, below, kept);
    const int moves = L - kept;
    over(hi, [&](int p, int refs, int before) {
        before += base;
        if (refs <= 0) in.marks[p] = kUnheld;
        if (p < L && refs <= 0) copies[2 * (p - before + 1) + 1] = p;   // hole number p - before
        if (p >= L && refs > 0) copies[2 * (before - kept + 1)] = p;
    });
    sync_all();
    for (int k = first; k < moves; k += threads) {
        const int src = __ldcg(copies + 2 * (k + 1)), dst = __ldcg(copies + 2 * (k + 1) + 1);
        in.marks[src] = dst;
        out.refs[dst] = __ldcg(in.refs + src);
    }
    sync_all();
    unsigned flags = 0;
    for (int64_t e0 = first; e0 < entries; e0 += (int64_t)threads * kUnroll) {
        int p[kUnroll], m[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            p[k] = e0 + (int64_t)k * threads < entries ? __ldcg(table + e0 + (int64_t)k * threads) : -1;
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            m[k] = p[k] < 0               ? kIdle
                   : p[k] >= in.num_pages ? kUnheld
                                          : __ldcg(in.marks + p[k]);
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            if (m[k] == kUnheld) flags |= HPC_FLAG_BAD_PAGE;
            if (e0 + (int64_t)k * threads < entries)
                table_out[e0 + (int64_t)k * threads] = m[k] != kIdle ? m[k] : p[k];
        }
    }
    for (int p = first; p < in.num_pages; p += threads) {
        if (p >= L) {
            out.refs[p] = 0;
        } else if (out.refs != in.refs) {
            const int r = __ldcg(in.refs + p);
            if (r > 0) out.refs[p] = r;
        }
        if (p < in.num_pages - L) out.stack[p] = in.num_pages - 1 - p;
    }
    if (first >= 1 && first < 4 && out.state != in.state) out.state[first] = __ldcg(in.state + first);
    if (first == 0) {
        copies[0] = moves;
        copies[1] = 0;
        out.state[0] = in.num_pages - L;
    }
    sync_all();
    for (int p = first; p < in.num_pages; p += threads) in.marks[p] = kIdle;
    flags = __reduce_or_sync(kAll, flags);
    if (flags && lane == 0) atomicOr(out.state + 1, (int)flags);
}

// ------------------------------------------------------------------ copy
constexpr int kPieceBytes = 8192;  // of a page of K or V (the smallest page's)
constexpr int kCopyStages = 8;     // pieces of a CTA in shared memory
constexpr int kCopyLead = 4;       // loads ahead of the stores
constexpr int kCopyCtas = 3;       // of an SM
constexpr int kCopySmem = kCopyStages * kPieceBytes;

__device__ __forceinline__ void bulk_store(void *dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
                 "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}

// Page copies[1 + c][0] to page copies[1 + c][1], K, V and (where there are block
// scales) their scales.  One warp per CTA, whose first lane keeps a ring of pieces
// moving through shared memory by bulk copies: four loads ahead of the stores.
__global__ void __launch_bounds__(32)
    copy_pages_kernel(const int32_t *copies, int cap, char *k, char *v, float *scale,
                      int num_pages, int pieces, int scale_vecs, int32_t *flags) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[kCopyStages];
    __shared__ char *to[kCopyStages];
    const int lane = threadIdx.x;
    if (lane == 0) {
        for (int s = 0; s < kCopyStages; ++s) mbar_init(&full[s], 1);
        fence_barrier_init();
    }
    __syncwarp();
    grid_dependency_wait();
    grid_launch_dependents();
    const int n = min(max(__ldg(copies), 0), cap);
    auto pair_of = [&](int c, int &src, int &dst) {
        src = __ldg(copies + 2 * (c + 1)), dst = __ldg(copies + 2 * (c + 1) + 1);
        return src >= 0 && src < num_pages && dst >= 0 && dst < num_pages;
    };
    if (lane == 0) {
        const long long items = (long long)n * 2 * pieces;
        const size_t page = (size_t)pieces * kPieceBytes;
        volatile int abort = 0;
        uint32_t loads = 0, stores = 0;
        auto store = [&]() {  // the next piece that has landed goes out
            const uint32_t s = stores % kCopyStages;
            if (!mbar_wait(&full[s], (stores / kCopyStages) & 1u, &abort)) return false;
            bulk_store(to[s], ring + s * kPieceBytes, kPieceBytes);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            ++stores;
            return true;
        };
        bool ok = true;
        for (long long it = blockIdx.x; ok && it < items; it += gridDim.x) {
            const int c = (int)(it / (2 * pieces)), piece = (int)(it - (long long)c * 2 * pieces);
            int src, dst;
            if (!pair_of(c, src, dst)) {
                if (piece == 0 && flags) atomicOr(flags, (int)HPC_FLAG_BAD_PAGE);
                continue;
            }
            char *cache = piece < pieces ? k : v;
            const size_t off = (size_t)(piece < pieces ? piece : piece - pieces) * kPieceBytes;
            const uint32_t s = loads % kCopyStages;
            // the piece that was in this place has been read out
            asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kCopyStages - 1 - kCopyLead)
                         : "memory");
            to[s] = cache + dst * page + off;
            mbar_arrive_expect_tx(&full[s], kPieceBytes);
            bulk_load(ring + s * kPieceBytes, cache + src * page + off, kPieceBytes, &full[s]);
            ++loads;
            if (loads - stores > kCopyLead) ok = store();
        }
        while (ok && stores < loads) ok = store();
        if (!ok) {  // no copy may land after the CTA has left (bounded)
            volatile int no_abort = 0;
            for (; stores < loads; ++stores)
                mbar_wait(&full[stores % kCopyStages], (stores / kCopyStages) & 1u, &no_abort);
            if (flags) atomicOr(flags, (int)HPC_FLAG_TIMEOUT);
        }
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    __syncwarp();
    for (int c = blockIdx.x; scale_vecs > 0 && c < n; c += gridDim.x) {
        int src, dst;
        if (!pair_of(c, src, dst)) continue;
        const float4 *a = reinterpret_cast<const float4 *>(scale) + (size_t)src * scale_vecs;
        float4 *b = reinterpret_cast<float4 *>(scale) + (size_t)dst * scale_vecs;
        for (int i = lane; i < scale_vecs; i += 32) b[i] = a[i];
    }
}

// ------------------------------------------------------------------ host side
bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

hpc_status status_of(cudaError_t e) { return e == cudaSuccess ? HPC_OK : HPC_ERR_CUDA; }

// A launch as a programmatic dependent of the previous kernel, as one cluster where
// `cluster` says so.
template <class... P, class... A>
cudaError_t launch_one(void (*kernel)(P...), int ctas, int threads, bool cluster, hpc_stream_t s,
                       A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = cluster ? 0 : kCopySmem;
    cfg.stream = static_cast<cudaStream_t>(s);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    if (cluster && ctas > 8) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The CTAs (a power of two) that hold `entries` with `own` to a thread.
int pool_ctas(int64_t entries, int own) {
    int n = 1;
    while (n < kPoolCtas && (int64_t)n * kPoolThreads * own < entries) n *= 2;
    return n;
}

// A call over list entries: few or many to a thread, in rounds.
template <class F, class... A>
hpc_status launch_list(F few, F many, int64_t entries, hpc_stream_t stream, A... args) {
    const int own = entries <= (int64_t)kPoolCtas * kPoolThreads * kFew ? kFew : kMany;
    const int ctas = pool_ctas(entries, own);
    const int64_t at_once = (int64_t)ctas * kPoolThreads * own;
    return status_of(launch_one(own == kFew ? few : many, ctas, kPoolThreads, true, stream, args...,
                                (int)((entries + at_once - 1) / at_once)));
}

hpc_status check_pool(const hpc_page_pool *p) {
    if (!p || !p->refs || !p->free_list || !p->state || !p->marks || p->num_pages <= 0)
        return HPC_ERR_ARG;
    return p->num_pages < kCodes ? HPC_OK : HPC_ERR_UNSUPPORTED;
}

Pool pool_of(const hpc_page_pool &p) {
    return {p.refs, p.free_list, p.state, p.marks, p.num_pages};
}

hpc_status check_rows(const int32_t *table, int32_t B, int32_t max_pages, const int32_t *rows,
                      int32_t n) {
    if (B < 0 || n < 0 || max_pages <= 0) return HPC_ERR_ARG;
    if (B > HPC_MAX_BATCH || n > HPC_MAX_BATCH) return HPC_ERR_UNSUPPORTED;
    // list entries and token indices stay in int32
    if ((int64_t)n * max_pages >= kCodes ||
        (int64_t)max_pages * HPC_PAGE_SIZE >= (int64_t)1 << 30)
        return HPC_ERR_UNSUPPORTED;
    if (!rows && n > B) return HPC_ERR_ARG;
    if (n > 0 && !table) return HPC_ERR_ARG;
    return HPC_OK;
}

}  // namespace
}  // namespace hpc

using namespace hpc;

extern "C" {

hpc_status hpc_kv_free(const hpc_page_pool *pool, int32_t *d_block_table, int32_t B,
                       int32_t max_pages_per_req, const int32_t *d_rows, const int32_t *d_keep,
                       int32_t n, hpc_stream_t stream) {
    hpc_status st = check_pool(pool);
    if (st == HPC_OK) st = check_rows(d_block_table, B, max_pages_per_req, d_rows, n);
    if (st != HPC_OK || n == 0) return st;
    const Rows t = {d_block_table, d_rows, B, max_pages_per_req, n};
    return launch_list(free_kernel<kFew>, free_kernel<kMany>, (int64_t)n * max_pages_per_req,
                       stream, pool_of(*pool), t, d_keep);
}

hpc_status hpc_kv_extend(const hpc_page_pool *pool, int32_t *d_block_table, int32_t B,
                         int32_t max_pages_per_req, const int32_t *d_rows, const int32_t *d_lens,
                         int32_t n, hpc_stream_t stream) {
    hpc_status st = check_pool(pool);
    if (st == HPC_OK) st = check_rows(d_block_table, B, max_pages_per_req, d_rows, n);
    if (st != HPC_OK || n == 0) return st;
    if (!d_lens) return HPC_ERR_ARG;
    const Rows t = {d_block_table, d_rows, B, max_pages_per_req, n};
    return launch_list(extend_kernel<kFew>, extend_kernel<kMany>, (int64_t)n * max_pages_per_req,
                       stream, pool_of(*pool), t, d_lens);
}

hpc_status hpc_kv_fork(const hpc_page_pool *pool, int32_t *d_block_table, int32_t B,
                       int32_t max_pages_per_req, const int32_t *d_src, const int32_t *d_dst,
                       const int32_t *d_lens, int32_t n, int32_t *d_copies, int32_t cap_copies,
                       hpc_stream_t stream) {
    hpc_status st = check_pool(pool);
    if (st == HPC_OK) st = check_rows(d_block_table, B, max_pages_per_req, d_dst, n);
    if (st != HPC_OK) return st;
    if (cap_copies < 0 || !d_copies) return HPC_ERR_ARG;
    if (cap_copies < n) return HPC_ERR_WORKSPACE;
    if (n > 0 && (!d_src || !d_dst || !d_lens)) return HPC_ERR_ARG;
    const Rows t = {d_block_table, d_dst, B, max_pages_per_req, n};
    const Fork f = {d_src, d_lens, d_copies};
    // (a warp takes kForkPages entries at a time)
    return status_of(launch_one(fork_kernel,
                                pool_ctas((int64_t)n * max_pages_per_req, kForkPages / 32),
                                kPoolThreads, true, stream, pool_of(*pool), t, f));
}

hpc_status hpc_kv_compact(const hpc_page_pool *pool, const int32_t *d_block_table, int32_t B,
                          int32_t max_pages_per_req, int32_t *d_copies, int32_t cap_copies,
                          int32_t *d_block_table_out, const hpc_page_pool *pool_out,
                          hpc_stream_t stream) {
    hpc_status st = check_pool(pool);
    if (st == HPC_OK) st = check_pool(pool_out);
    if (st != HPC_OK) return st;
    if (B < 0 || max_pages_per_req <= 0 || cap_copies < 0 || !d_copies) return HPC_ERR_ARG;
    if (pool_out->num_pages != pool->num_pages) return HPC_ERR_ARG;
    // one pool, or two that share nothing that is written
    const bool one = pool_out->refs == pool->refs;
    if ((pool_out->free_list == pool->free_list) != one || (pool_out->state == pool->state) != one)
        return HPC_ERR_ARG;
    if (B > 0 && (!d_block_table || !d_block_table_out)) return HPC_ERR_ARG;
    if (cap_copies < pool->num_pages / 2) return HPC_ERR_WORKSPACE;
    const int64_t entries = (int64_t)B * max_pages_per_req;
    return status_of(launch_one(compact_kernel,
                                pool_ctas(std::max<int64_t>(entries, pool->num_pages), kUnroll),
                                kPoolThreads, true, stream, pool_of(*pool), pool_of(*pool_out),
                                d_block_table, d_block_table_out, entries, d_copies));
}

hpc_status hpc_kv_copy_pages(const int32_t *d_copies, int32_t cap_copies, void *d_k_cache,
                             void *d_v_cache, float *d_kv_scale, hpc_kv_dtype kv_dtype,
                             int32_t num_pages, int32_t Hkv, int32_t head_dim, int32_t *d_flags,
                             hpc_stream_t stream) {
    if (cap_copies < 0 || num_pages <= 0 || Hkv <= 0) return HPC_ERR_ARG;
    if (head_dim != HPC_HEAD_DIM) return HPC_ERR_UNSUPPORTED;
    if (kv_dtype != HPC_KV_BF16 && kv_dtype != HPC_KV_FP8_E4M3 && kv_dtype != HPC_KV_E4M3_BLOCK)
        return HPC_ERR_ARG;
    if ((kv_dtype == HPC_KV_E4M3_BLOCK) != (d_kv_scale != nullptr)) return HPC_ERR_ARG;
    if (!d_copies || !d_k_cache || !d_v_cache) return HPC_ERR_ARG;
    if (!aligned(d_k_cache, 16) || !aligned(d_v_cache, 16) || !aligned(d_kv_scale, 16))
        return HPC_ERR_ARG;
    const int64_t page = (int64_t)HPC_PAGE_SIZE * Hkv * HPC_HEAD_DIM *
                         (kv_dtype == HPC_KV_BF16 ? 2 : 1);
    if (page >= (int64_t)1 << 30) return HPC_ERR_UNSUPPORTED;
    if (cap_copies == 0) return HPC_OK;
    const int pieces = (int)(page / kPieceBytes);
    const int scale_vecs = kv_dtype == HPC_KV_E4M3_BLOCK ? Hkv * 2 : 0;
    static std::atomic<int> sms_of[64];  // per device, once the kernel's attribute is set
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return HPC_ERR_CUDA;
    int sms = sms_of[dev].load();
    if (sms == 0) {
        if (cudaFuncSetAttribute(copy_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kCopySmem) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return HPC_ERR_CUDA;
        sms_of[dev].store(sms);
    }
    const int grid = (int)std::min<int64_t>((int64_t)cap_copies * 2 * pieces, (int64_t)sms * kCopyCtas);
    return status_of(launch_one(copy_pages_kernel, grid, 32, false, stream, d_copies, cap_copies,
                                static_cast<char *>(d_k_cache), static_cast<char *>(d_v_cache),
                                d_kv_scale, num_pages, pieces, scale_vecs, d_flags));
}

}  // extern "C"
