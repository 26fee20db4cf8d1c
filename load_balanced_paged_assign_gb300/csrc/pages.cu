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
// Each call's bookkeeping is one launch of one cluster of CTAs: its phases (count,
// place, write) follow one another at cluster barriers, the warps' totals pass
// through distributed shared memory.  A warp holds consecutive entries, so a prefix
// sum is a ballot per 32 entries and one sum over the warps.
//
// All of it is latency: a few dependent reads per entry (table, count, stack).  The
// copies that a fork or a compaction lists (pages moved in every layer's cache) are
// a kernel of their own, which HBM bounds.
#include <cooperative_groups.h>

#include <algorithm>
#include <climits>

#include "internal.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace hpc {
namespace {

constexpr int kPoolThreads = 1024;
constexpr int kPoolWarps = kPoolThreads / 32;
constexpr int kPoolCtas = 8;          // of a cluster (the portable limit)
constexpr int kOneCtaEntries = 4096;  // up to here one CTA is quicker than a cluster
constexpr int kIdle = INT_MAX;        // marks[p] between calls
// Numbers below -2^30 in the table are the calls' own, and gone when they end: a page
// taken from an entry, or the list's place that claims an empty one (the smaller wins).
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

__device__ __forceinline__ int row_of(const Rows &t, int i) { return t.rows ? __ldg(t.rows + i) : i; }

// The entries of one warp: a consecutive range of the call's.
struct Part {
    int lo, hi;
};

__device__ __forceinline__ Part part_of(int entries) {
    const int warps = (int)gridDim.x * kPoolWarps;
    const int w = (int)blockIdx.x * kPoolWarps + (int)(threadIdx.x >> 5);
    const int per = ((entries + warps - 1) / warps + 31) & ~31;
    const long long lo = (long long)w * per;
    return {(int)min(lo, (long long)entries), (int)min(lo + per, (long long)entries)};
}

struct Totals {
    int warp[kPoolWarps];
    int cta;
};

// The entries counted by the warps before this one, and by all: `count` is the
// warp's.  A barrier of the cluster: what its threads wrote before, all of them see.
__device__ int cluster_base(int count, Totals &t, int &total) {
    cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    if (lane == 0) t.warp[w] = count;
    __syncthreads();
    int mine = t.warp[lane], before = 0;
    const int cta = __reduce_add_sync(kAll, mine);
    before = __reduce_add_sync(kAll, lane < w ? mine : 0);
    if (threadIdx.x == 0) t.cta = cta;
    cluster.sync();
    total = 0;
    for (unsigned c = 0; c < cluster.num_blocks(); ++c) {
        const int n = cluster.map_shared_rank(&t, c)->cta;
        if (c < cluster.block_rank()) before += n;
        total += n;
    }
    return before;
}

// Goes over the warp's entries 32 at a time: pred(e) for each, emit(e, rank) for
// those that it holds for, ranked from `base`.  Returns how many there were.
template <class Pred, class Emit>
__device__ __forceinline__ int ranked(const Part &part, int base, Pred pred, Emit emit) {
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (int e0 = part.lo; e0 < part.hi; e0 += 32) {
        const int e = e0 + lane;
        const bool yes = e < part.hi && pred(e);
        const unsigned vote = __ballot_sync(kAll, yes);
        if (yes) emit(e, base + n + __popc(vote & ((1u << lane) - 1u)));
        n += __popc(vote);
    }
    return n;
}

struct Nothing {
    __device__ void operator()(int, int) const {}
};

__device__ __forceinline__ int code_of(int x) { return INT_MIN + x; }
// what an entry's code stands for, -1 if it holds none below `limit`
__device__ __forceinline__ int decoded(int v, int limit) {
    const unsigned x = (unsigned)v ^ 0x80000000u;
    return x < (unsigned)limit ? (int)x : -1;
}

// How many pages the stack can hold or hand out, whatever its count says.
__device__ __forceinline__ int stack_top(const Pool &pool) {
    return min(max(__ldcg(pool.state), 0), pool.num_pages);
}

// ------------------------------------------------------------------ give back
// Entries from ceil(keep / 64) on: each loses its page; a page that none holds any
// more goes back on the stack.  An entry is taken by exchanging a code of its page
// for it, so a row that is named twice gives its pages back once; of a page's entries
// taken here the first in the list places it (marks).
__global__ void __launch_bounds__(kPoolThreads) free_kernel(const Pool pool, const Rows t,
                                                            const int32_t *keep) {
    __shared__ Totals totals;
    cg::cluster_group cluster = cg::this_cluster();
    grid_dependency_wait();
    grid_launch_dependents();
    const int entries = t.n * t.max_pages;
    const Part part = part_of(entries);
    unsigned flags = 0;
    // the table entry of list entry e, or null
    auto entry = [&](int e) -> int32_t * {
        const int i = e / t.max_pages, j = e - i * t.max_pages, r = row_of(t, i);
        const int k = keep ? __ldg(keep + i) : 0;
        if (r < 0 || r >= t.B || k < 0 || k > t.max_pages * kTile) {
            flags |= HPC_FLAG_BAD_SEQLEN;
            return nullptr;
        }
        return j < (k + kTile - 1) / kTile ? nullptr : t.table + (size_t)r * t.max_pages + j;
    };
    const int top = stack_top(pool);
    for (int e = part.lo + (int)(threadIdx.x & 31); e < part.hi; e += 32) {
        int32_t *at = entry(e);
        if (!at) continue;
        int p = __ldcg(at);
        if (p < 0) continue;
        const bool good = p < pool.num_pages;
        p = atomicExch(at, good ? code_of(p) : -1);
        if (p < 0) continue;  // taken by another entry of the same row
        if (!good) {
            flags |= HPC_FLAG_BAD_PAGE;
        } else if (atomicSub(pool.refs + p, 1) <= 0) {  // held by none
            atomicAdd(pool.refs + p, 1);
            atomicExch(at, -1);
            flags |= HPC_FLAG_BAD_PAGE;
        } else {
            atomicMin(pool.marks + p, e);
        }
    }
    cluster.sync();
    // the page that entry e puts on the stack, or -1
    auto back = [&](int e) {
        const int32_t *at = entry(e);
        if (!at) return -1;
        const int p = decoded(__ldcg(at), pool.num_pages);
        return p >= 0 && __ldcg(pool.marks + p) == e && __ldcg(pool.refs + p) == 0 ? p : -1;
    };
    const int mine = ranked(part, 0, [&](int e) { return back(e) >= 0; }, Nothing());
    int total;
    const int base = cluster_base(mine, totals, total);
    if (mine > 0)  // the list's first page comes to lie on top
        ranked(part, base, [&](int e) { return back(e) >= 0; },
               [&](int e, int rank) {
                   const int at = top + total - 1 - rank;
                   if (at < pool.num_pages) pool.stack[at] = back(e);
               });
    cluster.sync();
    for (int e = part.lo + (int)(threadIdx.x & 31); e < part.hi; e += 32) {
        int32_t *at = entry(e);
        if (!at) continue;
        const int p = decoded(__ldcg(at), pool.num_pages);
        if (p < 0) continue;
        pool.marks[p] = kIdle;
        *at = -1;
    }
    if (top + total > pool.num_pages) flags |= HPC_FLAG_BAD_PAGE;
    flags = __reduce_or_sync(kAll, flags);
    if (flags && (threadIdx.x & 31) == 0) atomicOr(pool.state + 1, (int)flags);
    if (blockIdx.x == 0 && threadIdx.x == 0) pool.state[0] = min(top + total, pool.num_pages);
}

// ------------------------------------------------------------------ take
// Negative entries below ceil(lens / 64) take a page each, or, where the stack has
// not enough for all, none does.  An entry is claimed first, and the first of the list
// wins, so a row that is named twice is served once.
__global__ void __launch_bounds__(kPoolThreads) extend_kernel(const Pool pool, const Rows t,
                                                              const int32_t *lens) {
    __shared__ Totals totals;
    cg::cluster_group cluster = cg::this_cluster();
    grid_dependency_wait();
    grid_launch_dependents();
    const int entries = t.n * t.max_pages;
    const Part part = part_of(entries);
    unsigned flags = 0;
    auto entry = [&](int e) -> int32_t * {
        const int i = e / t.max_pages, j = e - i * t.max_pages, r = row_of(t, i);
        const int L = __ldg(lens + i);
        if (r < 0 || r >= t.B || L < 0 || L > t.max_pages * kTile) {
            flags |= HPC_FLAG_BAD_SEQLEN;
            return nullptr;
        }
        return j < (L + kTile - 1) / kTile ? t.table + (size_t)r * t.max_pages + j : nullptr;
    };
    auto claimed = [&](int e) {
        const int32_t *at = entry(e);
        return at && __ldcg(at) == code_of(e);
    };
    const int top = stack_top(pool);
    for (int e = part.lo + (int)(threadIdx.x & 31); e < part.hi; e += 32) {
        int32_t *at = entry(e);
        if (!at) continue;
        if (__ldcg(at) < 0) atomicMin(at, code_of(e));
    }
    cluster.sync();
    const int mine = ranked(part, 0, claimed, Nothing());
    int total;
    const int base = cluster_base(mine, totals, total);
    const bool enough = total <= top;
    if (mine > 0)
        ranked(part, base, claimed, [&](int e, int rank) {
            int32_t *at = entry(e);
            const int p = enough ? __ldcg(pool.stack + (top - 1 - rank)) : -1;
            if (enough && (p < 0 || p >= pool.num_pages)) {
                flags |= HPC_FLAG_BAD_PAGE;
                *at = -1;
                return;
            }
            *at = p;
            if (enough) pool.refs[p] = 1;
        });
    if (!enough) flags |= HPC_FLAG_NO_PAGES;
    flags = __reduce_or_sync(kAll, flags);
    if (flags && (threadIdx.x & 31) == 0) atomicOr(pool.state + 1, (int)flags);
    if (enough && blockIdx.x == 0 && threadIdx.x == 0) pool.state[0] = top - total;
    cluster.sync();  // no CTA leaves while another may read its shared memory
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
    const int first = (int)blockIdx.x * kPoolThreads + threadIdx.x;
    const int threads = (int)gridDim.x * kPoolThreads;
    for (int i = threadIdx.x; i < HPC_MAX_BATCH / 32; i += kPoolThreads) bad[i] = 0;
    cluster.sync();
    unsigned flags = 0;
    unsigned *bad0 = cluster.map_shared_rank(bad, 0);
    auto refuse = [&](int i) { atomicOr(bad0 + (i >> 5), 1u << (i & 31)); };
    const int cap = t.max_pages * kTile, top = stack_top(pool);
    for (int i = first; i < t.n; i += threads) {
        const int s = __ldg(f.src + i), d = row_of(t, i), L = __ldg(f.lens + i);
        if (s < 0 || s >= t.B || d < 0 || d >= t.B || s == d || L < 0 || L > cap) {
            flags |= HPC_FLAG_BAD_SEQLEN;
            refuse(i);
        } else if (L > 0) {
            int32_t *at = t.table + (size_t)d * t.max_pages;
            if (__ldcg(at) < 0) atomicMin(at, code_of(i));
        }
    }
    cluster.sync();
    const int entries = t.n * t.max_pages;
    for (int e = first; e < entries; e += threads) {
        const int i = e / t.max_pages, j = e - i * t.max_pages;
        const int s = __ldg(f.src + i), d = row_of(t, i), L = __ldg(f.lens + i);
        if (s < 0 || s >= t.B || d < 0 || d >= t.B || s == d || L < 0 || L > cap) continue;
        if (j >= (L + kTile - 1) / kTile) continue;
        const int p = __ldcg(t.table + (size_t)s * t.max_pages + j);
        const int q = __ldcg(t.table + (size_t)d * t.max_pages + j);
        if (p < 0 || p >= pool.num_pages || __ldcg(pool.refs + p) <= 0) {
            flags |= HPC_FLAG_BAD_PAGE;
            refuse(i);
        } else if (j == 0 ? q != code_of(i) : q >= 0) {
            flags |= HPC_FLAG_BAD_SEQLEN;  // the row is not empty, or another child's
            refuse(i);
        }
    }
    cluster.sync();
    for (int w = threadIdx.x; w < (t.n + 31) / 32; w += kPoolThreads)
        if (blockIdx.x > 0) bad[w] = bad0[w];
    __syncthreads();
    auto refused = [&](int i) { return (bad[i >> 5] >> (i & 31) & 1u) != 0; };
    // the children that need a page of their own
    auto partial = [&](int i) { return !refused(i) && __ldg(f.lens + i) % kTile != 0; };
    const Part part = part_of(t.n);
    const int mine = ranked(part, 0, partial, Nothing());
    int total;
    const int base = cluster_base(mine, totals, total);
    const bool enough = total <= top;
    if (enough && mine > 0)
        ranked(part, base, partial, [&](int i, int rank) {
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
        });
    for (int e = first; e < entries; e += threads) {
        const int i = e / t.max_pages, j = e - i * t.max_pages;
        const int d = row_of(t, i);
        if (refused(i) || !enough) {  // the claim, where it is this child's, is withdrawn
            if (j == 0 && d >= 0 && d < t.B)
                atomicCAS(t.table + (size_t)d * t.max_pages, code_of(i), -1);
        } else if (j < __ldg(f.lens + i) / kTile) {
            const int p = __ldcg(t.table + (size_t)__ldg(f.src + i) * t.max_pages + j);
            t.table[(size_t)d * t.max_pages + j] = p;
            atomicAdd(pool.refs + p, 1);
        }
    }
    if (!enough) flags |= HPC_FLAG_NO_PAGES;
    flags = __reduce_or_sync(kAll, flags);
    if (flags && (threadIdx.x & 31) == 0) atomicOr(pool.state + 1, (int)flags);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        f.copies[0] = enough ? total : 0;
        f.copies[1] = 0;
        if (enough) pool.state[0] = top - total;
    }
    cluster.sync();  // no CTA leaves while another may read its shared memory
}

// ------------------------------------------------------------------ compact
// The live pages behind the first L places (L live ones in all) move, in order,
// into the holes among those; marks[p] holds a moved page's new place meanwhile.
__global__ void __launch_bounds__(kPoolThreads)
    compact_kernel(const Pool in, const Pool out, const int32_t *table, int32_t *table_out,
                   int64_t entries, int32_t *copies) {
    __shared__ Totals totals;
    cg::cluster_group cluster = cg::this_cluster();
    grid_dependency_wait();
    grid_launch_dependents();
    const int first = (int)blockIdx.x * kPoolThreads + threadIdx.x;
    const int threads = (int)gridDim.x * kPoolThreads;
    const Part part = part_of(in.num_pages);
    auto live = [&](int p) { return __ldcg(in.refs + p) > 0; };
    int L, holes;
    const int n_live = ranked(part, 0, live, Nothing());
    cluster_base(n_live, totals, L);
    auto hole = [&](int p) { return p < L && !live(p); };
    auto far = [&](int p) { return p >= L && live(p); };
    const int n_holes = ranked(part, 0, hole, Nothing());
    cluster.sync();
    const int hole_base = cluster_base(n_holes, totals, holes);
    const int n_far = ranked(part, 0, far, Nothing());
    cluster.sync();
    int moves;
    const int far_base = cluster_base(n_far, totals, moves);  // (as many as holes)
    if (n_holes > 0)
        ranked(part, hole_base, hole, [&](int p, int k) { copies[2 * (k + 1) + 1] = p; });
    if (n_far > 0) ranked(part, far_base, far, [&](int p, int k) { copies[2 * (k + 1)] = p; });
    cluster.sync();
    for (int k = first; k < moves; k += threads) {
        const int src = __ldcg(copies + 2 * (k + 1)), dst = __ldcg(copies + 2 * (k + 1) + 1);
        in.marks[src] = dst;
        out.refs[dst] = __ldcg(in.refs + src);
    }
    cluster.sync();
    for (int64_t e = first; e < entries; e += threads) {
        const int p = __ldcg(table + e);
        int to = p;
        if (p >= 0 && p < in.num_pages) {
            const int m = __ldcg(in.marks + p);
            if (m != kIdle) to = m;
        }
        table_out[e] = to;
    }
    for (int p = first; p < in.num_pages; p += threads) {
        if (p >= L) out.refs[p] = 0;
        else if (out.refs != in.refs && live(p)) out.refs[p] = __ldcg(in.refs + p);
        if (p < in.num_pages - L) out.stack[p] = in.num_pages - 1 - p;
    }
    if (first >= 1 && first < 4 && out.state != in.state) out.state[first] = __ldcg(in.state + first);
    if (first == 0) {
        copies[0] = moves;
        copies[1] = 0;
        out.state[0] = in.num_pages - L;
    }
    cluster.sync();
    for (int k = first; k < moves; k += threads) in.marks[__ldcg(copies + 2 * (k + 1))] = kIdle;
}

// ------------------------------------------------------------------ copy
constexpr int kCopyThreads = 256;
constexpr int kPieceBytes = 4096;  // of a page of K or V, for one warp

__device__ __forceinline__ void load32(const void *p, uint32_t (&r)[8]) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "l"(p)
                 : "memory");
}

__device__ __forceinline__ void store32(void *p, const uint32_t (&r)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Page copies[1 + c][0] to page copies[1 + c][1], K, V and (where there are block
// scales) their scales.  A warp takes a piece of 4 KB at a time, all of its loads in
// flight together.
__global__ void __launch_bounds__(kCopyThreads)
    copy_pages_kernel(const int32_t *copies, int cap, char *k, char *v, float *scale,
                      int num_pages, int pieces, int scale_vecs, int32_t *flags) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int warps = (int)gridDim.x * (kCopyThreads / 32);
    const int n = min(max(__ldg(copies), 0), cap);
    const int per = 2 * pieces + (scale_vecs > 0 ? 1 : 0);  // a copy's items
    const long long items = (long long)n * per;
    for (long long it = (long long)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5);
         it < items; it += warps) {
        const int c = (int)(it / per), piece = (int)(it - (long long)c * per);
        const int src = __ldg(copies + 2 * (c + 1)), dst = __ldg(copies + 2 * (c + 1) + 1);
        if (src < 0 || src >= num_pages || dst < 0 || dst >= num_pages) {
            if (lane == 0 && piece == 0 && flags) atomicOr(flags, (int)HPC_FLAG_BAD_PAGE);
            continue;
        }
        if (piece == 2 * pieces) {
            const float4 *a = reinterpret_cast<const float4 *>(scale) + (size_t)src * scale_vecs;
            float4 *b = reinterpret_cast<float4 *>(scale) + (size_t)dst * scale_vecs;
            for (int i = lane; i < scale_vecs; i += 32) b[i] = a[i];
            continue;
        }
        char *cache = piece < pieces ? k : v;
        const size_t off = (size_t)(piece < pieces ? piece : piece - pieces) * kPieceBytes + lane * 32;
        const size_t page = (size_t)pieces * kPieceBytes;
        const char *a = cache + src * page + off;
        char *b = cache + dst * page + off;
        uint32_t x[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) load32(a + i * 1024, x[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) store32(b + i * 1024, x[i]);
    }
}

// ------------------------------------------------------------------ host side
bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A launch as a programmatic dependent of the previous kernel, as one cluster where
// `cluster` says so.
template <class... P, class... A>
cudaError_t launch_one(void (*kernel)(P...), int ctas, int threads, bool cluster, hpc_stream_t s,
                       A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = static_cast<cudaStream_t>(s);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

int pool_ctas(int64_t entries) { return entries <= kOneCtaEntries ? 1 : kPoolCtas; }

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

hpc_status status_of(cudaError_t e) { return e == cudaSuccess ? HPC_OK : HPC_ERR_CUDA; }

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
    return status_of(launch_one(free_kernel, pool_ctas((int64_t)n * max_pages_per_req),
                                kPoolThreads, true, stream, pool_of(*pool), t, d_keep));
}

hpc_status hpc_kv_extend(const hpc_page_pool *pool, int32_t *d_block_table, int32_t B,
                         int32_t max_pages_per_req, const int32_t *d_rows, const int32_t *d_lens,
                         int32_t n, hpc_stream_t stream) {
    hpc_status st = check_pool(pool);
    if (st == HPC_OK) st = check_rows(d_block_table, B, max_pages_per_req, d_rows, n);
    if (st != HPC_OK || n == 0) return st;
    if (!d_lens) return HPC_ERR_ARG;
    const Rows t = {d_block_table, d_rows, B, max_pages_per_req, n};
    return status_of(launch_one(extend_kernel, pool_ctas((int64_t)n * max_pages_per_req),
                                kPoolThreads, true, stream, pool_of(*pool), t, d_lens));
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
    return status_of(launch_one(fork_kernel, pool_ctas((int64_t)n * max_pages_per_req),
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
                                pool_ctas(std::max<int64_t>(entries, pool->num_pages)),
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
    if (!aligned(d_k_cache, 32) || !aligned(d_v_cache, 32) || !aligned(d_kv_scale, 16))
        return HPC_ERR_ARG;
    const int64_t page = (int64_t)HPC_PAGE_SIZE * Hkv * HPC_HEAD_DIM *
                         (kv_dtype == HPC_KV_BF16 ? 2 : 1);
    if (page >= (int64_t)1 << 30) return HPC_ERR_UNSUPPORTED;
    if (cap_copies == 0) return HPC_OK;
    const int pieces = (int)(page / kPieceBytes);
    const int scale_vecs = kv_dtype == HPC_KV_E4M3_BLOCK ? Hkv * 2 : 0;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return HPC_ERR_CUDA;
    const int64_t warps = (int64_t)cap_copies * (2 * pieces + (scale_vecs > 0));
    const int grid = (int)std::min<int64_t>((warps + kCopyThreads / 32 - 1) / (kCopyThreads / 32),
                                            (int64_t)sms * 6);
    return status_of(launch_one(copy_pages_kernel, grid, kCopyThreads, false, stream, d_copies,
                                cap_copies, static_cast<char *>(d_k_cache),
                                static_cast<char *>(d_v_cache), d_kv_scale, num_pages, pieces,
                                scale_vecs, d_flags));
}

}  // extern "C"
