// fd_pages.cu -- page bookkeeping of a paged cache: freeing, forking,
// reserving (with copy on write), compacting, and the copies of pages that
// the last two ask for.
//
// refs[p] counts the block-table entries that name page p; a page with no
// reference is free.  Every choice is by number (lowest free page, sequences
// in order), and the integer atomics only add or take minima, so the same
// books give the same books whatever order blocks run in.
//
// What bounds these: a few thousand table entries and reference counts are
// read and written, so the time is dependent loads and barriers, not bytes.
// reserve and compact need ranks over the whole pool, hence barriers; they run
// as one thread-block cluster, whose barrier costs far less than another
// launch, with a warp per run of sequences and per run of pages.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <atomic>

#include "fd.h"
#include "fd_internal.h"
#include "fd_pages.h"

namespace fd {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ void flag(const Books &k, int bit) { atomicOr(k.status, bit); }

__device__ __forceinline__ int pages_of(int64_t positions, int page_size) {
    return (int)((positions + page_size - 1) / page_size);
}

// Takes back one reference to page e (a page that has none left is flagged).
__device__ __forceinline__ void drop(const Books &k, int e) {
    if (e < 0) return;
    if (e >= k.num_pages) {
        flag(k, FD_DEV_BAD_INDEX);
        return;
    }
    if (atomicSub(k.refs + e, 1) <= 0) {
        atomicAdd(k.refs + e, 1);
        flag(k, FD_DEV_BAD_INDEX);
    }
}

// The sequence's length, kept within what its row can hold.
__device__ __forceinline__ int64_t held(const Books &k, int b) {
    const int64_t raw = k.lengths[b], cap = (int64_t)k.max_pages * k.page_size;
    if (raw < 0 || raw > cap) flag(k, FD_DEV_BAD_LENGTH);
    return clamp_len(raw, cap);
}

// One block per listed sequence.  A sequence listed twice ends at the smaller
// length: an entry is released by whoever exchanges it for -1.
__global__ void free_kernel(const Books k, const int32_t *seqs, const int32_t *lengths, int n) {
    const int i = blockIdx.x;
    const int b = seqs ? seqs[i] : i;
    if (b < 0 || b >= k.B) {
        if (threadIdx.x == 0) flag(k, FD_DEV_BAD_INDEX);
        return;
    }
    int64_t L = 0;
    if (lengths) {
        const int64_t want = lengths[i];
        L = min(held(k, b), want < 0 ? (int64_t)0 : want);
    }
    int32_t *row = k.table + (int64_t)b * k.max_pages;
    for (int j = pages_of(L, k.page_size) + threadIdx.x; j < k.max_pages; j += blockDim.x)
        if (row[j] != -1) drop(k, atomicExch(row + j, -1));
    if (threadIdx.x == 0) {
        if (L == 0) k.lengths[b] = 0;
        else atomicMin(k.lengths + b, (int)L);
    }
}

// One block per (src, dst).  Rows are read as they stood before the call: an
// entry whose dst is another entry's source, or an earlier entry's dst, is
// left out and flagged.
__global__ void fork_kernel(const Books k, const int32_t *src, const int32_t *dst,
                            const int32_t *lengths, int n) {
    const int i = blockIdx.x;
    const int s = src[i], d = dst[i];
    bool bad = s < 0 || s >= k.B || d < 0 || d >= k.B;
    if (!bad && s == d) return;
    if (!bad)
        for (int o = threadIdx.x; o < n; o += blockDim.x)
            bad |= (o < i && dst[o] == d) || (o != i && src[o] == d && dst[o] != d);
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) flag(k, FD_DEV_BAD_INDEX);
        return;
    }
    int64_t L = held(k, s);
    if (lengths) {
        const int64_t want = lengths[i];
        L = min(L, want < 0 ? (int64_t)0 : want);
    }
    const int share = pages_of(L, k.page_size);
    const int32_t *from = k.table + (int64_t)s * k.max_pages;
    int32_t *to = k.table + (int64_t)d * k.max_pages;
    for (int j = threadIdx.x; j < k.max_pages; j += blockDim.x) {
        int e = j < share ? from[j] : -1;
        if (e >= k.num_pages || (e < 0 && j < share)) {
            flag(k, FD_DEV_BAD_INDEX);
            e = -1;
        }
        const int old = to[j];
        if (old == e) continue;
        if (e >= 0) atomicAdd(k.refs + e, 1);
        drop(k, old);
        to[j] = e;
    }
    if (threadIdx.x == 0) k.lengths[d] = (int)L;
}

// ------------------------------------------------------------ one cluster
// Totals that each warp of the cluster contributes, and the sums over the
// warps before this one and over all.
struct Totals {
    int need, spare, copies;
};

struct Cluster {
    int rank, size, warp, warps;   // block in the cluster; warp in the cluster
    __device__ __forceinline__ Cluster() {
        auto c = cg::this_cluster();
        rank = (int)c.block_rank();
        size = (int)c.num_blocks();
        warp = rank * kWarps + (int)(threadIdx.x >> 5);
        warps = size * kWarps;
    }
    __device__ __forceinline__ void sync() const {
        if (size == 1) __syncthreads();
        else cg::this_cluster().sync();
    }
};

// Sums `mine` over the warps before this one (before) and over all (all).
// `shared`: kWarps entries of this block; every thread of the cluster calls
// it, `mine` is uniform over a warp.
__device__ __forceinline__ void scan(const Cluster &c, Totals *shared, const Totals &mine,
                                     Totals &before, Totals &all) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) shared[threadIdx.x >> 5] = mine;
    c.sync();
    before = all = Totals{0, 0, 0};
    for (int r = 0; r < c.size; ++r) {
        const Totals *t = c.size == 1 ? shared : cg::this_cluster().map_shared_rank(shared, r);
        Totals x = t[lane], y = x;
        if (r * kWarps + lane >= c.warp) y = Totals{0, 0, 0};
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            x.need += __shfl_xor_sync(kAll, x.need, o);
            x.spare += __shfl_xor_sync(kAll, x.spare, o);
            x.copies += __shfl_xor_sync(kAll, x.copies, o);
            y.need += __shfl_xor_sync(kAll, y.need, o);
            y.spare += __shfl_xor_sync(kAll, y.spare, o);
            y.copies += __shfl_xor_sync(kAll, y.copies, o);
        }
        all.need += x.need; all.spare += x.spare; all.copies += x.copies;
        before.need += y.need; before.spare += y.spare; before.copies += y.copies;
    }
}

struct ReserveArgs {
    Books k;
    const int32_t *n_new;
    int32_t n_each;
    int32_t *pairs, *count;
    int32_t *writers, *first, *list;   // scratch, num_pages words each
};

// Table entries [lo, hi) of sequence b that will be written, and its length.
__device__ __forceinline__ void write_range(const ReserveArgs &a, int b, int &lo, int &hi, int64_t &L,
                                            bool report) {
    const Books &k = a.k;
    const int64_t cap = (int64_t)k.max_pages * k.page_size;
    const int64_t raw = k.lengths[b];
    const int64_t want = a.n_new ? a.n_new[b] : a.n_each;
    L = clamp_len(raw, cap);
    const int64_t end = clamp_len(L + (want < 0 ? 0 : want), cap);
    if (report && (raw != L || want < 0 || L + want > cap)) flag(k, FD_DEV_BAD_LENGTH);
    lo = (int)(L / k.page_size);
    hi = end > L ? pages_of(end, k.page_size) : lo;
}

// Entries of the write ranges that name no page, or a page that others name
// too, get pages of their own; the rest stay.  A sharer keeps the page when
// every holder writes in this call and it is the first of them (in order of
// sequences, then pages).
__global__ void __launch_bounds__(kThreads) reserve_kernel(const ReserveArgs a) {
    __shared__ Totals sums[kWarps], sums2[kWarps];
    const Books &k = a.k;
    const Cluster c;
    const int lane = threadIdx.x & 31;
    // sequences [b0, b1) and pages [p0, p1) of this warp
    const int per_b = (k.B + c.warps - 1) / c.warps;
    const int b0 = min(k.B, c.warp * per_b), b1 = min(k.B, b0 + per_b);
    const int per_p = ((k.num_pages + c.warps - 1) / c.warps + 31) / 32 * 32;
    const int p0 = (int)min((int64_t)k.num_pages, (int64_t)c.warp * per_p);
    const int p1 = min(k.num_pages, p0 + per_p);

    Totals mine{0, 0, 0}, before, all;
    // free pages of the warp's run, and how many of its entries are shared
    for (int q = p0; q < p1; q += 32)
        mine.spare += __popc(__ballot_sync(kAll, q + lane < p1 && k.refs[q + lane] <= 0));
    int shared = 0;
    for (int b = b0; b < b1; ++b) {
        int lo, hi;
        int64_t L;
        write_range(a, b, lo, hi, L, lane == 0);
        int32_t *row = k.table + (int64_t)b * k.max_pages;
        for (int j = lo + lane; j < hi; j += 32) {
            const int e = row[j];
            if (e < 0 || e >= k.num_pages) {
                if (e != -1) row[j] = -1;
                ++mine.need;
            } else if (k.refs[e] > 1) {
                a.writers[e] = 0;
                a.first[e] = 0x7fffffff;
                ++shared;
            }
        }
    }
    mine.need = __reduce_add_sync(kAll, mine.need);
    mine.copies = __reduce_add_sync(kAll, shared);
    scan(c, sums, mine, before, all);
    if (all.copies > 0) {
        // some written pages are shared: find each one's writers, then mark
        // the entries that part from it as -(page + 2)
        for (int b = b0; b < b1; ++b) {
            int lo, hi;
            int64_t L;
            write_range(a, b, lo, hi, L, false);
            const int32_t *row = k.table + (int64_t)b * k.max_pages;
            for (int j = lo + lane; j < hi; j += 32) {
                const int e = row[j];
                if (e >= 0 && k.refs[e] > 1) {
                    atomicAdd(a.writers + e, 1);
                    atomicMin(a.first + e, (int)((int64_t)b * k.max_pages + j));
                }
            }
        }
        c.sync();
        int parted = 0, copies = 0;
        for (int b = b0; b < b1; ++b) {
            int lo, hi;
            int64_t L;
            write_range(a, b, lo, hi, L, false);
            int32_t *row = k.table + (int64_t)b * k.max_pages;
            for (int j = lo + lane; j < hi; j += 32) {
                const int e = row[j];
                if (e < 0 || k.refs[e] <= 1) continue;
                if (a.writers[e] == k.refs[e] && a.first[e] == (int)((int64_t)b * k.max_pages + j)) continue;
                row[j] = -(e + 2);
                ++parted;
                if ((int64_t)j * k.page_size < L) ++copies;
            }
        }
        mine.need += __reduce_add_sync(kAll, parted);
        mine.copies = __reduce_add_sync(kAll, copies);
        scan(c, sums2, mine, before, all);
    }
    const bool fits = all.need <= all.spare;

    // the free pages, lowest first, as far as they are needed
    if (fits && before.spare < all.need) {
        int rank = before.spare;
        for (int q = p0; q < p1 && rank < all.need; q += 32) {
            const bool is = q + lane < p1 && k.refs[q + lane] <= 0;
            const unsigned m = __ballot_sync(kAll, is);
            if (is) a.list[rank + __popc(m & ((1u << lane) - 1))] = q + lane;
            rank += __popc(m);
        }
    }
    c.sync();
    int rank = before.need, pair = before.copies;
    for (int b = b0; b < b1; ++b) {
        int lo, hi;
        int64_t L;
        write_range(a, b, lo, hi, L, false);
        int32_t *row = k.table + (int64_t)b * k.max_pages;
        for (int j0 = lo; j0 < hi; j0 += 32) {
            const int j = j0 + lane;
            const int e = j < hi ? row[j] : 0;
            const bool need = e < 0;
            const unsigned m = __ballot_sync(kAll, need);
            const bool copy = e <= -2 && (int64_t)j * k.page_size < L;
            const unsigned mc = __ballot_sync(kAll, copy);
            if (need) {
                if (!fits) {
                    if (e <= -2) row[j] = -(e + 2);   // as it was
                } else {
                    const int got = a.list[rank + __popc(m & ((1u << lane) - 1))];
                    if (e <= -2) atomicSub(k.refs - (e + 2), 1);
                    if (copy) {
                        const int at = pair + __popc(mc & ((1u << lane) - 1));
                        a.pairs[2 * at] = -(e + 2);
                        a.pairs[2 * at + 1] = got;
                    }
                    k.refs[got] = 1;
                    row[j] = got;
                }
            }
            rank += __popc(m);
            pair += __popc(mc);
        }
    }
    if (c.warp == 0 && lane == 0) {
        *a.count = fits ? all.copies : -(all.need - all.spare);
        if (!fits) flag(k, FD_DEV_NO_PAGES);
    }
    // no block leaves while another may still read its shared memory
    c.sync();
}

struct CompactArgs {
    Books k;
    int32_t *pairs, *count;
    int32_t *goes;             // scratch [num_pages]: where a page past the used ones goes
    int32_t *holes, *movers;   // scratch [num_pages / 2] each
    int32_t *n_used;           // scratch [1]
};

// The i-th used page at or past n_used moves to the i-th free page below it.
__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactArgs a) {
    __shared__ Totals sums[kWarps], sums2[kWarps];
    const Books &k = a.k;
    const Cluster c;
    const int lane = threadIdx.x & 31;
    const int per_p = ((k.num_pages + c.warps - 1) / c.warps + 31) / 32 * 32;
    const int p0 = (int)min((int64_t)k.num_pages, (int64_t)c.warp * per_p);
    const int p1 = min(k.num_pages, p0 + per_p);
    Totals mine{0, 0, 0}, before, all;
    for (int q = p0; q < p1; q += 32)
        mine.need += __popc(__ballot_sync(kAll, q + lane < p1 && k.refs[q + lane] > 0));
    scan(c, sums, mine, before, all);
    const int used = all.need;
    mine = Totals{0, 0, 0};
    for (int q = p0; q < p1; q += 32) {
        const int at = q + lane;
        const bool in = at < p1, is = in && k.refs[at] > 0;
        mine.spare += __popc(__ballot_sync(kAll, in && !is && at < used));
        mine.copies += __popc(__ballot_sync(kAll, is && at >= used));
        if (in && !is && at >= used) a.goes[at] = -1;
    }
    scan(c, sums2, mine, before, all);
    int hole = before.spare, mover = before.copies;
    for (int q = p0; q < p1; q += 32) {
        const int at = q + lane;
        const bool in = at < p1, is = in && k.refs[at] > 0;
        const bool h = in && !is && at < used, m = is && at >= used;
        const unsigned bh = __ballot_sync(kAll, h), bm = __ballot_sync(kAll, m);
        const unsigned below = (1u << lane) - 1;
        if (h) a.holes[hole + __popc(bh & below)] = at;
        if (m) a.movers[mover + __popc(bm & below)] = at;
        hole += __popc(bh);
        mover += __popc(bm);
    }
    c.sync();
    for (int i = c.warp * 32 + lane; i < all.copies; i += c.warps * 32) {
        const int from = a.movers[i], to = a.holes[i];
        a.pairs[2 * i] = from;
        a.pairs[2 * i + 1] = to;
        a.goes[from] = to;
        k.refs[to] = k.refs[from];
        k.refs[from] = 0;
    }
    if (c.warp == 0 && lane == 0) {
        *a.count = all.copies;
        *a.n_used = used;
    }
    c.sync();
}

__global__ void renumber_kernel(const CompactArgs a) {
    const Books &k = a.k;
    const int used = *a.n_used;
    const int64_t n = (int64_t)k.B * k.max_pages;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int e = k.table[i];
        if (e < used) continue;
        const int to = e < k.num_pages ? a.goes[e] : -1;
        if (to < 0) flag(k, FD_DEV_BAD_INDEX);
        k.table[i] = to;
    }
}

// ---------------------------------------------------------------- copies
constexpr int kUnit = 4096;       // bytes a warp copies at a time
constexpr int kCopyThreads = 512;

struct CopyArgs {
    Pools q;
    const int32_t *pairs, *count;
    int32_t max_pairs, num_pages;
    int32_t *status;
};

template <typename V>
__device__ __forceinline__ void copy_unit(const uint8_t *src, uint8_t *dst, int bytes, int lane) {
    constexpr int W = (int)sizeof(V), N = 8;
    int at = lane * W;
    for (; at + (N - 1) * 32 * W < bytes; at += N * 32 * W) {
        V x[N];
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = *reinterpret_cast<const V *>(src + at + i * 32 * W);
#pragma unroll
        for (int i = 0; i < N; ++i) *reinterpret_cast<V *>(dst + at + i * 32 * W) = x[i];
    }
    for (; at < bytes; at += 32 * W) *reinterpret_cast<V *>(dst + at) = *reinterpret_cast<const V *>(src + at);
}

// Units (pair, pool, 4 KiB of the page) strided over the grid's warps.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyArgs a) {
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * (kCopyThreads / 32);
    const int per = a.q.units[a.q.n];
    const int pairs = max(0, min(*a.count, a.max_pairs));
    const int64_t units = (int64_t)pairs * per;
    for (int64_t u = (int64_t)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); u < units; u += warps) {
        const int i = (int)(u / per), x = (int)(u - (int64_t)i * per);
        const int from = a.pairs[2 * i], to = a.pairs[2 * i + 1];
        if (from < 0 || from >= a.num_pages || to < 0 || to >= a.num_pages) {
            if (lane == 0) atomicOr(a.status, FD_DEV_BAD_INDEX);
            continue;
        }
        int lo = 0, hi = a.q.n;   // the pool whose units hold x
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.q.units[mid] <= x) lo = mid;
            else hi = mid;
        }
        const int64_t off = (int64_t)(x - a.q.units[lo]) * kUnit;
        const int bytes = (int)min((int64_t)kUnit, a.q.bytes[lo] - off);
        const uint8_t *src = a.q.base[lo] + (int64_t)from * a.q.step[lo] + off;
        uint8_t *dst = a.q.base[lo] + (int64_t)to * a.q.step[lo] + off;
        const uint64_t low = (uint64_t)(uintptr_t)src | (uint64_t)(uintptr_t)dst | (uint64_t)bytes;
        if ((low & 15) == 0) copy_unit<uint4>(src, dst, bytes, lane);
        else if ((low & 3) == 0) copy_unit<uint32_t>(src, dst, bytes, lane);
        else copy_unit<uint8_t>(src, dst, bytes, lane);
    }
}

int cluster_for(const Books &k) { return k.num_pages > 4096 || k.B > 64 ? kMaxCluster : 1; }

template <typename Args>
int launch_cluster(void (*kernel)(const Args), const Args &a, int size, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)size);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)size;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? 0 : -5;
}

}  // namespace

int pages_unit_bytes() { return kUnit; }

int64_t pages_scratch_words(int64_t num_pages) { return 3 * num_pages + 32; }

int launch_pages_free(const Books &k, const int32_t *seqs, const int32_t *lengths, int n,
                      cudaStream_t st) {
    free_kernel<<<n, 256, 0, st>>>(k, seqs, lengths, n);
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

int launch_pages_fork(const Books &k, const int32_t *src, const int32_t *dst, const int32_t *lengths,
                      int n, cudaStream_t st) {
    fork_kernel<<<n, 256, 0, st>>>(k, src, dst, lengths, n);
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

int launch_pages_reserve(const Books &k, const int32_t *n_new, int n_each, int32_t *pairs,
                         int32_t *count, int32_t *scratch, cudaStream_t st) {
    ReserveArgs a{k, n_new, n_each, pairs, count, scratch, scratch + k.num_pages,
                  scratch + 2 * (int64_t)k.num_pages};
    return launch_cluster(reserve_kernel, a, cluster_for(k), st);
}

int launch_pages_compact(const Books &k, int32_t *pairs, int32_t *count, int32_t *scratch,
                         cudaStream_t st) {
    const int64_t P = k.num_pages;
    CompactArgs a{k, pairs, count, scratch + 32, scratch + 32 + P, scratch + 32 + 2 * P, scratch};
    const int rc = launch_cluster(compact_kernel, a, cluster_for(k), st);
    if (rc != 0) return rc;
    const int64_t n = (int64_t)k.B * k.max_pages;
    const int64_t blocks = ceil_div(n, 256) < 1024 ? ceil_div(n, 256) : 1024;
    renumber_kernel<<<(unsigned)blocks, 256, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

int launch_pages_copy(const Pools &q, const int32_t *pairs, const int32_t *count, int max_pairs,
                      int num_pages, int32_t *status, int sms, cudaStream_t st) {
    CopyArgs a{q, pairs, count, max_pairs, num_pages, status};
    const int64_t warps = (int64_t)max_pairs * q.units[q.n];
    int64_t blocks = ceil_div(warps, kCopyThreads / 32);
    if (blocks > 4 * (int64_t)sms) blocks = 4 * (int64_t)sms;
    copy_kernel<<<(unsigned)blocks, kCopyThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

}  // namespace fd
