// fd_pages.cu -- page bookkeeping of a paged cache: freeing, forking, reordering,
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
// as one block, or one thread-block cluster for large pools, whose barrier costs
// far less than another launch, with a thread per table entry and 128 pages per
// warp step.  64 sequences leave and 64 come in 256 of 512 entries: 16.0 us for
// the two calls; 3 children of one sequence freed, forked, reserved for and their
// page copied: 15 to 18 us for the four; 10,192 pages ranked 9 to 12 us, renumbered
// 4, and 45 MB of them copied 15.7, the rate of a plain copy.  A reordering is one launch:
// 4 rows of 128 pages 6 us, 256 rows of 2,048 13 (eight columns a block; 19 by one).
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
constexpr int kReorderThreads = 256, kReorderShift = 3;   // 8 columns a block
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

// Rows change places only within a column, so a block takes some columns of
// every row into shared memory and writes them back in their new places; the
// lengths, which every block reads, are written by the last one to finish.
__global__ void __launch_bounds__(kReorderThreads) reorder_kernel(const Books k, const int32_t *src, int shift,
                                                                  int32_t *ticket) {
    extern __shared__ int32_t old[];
    const int cols = 1 << shift, c0 = blockIdx.x << shift, width = min(cols, k.max_pages - c0);
    const int cells = k.B << shift;
#pragma unroll 4
    for (int e = threadIdx.x; e < cells; e += kReorderThreads) {
        const int b = e >> shift, c = e & (cols - 1);
        if (c < width) old[e] = k.table[(int64_t)b * k.max_pages + c0 + c];
    }
    __syncthreads();
#pragma unroll 2
    for (int e = threadIdx.x; e < cells; e += kReorderThreads) {
        const int b = e >> shift, c = e & (cols - 1);
        if (c >= width) continue;
        const int s = src[b];
        if (s == b) continue;
        if (s >= k.B) {
            if (c0 + c == 0) flag(k, FD_DEV_BAD_INDEX);
            continue;
        }
        const int j = c0 + c, was = old[e];
        int to = -1;
        if (s >= 0 && j < pages_of(held(k, s), k.page_size)) {
            to = old[(s << shift) + c];
            if (to < 0 || to >= k.num_pages) {
                flag(k, FD_DEV_BAD_INDEX);
                to = -1;
            }
        }
        if (to == was) continue;
        if (to >= 0) atomicAdd(k.refs + to, 1);
        drop(k, was);
        k.table[(int64_t)b * k.max_pages + j] = to;
    }
    __shared__ int last;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(ticket, 1) == (int)gridDim.x - 1;
        if (last) __threadfence();
    }
    __syncthreads();
    if (!last) return;
    for (int b = threadIdx.x; b < k.B; b += kReorderThreads) {
        const int s = src[b];
        old[b] = s == b || s >= k.B ? k.lengths[b] : s < 0 ? 0 : (int)held(k, s);
    }
    __syncthreads();
    for (int b = threadIdx.x; b < k.B; b += kReorderThreads) k.lengths[b] = old[b];
    if (threadIdx.x == 0) *ticket = 0;
}

// ------------------------------------------------------------ one cluster
// What a thread contributes to the ranks, and the sums over the threads before
// it and over all.
struct __align__(16) Totals {
    int need, spare, copies, unused;
};

__device__ __forceinline__ Totals operator+(const Totals &a, const Totals &b) {
    return Totals{a.need + b.need, a.spare + b.spare, a.copies + b.copies, 0};
}

__device__ __forceinline__ Totals shift_up(const Totals &x, int by) {
    return Totals{__shfl_up_sync(kAll, x.need, by), __shfl_up_sync(kAll, x.spare, by),
                  __shfl_up_sync(kAll, x.copies, by), 0};
}

struct Cluster {
    int rank, size, thread, threads;   // block in the cluster; thread in the cluster
    __device__ __forceinline__ Cluster() {
        auto c = cg::this_cluster();
        rank = (int)c.block_rank();
        size = (int)c.num_blocks();
        thread = rank * kThreads + (int)threadIdx.x;
        threads = size * kThreads;
    }
    __device__ __forceinline__ void sync() const {
        if (size == 1) __syncthreads();
        else cg::this_cluster().sync();
    }
};

// Inclusive sums over the lanes of a warp.
__device__ __forceinline__ Totals warp_scan(Totals x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Totals y = shift_up(x, o);
        if (lane >= o) x = x + y;
    }
    return x;
}

__device__ __forceinline__ Totals from_lane(const Totals &x, int src) {
    return Totals{__shfl_sync(kAll, x.need, src), __shfl_sync(kAll, x.spare, src),
                  __shfl_sync(kAll, x.copies, src), 0};
}

// Sums `mine` over the threads before this one (before) and over all (all).
// `at`: kWarps + 1 entries of this block's shared memory that nothing else
// uses until the next barrier; every thread of the cluster calls it.  One
// barrier of the block, one of the cluster, one read from each other block.
__device__ __forceinline__ void scan(const Cluster &c, Totals *at, const Totals &mine, Totals &before,
                                     Totals &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Totals upto = warp_scan(mine);
    if (lane == 31) at[warp] = upto;
    __syncthreads();
    const Totals warps = warp_scan(at[lane]);
    const Totals block = from_lane(warps, 31);
    const Totals early = from_lane(warps, warp > 0 ? warp - 1 : 0);
    before = shift_up(upto, 1);
    if (lane == 0) before = Totals{0, 0, 0, 0};
    if (warp > 0) before = before + early;
    all = block;
    if (c.size > 1) {
        if (threadIdx.x == 0) at[kWarps] = block;
        c.sync();
        Totals x{0, 0, 0, 0};
        if (lane < c.size) x = *cg::this_cluster().map_shared_rank(at + kWarps, lane);
        x = warp_scan(x);
        all = from_lane(x, 31);
        if (c.rank > 0) before = before + from_lane(x, c.rank - 1);
    }
}

// The pages of a pool in runs of 128 per warp step, four to a lane; bit i of a
// flag word's nibble n says whether page i of this lane's four in step n is
// free.  A warp's steps are consecutive, so ranks follow the numbers.
struct PageRun {
    int p0, steps;   // first page of this warp, and its steps
    int P;
    const int32_t *refs;
    uint32_t kept;   // the flags, where there are at most 8 steps
    __device__ __forceinline__ PageRun(const Books &k, const Cluster &c) : P(k.num_pages), refs(k.refs), kept(0) {
        const int warps = c.threads / 32, warp = c.thread / 32;
        const int all = (P + 127) / 128, per = (all + warps - 1) / warps;
        p0 = (int)min((int64_t)P, (int64_t)warp * per * 128);
        steps = min(per, (P - p0 + 127) / 128);
    }
    __device__ __forceinline__ int page(int step) const { return p0 + step * 128 + (int)(threadIdx.x & 31) * 4; }
    // Free pages among this lane's four in `step`, as bits.
    __device__ __forceinline__ uint32_t look(int step) const {
        const int q = page(step);
        int4 r = make_int4(1, 1, 1, 1);
        if (q + 3 < P && (reinterpret_cast<uintptr_t>(refs) & 15) == 0) {
            r = *reinterpret_cast<const int4 *>(refs + q);
        } else {
            if (q < P) r.x = refs[q];
            if (q + 1 < P) r.y = refs[q + 1];
            if (q + 2 < P) r.z = refs[q + 2];
            if (q + 3 < P) r.w = refs[q + 3];
        }
        return (r.x <= 0 ? 1u : 0u) | (r.y <= 0 ? 2u : 0u) | (r.z <= 0 ? 4u : 0u) | (r.w <= 0 ? 8u : 0u);
    }
    // Free pages of this lane.
    __device__ __forceinline__ int count() {
        int n = 0;
        if (steps <= 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < steps) kept |= look(i) << (4 * i);
            n = __popc(kept);
        } else {
#pragma unroll 4
            for (int i = 0; i < steps; ++i) n += __popc(look(i));
        }
        return n;
    }
    __device__ __forceinline__ uint32_t flags(int step) const {
        return steps <= 8 ? (kept >> (4 * step)) & 15u : look(step);
    }
    // Pages that exist among this lane's four.
    __device__ __forceinline__ uint32_t real(int step) const {
        const int left = P - page(step);
        return left >= 4 ? 15u : (left <= 0 ? 0u : (1u << left) - 1u);
    }
};

// Rank within the warp's step of the lowest page of this lane that `bits`
// marks (those of one lane follow one another), and how many there are.
__device__ __forceinline__ int step_rank(uint32_t bits, int &all) {
    const int lane = threadIdx.x & 31, mine = __popc(bits);
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kAll, upto, o);
        if (lane >= o) upto += y;
    }
    all = __shfl_sync(kAll, upto, 31);
    return upto - mine;
}

struct ReserveArgs {
    Books k;
    const int32_t *n_new;
    int32_t n_each;
    int32_t *pairs, *count;
    int32_t *writers, *first, *list;   // scratch, num_pages words each
};

constexpr int kSeqs = 4096;   // sequences whose ranges are looked at together

// The table entries that a run of sequences will write, numbered in order:
// entries start[b] .. start[b + 1] - 1 belong to sequence c0 + b, whose length
// is len[b].
struct Ranges {
    int *start, *len;
    int n, total;        // sequences and entries
    int c0;
    __device__ __forceinline__ void load(const ReserveArgs &a, int from, Totals *at, bool report) {
        const Books &k = a.k;
        const int64_t cap = (int64_t)k.max_pages * k.page_size;
        c0 = from;
        n = min(kSeqs, k.B - from);
        __syncthreads();   // the last run's ranges are done with
        int base = 0;
        for (int i0 = 0; i0 < n; i0 += kThreads) {
            const int i = i0 + (int)threadIdx.x;
            int entries = 0;
            if (i < n) {
                const int64_t raw = k.lengths[from + i];
                const int64_t want = a.n_new ? a.n_new[from + i] : a.n_each;
                const int64_t L = clamp_len(raw, cap);
                const int64_t end = clamp_len(L + (want < 0 ? 0 : want), cap);
                if (report && (raw != L || want < 0 || L + want > cap)) flag(k, FD_DEV_BAD_LENGTH);
                if (end > L) entries = pages_of(end, k.page_size) - (int)(L / k.page_size);
                len[i] = (int)L;
            }
            const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
            int upto = entries;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kAll, upto, o);
                if (lane >= o) upto += y;
            }
            if (lane == 31) at[warp].need = upto;
            __syncthreads();
            int w = at[lane].need;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kAll, w, o);
                if (lane >= o) w += y;
            }
            const int before = warp > 0 ? __shfl_sync(kAll, w, warp - 1) : 0;
            const int sum = __shfl_sync(kAll, w, 31);
            if (i < n) start[i + 1] = base + before + upto;
            base += sum;
            __syncthreads();
        }
        if (threadIdx.x == 0) start[0] = 0;
        total = base;
        __syncthreads();
    }
    // Calls f(entry's address, key, whether it holds positions that are kept)
    // for this thread's entries, in order.
    template <typename F>
    __device__ __forceinline__ void each(const Books &k, const Cluster &c, F f) const {
        const Run run = run_of(total, c.threads, c.thread);
        const int lo = run.lo, hi = run.hi;
        if (lo >= hi) return;
        int b = 0, top = n;   // the last sequence that starts at or before lo
        while (top - b > 1) {
            const int mid = (b + top) >> 1;
            if (start[mid] <= lo) b = mid;
            else top = mid;
        }
        for (int t = lo; t < hi; ++t) {
            while (t >= start[b + 1]) ++b;
            const int j = len[b] / k.page_size + (t - start[b]);
            const int64_t key = (int64_t)(c0 + b) * k.max_pages + j;
            f(k.table + key, (int)key, (int64_t)j * k.page_size < len[b]);
        }
    }
};

// Entries of the write ranges that name no page, or a page that others name
// too, get pages of their own; the rest stay.  A sharer keeps the page when
// every holder writes in this call and it is the first of them (in order of
// sequences, then pages).
__global__ void __launch_bounds__(kThreads) reserve_kernel(const ReserveArgs a) {
    __shared__ Totals sums[4][kWarps + 1];
    __shared__ int starts[kSeqs + 1], lens[kSeqs];
    const Books &k = a.k;
    const Cluster c;
    PageRun run(k, c);
    const int spare = run.count();
    Ranges r{starts, lens, 0, 0, 0};
    const bool one = k.B <= kSeqs;

    Totals mine{0, spare, 0, 0}, before, all;
    for (int c0 = 0; c0 < k.B; c0 += kSeqs) {
        r.load(a, c0, sums[0], c.rank == 0);
        r.each(k, c, [&](int32_t *at, int, bool) {
            const int e = *at;
            if (e < 0 || e >= k.num_pages) {
                if (e != -1) *at = -1;
                ++mine.need;
            } else if (k.refs[e] > 1) {
                a.writers[e] = 0;
                a.first[e] = 0x7fffffff;
                ++mine.copies;
            }
        });
    }
    scan(c, sums[1], mine, before, all);
    if (all.copies > 0) {
        // some written pages are shared: find each one's writers, then mark
        // the entries that part from it as -(page + 2)
        for (int c0 = 0; c0 < k.B; c0 += kSeqs) {
            if (!one) r.load(a, c0, sums[0], false);
            r.each(k, c, [&](int32_t *at, int key, bool) {
                const int e = *at;
                if (e >= 0 && k.refs[e] > 1) {
                    atomicAdd(a.writers + e, 1);
                    atomicMin(a.first + e, key);
                }
            });
        }
        c.sync();
        mine.copies = 0;
        for (int c0 = 0; c0 < k.B; c0 += kSeqs) {
            if (!one) r.load(a, c0, sums[0], false);
            r.each(k, c, [&](int32_t *at, int key, bool held) {
                const int e = *at;
                if (e < 0 || k.refs[e] <= 1) return;
                if (a.writers[e] == k.refs[e] && a.first[e] == key) return;
                *at = -(e + 2);
                ++mine.need;
                if (held) ++mine.copies;
            });
        }
        scan(c, sums[2], mine, before, all);
    }
    const bool fits = all.need <= all.spare;

    // the free pages, lowest first, as far as they are needed
    if (fits) {
        int rank = __shfl_sync(kAll, before.spare, 0);   // of the warp's first
        for (int i = 0; i < run.steps && rank < all.need; ++i) {
            const uint32_t bits = run.flags(i) & run.real(i);
            int got;
            int at = rank + step_rank(bits, got);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if ((bits >> q) & 1u) a.list[at++] = run.page(i) + q;
            rank += got;
        }
    }
    c.sync();
    Totals base{0, 0, 0, 0};   // of the runs of sequences before
    for (int c0 = 0; c0 < k.B; c0 += kSeqs) {
        int rank = before.need, pair = before.copies;
        if (!one) {
            // this run's share of the ranks
            r.load(a, c0, sums[0], false);
            Totals here{0, 0, 0, 0}, early, sum;
            r.each(k, c, [&](int32_t *at, int, bool held) {
                if (*at < 0) ++here.need;
                if (*at <= -2 && held) ++here.copies;
            });
            scan(c, sums[3], here, early, sum);
            rank = base.need + early.need;
            pair = base.copies + early.copies;
            base = base + sum;
            c.sync();
        }
        r.each(k, c, [&](int32_t *at, int, bool held) {
            const int e = *at;
            if (e >= 0) return;
            if (!fits) {
                if (e <= -2) *at = -(e + 2);   // as it was
                return;
            }
            const int got = a.list[rank++];
            if (e <= -2) {
                atomicSub(k.refs - (e + 2), 1);
                if (held) {
                    a.pairs[2 * pair] = -(e + 2);
                    a.pairs[2 * pair + 1] = got;
                    ++pair;
                }
            }
            k.refs[got] = 1;
            *at = got;
        });
    }
    if (c.thread == 0) {
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
    __shared__ Totals sums[2][kWarps + 1];
    const Books &k = a.k;
    const Cluster c;
    PageRun run(k, c);
    Totals mine{0, run.count(), 0, 0}, before, all;
    scan(c, sums[0], mine, before, all);
    const int used = k.num_pages - all.spare;
    // bits of the pages below `used`
    const auto low = [&](int i) {
        const int left = used - run.page(i);
        return left >= 4 ? 15u : (left <= 0 ? 0u : (1u << left) - 1u);
    };
    mine = Totals{0, 0, 0, 0};
    for (int i = 0; i < run.steps; ++i) {
        const uint32_t free = run.flags(i), real = run.real(i);
        mine.spare += __popc(free & low(i) & real);
        mine.copies += __popc(~free & ~low(i) & real);
    }
    scan(c, sums[1], mine, before, all);
    int hole = __shfl_sync(kAll, before.spare, 0), mover = __shfl_sync(kAll, before.copies, 0);
    for (int i = 0; i < run.steps; ++i) {
        const uint32_t free = run.flags(i), real = run.real(i);
        const uint32_t h = free & low(i) & real, m = ~free & ~low(i) & real, none = free & ~low(i) & real;
        int got;
        int at = hole + step_rank(h, got);
        hole += got;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if ((h >> q) & 1u) a.holes[at++] = run.page(i) + q;
        at = mover + step_rank(m, got);
        mover += got;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if ((m >> q) & 1u) a.movers[at++] = run.page(i) + q;
            if ((none >> q) & 1u) a.goes[run.page(i) + q] = -1;
        }
    }
    c.sync();
    for (int i = c.thread; i < all.copies; i += c.threads) {
        const int from = a.movers[i], to = a.holes[i];
        a.pairs[2 * i] = from;
        a.pairs[2 * i + 1] = to;
        a.goes[from] = to;
        k.refs[to] = k.refs[from];
        k.refs[from] = 0;
    }
    if (c.thread == 0) {
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

// One block or eight, in us (half the pages in use):
//   pages      8,000        16,000       32,000       130,000      400,000
//   reserve    7.1 / 8.5    7.6 / 8.4    10.4 / 9.4   20 / 11      43 / 20
//   compact    9.3 / 10.5   13.8 / 11.5  22 / 11      80 / 20      233 / 47
constexpr int kReserveAlone = 24576, kCompactAlone = 12288;
int cluster_for(const Books &k, int alone) { return k.num_pages > alone ? kMaxCluster : 1; }

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

int launch_pages_reorder(const Books &k, const int32_t *src, int32_t *ticket, cudaStream_t st) {
    int shift = kReorderShift;
    while (shift > 0 && ((int64_t)k.B << shift) > kReorderRows) --shift;
    const int bytes = (k.B << shift) * 4;
    // (48 KB need no leave, the kernel's own few bytes among them)
    if (bytes + 128 > 48 * 1024 && cudaFuncSetAttribute(reorder_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                        kReorderRows * 4) != cudaSuccess)
        return -5;
    const unsigned blocks = (unsigned)ceil_div(k.max_pages, 1 << shift);
    reorder_kernel<<<blocks, kReorderThreads, bytes, st>>>(k, src, shift, ticket);
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

int launch_pages_reserve(const Books &k, const int32_t *n_new, int n_each, int32_t *pairs,
                         int32_t *count, int32_t *scratch, cudaStream_t st) {
    ReserveArgs a{k, n_new, n_each, pairs, count, scratch, scratch + k.num_pages,
                  scratch + 2 * (int64_t)k.num_pages};
    return launch_cluster(reserve_kernel, a, cluster_for(k, kReserveAlone), st);
}

int launch_pages_compact(const Books &k, int32_t *pairs, int32_t *count, int32_t *scratch,
                         cudaStream_t st) {
    const int64_t P = k.num_pages;
    CompactArgs a{k, pairs, count, scratch + 32, scratch + 32 + P, scratch + 32 + 2 * P, scratch};
    const int rc = launch_cluster(compact_kernel, a, cluster_for(k, kCompactAlone), st);
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
