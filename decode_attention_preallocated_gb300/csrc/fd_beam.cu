// fd_beam.cu -- one step of a beam search: the best n_out of a request's beams
// times words, from the logits.
//
// A word of beam k scores s_k + (x - lse_k), lse_k = m + log sum exp(x - m).  Within
// a beam the order is that of the logits, so the logits are read once: a block
// takes a slice of one beam's row, leaves its maximum, its sum of exponentials and its
// n_out best words (logit, lowest word first), and the last block of a request joins the
// slices of all its beams.
//
// The best n of many: at least n of the threads' largest lie at or above a bound
// that warp maxima give (bound_of), and few more numbers do.  A block streams its
// slice, each thread 32 bytes a step, keeping the maximum of each thread's step;
// the few steps that reach the bound are read again (from L2) for the words that
// do.  Those are ranked by counting how many are better than each.  The join
// ranks what the slices left the same way, by scores in single precision widened
// by what those may be off, and orders the few that remain by their exact scores.
// lse is an fp32 number off by some 2^-20 (exponentials by the special function unit, sums
// in fp32); its terms are added in an order that is the same for every row of a call.
//
// Times (us, floors by the copy rate): 4 beams of 32,000 fp32 words 13.6, of which the
// read is 0.1: dependent steps of one slice (load, bound, read again, rank) and of the
// join.  32 x 8 beams of 128,000 bf16 words, a fifth of them ended, 26.7 (floor 7.8): a block
// streams for a third of that, and spends as long on its bound, the second look and the
// ranking, with barriers between, and the last one on the join.  Four steps' loads in
// flight and three blocks an SM: 30.6, before the join took its candidates in another
// order; two and four, three and four 31.3; six and three 31.3; six or eight and two 36.
// Rows that start off a 16-byte boundary bring 16 bytes more a thread and shift their words
// out of them: 32 x 16 beams of 10,623 bf16 words 26.8 us (fp32 29.7; two steps ahead, 27.1
// and 29.5 with three, 28.0 and 28.9 with four).  Words counted from the boundary took 26.0
// and 27.7, but rows of the same logits then had other sums, and did not tie.
// More than kFinals candidates as good as the bound (all words alike) are picked one
// by one: 4 x 8 beams of 50,000 words, 32 best, 395 us.
#include <cuda_runtime.h>

#include <math.h>

#include <initializer_list>

#include "fd_device.cuh"
#include "fd_packed.cuh"
#include "fd_serve.h"

namespace fd {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
// Words a thread, and a block, looks at in one step: 32 bytes a thread.
template <typename T>
constexpr int kPer = 32 / (int)sizeof(T);
template <typename T>
constexpr int kStep = kPer<T> * kThreads;
constexpr int kSteps = 16;         // steps of a slice at most
constexpr int kAgain = 64;         // threads' steps read again at a time
constexpr int kKeep = 512;         // a longer list is cut before more comes
constexpr int kList = kKeep + kAgain * kPer<uint16_t>;
constexpr int kHeld = 8;           // of the join's candidates, those that a thread holds
constexpr int kFinals = 512;       // the join's list
constexpr int kAhead = 4, kAheadOdd = 2;   // steps whose loads are in flight (rows on 16-byte boundaries, others)
constexpr int kBlocks = 3;         // blocks an SM holds
constexpr unsigned kAll = 0xffffffffu;

// Unsigned numbers in the order of the floats, both zeros alike; 0 for what is
// no candidate (-inf, NaN).
__device__ __forceinline__ uint32_t order_of(float x) {
    if (!(x > neg_inf())) return 0;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float float_of(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// The order of the lowest finite number.
constexpr uint32_t kLowest = 0x00800000u;
constexpr float kLog2e = 1.4426950408889634f;

// Both numbers of a pair times f.
__device__ __forceinline__ uint64_t scaled(uint64_t a, float f) { return mul2(a, pair(f, f)); }

// What a slice leaves behind: then room for 2 n_out keys (order of the logit,
// ~word), its n_out best among them, 0 past the last.
struct Slice {
    float top, sum;    // of its logits: maximum, and sum of exp(x - top), NaN with a NaN among them
};

__device__ __forceinline__ Slice *head_of(char *scratch, int64_t slice, int n_out) {
    return reinterpret_cast<Slice *>(scratch + slice * (int64_t)(8 + 16 * n_out));
}
__device__ __forceinline__ uint64_t *keys_of(Slice *h) { return reinterpret_cast<uint64_t *>(h + 1); }

// The i-th largest of the warp's keys (1 <= i <= lanes whose key is not 0).
__device__ __forceinline__ uint64_t warp_largest(uint64_t mine, int i) {
    uint32_t hi = (uint32_t)(mine >> 32), lo = (uint32_t)mine, top = 0, low = 0;
    for (; i > 0; --i) {
        top = __reduce_max_sync(kAll, hi);
        low = __reduce_max_sync(kAll, hi == top ? lo : 0u);
        const uint32_t who = __ballot_sync(kAll, hi == top && lo == low);
        if ((threadIdx.x & 31) == __ffs(who) - 1) hi = lo = 0;
    }
    return (uint64_t)top << 32 | low;
}

// A bound that at least n of the block's keys reach, from each thread's largest (0:
// it has none); 0 where fewer than n threads have one.  Warps with few such
// lanes give fewer.
__device__ __forceinline__ uint64_t bound_of(uint64_t mine, int n, int *counts, uint64_t *bounds) {
    const int warp = threadIdx.x >> 5, have = __popc(__ballot_sync(kAll, mine != 0));
    int m = (n + kWarps - 1) / kWarps;
    uint64_t b = have > 0 ? warp_largest(mine, min(have, m)) : ~0ull;
    if ((threadIdx.x & 31) == 0) {
        counts[warp] = have;
        bounds[warp] = b;
    }
    __syncthreads();
    int got = 0, all = 0;
    b = ~0ull;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        got += min(counts[w], m);
        all += counts[w];
        b = b < bounds[w] ? b : bounds[w];
    }
    if (got >= n) return b;
    if (all < n) return 0;
    do {
        ++m;
        got = 0;
        for (int w = 0; w < kWarps; ++w) got += min(counts[w], m);
    } while (got < n);
    b = have > 0 ? warp_largest(mine, min(have, m)) : ~0ull;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) bounds[warp] = b;
    __syncthreads();
    b = ~0ull;
    for (int w = 0; w < kWarps; ++w) b = b < bounds[w] ? b : bounds[w];
    return b;
}

struct __align__(16) Room {
    union {
        uint64_t list[kList];
        struct {
            uint64_t score[kFinals], at[kFinals];
        } finals;
    };
    float lse[128];
    float tops_of[kSteps][kThreads];   // of each thread's steps
    uint16_t again[kSteps * kThreads];   // steps to read again: step * kThreads + thread
    int n_again;
    uint64_t bounds[kWarps];
    int counts[kWarps];
    float tops[kWarps], sums[kWarps];
    int count, last;
};

struct BeamArgs {
    BeamParams p;
    int32_t slices, steps;     // a row's slices, of so many steps each
};

// A number's bits in the order of the numbers (no NaN).
__device__ __forceinline__ uint64_t order_of(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x);
    return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ double double_of(uint64_t k) {
    return __longlong_as_double((long long)(k ^ ((k >> 63) ? 1ull << 63 : ~0ull)));
}

// Cuts the list of `count` keys (at most MINE a thread) to its n best, in order;
// every thread.
template <int MINE>
__device__ __forceinline__ void cut(Room &sm, int count, int n) {
    uint64_t key[MINE], top = 0;
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
        const int at = threadIdx.x + i * kThreads;
        key[i] = at < count ? sm.list[at] : 0;
        top = key[i] > top ? key[i] : top;
    }
    if (count > kThreads / 4) {
        // first those that can be among them
        const uint64_t least = bound_of(top, n, sm.counts, sm.bounds);
        if (threadIdx.x == 0) sm.count = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MINE; ++i)
            if (key[i] && key[i] >= least) sm.list[atomicAdd(&sm.count, 1)] = key[i];
        __syncthreads();
        count = sm.count;
#pragma unroll
        for (int i = 0; i < MINE; ++i) {
            const int at = threadIdx.x + i * kThreads;
            key[i] = at < count ? sm.list[at] : 0;
        }
    }
    int rank[MINE];
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
        rank[i] = 0;
        if (i * kThreads >= count) break;
#pragma unroll 4
        for (int j = 0; j < count; ++j) rank[i] += sm.list[j] > key[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
        if (i * kThreads >= count) break;
        if (key[i] && rank[i] < n) sm.list[rank[i]] = key[i];
    }
    if (threadIdx.x == 0) sm.count = min(count, n);
    __syncthreads();
}

// The same for a list of any length, out of line: it is rarely long.
__device__ __noinline__ void cut_long(Room &sm, int count, int n) {
    cut<(kList + kThreads - 1) / kThreads>(sm, count, n);
}

// Joins the slices of request b.
__device__ __noinline__ void join(const BeamArgs &a, int b, Room &sm) {
    const BeamParams &p = a.p;
    const int tid = threadIdx.x, K = p.K, S = a.slices, n = p.n_out;
    const int64_t first = (int64_t)b * K * S;
    const int room = 2 * n, total = K * S * room;
    // the first of this thread's candidates set out before the sums are joined
    // (every warp takes some of every beam: the worst warp's largest bound them all, and
    // beams lie far apart.  32 x 16 beams, 32 best, a warp by beams: 51 to 320 us, 25 to 37 so)
    const int mine = (tid & 31) * kWarps + (tid >> 5);
    uint64_t held[kHeld];
    const auto key_at = [&](int e) {
        const int slice = e / room;
        return __ldcg(keys_of(head_of(p.scratch, first + slice, n)) + (e - slice * room));
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i) held[i] = mine + i * kThreads < total ? key_at(mine + i * kThreads) : 0;
    for (int k = tid >> 5; k < K; k += kWarps) {
        const int lane = tid & 31;
        float top = neg_inf(), sum = 0.f;
        bool nan = false;
        for (int s = lane; s < S; s += 32) {
            const float2 h = __ldcg(reinterpret_cast<const float2 *>(head_of(p.scratch, first + (int64_t)k * S + s, n)));
            nan |= h.y != h.y;
            if (h.x > neg_inf()) {
                const float now = fmaxf(top, h.x);
                sum = sum * expf(top - now) + h.y * expf(h.x - now);
                top = now;
            }
        }
        nan = __any_sync(kAll, nan);
        float most = top;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(kAll, most, o));
        sum = top > neg_inf() ? sum * expf(top - most) : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        if (lane == 0) {
            // sum = 2^e f, f in [0.75, 1.5): the logarithm of f is small, and so
            // is what it is off by; the three are added in 64 bits
            const int e = (__float_as_int(sum) - 0x3f400000) >> 23;
            const float f = __int_as_float(__float_as_int(sum) - (e << 23));
            float x = (float)((double)most + ((double)e * 0.693147180559945309 + (double)logf(f)));
            if (!(sum > 0.f && sum < INFINITY)) x = most + logf(sum);   // no word, or no number
            if (nan) x = __uint_as_float(0x7fffffffu);
            if (p.finished && p.finished[(int64_t)b * K + k]) x = 0.f;
            sm.lse[k] = x;
        }
    }
    if (tid == 0) sm.count = 0;
    __syncthreads();
    // f(beam, key, score in single precision, what that may be off) of this thread's
    // candidates
    const float *scores = p.scores + (int64_t)b * K;
    const auto one = [&](int e, uint64_t key, auto f) {
        if (!key) return;
        const int k = e / (room * S);
        const float s = __ldg(scores + k), d = float_of((uint32_t)(key >> 32)) - sm.lse[k], score = s + d;
        if (score > neg_inf()) f(k, key, score, ldexpf(fabsf(s) + fabsf(d), -22));
    };
    const auto visit = [&](auto f) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (mine + i * kThreads < total) one(mine + i * kThreads, held[i], f);
        for (int e = mine + kHeld * kThreads; e < total; e += kThreads) one(e, key_at(e), f);
    };
    float low = neg_inf();
    visit([&](int, uint64_t, float score, float off) { low = fmaxf(low, score - off); });
    const uint32_t least = (uint32_t)(bound_of((uint64_t)order_of(low) << 32, n, sm.counts, sm.bounds) >> 32);
    const auto exactly = [&](int k, uint64_t key) {
        return order_of((double)__ldg(scores + k) + ((double)float_of((uint32_t)(key >> 32)) - (double)sm.lse[k]));
    };
    visit([&](int k, uint64_t key, float score, float off) {
        if (order_of(score + off) < least) return;
        const int i = atomicAdd(&sm.count, 1);
        if (i >= kFinals) return;
        sm.finals.score[i] = key;
        sm.finals.at[i] = (uint64_t)k << 32 | (uint32_t)~(uint32_t)key;
    });
    __syncthreads();
    const int count = sm.count;
    const int64_t out = (int64_t)b * n;
    const auto put = [&](int rank, uint64_t score, uint64_t at) {
        p.scores_out[out + rank] = (float)double_of(score);
        p.beams_out[out + rank] = b * K + (int)(at >> 32);
        p.tokens_out[out + rank] = (int)(uint32_t)at;
    };
    // higher scores, then lower numbers
    const auto better = [](uint64_t s, uint64_t a, uint64_t t, uint64_t b) { return s > t || (s == t && a < b); };
    int found = count;
    if (count <= kFinals) {
        for (int i = tid; i < count; i += kThreads) sm.finals.score[i] = exactly((int)(sm.finals.at[i] >> 32), sm.finals.score[i]);
        __syncthreads();
        for (int i = tid; i < count; i += kThreads) {
            const uint64_t s = sm.finals.score[i], at = sm.finals.at[i];
            int rank = 0;
#pragma unroll 8
            for (int j = 0; j < count; ++j) {
                const uint64_t t = sm.finals.score[j], u = sm.finals.at[j];
                rank += (int)(t > s) | ((int)(t == s) & (int)(u < at));
            }
            if (rank < n) put(rank, s, at);
        }
    } else {
        // more are as good as that: the next best, n times
        uint64_t ps = 0, pa = 0;
        for (found = 0; found < n; ++found) {
            uint64_t bs = 0, ba = ~0ull;
            visit([&](int k, uint64_t key, float, float) {
                const uint64_t t = exactly(k, key), at = (uint64_t)k << 32 | (uint32_t)~(uint32_t)key;
                if ((found == 0 || better(ps, pa, t, at)) && better(t, at, bs, ba)) {
                    bs = t;
                    ba = at;
                }
            });
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const uint64_t s = __shfl_xor_sync(kAll, bs, o), at = __shfl_xor_sync(kAll, ba, o);
                if (better(s, at, bs, ba)) {
                    bs = s;
                    ba = at;
                }
            }
            __syncthreads();
            if ((tid & 31) == 0) {
                sm.finals.score[tid >> 5] = bs;
                sm.finals.at[tid >> 5] = ba;
            }
            __syncthreads();
            for (int j = 0; j < kWarps; ++j)
                if (better(sm.finals.score[j], sm.finals.at[j], bs, ba)) {
                    bs = sm.finals.score[j];
                    ba = sm.finals.at[j];
                }
            __syncthreads();
            if (ba == ~0ull) break;
            if (tid == 0) put(found, bs, ba);
            ps = bs;
            pa = ba;
        }
    }
    for (int i = found + tid; i < n; i += kThreads) {
        p.scores_out[out + i] = -INFINITY;
        p.beams_out[out + i] = -1;
        p.tokens_out[out + i] = -1;
    }
}

// This thread's words of one step: neighbours, the same of every row wherever it starts
// (rows of the same numbers then have the same sums, and tie).  ODD: base is the 16-byte
// boundary at or before the row, `off` words before it, and one load more brings what the
// words are shifted out of.
template <typename T, bool ODD>
struct Words {
    static constexpr int PER = kPer<T>, N = PER * (int)sizeof(T) / 16, EACH = 16 / (int)sizeof(T);
    uint4 w[N + ODD];
    // Every load lies in the row.
    __device__ __forceinline__ static bool whole(int v, int off, int end) {
        return ODD ? v >= off && v + PER + EACH - off <= end : v + PER <= end;
    }
    __device__ __forceinline__ void load(const T *base, int off, int end, int v) {
#pragma unroll
        for (int i = 0; i < N + ODD; ++i) {
            w[i] = make_uint4(0, 0, 0, 0);
            if (whole(v, off, end)) w[i] = ldg_stream(reinterpret_cast<const uint4 *>(base + v) + i);
        }
    }
    __device__ __forceinline__ static float number(const T *at) {
        if constexpr (sizeof(T) == 4) return __ldg(at);
        else return __uint_as_float((uint32_t)__ldg(at) << 16);
    }
    // Words v .. v + PER - 1 as numbers; the row's first and last few one by one.
    __device__ __forceinline__ void get(const T *base, int off, int end, int v, float *to) const {
        constexpr int U = 4 * N;
        uint32_t u[4 * (N + ODD)];
#pragma unroll
        for (int i = 0; i < N + ODD; ++i) {
            u[4 * i] = w[i].x;
            u[4 * i + 1] = w[i].y;
            u[4 * i + 2] = w[i].z;
            u[4 * i + 3] = w[i].w;
        }
        if constexpr (ODD) {
            // by two, by one and by half a 32-bit word
            const int half = sizeof(T) == 4 ? 2 * off : off;
            if (half & 4) {
#pragma unroll
                for (int e = 0; e < U + 2; ++e) u[e] = u[e + 2];
            }
            if (half & 2) {
#pragma unroll
                for (int e = 0; e < U + 1; ++e) u[e] = u[e + 1];
            }
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int e = 0; e < U; ++e) u[e] = __funnelshift_r(u[e], u[e + 1], (half & 1) * 16);
            }
        }
#pragma unroll
        for (int e = 0; e < U; ++e) {
            if (sizeof(T) == 4) {
                to[e] = __uint_as_float(u[e]);
            } else {
                to[2 * e] = bf16lo(u[e]);
                to[2 * e + 1] = bf16hi(u[e]);
            }
        }
        if (!whole(v, off, end)) {
#pragma unroll
            for (int e = 0; e < PER; ++e) to[e] = v + e < end ? number(base + off + v + e) : neg_inf();
        }
    }
};

// blockIdx.x: slice of a row (beam of a request).  ODD: some row starts off a 16-byte
// boundary.
template <typename T, bool ODD>
__global__ void __launch_bounds__(kThreads, kBlocks) beam_kernel(const __grid_constant__ BeamArgs a) {
    constexpr int PER = kPer<T>, STEP = kStep<T>;
    __shared__ Room sm;
    const BeamParams &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = p.n_out;
    const int64_t row = blockIdx.x / (unsigned)a.slices;
    const int slice = (int)(blockIdx.x % (unsigned)a.slices);
    const int b = (int)(row / p.K), k = (int)(row % p.K);
    Slice *head = head_of(p.scratch, row * a.slices + slice, n);
    uint64_t *keys = keys_of(head);
    if (p.finished && __ldg(p.finished + row)) {
        if (tid == 0) *head = Slice{neg_inf(), 0.f};
        for (int i = tid; i < 2 * n; i += kThreads)
            keys[i] = slice == 0 && i == 0 ? (uint64_t)order_of(0.f) << 32 | (uint32_t)~p.end_token : 0ull;
    } else {
        constexpr int AHEAD = ODD ? kAheadOdd : kAhead;
        const T *base = static_cast<const T *>(p.logits) + b * p.ls[0] + k * p.ls[1];
        const int off = ODD ? (int)(reinterpret_cast<uintptr_t>(base) % 16 / sizeof(T)) : 0, end = p.V;
        base -= off;
        const int first = slice * a.steps * STEP;
        const int steps = min(a.steps, (end - first + STEP - 1) / STEP);   // (0 or less: it has no words)
        if (tid == 0) sm.count = sm.n_again = 0;
        Words<T, ODD> next[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (i < steps) next[i].load(base, off, end, first + i * STEP + tid * PER);
        // of this thread's words so far: maximum, and sum of exp(x - top) (two halves)
        float top = neg_inf();
        uint64_t sum = 0;
        for (int i0 = 0; i0 < steps; i0 += AHEAD) {
#pragma unroll
            for (int q = 0; q < AHEAD; ++q) {
                const int i = i0 + q, at = first + i * STEP + tid * PER;
                if (i >= steps) break;
                float x[PER];
                next[q].get(base, off, end, at, x);
                if (i + AHEAD < steps) next[q].load(base, off, end, at + AHEAD * STEP);
                float most = x[0];
#pragma unroll
                for (int e = 1; e < PER; ++e) most = fmaxf(most, x[e]);
                sm.tops_of[i][tid] = most;
                if (most > top) {
                    if (top > neg_inf()) sum = scaled(sum, fast_exp2((top - most) * kLog2e));
                    top = most;
                }
                // (the difference first: a rounded product of the reference would
                // scale the whole sum; a NaN makes the sum one)
                const float ref = top > neg_inf() ? -top : 0.f;
#pragma unroll
                for (int e = 0; e < PER; e += 2) {
                    const float2 y = unpair(mul2(add2(pair(x[e], x[e + 1]), pair(ref, ref)), pair(kLog2e, kLog2e)));
                    sum = add2(sum, pair(fast_exp2(y.x), fast_exp2(y.y)));
                }
            }
        }
        // the block's maximum and sum, and the steps that reach the bound
        float all = top;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) all = fmaxf(all, __shfl_xor_sync(kAll, all, o));
        if (lane == 0) sm.tops[warp] = all;
        const uint32_t least = max(kLowest, (uint32_t)(bound_of((uint64_t)order_of(top) << 32, n, sm.counts, sm.bounds) >> 32));
        const float edge = float_of(least);
        if (top >= edge)
            for (int i = 0; i < steps; ++i)
                if (sm.tops_of[i][tid] >= edge) sm.again[atomicAdd(&sm.n_again, 1)] = (uint16_t)(i * kThreads + tid);
        all = sm.tops[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) all = fmaxf(all, sm.tops[w]);
        const float2 halves = unpair(sum);
        float mine = halves.x + halves.y;
        if (top > neg_inf()) mine *= fast_exp2((top - all) * kLog2e);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(kAll, mine, o);
        if (lane == 0) sm.sums[warp] = mine;
        __syncthreads();
        if (tid == 0) {
            mine = 0.f;
            for (int w = 0; w < kWarps; ++w) mine += sm.sums[w];
            *head = Slice{all, mine};
        }
        for (int i0 = 0; i0 < sm.n_again; i0 += kAgain) {
            bool over = false;
            if (tid < kAgain && i0 + tid < sm.n_again) {
                const int e0 = sm.again[i0 + tid], at = first + e0 / kThreads * STEP + e0 % kThreads * PER;
                float x[PER];
                next[0].load(base, off, end, at);
                next[0].get(base, off, end, at, x);
#pragma unroll
                for (int e = 0; e < PER; ++e)
                    if (x[e] >= edge) {
                        const int to = atomicAdd(&sm.count, 1);
                        over |= to >= kKeep;
                        sm.list[to] = (uint64_t)order_of(x[e]) << 32 | ~(uint32_t)(at + e);
                    }
            }
            if (__syncthreads_or(over)) cut_long(sm, sm.count, n);
        }
        int count = sm.count;
        if (count > 2 * n) {
            __syncthreads();
            if (count <= kThreads) cut<1>(sm, count, n);
            else cut_long(sm, count, n);
            count = sm.count;
        }
        for (int i = tid; i < 2 * n; i += kThreads) keys[i] = i < count ? sm.list[i] : 0;
    }
    // the last block of a request joins its slices
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        sm.last = atomicAdd(p.tickets + b, 1) == p.K * a.slices - 1;
        if (sm.last) __threadfence();
    }
    __syncthreads();
    if (!sm.last) return;
    join(a, b, sm);
    if (tid == 0) p.tickets[b] = 0;
}

// Steps a slice: all rows in one round of the blocks that 152 SMs hold where there are
// not more rows than blocks (32 x 8 rows of 128,000 bf16 words, a fifth of them ended:
// 30.6 us when tried; with more blocks than that 35 to 40), else a row a block;
// kSteps at most.  And no more slices than leave the join what its threads hold (each
// slice leaves up to `per` keys of a request): 8 beams of 128,000 words, 16 best, 20.5
// us against 41 in single steps; 128 beams of 32,000, 64 best, 92 against 192; half of
// that changed nothing.
int steps_of(int64_t rows, int64_t V, int step, int per) {
    const int64_t steps = ceil_div(V, step), room = 152 * kBlocks;
    const int64_t most = kHeld * kThreads / per < 1 ? 1 : kHeld * kThreads / per;
    const int64_t full = rows <= room ? room / rows : 1, slices = full < most ? full : most;
    const int64_t each = ceil_div(steps, slices < steps ? slices : steps);
    return (int)(each < kSteps ? each : kSteps);
}

}  // namespace

int64_t beam_scratch_bytes(int64_t B, int K, int64_t V, int n_out) {
    // (the more slices of the two types')
    int64_t slices = 0;
    for (const int step : {kStep<float>, kStep<uint16_t>}) {
        const int64_t n = ceil_div(V, (int64_t)steps_of(B * K, V, step, K * 2 * n_out) * step);
        slices = n > slices ? n : slices;
    }
    return B * K * slices * (int64_t)(8 + 16 * n_out);
}

int launch_beam_select(const BeamParams &p, cudaStream_t st) {
    const int64_t rows = (int64_t)p.B * p.K;
    const int es = p.bf16 ? 2 : 4, step = p.bf16 ? kStep<uint16_t> : kStep<float>;
    const int steps = steps_of(rows, p.V, step, p.K * 2 * p.n_out);
    const BeamArgs a{p, (int32_t)ceil_div(p.V, (int64_t)steps * step), steps};
    const int64_t blocks = rows * a.slices;
    if (blocks >= (int64_t)1 << 31) return -2;
    const bool odd = reinterpret_cast<uintptr_t>(p.logits) % 16 || (p.B > 1 && p.ls[0] * es % 16) || (p.K > 1 && p.ls[1] * es % 16);
    const auto kernel = p.bf16 ? (odd ? beam_kernel<uint16_t, true> : beam_kernel<uint16_t, false>)
                               : (odd ? beam_kernel<float, true> : beam_kernel<float, false>);
    kernel<<<(unsigned)blocks, kThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

}  // namespace fd
