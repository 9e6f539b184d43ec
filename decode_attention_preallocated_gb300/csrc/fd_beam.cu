// fd_beam.cu -- one step of a beam search: the best n_out of a request's beams
// times words, from the logits.
//
// A word of beam k scores s_k + (x - lse_k), lse_k = m + log sum exp(x - m).  Within
// a beam the order is that of the logits, so the logits are read once: a block
// takes a slice of one beam's row into registers, leaves its maximum, its sum
// of exponentials and its n_out best words (logit, lowest word first), and the
// last block of a request joins the slices of all its beams.
//
// The best n of many: each of W warps finds the ceil(n / W)-th largest of its
// lanes' maxima; at least n numbers lie at or above the least of these, and
// few more do, so they are collected in shared memory and ranked by counting.
// More than the list holds (logits with many equal maxima) go by n rounds of
// one maximum each.
#include <cuda_runtime.h>

#include <math.h>

#include "fd_device.cuh"
#include "fd_serve.h"

namespace fd {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kList = 1024;        // collected candidates
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

// What a slice leaves behind: then n_out keys, (order of the logit, ~word)
// falling, 0 past the last.
struct Slice {
    float top, sum;    // of its logits: maximum, and sum of exp(x - top)
};

__device__ __forceinline__ Slice *head_of(char *scratch, int64_t slice, int n_out) {
    return reinterpret_cast<Slice *>(scratch + slice * (int64_t)(8 + 8 * n_out));
}
__device__ __forceinline__ uint64_t *keys_of(Slice *h) { return reinterpret_cast<uint64_t *>(h + 1); }

// A bound that at least n of the block's numbers reach, from each thread's
// largest: 0 where there may be fewer.
__device__ __forceinline__ uint32_t bound_of(uint32_t mine, int n, uint32_t *warp_bounds) {
    const int lane = threadIdx.x & 31;
    uint32_t x = mine, b = 0;
    for (int k = (n + kWarps - 1) / kWarps; k > 0; --k) {
        b = __reduce_max_sync(kAll, x);
        const uint32_t who = __ballot_sync(kAll, x == b);
        if (lane == __ffs(who) - 1) x = 0;
    }
    if (lane == 0) warp_bounds[threadIdx.x >> 5] = b;
    __syncthreads();
    b = warp_bounds[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) b = min(b, warp_bounds[w]);
    return b;
}

__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint64_t block_max(uint64_t x, uint64_t *room) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = max64(x, __shfl_xor_sync(kAll, x, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) room[threadIdx.x >> 5] = x;
    __syncthreads();
    x = room[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) x = max64(x, room[w]);
    return x;
}

struct __align__(8) Room {
    uint64_t list[kList];
    uint64_t room[kWarps];
    uint32_t bounds[kWarps];
    float tops[kWarps], sums[kWarps];
    int count, last;
};

struct BeamArgs {
    BeamParams p;
    int32_t slices;
};

// Values of the final ranking: the score in 64 bits and the candidate's number
// (beam, word); better: higher, then lower number.
struct __align__(16) Final {
    double score;
    uint64_t at;       // beam << 32 | word
};

// Joins the slices of request b.
__device__ __noinline__ void join(const BeamArgs &a, int b, Room &sm, Final *finals, float *lse) {
    const BeamParams &p = a.p;
    const int tid = threadIdx.x, K = p.K, S = a.slices, n = p.n_out;
    const int64_t first = (int64_t)b * K * S;
    for (int k = tid >> 5; k < K; k += kWarps) {
        const int lane = tid & 31;
        float top = neg_inf();
        bool nan = false;
        for (int s = lane; s < S; s += 32) {
            const float t = __ldcg(&head_of(p.scratch, first + (int64_t)k * S + s, n)->top);
            nan |= t != t;
            top = fmaxf(top, t);
        }
        nan = __any_sync(kAll, nan);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
        double sum = 0;
        for (int s = lane; s < S; s += 32) {
            const Slice *h = head_of(p.scratch, first + (int64_t)k * S + s, n);
            const float t = __ldcg(&h->top);
            if (t > neg_inf()) sum += (double)(__ldcg(&h->sum) * expf(t - top));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        if (lane == 0) {
            float x = (float)((double)top + log(sum));
            if (nan) x = __uint_as_float(0x7fffffffu);
            if (p.finished && p.finished[(int64_t)b * K + k]) x = 0.f;
            lse[k] = x;
        }
    }
    if (tid == 0) sm.count = 0;
    __syncthreads();
    // candidates in single precision, widened by what that may be off
    const int total = K * S * n;
    const float *scores = p.scores + (int64_t)b * K;
    const auto visit = [&](auto f) {
        for (int e = tid; e < total; e += kThreads) {
            const int row = e / n, k = row / S;
            const uint64_t key = __ldcg(keys_of(head_of(p.scratch, first + row, n)) + (e - row * n));
            if (!key) continue;
            const float x = float_of((uint32_t)(key >> 32)), s = __ldg(scores + k), d = x - lse[k];
            const float score = s + d;
            if (!(score > neg_inf())) continue;
            f(k, key, x, s, score, ldexpf(fabsf(s) + fabsf(d), -22));
        }
    };
    float low = neg_inf();
    visit([&](int, uint64_t, float, float, float score, float off) { low = fmaxf(low, score - off); });
    const uint32_t least = bound_of(order_of(low), n, sm.bounds);
    const auto exactly = [&](int k, float x, float s) { return (double)s + ((double)x - (double)lse[k]); };
    visit([&](int k, uint64_t key, float x, float s, float score, float off) {
        if (order_of(score + off) < least) return;
        const int i = atomicAdd(&sm.count, 1);
        if (i < kList) finals[i] = Final{exactly(k, x, s), (uint64_t)k << 32 | (uint32_t)~(uint32_t)key};
    });
    __syncthreads();
    const int count = sm.count;
    const int64_t out = (int64_t)b * n;
    const auto put = [&](int rank, const Final &f) {
        p.scores_out[out + rank] = (float)f.score;
        p.beams_out[out + rank] = b * K + (int)(f.at >> 32);
        p.tokens_out[out + rank] = (int)(uint32_t)f.at;
    };
    const auto better = [](const Final &x, const Final &y) { return x.score > y.score || (x.score == y.score && x.at < y.at); };
    int found = count;
    if (count <= kList) {
        for (int i = tid; i < count; i += kThreads) {
            const Final mine = finals[i];
            int rank = 0;
            for (int j = 0; j < count; ++j) rank += better(finals[j], mine);
            if (rank < n) put(rank, mine);
        }
    } else {
        // the next best, n times
        Final prev{INFINITY, 0};
        for (found = 0; found < n; ++found) {
            Final best{-INFINITY, ~0ull};
            visit([&](int k, uint64_t key, float x, float s, float, float) {
                const Final f{exactly(k, x, s), (uint64_t)k << 32 | (uint32_t)~(uint32_t)key};
                if ((found == 0 || better(prev, f)) && better(f, best)) best = f;
            });
            __syncthreads();
            finals[tid] = best;
            __syncthreads();
            for (int j = 0; j < kThreads; ++j)
                if (better(finals[j], best)) best = finals[j];
            __syncthreads();
            if (best.at == ~0ull) break;
            if (tid == 0) put(found, best);
            prev = best;
        }
    }
    for (int i = found + tid; i < n; i += kThreads) {
        p.scores_out[out + i] = -INFINITY;
        p.beams_out[out + i] = -1;
        p.tokens_out[out + i] = -1;
    }
}

// grid: (slices, beams of all requests).  PER words a thread; VEC: rows are read
// 16 bytes at a time.
template <typename T, int PER, bool VEC>
__global__ void __launch_bounds__(kThreads) beam_kernel(const __grid_constant__ BeamArgs a) {
    __shared__ Room sm;
    __shared__ Final finals[kList];
    __shared__ float lse[128];
    const BeamParams &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = p.n_out;
    const int64_t row = blockIdx.x / (unsigned)a.slices;
    const int slice = (int)(blockIdx.x % (unsigned)a.slices);
    const int b = (int)(row / p.K), k = (int)(row % p.K);
    Slice *head = head_of(p.scratch, row * a.slices + slice, n);
    uint64_t *keys = keys_of(head);
    if (p.finished && __ldg(p.finished + row)) {
        if (tid == 0) *head = Slice{neg_inf(), 0.f};
        for (int i = tid; i < n; i += kThreads)
            keys[i] = slice == 0 && i == 0 ? (uint64_t)order_of(0.f) << 32 | (uint32_t)~p.end_token : 0ull;
    } else {
        constexpr int W = VEC ? 16 / (int)sizeof(T) : 1;
        const T *src = static_cast<const T *>(p.logits) + b * p.ls[0] + k * p.ls[1];
        const int first = slice * (kThreads * PER);
        float x[PER];
        bool bad = false;
#pragma unroll
        for (int j = 0; j < PER / W; ++j) {
            const int v = first + (j * kThreads + tid) * W;
            if (VEC && v + W <= p.V) {
                const uint4 w = ldg_stream(src + v);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < W; ++e)
                    x[j * W + e] = sizeof(T) == 4 ? __uint_as_float(u[e])
                                                  : (e & 1) ? bf16hi(u[e / 2]) : bf16lo(u[e / 2]);
            } else {
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    x[j * W + e] = neg_inf();
                    if (v + e < p.V) {
                        if constexpr (sizeof(T) == 4) x[j * W + e] = src[v + e];
                        else x[j * W + e] = __uint_as_float((uint32_t)src[v + e] << 16);
                    }
                }
            }
        }
        float top = neg_inf();
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            bad |= x[e] != x[e];
            top = fmaxf(top, x[e]);
        }
        const uint32_t mine = order_of(top);
        float all = top;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) all = fmaxf(all, __shfl_xor_sync(kAll, all, o));
        if (lane == 0) sm.tops[warp] = all;
        if (tid == 0) sm.count = 0;
        const uint32_t least = max(bound_of(mine, n, sm.bounds), 1u);
        all = sm.tops[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) all = fmaxf(all, sm.tops[w]);
        // sum of exp(x - all), and the candidates
        // (the difference first: a rounded product of the maximum would scale
        // the whole sum)
        const float base = all > neg_inf() ? all : 0.f;
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < PER; ++e) sum += fast_exp2((x[e] - base) * 1.4426950408889634f);
        if (mine >= least) {
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const uint32_t o = order_of(x[e]);
                if (o >= least) {
                    const int i = atomicAdd(&sm.count, 1);
                    const uint32_t word = first + ((e / W) * kThreads + tid) * W + e % W;
                    if (i < kList) sm.list[i] = (uint64_t)o << 32 | (uint32_t)~word;
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        if (lane == 0) sm.sums[warp] = sum;
        bad = __syncthreads_or(bad);
        const int count = sm.count;
        if (tid == 0) {
            sum = 0.f;
            for (int w = 0; w < kWarps; ++w) sum += sm.sums[w];
            *head = Slice{bad ? __uint_as_float(0x7fffffffu) : all, sum};
        }
        if (count <= kList) {
            for (int i = tid; i < count; i += kThreads) {
                const uint64_t key = sm.list[i];
                int rank = 0;
                for (int j = 0; j < count; ++j) rank += sm.list[j] > key;
                if (rank < n) keys[rank] = key;
            }
            for (int i = count + tid; i < n; i += kThreads) keys[i] = 0;
        } else {
            uint64_t prev = ~0ull;
            for (int i = 0; i < n; ++i) {
                uint64_t best = 0;
#pragma unroll
                for (int e = 0; e < PER; ++e) {
                    const uint32_t o = order_of(x[e]);
                    const uint32_t word = first + ((e / W) * kThreads + tid) * W + e % W;
                    const uint64_t key = (uint64_t)o << 32 | (uint32_t)~word;
                    if (o && key < prev) best = max64(best, key);
                }
                prev = block_max(best, sm.room);
                if (tid == 0) keys[i] = prev;
            }
        }
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
    join(a, b, sm, finals, lse);
    if (tid == 0) p.tickets[b] = 0;
}

// Words a thread of the slices of a call: see launch_beam_select.
int per_thread(int64_t rows, int64_t V) { return rows * ceil_div(V, kThreads * 32) >= 152 ? 32 : 8; }

template <typename T, int PER>
void launch(const BeamArgs &a, bool vec, unsigned blocks, cudaStream_t st) {
    if (vec) beam_kernel<T, PER, true><<<blocks, kThreads, 0, st>>>(a);
    else beam_kernel<T, PER, false><<<blocks, kThreads, 0, st>>>(a);
}

}  // namespace

int64_t beam_scratch_bytes(int64_t B, int K, int64_t V, int n_out) {
    return B * K * ceil_div(V, kThreads * per_thread(B * K, V)) * (int64_t)(8 + 8 * n_out);
}

int launch_beam_select(const BeamParams &p, cudaStream_t st) {
    const int64_t rows = (int64_t)p.B * p.K;
    const int per = per_thread(rows, p.V);
    BeamArgs a{p, (int32_t)ceil_div(p.V, kThreads * per)};
    const int64_t blocks = rows * a.slices;
    if (blocks >= (int64_t)1 << 31) return -2;
    const int es = p.bf16 ? 2 : 4;
    const bool vec = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 && p.ls[0] * es % 16 == 0 && p.ls[1] * es % 16 == 0;
    if (p.bf16 && per == 32) launch<uint16_t, 32>(a, vec, (unsigned)blocks, st);
    else if (p.bf16) launch<uint16_t, 8>(a, vec, (unsigned)blocks, st);
    else if (per == 32) launch<float, 32>(a, vec, (unsigned)blocks, st);
    else launch<float, 8>(a, vec, (unsigned)blocks, st);
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

}  // namespace fd
