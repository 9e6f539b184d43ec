// fd_rows.cu -- new rows into a bf16 or int8 cache, keys and queries rotated to
// their positions on the way.
//
// A pair of values (a, b) at position p turns to (a cos - b sin, b cos + a sin) by the
// table's row of p; an int8 row is codes rint(x / s) and s = max|x| / 127.  Every
// number is read once and written once, so memory bounds long prompts and the launch
// a single token.
//
// A thread block per token: its heads' loads are independent, eight (d 128) or sixteen
// lanes take a head in runs of 16 bytes, and a row's maximum is one reduction over
// them.  Loads of three heads set out together (8 prompts of 300 .. 2,048 tokens, 32
// heads of 8, pages of 64: 54 us with three, 60 with two, 62 with four or six, which
// hold more registers; 77 one after the other), and at most 80 registers let six blocks
// share an SM (53; 50 with eight, whose spills cost a single token 1.5 of 4.1 us).
// That is 5.0 TB/s for 262 MB (52 us, floor 38.6): reads and writes of 256-byte rows of
// many pages in turn.  4 prompts into an int8 cache at d 256: 20 us (floor 9.9); one token of
// 64 sequences 4.3.
#include <cuda_runtime.h>

#include "fd_device.cuh"
#include "fd_serve.h"

namespace fd {

namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 3;      // heads whose loads a thread has in flight
constexpr int kBlocks = 6;     // blocks an SM holds at least

__device__ __forceinline__ void write_length(const RowsParams &p, int b) {
    const int64_t raw = p.lengths[b], base = clamp_len(raw, p.c.cap);
    const int64_t want = p.new_lengths ? p.new_lengths[b] : p.n, real = clamp_len(want, p.n);
    if (raw != base || want != real || base + real > p.c.cap) atomicOr(p.status, kDevBadLength);
    if (p.lengths_out) p.lengths_out[b] = (int32_t)clamp_len(base + real, p.c.cap);
}

// Sixteen values of a row: those that unit `u` of a head's d/16 holds.  The units
// of the first r values hold eight pairs each: values 8u .. 8u+7 and their
// partners r/2 further on, or, interleaved, values 16u .. 16u+15.
struct Unit {
    int lo, hi;        // where the two runs of eight values start
    bool turns, across;
    __device__ __forceinline__ Unit(const RowsParams &p, int u) {
        turns = p.rope && 16 * u < p.r;
        across = turns && !p.interleaved;
        lo = across ? 8 * u : 16 * u;
        hi = across ? lo + p.r / 2 : lo + 8;
    }
};

__device__ __forceinline__ void widen(const uint4 &w, float *x) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[2 * e] = bf16lo(v[e]);
        x[2 * e + 1] = bf16hi(v[e]);
    }
}

__device__ __forceinline__ uint4 narrow(const float *x) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// One pair turned by its angle: every product rounded, then the sum.
__device__ __forceinline__ void turn(float &a, float &b, float c, float s) {
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = x;
}

// x / s to the nearest whole number, at most 127 in magnitude, as a byte.
__device__ __forceinline__ uint32_t code_of(float x, float s) {
    const float y = fminf(fmaxf(rintf(__fdiv_rn(x, s)), -127.f), 127.f);
    return (uint32_t)(int)y & 0xffu;
}

__device__ __forceinline__ uint2 codes_of(const float *x, float s) {
    uint32_t w[2] = {0, 0};
    if (s > 0.f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e >> 2] |= code_of(x[e], s) << (8 * (e & 3));
    }
    return make_uint2(w[0], w[1]);
}

// One block per token: its heads of q, k and v, LANES threads a head.
template <int LANES, bool INT8>
__global__ void __launch_bounds__(kThreads, kBlocks) append_rows_kernel(const __grid_constant__ RowsParams p) {
    constexpr int kSlots = kThreads / LANES;   // heads side by side
    const int b = (int)(blockIdx.x / (uint32_t)p.n), i = (int)(blockIdx.x % (uint32_t)p.n);
    const int64_t base = clamp_len(__ldg(p.lengths + b), p.c.cap);
    const int real = p.new_lengths ? (int)clamp_len(__ldg(p.new_lengths + b), p.n) : p.n;
    const int64_t pos = base + i;
    bool mine = i < real;
    if (mine && p.rope && pos >= p.positions) {
        if (threadIdx.x == 0) atomicOr(p.status, kDevBadIndex);
        mine = false;
    }
    if (mine) {
        // where the token's row lives
        int64_t lead = b, row = pos;
        bool kept = pos < p.c.cap;
        if (kept && p.c.block_table) {
            const int32_t at = (int32_t)pos;
            const int32_t j = p.c.page_shift >= 0 ? at >> p.c.page_shift : at / p.c.page_size;
            lead = __ldg(p.c.block_table + (int64_t)b * p.c.max_pages + j);
            row = at - j * p.c.page_size;
            if (lead < 0 || lead >= p.c.lead) {
                if (threadIdx.x == 0) atomicOr(p.status, kDevBadIndex);
                kept = false;
            }
        }
        const int u = (int)threadIdx.x % LANES;
        const Unit unit(p, u);
        float cs[8], sn[8];
        if (unit.turns) {
            const float4 *t = reinterpret_cast<const float4 *>(p.rope + pos * p.rope_stride + 8 * u);
            const float4 *s = reinterpret_cast<const float4 *>(p.rope + pos * p.rope_stride + p.r / 2 + 8 * u);
            *reinterpret_cast<float4 *>(cs) = __ldg(t);
            *reinterpret_cast<float4 *>(cs + 4) = __ldg(t + 1);
            *reinterpret_cast<float4 *>(sn) = __ldg(s);
            *reinterpret_cast<float4 *>(sn + 4) = __ldg(s + 1);
        }
        const int Hq = p.q ? p.Hq : 0, heads = Hq + 2 * p.c.Hkv;
        // kBatch heads' loads set out together; every thread of a head's lanes
        // takes the same turns of these loops
        for (int h0 = (int)threadIdx.x / LANES; h0 < heads; h0 += kBatch * kSlots) {
            uint4 wl[kBatch], wh[kBatch];
#pragma unroll
            for (int e = 0; e < kBatch; ++e) {
                const int h = h0 + e * kSlots;
                const bool is_q = h < Hq, is_v = h >= Hq + p.c.Hkv;
                if (h >= heads || (!is_q && !kept)) continue;
                const int hh = is_q ? h : h - Hq - (is_v ? p.c.Hkv : 0);
                const uint16_t *src = is_q ? p.q + b * p.qs[0] + i * p.qs[1] + hh * p.qs[2]
                                           : is_v ? p.v_new + b * p.vns[0] + i * p.vns[1] + hh * p.vns[2]
                                                  : p.k_new + b * p.kns[0] + i * p.kns[1] + hh * p.kns[2];
                wl[e] = *reinterpret_cast<const uint4 *>(src + (is_v ? 16 * u : unit.lo));
                wh[e] = *reinterpret_cast<const uint4 *>(src + (is_v ? 16 * u + 8 : unit.hi));
            }
#pragma unroll
            for (int e = 0; e < kBatch; ++e) {
                const int h = h0 + e * kSlots;
                const bool is_q = h < Hq, is_v = h >= Hq + p.c.Hkv;
                if (h >= heads || (!is_q && !kept)) continue;
                const int hh = is_q ? h : h - Hq - (is_v ? p.c.Hkv : 0);
                const int lo = is_v ? 16 * u : unit.lo, hi = is_v ? 16 * u + 8 : unit.hi;
                if (!INT8 && (is_v || !unit.turns)) {
                    // nothing to compute
                    uint16_t *dst = is_q ? p.q_out + b * p.qos[0] + i * p.qos[1] + hh * p.qos[2]
                                         : is_v ? static_cast<uint16_t *>(p.c.v) + lead * p.c.vs[0] + hh * p.c.vs[1] + row * p.c.vs[2]
                                                : static_cast<uint16_t *>(p.c.k) + lead * p.c.ks[0] + hh * p.c.ks[1] + row * p.c.ks[2];
                    *reinterpret_cast<uint4 *>(dst + lo) = wl[e];
                    *reinterpret_cast<uint4 *>(dst + hi) = wh[e];
                    continue;
                }
                float x[16];
                widen(wl[e], x);
                widen(wh[e], x + 8);
                if (!is_v && unit.turns) {
                    if (unit.across) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) turn(x[k], x[k + 8], cs[k], sn[k]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k) turn(x[2 * k], x[2 * k + 1], cs[k], sn[k]);
                    }
                }
                if (is_q || !INT8) {
                    uint16_t *dst = is_q ? p.q_out + b * p.qos[0] + i * p.qos[1] + hh * p.qos[2]
                                         : static_cast<uint16_t *>(p.c.k) + lead * p.c.ks[0] + hh * p.c.ks[1] + row * p.c.ks[2];
                    *reinterpret_cast<uint4 *>(dst + lo) = narrow(x);
                    *reinterpret_cast<uint4 *>(dst + hi) = narrow(x + 8);
                    continue;
                }
                // the largest magnitude of the row, by its bits (a NaN's are the
                // largest of all)
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < 16; ++k) top = max(top, __float_as_uint(x[k]) & 0x7fffffffu);
                const uint32_t lanes = LANES == 16 ? 0xffffu << (threadIdx.x & 16) : 0xffu << (threadIdx.x & 24);
                top = __reduce_max_sync(lanes, top);
                const float s = top < 0x7f800000u ? __fdiv_rn(__uint_as_float(top), 127.f) : __uint_as_float(0x7fffffffu);
                char *dst = is_v ? static_cast<char *>(p.c.v) + lead * p.c.vs[0] + hh * p.c.vs[1] + row * p.c.vs[2]
                                 : static_cast<char *>(p.c.k) + lead * p.c.ks[0] + hh * p.c.ks[1] + row * p.c.ks[2];
                *reinterpret_cast<uint2 *>(dst + lo) = codes_of(x, s);
                *reinterpret_cast<uint2 *>(dst + hi) = codes_of(x + 8, s);
                if (u == 0) {
                    float *to = is_v ? p.c.v_scale + lead * p.c.vss[0] + hh * p.c.vss[1] + row * p.c.vss[2]
                                     : p.c.k_scale + lead * p.c.kss[0] + hh * p.c.kss[1] + row * p.c.kss[2];
                    *to = s;
                }
            }
        }
    }
    if (!p.grid) {
        if (i == 0 && threadIdx.x == 0) write_length(p, b);
        return;
    }
    // the lengths are updated in place: by the last block, when none reads them
    // any more
    __shared__ int last;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(p.grid, 1) == (int)gridDim.x - 1;
        if (last) __threadfence();
    }
    __syncthreads();
    if (!last) return;
    for (int e = threadIdx.x; e < p.B; e += kThreads) write_length(p, e);
    if (threadIdx.x == 0) *p.grid = 0;
}

}  // namespace

int launch_append_rows(const RowsParams &p, cudaStream_t st) {
    const unsigned blocks = (unsigned)p.B * (unsigned)p.n;
    if (p.c.d == 128 && !p.c.int8) append_rows_kernel<8, false><<<blocks, kThreads, 0, st>>>(p);
    else if (p.c.d == 128) append_rows_kernel<8, true><<<blocks, kThreads, 0, st>>>(p);
    else if (!p.c.int8) append_rows_kernel<16, false><<<blocks, kThreads, 0, st>>>(p);
    else append_rows_kernel<16, true><<<blocks, kThreads, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

}  // namespace fd
