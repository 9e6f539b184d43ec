// fd_fp4_rows.cu -- the 4-bit cache's writer and its plain reader.
//
// append: a group of 16 values x becomes s = e4m3(max|x| / (6 g)) and codes
// e2m1(x / (s g)), both rounded to nearest even; s = 0 leaves zero codes, and
// a group that holds a NaN or an infinity gets the NaN scale, so that what
// reads it gives NaN and not a wrong number.
// read: code * s is exact in fp16; times g in fp32, rounded once to the
// output's type.
//
// Both move bytes and little else (2 + 9/16 bytes a value), so a thread takes
// one group of K and the same group of V, neighbouring lanes neighbouring
// groups of a row, and each bf16 group moves as one 32-byte access (two of 16
// where the rows are not 32-byte aligned).  What competes with the bytes is
// arithmetic: the quotients run on paired fp32 operations, and offsets are
// 32-bit products widened to 64.
#include <cuda_runtime.h>

#include <initializer_list>

#include "fd_device.cuh"
#include "fd_fp4.cuh"
#include "fd_fp4_launch.h"

namespace fd {

namespace {

using namespace fp4;

constexpr int kThreads = 256;

// Where row `pos` of sequence b lives: page (or sequence) and row in it.
// False, with FD_DEV_BAD_INDEX set, where the table names no page of the pool.
__device__ __forceinline__ bool locate(const Fp4Rows &p, int b, int64_t pos, int64_t &lead, int64_t &row) {
    if (!p.block_table) {
        lead = b;
        row = pos;
        return true;
    }
    const int32_t at = (int32_t)pos;
    const int32_t j = p.page_shift >= 0 ? at >> p.page_shift : at / p.page_size;
    const int32_t e = __ldg(p.block_table + (int64_t)b * p.max_pages + j);
    if (e < 0 || e >= p.num_pages) {
        atomicOr(p.status, kDevBadIndex);
        return false;
    }
    lead = e;
    row = at - j * p.page_size;
    return true;
}

// 32 bytes from or to global memory in one access.
__device__ __forceinline__ void load32(const void *src, uint32_t *w) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]),
                   "=r"(w[7])
                 : "l"(src));
}
__device__ __forceinline__ void store32(void *dst, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Two fp32 numbers in one 64-bit register, and operations on both.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Four pairs (y1, y0) .. of quotients -> four bytes of codes.
__device__ __forceinline__ uint32_t codes4(const uint64_t *y) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, e;\n\t.reg .f32 l0, h0, l1, h1, l2, h2, l3, h3;\n\t"
        "mov.b64 {l0, h0}, %1;\n\t"
        "mov.b64 {l1, h1}, %2;\n\t"
        "mov.b64 {l2, h2}, %3;\n\t"
        "mov.b64 {l3, h3}, %4;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, h0, l0;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, h1, l1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, h2, l2;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 e, h3, l3;\n\t"
        "mov.b32 %0, {a, b, c, e};\n\t}"
        : "=r"(r)
        : "l"(y[0]), "l"(y[1]), "l"(y[2]), "l"(y[3]));
    return r;
}

// 16 bf16 values (eight words of two) -> eight bytes of codes and the scale.
// g6 = 6 g.
__device__ __forceinline__ uint2 quantise(const uint32_t *w, float g, float g6, uint32_t &scale) {
    uint32_t top = 0;   // |x| of bf16 values orders as its bits do
#pragma unroll
    for (int e = 0; e < 8; ++e) top = __vmaxu2(top, w[e] & 0x7fff7fffu);
    top = max(top & 0xffffu, top >> 16);
    const float amax = __uint_as_float(top << 16);
    uint16_t two;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.f), "f"(__fdiv_rn(amax, g6)));
    scale = (uint32_t)two & 0xffu;
    const float sg = __half2float(__ushort_as_half((unsigned short)(scales_to_f16x2(two) & 0xffffu))) * g;
    if (top >= 0x7f80u || scale == 0x7eu) {
        // a value that is not finite, or the largest scale, past which values
        // saturate: one at a time
        if (top >= 0x7f80u) {
            scale = 0x7fu;
            return make_uint2(0, 0);
        }
        uint64_t y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            y[e] = pair(fminf(fmaxf(__fdiv_rn(bf16lo(w[e]), sg), -8.f), 8.f),
                        fminf(fmaxf(__fdiv_rn(bf16hi(w[e]), sg), -8.f), 8.f));
        return make_uint2(codes4(y), codes4(y + 4));
    }
    // x / (s g) correctly rounded from the rounded reciprocal and one residual
    // (Markstein, "Computation of elementary functions on the IBM RISC
    // System/6000 processor", 1990), so that a value halfway between two
    // codes is seen as such.  The residual is taken as q s g - x, which keeps
    // the sign of a zero.  s = 0: every quotient is a zero.
    const float r1 = sg > 0.f ? __frcp_rn(sg) : 0.f;
    const uint64_t r = pair(r1, r1), d = pair(sg, sg), less = pair(-r1, -r1);
    uint64_t y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint64_t x = pair(bf16lo(w[e]), bf16hi(w[e]));
        const uint64_t q = mul2(x, r);
        const uint64_t minus = pair(bf16lo(w[e] ^ 0x80008000u), bf16hi(w[e] ^ 0x80008000u));
        y[e] = fma2(fma2(q, d, minus), less, q);
    }
    return make_uint2(codes4(y), codes4(y + 4));
}

__device__ __forceinline__ int64_t base_of(const Fp4Rows &p, int b) {
    return clamp_len((int64_t)__ldg(p.lengths + b), p.cap);
}

__device__ __forceinline__ int new_of(const Fp4Rows &p, int b) {
    if (!p.new_lengths) return p.n;
    const int x = __ldg(p.new_lengths + b);
    return x < 0 ? 0 : (x > p.n ? p.n : x);
}

__device__ __forceinline__ void write_length(const Fp4Rows &p, int b) {
    const int64_t raw = (int64_t)p.lengths[b], base = clamp_len(raw, p.cap);
    const int real = new_of(p, b);
    if (raw != base || base + real > p.cap || (p.new_lengths && p.new_lengths[b] != real))
        atomicOr(p.status, kDevBadLength);
    if (p.lengths_out) p.lengths_out[b] = (int32_t)clamp_len(base + real, p.cap);
}

// a * stride, by one 32-bit widening product where the strides allow it.
template <bool NARROW>
__device__ __forceinline__ int64_t times(int64_t a, int64_t stride) {
    return NARROW ? (int64_t)(uint64_t)((uint64_t)(uint32_t)a * (uint32_t)stride) : a * stride;
}

// Item `it` of a sequence's (row, kv head, group) items.
template <int GROUPS>
__device__ __forceinline__ void item_of(const Fp4Rows &p, int64_t it, int64_t &i, int &hk, int &grp) {
    grp = (int)(it % GROUPS);
    const int64_t rest = it / GROUPS;
    if (p.head_shift >= 0) {
        i = rest >> p.head_shift;
        hk = (int)(rest - (i << p.head_shift));
    } else if (rest < ((int64_t)1 << 31)) {
        i = (uint32_t)rest / (uint32_t)p.Hkv;
        hk = (int)((uint32_t)rest - (uint32_t)i * (uint32_t)p.Hkv);
    } else {
        i = rest / p.Hkv;
        hk = (int)(rest % p.Hkv);
    }
}

// grid.y: sequences; grid.x strides over the sequence's (row, kv head, group).
template <int GROUPS, bool NARROW>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ Fp4Rows p) {
    const float k6 = 6.f * p.k_global, v6 = 6.f * p.v_global;
    for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
        const int64_t base = base_of(p, b);
        const int64_t rows = min((int64_t)new_of(p, b), p.cap - base);
        const int64_t items = rows * p.Hkv * GROUPS;
        for (int64_t it = (int64_t)blockIdx.x * kThreads + threadIdx.x; it < items;
             it += (int64_t)gridDim.x * kThreads) {
            int64_t i;
            int hk, grp;
            item_of<GROUPS>(p, it, i, hk, grp);
            const uint16_t *ksrc = p.k_new + times<NARROW>(b, p.kns[0]) + times<NARROW>(i, p.kns[1]) +
                                   times<NARROW>(hk, p.kns[2]) + grp * kGroup;
            const uint16_t *vsrc = p.v_new + times<NARROW>(b, p.vns[0]) + times<NARROW>(i, p.vns[1]) +
                                   times<NARROW>(hk, p.vns[2]) + grp * kGroup;
            uint32_t kw[8], vw[8];
            if (p.aligned32) {
                load32(ksrc, kw);
                load32(vsrc, vw);
            } else {
                const uint4 k0 = ldg_stream(ksrc), k1 = ldg_stream(ksrc + 8);
                const uint4 v0 = ldg_stream(vsrc), v1 = ldg_stream(vsrc + 8);
                kw[0] = k0.x; kw[1] = k0.y; kw[2] = k0.z; kw[3] = k0.w;
                kw[4] = k1.x; kw[5] = k1.y; kw[6] = k1.z; kw[7] = k1.w;
                vw[0] = v0.x; vw[1] = v0.y; vw[2] = v0.z; vw[3] = v0.w;
                vw[4] = v1.x; vw[5] = v1.y; vw[6] = v1.z; vw[7] = v1.w;
            }
            int64_t lead, row;
            if (!locate(p, b, base + i, lead, row)) continue;
            uint32_t sc;
            uint2 c = quantise(kw, p.k_global, k6, sc);
            *reinterpret_cast<uint2 *>(p.k + times<NARROW>(lead, p.kst[0]) + times<NARROW>(hk, p.kst[1]) +
                                       times<NARROW>(row, p.kst[2]) + grp * 8) = c;
            p.ks[times<NARROW>(lead, p.kss[0]) + times<NARROW>(hk, p.kss[1]) + times<NARROW>(row, p.kss[2]) + grp] =
                (uint8_t)sc;
            c = quantise(vw, p.v_global, v6, sc);
            *reinterpret_cast<uint2 *>(p.v + times<NARROW>(lead, p.vst[0]) + times<NARROW>(hk, p.vst[1]) +
                                       times<NARROW>(row, p.vst[2]) + grp * 8) = c;
            p.vs[times<NARROW>(lead, p.vss[0]) + times<NARROW>(hk, p.vss[1]) + times<NARROW>(row, p.vss[2]) + grp] =
                (uint8_t)sc;
        }
        if (!p.grid && blockIdx.x == 0 && threadIdx.x == 0) write_length(p, b);
    }
    if (!p.grid) return;
    // the lengths are updated in place: by the last block, when none reads
    // them any more
    __shared__ int last;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(p.grid, 1) == (int)(gridDim.x * gridDim.y) - 1;
        if (last) __threadfence();
    }
    __syncthreads();
    if (!last) return;
    for (int b = threadIdx.x; b < p.B; b += kThreads) write_length(p, b);
    if (threadIdx.x == 0) *p.grid = 0;
}

// Eight bytes of codes and their scale -> 16 outputs.
__device__ __forceinline__ void expand(uint2 c, uint32_t scale, float g, bool f32, bool aligned32, void *out,
                                       int64_t off) {
    uint32_t p[8];
    codes_to_f16x2(c.x, p[0], p[1], p[2], p[3]);
    codes_to_f16x2(c.y, p[4], p[5], p[6], p[7]);
    const uint32_t s = scales_to_f16x2(scale | (scale << 8));
    float2 x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t v = mul_f16x2(p[e], s);
        x[e] = __half22float2(*reinterpret_cast<const __half2 *>(&v));
        x[e].x *= g;
        x[e].y *= g;
    }
    if (f32) {
        float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(out) + off);
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[e] = make_float4(x[2 * e].x, x[2 * e].y, x[2 * e + 1].x, x[2 * e + 1].y);
    } else {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = pack_bf16x2(x[e].x, x[e].y);
        if (aligned32) {
            store32(static_cast<uint16_t *>(out) + off, w);
        } else {
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + off);
            dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
            dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
}

template <int GROUPS, bool NARROW>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ Fp4Rows p) {
    const int64_t items = (int64_t)p.n * p.Hkv * GROUPS;
    for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
        const int64_t raw = (int64_t)__ldg(p.lengths + b), len = clamp_len(raw, p.cap);
        const int64_t start = p.start ? (int64_t)__ldg(p.start + b) : 0;
        if (blockIdx.x == 0 && threadIdx.x == 0 && (raw != len || start < 0))
            atomicOr(p.status, kDevBadLength);
        for (int64_t it = (int64_t)blockIdx.x * kThreads + threadIdx.x; it < items;
             it += (int64_t)gridDim.x * kThreads) {
            int64_t i;
            int hk, grp;
            item_of<GROUPS>(p, it, i, hk, grp);
            const int64_t pos = start + i;
            int64_t lead = 0, row = 0;
            // (zero codes and scales where there is no such position)
            uint2 kc = make_uint2(0, 0), vc = make_uint2(0, 0);
            uint32_t ksc = 0, vsc = 0;
            if (pos >= 0 && pos < len && locate(p, b, pos, lead, row)) {
                kc = __ldg(reinterpret_cast<const uint2 *>(p.k + times<NARROW>(lead, p.kst[0]) +
                                                           times<NARROW>(hk, p.kst[1]) +
                                                           times<NARROW>(row, p.kst[2]) + grp * 8));
                vc = __ldg(reinterpret_cast<const uint2 *>(p.v + times<NARROW>(lead, p.vst[0]) +
                                                           times<NARROW>(hk, p.vst[1]) +
                                                           times<NARROW>(row, p.vst[2]) + grp * 8));
                ksc = __ldg(p.ks + times<NARROW>(lead, p.kss[0]) + times<NARROW>(hk, p.kss[1]) +
                            times<NARROW>(row, p.kss[2]) + grp);
                vsc = __ldg(p.vs + times<NARROW>(lead, p.vss[0]) + times<NARROW>(hk, p.vss[1]) +
                            times<NARROW>(row, p.vss[2]) + grp);
            }
            expand(kc, ksc, p.k_global, p.out_f32, p.aligned32, p.k_out,
                   times<NARROW>(b, p.kos[0]) + times<NARROW>(i, p.kos[1]) + times<NARROW>(hk, p.kos[2]) +
                       grp * kGroup);
            expand(vc, vsc, p.v_global, p.out_f32, p.aligned32, p.v_out,
                   times<NARROW>(b, p.vos[0]) + times<NARROW>(i, p.vos[1]) + times<NARROW>(hk, p.vos[2]) +
                       grp * kGroup);
        }
    }
}

// Blocks: one item a thread, up to 2^15 blocks per sequence.
dim3 grid_of(const Fp4Rows &p) {
    const int64_t items = (int64_t)p.n * p.Hkv * (p.d / kGroup);
    int64_t x = ceil_div(items, kThreads);
    if (x > 32768) x = 32768;
    if (x < 1) x = 1;
    return dim3((unsigned)x, (unsigned)(p.B < 65535 ? p.B : 65535));
}

// Every stride, and every number that multiplies one, below 2^32.
bool narrow(const Fp4Rows &p, const int64_t *k_rows, const int64_t *v_rows) {
    int64_t most = 0;
    for (int i = 0; i < 3; ++i)
        for (const int64_t s : {p.kst[i], p.vst[i], p.kss[i], p.vss[i], k_rows[i], v_rows[i]})
            most = s > most ? s : most;
    return most < ((int64_t)1 << 32);
}

}  // namespace

int launch_fp4_append(const Fp4Rows &p, cudaStream_t st) {
    const dim3 grid = grid_of(p);
    const bool n = narrow(p, p.kns, p.vns);
    if (p.d == 128 && n) append_kernel<8, true><<<grid, kThreads, 0, st>>>(p);
    else if (p.d == 128) append_kernel<8, false><<<grid, kThreads, 0, st>>>(p);
    else if (p.d == 256 && n) append_kernel<16, true><<<grid, kThreads, 0, st>>>(p);
    else if (p.d == 256) append_kernel<16, false><<<grid, kThreads, 0, st>>>(p);
    else return -2;
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

int launch_fp4_read(const Fp4Rows &p, cudaStream_t st) {
    const dim3 grid = grid_of(p);
    const bool n = narrow(p, p.kos, p.vos);
    if (p.d == 128 && n) read_kernel<8, true><<<grid, kThreads, 0, st>>>(p);
    else if (p.d == 128) read_kernel<8, false><<<grid, kThreads, 0, st>>>(p);
    else if (p.d == 256 && n) read_kernel<16, true><<<grid, kThreads, 0, st>>>(p);
    else if (p.d == 256) read_kernel<16, false><<<grid, kThreads, 0, st>>>(p);
    else return -2;
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

}  // namespace fd
