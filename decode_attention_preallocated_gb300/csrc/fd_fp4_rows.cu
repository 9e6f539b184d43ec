// fd_fp4_rows.cu -- the 4-bit cache's writer and its plain reader.
//
// append: a group of 16 values x becomes s = e4m3(max|x| / (6 g)) and codes
// e2m1(x / (s g)), both rounded to nearest even; s = 0 leaves zero codes, and
// a group that holds a NaN or an infinity gets the NaN scale, so that what
// reads it gives NaN and not a wrong number.
// read: code * s is exact in fp16; times g in fp32, rounded once to the
// output's type.
//
// Both move bytes and little else (2 + 9/16 bytes a value).  A thread takes two
// neighbouring groups of K and the same two of V, neighbouring lanes
// neighbouring groups of a row: addresses and page lookups serve 64 values, 64
// bytes of bf16 move as two 32-byte accesses (as four of 16 where the rows are
// not 32-byte aligned, 62 us instead of 51 below), and the next loads set out
// before the last values are worked on.  The quotients run on paired fp32
// operations, offsets are 32-bit products widened to 64.
//   Four prompts of 1,000 to 8,192 rows (8 heads x 128) into pages of 64 and
// 8,192 positions of each read back: 51.0 us for both calls, 251 MB moved, 0.73
// of the copy rate.  Alone: append 24 us, 0.70; read 28.9, 0.81, and into fp32
// 120, 0.36, as each 16-byte store lies 128 bytes from the next lane's.
// With one group a thread 55.1 for both, with one and no loads ahead 58.1.
#include <cuda_runtime.h>

#include <initializer_list>

#include "fd_device.cuh"
#include "fd_fp4.cuh"
#include "fd_fp4_launch.h"

namespace fd {

namespace {

using namespace fp4;

constexpr int kThreads = 128;
constexpr int kBlocks = 6;   // an SM: 85 registers a thread

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
__device__ __forceinline__ float2 unpair(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
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

// The larger magnitude of two pairs of bf16 numbers, NaN where one is; the
// signs of the result mean nothing.
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// What a call divides the largest magnitudes by, 6 g, and its reciprocal.
struct Factor {
    float g, g6, r6;
};
__device__ __forceinline__ Factor factor(float g) { return Factor{g, 6.f * g, __frcp_rn(6.f * g)}; }

// 16 bf16 values (eight words of two) -> eight bytes of codes and the scale.
// Quotients are correctly rounded from the rounded reciprocal of the divisor
// and one residual (Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990; within one unit where the divisor's
// mantissa is all ones), so that a value halfway between two codes is seen as
// such.
__device__ __forceinline__ uint2 quantise(const uint32_t *w, const Factor &f, uint32_t &scale) {
    const float g = f.g;
    uint32_t top = larger(larger(larger(w[0], w[1]), larger(w[2], w[3])),
                          larger(larger(w[4], w[5]), larger(w[6], w[7]))) & 0x7fff7fffu;
    top = max(top & 0xffffu, top >> 16);
    const float amax = __uint_as_float(top << 16);
    float want = amax * f.r6;
    if (want < 1024.f) want = __fmaf_rn(__fmaf_rn(-want, f.g6, amax), f.r6, want);   // (else 448)
    uint16_t two;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.f), "f"(want));
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
    // x / (s g), all of it negated, -q, x + (-q) s g and -q - r times that, which
    // keeps the sign of a zero; the codes' signs are turned at the end.  s = 0:
    // every quotient is a zero.
    const float r1 = sg > 0.f ? -__frcp_rn(sg) : -0.f;
    const uint64_t r = pair(r1, r1), d = pair(sg, sg);
    uint64_t y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint64_t x = pair(bf16lo(w[e]), bf16hi(w[e]));
        const uint64_t q = mul2(x, r);
        y[e] = fma2(fma2(q, d, x), r, q);
    }
    return make_uint2(codes4(y) ^ 0x88888888u, codes4(y + 4) ^ 0x88888888u);
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

// A thread's work: two neighbouring groups of units (row i, kv head hk) of a
// sequence, kPer units apart; `lane` counts the pairs of groups in a row.  A
// block takes p.span units of a sequence.
template <int LANES>
struct Walk {
    static constexpr int kPer = kThreads / LANES;
    int i, hk, lane, left;   // left: units from here on
    __device__ __forceinline__ Walk(const Fp4Rows &p, int64_t rows) {
        lane = (int)threadIdx.x % LANES;
        const int64_t first = (int64_t)blockIdx.x * p.span, end = min(rows * p.Hkv, first + p.span);
        const int64_t u = first + (int)threadIdx.x / LANES;
        left = u < end ? (int)((end - u + (kPer - 1)) / kPer) : 0;
        if (u < ((int64_t)1 << 31)) {
            i = (int)((uint32_t)u / (uint32_t)p.Hkv);
            hk = (int)((uint32_t)u - (uint32_t)i * (uint32_t)p.Hkv);
        } else {
            i = (int)(u / p.Hkv);
            hk = (int)(u % p.Hkv);
        }
    }
    __device__ __forceinline__ void next(const Fp4Rows &p) {
        --left;
        i += p.step_i;
        hk += p.step_hk;
        if (hk >= p.Hkv) {
            hk -= p.Hkv;
            ++i;
        }
    }
};

template <bool NARROW, typename T>
__device__ __forceinline__ T *at(T *base, const int64_t *strides, int64_t lead, int64_t row, int64_t hk) {
    return base + times<NARROW>(lead, strides[0]) + times<NARROW>(hk, strides[1]) + times<NARROW>(row, strides[2]);
}

// 32 bf16 values, in two accesses where the rows allow it.
__device__ __forceinline__ void load_pair(const uint16_t *src, bool whole, uint32_t *w) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (whole) {
            load32(src + h * kGroup, w + h * 8);
        } else {
            const uint4 a = ldg_stream(src + h * kGroup), b = ldg_stream(src + h * kGroup + 8);
            w[h * 8] = a.x; w[h * 8 + 1] = a.y; w[h * 8 + 2] = a.z; w[h * 8 + 3] = a.w;
            w[h * 8 + 4] = b.x; w[h * 8 + 5] = b.y; w[h * 8 + 6] = b.z; w[h * 8 + 7] = b.w;
        }
    }
}

// 32 bf16 values -> 16 bytes of codes and two scales.
__device__ __forceinline__ uint4 quantise_pair(const uint32_t *w, const Factor &f, uint16_t &scales) {
    uint32_t s0, s1;
    const uint2 a = quantise(w, f, s0), b = quantise(w + 8, f, s1);
    scales = (uint16_t)(s0 | (s1 << 8));
    return make_uint4(a.x, a.y, b.x, b.y);
}

// grid.y: sequences; grid.x: their units.  A thread's next values of K set out
// when its last are quantised, and the same for V.
template <int LANES, bool NARROW>
__global__ void __launch_bounds__(kThreads, kBlocks) append_kernel(const __grid_constant__ Fp4Rows p) {
    const Factor kf = factor(p.k_global), vf = factor(p.v_global);
    for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
        const int64_t base = base_of(p, b);
        Walk<LANES> w(p, min((int64_t)new_of(p, b), p.cap - base));
        const uint16_t *kb = p.k_new + times<NARROW>(b, p.kns[0]) + w.lane * 32;
        const uint16_t *vb = p.v_new + times<NARROW>(b, p.vns[0]) + w.lane * 32;
        uint32_t kw[16], vw[16];
        if (w.left > 0) {
            load_pair(kb + times<NARROW>(w.i, p.kns[1]) + times<NARROW>(w.hk, p.kns[2]), p.aligned32, kw);
            load_pair(vb + times<NARROW>(w.i, p.vns[1]) + times<NARROW>(w.hk, p.vns[2]), p.aligned32, vw);
        }
        while (w.left > 0) {
            int64_t lead = 0, row = 0;
            const bool to = locate(p, b, base + w.i, lead, row);
            const int hk = w.hk;
            w.next(p);
            uint16_t sc;
            uint4 c = quantise_pair(kw, kf, sc);
            if (w.left > 0)
                load_pair(kb + times<NARROW>(w.i, p.kns[1]) + times<NARROW>(w.hk, p.kns[2]), p.aligned32, kw);
            if (to) {
                *reinterpret_cast<uint4 *>(at<NARROW>(p.k + w.lane * 16, p.kst, lead, row, hk)) = c;
                *reinterpret_cast<uint16_t *>(at<NARROW>(p.ks + w.lane * 2, p.kss, lead, row, hk)) = sc;
            }
            c = quantise_pair(vw, vf, sc);
            if (w.left > 0)
                load_pair(vb + times<NARROW>(w.i, p.vns[1]) + times<NARROW>(w.hk, p.vns[2]), p.aligned32, vw);
            if (to) {
                *reinterpret_cast<uint4 *>(at<NARROW>(p.v + w.lane * 16, p.vst, lead, row, hk)) = c;
                *reinterpret_cast<uint16_t *>(at<NARROW>(p.vs + w.lane * 2, p.vss, lead, row, hk)) = sc;
            }
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

// Eight bytes of codes and their scale (twice) -> 16 outputs at `out`.
template <bool F32>
__device__ __forceinline__ void expand(uint32_t c0, uint32_t c1, uint32_t s, float g, bool aligned32, void *out) {
    uint32_t p[8];
    codes_to_f16x2(c0, p[0], p[1], p[2], p[3]);
    codes_to_f16x2(c1, p[4], p[5], p[6], p[7]);
    const uint64_t gg = pair(g, g);
    float2 x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t v = mul_f16x2(p[e], s);
        const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&v));
        x[e] = unpair(mul2(pair(y.x, y.y), gg));
    }
    if (F32) {
        float4 *dst = static_cast<float4 *>(out);
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[e] = make_float4(x[2 * e].x, x[2 * e].y, x[2 * e + 1].x, x[2 * e + 1].y);
    } else {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = pack_bf16x2(x[e].x, x[e].y);
        if (aligned32) {
            store32(out, w);
        } else {
            uint4 *dst = static_cast<uint4 *>(out);
            dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
            dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
}

// What a thread reads of a unit: codes and scales of K and V, zeros where there
// is no such position.
struct Read {
    uint4 kc, vc;
    uint32_t ksc, vsc;
};

template <bool NARROW>
__device__ __forceinline__ Read fetch(const Fp4Rows &p, int b, int64_t pos, int64_t len, int hk, int lane) {
    Read r{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0), 0, 0};
    int64_t lead = 0, row = 0;
    if (pos >= 0 && pos < len && locate(p, b, pos, lead, row)) {
        r.kc = ldg_stream(at<NARROW>(p.k + lane * 16, p.kst, lead, row, hk));
        r.vc = ldg_stream(at<NARROW>(p.v + lane * 16, p.vst, lead, row, hk));
        r.ksc = __ldg(reinterpret_cast<const uint16_t *>(at<NARROW>(p.ks + lane * 2, p.kss, lead, row, hk)));
        r.vsc = __ldg(reinterpret_cast<const uint16_t *>(at<NARROW>(p.vs + lane * 2, p.vss, lead, row, hk)));
    }
    return r;
}

template <bool F32>
__device__ __forceinline__ void expand_pair(uint4 c, uint32_t scales, float g, bool aligned32, uint8_t *out) {
    const uint32_t s = scales_to_f16x2(scales);
    expand<F32>(c.x, c.y, __byte_perm(s, 0, 0x1010), g, aligned32, out);
    expand<F32>(c.z, c.w, __byte_perm(s, 0, 0x3232), g, aligned32, out + kGroup * (F32 ? 4 : 2));
}

// As append_kernel; the next unit's codes set out before the last one's values
// are written.
template <int LANES, bool NARROW, bool F32>
__global__ void __launch_bounds__(kThreads, kBlocks) read_kernel(const __grid_constant__ Fp4Rows p) {
    constexpr int kSize = F32 ? 4 : 2;
    for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
        const int64_t raw = (int64_t)__ldg(p.lengths + b), len = clamp_len(raw, p.cap);
        const int64_t start = p.start ? (int64_t)__ldg(p.start + b) : 0;
        if (blockIdx.x == 0 && threadIdx.x == 0 && (raw != len || start < 0))
            atomicOr(p.status, kDevBadLength);
        Walk<LANES> w(p, p.n);
        if (w.left == 0) continue;
        uint8_t *kb = static_cast<uint8_t *>(p.k_out) + (times<NARROW>(b, p.kos[0]) + w.lane * 32) * kSize;
        uint8_t *vb = static_cast<uint8_t *>(p.v_out) + (times<NARROW>(b, p.vos[0]) + w.lane * 32) * kSize;
        Read now = fetch<NARROW>(p, b, start + w.i, len, w.hk, w.lane);
        while (true) {
            uint8_t *kd = kb + (times<NARROW>(w.i, p.kos[1]) + times<NARROW>(w.hk, p.kos[2])) * kSize;
            uint8_t *vd = vb + (times<NARROW>(w.i, p.vos[1]) + times<NARROW>(w.hk, p.vos[2])) * kSize;
            w.next(p);
            Read next = now;
            if (w.left > 0) next = fetch<NARROW>(p, b, start + w.i, len, w.hk, w.lane);
            expand_pair<F32>(now.kc, now.ksc, p.k_global, p.aligned32, kd);
            expand_pair<F32>(now.vc, now.vsc, p.v_global, p.aligned32, vd);
            if (w.left == 0) break;
            now = next;
        }
    }
}

// Threads take kSpan units each where that still makes kLeastBlocks blocks, else
// one; more where the grid would pass 2^16 blocks a sequence.  The prompts above:
// 54.2 us with 1, 51.0 with 2, 51.9 with 3; one token of 64 sequences is 64
// blocks with 1 and would be half idle with 2.
constexpr int kSpan = 2, kLeastBlocks = 304;
dim3 grid_of(Fp4Rows &p) {
    const int per = kThreads / (p.d / 32);
    const int64_t units = (int64_t)p.n * p.Hkv;
    int64_t each = p.B * units >= (int64_t)kLeastBlocks * per * kSpan ? kSpan : 1;
    const int64_t most = ceil_div(units, (int64_t)per << 16);
    if (each < most) each = most;
    p.span = each * per;
    p.step_i = per / p.Hkv;
    p.step_hk = per % p.Hkv;
    return dim3((unsigned)ceil_div(units, p.span), (unsigned)(p.B < 65535 ? p.B : 65535));
}

// Every stride, and every number that multiplies one, below 2^32: the prompts
// above take 50.9 us, with full products 51.9.
bool narrow(const Fp4Rows &p, const int64_t *k_rows, const int64_t *v_rows) {
    int64_t most = 0;
    for (int i = 0; i < 3; ++i)
        for (const int64_t s : {p.kst[i], p.vst[i], p.kss[i], p.vss[i], k_rows[i], v_rows[i]})
            most = s > most ? s : most;
    return most < ((int64_t)1 << 32);
}

}  // namespace

int launch_fp4_append(Fp4Rows p, cudaStream_t st) {
    const dim3 grid = grid_of(p);
    const bool n = narrow(p, p.kns, p.vns);
    if (p.d == 128 && n) append_kernel<4, true><<<grid, kThreads, 0, st>>>(p);
    else if (p.d == 128) append_kernel<4, false><<<grid, kThreads, 0, st>>>(p);
    else if (p.d == 256 && n) append_kernel<8, true><<<grid, kThreads, 0, st>>>(p);
    else if (p.d == 256) append_kernel<8, false><<<grid, kThreads, 0, st>>>(p);
    else return -2;
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

template <int LANES, bool NARROW>
static void launch_read(const Fp4Rows &p, dim3 grid, cudaStream_t st) {
    if (p.out_f32) read_kernel<LANES, NARROW, true><<<grid, kThreads, 0, st>>>(p);
    else read_kernel<LANES, NARROW, false><<<grid, kThreads, 0, st>>>(p);
}

int launch_fp4_read(Fp4Rows p, cudaStream_t st) {
    const dim3 grid = grid_of(p);
    const bool n = narrow(p, p.kos, p.vos);
    if (p.d == 128 && n) launch_read<4, true>(p, grid, st);
    else if (p.d == 128) launch_read<4, false>(p, grid, st);
    else if (p.d == 256 && n) launch_read<8, true>(p, grid, st);
    else if (p.d == 256) launch_read<8, false>(p, grid, st);
    else return -2;
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

}  // namespace fd
