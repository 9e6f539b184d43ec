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
// one group of K and the same group of V: two 16-byte loads of each (append)
// are in flight per thread, and neighbouring lanes hold neighbouring groups
// of a row.
#include <cuda_runtime.h>

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

// 16 bf16 values (eight words of two) -> eight bytes of codes and the scale.
__device__ __forceinline__ uint2 quantise(const uint32_t *w, float g, uint32_t &scale) {
    uint32_t top = 0;   // |x| of bf16 values orders as its bits do
#pragma unroll
    for (int e = 0; e < 8; ++e) top = __vmaxu2(top, w[e] & 0x7fff7fffu);
    top = max(top & 0xffffu, top >> 16);
    const float amax = __uint_as_float(top << 16);
    const bool finite = top < 0x7f80u;
    float sg, r;
    {
        uint16_t two;
        const float want = __fdiv_rn(amax, 6.f * g);
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.f), "f"(want));
        scale = finite ? (uint32_t)two & 0xffu : 0x7fu;
        const __half s = __ushort_as_half((unsigned short)(scales_to_f16x2(two) & 0xffffu));
        sg = finite ? __half2float(s) * g : 0.f;
        r = sg > 0.f ? __frcp_rn(sg) : 0.f;
    }
    // a scale at its largest (448) leaves values past 6 s g: they saturate
    const float most = 8.f * sg;
    const bool past = amax > most && sg > 0.f;
    uint32_t out[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float x = i ? bf16hi(w[e]) : bf16lo(w[e]);
            if (past) x = fminf(fmaxf(x, -most), most);
            if (!finite) x = 0.f;
            // x / (s g) correctly rounded from the rounded reciprocal and one
            // residual (Markstein, "Computation of elementary functions on
            // the IBM RISC System/6000 processor", 1990), so that a value
            // halfway between two codes is seen as such
            const float q = x * r;
            // (and with x's sign, which the sum of a zero loses)
            y[i] = copysignf(__fmaf_rn(__fmaf_rn(-q, sg, x), r, q), x);
        }
        asm("{\n\t.reg .b8 c;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 c, %1, %2;\n\t"
            "mov.b32 %0, {c, 0, 0, 0};\n\t}"
            : "=r"(out[e])
            : "f"(y[1]), "f"(y[0]));
    }
    return make_uint2(out[0] | (out[1] << 8) | (out[2] << 16) | (out[3] << 24),
                      out[4] | (out[5] << 8) | (out[6] << 16) | (out[7] << 24));
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

// grid.y: sequences; grid.x strides over the sequence's (row, kv head, group).
template <int GROUPS>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ Fp4Rows p) {
    for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
        const int64_t base = base_of(p, b);
        const int64_t rows = min((int64_t)new_of(p, b), p.cap - base);
        const int64_t items = rows * p.Hkv * GROUPS;
        for (int64_t it = (int64_t)blockIdx.x * kThreads + threadIdx.x; it < items;
             it += (int64_t)gridDim.x * kThreads) {
            const int grp = (int)(it % GROUPS);
            const int64_t rest = it / GROUPS;
            int64_t i;
            int hk;
            if (rest < (1 << 30)) {   // the usual case: 32-bit division
                i = (uint32_t)rest / (uint32_t)p.Hkv;
                hk = (int)((uint32_t)rest - (uint32_t)i * (uint32_t)p.Hkv);
            } else {
                i = rest / p.Hkv;
                hk = (int)(rest % p.Hkv);
            }
            int64_t lead, row;
            if (!locate(p, b, base + i, lead, row)) continue;
            const uint4 *ksrc = reinterpret_cast<const uint4 *>(
                p.k_new + (int64_t)b * p.kns[0] + i * p.kns[1] + (int64_t)hk * p.kns[2] + grp * kGroup);
            const uint4 *vsrc = reinterpret_cast<const uint4 *>(
                p.v_new + (int64_t)b * p.vns[0] + i * p.vns[1] + (int64_t)hk * p.vns[2] + grp * kGroup);
            const uint4 k0 = ldg_stream(ksrc), k1 = ldg_stream(ksrc + 1);
            const uint4 v0 = ldg_stream(vsrc), v1 = ldg_stream(vsrc + 1);
            const uint32_t kw[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
            const uint32_t vw[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
            uint32_t sc;
            uint2 c = quantise(kw, p.k_global, sc);
            *reinterpret_cast<uint2 *>(p.k + lead * p.kst[0] + hk * p.kst[1] + row * p.kst[2] + grp * 8) = c;
            p.ks[lead * p.kss[0] + hk * p.kss[1] + row * p.kss[2] + grp] = (uint8_t)sc;
            c = quantise(vw, p.v_global, sc);
            *reinterpret_cast<uint2 *>(p.v + lead * p.vst[0] + hk * p.vst[1] + row * p.vst[2] + grp * 8) = c;
            p.vs[lead * p.vss[0] + hk * p.vss[1] + row * p.vss[2] + grp] = (uint8_t)sc;
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
__device__ __forceinline__ void expand(uint2 c, uint32_t scale, float g, bool ok, bool f32, void *out,
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
        x[e].x = ok ? x[e].x * g : 0.f;
        x[e].y = ok ? x[e].y * g : 0.f;
    }
    if (f32) {
        float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(out) + off);
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[e] = make_float4(x[2 * e].x, x[2 * e].y, x[2 * e + 1].x, x[2 * e + 1].y);
    } else {
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + off);
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = pack_bf16x2(x[e].x, x[e].y);
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

template <int GROUPS>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ Fp4Rows p) {
    const int64_t items = (int64_t)p.n * p.Hkv * GROUPS;
    for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
        const int64_t raw = (int64_t)__ldg(p.lengths + b), len = clamp_len(raw, p.cap);
        const int64_t start = p.start ? (int64_t)__ldg(p.start + b) : 0;
        if (blockIdx.x == 0 && threadIdx.x == 0 && (raw != len || start < 0))
            atomicOr(p.status, kDevBadLength);
        for (int64_t it = (int64_t)blockIdx.x * kThreads + threadIdx.x; it < items;
             it += (int64_t)gridDim.x * kThreads) {
            const int grp = (int)(it % GROUPS);
            const int64_t rest = it / GROUPS;
            int64_t i;
            int hk;
            if (rest < (1 << 30)) {
                i = (uint32_t)rest / (uint32_t)p.Hkv;
                hk = (int)((uint32_t)rest - (uint32_t)i * (uint32_t)p.Hkv);
            } else {
                i = rest / p.Hkv;
                hk = (int)(rest % p.Hkv);
            }
            const int64_t pos = start + i;
            int64_t lead = 0, row = 0;
            const bool ok = pos >= 0 && pos < len && locate(p, b, pos, lead, row);
            uint2 kc = make_uint2(0, 0), vc = make_uint2(0, 0);
            uint32_t ksc = 0, vsc = 0;
            if (ok) {
                kc = *reinterpret_cast<const uint2 *>(p.k + lead * p.kst[0] + hk * p.kst[1] + row * p.kst[2] + grp * 8);
                vc = *reinterpret_cast<const uint2 *>(p.v + lead * p.vst[0] + hk * p.vst[1] + row * p.vst[2] + grp * 8);
                ksc = p.ks[lead * p.kss[0] + hk * p.kss[1] + row * p.kss[2] + grp];
                vsc = p.vs[lead * p.vss[0] + hk * p.vss[1] + row * p.vss[2] + grp];
            }
            expand(kc, ksc, p.k_global, ok, p.out_f32, p.k_out,
                   (int64_t)b * p.kos[0] + i * p.kos[1] + (int64_t)hk * p.kos[2] + grp * kGroup);
            expand(vc, vsc, p.v_global, ok, p.out_f32, p.v_out,
                   (int64_t)b * p.vos[0] + i * p.vos[1] + (int64_t)hk * p.vos[2] + grp * kGroup);
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

}  // namespace

int launch_fp4_append(const Fp4Rows &p, cudaStream_t st) {
    if (p.d == 128) append_kernel<8><<<grid_of(p), kThreads, 0, st>>>(p);
    else if (p.d == 256) append_kernel<16><<<grid_of(p), kThreads, 0, st>>>(p);
    else return -2;
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

int launch_fp4_read(const Fp4Rows &p, cudaStream_t st) {
    if (p.d == 128) read_kernel<8><<<grid_of(p), kThreads, 0, st>>>(p);
    else if (p.d == 256) read_kernel<16><<<grid_of(p), kThreads, 0, st>>>(p);
    else return -2;
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

}  // namespace fd
