// fd_prefill.cu -- attention of a chunk of new tokens over a cache by warp-level
// matrix instructions (mma.sync): every layout of caches.
//
// A block holds 64 of a kv head's packed rows (row r is token r / g, head
// r % g of the group), 16 to a warp, and walks the positions they see 64 at a
// time: K and V come to shared memory (int8 codes widened to bf16, which holds
// them exactly), S = Q K^T and O += P V in bf16 with fp32 sums, and the softmax
// keeps a running maximum and sum a row.
//
// It takes the calls that the tcgen05 kernel does not (a factor of 0 or below, strides
// that no tensor map has): 4 x 5 .. 16 tokens about 30,000 .. 65,536 positions 7,675 us,
// 2,048 tokens behind 30,720 9,653 us, 50 and 12 times what that one takes: its rows are not
// split over positions, and K and V wait for the products of the tile before.
#include <cuda_runtime.h>

#include "fd_device.cuh"
#include "fd_packed.cuh"
#include "fd_ptx.cuh"
#include "fd_prefill.h"

namespace fd {

namespace {

constexpr int kThreads = 128, kRows = 64, kTile = 64;

__device__ __forceinline__ void mma(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm(uint32_t *r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t *r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}


template <int D>
struct Smem {
    static constexpr int LD = D + 8;   // elements a row: 16 bytes more than a multiple of 128
    uint16_t q[kRows * LD], k[kTile * LD], v[kTile * LD];
    float ks[kTile], vs[kTile];
    int64_t rk[kTile], rv[kTile];      // where the tile's rows start (elements), -1: nowhere
};

template <int D, bool I8>
__global__ void __launch_bounds__(kThreads) prefill_simple_kernel(const __grid_constant__ PrefillParams p,
                                                                  int row_blocks) {
    extern __shared__ __align__(16) unsigned char raw[];
    Smem<D> &sm = *reinterpret_cast<Smem<D> *>(raw);
    constexpr int LD = Smem<D>::LD, CH = D / 8;
    const int rb = (int)(blockIdx.x % (unsigned)row_blocks);
    const int hk = (int)(blockIdx.x / (unsigned)row_blocks) % p.c.Hkv;
    const int b = (int)(blockIdx.x / (unsigned)row_blocks) / p.c.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t raw_len = __ldg(p.lengths + b), L = clamp_len(raw_len, p.c.cap);
    const int64_t raw_new = p.new_lengths ? __ldg(p.new_lengths + b) : p.n, fresh = clamp_len(raw_new, p.n);
    if (tid == 0 && (L != raw_len || fresh != raw_new)) atomicOr(p.status, kDevBadLength);
    const int64_t rows = fresh * p.g, r0 = (int64_t)rb * kRows;
    if (r0 >= rows) return;

    // the rows' queries; what is past them as zeros
    for (int e = tid; e < kRows * CH; e += kThreads) {
        const int r = e / CH, c = e % CH;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r0 + r < rows) {
            const int64_t i = (r0 + r) / p.g, h = (int64_t)hk * p.g + (r0 + r) % p.g;
            x = *reinterpret_cast<const uint4 *>(p.q + b * p.qs[0] + i * p.qs[1] + h * p.qs[2] + c * 8);
        }
        *reinterpret_cast<uint4 *>(&sm.q[r * LD + c * 8]) = x;
    }
    // the last position that this thread's two rows see (their tokens)
    int64_t last[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int64_t r = r0 + warp * 16 + (lane >> 2) + 8 * e;
        last[e] = r >= rows ? -1 : p.causal ? L - fresh + r / p.g : L - 1;
    }
    const int64_t top = min(rows - 1, r0 + kRows - 1) / p.g;
    const int64_t end = p.causal ? min(L, max((int64_t)0, L - fresh + top + 1)) : L;

    float o[D / 8][4], m[2] = {neg_inf(), neg_inf()}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.f;

    for (int64_t t0 = 0; t0 < end; t0 += kTile) {
        __syncthreads();
        if (tid < kTile) {
            const int64_t pos = t0 + tid;
            int64_t lead = b, row = pos;
            bool there = pos < end;
            if (there && p.c.block_table) {
                const int32_t at = (int32_t)pos;
                const int32_t j = p.c.page_shift >= 0 ? at >> p.c.page_shift : at / p.c.page_size;
                lead = __ldg(p.c.block_table + (int64_t)b * p.c.max_pages + j);
                row = at - j * p.c.page_size;
                there = lead >= 0 && lead < p.c.lead;
                if (!there) atomicOr(p.status, kDevBadIndex);
            }
            sm.rk[tid] = there ? lead * p.c.ks[0] + hk * p.c.ks[1] + row * p.c.ks[2] : -1;
            sm.rv[tid] = there ? lead * p.c.vs[0] + hk * p.c.vs[1] + row * p.c.vs[2] : -1;
            if (I8) {
                sm.ks[tid] = there ? p.c.k_scale[lead * p.c.kss[0] + hk * p.c.kss[1] + row * p.c.kss[2]] : 0.f;
                sm.vs[tid] = there ? p.c.v_scale[lead * p.c.vss[0] + hk * p.c.vss[1] + row * p.c.vss[2]] : 0.f;
            }
        }
        __syncthreads();
        if (!I8) {
            const uint16_t *kc = static_cast<const uint16_t *>(p.c.k), *vc = static_cast<const uint16_t *>(p.c.v);
#pragma unroll 4
            for (int e = tid; e < kTile * CH; e += kThreads) {
                const int r = e / CH, c = e % CH;
                uint4 x = make_uint4(0, 0, 0, 0), y = x;
                if (sm.rk[r] >= 0) {
                    x = *reinterpret_cast<const uint4 *>(kc + sm.rk[r] + c * 8);
                    y = *reinterpret_cast<const uint4 *>(vc + sm.rv[r] + c * 8);
                }
                *reinterpret_cast<uint4 *>(&sm.k[r * LD + c * 8]) = x;
                *reinterpret_cast<uint4 *>(&sm.v[r * LD + c * 8]) = y;
            }
        } else {
            const char *kc = static_cast<const char *>(p.c.k), *vc = static_cast<const char *>(p.c.v);
#pragma unroll 2
            for (int e = tid; e < kTile * CH / 2; e += kThreads) {
                const int r = e / (CH / 2), c = e % (CH / 2);
                uint4 x = make_uint4(0, 0, 0, 0), y = x;
                if (sm.rk[r] >= 0) {
                    x = *reinterpret_cast<const uint4 *>(kc + sm.rk[r] + c * 16);
                    y = *reinterpret_cast<const uint4 *>(vc + sm.rv[r] + c * 16);
                }
                const uint2 x0 = widen4(x.x), x1 = widen4(x.y), x2 = widen4(x.z), x3 = widen4(x.w);
                const uint2 y0 = widen4(y.x), y1 = widen4(y.y), y2 = widen4(y.z), y3 = widen4(y.w);
                uint4 *kd = reinterpret_cast<uint4 *>(&sm.k[r * LD + c * 16]);
                uint4 *vd = reinterpret_cast<uint4 *>(&sm.v[r * LD + c * 16]);
                kd[0] = make_uint4(x0.x, x0.y, x1.x, x1.y);
                kd[1] = make_uint4(x2.x, x2.y, x3.x, x3.y);
                vd[0] = make_uint4(y0.x, y0.y, y1.x, y1.y);
                vd[1] = make_uint4(y2.x, y2.y, y3.x, y3.y);
            }
        }
        __syncthreads();

        // S: 16 rows x 64 positions
        float s[kTile / 8][4];
#pragma unroll
        for (int n = 0; n < kTile / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
        const uint32_t qa = ptx::smem_u32(&sm.q[(warp * 16 + (lane & 15)) * LD + (lane >> 4) * 8]);
        const uint32_t ka = ptx::smem_u32(&sm.k[((lane & 7) + ((lane >> 4) & 1) * 8) * LD + ((lane >> 3) & 1) * 8]);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t a[4];
            ldsm(a, qa + kk * 32);
#pragma unroll
            for (int n = 0; n < kTile / 16; ++n) {
                uint32_t k4[4];
                ldsm(k4, ka + n * 16 * LD * 2 + kk * 32);
                mma(s[2 * n], a, k4[0], k4[1]);
                mma(s[2 * n + 1], a, k4[2], k4[3]);
            }
        }
        // softmax of this thread's two rows (four lanes share a row)
        float top2[2] = {m[0], m[1]};
#pragma unroll
        for (int n = 0; n < kTile / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = n * 8 + (lane & 3) * 2 + (e & 1);
                float x = s[n][e] * p.scale_log2;
                if (I8) x *= sm.ks[c];
                x = t0 + c <= last[e >> 1] && sm.rk[c] >= 0 ? x : neg_inf();
                s[n][e] = x;
                top2[e >> 1] = fmaxf(top2[e >> 1], x);
            }
        float shift[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            top2[e] = fmaxf(top2[e], __shfl_xor_sync(0xffffffffu, top2[e], 1));
            top2[e] = fmaxf(top2[e], __shfl_xor_sync(0xffffffffu, top2[e], 2));
            shift[e] = top2[e] == neg_inf() ? 0.f : top2[e];
            const float f = fast_exp2(m[e] - shift[e]);
            m[e] = top2[e];
            l[e] *= f;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
                o[n][2 * e] *= f;
                o[n][2 * e + 1] *= f;
            }
        }
        uint32_t w[kTile / 8][2];
#pragma unroll
        for (int n = 0; n < kTile / 8; ++n) {
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = fast_exp2(s[n][e] - shift[e >> 1]);
                l[e >> 1] += x[e];
                // (a hidden position's scale may be a NaN)
                if (I8) x[e] = s[n][e] == neg_inf() ? 0.f : x[e] * sm.vs[n * 8 + (lane & 3) * 2 + (e & 1)];
            }
            w[n][0] = pack_bf16x2(x[0], x[1]);
            w[n][1] = pack_bf16x2(x[2], x[3]);
        }
        // O += P V
        const uint32_t va = ptx::smem_u32(&sm.v[(lane & 15) * LD + (lane >> 4) * 8]);
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk) {
            const uint32_t a[4] = {w[2 * kk][0], w[2 * kk][1], w[2 * kk + 1][0], w[2 * kk + 1][1]};
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
                uint32_t v4[4];
                ldsm_t(v4, va + kk * 16 * LD * 2 + n * 32);
                mma(o[2 * n], a, v4[0], v4[1]);
                mma(o[2 * n + 1], a, v4[2], v4[3]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        const float inv = l[e] > 0.f ? 1.f / l[e] : 0.f;
        const int64_t r = r0 + warp * 16 + (lane >> 2) + 8 * e;
        if (r >= rows) continue;
        uint16_t *dst = p.out + b * p.os[0] + (r / p.g) * p.os[1] + ((int64_t)hk * p.g + r % p.g) * p.os[2] + (lane & 3) * 2;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
            *reinterpret_cast<uint32_t *>(dst + n * 8) = pack_bf16x2(o[n][2 * e] * inv, o[n][2 * e + 1] * inv);
    }
}

template <int D, bool I8>
int launch(const PrefillParams &p, cudaStream_t st) {
    const int64_t row_blocks = ceil_div((int64_t)p.n * p.g, kRows);
    const int64_t blocks = row_blocks * p.c.Hkv * p.B;
    if (blocks >= (int64_t)1 << 31) return -2;
    if (cudaFuncSetAttribute(prefill_simple_kernel<D, I8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)sizeof(Smem<D>)) != cudaSuccess)
        return -5;
    prefill_simple_kernel<D, I8><<<(unsigned)blocks, kThreads, sizeof(Smem<D>), st>>>(p, (int)row_blocks);
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

}  // namespace

int launch_prefill_simple(const PrefillParams &p, cudaStream_t st) {
    if (p.c.d == 128) return p.c.int8 ? launch<128, true>(p, st) : launch<128, false>(p, st);
    return p.c.int8 ? launch<256, true>(p, st) : launch<256, false>(p, st);
}

}  // namespace fd
