// fd_fp4_decode.cu -- decode attention over a cache held in 4 bits (format in
// fd_fp4.cuh), flat or paged, head_dim 128 and 256.
//
// What it computes, per query row: s_j = scale * q . k_j over the visible
// positions, w_j = 2^(s_j log2 e - m), out = sum_j w_j v_j / sum_j w_j, in one
// pass with a running reference m.  A position costs d/2 + d/16 bytes of K and
// as many of V, a quarter of a bf16 cache.
//
// Layout.  Every warp is on its own: it walks 32 (d = 128) or 16 (d = 256)
// positions at a time through a private cp.async ring, turns the codes into
// fp16 operands in registers and feeds mma.sync m16n8k16, so nothing is
// written back to shared memory and no warp waits for another until its piece
// of the prefix ends.  Positions are the M side of S^T = K Q^T and head
// dimensions the M side of O^T = V^T P^T; the query rows are N, in eights, so
// a group of up to 8 rows wastes nothing.
//   K: lane 4*gid + t holds 32 consecutive values (two scale groups) of
//   position gid; the contraction runs over values in the order the lanes hold
//   them, and Q's fragments are laid out in that order.
//   V: lane 4*gid + t holds scale group gid of positions 2t, 2t+1, 2t+8,
//   2t+9; the nibbles of two positions are merged into one byte each, so that
//   one conversion yields the pair along positions that the MMA wants.
//   P: the S^T accumulator turned by movmatrix.
// code * scale is exact in fp16 (fd_fp4.cuh).  Q is scaled per row by a power
// of two so that its largest entry lies in [1, 2): a bf16 entry is then exact
// in fp16 down to 2^-14 of the largest, and below that off by at most 2^-25
// of it.  The weights are kept as w * 2^4 (up to 2^14, see kGrow) and
// rounded to fp16: off by up to 2^-11 of the weight, or by 2^-29 of the row's
// largest weight where that is more; the sums, the reference and both
// accumulators are fp32.
#include <cuda_runtime.h>

#include <atomic>

#include "fd_device.cuh"
#include "fd_fp4.cuh"
#include "fd_fp4_launch.h"

namespace fd {

namespace {

using namespace fp4;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
// The reference of a row is its running maximum less 4 when it was last set;
// it is set again only when a weight would pass 2^14, which keeps every weight
// within fp16 and spares most tiles the shuffles and the rescaling.
constexpr float kBelow = 4.f, kGrow = 14.f;

template <int NH, int NT>
struct Cfg {
    static constexpr int D = NH * 128;
    static constexpr int MT = 2 / NH;            // 16-position blocks per step
    static constexpr int SUB = 16 * MT;          // positions per warp step
    static constexpr int TILE = SUB * kWarps;    // positions per partition tile
    static constexpr int ROWS = 8 * NT;
    static constexpr int CODE = SUB * D / 2;     // bytes of K (or V) codes per step
    static constexpr int SCALE = SUB * D / 16;
    static constexpr int STAGE = 2 * CODE + 2 * SCALE;
    // accumulators of NH * NT * 32 registers: up to 32 of them leave room for
    // two blocks per SM
    static constexpr int OCC = NH * NT == 1 ? 2 : (NH * NT == 2 ? 2 : 1);
    static constexpr int NST = OCC == 2 ? 3 : 4;
    static constexpr int RING = kWarps * NST * STAGE;
    static constexpr int MERGE = kWarps * ROWS * (D + 4) * 4;
    static constexpr int QFRAG = NH * NT * 8 * 32 * 8;
    static constexpr int BODY = RING > MERGE ? RING : MERGE;
    static constexpr int SMEM = BODY + QFRAG + ROWS * 4 + kWarps * NST * 4;
    static_assert((SMEM + 64 + 1024) * OCC <= 228 * 1024, "shared memory");
    static_assert(QFRAG >= 2 * kWarps * ROWS * 4, "the warps' statistics reuse the Q fragments");
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 (or 8) bytes into shared memory; zeros when !ok (src is then not read).
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const uint8_t *src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src),
                 "r"(ok ? 8 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// Where 16-byte chunk c of position p's 64-byte half row lies in its array.
// Two positions share 128 bytes, and pairs of positions are rotated so that
// the K reads (8 lanes: 2 positions x 4 chunks) and the V reads (16 lanes: 4
// even or 4 odd positions x 2 chunks) each touch all 32 banks once.
__device__ __forceinline__ uint32_t chunk_at(int p, int c) {
    return (uint32_t)((p >> 1) * 128 + ((((p & 1) * 4 + c) ^ (2 * ((p >> 1) & 3))) * 16));
}

struct Seg {
    int b, hk, row0, rows;   // sequence, kv head, first row of the part, its rows
    int64_t len;
};

template <int NH, int NT, bool PAGED>
__global__ void __launch_bounds__(kThreads, (Cfg<NH, NT>::OCC))
fp4_decode_kernel(const __grid_constant__ Fp4Params fp) {
    using C = Cfg<NH, NT>;
    constexpr int D = C::D, MT = C::MT, SUB = C::SUB, NST = C::NST, ROWS = C::ROWS;
    const Params &p = fp.p;
    extern __shared__ __align__(128) unsigned char smem[];
    uint2 *qfrag = reinterpret_cast<uint2 *>(smem + C::BODY);          // [NH][NT][8][32]
    float *qmul = reinterpret_cast<float *>(smem + C::BODY + C::QFRAG);   // [ROWS]
    uint32_t *seen = reinterpret_cast<uint32_t *>(qmul + ROWS);        // [kWarps][NST]: valid positions
    // reference and sum of each warp's rows, once the Q fragments are done with
    float *wm = reinterpret_cast<float *>(qfrag), *wl = wm + kWarps * ROWS;   // [kWarps][ROWS]
    __shared__ int64_t sh_total, sh_seg, sh_first, sh_n;
    __shared__ int sh_last;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gid = lane >> 2, t4 = lane & 3;
    const int G = gridDim.x, cta = blockIdx.x;

    if (warp == 0) {
        const int64_t tot = total_tiles_warp(p);
        if (lane == 0) sh_total = tot;
    }
    __syncthreads();
    const int64_t total = sh_total;

    const auto seg_of = [&](int64_t s) {
        Seg g;
        const int hp = (int)(s % p.Hkv);
        g.b = (int)(s / p.Hkv);
        g.hk = hp / fp.parts;
        g.row0 = (hp % fp.parts) * p.rows;
        g.rows = min(p.rows, fp.all_rows - g.row0);
        g.len = seq_len(p, g.b);
        return g;
    };
    // Output pointer offset of row r of a segment.
    const auto out_off = [&](const Seg &g, int r) {
        const int rr = g.row0 + r;
        return (int64_t)g.b * p.os[0] + (int64_t)(rr % p.n_q) * p.os[1] +
               (int64_t)(g.hk * p.g + rr / p.n_q) * p.os[2];
    };
    const auto store8 = [&](int64_t off, const float *o) {
        if (p.out_f32) {
            float *dst = reinterpret_cast<float *>(p.out) + off;
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e] = o[e];
        } else {
            uint16_t *dst = reinterpret_cast<uint16_t *>(p.out) + off;
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(o[2 * e], o[2 * e + 1]);
            if ((reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
                *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    dst[2 * e] = (uint16_t)(w[e] & 0xffffu);
                    dst[2 * e + 1] = (uint16_t)(w[e] >> 16);
                }
            }
        }
    };

    // Segments with nothing to attend still need their output rows zeroed.
    for (int64_t s = cta; s < p.nseg; s += G) {
        if (seg_tiles(p, s) != 0) continue;
        const Seg g = seg_of(s);
        const float z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int e = tid; e < g.rows * (D / 8); e += kThreads)
            store8(out_off(g, e / (D / 8)) + (e % (D / 8)) * 8, z);
    }
    if (total == 0) return;
    const int32_t Gw = working_blocks(total, G);
    if (cta >= Gw) return;
    const Split sp{total, Gw};
    const int64_t t_begin = sp.start(cta), t_end = sp.start(cta + 1);

    unsigned char *ring = smem + warp * (NST * C::STAGE);
    const uint32_t ring_a = smem_addr(ring);

    int64_t t = t_begin;
    while (t < t_end) {
        __syncthreads();
        if (warp == 0) {
            SegPos pos;
            const int64_t s = seg_of_tile_warp(p, t, &pos);
            if (lane == 0) { sh_seg = s; sh_first = pos.first; sh_n = pos.ntiles; }
        }
        __syncthreads();
        const int64_t s = sh_seg, first = sh_first, nt = sh_n;
        if (s < 0 || nt <= 0) break;   // cannot happen for t < total
        const int64_t piece_end = min(t_end, first + nt);
        const Seg g = seg_of(s);
        const int len = (int)g.len;

        // ---- the warp's steps: step n covers positions start + n * TILE ..
        const int start = (int)((t - first) * C::TILE) + warp * SUB;
        const int ntile = (int)(piece_end - t);
        // steps whose first position lies in the prefix
        const int steps = start >= len ? 0 : min(ntile, (int)(((unsigned)(len - start) + (C::TILE - 1u)) / C::TILE));

        const uint8_t *kb = static_cast<const uint8_t *>(p.k) + (int64_t)g.hk * p.ks[1];
        const uint8_t *vb = static_cast<const uint8_t *>(p.v) + (int64_t)g.hk * p.vs[1];
        const uint8_t *ksb = fp.ks + (int64_t)g.hk * fp.kss[1];
        const uint8_t *vsb = fp.vs + (int64_t)g.hk * fp.vss[1];
        if (!PAGED) {
            kb += (int64_t)g.b * p.ks[0];
            vb += (int64_t)g.b * p.vs[0];
            ksb += (int64_t)g.b * fp.kss[0];
            vsb += (int64_t)g.b * fp.vss[0];
        }
        // Copies step n into ring slot n % NST.  Lane = position while the
        // rows are located (page lookup), then lane = 16-byte chunk.
        const auto fetch = [&](int n) {
            if (n < steps) {
                const int pos0 = start + n * C::TILE;
                const int slot = n % NST;
                const uint32_t dst = ring_a + slot * C::STAGE;
                const int mine = pos0 + lane;
                bool ok = lane < min(SUB, len - pos0);
                int page = 0, row = mine;
                if (PAGED) {
                    if (ok) {
                        page = page_of(p, g.b, mine);
                        row = page_row(p, mine);
                        ok = page >= 0;
                    }
                    if (!ok) { page = 0; row = 0; }
                }
                const uint32_t valid = __ballot_sync(0xffffffffu, ok);
                constexpr int CPR = D / 32;          // 16-byte chunks per row
                constexpr int RPI = 32 / CPR;        // rows per copy instruction
#pragma unroll
                for (int i = 0; i < SUB / RPI; ++i) {
                    const int r = i * RPI + lane / CPR, c = lane % CPR;
                    const bool in = (valid >> r) & 1u;
                    int64_t ko, vo;
                    if (PAGED) {
                        const int pg = __shfl_sync(0xffffffffu, page, r);
                        const int rw = __shfl_sync(0xffffffffu, row, r);
                        ko = (int64_t)pg * p.ks[0] + (int64_t)rw * p.ks[2];
                        vo = (int64_t)pg * p.vs[0] + (int64_t)rw * p.vs[2];
                    } else {
                        const int64_t rw = in ? pos0 + r : 0;
                        ko = rw * p.ks[2];
                        vo = rw * p.vs[2];
                    }
                    const uint32_t a = dst + (NH == 2 ? (c >> 2) * (SUB * 64) : 0) + chunk_at(r, c & 3);
                    copy16(a, kb + ko + c * 16, in);
                    copy16(a + C::CODE, vb + vo + c * 16, in);
                }
                const uint32_t sd = dst + 2 * C::CODE;
                if (NH == 1) {
                    const int64_t rw = PAGED || ok ? row : 0;
                    copy8(sd + lane * 8, ksb + (PAGED ? (int64_t)page * fp.kss[0] : 0) + rw * fp.kss[2], ok);
                    copy8(sd + C::SCALE + lane * 8,
                          vsb + (PAGED ? (int64_t)page * fp.vss[0] : 0) + rw * fp.vss[2], ok);
                } else {
                    // lanes 0-15 the K scales, lanes 16-31 the V scales
                    const int r = lane & 15;
                    const bool in = (valid >> r) & 1u;
                    int64_t pg = 0, rw = in ? pos0 + r : 0;
                    if (PAGED) {
                        pg = __shfl_sync(0xffffffffu, page, r);
                        rw = __shfl_sync(0xffffffffu, row, r);
                    }
                    const uint8_t *src = lane < 16 ? ksb + pg * fp.kss[0] * (PAGED ? 1 : 0) + rw * fp.kss[2]
                                                   : vsb + pg * fp.vss[0] * (PAGED ? 1 : 0) + rw * fp.vss[2];
                    copy16(sd + lane * 16, src, in);
                }
                if (lane == 0) seen[warp * NST + slot] = valid;
            }
            copy_commit();
        };
#pragma unroll
        for (int n = 0; n < NST - 1; ++n) fetch(n);

        // ---- Q: fp16 fragments and each row's factor, while K and V arrive
        for (int r = warp; r < ROWS; r += kWarps) {
            float x[NH][4];
            float amax = 0.f;
            const int rr = g.row0 + r;
            const uint16_t *src = p.q + (int64_t)g.b * p.qs[0] + (int64_t)(rr % p.n_q) * p.qs[1] +
                                  (int64_t)(g.hk * p.g + rr / p.n_q) * p.qs[2];
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[h][e] = r < g.rows ? __uint_as_float((uint32_t)src[h * 128 + lane * 4 + e] << 16) : 0.f;
                    amax = fmaxf(amax, fabsf(x[h][e]));
                }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            // 2^e <= amax < 2^(e+1); e within what 2^-e and 2^e can hold
            int e = (int)((__float_as_uint(amax) >> 23) & 255u) - 127;
            e = amax > 0.f ? max(-126, min(126, e)) : 0;
            const float down = __uint_as_float((uint32_t)(127 - e) << 23);
            if (lane == 0) qmul[r] = p.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const uint2 f = make_uint2(pack_f16x2(x[h][0] * down, x[h][1] * down),
                                           pack_f16x2(x[h][2] * down, x[h][3] * down));
                // values 4*lane .. +3 of the half: owner lane t = lane / 8, k step lane % 8
                qfrag[((h * NT + (r >> 3)) * 8 + (lane & 7)) * 32 + (r & 7) * 4 + (lane >> 3)] = f;
            }
        }
        __syncthreads();

        float mul[NT][2];    // rows 8*n + 2*t4 and the next: factor on q.k
        int lim[NT][2];      // last position each row sees
        float mr[NT][2], l[NT][2];
        float O[NH][8][NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = n * 8 + 2 * t4 + c;
                mul[n][c] = qmul[r];
                lim[n][c] = p.causal ? len - p.n_q + (g.row0 + r) % p.n_q : len - 1;
                mr[n][c] = neg_inf();
                l[n][c] = 0.f;
            }
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) O[h][j][n][e] = 0.f;

        for (int n0 = 0; n0 < steps; ++n0) {
            copy_wait<NST - 2>();
            __syncwarp();
            fetch(n0 + NST - 1);
            const unsigned char *st = ring + (n0 % NST) * C::STAGE;
            const int pos0 = start + n0 * C::TILE;

            // ---- S^T = K Q^T
            float S[MT][NT][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[m][n][e] = 0.f;
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const unsigned char *kh = st + h * (SUB * 64);
                const unsigned char *sc = st + 2 * C::CODE + h * 8 + 2 * t4;
                uint4 ka[MT], kc[MT];
                uint32_t sa[MT], sb[MT];
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    ka[m] = *reinterpret_cast<const uint4 *>(kh + chunk_at(m * 16 + gid, t4));
                    kc[m] = *reinterpret_cast<const uint4 *>(kh + chunk_at(m * 16 + gid + 8, t4));
                    sa[m] = scales_to_f16x2(*reinterpret_cast<const uint16_t *>(sc + (m * 16 + gid) * (NH * 8)));
                    sb[m] = scales_to_f16x2(*reinterpret_cast<const uint16_t *>(sc + (m * 16 + gid + 8) * (NH * 8)));
                }
#pragma unroll
                for (int w = 0; w < 4; ++w) {   // word w: k steps 2w and 2w + 1
                    uint2 qf[2][NT];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            qf[i][n] = qfrag[((h * NT + n) * 8 + 2 * w + i) * 32 + lane];
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const uint32_t wa = w == 0 ? ka[m].x : w == 1 ? ka[m].y : w == 2 ? ka[m].z : ka[m].w;
                        const uint32_t wb = w == 0 ? kc[m].x : w == 1 ? kc[m].y : w == 2 ? kc[m].z : kc[m].w;
                        const uint32_t ga = __byte_perm(sa[m], 0, w < 2 ? 0x1010 : 0x3232);
                        const uint32_t gb = __byte_perm(sb[m], 0, w < 2 ? 0x1010 : 0x3232);
                        uint32_t a[4], b[4];
                        codes_to_f16x2(wa, a[0], a[1], a[2], a[3]);
                        codes_to_f16x2(wb, b[0], b[1], b[2], b[3]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            a[e] = mul_f16x2(a[e], ga);
                            b[e] = mul_f16x2(b[e], gb);
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma(S[m][n], a[2 * i], b[2 * i], a[2 * i + 1], b[2 * i + 1], qf[i][n].x, qf[i][n].y);
                    }
                }
            }

            // ---- mask, reference, weights
            const uint32_t valid = seen[warp * NST + n0 % NST];
            const bool whole = valid == (SUB == 32 ? 0xffffffffu : 0xffffu) &&
                               (!p.causal || pos0 + SUB - 1 <= len - p.n_q);
            float top[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                top[n][0] = top[n][1] = neg_inf();
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int c = e & 1, at = m * 16 + gid + (e >> 1) * 8;
                        float x = S[m][n][e] * mul[n][c];
                        if (!whole && (!((valid >> at) & 1u) || pos0 + at > lim[n][c])) x = neg_inf();
                        S[m][n][e] = x;
                        top[n][c] = fmaxf(top[n][c], x);
                    }
            }
            bool grow = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) grow |= top[n][c] - mr[n][c] > kGrow;
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float x = top[n][c];
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                        const float to = fmaxf(mr[n][c], x - kBelow);
                        const float by = mr[n][c] == neg_inf() ? 0.f : fast_exp2(mr[n][c] - to);
                        mr[n][c] = to;
                        l[n][c] *= by;
#pragma unroll
                        for (int h = 0; h < NH; ++h)
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                O[h][j][n][c] *= by;
                                O[h][j][n][c + 2] *= by;
                            }
                    }
            }
            uint32_t P[MT][NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float m0 = mr[n][0] == neg_inf() ? 0.f : mr[n][0];
                const float m1 = mr[n][1] == neg_inf() ? 0.f : mr[n][1];
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const float w0 = fast_exp2(S[m][n][0] - m0), w1 = fast_exp2(S[m][n][1] - m1);
                    const float w2 = fast_exp2(S[m][n][2] - m0), w3 = fast_exp2(S[m][n][3] - m1);
                    l[n][0] += w0 + w2;
                    l[n][1] += w1 + w3;
                    P[m][n][0] = transpose8x8(pack_f16x2(w0, w1));
                    P[m][n][1] = transpose8x8(pack_f16x2(w2, w3));
                }
            }

            // ---- O^T += V^T P^T
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const unsigned char *vh = st + C::CODE + h * (SUB * 64) + (gid & 1) * 8;
                const unsigned char *sc = st + 2 * C::CODE + C::SCALE + h * 8 + gid;
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    uint2 x[4];
                    uint32_t s8[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int at = m * 16 + 2 * t4 + (e & 1) + (e >> 1) * 8;
                        x[e] = *reinterpret_cast<const uint2 *>(vh + chunk_at(at, gid >> 1));
                        s8[e] = sc[at * (NH * 8)];
                    }
                    const uint32_t g01 = scales_to_f16x2(s8[0] | (s8[1] << 8));
                    const uint32_t g23 = scales_to_f16x2(s8[2] | (s8[3] << 8));
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const uint32_t x0 = w ? x[0].y : x[0].x, x1 = w ? x[1].y : x[1].x;
                        const uint32_t x2 = w ? x[2].y : x[2].x, x3 = w ? x[3].y : x[3].x;
                        constexpr uint32_t lo = 0x0f0f0f0fu;
                        uint32_t a0[4], a1[4], a2[4], a3[4];
                        codes_to_f16x2((x0 & lo) | ((x1 << 4) & ~lo), a0[0], a0[1], a0[2], a0[3]);
                        codes_to_f16x2(((x0 >> 4) & lo) | (x1 & ~lo), a1[0], a1[1], a1[2], a1[3]);
                        codes_to_f16x2((x2 & lo) | ((x3 << 4) & ~lo), a2[0], a2[1], a2[2], a2[3]);
                        codes_to_f16x2(((x2 >> 4) & lo) | (x3 & ~lo), a3[0], a3[1], a3[2], a3[3]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t f0 = mul_f16x2(a0[i], g01), f1 = mul_f16x2(a1[i], g01);
                            const uint32_t f2 = mul_f16x2(a2[i], g23), f3 = mul_f16x2(a3[i], g23);
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma(O[h][4 * w + i][n], f0, f1, f2, f3, P[m][n][0], P[m][n][1]);
                        }
                    }
                }
            }
            __syncwarp();   // the slot may be filled again
        }
        copy_wait<0>();
        __syncthreads();   // every warp is past its ring and the Q fragments

        // ---- the block's warps together
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], o);
                if (gid == 0) {
                    wm[warp * ROWS + n * 8 + 2 * t4 + c] = mr[n][c];
                    wl[warp * ROWS + n * 8 + 2 * t4 + c] = l[n][c];
                }
            }
        __syncthreads();
        float *sums = reinterpret_cast<float *>(smem);   // [kWarps][ROWS][D + 4]
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = n * 8 + 2 * t4 + c;
                float M = neg_inf();
#pragma unroll
                for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w * ROWS + r]);
                const float by = mr[n][c] == neg_inf() ? 0.f : fast_exp2(mr[n][c] - M);
                // rows 2t and 2t + 1 apart, so that the 8 lanes of a 128-byte
                // store (4 rows, 2 groups) fall on different banks
                float *dst = sums + (warp * ROWS + n * 8 + c * 4 + t4) * (D + 4) + 16 * gid;
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<float4 *>(dst + h * 128 + j * 4) =
                            make_float4(O[h][2 * j][n][c] * by, O[h][2 * j][n][c + 2] * by,
                                        O[h][2 * j + 1][n][c] * by, O[h][2 * j + 1][n][c + 2] * by);
            }
        __syncthreads();
        const int c_first = sp.owner(first), c_last = sp.owner(first + nt - 1);
        const bool alone = c_first == c_last;
        float *slot = slot_ptr(p, s, cta);
        for (int e = tid; e < g.rows * (D / 8); e += kThreads) {
            const int r = e / (D / 8), col = (e % (D / 8)) * 8;
            float M = neg_inf(), L = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w * ROWS + r]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float x = wm[w * ROWS + r];
                L += x == neg_inf() ? 0.f : wl[w * ROWS + r] * fast_exp2(x - M);
            }
            float o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            const int at = (r & ~7) + (r & 1) * 4 + ((r & 7) >> 1);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 *src = reinterpret_cast<const float4 *>(sums + (w * ROWS + at) * (D + 4) + col);
                const float4 a = src[0], b = src[1];
                o[0] += a.x; o[1] += a.y; o[2] += a.z; o[3] += a.w;
                o[4] += b.x; o[5] += b.y; o[6] += b.z; o[7] += b.w;
            }
            if (alone) {
                const float by = L > 0.f || L != L ? fp.v_global / L : 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] *= by;
                store8(out_off(g, r) + col, o);
            } else {
                float4 *dst = reinterpret_cast<float4 *>(slot + (int64_t)r * D + col);
                dst[0] = make_float4(o[0], o[1], o[2], o[3]);
                dst[1] = make_float4(o[4], o[5], o[6], o[7]);
                if (col == 0) {
                    slot[(int64_t)p.rows * D + r] = M;
                    slot[(int64_t)p.rows * D + p.rows + r] = L;
                }
            }
        }

        // ---- split segments: the last block to finish joins the pieces
        if (!alone) {
            __threadfence();
            __syncthreads();
            if (tid == 0) sh_last = atomicAdd(p.counters + s, 1) == c_last - c_first;
            __syncthreads();
            if (sh_last) {
                __threadfence();
                for (int e = tid; e < g.rows * (D / 8); e += kThreads) {
                    const int r = e / (D / 8), col = (e % (D / 8)) * 8;
                    float M = neg_inf(), L = 0.f;
                    float o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
                    for (int c2 = c_first; c2 <= c_last; ++c2) {
                        const float *sl = slot_ptr(p, s, c2);
                        const float mv = __ldcg(sl + (int64_t)p.rows * D + r);
                        const float lv = __ldcg(sl + (int64_t)p.rows * D + p.rows + r);
                        const float4 a = __ldcg(reinterpret_cast<const float4 *>(sl + (int64_t)r * D + col));
                        const float4 b = __ldcg(reinterpret_cast<const float4 *>(sl + (int64_t)r * D + col + 4));
                        const float to = fmaxf(M, mv);
                        const float u = M == neg_inf() ? 0.f : fast_exp2(M - to);
                        const float w = mv == neg_inf() ? 0.f : fast_exp2(mv - to);
                        M = to;
                        L = L * u + w * lv;
                        const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = o[i] * u + w * x[i];
                    }
                    const float by = L > 0.f || L != L ? fp.v_global / L : 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] *= by;
                    store8(out_off(g, r) + col, o);
                }
                if (tid == 0) p.counters[s] = 0;
            }
        }
        t = piece_end;
    }
}

template <int NH, int NT, bool PAGED>
int launch(const Fp4Params &p, int G, cudaStream_t st) {
    using C = Cfg<NH, NT>;
    static std::atomic<uint64_t> opted{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -5;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (!bit || !(opted.load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(fp4_decode_kernel<NH, NT, PAGED>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
            return -5;
        opted.fetch_or(bit, std::memory_order_release);
    }
    fp4_decode_kernel<NH, NT, PAGED><<<G, kThreads, C::SMEM, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

template <int NH, int NT>
int launch_layout(const Fp4Params &p, int G, cudaStream_t st) {
    return p.p.mode == kPaged ? launch<NH, NT, true>(p, G, st) : launch<NH, NT, false>(p, G, st);
}

}  // namespace

int fp4_max_rows(int d) { return d == 128 ? 32 : 16; }

int fp4_tile_tokens(int d) { return d == 128 ? Cfg<1, 1>::TILE : Cfg<2, 1>::TILE; }

int fp4_blocks_per_sm(int d, int rows) {
    const int nt = (rows + 7) / 8;
    if (d == 128) return nt <= 1 ? Cfg<1, 1>::OCC : nt == 2 ? Cfg<1, 2>::OCC : 1;
    return nt <= 1 ? Cfg<2, 1>::OCC : 1;
}

int launch_fp4_decode(const Fp4Params &p, int G, cudaStream_t st) {
    const int nt = (p.p.rows + 7) / 8;
    if (p.p.d == 128) {
        if (nt <= 1) return launch_layout<1, 1>(p, G, st);
        if (nt == 2) return launch_layout<1, 2>(p, G, st);
        if (nt == 3) return launch_layout<1, 3>(p, G, st);
        if (nt == 4) return launch_layout<1, 4>(p, G, st);
    } else if (p.p.d == 256) {
        if (nt <= 1) return launch_layout<2, 1>(p, G, st);
        if (nt == 2) return launch_layout<2, 2>(p, G, st);
    }
    return -2;
}

}  // namespace fd
