// fd_fp4_decode.cuh -- decode attention over a cache held in 4 bits (format in
// fd_fp4.cuh), flat or paged, head_dim 128 and 256; compiled for bf16 outputs in
// fd_fp4_decode.cu and for fp32 ones in fd_fp4_decode_f32.cu.
//
// What it computes, per query row: s_j = scale * q . k_j over the visible
// positions, w_j = 2^(s_j log2 e - m), out = sum_j w_j v_j / sum_j w_j, in one
// pass with a running reference m.  A position costs d/2 + d/16 bytes of K and
// as many of V, 0.28 of a bf16 cache's.
//
// Layout.  A warp walks 32 positions at a time through a private cp.async ring,
// turns the codes into fp16 operands in registers and feeds mma.sync m16n8k16,
// so nothing is written back to shared memory.  Positions are the M side of
// S^T = K Q^T and head dimensions the M side of O^T = V^T P^T; the query rows
// are N, in eights, so a group of up to 8 rows wastes nothing.
//   A warp takes 128 values of each row: at d = 128 it is on its own until its
//   piece of the prefix ends; at d = 256 two warps share the positions, each
//   with one half of the row, and add their partial scores through shared
//   memory, so that no code is converted twice and a warp's accumulators hold
//   128 dimensions in either case.
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
// of it.  The weights are kept as w * 2^4 (up to 2^14, see Reference) and
// rounded to fp16: off by up to 2^-11 of the weight, or by 2^-29 of the row's
// largest weight where that is more, which the rounding of a bf16 output hides.
// For fp32 outputs a weight, kept as w * 2^12 (up to 2^15), is the sum of two
// fp16 numbers, the second what the first's rounding left: off by up to 2^-22 of
// the weight or 2^-37 of the largest, for twice the MMAs on V.  The sums, the
// reference and both accumulators are fp32.
//
// What bounds it.  4 rows at d = 128, 4 sequences of 131,072 positions: 113.7 us,
// 5.3 TB/s (0.78 of a copy), DRAM and about 10 us of start and end.  24 rows at
// d = 256, 8 ragged sequences up to 32,768: 79.0 us; 8 of 16,384 66.4, in which
// the tensor pipe is busy for 26 us and the issue slots for 29: the latency of a
// step with 8 warps an SM.  64 ragged sequences up to 4,096 over pages of 16:
// 60.4 us, with 2.4 pieces a block.  A step of 32 positions is 640 instructions
// (one eight of rows, flat), half of them widening codes.  More than 32 rows are
// two parts, each of which reads and widens the whole prefix: 60 rows at d = 256,
// 8 sequences of 16,384, 145 us against 87 for 30.
//   fp32 outputs: 4 sequences of 131,072 positions 126.6 us against 113.4 for
// bf16; 24 rows at d = 256, 8 sequences of 16,384, 82 against 66.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "fd_fp4_split.cuh"

namespace fd {

namespace {

using namespace fp4;

constexpr int kSub = 32;               // positions per warp step
constexpr int kCode = kSub * 64;       // a step's K (or V) codes of 128 dimensions
constexpr int kScale = kSub * 8;
constexpr int kStage = 2 * kCode + 2 * kScale;

template <int NH, int NT>
struct Cfg {
    static constexpr int D = NH * 128;
    static constexpr int ROWS = 8 * NT;
    // Accumulators take 32 * NT registers: 16 warps an SM fit with one eight
    // of rows, 12 with two (as two blocks, so that one's start and end overlap
    // the other's middle), 8 beyond.  One block of 16 warps for one eight: long
    // 106.5 us against 109.7, paged 80 against 62; four of 4: long 113.6, d =
    // 256 61 against 48.  Two blocks of 6 with three eights spill: 102 against
    // 81.
    static constexpr int OCC = NT <= 2 ? 2 : 1;
    static constexpr int WARPS = NT == 2 ? 6 : 8;
    static constexpr int THREADS = WARPS * 32;
    static constexpr int STREAMS = WARPS / NH;         // warps (pairs) side by side
    static constexpr int TILE = kSub * STREAMS;        // positions per partition tile
    static constexpr int MERGE = STREAMS * ROWS * (D + 4) * 4;
    static constexpr int SWAP = NH == 2 ? 2 * WARPS * NT * 1024 : 0;   // partial scores, two steps
    static constexpr int QFRAG = NH * NT * 2048;
    // The ring is apart from what the end of a piece uses: the next piece's
    // first steps are on their way meanwhile.
    static constexpr int TAIL = (SWAP > MERGE ? SWAP : MERGE) + QFRAG + ROWS * 4 + 2 * STREAMS * ROWS * 4 + WARPS * 12;
    static constexpr int NST = (WARPS * 3 * kStage + TAIL + 1280) * OCC <= 228 * 1024 ? 3 : 2;
    static constexpr int RING = WARPS * NST * kStage;
    static constexpr int SMEM = RING + TAIL;
    static_assert((SMEM + 256 + 1024) * OCC <= 228 * 1024, "shared memory");
    static constexpr int QROWS = (ROWS + WARPS - 1) / WARPS;   // query rows a warp prepares
};

// A page or row number times a stride (neither is negative).
__device__ __forceinline__ uint64_t wide(uint32_t x, int64_t stride) { return x * (uint64_t)stride; }

template <int NH, int NT, bool PAGED, bool F32>
__global__ void __launch_bounds__((Cfg<NH, NT>::THREADS), (Cfg<NH, NT>::OCC))
fp4_decode_kernel(const __grid_constant__ Fp4Params fp) {
    using C = Cfg<NH, NT>;
    using R = Reference<F32>;
    constexpr int D = C::D, NST = C::NST, ROWS = C::ROWS, STREAMS = C::STREAMS, kThreads = C::THREADS;
    const Params &p = fp.p;
    extern __shared__ __align__(128) unsigned char smem[];
    // what the end of a piece sums, and during one the partial scores
    float *sums = reinterpret_cast<float *>(smem + C::RING);         // [STREAMS][ROWS][D + 4]
    float4 *swap = reinterpret_cast<float4 *>(smem + C::RING);       // [2][WARPS][2 * NT][32]
    uint4 *qfrag = reinterpret_cast<uint4 *>(smem + C::RING + (C::SWAP > C::MERGE ? C::SWAP : C::MERGE));
    float *qmul = reinterpret_cast<float *>(qfrag) + C::QFRAG / 4;   // qfrag: [NH][NT][4][32]; [ROWS]
    float *wm = qmul + ROWS, *wl = wm + STREAMS * ROWS;              // each stream's references and sums
    uint32_t *seen = reinterpret_cast<uint32_t *>(wl + STREAMS * ROWS);   // [WARPS][NST]: valid positions (paged)
    __shared__ int sh_last;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gid = lane >> 2, t4 = lane & 3;
    const int half = NH == 2 ? warp & 1 : 0, stream = warp / NH;
    const int G = gridDim.x, cta = blockIdx.x;

    Finder<C::TILE> finder(fp);
    const Share share(finder.total(), G);
    if (cta >= share.blocks && share.total > 0) return;
    const uint32_t t_begin = share.begin(cta), t_end = share.begin(cta + 1);

    unsigned char *ring = smem + warp * (NST * kStage);
    const uint32_t ring_a = smem_addr(ring);

    // ---- a piece: the tiles of one segment that are this block's.  Step n of a
    // warp covers positions start + n * TILE ..
    const int t4x16 = t4 * 16 + half * 64;
    const uint32_t to = ring_a + chunk_at(gid, t4);    // rows 8 further lie 512 bytes on
    // Pages whose size is a power of two from 8 on are looked up by runs of 8 or
    // 16 rows, others row by row.  64 sequences of 2,040 positions over pages of
    // 8: 54.7 us; of 12: 57.0; of 24: 56.2, by runs with a division each 60.5.
    const bool runs = PAGED && p.page_shift >= 3, runs16 = PAGED && p.page_shift >= 4;
    int start = 0, steps = 0, len = 0, seq = 0;
    const uint8_t *kb = nullptr, *vb = nullptr, *ksb = nullptr, *vsb = nullptr;
    // Pages of the runs of 8 rows of eight steps: lane 4 * (n % 8) + i has run i
    // of step n, -1 past the steps and where there is none.  The next eight are
    // looked up halfway through these.
    int pages = 0, later = 0;
    const auto lookup = [&](int n0) {
        const int n = n0 + (lane >> 2), i = lane & 3;
        const int pos0 = start + n * C::TILE;
        return n < steps && 8 * i < len - pos0 ? page_of(p, seq, pos0 + 8 * i) : -1;
    };
    // Copies step n into ring slot n % NST.  This lane's part: 16-byte chunk
    // lane & 3 of rows lane >> 2, + 8, .. (codes) and the scales of row `lane`.
    const auto fetch = [&](int n) {
        if (n < steps) {
            const int pos0 = start + n * C::TILE, left = len - pos0;   // positions that exist from here on
            const int slot = n % NST;
            const uint32_t dst = to + slot * kStage;
            const uint32_t sd = ring_a + slot * kStage + 2 * kCode + lane * 8;
            if (!PAGED) {
                const int64_t k8 = 8 * p.ks[2], v8 = 8 * p.vs[2];
                if (left >= kSub) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        copy16(dst + i * 512, kb + i * k8);
                        copy16(dst + i * 512 + kCode, vb + i * v8);
                    }
                    copy8(sd, ksb);
                    copy8(sd + kScale, vsb);
                } else {   // rows past the length: zeros, from an address that exists
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool in = 8 * i + gid < left;
                        copy16(dst + i * 512, in ? kb + i * k8 : static_cast<const uint8_t *>(p.k), in);
                        copy16(dst + i * 512 + kCode, in ? vb + i * v8 : static_cast<const uint8_t *>(p.v), in);
                    }
                    const bool in = lane < left;
                    copy8(sd, in ? ksb : fp.ks, in);
                    copy8(sd + kScale, in ? vsb : fp.vs, in);
                }
                // (steps are fetched in order)
                kb += C::TILE * p.ks[2];
                vb += C::TILE * p.vs[2];
                ksb += C::TILE * fp.kss[2];
                vsb += C::TILE * fp.vss[2];
            } else {
                uint32_t valid;
                if (runs) {
                    // runs of 8 rows lie on one page: four pages a step, or two
                    // where the pages hold whole runs of 16
                    if ((n & 7) == 4) later = lookup(n + 4);
                    if ((n & 7) == 0 && n > 0) pages = later;
                    const int at = (n & 7) * 4;
                    const int mine = __shfl_sync(0xffffffffu, pages, at + (lane >> 3));
                    const bool ok = lane < left && mine >= 0;
                    valid = __ballot_sync(0xffffffffu, ok);
                    const uint8_t *k0 = kb, *v0 = vb;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        bool in = (valid >> (8 * i + gid)) & 1u;
                        if (i % 2 && runs16) {
                            k0 += 8 * p.ks[2];
                            v0 += 8 * p.vs[2];
                        } else {
                            const int pg = __shfl_sync(0xffffffffu, pages, at + i);
                            const uint32_t first = pg >= 0 ? pg : 0, row = ((pos0 + 8 * i) & (p.page_size - 1)) + gid;
                            k0 = kb + wide(first, p.ks[0]) + wide(row, p.ks[2]);
                            v0 = vb + wide(first, p.vs[0]) + wide(row, p.vs[2]);
                        }
                        copy16(dst + i * 512, in ? k0 : kb, in);
                        copy16(dst + i * 512 + kCode, in ? v0 : vb, in);
                    }
                    const uint32_t first = ok ? mine : 0, row = ok ? (pos0 + lane) & (p.page_size - 1) : 0;
                    copy8(sd, ksb + wide(first, fp.kss[0]) + wide(row, fp.kss[2]), ok);
                    copy8(sd + kScale, vsb + wide(first, fp.vss[0]) + wide(row, fp.vss[2]), ok);
                } else {
                    // any page size: row by row
                    int page = lane < left ? page_of(p, seq, pos0 + lane) : -1;
                    const bool ok = page >= 0;
                    const int row = ok ? page_row(p, pos0 + lane) : 0;
                    if (!ok) page = 0;
                    valid = __ballot_sync(0xffffffffu, ok);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int pg = __shfl_sync(0xffffffffu, page, 8 * i + gid);
                        const int rw = __shfl_sync(0xffffffffu, row, 8 * i + gid);
                        const bool in = (valid >> (8 * i + gid)) & 1u;
                        copy16(dst + i * 512, kb + (int64_t)pg * p.ks[0] + (int64_t)rw * p.ks[2], in);
                        copy16(dst + i * 512 + kCode, vb + (int64_t)pg * p.vs[0] + (int64_t)rw * p.vs[2], in);
                    }
                    copy8(sd, ksb + (int64_t)page * fp.kss[0] + (int64_t)row * fp.kss[2], ok);
                    copy8(sd + kScale, vsb + (int64_t)page * fp.vss[0] + (int64_t)row * fp.vss[2], ok);
                }
                if (lane == 0) seen[warp * NST + slot] = valid;
            }
        }
        copy_commit();
    };
    // The query rows this warp prepares, as bf16 pairs.
    uint2 qraw[C::QROWS][NH];
    // Starts on the piece [t0, t1) of segment g: its first copies and its query.
    const auto begin_piece = [&](const Seg &g, uint32_t t0, uint32_t t1) {
        len = g.len;
        seq = g.b;
        const uint32_t from = (t0 - g.first) * C::TILE + stream * kSub;
        start = (int)from;   // (not used where it passes 2^31: there are no steps)
        steps = steps_from(from, len, t1 - t0, C::TILE);
        kb = static_cast<const uint8_t *>(p.k) + (int64_t)g.hk * p.ks[1] + t4x16;
        vb = static_cast<const uint8_t *>(p.v) + (int64_t)g.hk * p.vs[1] + t4x16;
        ksb = fp.ks + (int64_t)g.hk * fp.kss[1] + half * 8;
        vsb = fp.vs + (int64_t)g.hk * fp.vss[1] + half * 8;
        if (!PAGED) {
            kb += (int64_t)g.b * p.ks[0] + (int64_t)(start + gid) * p.ks[2];
            vb += (int64_t)g.b * p.vs[0] + (int64_t)(start + gid) * p.vs[2];
            ksb += (int64_t)g.b * fp.kss[0] + (int64_t)(start + lane) * fp.kss[2];
            vsb += (int64_t)g.b * fp.vss[0] + (int64_t)(start + lane) * fp.vss[2];
        }
        if (runs) pages = lookup(0);
#pragma unroll
        for (int n = 0; n < NST - 1; ++n) fetch(n);
#pragma unroll
        for (int i = 0; i < C::QROWS; ++i) load_query<NH>(fp, g, warp + i * C::WARPS, qraw[i]);
    };
    Seg g;
    uint32_t t0 = 0, t1 = 0;
    bool more = share.total > 0 && first_piece(finder, t_begin, t_end, g, t0, t1);
    if (more) begin_piece(g, t0, t1);
    // Sequences with nothing to attend still need their output rows zeroed.
    zero_empty<D>(p, finder, cta, share.total > 0 ? share.blocks : G, tid, kThreads);

    while (more) {
        // ---- Q: fp16 fragments and each row's factor, while K and V arrive
#pragma unroll
        for (int i = 0; i < C::QROWS; ++i) {
            const int r = warp + i * C::WARPS;
            if (r >= ROWS) break;
            const float factor = scale_query<NH>(p, qraw[i]);
            if (lane == 0) qmul[r] = factor;
#pragma unroll
            for (int h = 0; h < NH; ++h)
                // values 4*lane .. +3 of the half: owner lane t = lane / 8, k step lane % 8
                reinterpret_cast<uint2 *>(qfrag)[((((h * NT + (r >> 3)) * 4 + ((lane & 7) >> 1)) * 32 +
                                                   (r & 7) * 4 + (lane >> 3)) * 2) + (lane & 1)] = qraw[i][h];
        }
        __syncthreads();

        float mr[NT][2], l[NT][2];
        float O[8][NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                mr[n][c] = kNone;
                l[n][c] = 0.f;
            }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) O[j][n][e] = 0.f;
        const uint4 *qf = qfrag + half * NT * 128 + lane;
        uint4 qr[4];         // one eight of rows keeps its fragments in registers
        if (NT == 1)
#pragma unroll
            for (int w = 0; w < 4; ++w) qr[w] = qf[w * 32];
        const float2 mul1 = *reinterpret_cast<const float2 *>(qmul + 2 * t4);

        for (int at_step = 0; at_step < steps; ++at_step) {
            copy_wait<NST - 2>();
            __syncwarp();
            fetch(at_step + NST - 1);
            unsigned char *st = ring + (at_step % NST) * kStage;
            const int pos0 = start + at_step * C::TILE;

            // ---- S^T = K Q^T over this warp's 128 values
            float S[2][NT][4];
            {
                const unsigned char *kh = st + chunk_at(gid, t4);
                const unsigned char *sc = st + 2 * kCode + gid * 8 + 2 * t4;
                uint4 ka[2], kc[2];
                uint32_t sa[2], sb[2];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) S[m][n][e] = 0.f;
                    ka[m] = *reinterpret_cast<const uint4 *>(kh + m * 1024);
                    kc[m] = *reinterpret_cast<const uint4 *>(kh + m * 1024 + 512);
                    sa[m] = scales_to_f16x2(*reinterpret_cast<const uint16_t *>(sc + m * 128));
                    sb[m] = scales_to_f16x2(*reinterpret_cast<const uint16_t *>(sc + m * 128 + 64));
                }
#pragma unroll
                for (int w = 0; w < 4; ++w) {   // word w: k steps 2w and 2w + 1
                    uint4 q4[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) q4[n] = NT == 1 ? qr[w] : qf[(n * 4 + w) * 32];
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
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
                        for (int n = 0; n < NT; ++n) mma(S[m][n], a[0], b[0], a[1], b[1], q4[n].x, q4[n].y);
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma(S[m][n], a[2], b[2], a[3], b[3], q4[n].z, q4[n].w);
                    }
                }
            }
            // d = 256: both halves' parts of the scores meet in shared memory;
            // both warps add the same two numbers, so they agree on everything
            // that follows.  Two buffers: one is written again only after the
            // next step's barrier, when the partner has read it.
            if (NH == 2) {
                float4 *mine = swap + (((at_step & 1) * C::WARPS + warp) * (2 * NT)) * 32 + lane;
                const float4 *theirs = swap + (((at_step & 1) * C::WARPS + (warp ^ 1)) * (2 * NT)) * 32 + lane;
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mine[(m * NT + n) * 32] = make_float4(S[m][n][0], S[m][n][1], S[m][n][2], S[m][n][3]);
                asm volatile("bar.sync %0, 64;" ::"r"(1 + stream) : "memory");
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float4 o = theirs[(m * NT + n) * 32];
                        S[m][n][0] += o.x; S[m][n][1] += o.y; S[m][n][2] += o.z; S[m][n][3] += o.w;
                    }
            }
            uint32_t valid;
            if (PAGED) valid = seen[warp * NST + at_step % NST];
            else valid = len - pos0 >= kSub ? 0xffffffffu : (1u << (len - pos0)) - 1u;
            const bool masked = valid != 0xffffffffu || (p.causal && pos0 + (kSub - 1) > len - p.n_q);

            // ---- mask, reference, weights
            if (masked) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        // last position the row sees
                        const int lim = p.causal ? len - p.n_q + (g.row0 + n * 8 + 2 * t4 + c) % p.n_q : len - 1;
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int e = c; e < 4; e += 2) {
                                const int at = m * 16 + gid + (e >> 1) * 8;
                                if (!((valid >> at) & 1u) || at > lim - pos0) S[m][n][e] = neg_inf();
                            }
                    }
            }
            // Scores in the log2 domain, each rounded to fp32 before the reference
            // is taken from them and from it: at 2^27 and more a product that kept
            // its low bits could lie 2^15 and more above or below a rounded reference.
            float top[NT][2];
            bool grow = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                // rows 8*n + 2*t4 and the next: factor on q.k
                const float2 mul = NT == 1 ? mul1 : *reinterpret_cast<const float2 *>(qmul + n * 8 + 2 * t4);
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        S[m][n][e] = __fmul_rn(S[m][n][e], mul.x);
                        S[m][n][e + 1] = __fmul_rn(S[m][n][e + 1], mul.y);
                    }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    top[n][c] = fmaxf(fmaxf(S[0][n][c], S[0][n][c + 2]), fmaxf(S[1][n][c], S[1][n][c + 2]));
                    grow |= __fsub_rn(top[n][c], mr[n][c]) > R::kGrow;
                }
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float x = top[n][c];
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                        // (a row that still sees nothing keeps kNone)
                        const float ref = fmaxf(mr[n][c], R::of(x));
                        const float by = fast_exp2(mr[n][c] - ref);
                        mr[n][c] = ref;
                        l[n][c] *= by;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            O[j][n][c] *= by;
                            O[j][n][c + 2] *= by;
                        }
                    }
            }
            // The weights of 16 positions as the MMA's operand, in fp16; for fp32
            // outputs with what that rounding left in a second one.
            const auto weigh = [&](int m, int n, uint32_t *hi, uint32_t *lo) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = fast_exp2(__fsub_rn(S[m][n][e], mr[n][e & 1]));
                l[n][0] += w[0] + w[2];
                l[n][1] += w[1] + w[3];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t h = pack_f16x2(w[2 * i], w[2 * i + 1]);
                    hi[i] = transpose8x8(h);
                    if (F32) {
                        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                        lo[i] = transpose8x8(pack_f16x2(w[2 * i] - x.x, w[2 * i + 1] - x.y));
                    }
                }
            };
            uint32_t P[2][NT][2], P2[NT][2];
            if (!F32)   // (fp32 outputs: half at a time, below, as registers are short)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int m = 0; m < 2; ++m) weigh(m, n, P[m][n], P2[n]);

            // A weight of 0 does not hide a NaN: where the window hides positions
            // from some rows, NaN scales of V become 0 and what they stand for
            // goes to the sums of the rows that see them.
            if (masked && p.causal) {
                uint2 *mine = reinterpret_cast<uint2 *>(st + 2 * kCode + kScale) + lane;
                const uint2 s8 = *mine;
                const uint2 hit = make_uint2(__vcmpeq4(s8.x & 0x7f7f7f7fu, 0x7f7f7f7fu),
                                             __vcmpeq4(s8.y & 0x7f7f7f7fu, 0x7f7f7f7fu));
                if (__any_sync(0xffffffffu, (hit.x | hit.y) != 0)) {
                    uint32_t bad = 0;   // positions of this lane's 16 dimensions
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t at = __ballot_sync(0xffffffffu, (((i < 4 ? hit.x : hit.y) >> (8 * (i & 3))) & 1u) != 0);
                        if (gid == i) bad = at;
                    }
                    *mine = make_uint2(s8.x & ~hit.x, s8.y & ~hit.y);
                    __syncwarp();
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int see = len - p.n_q + (g.row0 + n * 8 + 2 * t4 + c) % p.n_q + 1 - pos0;
                            const uint32_t seen_at = see >= kSub ? 0xffffffffu : see > 0 ? (1u << see) - 1u : 0u;
                            if (bad & valid & seen_at)
#pragma unroll
                                for (int j = 0; j < 8; ++j) O[j][n][c] = O[j][n][c + 2] = __uint_as_float(0x7fffffffu);
                        }
                }
            }

            // ---- O^T += V^T P^T over this warp's 128 dimensions
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                if (F32)
#pragma unroll
                    for (int n = 0; n < NT; ++n) weigh(m, n, P[m][n], P2[n]);
                const unsigned char *sc = st + 2 * kCode + kScale + m * 128 + 16 * t4 + gid;
                uint2 x[4];
                uint32_t s8[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int at = 2 * t4 + (e & 1) + (e >> 1) * 8;
                    x[e] = *reinterpret_cast<const uint2 *>(st + kCode + m * 1024 + chunk_at(at, gid >> 1) +
                                                            (gid & 1) * 8);
                    s8[e] = sc[(e & 1) * 8 + (e >> 1) * 64];
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
                            mma(O[4 * w + i][n], f0, f1, f2, f3, P[m][n][0], P[m][n][1]);
                        if (F32)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma(O[4 * w + i][n], f0, f1, f2, f3, P2[n][0], P2[n][1]);
                    }
                }
            }
            __syncwarp();   // the slot may be filled again
        }
        copy_wait<0>();

        // ---- the next piece sets out (the ring is this warp's own)
        const Seg now = g;
        const uint32_t n0 = t0, n1 = t1;
        more = next_piece(finder, p, t_end, g, t0, t1);
        if (more) begin_piece(g, t0, t1);

        // ---- the block's warps together
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], o);
                if (gid == 0 && half == 0) {
                    wm[stream * ROWS + n * 8 + 2 * t4 + c] = mr[n][c];
                    wl[stream * ROWS + n * 8 + 2 * t4 + c] = l[n][c];
                }
            }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = n * 8 + 2 * t4 + c;
                float M = kNone;
#pragma unroll
                for (int w = 0; w < STREAMS; ++w) M = fmaxf(M, wm[w * ROWS + r]);
                const float by = fast_exp2(mr[n][c] - M);
                // rows 2t and 2t + 1 apart, so that the 8 lanes of a 128-byte
                // store (4 rows, 2 groups) fall on different banks
                float *dst = sums + (stream * ROWS + n * 8 + c * 4 + t4) * (D + 4) + half * 128 + 16 * gid;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<float4 *>(dst + j * 4) =
                        make_float4(O[2 * j][n][c] * by, O[2 * j][n][c + 2] * by,
                                    O[2 * j + 1][n][c] * by, O[2 * j + 1][n][c + 2] * by);
            }
        __syncthreads();
        const bool alone = n1 - n0 == now.tiles;
        add_streams<D, ROWS, STREAMS, kThreads>(fp, now, alone, cta, sums, wm, wl);
        if (!alone)
            join_pieces<D, kThreads>(fp, share, now, cta, tid, sums, &sh_last, [] { __syncthreads(); });
    }
}

template <int NH, int NT, bool PAGED, bool F32>
int launch(const Fp4Params &p, int G, cudaStream_t st) {
    using C = Cfg<NH, NT>;
    static std::atomic<uint64_t> opted{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -5;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (!bit || !(opted.load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(fp4_decode_kernel<NH, NT, PAGED, F32>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
            return -5;
        opted.fetch_or(bit, std::memory_order_release);
    }
    fp4_decode_kernel<NH, NT, PAGED, F32><<<G, C::THREADS, C::SMEM, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

template <int NH, int NT, bool F32>
int launch_layout(const Fp4Params &p, int G, cudaStream_t st) {
    return p.p.mode == kPaged ? launch<NH, NT, true, F32>(p, G, st) : launch<NH, NT, false, F32>(p, G, st);
}

template <int NH, bool F32>
int launch_rows(const Fp4Params &p, int G, cudaStream_t st) {
    switch ((p.p.rows + 7) / 8) {
        case 1: return launch_layout<NH, 1, F32>(p, G, st);
        case 2: return launch_layout<NH, 2, F32>(p, G, st);
        case 3: return launch_layout<NH, 3, F32>(p, G, st);
        case 4: return launch_layout<NH, 4, F32>(p, G, st);
        default: return -2;
    }
}

template <bool F32>
int launch_decode(const Fp4Params &p, int G, cudaStream_t st) {
    return p.p.d == 128 ? launch_rows<1, F32>(p, G, st) : p.p.d == 256 ? launch_rows<2, F32>(p, G, st) : -2;
}

}  // namespace

}  // namespace fd
