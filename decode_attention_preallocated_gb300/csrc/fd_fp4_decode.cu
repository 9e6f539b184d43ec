// fd_fp4_decode.cu -- decode attention over a cache held in 4 bits (format in
// fd_fp4.cuh), flat or paged, head_dim 128 and 256.
//
// What it computes, per query row: s_j = scale * q . k_j over the visible
// positions, w_j = 2^(s_j log2 e - m), out = sum_j w_j v_j / sum_j w_j, in one
// pass with a running reference m.  A position costs d/2 + d/16 bytes of K and
// as many of V, a quarter of a bf16 cache.
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

// The reference of a row is its running maximum less 4 when it was last set;
// it is set again only when a weight would pass 2^14, which keeps every weight
// within fp16 and spares most steps the shuffles and the rescaling.
constexpr float kBelow = 4.f, kGrow = 14.f;
// The reference of a row that has seen nothing yet.
constexpr float kNone = -3.402823466e38f;

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
    // the other's middle), 8 beyond.
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

// Pieces of a segment that are joined in groups of this many, when there are
// more than kOneJoin of them.
constexpr int kGroup8 = 8, kOneJoin = 12;

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 (or 8) bytes into shared memory; with `ok`, zeros where that is false
// (src is then not read).
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const uint8_t *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
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

// A segment: one part of the query rows of one (sequence, kv head).
struct Seg {
    int b, hp;               // sequence; kv head and part, hp = hk * parts + part
    int hk, row0, rows;      // kv head; first row of the part and its rows
    int len;
    uint32_t first, tiles;   // work unit of its first tile, and number of tiles
};

// Walks the launch's work units in order: every segment that has tiles holds
// p.seg_units units, the price of a piece's start and end, and then one per
// tile.  Every warp keeps its own copy (lane l holds the tile count of sequence
// 32 * chunk + l), so that no barrier is needed to find the next segment.
template <int TILE>
struct Finder {
    const Fp4Params &fp;
    int lane, chunk;
    uint32_t n;              // tiles per segment of this lane's sequence
    __device__ __forceinline__ Finder(const Fp4Params &f) : fp(f), lane(threadIdx.x & 31), chunk(0) { load(0); }
    __device__ __forceinline__ void load(int c) {
        chunk = c;
        const int b = c * 32 + lane;
        n = b < fp.p.B ? ((uint32_t)seq_len(fp.p, b) + (TILE - 1)) / TILE : 0;
    }
    __device__ __forceinline__ uint32_t units() const { return n > 0 ? n + fp.p.seg_units : 0; }
    __device__ __forceinline__ uint32_t total() {
        uint32_t sum = 0;
        for (int c = 0; c * 32 < fp.p.B; ++c) {
            if (c != chunk) load(c);
            sum += units();
        }
        return __reduce_add_sync(0xffffffffu, sum) * (uint32_t)fp.p.Hkv;
    }
    __device__ __forceinline__ void fill(Seg &g) const {
        g.hk = fp.parts == 1 ? g.hp : g.hp / fp.parts;
        g.row0 = (g.hp - g.hk * fp.parts) * fp.p.rows;
        g.rows = min(fp.p.rows, fp.all_rows - g.row0);
    }
    // The segment that holds unit t (below the total).
    __device__ __forceinline__ void find(uint32_t t, Seg &g) {
        uint32_t base = 0;
        for (int c = 0; c * 32 < fp.p.B; ++c) {
            if (c != chunk) load(c);
            const uint32_t mine = units() * (uint32_t)fp.p.Hkv;
            uint32_t upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += x;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, t - base < upto);
            if (hit) {
                const int src = __ffs(hit) - 1;
                const uint32_t before = base + __shfl_sync(0xffffffffu, upto - mine, src);
                g.tiles = __shfl_sync(0xffffffffu, n, src);
                const uint32_t each = g.tiles + fp.p.seg_units;
                g.b = c * 32 + src;
                g.hp = (int)((t - before) / each);
                g.first = before + (uint32_t)g.hp * each + fp.p.seg_units;
                g.len = (int)seq_len(fp.p, g.b);
                fill(g);
                return;
            }
            base += __shfl_sync(0xffffffffu, upto, 31);
        }
    }
    // The segment after g (one exists: the caller has units left).
    __device__ __forceinline__ void next(Seg &g) {
        g.first += g.tiles + fp.p.seg_units;
        if (++g.hp == fp.p.Hkv) {
            g.hp = 0;
            for (int c = (g.b + 1) / 32; c * 32 < fp.p.B; ++c) {
                if (c != chunk) load(c);
                const unsigned live = __ballot_sync(0xffffffffu, n > 0 && c * 32 + lane > g.b);
                if (live) {
                    const int src = __ffs(live) - 1;
                    g.b = c * 32 + src;
                    g.tiles = __shfl_sync(0xffffffffu, n, src);
                    break;
                }
            }
            g.len = (int)seq_len(fp.p, g.b);
        }
        fill(g);
    }
};

template <int NH, int NT, bool PAGED>
__global__ void __launch_bounds__((Cfg<NH, NT>::THREADS), (Cfg<NH, NT>::OCC))
fp4_decode_kernel(const __grid_constant__ Fp4Params fp) {
    using C = Cfg<NH, NT>;
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

    Finder<C::TILE> finder(fp);
    const uint32_t total = finder.total();
    // Blocks [0, Gw) share the units; with few of them a block takes at least
    // two, which costs less than one more piece to join.
    const int32_t Gw = (int32_t)min((uint32_t)G, (total + 1) / 2);
    if (cta >= Gw && total > 0) return;
    // floor(c * total / Gw) in 32 bits: c and the remainder are below Gw
    const uint32_t per = total > 0 ? total / (uint32_t)Gw : 0, rest = total - per * (uint32_t)Gw;
    const auto begins = [&](int c) { return (uint32_t)c * per + (uint32_t)c * rest / (uint32_t)Gw; };
    const Split sp{(int64_t)total, Gw};
    const uint32_t t_begin = begins(cta), t_end = begins(cta + 1);

    unsigned char *ring = smem + warp * (NST * kStage);
    const uint32_t ring_a = smem_addr(ring);

    // ---- a piece: the tiles of one segment that are this block's.  Step n of a
    // warp covers positions start + n * TILE ..
    const int t4x16 = t4 * 16 + half * 64;
    const uint32_t to = ring_a + chunk_at(gid, t4);    // rows 8 further lie 512 bytes on
    const bool runs = PAGED && (p.page_size & 7) == 0;
    int start = 0, steps = 0, len = 0, seq = 0;
    const uint8_t *kb = nullptr, *vb = nullptr, *ksb = nullptr, *vsb = nullptr;
    // Page of each of a step's four runs of 8 rows (in lanes 0 .. 3), looked up
    // a step ahead; -1 past the steps and where there is none.
    int ahead = 0;
    const auto lookup = [&](int n) {
        int e = -1;
        const int pos0 = start + n * C::TILE;
        if (n < steps && lane < 4 && 8 * lane < len - pos0) e = page_of(p, seq, pos0 + 8 * lane);
        return e;
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
                const int64_t far = (int64_t)n * C::TILE;
                const uint8_t *k0 = kb + far * p.ks[2], *v0 = vb + far * p.vs[2];
                const uint8_t *k1 = ksb + far * fp.kss[2], *v1 = vsb + far * fp.vss[2];
                const int64_t k8 = 8 * p.ks[2], v8 = 8 * p.vs[2];
                if (left >= kSub) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        copy16(dst + i * 512, k0 + i * k8);
                        copy16(dst + i * 512 + kCode, v0 + i * v8);
                    }
                    copy8(sd, k1);
                    copy8(sd + kScale, v1);
                } else {   // rows past the length: zeros, from an address that exists
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool in = 8 * i + gid < left;
                        copy16(dst + i * 512, in ? k0 + i * k8 : static_cast<const uint8_t *>(p.k), in);
                        copy16(dst + i * 512 + kCode, in ? v0 + i * v8 : static_cast<const uint8_t *>(p.v), in);
                    }
                    const bool in = lane < left;
                    copy8(sd, in ? k1 : fp.ks, in);
                    copy8(sd + kScale, in ? v1 : fp.vs, in);
                }
            } else {
                // row `lane`: its page and row in it
                int page, row;
                if (runs) {
                    page = __shfl_sync(0xffffffffu, ahead, lane >> 3);
                    row = page_row(p, pos0 + (lane & ~7)) + (lane & 7);
                } else {
                    page = lane < left ? page_of(p, seq, pos0 + lane) : -1;
                    row = lane < left ? page_row(p, pos0 + lane) : 0;
                }
                const bool ok = lane < left && page >= 0;
                if (page < 0) page = 0;
                if (!ok) row = 0;
                const uint32_t valid = __ballot_sync(0xffffffffu, ok);
                if (lane == 0) seen[warp * NST + slot] = valid;
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
                if (runs) ahead = lookup(n + 1);
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
        start = (int)((t0 - g.first) * C::TILE) + stream * kSub;
        steps = start >= len ? 0 : min((int)(t1 - t0), (int)(((unsigned)(len - start) + (C::TILE - 1u)) / C::TILE));
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
        ahead = runs ? lookup(0) : 0;
#pragma unroll
        for (int n = 0; n < NST - 1; ++n) fetch(n);
#pragma unroll
        for (int i = 0; i < C::QROWS; ++i) {
            const int r = warp + i * C::WARPS, rr = g.row0 + r;
            const uint16_t *src = p.q + (int64_t)g.b * p.qs[0] + (int64_t)(rr % p.n_q) * p.qs[1] +
                                  (int64_t)(g.hk * p.g + rr / p.n_q) * p.qs[2] + lane * 4;
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                qraw[i][h] = make_uint2(0, 0);
                if (r < g.rows) {
                    if (fp.q_aligned8) qraw[i][h] = __ldg(reinterpret_cast<const uint2 *>(src + h * 128));
                    else {
                        const uint16_t *x = src + h * 128;
                        qraw[i][h] = make_uint2(__ldg(x) | ((uint32_t)__ldg(x + 1) << 16),
                                                __ldg(x + 2) | ((uint32_t)__ldg(x + 3) << 16));
                    }
                }
            }
        }
    };
    // The next piece of this block at or after unit t: false when there is none.
    const auto piece_at = [&](Seg &g, uint32_t t, uint32_t &t0, uint32_t &t1) {
        t0 = max(t, g.first);
        t1 = min(t_end, g.first + g.tiles);
        return t0 < t1;
    };

    Seg g;
    uint32_t t0 = 0, t1 = 0;
    bool more = false;
    if (total > 0) {
        finder.find(t_begin, g);
        more = piece_at(g, t_begin, t0, t1);
        if (!more && g.first + g.tiles < t_end) {   // (only the price of a segment that ends before it)
            finder.next(g);
            more = piece_at(g, t_begin, t0, t1);
        }
        if (more) begin_piece(g, t0, t1);
    }
    // Sequences with nothing to attend still need their output rows zeroed.
    for (int c = 0; c * 32 < p.B; ++c) {
        if (c != finder.chunk) finder.load(c);
        unsigned empty = __ballot_sync(0xffffffffu, finder.n == 0 && c * 32 + lane < p.B);
        for (; empty; empty &= empty - 1) {
            const int b = c * 32 + __ffs(empty) - 1, Gz = total > 0 ? Gw : G;
            const int64_t s0 = (int64_t)b * p.Hkv;
            for (int hp = (int)(((int64_t)cta - s0 % Gz + Gz) % Gz); hp < p.Hkv; hp += Gz) {
                Seg z;
                z.b = b;
                z.hp = hp;
                finder.fill(z);
                const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                for (int e = tid; e < z.rows * (D / 8); e += kThreads)
                    store8(out_off(z, e / (D / 8)) + (e % (D / 8)) * 8, zero);
            }
        }
    }

    while (more) {
        // ---- Q: fp16 fragments and each row's factor, while K and V arrive
#pragma unroll
        for (int i = 0; i < C::QROWS; ++i) {
            const int r = warp + i * C::WARPS;
            if (r >= ROWS) break;
            float x[NH][4];
            float amax = 0.f;
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                x[h][0] = bf16lo(qraw[i][h].x); x[h][1] = bf16hi(qraw[i][h].x);
                x[h][2] = bf16lo(qraw[i][h].y); x[h][3] = bf16hi(qraw[i][h].y);
#pragma unroll
                for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fabsf(x[h][e]));
            }
            // (of non-negative numbers: their bits order as they do)
            amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
            // 2^e <= amax < 2^(e+1); e within what 2^-e and 2^e can hold
            int e = (int)((__float_as_uint(amax) >> 23) & 255u) - 127;
            e = amax > 0.f ? max(-126, min(126, e)) : 0;
            // a negative scale turns the query instead: the factors stay >= 0
            // (and above 0, so that -inf stays -inf when multiplied)
            const float down = copysignf(__uint_as_float((uint32_t)(127 - e) << 23), p.scale_log2);
            if (lane == 0)
                qmul[r] = fmaxf(fabsf(p.scale_log2) * __uint_as_float((uint32_t)(127 + e) << 23), 1.1754944e-38f);
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const uint2 f = make_uint2(pack_f16x2(x[h][0] * down, x[h][1] * down),
                                           pack_f16x2(x[h][2] * down, x[h][3] * down));
                // values 4*lane .. +3 of the half: owner lane t = lane / 8, k step lane % 8
                reinterpret_cast<uint2 *>(qfrag)[((((h * NT + (r >> 3)) * 4 + ((lane & 7) >> 1)) * 32 +
                                                   (r & 7) * 4 + (lane >> 3)) * 2) + (lane & 1)] = f;
            }
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
            const unsigned char *st = ring + (at_step % NST) * kStage;
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
            float mul[NT][2];    // rows 8*n + 2*t4 and the next: factor on q.k
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 x = NT == 1 ? mul1 : *reinterpret_cast<const float2 *>(qmul + n * 8 + 2 * t4);
                mul[n][0] = x.x;
                mul[n][1] = x.y;
            }
            float top[NT][2];
            bool grow = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    top[n][c] = fmaxf(fmaxf(S[0][n][c], S[0][n][c + 2]), fmaxf(S[1][n][c], S[1][n][c + 2]));
                    grow |= __fmaf_rn(top[n][c], mul[n][c], -mr[n][c]) > kGrow;
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
                        const float ref = fmaxf(mr[n][c], x * mul[n][c] - kBelow);
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
            uint32_t P[2][NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const float w0 = fast_exp2(__fmaf_rn(S[m][n][0], mul[n][0], -mr[n][0]));
                    const float w1 = fast_exp2(__fmaf_rn(S[m][n][1], mul[n][1], -mr[n][1]));
                    const float w2 = fast_exp2(__fmaf_rn(S[m][n][2], mul[n][0], -mr[n][0]));
                    const float w3 = fast_exp2(__fmaf_rn(S[m][n][3], mul[n][1], -mr[n][1]));
                    l[n][0] += w0 + w2;
                    l[n][1] += w1 + w3;
                    P[m][n][0] = transpose8x8(pack_f16x2(w0, w1));
                    P[m][n][1] = transpose8x8(pack_f16x2(w2, w3));
                }

            // ---- O^T += V^T P^T over this warp's 128 dimensions
#pragma unroll
            for (int m = 0; m < 2; ++m) {
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
                    }
                }
            }
            __syncwarp();   // the slot may be filled again
        }
        copy_wait<0>();

        // ---- the next piece sets out (the ring is this warp's own)
        const Seg now = g;
        const uint32_t n0 = t0, n1 = t1;
        more = t1 + p.seg_units < t_end;   // (t1 < t_end: the segment ended)
        if (more) {
            finder.next(g);
            more = piece_at(g, t1, t0, t1);
        }
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
        const int64_t s = (int64_t)now.b * p.Hkv + now.hp;
        const bool alone = n1 - n0 == now.tiles;
        float *slot = slot_ptr(p, s, cta);
        for (int e = tid; e < now.rows * (D / 8); e += kThreads) {
            const int r = e / (D / 8), col = (e % (D / 8)) * 8;
            float M = kNone, L = 0.f;
#pragma unroll
            for (int w = 0; w < STREAMS; ++w) M = fmaxf(M, wm[w * ROWS + r]);
#pragma unroll
            for (int w = 0; w < STREAMS; ++w) L += wl[w * ROWS + r] * fast_exp2(wm[w * ROWS + r] - M);
            float o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            const int at = (r & ~7) + (r & 1) * 4 + ((r & 7) >> 1);
#pragma unroll
            for (int w = 0; w < STREAMS; ++w) {
                const float4 *src = reinterpret_cast<const float4 *>(sums + (w * ROWS + at) * (D + 4) + col);
                const float4 a = src[0], b = src[1];
                o[0] += a.x; o[1] += a.y; o[2] += a.z; o[3] += a.w;
                o[4] += b.x; o[5] += b.y; o[6] += b.z; o[7] += b.w;
            }
            if (alone) {
                const float by = L > 0.f || L != L ? fp.v_global / L : 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] *= by;
                store8(out_off(now, r) + col, o);
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
        if (alone) continue;

        // ---- split segments: whoever finishes last joins the pieces; many of
        // them in two levels, groups of 8 and then the groups
        const int c_first = sp.owner(now.first), c_last = sp.owner((int64_t)now.first + now.tiles - 1);
        const int pieces = c_last - c_first + 1;
        const auto last_of = [&](int32_t *counter, int of) {
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                sh_last = atomicAdd(counter, 1) == of - 1;
                if (sh_last) *counter = 0;
            }
            __syncthreads();
            const bool yes = sh_last;
            if (yes) __threadfence();
            return yes;
        };
        // Joins pieces c0, c0 + step, .. (`count` of them) into the slot of
        // c0, or into the output.
        const auto join = [&](int c0, int step, int count, bool final) {
            // (row, 8 columns) items, and `ways` groups of threads that take
            // every ways-th piece each
            const int items = now.rows * (D / 8);
            const int ways = max(1, kThreads / items);
            for (int e0 = 0; e0 < items; e0 += kThreads) {
                const int way = items < kThreads ? tid / items : 0;
                const int e = items < kThreads ? tid - way * items : e0 + tid;
                const int r = e / (D / 8), col = (e % (D / 8)) * 8;
                float M = kNone, L = 0.f;
                float o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                if (way < ways && e < items) {
#pragma unroll 4
                    for (int k = way; k < count; k += ways) {
                        const float *sl = slot_ptr(p, s, c0 + k * step);
                        const float mv = __ldcg(sl + (int64_t)p.rows * D + r);
                        const float lv = __ldcg(sl + (int64_t)p.rows * D + p.rows + r);
                        const float4 a = __ldcg(reinterpret_cast<const float4 *>(sl + (int64_t)r * D + col));
                        const float4 b = __ldcg(reinterpret_cast<const float4 *>(sl + (int64_t)r * D + col + 4));
                        const float ref = fmaxf(M, mv);
                        const float u = fast_exp2(M - ref), w = fast_exp2(mv - ref);
                        M = ref;
                        L = L * u + w * lv;
                        const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = o[i] * u + w * x[i];
                    }
                }
                if (way > 0 && way < ways) {
                    float *dst = sums + ((way - 1) * items + e) * 10;   // [ways - 1][items][10]
                    dst[0] = M;
                    dst[1] = L;
#pragma unroll
                    for (int i = 0; i < 8; ++i) dst[2 + i] = o[i];
                }
                __syncthreads();
                if (way == 0 && e < items) {
                    for (int k = 0; k < ways - 1; ++k) {
                        const float *src = sums + (k * items + e) * 10;
                        const float ref = fmaxf(M, src[0]);
                        const float u = fast_exp2(M - ref), w = fast_exp2(src[0] - ref);
                        M = ref;
                        L = L * u + w * src[1];
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = o[i] * u + w * src[2 + i];
                    }
                    if (final) {
                        const float by = L > 0.f || L != L ? fp.v_global / L : 0.f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] *= by;
                        store8(out_off(now, r) + col, o);
                    } else {
                        float *sl = slot_ptr(p, s, c0);
                        float4 *dst = reinterpret_cast<float4 *>(sl + (int64_t)r * D + col);
                        dst[0] = make_float4(o[0], o[1], o[2], o[3]);
                        dst[1] = make_float4(o[4], o[5], o[6], o[7]);
                        if (col == 0) {
                            sl[(int64_t)p.rows * D + r] = M;
                            sl[(int64_t)p.rows * D + p.rows + r] = L;
                        }
                    }
                }
            }
        };
        if (pieces <= kOneJoin) {
            if (last_of(p.counters + s, pieces)) join(c_first, 1, pieces, true);
        } else {
            const int group = (cta - c_first) / kGroup8, lead = c_first + group * kGroup8;
            const int groups = (pieces + kGroup8 - 1) / kGroup8;
            const int size = min(kGroup8, pieces - group * kGroup8);
            if (last_of(fp.groups + (s + lead), size)) {
                if (size > 1) join(lead, 1, size, false);
                if (last_of(p.counters + s, groups)) join(c_first, kGroup8, groups, true);
            }
        }
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
    fp4_decode_kernel<NH, NT, PAGED><<<G, C::THREADS, C::SMEM, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

template <int NH, int NT>
int launch_layout(const Fp4Params &p, int G, cudaStream_t st) {
    return p.p.mode == kPaged ? launch<NH, NT, true>(p, G, st) : launch<NH, NT, false>(p, G, st);
}

}  // namespace

int fp4_max_rows(int) { return 32; }

int fp4_tile_tokens(int d, int rows) {
    static const int tile[4] = {Cfg<1, 1>::TILE, Cfg<1, 2>::TILE, Cfg<1, 3>::TILE, Cfg<1, 4>::TILE};
    return tile[(rows - 1) / 8] / (d / 128);   // pairs of warps at d = 256
}

int fp4_seg_units() { return 2; }

int fp4_blocks_per_sm(int rows) { return rows <= 16 ? Cfg<1, 1>::OCC : Cfg<1, 3>::OCC; }

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
        if (nt == 3) return launch_layout<2, 3>(p, G, st);
        if (nt == 4) return launch_layout<2, 4>(p, G, st);
    }
    return -2;
}

}  // namespace fd
