// fd_fp4_split.cuh -- what the decode kernel over a 4-bit cache is built on: the
// walk over the launch's work, copies into shared memory, and the end of a
// piece (stores, and joining the pieces of a split segment).
#pragma once

#include "fd_device.cuh"
#include "fd_fp4.cuh"
#include "fd_fp4_launch.h"

namespace fd {
namespace fp4 {

// The reference of a row is its running maximum less kBelow when it was last
// set; it is set again only when a weight would pass 2^kGrow, which keeps every
// weight within fp16 and spares most steps the shuffles and the rescaling.  fp32
// outputs keep their weights larger, so that small ones stay above fp16's least.
template <bool F32>
struct Reference {
    static constexpr float kBelow = F32 ? 12.f : 4.f, kGrow = F32 ? 15.f : 14.f;
    // Of a row whose largest score is x (in the log2 domain).  From 2^26 on
    // x - kBelow is rounded to a multiple of 8 or more; it lies at most 8 below x
    // where kBelow is 4, and is x itself where it would lie too far below.
    static __device__ __forceinline__ float of(float x) {
        const float ref = __fsub_rn(x, kBelow);
        return F32 && __fsub_rn(x, ref) > kGrow ? x : ref;
    }
};
// The reference of a row that has seen nothing yet.
constexpr float kNone = -3.402823466e38f;

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
    int hk, row0, rows;      // kv head; first row of the part, and its rows
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

// Work units that a block takes at least.  4 rows x 4 heads over 3,000 positions
// of a 256-wide cache: 19.3 us with 3, 18.9 with 4, 23.5 with 6; 4 x 2 heads
// over 1,000 of a 128-wide one: 9.5, 8.6, 8.8.
constexpr uint32_t kLeastUnits = 4;

// The range of work units of each of the launch's working blocks.
struct Share {
    uint32_t total, per, rest;
    int32_t blocks;          // working blocks
    // With few units a block takes at least kLeastUnits, which costs less than
    // more pieces to join.
    __device__ __forceinline__ Share(uint32_t units, int grid)
        : total(units), blocks(max(1, (int32_t)min((uint32_t)grid, units / kLeastUnits))) {
        per = units > 0 ? units / (uint32_t)blocks : 0;
        rest = units - per * (uint32_t)blocks;
    }
    // floor(c * total / blocks) in 32 bits: c and the remainder are below 2^16
    __device__ __forceinline__ uint32_t begin(int c) const {
        return (uint32_t)c * per + (uint32_t)c * rest / (uint32_t)blocks;
    }
    __device__ __forceinline__ int owner(uint32_t unit) const {
        return Split{(int64_t)total, blocks}.owner((int64_t)unit);
    }
};

// The part of segment g that lies in units [t, t_end): false when there is none.
__device__ __forceinline__ bool piece_at(const Seg &g, uint32_t t, uint32_t t_end, uint32_t &t0,
                                         uint32_t &t1) {
    t0 = max(t, g.first);
    t1 = min(t_end, g.first + g.tiles);
    return t0 < t1;
}

// The first piece of units [t, t_end).  (Where t lies in the price of a segment
// whose tiles another block has, the block has none: t_end is at most the first
// of them.)
template <int TILE>
__device__ __forceinline__ bool first_piece(Finder<TILE> &f, uint32_t t, uint32_t t_end, Seg &g,
                                            uint32_t &t0, uint32_t &t1) {
    f.find(t, g);
    return piece_at(g, t, t_end, t0, t1);
}

// The piece after [t0, t1) of g.
template <int TILE>
__device__ __forceinline__ bool next_piece(Finder<TILE> &f, const Params &p, uint32_t t_end, Seg &g,
                                           uint32_t &t0, uint32_t &t1) {
    if (t1 + p.seg_units >= t_end) return false;   // (t1 < t_end: the segment ended)
    f.next(g);
    return piece_at(g, t1, t_end, t0, t1);
}

// Element offset of query row r of a segment in q or the output.
__device__ __forceinline__ int64_t row_at(const Params &p, const Seg &g, int r, const int64_t *strides) {
    r += g.row0;
    return (int64_t)g.b * strides[0] + (int64_t)(r % p.n_q) * strides[1] +
           (int64_t)(g.hk * p.g + r / p.n_q) * strides[2];
}

// Eight consecutive output values at element `off`.
__device__ __forceinline__ void put8(const Params &p, int64_t off, const float *o) {
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
}

// Output rows of the sequences with nothing to attend, spread over the blocks.
template <int D, int TILE>
__device__ __forceinline__ void zero_empty(const Params &p, Finder<TILE> &f, int block, int blocks,
                                           int tid, int threads) {
    const int lane = threadIdx.x & 31;
    for (int c = 0; c * 32 < p.B; ++c) {
        if (c != f.chunk) f.load(c);
        unsigned empty = __ballot_sync(0xffffffffu, f.n == 0 && c * 32 + lane < p.B);
        for (; empty; empty &= empty - 1) {
            Seg g;
            g.b = c * 32 + __ffs(empty) - 1;
            const int64_t s0 = (int64_t)g.b * p.Hkv;
            for (g.hp = (int)(((int64_t)block - s0 % blocks + blocks) % blocks); g.hp < p.Hkv; g.hp += blocks) {
                f.fill(g);
                const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                for (int e = tid; e < g.rows * (D / 8); e += threads)
                    put8(p, row_at(p, g, e / (D / 8), p.os) + (e % (D / 8)) * 8, zero);
            }
        }
    }
}

// 2^-reference-scaled sums become the output: v_global / L, or 0 for a row
// that saw nothing.
__device__ __forceinline__ float out_factor(const Fp4Params &fp, float L) {
    return L > 0.f || L != L ? fp.v_global / L : 0.f;
}

// Adds up a block's streams, each with its own reference: sums [STREAMS][ROWS]
// [D + 4] already scaled to the common reference (row r at (r & ~7) + (r & 1) *
// 4 + (r & 7) / 2), their references wm and weight sums wl [STREAMS][ROWS]; into
// the output where the segment is this block's alone, else into its slot.
template <int D, int ROWS, int STREAMS, int THREADS>
__device__ __forceinline__ void add_streams(const Fp4Params &fp, const Seg &g, bool alone, int cta,
                                            const float *sums, const float *wm, const float *wl) {
    const Params &p = fp.p;
    float *slot = slot_ptr(p, (int64_t)g.b * p.Hkv + g.hp, cta);
    for (int e = threadIdx.x; e < g.rows * (D / 8); e += THREADS) {
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
            const float by = out_factor(fp, L);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] *= by;
            put8(p, row_at(p, g, r, p.os) + col, o);
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
}

// The query rows of a segment as a warp loads them: lane l holds values 4l ..
// 4l + 3 of each 128.
template <int NH>
__device__ __forceinline__ void load_query(const Fp4Params &fp, const Seg &g, int r, uint2 *q) {
    const int lane = threadIdx.x & 31;
    const uint16_t *src = fp.p.q + row_at(fp.p, g, r, fp.p.qs) + lane * 4;
#pragma unroll
    for (int h = 0; h < NH; ++h) {
        q[h] = make_uint2(0, 0);
        if (r < g.rows) {
            const uint16_t *x = src + h * 128;
            if (fp.q_aligned8) q[h] = __ldg(reinterpret_cast<const uint2 *>(x));
            else q[h] = make_uint2(__ldg(x) | ((uint32_t)__ldg(x + 1) << 16),
                                   __ldg(x + 2) | ((uint32_t)__ldg(x + 3) << 16));
        }
    }
}

// Scales a loaded row by a power of two so that its largest entry lies in [1,
// 2), and turns it into fp16 pairs.  Returns the factor on q.k: its sign is in
// the row, so it is >= 0, and it is above 0, so that -inf stays -inf when
// multiplied.
template <int NH>
__device__ __forceinline__ float scale_query(const Params &p, uint2 *q) {
    float x[NH][4];
    float amax = 0.f;
#pragma unroll
    for (int h = 0; h < NH; ++h) {
        x[h][0] = bf16lo(q[h].x); x[h][1] = bf16hi(q[h].x);
        x[h][2] = bf16lo(q[h].y); x[h][3] = bf16hi(q[h].y);
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fabsf(x[h][e]));
    }
    // (of non-negative numbers: their bits order as they do)
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    // 2^e <= amax < 2^(e+1); e within what 2^-e and 2^e can hold
    int e = (int)((__float_as_uint(amax) >> 23) & 255u) - 127;
    e = amax > 0.f ? max(-126, min(126, e)) : 0;
    const float down = copysignf(__uint_as_float((uint32_t)(127 - e) << 23), p.scale_log2);
#pragma unroll
    for (int h = 0; h < NH; ++h)
        q[h] = make_uint2(pack_f16x2(x[h][0] * down, x[h][1] * down), pack_f16x2(x[h][2] * down, x[h][3] * down));
    return fmaxf(fabsf(p.scale_log2) * __uint_as_float((uint32_t)(127 + e) << 23), 1.1754944e-38f);
}

// Pieces of a segment are joined in groups of 8 where a thread of a single join
// would walk over more than kOneJoin of them.  24 rows at d = 256, 32,768
// positions (38 pieces, one way): 40 us in groups, 48 at once.  4 rows at d =
// 128 (four ways, 9 or 10 pieces each): 17.7 in groups, 15.1 at once.  16 at d =
// 256 over 3,000 positions: 21.8 in groups, 18.1 at once.
constexpr int kGroup8 = 8, kOneJoin = 12;

// The end of a piece of a split segment whose partial result is in this
// block's slot: whoever finishes last joins the pieces; many of them in two
// levels, groups of 8 and then the groups.  Called by `THREADS` threads, tid
// 0 .. THREADS - 1, that `sync` brings together; room: shared memory, 10 *
// THREADS floats; flag: one shared int.
template <int D, int THREADS, typename Sync>
__device__ __forceinline__ void join_pieces(const Fp4Params &fp, const Share &share, const Seg &g, int cta,
                                            int tid, float *room, int *flag, Sync sync) {
    const Params &p = fp.p;
    const int64_t s = (int64_t)g.b * p.Hkv + g.hp;
    const int c_first = share.owner(g.first), c_last = share.owner(g.first + g.tiles - 1);
    const int pieces = c_last - c_first + 1;
    const auto last_of = [&](int32_t *counter, int of) {
        __threadfence();
        sync();
        if (tid == 0) {
            *flag = atomicAdd(counter, 1) == of - 1;
            if (*flag) *counter = 0;
        }
        sync();
        const bool yes = *flag;
        if (yes) __threadfence();
        return yes;
    };
    // (row, 8 columns) items, and `ways` groups of threads that take every
    // ways-th piece each
    const int items = g.rows * (D / 8), ways = max(1, THREADS / items);
    // Joins pieces c0, c0 + step, .. (`count` of them) into the slot of c0, or
    // into the output.
    const auto join = [&](int c0, int step, int count, bool final) {
        for (int e0 = 0; e0 < items; e0 += THREADS) {
            const int way = items < THREADS ? tid / items : 0;
            const int e = items < THREADS ? tid - way * items : e0 + tid;
            const int r = e / (D / 8), col = (e % (D / 8)) * 8;
            float M = kNone, L = 0.f;
            float o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (way < ways && e < items) {
#pragma unroll 8
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
                float *dst = room + ((way - 1) * items + e) * 10;   // [ways - 1][items][10]
                dst[0] = M;
                dst[1] = L;
#pragma unroll
                for (int i = 0; i < 8; ++i) dst[2 + i] = o[i];
            }
            sync();
            if (way == 0 && e < items) {
                for (int k = 0; k < ways - 1; ++k) {
                    const float *src = room + (k * items + e) * 10;
                    const float ref = fmaxf(M, src[0]);
                    const float u = fast_exp2(M - ref), w = fast_exp2(src[0] - ref);
                    M = ref;
                    L = L * u + w * src[1];
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = o[i] * u + w * src[2 + i];
                }
                if (final) {
                    const float by = out_factor(fp, L);
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] *= by;
                    put8(p, row_at(p, g, r, p.os) + col, o);
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
    if (pieces <= kOneJoin * ways) {
        if (last_of(p.counters + s, pieces)) join(c_first, 1, pieces, true);
        return;
    }
    const int group = (cta - c_first) / kGroup8, lead = c_first + group * kGroup8;
    const int groups = (pieces + kGroup8 - 1) / kGroup8;
    const int size = min(kGroup8, pieces - group * kGroup8);
    if (last_of(fp.groups + (s + lead), size)) {
        if (size > 1) join(lead, 1, size, false);
        if (last_of(p.counters + s, groups)) join(c_first, kGroup8, groups, true);
    }
}

}  // namespace fp4
}  // namespace fd
