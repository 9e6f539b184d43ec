// fd_prefill_tc.cu -- attention of a chunk of new tokens over a cache on the
// tensor cores (tcgen05, TMEM accumulators, TMA loads).
//
// Rows.  The query heads of a kv head share its K and V, so a tile holds T =
// 128 / g tokens of all g heads: row r is token r / g, head r % g.  A segment is
// one tile, or two where a chunk has more rows than one holds (head_dim 128):
// each position's K and V then serve 256 rows.
//
// Work.  Segments (sequence, kv head, tiles) follow one another in units of 128
// positions: a charge for its start and end, then its blocks of positions (a
// bound on them that sums in closed form).  The grid's blocks, one an SM, take
// equal consecutive shares of the units.  A segment that is cut leaves partial sums
// in the workspace, which a second launch, set out ahead, joins in the order of the
// pieces.
//
// Roles in a block:
//   warps 8, 11  TMA producers: Q of a segment, then K and V tiles of 128 positions
//            in halves of 128 dimensions, into a ring of shared-memory slots.  Each
//            brings 64 of the 128 dimensions: small pages take a copy for each run
//            of rows, and a warp sets out one in some 100 cycles.
//   warps 9, 10  MMA issuers (one thread each): S = Q K^T (128 x 128) into TMEM,
//            O += P V with P from TMEM.  Two tiles: one issuer a tile; one tile: one
//            for the scores, one for P V.  The queue of issued MMAs is short, and
//            what a thread does between them (barriers, commits: half the time with
//            one issuer) leaves the tensor pipe idle unless the other's are there.
//   warps 0-7  softmax: a thread owns a row (two tiles: of its group's tile) or
//            half the columns of one (one tile, S then double buffered).  P
//            overwrites S in TMEM in bf16.  A row's reference is its running
//            maximum, refreshed, and O rescaled, only where a score passes it
//            by 2^8.
// K and V of most paged calls do not come by TMA: warps 8-11 copy them by cp.async.
// int8 caches: codes are copied by TMA into the second half of their slot, and
// warps 8-11 widen them in place to bf16 (exactly); the position's K scale
// multiplies its scores, its V scale its weights.  In both the producer is warp 12,
// the issuers 13 and 14.
//
// Weights are rounded to bf16, the output's own type, over either cache: the sum of their
// errors is then like the output's rounding (0.0024 off 64 bits in all, 0.0017 with exact
// weights).  Over int8 caches finer ones were tried: two bf16 numbers a weight, twice the
// products on V, take the int8 chunks below from 250 to 328 us; one fp16 number, V's codes in
// fp16 and references that follow the V scales too, 274 us, and what is less than some 2^-31
// of the largest is lost, where bf16 keeps eight bits of it.
//
// Bounds and times (us; 32 heads of 8 at head_dim 128, rates of a 6,787 GB/s copy and a
// 1,906 TFLOP/s product):
//   2,048 tokens behind 30,720, pages of 64: 780, 1.4 PFLOP/s (floor 559).  Softmax and
//     the matrix pipe take turns of a similar length; some of each shows.
//   4 x 5 .. 16 tokens about 30,000 .. 65,536 positions: 148, 5.9 TB/s (floor 129): the
//     memory; ends and the join take 15.
//   8 prompts of 500 .. 4,096 tokens, 16 heads of 4, head_dim 256: 430, 1.1 PFLOP/s (floor
//     254).  O fills half of TMEM, so one tile is held; its scores, softmax and products
//     wait for one another, and two blocks in flight do not cover that (the matrix pipe is
//     busy half of the time, and its operands fill what shared memory passes).
//   4 x 200 .. 512 tokens behind up to 8,000 int8 positions: 239, 0.58 PFLOP/s (floor 73):
//     widening the codes and the scales of every score and weight.
//   37 tokens behind 963, 8 heads of 2: 16.5: two launches of dependent steps.
// Code is kept small: the roles' instructions together pass what the caches hold, and a
// third less of them took prompts at d 256 from 640 to 503 us.
#include <cuda_runtime.h>

#include <cstring>
#include <type_traits>

#include "fd_api.h"
#include "fd_device.cuh"
#include "fd_packed.cuh"
#include "fd_prefill.h"
#include "fd_ptx.cuh"
#include "fd_tensor_map.h"

namespace fd {

namespace {

constexpr int TT = 128;
constexpr int kDevTimeout = 4;          // mirrors FD_DEV_INTERNAL
constexpr uint64_t kDrainNs = 2000000000ull;
constexpr float kSlack = 8.f;           // log2: how far a score may pass the reference
constexpr unsigned kAll = 0xffffffffu;

struct PfArgs {
    CUtensorMap tq, tk, tv;   // tk, tv: boxes of prow rows (flat: 128)
    CUtensorMap gk, gv;       // paged: single rows, gathered four at a time
    PrefillParams p;
    int32_t T, R;             // tokens and rows a tile
    int32_t prow;             // rows a box; 0: every tile is gathered
    int64_t gs[3];            // pool row of (page, kv head, row) in gk, gv
    float *slots;             // partial sums, two a block
};

struct Bars {
    uint64_t slot_full[8], slot_empty[8], raw_full[8];   // raw: int8 codes
    uint64_t q_full[2], q_free[2], s_full[2], p_full[2], o_full[2];
    uint64_t cross, pv_done[2], drain[2];
    uint32_t tmem_base;
    int abort_flag;          // the site of the first wait that ran out, else 0
    int turn;                // held by the issuer whose tile's MMAs go out
    uint32_t armed[2];       // two producers: slots that each has set out, at its end
};

// How K and V come: whole slots by TMA; int8 codes by TMA, widened; by cp.async.
enum Load { kTma, kCodes, kCopies };

template <int D, bool TWO, int LOAD>
struct Cfg {
    static constexpr bool I8 = LOAD == kCodes, MORE = LOAD != kTma;   // MORE: a warpgroup that widens or copies
    static_assert(!TWO || D == 128, "two tiles' O and S fill TMEM at head_dim 128");
    // Warpgroups of softmax (two), of widening or copying, and of the producers and
    // issuers; softmax takes registers that the others give up.
    static constexpr int THREADS = MORE ? 512 : 384;
    static constexpr int LAUNCH_REGS = MORE ? 128 : 168, SOFTMAX_REGS = MORE ? 184 : 200, MORE_REGS = MORE ? 72 : 0,
                         OTHER_REGS = MORE ? 72 : 104;
    static_assert(256 * SOFTMAX_REGS + 128 * (MORE_REGS + OTHER_REGS) <= THREADS * LAUNCH_REGS, "registers of the launch");
    static constexpr int PRODUCER = MORE ? 12 : 8, PRODUCER2 = MORE ? -1 : 11, ISSUER = PRODUCER + 1;   // warps; issuers: two
    // One tile by TMA is of a flat cache (copied()).
    static constexpr bool PAGED = MORE || TWO;
    static constexpr int NH = D / 128, QT = TWO ? 2 : 1;
    static constexpr uint32_t BOX = TT * 128;        // 128 rows x 64 numbers
    static constexpr uint32_t SLOT = 2 * BOX;        // 128 rows x 128 numbers
    static constexpr uint32_t QTILE = NH * SLOT;
    static constexpr uint32_t OFF_RED = 512;         // [2][2][128] floats
    static constexpr uint32_t OFF_BAD = OFF_RED + 2048;   // [8][8] words
    static constexpr uint32_t OFF_SCALES = OFF_BAD + 256;   // int8: [8][2][128] floats
    static constexpr uint32_t OFF_Q = (OFF_SCALES + (I8 ? 8192 : 0) + 1023) / 1024 * 1024;
    static constexpr uint32_t BUDGET = 232448;
    static constexpr int NS = (int)((BUDGET - OFF_Q - QT * QTILE) / SLOT);
    static_assert(NS >= 4 && NS <= 8, "ring");
    static constexpr uint32_t OFF_SLOTS = OFF_Q + QT * QTILE;
    static constexpr uint32_t SMEM = OFF_SLOTS + NS * SLOT;
    static constexpr int NC = TWO ? 128 : 64;        // score columns a softmax thread
    static constexpr int OC = TWO ? D : D / 2;       // output columns a softmax thread
    static constexpr uint32_t TMEM_O = 256;          // S: columns 0 .. 255
    static constexpr int ROWS = QT * TT;             // rows a partial slot
    static constexpr int64_t SLOT_FLOATS = (int64_t)ROWS * (D + 2);
    static constexpr uint32_t IDESC_QK = ptx::idesc_bf16(128, 128, 0, 0);
    static constexpr uint32_t IDESC_PV = ptx::idesc_bf16(128, 128, 0, 1);
};
static_assert(sizeof(Bars) <= 512, "barrier block");

// ------------------------------------------------------------------ work
// Blocks of positions that a segment's start and end are charged as (prompts at d 256
// with 1, 2, 3, 4, 6: 520, 494, 478, 482, 496 us).
constexpr int kCharge = 3;

// Blocks that hold x positions (lengths go up to 2^31 - 1: sums with them are unsigned).
__device__ __forceinline__ int blocks_of(int x) { return (int)(((unsigned)x + TT - 1) / TT); }

// What a launch's share of the work goes by: B sequences of L_b positions, fresh_b
// of them new.
struct Seq {
    int L, fresh, nq;        // nq: segments a kv head
    __device__ __forceinline__ int base() const { return L - fresh; }
};

__device__ __forceinline__ Seq seq_of(const PrefillParams &p, int b, int S, bool flag = false) {
    const int cap = (int)p.c.cap, raw = __ldg(p.lengths + b), L = max(0, min(raw, cap));
    const int want = p.new_lengths ? __ldg(p.new_lengths + b) : p.n, fresh = max(0, min(want, p.n));
    if (flag && (raw != L || want != fresh)) atomicOr(p.status, kDevBadLength);
    return Seq{L, fresh, (fresh + S - 1) / S};
}

// Units of a segment, and of the first q of a kv head.  Causal segments see the
// positions before the chunk and (q + 1) S new ones, in at most ceil((q + 1) /
// per) blocks, per = 128 / S whole segments a block (S = 256: 2 (q + 1) blocks).
__device__ __forceinline__ int cost_of(const PrefillParams &p, const Seq &s, int S, int q) {
    if (!p.causal) return kCharge + blocks_of(s.L);
    const int per = p.per;
    return kCharge + blocks_of(max(s.base(), 0)) + (S > TT ? 2 * (q + 1) : (q + per) / per);
}
__device__ __forceinline__ int units_of(const PrefillParams &p, const Seq &s, int S, int q) {
    if (!p.causal) return q * (kCharge + blocks_of(s.L));
    const int before = q * (kCharge + blocks_of(max(s.base(), 0)));
    if (S > TT) return before + q * (q + 1);
    const int per = p.per, m = q / per;
    return before + per * (m * (m + 1) / 2) + (q - m * per) * (m + 1);
}

// All units (below 2^31), and the blocks that share them: the first `rest` take
// one more.
struct Total {
    int units, each, G, rest;
    int first;               // units of this lane's first sequence, of one kv head
    __device__ __forceinline__ int start(int c) const { return c * each + min(c, rest); }
    __device__ __forceinline__ int owner(int u) const {
        const int more = rest * (each + 1);
        return u < more ? u / (each + 1) : rest + (u - more) / each;
    }
};

// Every lane of a warp.
__device__ __forceinline__ Total total_of(const PrefillParams &p, int S, int grid, bool flag) {
    Total t;
    t.first = 0;
    int sum = 0;
#pragma unroll 1
    for (int i = threadIdx.x & 31; i < p.B; i += 32) {
        const Seq x = seq_of(p, i, S, flag);
        const int mine = units_of(p, x, S, x.nq);
        if (i < 32) t.first = mine;
        sum += mine;
    }
    t.units = __reduce_add_sync(kAll, sum) * p.c.Hkv;
    t.G = max(1, min(t.units, grid));
    t.each = t.units / t.G;
    t.rest = t.units - t.each * t.G;
    return t;
}

// A walk over the segments of a share: the current one, and where the share starts
// and ends, in blocks of it.
struct Walk {
    int from, to;
    Seq s;
    int b, hk, q;

    // The segment that holds unit u0 of a share [u0, u1); every lane of a warp.
    __device__ __forceinline__ void seek(const PrefillParams &p, int S, const Total &t, int u0, int u1) {
        const int lane = threadIdx.x & 31;
        int before = 0, mine = t.first * p.c.Hkv;
#pragma unroll 1
        for (int b0 = 0;; b0 += 32) {
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kAll, upto, o);
                if (lane >= o) upto += y;
            }
            const unsigned in = __ballot_sync(kAll, before + upto > u0);
            if (in) {
                const int at = __ffs(in) - 1;
                int x = u0 - before - __shfl_sync(kAll, upto - mine, at);
                b = b0 + at;
                s = seq_of(p, b, S);
                const int head = units_of(p, s, S, s.nq);
                hk = x / head;
                x -= hk * head;
                if (p.causal) {
                    // about S / 256 q^2 + k q = x
                    const float k = (float)cost_of(p, s, S, 0), w = S * (1.f / 128);
                    q = max(0, min((int)((sqrtf(k * k + 2.f * w * (float)x) - k) / w), s.nq - 1));
                    while (q > 0 && units_of(p, s, S, q) > x) --q;
                    while (q + 1 < s.nq && units_of(p, s, S, q + 1) <= x) ++q;
                } else {
                    q = x / cost_of(p, s, S, 0);
                }
                from = x - units_of(p, s, S, q) - kCharge;
                to = from + (u1 - u0);
                return;
            }
            before += __shfl_sync(kAll, upto, 31);
            const int i = b0 + 32 + lane;
            mine = 0;
            if (i < p.B) {
                const Seq x = seq_of(p, i, S);
                mine = units_of(p, x, S, x.nq) * p.c.Hkv;
            }
        }
    }
    __device__ __forceinline__ bool next(const PrefillParams &p, int S) {
        const int cost = cost_of(p, s, S, q);
        from -= cost;
        to -= cost;
        if (to + kCharge <= 0) return false;
        if (++q == s.nq) {
            q = 0;
            if (++hk == p.c.Hkv) {
                hk = 0;
                do {
                    if (++b >= p.B) return false;
                    s = seq_of(p, b, S);
                } while (s.nq == 0);
            }
        }
        return true;
    }
    // Positions that the first `tokens` of this segment see.
    __device__ __forceinline__ int seen(const PrefillParams &p, int S, int tokens) const {
        if (!p.causal) return s.L;
        return max(0, min(s.L, s.base() + min(s.fresh, q * S + tokens)));
    }
    __device__ __forceinline__ int blocks(const PrefillParams &p, int S) const { return blocks_of(seen(p, S, S)); }
};

// The blocks of positions of the current segment that are this share's, and of
// them those that each tile sees.
struct Piece {
    int j0, j1, all;         // of `all`
    int hi[2];               // tile t works on j0 .. hi[t] - 1
    __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == all; }
};

template <int QT>
__device__ __forceinline__ Piece piece_of(const PfArgs &a, const Walk &w) {
    const PrefillParams &p = a.p;
    const int S = QT * a.T;
    Piece x;
    x.all = w.blocks(p, S);
    x.j0 = max(0, min(x.all, w.from));
    x.j1 = max(0, min(x.all, w.to));
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        x.hi[t] = x.j0;
        if (t < QT && w.q * S + t * a.T < w.s.fresh)
            x.hi[t] = max(x.j0, min(x.j1, blocks_of(w.seen(p, S, (t + 1) * a.T))));
    }
    return x;
}

// ----------------------------------------------------------------- helpers
// A wait within the launch's limit, counted in rounds of a microsecond's suspension
// (no clock, no call: some thirty places wait, and instruction caches are
// small).  One that runs out stops the block's others, and its site is reported
// when the block ends.
__device__ __forceinline__ bool wait_on(Bars *bs, const PrefillParams &p, uint64_t *bar, uint32_t parity, int site) {
    volatile int *abort = &bs->abort_flag;
    for (int n = p.wait_rounds; !ptx::mbar_try_wait_for(bar, parity & 1, 1000); --n) {
        if (n == 0) *abort = site;
        if (*abort) return false;
    }
    return true;
}

// The same for a whole warp, which goes on or gives up as one: what follows (votes,
// loads from TMEM) wants all of its lanes.
__device__ __forceinline__ bool warp_wait_on(Bars *bs, const PrefillParams &p, uint64_t *bar, uint32_t parity, int site) {
    return __all_sync(kAll, wait_on(bs, p, bar, parity, site));
}

// Waits for a block's own copies or MMAs, which must end even when another role
// gave up; until kDrainNs after t0.
__device__ __forceinline__ void drain_on(uint64_t *bar, uint32_t parity, uint64_t t0) {
    for (uint32_t n = 1; !ptx::mbar_try_wait(bar, parity); ++n)
        if ((n & 63) == 0 && ptx::globaltimer_ns() - t0 > kDrainNs) return;
}

// The issuers' turn, taken (the other holds it for a microsecond or so; a thousand
// tries of some 100 cycles a round) and given back.
__device__ __forceinline__ bool take_turn(Bars *bs, const PrefillParams &p) {
    volatile int *abort = &bs->abort_flag;
    for (int64_t n = 1000 * (int64_t)p.wait_rounds; atomicCAS(&bs->turn, 0, 1) != 0; --n) {
        if (n == 0) *abort = 12;
        if (*abort) return false;
    }
    return true;
}
__device__ __forceinline__ void give_turn(Bars *bs) { atomicExch(&bs->turn, 0); }

__device__ __forceinline__ void store32(void *dst, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Row `row` of tile t of the current segment: its token, where it is stored.
template <int QT>
__device__ __forceinline__ bool row_at(const PfArgs &a, const Walk &w, int t, int row, int &token, int64_t &off) {
    const PrefillParams &p = a.p;
    token = (w.q * QT + t) * a.T + row / p.g;
    off = w.b * p.os[0] + token * p.os[1] + ((int64_t)w.hk * p.g + row % p.g) * p.os[2];
    return row < a.R && token < w.s.fresh;
}

// ---------------------------------------------------------------- widening

// One warp of the widening warpgroup: its 32 rows of every fill, in place.  A thread
// takes 16 of a row's 128 codes, of every fourth row, all of them into registers
// before the warp writes; it also brings the scales of position tid of each block,
// which are loaded a block before they are wanted.
template <int D, bool TWO>
__device__ __forceinline__ void widen_role(const PfArgs &a, Bars *bs, unsigned char *smem, Walk w, bool has) {
    using C = Cfg<D, TWO, kCodes>;
    const PrefillParams &p = a.p;
    const int tid = (int)threadIdx.x - 256, S = C::QT * a.T;
    const int chunk = tid & 7, row0 = (tid & ~31) + ((tid & 31) >> 3);   // rows row0 + 4 e
    uint32_t fills = 0, seen = 0;
    bool ok = true;
    for (bool more = has; more && ok; more = w.next(p, S)) {
        const Piece x = piece_of<C::QT>(a, w);
        const int n = x.j1 - x.j0;
        if (n <= 0) continue;
        // what column tid of block i of the piece stands for: its page, and its scales
        const auto position = [&](int i) {
            const int pos0 = (x.j0 + i) * TT;
            return (p.c.block_table ? pos0 : min(pos0, w.s.L - TT)) + tid;
        };
        const auto lead_of = [&](int i) {
            if (i >= n) return -1;
            const int pos = position(i);
            if (pos < 0 || pos >= w.s.L) return -1;
            if (!p.c.block_table) return w.b;
            const int e = __ldg(p.c.block_table + (int64_t)w.b * p.c.max_pages +
                                (p.c.page_shift >= 0 ? pos >> p.c.page_shift : pos / p.c.page_size));
            return e < p.c.lead ? e : -1;
        };
        float k_scale = 0.f, v_scale = 0.f;
        const auto bring = [&](int i, int lead) {
            k_scale = v_scale = 0.f;
            if (lead < 0) return;
            const int pos = position(i);
            const int64_t row = !p.c.block_table ? pos : p.c.page_shift >= 0 ? pos & (p.c.page_size - 1) : pos % p.c.page_size;
            k_scale = __ldg(p.c.k_scale + lead * p.c.kss[0] + w.hk * p.c.kss[1] + row * p.c.kss[2]);
            v_scale = __ldg(p.c.v_scale + lead * p.c.vss[0] + w.hk * p.c.vss[1] + row * p.c.vss[2]);
        };
        bring(0, lead_of(0));
        int lead = lead_of(1);
        // fills: K(0), K(1), V(0), K(2), V(1) .. V(n - 1), NH halves each; two tiles:
        // K(0), V(0), K(1), V(1) ..
        int i = 0;                                             // the next block of K
        for (int g = 0; g < 2 * n && ok; ++g) {
            const bool k = TWO ? (g & 1) == 0 : g == 0 || ((g & 1) == 1 && g != 2 * n - 1);
            if (k) {
                float *to = reinterpret_cast<float *>(smem + C::OFF_SCALES + ((seen + i) & 7) * 1024);
                to[tid] = k_scale;
                to[128 + tid] = v_scale;
                ++i;
                bring(i, lead);
                lead = lead_of(i + 1);
            }
            for (int h = 0; h < C::NH; ++h) {
                const uint32_t slot = fills % C::NS, use = fills / C::NS;
                ok = warp_wait_on(bs, p, &bs->raw_full[slot], use, 11);
                if (!ok) break;
                ++fills;
                unsigned char *const box = smem + C::OFF_SLOTS + slot * C::SLOT;
                uint4 codes[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int r = row0 + 4 * e;
                    codes[e] = *reinterpret_cast<const uint4 *>(box + C::BOX + r * 128 + ((chunk ^ (r & 7)) * 16));
                }
                __syncwarp();
                unsigned char *const dst = box + (chunk >> 2) * C::BOX;
                const int c0 = (chunk & 3) * 2;
                // (lanes of the other box take the other chunk first: no bank twice)
                const int turn = chunk >> 2;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int r = row0 + 4 * e;
                    const uint2 q0 = widen4(codes[e].x), q1 = widen4(codes[e].y), q2 = widen4(codes[e].z), q3 = widen4(codes[e].w);
                    const uint4 first = make_uint4(q0.x, q0.y, q1.x, q1.y), second = make_uint4(q2.x, q2.y, q3.x, q3.y);
                    *reinterpret_cast<uint4 *>(dst + r * 128 + (((c0 + turn) ^ (r & 7)) * 16)) = turn ? second : first;
                    *reinterpret_cast<uint4 *>(dst + r * 128 + (((c0 + 1 - turn) ^ (r & 7)) * 16)) = turn ? first : second;
                }
                ptx::fence_proxy_async_smem();
                ptx::mbar_arrive(&bs->slot_full[slot]);
            }
        }
        seen += n;
    }
}

// ----------------------------------------------------------------- copying
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// One warp of the copying warpgroup: its 32 rows of every fill, zeros where there is
// none, in the slots' 128-byte swizzle.  Two fills are on their way while a third
// sets out; one that has come is fenced and announced.
template <int D, bool TWO>
__device__ __forceinline__ void copy_role(const PfArgs &a, Bars *bs, unsigned char *smem, Walk w, bool has) {
    using C = Cfg<D, TWO, kCopies>;
    const PrefillParams &p = a.p;
    const int tid = (int)threadIdx.x - 256, lane = tid & 31, S = C::QT * a.T;
    // in a round the warp copies two rows: 16 lanes take a row's 16 chunks
    const int chunk = lane & 15, row0 = (tid & ~31) + (lane >> 4);       // rows row0 + 2 e
    const uint32_t slots = ptx::smem_u32(smem) + C::OFF_SLOTS + (chunk >> 3) * C::BOX + row0 * 128;
    const uint16_t *const bases[2] = {static_cast<const uint16_t *>(p.c.k), static_cast<const uint16_t *>(p.c.v)};
    uint32_t fills = 0, told = 0, seen = 0;
    bool ok = true;
    const auto tell = [&]() {
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(&bs->slot_full[told % C::NS]);
        ++told;
    };
    const auto tell_all = [&]() {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        while (told < fills) tell();
    };
    for (bool more = has; more && ok; more = w.next(p, S)) {
        const Piece x = piece_of<C::QT>(a, w);
        const int n = x.j1 - x.j0;
        if (n <= 0) continue;
        const int32_t *table = p.c.block_table + (int64_t)w.b * p.c.max_pages;
        // position tid of block i: its table entry, and where its row lies (elements)
        const auto entry_of = [&](int i) {
            if (i >= n) return -1;
            const int pos = (x.j0 + i) * TT + tid;
            return pos < w.s.L ? __ldg(table + (p.c.page_shift >= 0 ? pos >> p.c.page_shift : pos / p.c.page_size)) : -1;
        };
        int entry = entry_of(0);
        int64_t k_row = -1, v_row = -1, v_next = -1;
        const auto look = [&](int i) {
            const int pos = (x.j0 + i) * TT + tid;
            const int row = p.c.page_shift >= 0 ? pos & (p.c.page_size - 1) : pos % p.c.page_size;
            const bool there = entry >= 0 && entry < p.c.lead, hole = pos < w.s.L && !there;
            if (hole) atomicOr(p.status, kDevBadIndex);
            k_row = there ? entry * p.c.ks[0] + w.hk * p.c.ks[1] + row * p.c.ks[2] : -1;
            v_row = v_next;
            v_next = there ? entry * p.c.vs[0] + w.hk * p.c.vs[1] + row * p.c.vs[2] : -1;
            entry = entry_of(i + 1);
            const unsigned word = __ballot_sync(kAll, hole);
            if (lane == 0) reinterpret_cast<uint32_t *>(smem + C::OFF_BAD)[((seen + i) & 7) * 8 + 1 + (tid >> 5)] = word;
        };
        // fills: K(0), K(1), V(0), K(2), V(1) .. V(n - 1), NH halves each; two tiles:
        // K(0), V(0), K(1), V(1) ..
        int i = 0;                                             // the next block of K
#pragma unroll 1
        for (int g = 0; g < 2 * n && ok; ++g) {
            const bool k = TWO ? (g & 1) == 0 : g == 0 || ((g & 1) == 1 && g != 2 * n - 1);
            if (k) look(i++);
            // (V of the block before the last of K, or of the last where no K follows)
            const int64_t mine = k ? k_row : TWO || g == 2 * n - 1 ? v_next : v_row;
#pragma unroll 1
            for (int h = 0; h < C::NH; ++h) {
                const uint32_t slot = fills % C::NS, use = fills / C::NS;
                if (!ptx::mbar_try_wait(&bs->slot_empty[slot], (use + 1) & 1)) {
                    tell_all();      // what has been copied may be what is waited for
                    ok = wait_on(bs, p, &bs->slot_empty[slot], use + 1, 2);
                }
                ok = __all_sync(kAll, ok);
                if (!ok) break;
                const uint32_t dst = slots + slot * C::SLOT;
                const uint16_t *src = bases[k ? 0 : 1] + h * 128 + chunk * 8;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int64_t row = __shfl_sync(kAll, mine, 2 * e + (lane >> 4));
                    copy16(dst + e * 256 + (((chunk & 7) ^ ((row0 + 2 * e) & 7)) * 16), src + (row < 0 ? 0 : row), row >= 0);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                ++fills;
                if (fills - told > 2) {
                    asm volatile("cp.async.wait_group 2;" ::: "memory");
                    tell();
                }
            }
        }
        seen += n;
    }
    tell_all();
}

// ------------------------------------------------------------------ kernel
template <int D, bool TWO, int LOAD>
__global__ void __launch_bounds__(Cfg<D, TWO, LOAD>::THREADS, 1) prefill_tc_kernel(const __grid_constant__ PfArgs a) {
    using C = Cfg<D, TWO, LOAD>;
    constexpr bool I8 = C::I8;
    const PrefillParams &p = a.p;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t base = ptx::smem_u32(smem);
    Bars *bs = reinterpret_cast<Bars *>(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;");   // (the join waits for this kernel's end)
    if (base & 1023u) {   // the swizzled layouts want aligned buffers
        if (tid == 0) atomicOr(p.status, kDevTimeout);
        return;
    }
    if (warp == C::PRODUCER && lane == 0) {
        ptx::prefetch_tmap(&a.tq);
        ptx::prefetch_tmap(&a.tk);
        ptx::prefetch_tmap(&a.tv);
        for (int i = 0; i < C::NS; ++i) {
            ptx::mbar_init(&bs->slot_full[i], C::MORE ? 128 : 2);
            ptx::mbar_init(&bs->raw_full[i], 1);
            ptx::mbar_init(&bs->slot_empty[i], C::QT);   // two tiles: by both issuers
        }
        for (int t = 0; t < 2; ++t) {
            ptx::mbar_init(&bs->q_full[t], 1);
            ptx::mbar_init(&bs->q_free[t], 1);
            ptx::mbar_init(&bs->s_full[t], 1);
            ptx::mbar_init(&bs->p_full[t], TWO ? 128 : 256);
            ptx::mbar_init(&bs->o_full[t], 1);
            ptx::mbar_init(&bs->pv_done[t], 1);
            ptx::mbar_init(&bs->drain[t], 1);
        }
        ptx::mbar_init(&bs->cross, 256);
        bs->abort_flag = 0;
        bs->turn = 0;
        ptx::mbar_fence_init();
    }
    if (warp == C::ISSUER) {
        ptx::tmem_alloc(&bs->tmem_base, 512);
        ptx::tmem_relinquish();
    }
    const int S = C::QT * a.T;           // tokens a segment
    Walk w;
    bool has;
    {
        const Total total = total_of(p, S, gridDim.x, warp == C::PRODUCER && blockIdx.x == 0);
        has = (int)blockIdx.x < total.G && total.units > 0;
        if (has) w.seek(p, S, total, total.start(blockIdx.x), total.start(blockIdx.x + 1));
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = bs->tmem_base;

    if (C::MORE && warp >= 8 && warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::MORE ? C::MORE_REGS : 24));
        if constexpr (LOAD == kCodes) widen_role<D, TWO>(a, bs, smem, w, has);
        if constexpr (LOAD == kCopies) copy_role<D, TWO>(a, bs, smem, w, has);
    } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
    if (warp == C::PRODUCER || warp == C::PRODUCER2) {
        // ------------------------------------------------------ producers
        const int part = warp == C::PRODUCER ? 0 : 1;
        uint32_t fills = 0, loads[2] = {0, 0}, seen = 0;   // seen: blocks of positions
        bool ok = true;
        // rows of a block of positions: a box's page and first row, or the
        // pool's rows of positions 4 lane .. 4 lane + 3
        struct Rows {
            int y[4];
        };
        const bool paged = C::PAGED && p.c.block_table;
        for (bool more = has; more && ok; more = w.next(p, S)) {
            const Piece x = piece_of<C::QT>(a, w);
            if (x.j0 >= x.j1) continue;
#pragma unroll
            for (int t = 0; t < C::QT; ++t) {
                if (part || x.hi[t] <= x.j0 || !ok) continue;
                if (lane == 0) {
                    if (loads[t] > 0) ok = wait_on(bs, p, &bs->q_free[t], loads[t] - 1, 1);
                    if (ok) {
                        ++loads[t];
                        ptx::mbar_arrive_expect_tx(&bs->q_full[t], (uint32_t)(a.R * 128 * (D / 64)));
                        for (int cb = 0; cb < D / 64; ++cb)
                            ptx::tma_load_4d(smem + C::OFF_Q + t * C::QTILE + cb * C::BOX, &a.tq, &bs->q_full[t], cb * 64,
                                             w.hk * p.g, w.q * S + t * a.T, w.b);
                    }
                }
                ok = __shfl_sync(kAll, ok, 0);
            }
            if (LOAD == kCopies) continue;      // (Q only)
            const auto tiled = [&](int j) { return !paged || (a.prow > 0 && (int64_t)(j + 1) * TT <= w.s.L); };
            // entries of the runs of the next blocks, one a lane: a load's latency in
            // every block held the copies up (2,048 tokens at d 256 over pages of 128:
            // 2,095 -> 1,975 us)
            int window = 0, window_end = -1, entry = -1;
            const auto look = [&](int j) {
                Rows r{{-1, -1, -1, -1}};
                if (!paged || j >= x.j1) return r;
                const int32_t *table = p.c.block_table + (int64_t)w.b * p.c.max_pages;
                const bool box = tiled(j);
                // (the window's last runs may lie past 2^31)
                const unsigned pos = (unsigned)(j * TT) + lane * (box ? a.prow : 4), page_size = p.c.page_size;
                int i = (int)(p.c.page_shift >= 0 ? pos >> p.c.page_shift : pos / page_size), row = (int)(pos - i * page_size);
                if (box) {
                    const int runs = TT / a.prow;
                    if (j >= window_end) {
                        window = j;
                        window_end = j + 32 / runs;
                        entry = pos < (unsigned)w.s.L ? __ldg(table + i) : -1;
                    }
                    const int page = __shfl_sync(kAll, entry, ((j - window) * runs + lane) & 31);
                    if (lane >= runs) return r;
                    r.y[0] = page < p.c.lead ? page : -1;
                    r.y[1] = row;
                    return r;
                }
                // four positions, on one page or more
                int page[4], at[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    at[e] = row;
                    page[e] = pos + e < (unsigned)w.s.L ? __ldg(table + i) : -1;
                    if (++row == p.c.page_size) {
                        row = 0;
                        ++i;
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (page[e] >= 0 && page[e] < p.c.lead) r.y[e] = (int)(page[e] * a.gs[0] + w.hk * a.gs[1] + at[e] * a.gs[2]);
                return r;
            };
            // one half of K or V of block j
            const auto fill = [&](int j, int h, bool v, const Rows &r) {
                const uint32_t slot = fills % C::NS, use = fills / C::NS;
                uint64_t *const full = I8 ? &bs->raw_full[slot] : &bs->slot_full[slot];
                if (lane == 0) {
                    ok = wait_on(bs, p, &bs->slot_empty[slot], use + 1, 2);
                    if (ok) ptx::mbar_arrive_expect_tx(full, C::BOX);
                }
                ok = __shfl_sync(kAll, ok, 0);
                if (!ok) return;
                ++fills;
                // (codes as pairs, into the second half)
                unsigned char *dst = smem + C::OFF_SLOTS + slot * C::SLOT + (I8 ? 1 : part) * C::BOX;
                const int dim = I8 ? h * 64 : h * 128 + part * 64;
                if (!paged) {
                    const int y = min(j * TT, w.s.L - TT);   // the last tile ends at the length
                    if (lane == 0) ptx::tma_load_4d(dst, v ? &a.tv : &a.tk, full, dim, y, w.hk, w.b);
                } else if (tiled(j)) {
                    if (lane < TT / a.prow)
                        ptx::tma_load_4d(dst + lane * a.prow * 128, v ? &a.tv : &a.tk, full, dim, r.y[1],
                                         w.hk, r.y[0]);
                } else {
                    ptx::tma_gather4(dst + 4 * lane * 128, v ? &a.gv : &a.gk, full, dim, r.y[0], r.y[1],
                                     r.y[2], r.y[3]);
                }
            };
            // which of the block's positions lie on a page that the table does
            // not name, for the softmax
            const auto mark = [&](int j, const Rows &r) {
                if (!paged || part) return;
                uint32_t *ring = reinterpret_cast<uint32_t *>(smem + C::OFF_BAD) + ((seen + j - x.j0) & 7) * 8;
                uint32_t bad = 0;   // of positions 4 lane .. 4 lane + 3
                if (tiled(j)) {
                    const unsigned runs = __ballot_sync(kAll, lane < TT / a.prow && r.y[0] < 0);
                    if (runs)
#pragma unroll
                        for (int e = 0; e < 4; ++e) bad |= ((runs >> ((4 * lane + e) / a.prow)) & 1u) << e;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if ((int64_t)j * TT + 4 * lane + e < w.s.L && r.y[e] < 0) bad |= 1u << e;
                }
                const bool any = __any_sync(kAll, bad != 0);
                if (any) {
                    if (bad) atomicOr(p.status, kDevBadIndex);
                    uint32_t word = bad << (4 * (lane & 7));
#pragma unroll
                    for (int o = 1; o < 8; o <<= 1) word |= __shfl_xor_sync(kAll, word, o);
                    if ((lane & 7) == 0) ring[1 + lane / 8] = word;
                }
                __syncwarp();
                if (lane == 0) ring[0] = any;
                __syncwarp();
            };
            // K(0), K(1), V(0), K(2), V(1) .. V(n - 1); two tiles: K(0), V(0), K(1), ..
            const int n = x.j1 - x.j0;
            Rows of_v{{-1, -1, -1, -1}}, of_k = look(x.j0), then = of_v;
            int kb = 0, vb = 0;
#pragma unroll 1
            for (int f = 0; f < 2 * n && ok; ++f) {
                const bool v = TWO ? (f & 1) : f == 2 * n - 1 || (f > 0 && (f & 1) == 0);
                const int j = x.j0 + (v ? vb : kb);
                if (!v) mark(j, of_k);
#pragma unroll 1
                for (int h = 0; h < C::NH && ok; ++h) fill(j, h, v, v ? of_v : of_k);
                if (!v) {
                    const Rows r = look(j + 1);
                    if (TWO || f == 0) {
                        of_v = of_k;
                        of_k = r;
                    } else {
                        then = r;
                    }
                    ++kb;
                } else {
                    if (!TWO) {
                        of_v = of_k;
                        of_k = then;
                    }
                    ++vb;
                }
            }
            seen += x.j1 - x.j0;
        }
        // every copy that was issued lands before the block exits.  Two producers: one
        // that gave up may be up to a ring behind; it arrives, without bytes, for the
        // slots that the other has set out, whose phases would not end otherwise
        if (C::PRODUCER2 >= 0) {
            if (lane == 0) bs->armed[part] = fills;
            __syncwarp();
            asm volatile("barrier.sync 1, 64;" ::: "memory");
            const uint32_t most = max(fills, bs->armed[part ^ 1]);
            for (; fills < most; ++fills)
                if (lane == 0) ptx::mbar_arrive(&bs->slot_full[fills % C::NS]);
        }
        if (lane == 0) {
            const uint64_t t0 = ptx::globaltimer_ns();
            for (uint32_t i = fills > C::NS ? fills - C::NS : 0; i < fills; ++i)
                drain_on(I8 ? &bs->raw_full[i % C::NS] : &bs->slot_full[i % C::NS], (i / C::NS) & 1, t0);
            for (int t = 0; t < C::QT; ++t)
                if (loads[t] > 0) drain_on(&bs->q_full[t], (loads[t] - 1) & 1, t0);
        }
    } else if (warp == C::ISSUER || warp == C::ISSUER + 1) {
        // --------------------------------------------------------- issuers
        if (lane == 0) {
            const int me = warp - C::ISSUER;
            bool ok = true;
            uint32_t filled = 0;             // slots of the pieces before
            uint32_t pieces = 0, ctr = 0;
            const auto slot_at = [&](uint32_t i) { return base + C::OFF_SLOTS + (i % C::NS) * C::SLOT; };
            const auto wait_slot = [&](uint32_t i) {
                ok = ok && wait_on(bs, p, &bs->slot_full[i % C::NS], i / C::NS, 3);
            };
            const auto free_slot = [&](uint32_t i) { ptx::mma_commit(&bs->slot_empty[i % C::NS]); };
            // S[buf] (+)= Q_t K^T over one half of the dimensions
            const auto qk = [&](int t, uint32_t buf, uint32_t i, int h) {
                const uint64_t q = ptx::smem_desc(base + C::OFF_Q + t * C::QTILE + h * C::SLOT, 16, 1024, ptx::kLayoutSwizzle128);
                const uint64_t k = ptx::smem_desc(slot_at(i), 16, 1024, ptx::kLayoutSwizzle128);
                ptx::tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint64_t at = ((kk >> 2) * C::BOX + (kk & 3) * 32) >> 4;
                    ptx::mma_f16_ss(tmem + buf * 128, q + at, k + at, C::IDESC_QK, h > 0 || kk > 0);
                }
            };
            // O_t's dimensions of half h += P[buf] V
            const auto pv = [&](int t, uint32_t buf, uint32_t i, int h, bool first) {
                const uint64_t v = ptx::smem_desc(slot_at(i), C::BOX, 1024, ptx::kLayoutSwizzle128);
                ptx::tc_fence_after();
#pragma unroll
                for (int kt = 0; kt < 8; ++kt)
                    ptx::mma_f16_ts(tmem + C::TMEM_O + t * 128 + h * 128, tmem + buf * 128 + kt * 8, v + ((kt * 2048) >> 4),
                                    C::IDESC_PV, !(first && kt == 0));
            };
            for (bool more = has; more && ok; more = w.next(p, S)) {
                const Piece x = piece_of<C::QT>(a, w);
                const int n = x.j1 - x.j0;
                if (n <= 0) continue;
                if (TWO) {
                    // tile `me`: scores of the next block follow P V of the last,
                    // which reads P where they go; fills K(0) V(0) K(1) V(1) ..
                    const int mine = x.hi[me] - x.j0;
                    if (mine > 0) ok = wait_on(bs, p, &bs->q_full[me], pieces++, 4);
                    const auto pass = [&](uint32_t i) {   // a slot that this tile has no use for
                        wait_slot(i);
                        if (ok) ptx::mbar_arrive(&bs->slot_empty[i % C::NS]);
                    };
                    const auto scores = [&](int i) {
                        const uint32_t k = filled + 2 * i;
                        qk(me, me, k, 0);
                        ptx::mma_commit(&bs->s_full[me]);
                        free_slot(k);
                        if (i + 1 == mine) ptx::mma_commit(&bs->q_free[me]);
                    };
                    if (ok && mine > 0) {
                        wait_slot(filled);
                        if (ok) scores(0);
                    } else if (ok) {
                        pass(filled);
                    }
                    for (int i = 0; i < n && ok; ++i) {
                        const uint32_t v = filled + 2 * i + 1;
                        if (i >= mine) {
                            pass(v);
                            if (ok && i + 1 < n) pass(v + 1);
                            continue;
                        }
                        wait_slot(v);
                        if (i + 1 < mine) wait_slot(v + 1);
                        ok = ok && wait_on(bs, p, &bs->p_full[me], ctr++, 5);
                        // one tile's MMAs go out together: mixed with the other's,
                        // both tiles' softmax would wait for both (883 us of 32 heads
                        // x 2,048 rows x 32,768 positions became 952)
                        ok = ok && take_turn(bs, p);
                        if (!ok) break;
                        pv(me, me, v, 0, i == 0);
                        free_slot(v);
                        if (i + 1 == mine) ptx::mma_commit(&bs->o_full[me]);
                        else scores(i + 1);
                        give_turn(bs);
                        if (i + 1 == mine && i + 1 < n) pass(v + 1);
                    }
                    filled += 2 * n;
                } else if (me == 0) {
                    // scores; fills K(0) K(1) V(0) K(2) V(1) .. V(n - 1).  A slot's
                    // parity tells its next fill from its last only once the last
                    // one has come.  Each issuer takes half of the fills; what it
                    // waits for first (P V two blocks back; P of its own block)
                    // puts the others', up to a ring's length before, behind it.
                    ok = wait_on(bs, p, &bs->q_full[0], pieces++, 4);
                    for (int i = 0; i < n && ok; ++i, ++ctr) {
                        // P of two blocks before, which lies there, has been used
                        if (ctr >= 2) ok = wait_on(bs, p, &bs->pv_done[ctr & 1], (ctr >> 1) - 1, 10);
#pragma unroll
                        for (int h = 0; h < C::NH && ok; ++h) {
                            const uint32_t k = filled + (i == 0 ? 0 : 2 * i - 1) * C::NH + h;
                            wait_slot(k);
                            if (!ok) break;
                            qk(0, ctr & 1, k, h);
                            if (h == C::NH - 1) ptx::mma_commit(&bs->s_full[ctr & 1]);
                            free_slot(k);
                        }
                    }
                    if (ok) ptx::mma_commit(&bs->q_free[0]);
                    filled += 2 * n * C::NH;
                } else {
                    for (int i = 0; i < n && ok; ++i, ++ctr) {
                        const uint32_t v0 = filled + (i == n - 1 ? 2 * n - 1 : 2 * i + 2) * C::NH;
                        ok = wait_on(bs, p, &bs->p_full[ctr & 1], ctr >> 1, 5);
#pragma unroll
                        for (int h = 0; h < C::NH && ok; ++h) {
                            wait_slot(v0 + h);
                            if (!ok) break;
                            pv(0, ctr & 1, v0 + h, h, i == 0);
                            if (h == C::NH - 1) ptx::mma_commit(&bs->pv_done[ctr & 1]);
                            free_slot(v0 + h);
                        }
                        if (ok && i == n - 1) ptx::mma_commit(&bs->o_full[0]);
                    }
                    filled += 2 * n * C::NH;
                }
            }
            // every MMA that was issued ends before the block exits
            ptx::mma_commit(&bs->drain[me]);
            drain_on(&bs->drain[me], 0, ptx::globaltimer_ns());
        }
    }
    } else {
        // --------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SOFTMAX_REGS));
        const int group = warp >> 2, row = (warp & 3) * 32 + lane;
        const int t = TWO ? group : 0;                  // tile
        const int col0 = TWO ? 0 : group * 64;          // first score column
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // TMEM lane of the warp, << 16
        const uint32_t o_at = tmem + lanes + C::TMEM_O + (TWO ? t * 128 : group * C::OC);
        float *red = reinterpret_cast<float *>(smem + C::OFF_RED);
        uint32_t ctr = 0, pieces = 0, crossed = 0, seen = 0;
        bool ok = true;
        // one tile: this thread's number against that of the row's other half
        const auto other = [&](float mine) {
            float *room = red + (crossed & 1) * 256;
            room[group * 128 + row] = mine;
            ptx::tc_fence_before();
            ptx::mbar_arrive(&bs->cross);
            ok = ok && warp_wait_on(bs, p, &bs->cross, crossed, 6);
            ptx::tc_fence_after();
            ++crossed;
            return room[(group ^ 1) * 128 + row];
        };
        const float sc = p.scale_log2;
        for (bool more = has; more && ok; more = w.next(p, S)) {
            const Piece x = piece_of<C::QT>(a, w);
            int token;
            int64_t off;
            const bool real = row_at<C::QT>(a, w, t, row, token, off);
            if (x.all == 0) {
                // nobody sees anything: the block of the segment's first unit
                if (w.from + kCharge <= 0 && real)
                    for (int c = 0; c < C::OC; c += 8)
                        *reinterpret_cast<uint4 *>(p.out + off + (TWO ? 0 : group * C::OC) + c) = make_uint4(0, 0, 0, 0);
                continue;
            }
            if (x.j0 >= x.j1) continue;
            const int n = x.hi[t] - x.j0;
            const int first = w.q * S + t * a.T;            // the tile's first token
            const int last = p.causal ? min(w.s.base() + min(token, w.s.fresh), w.s.L - 1) : w.s.L - 1;
            const int all_see = p.causal ? min(w.s.base() + min(first, w.s.fresh), w.s.L - 1) : w.s.L - 1;
            float m = neg_inf(), l = 0.f;
            uint64_t sum0 = 0, sum1 = 0;
            // one block of positions, whose hidden scores are -inf already where some row
            // does not see all of it (masked; int8: the others scaled)
            const auto block = [&](int j, uint32_t buf, bool masked) {
                const uint32_t s_at = tmem + lanes + buf * 128;
                const auto most = [&](const float *s, float top) {
                    float t0 = fmaxf(s[0], s[1]), t1 = fmaxf(s[2], s[3]);
#pragma unroll
                    for (int e = 4; e < 32; e += 4) {
                        t0 = fmaxf(t0, fmaxf(s[e], s[e + 1]));
                        t1 = fmaxf(t1, fmaxf(s[e + 2], s[e + 3]));
                    }
                    return fmaxf(top, fmaxf(t0, t1));
                };
                // int8: the scores of 32 columns from c on, times their scales of K
                const ulonglong2 *scales = reinterpret_cast<const ulonglong2 *>(smem + C::OFF_SCALES + ((seen + j - x.j0) & 7) * 1024 + col0 * 4);
                const auto scale = [&](float *s, int c) {
                    if (!I8 || masked) return;
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const ulonglong2 k = scales[(c + e) / 4];
                        const float2 u = unpair(mul2(pair(s[e], s[e + 1]), k.x)), v = unpair(mul2(pair(s[e + 2], s[e + 3]), k.y));
                        s[e] = u.x;
                        s[e + 1] = u.y;
                        s[e + 2] = v.x;
                        s[e + 3] = v.y;
                    }
                };
                // the row's maximum; columns 0 .. 63 stay in registers, 64 .. 127 are
                // read again below (both loops stay loops: a block of 128 columns
                // unrolled came from memory more often than from the instruction cache)
                float s[64], h[32];
                float top = neg_inf();
#pragma unroll (I8 ? 1 : 2)
                for (int c = C::NC - 64; c >= 0; c -= 64) {
                    ptx::tmem_ld32(s_at + col0 + c, s);
                    ptx::tmem_ld32(s_at + col0 + c + 32, s + 32);
                    ptx::tmem_wait_ld();
                    scale(s, c);
                    scale(s + 32, c + 32);
                    top = most(s, most(s + 32, top));
                }
                if (!TWO) top = fmaxf(top, other(top));
                if (!ok) return;
                // a new reference where a score passes the old one by 2^8
                // (rows that are nobody's hold what was left in shared memory)
                const bool raise = real && ((top - m) * sc > kSlack || m == neg_inf());
                if (__any_sync(kAll, raise)) {
                    float f = 1.f;
                    if (raise) {
                        f = m == neg_inf() ? 0.f : fast_exp2((m - top) * sc);
                        m = top;
                        const float2 u = unpair(sum0), v = unpair(sum1);
                        sum0 = pair(u.x * f, u.y * f);
                        sum1 = pair(v.x * f, v.y * f);
                    }
                    if (j > x.j0) {
                        // two tiles: the last PV into O was issued before these
                        // scores, whose end was waited for; one tile: after
                        if (!TWO) {
                            ok = warp_wait_on(bs, p, &bs->pv_done[ctr & 1], (ctr - 2) >> 1, 9);
                            if (!ok) return;
                            ptx::tc_fence_after();
                        }
#pragma unroll 1
                        for (int c = 0; c < C::OC; c += 32) {
                            ptx::tmem_ld32(o_at + c, h);
                            ptx::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) h[e] *= f;
                            ptx::tmem_st16(o_at + c, h);
                            ptx::tmem_st16(o_at + c + 16, h + 16);
                        }
                    }
                }
                const float ref = m == neg_inf() ? 0.f : -m * sc;
                const uint64_t sc2 = pair(sc, sc), ref2 = pair(ref, ref);
                // the weights of 32 columns from c on, into P
                const auto weigh = [&](const float *s, int c) {
                    uint32_t word[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float2 u = unpair(fma2(pair(s[e], s[e + 1]), sc2, ref2));
                        const float2 v = unpair(fma2(pair(s[e + 2], s[e + 3]), sc2, ref2));
                        const float p0 = fast_exp2(u.x), p1 = fast_exp2(u.y), p2 = fast_exp2(v.x), p3 = fast_exp2(v.y);
                        sum0 = add2(sum0, pair(p0, p1));
                        sum1 = add2(sum1, pair(p2, p3));
                        if (I8) {
                            // (the scale of a position that is hidden may be a NaN)
                            const ulonglong2 y = scales[32 + (c + e) / 4];
                            float2 f = unpair(mul2(pair(p0, p1), y.x)), g = unpair(mul2(pair(p2, p3), y.y));
                            if (masked) {
                                f.x = s[e] == neg_inf() ? 0.f : f.x;
                                f.y = s[e + 1] == neg_inf() ? 0.f : f.y;
                                g.x = s[e + 2] == neg_inf() ? 0.f : g.x;
                                g.y = s[e + 3] == neg_inf() ? 0.f : g.y;
                            }
                            word[e / 2] = pack_bf16x2(f.x, f.y);
                            word[e / 2 + 1] = pack_bf16x2(g.x, g.y);
                        } else {
                            word[e / 2] = pack_bf16x2(p0, p1);
                            word[e / 2 + 1] = pack_bf16x2(p2, p3);
                        }
                    }
                    ptx::tmem_st16(s_at + (col0 + c) / 2, word);
                };
#pragma unroll (I8 ? 1 : 2)
                for (int c = 0; c < C::NC; c += 64) {
                    const bool more = c + 64 < C::NC;
                    weigh(s, c);
                    if (more) ptx::tmem_ld32(s_at + 64, s);
                    weigh(s + 32, c + 32);
                    if (more) {
                        ptx::tmem_ld32(s_at + 96, s + 32);
                        ptx::tmem_wait_ld();
                        scale(s, 64);
                        scale(s + 32, 96);
                    }
                }
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                ptx::mbar_arrive(&bs->p_full[buf]);
            };
            const int plain = (all_see + 1) / TT;      // blocks that every row sees whole
            for (int j = x.j0; j < x.hi[t] && ok; ++j) {
                const uint32_t buf = TWO ? t : ctr & 1, use = TWO ? ctr : ctr >> 1;
                ++ctr;
                ok = warp_wait_on(bs, p, &bs->s_full[buf], use, 7);
                if (!ok) break;
                ptx::tc_fence_after();
                const volatile uint32_t *bad = reinterpret_cast<const volatile uint32_t *>(smem + C::OFF_BAD) + ((seen + j - x.j0) & 7) * 8;
                const bool holes = C::PAGED && p.c.block_table && (LOAD == kCopies ? bad[1] | bad[2] | bad[3] | bad[4] : bad[0]) != 0;
                const bool masked = j >= plain || holes;
                if (masked) {
                    // in place first: blocks that a row does not see whole are few, and
                    // a second loop body would crowd the instruction caches
                    const uint32_t s_at = tmem + lanes + buf * 128 + col0;
                    const int pos0 = j * TT;
                    const int at = C::PAGED && p.c.block_table ? pos0 : min(pos0, w.s.L - TT);   // position of column 0
#pragma unroll 1
                    for (int c = 0; c < C::NC; c += 32) {
                        float s[32];
                        ptx::tmem_ld32(s_at + c, s);
                        // of these columns the row sees lo .. hi - 1, less those on no page
                        const int lo = min(max(pos0 - at - col0 - c, 0), 32), hi = min(max(last + 1 - at - col0 - c, 0), 32);
                        uint32_t sees = hi > lo ? (0xffffffffu >> (32 - (hi - lo))) << lo : 0u;
                        if (holes) sees &= ~bad[1 + (col0 + c) / 32];
                        ptx::tmem_wait_ld();
                        if (I8) {
                            const float *k = reinterpret_cast<const float *>(smem + C::OFF_SCALES + ((seen + j - x.j0) & 7) * 1024) + col0 + c;
#pragma unroll
                            for (int e = 0; e < 32; ++e) s[e] *= k[e];
                        }
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!((sees >> e) & 1u)) s[e] = neg_inf();
                        ptx::tmem_st16(s_at + c, s);
                        ptx::tmem_st16(s_at + c + 16, s + 16);
                    }
                    ptx::tmem_wait_st();
                }
                block(j, buf, masked);
            }
            if (!ok) break;
            seen += x.j1 - x.j0;
            {
                const float2 u = unpair(sum0), v = unpair(sum1);
                l = (u.x + u.y) + (v.x + v.y);
            }
            if (!TWO) l += other(l);
            if (!ok) break;
            if (n > 0) {
                ok = warp_wait_on(bs, p, &bs->o_full[t], pieces++, 8);
                if (!ok) break;
                ptx::tc_fence_after();
            }
            const int c0 = TWO ? 0 : group * C::OC;
            if (x.whole()) {
                const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
                // four neighbours trade their rows' runs of eight columns, so that they
                // store 64 bytes of one row at a time (a row each, 32 bytes at a time, made a
                // segment's end 7,000 cycles at d 256; 6,300 so)
                uint16_t *at[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t where = reinterpret_cast<uint64_t>(real ? p.out + off + c0 : nullptr);
                    const uint64_t theirs = __shfl_sync(kAll, where, (lane & ~3) + e);
                    at[e] = theirs ? reinterpret_cast<uint16_t *>(theirs) + (lane & 3) * 8 : nullptr;
                }
#pragma unroll 1
                for (int c = 0; c < C::OC; c += 32) {
                    float o[32];
                    uint32_t word[16];
                    if (n > 0) {
                        ptx::tmem_ld32(o_at + c, o);
                        ptx::tmem_wait_ld();
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        word[e] = n > 0 && inv != 0.f ? pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv) : 0u;
#pragma unroll
                    for (int by = 1; by < 4; by *= 2)
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            if (e & (4 * by)) continue;
                            uint32_t &lo = word[e], &hi = word[e + 4 * by];
                            const uint32_t got = __shfl_xor_sync(kAll, lane & by ? lo : hi, by);
                            (lane & by ? lo : hi) = got;
                        }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (at[e])
                            *reinterpret_cast<uint4 *>(at[e] + c) =
                                make_uint4(word[4 * e], word[4 * e + 1], word[4 * e + 2], word[4 * e + 3]);
                }
            } else {
                float *slot = a.slots + (2 * (int64_t)blockIdx.x + (x.j0 > 0 ? 0 : 1)) * C::SLOT_FLOATS;
                const int r = t * TT + row;
                if (real && (TWO || group == 0)) {
                    slot[C::ROWS * D + r] = n > 0 && m != neg_inf() ? m * sc : neg_inf();
                    slot[C::ROWS * (D + 1) + r] = l;
                }
                if (n > 0) {
                    // eight columns of every row, then the next eight: a warp's stores
                    // are one run
                    float *dst = slot + c0 * C::ROWS + r * 8;
#pragma unroll 1
                    for (int c = 0; c < C::OC; c += 32) {
                        float o[32];
                        ptx::tmem_ld32(o_at + c, o);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            if (real) store32(dst + (c + e) * C::ROWS, reinterpret_cast<const uint32_t *>(o + e));
                    }
                }
            }
            // (the next segment's PV overwrites O once this group's P is there)
            ptx::tc_fence_before();
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (tid == 0 && bs->abort_flag) {
        // (the launch's first is recorded, as in the decode kernel)
        atomicOr(p.status, kDevTimeout);
        atomicCAS(p.status + 1, 0, bs->abort_flag);
    }
    if (warp == C::ISSUER) ptx::tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------- join
// blockIdx.x: a place between two blocks' shares.  If it cuts a segment's blocks
// of positions, this place's part of the segment's rows (of kJoinParts) is
// joined from the pieces, in order.
constexpr int kJoinParts = 4, kJoinThreads = 256, kJoinAhead = 4;

template <int D, bool TWO>
__global__ void __launch_bounds__(kJoinThreads) prefill_join_kernel(const __grid_constant__ PfArgs a, int grid) {
    using C = Cfg<D, TWO, kTma>;
    const PrefillParams &p = a.p;
    const int c = blockIdx.x + 1;
    const int S = C::QT * a.T;
    const Total total = total_of(p, S, grid, false);
    int first = 0, last = 0;
    Walk w;
    if (c < total.G && total.units > 0) {
        const int u = total.start(c);
        w.seek(p, S, total, u, u);
        const int all = w.blocks(p, S), block0 = u - w.from;   // unit of the first block
        if (all > 0) {
            first = total.owner(block0);
            last = total.owner(block0 + all - 1);
        }
    }
    // (every thread: the launch behind this one may count on the pieces' kernel)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (c <= first || c > last) return;
    const int parts = (last - first) * kJoinParts, at = (c - first - 1) * kJoinParts + (int)blockIdx.y;
    const int r0 = C::ROWS * at / parts, r1 = C::ROWS * (at + 1) / parts;
    constexpr int PER = D / 8;
    // a warp: eight rows of four runs of eight columns
    for (int e = threadIdx.x; e < (r1 - r0 + 7) / 8 * 8 * PER; e += kJoinThreads) {
        const int r = r0 + e / (8 * PER) * 8 + (e & 7), d = (e >> 3) % PER * 8;
        int token;
        int64_t off;
        if (r >= r1 || !row_at<C::QT>(a, w, r / TT, r % TT, token, off)) continue;
        float top = neg_inf(), l = 0.f, o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int k0 = first; k0 <= last; k0 += kJoinAhead) {
            float m[kJoinAhead] = {}, more[kJoinAhead] = {};
            float4 y[kJoinAhead][2] = {};
#pragma unroll
            for (int i = 0; i < kJoinAhead; ++i) {
                // the first piece is its block's second slot, the others their first
                const int k = k0 + i;
                if (k > last) continue;
                const float *s = a.slots + (2 * (int64_t)k + (k == first)) * C::SLOT_FLOATS;
                m[i] = s[C::ROWS * D + r];
                more[i] = s[C::ROWS * (D + 1) + r];
                y[i][0] = *reinterpret_cast<const float4 *>(s + d * C::ROWS + r * 8);
                y[i][1] = *reinterpret_cast<const float4 *>(s + d * C::ROWS + r * 8 + 4);
            }
#pragma unroll
            for (int i = 0; i < kJoinAhead; ++i) {
                // (a piece that saw nothing for the row holds no O; one whose scores
                // were all NaN has a sum that is, and no maximum)
                const bool any = k0 + i <= last && (m[i] != neg_inf() || more[i] != more[i]);
                const float now = any ? fmaxf(top, m[i]) : top, f = now == neg_inf() ? 0.f : fast_exp2(top - now);
                const float g = any ? fast_exp2(m[i] - now) : 0.f;
                const float x[8] = {y[i][0].x, y[i][0].y, y[i][0].z, y[i][0].w, y[i][1].x, y[i][1].y, y[i][1].z, y[i][1].w};
                top = now;
                l = l * f + (any ? more[i] * g : 0.f);
#pragma unroll
                for (int z = 0; z < 8; ++z) o[z] = o[z] * f + (any ? x[z] * g : 0.f);
            }
        }
        const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
        *reinterpret_cast<uint4 *>(p.out + off + d) =
            make_uint4(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv),
                       pack_bf16x2(o[4] * inv, o[5] * inv), pack_bf16x2(o[6] * inv, o[7] * inv));
    }
}

// ------------------------------------------------------------- host side
// bf16 numbers, or pairs of int8 codes.
bool encode(CUtensorMap *m, cuuint32_t rank, const void *base, const cuuint64_t *dims, const cuuint64_t *strides,
            const cuuint32_t *box, bool codes = false) {
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return encode_tiled(m, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base),
                        dims, strides, box, one, CU_TENSOR_MAP_SWIZZLE_128B) == CUDA_SUCCESS;
}

// The pool's rows as one strided 2-D array: the smallest stride, rows, and the
// three strides in rows.
bool pool_rows(const KvCache &c, int64_t *rs, int64_t *rows, int64_t g[3]) {
    int64_t r = c.ks[0];
    for (int i = 0; i < 3; ++i) {
        if (c.vs[i] != c.ks[i]) return false;
        r = c.ks[i] < r ? c.ks[i] : r;
    }
    if (r < c.d) return false;
    for (int i = 0; i < 3; ++i) {
        if (c.ks[i] % r) return false;
        g[i] = c.ks[i] / r;
    }
    *rs = r;
    *rows = (c.lead - 1) * g[0] + (int64_t)(c.Hkv - 1) * g[1] + (int64_t)(c.page_size - 1) * g[2] + 1;
    return *rows < (int64_t)1 << 31;
}

// Rows of a box: a tile is runs of this many rows that each lie on one page;
// 0 where there is no such number (every tile is then gathered).
int box_rows(const KvCache &c) {
    if (!c.block_table || c.page_size % TT == 0) return TT;
    return c.page_size >= 8 && c.page_size < TT && TT % c.page_size == 0 ? c.page_size : 0;
}

// Two tiles of queries share the blocks where the longest chunk fills more than one.
bool two_tiles(const PrefillParams &p) { return p.c.d == 128 && p.n > TT / p.g; }

// Pages whose K and V are copied by cp.async and not by TMA.  us, by TMA / copied (32
// heads of 8; rows of one head 2 KB apart, 4 KB at d 256):
//   one tile, 4 x 16 tokens, 65,520 positions, pages of 8: 328 / 186, 16: 259 / 189,
//     24: 420 / 188, 32: 218 / 188, 64: 201 / 184, 128: 197 / 183
//   d 256, 2,048 tokens, 32,768 positions, pages of 64: 2,095 / 1,848, 128: 1,973 / 1,847
//   two tiles, 2,048 tokens, 32,768 positions, pages of 16: 927 / 902, 64: 770 / 900,
//     128: 768 / 903
bool copied(const PrefillParams &p) { return p.c.block_table && !p.c.int8 && (!two_tiles(p) || box_rows(p.c) < 64); }

template <int D, bool TWO, int LOAD>
int launch(const PfArgs &a, int grid, cudaStream_t st) {
    using C = Cfg<D, TWO, LOAD>;
    if (cudaFuncSetAttribute(prefill_tc_kernel<D, TWO, LOAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM) != cudaSuccess)
        return -5;
    prefill_tc_kernel<D, TWO, LOAD><<<grid, C::THREADS, C::SMEM, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return -5;
    if (grid == 1) return 0;
    // launched ahead: its blocks find their places while the last pieces are made
    cudaLaunchAttribute ahead;
    memset(&ahead, 0, sizeof ahead);
    ahead.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    ahead.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(grid - 1, kJoinParts);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cfg.attrs = &ahead;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prefill_join_kernel<D, TWO>, a, grid) == cudaSuccess ? 0 : -5;
}

}  // namespace

// Two tiles hold 256 rows' partial sums at head_dim 128, one 128 at 256.
int64_t prefill_slot_floats(int d) { return d == 128 ? Cfg<128, true, kTma>::SLOT_FLOATS : Cfg<256, false, kTma>::SLOT_FLOATS; }

bool prefill_tc_supports(const PrefillParams &p) {
    int64_t rs, rows, g[3];
    return p.scale_log2 > 0.f && (!p.c.block_table || copied(p) || pool_rows(p.c, &rs, &rows, g));
}

int launch_prefill_tc(const PrefillParams &p, int grid, cudaStream_t st) {
    PfArgs a;
    memset(&a, 0, sizeof a);
    a.p = p;
    a.T = TT / p.g;
    {
        // units are counted in 32 bits
        const int64_t S = a.T, nq = ceil_div(p.n, S);
        if ((int64_t)p.B * p.c.Hkv * nq * (kCharge + ceil_div(p.c.cap + p.n, TT) + 2) >= (int64_t)1 << 31) return -2;
    }
    a.R = a.T * p.g;
    a.prow = box_rows(p.c);
    a.slots = p.partials;
    {
        const cuuint64_t dims[4] = {(cuuint64_t)p.c.d, (cuuint64_t)p.Hq, (cuuint64_t)p.n, (cuuint64_t)p.B};
        const cuuint64_t strides[3] = {(cuuint64_t)p.qs[2] * 2, (cuuint64_t)p.qs[1] * 2, (cuuint64_t)p.qs[0] * 2};
        const cuuint32_t box[4] = {64, (cuuint32_t)p.g, (cuuint32_t)a.T, 1};
        if (!encode(&a.tq, 4, p.q, dims, strides, box)) return -2;
    }
    const int es = p.c.int8 ? 1 : 2;                 // bytes a number
    const cuuint64_t width = (cuuint64_t)p.c.d * es / 2;
    const bool two = two_tiles(p), copies = copied(p);
    const void *caches[2] = {p.c.k, p.c.v};
    const int64_t *strides_of[2] = {p.c.ks, p.c.vs};
    for (int i = 0; i < 2 && !copies; ++i) {
        const int64_t *s = strides_of[i];
        if (a.prow > 0) {
            const int64_t rows = p.c.block_table ? p.c.page_size : p.c.cap;
            const cuuint64_t dims[4] = {width, (cuuint64_t)rows, (cuuint64_t)p.c.Hkv, (cuuint64_t)p.c.lead};
            const cuuint64_t strides[3] = {(cuuint64_t)(s[2] * es), (cuuint64_t)(s[1] * es), (cuuint64_t)(s[0] * es)};
            const cuuint32_t box[4] = {64, (cuuint32_t)a.prow, 1, 1};
            if (!encode(i ? &a.tv : &a.tk, 4, caches[i], dims, strides, box, p.c.int8)) return -2;
        }
        int64_t rs, rows;
        if (p.c.block_table) {
            if (!pool_rows(p.c, &rs, &rows, a.gs)) return -2;
            const cuuint64_t dims[2] = {width, (cuuint64_t)rows};
            const cuuint64_t strides[1] = {(cuuint64_t)(rs * es)};
            const cuuint32_t box[2] = {64, 1};
            if (!encode(i ? &a.gv : &a.gk, 2, caches[i], dims, strides, box, p.c.int8)) return -2;
        }
    }
    if (copies) a.tk = a.tv = a.tq;                 // (unused)
    else if (a.prow == 0) { a.tk = a.gk; a.tv = a.gv; }   // (unused)
    a.p.per = TT / (two ? 2 * a.T : a.T);
    if (a.p.per < 1) a.p.per = 1;
    const auto go = [&](auto load) {
        constexpr int LOAD = decltype(load)::value;
        return p.c.d == 256 ? launch<256, false, LOAD>(a, grid, st)
               : two        ? launch<128, true, LOAD>(a, grid, st)
                            : launch<128, false, LOAD>(a, grid, st);
    };
    if (p.c.int8) return go(std::integral_constant<int, kCodes>());
    if (copies) return go(std::integral_constant<int, kCopies>());
    return go(std::integral_constant<int, kTma>());
}

}  // namespace fd
