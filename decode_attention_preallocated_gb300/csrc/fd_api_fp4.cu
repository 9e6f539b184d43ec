// fd_api_fp4.cu -- the C ABI of the 4-bit cache and of the page bookkeeping
// (declared in include/fd.h): host-side validation and the launches.  As in
// fd_api.cu every check runs before the first CUDA call, and nothing
// allocates, frees, synchronises or reads device data.
#include <cuda_runtime.h>

#include <math.h>
#include <stdint.h>
#include <string.h>

#include "fd.h"
#include "fd_api.h"
#include "fd_fp4_launch.h"
#include "fd_pages.h"

namespace {

using fd::aligned16;
using fd::check_tensor;
using fd::esize;

// What every call here wants of opts.
int check_opts(const fd_opts *o) {
    if (!o || o->reserved[0] || o->reserved[1] || o->num_ctas < 0 ||
        o->wait_limit_us < 0 || o->wait_limit_us > 2000000)
        return FD_ERR_ARG;
    if (o->kernel != FD_KERNEL_AUTO) return FD_ERR_ARG;
    return o->ws ? FD_OK : FD_ERR_WORKSPACE;
}

int status_of(int rc) { return rc == 0 ? FD_OK : (rc == -2 ? FD_ERR_UNSUPPORTED : FD_ERR_CUDA); }

// The four tensors of a 4-bit cache and how positions map to its rows.
struct Cache {
    int64_t lead, Hkv, rows, d, cap;
    int32_t page_size, page_shift, max_pages;
};

int check_global(float g) {
    return isfinite(g) && g >= 5.421010862427522e-20f && g <= 1.8446744073709552e19f ? FD_OK
                                                                                     : FD_ERR_ARG;
}

int check_cache(const fd_tensor *k, const fd_tensor *v, const fd_tensor *ks, const fd_tensor *vs,
                float k_global, float v_global, const int32_t *table, int32_t max_pages, Cache *c) {
    int rc;
    if ((rc = check_tensor(k, 4)) || (rc = check_tensor(v, 4)) || (rc = check_tensor(ks, 4)) ||
        (rc = check_tensor(vs, 4)))
        return rc;
    if (k->dtype != FD_U8 || v->dtype != FD_U8 || ks->dtype != FD_E4M3 || vs->dtype != FD_E4M3)
        return FD_ERR_ARG;
    for (int i = 0; i < 4; ++i) {
        if (v->shape[i] != k->shape[i]) return FD_ERR_ARG;
        if (i < 3 && (ks->shape[i] != k->shape[i] || vs->shape[i] != k->shape[i])) return FD_ERR_ARG;
    }
    c->lead = k->shape[0]; c->Hkv = k->shape[1]; c->rows = k->shape[2]; c->d = 2 * k->shape[3];
    if (c->lead < 1 || c->Hkv < 1 || c->rows < 1 || c->Hkv > 4096) return FD_ERR_ARG;
    if (c->d != 128 && c->d != 256) return FD_ERR_UNSUPPORTED;
    if (ks->shape[3] != c->d / 16 || vs->shape[3] != c->d / 16) return FD_ERR_ARG;
    if (k->stride[3] != 1 || v->stride[3] != 1 || ks->stride[3] != 1 || vs->stride[3] != 1)
        return FD_ERR_ARG;
    const int64_t sa = c->d / 16;
    if (!aligned16(k->data) || !aligned16(v->data) || reinterpret_cast<uintptr_t>(ks->data) % sa ||
        reinterpret_cast<uintptr_t>(vs->data) % sa)
        return FD_ERR_ALIGN;
    for (int i = 0; i < 3; ++i)
        if (k->stride[i] % 16 || v->stride[i] % 16 || ks->stride[i] % sa || vs->stride[i] % sa)
            return FD_ERR_ALIGN;
    if ((rc = check_global(k_global)) || (rc = check_global(v_global))) return rc;
    c->page_size = 0; c->page_shift = -1; c->max_pages = 0;
    if (table) {
        if (max_pages < 1) return FD_ERR_ARG;
        if (c->rows > INT32_MAX || c->lead > (1 << 30)) return FD_ERR_UNSUPPORTED;
        c->cap = (int64_t)max_pages * c->rows;
        if (c->cap >= ((int64_t)1 << 31)) return FD_ERR_UNSUPPORTED;
        c->page_size = (int32_t)c->rows;
        c->max_pages = max_pages;
        for (int sh = 0; sh < 31; ++sh)
            if (((int64_t)1 << sh) == c->rows) c->page_shift = sh;
    } else {
        if (max_pages != 0) return FD_ERR_ARG;
        c->cap = c->rows;
        if (c->cap >= ((int64_t)1 << 31)) return FD_ERR_UNSUPPORTED;
    }
    return FD_OK;
}

// New rows or read-out rows [B, n, Hkv, d]: 16-byte aligned, innermost dense.
int check_rows(const fd_tensor *t, int64_t B, int64_t n, const Cache &c) {
    const int rc = check_tensor(t, 4);
    if (rc) return rc;
    if (t->shape[0] != B || t->shape[1] != n || t->shape[2] != c.Hkv || t->shape[3] != c.d ||
        t->stride[3] != 1)
        return FD_ERR_ARG;
    if (!aligned16(t->data)) return FD_ERR_ALIGN;
    for (int i = 0; i < 3; ++i)
        if ((t->stride[i] * esize(t->dtype)) % 16) return FD_ERR_ALIGN;
    return FD_OK;
}

void fill_rows(fd::Fp4Rows *p, const fd_tensor *k, const fd_tensor *v, const fd_tensor *ks,
               const fd_tensor *vs, const Cache &c, float k_global, float v_global,
               const int32_t *table) {
    p->Hkv = (int32_t)c.Hkv; p->d = (int32_t)c.d; p->cap = c.cap;
    p->k = static_cast<uint8_t *>(k->data); p->v = static_cast<uint8_t *>(v->data);
    p->ks = static_cast<uint8_t *>(ks->data); p->vs = static_cast<uint8_t *>(vs->data);
    for (int i = 0; i < 3; ++i) {
        p->kst[i] = k->stride[i]; p->vst[i] = v->stride[i];
        p->kss[i] = ks->stride[i]; p->vss[i] = vs->stride[i];
    }
    p->k_global = k_global; p->v_global = v_global;
    p->block_table = table;
    p->page_size = c.page_size; p->page_shift = c.page_shift; p->max_pages = c.max_pages;
    p->num_pages = c.lead;
}

// Base and strides of bf16 rows are multiples of 32 bytes.
bool aligned32(const fd_tensor *t) {
    return reinterpret_cast<uintptr_t>(t->data) % 32 == 0 && t->stride[0] % 16 == 0 &&
           t->stride[1] % 16 == 0 && t->stride[2] % 16 == 0;
}

// The books of a paged cache.
int check_books(fd::Books *k, int32_t *table, int32_t B, int32_t max_pages, int32_t *lengths,
                int32_t page_size, int32_t *refs, int32_t num_pages, const fd_opts *o) {
    if (!table || !lengths || !refs) return FD_ERR_ARG;
    if (B < 1 || max_pages < 1 || page_size < 1 || num_pages < 1 || num_pages > (1 << 30))
        return FD_ERR_ARG;
    if ((int64_t)B * max_pages >= ((int64_t)1 << 31) ||
        (int64_t)max_pages * page_size >= ((int64_t)1 << 31))
        return FD_ERR_UNSUPPORTED;
    const int rc = check_opts(o);
    if (rc) return rc;
    *k = fd::Books{table, lengths, refs, B, max_pages, page_size, num_pages, o->ws->status};
    return FD_OK;
}

}  // namespace

extern "C" {

int fd_decode_fp4(const fd_tensor *q, const fd_tensor *k_cache, const fd_tensor *v_cache,
                  const fd_tensor *k_scale, const fd_tensor *v_scale, float k_global,
                  float v_global, const int32_t *block_table, int32_t max_pages,
                  const int32_t *kv_lengths, int32_t n_q, int32_t causal, float scale,
                  const fd_tensor *out, const fd_opts *opts) {
    int rc;
    if ((rc = check_tensor(q, 4)) || (rc = check_tensor(out, 4))) return rc;
    if (q->dtype != FD_BF16 || (out->dtype != FD_BF16 && out->dtype != FD_F32)) return FD_ERR_ARG;
    Cache c;
    if ((rc = check_cache(k_cache, v_cache, k_scale, v_scale, k_global, v_global, block_table,
                          max_pages, &c)))
        return rc;
    const int64_t B = q->shape[0], Hq = q->shape[2];
    for (int i = 0; i < 4; ++i)
        if (out->shape[i] != q->shape[i]) return FD_ERR_ARG;
    if (B < 1 || B > (1 << 24) || Hq < 1 || Hq > 4096 || Hq % c.Hkv || q->shape[3] != c.d ||
        q->shape[1] != n_q || (!block_table && c.lead != B))
        return FD_ERR_ARG;
    if (n_q < 1 || n_q > 6) return FD_ERR_UNSUPPORTED;
    const int64_t g = Hq / c.Hkv, rows = g * n_q;
    if (rows > FD_MAX_ROWS) return FD_ERR_UNSUPPORTED;
    if (q->stride[3] != 1 || out->stride[3] != 1 || !kv_lengths) return FD_ERR_ARG;
    if (causal != 0 && causal != 1) return FD_ERR_ARG;
    if (!isfinite(scale)) return FD_ERR_ARG;
    if ((rc = check_opts(opts))) return rc;

    fd_workspace *ws = opts->ws;
    const int parts = (int)((rows + fd::kFp4PartRows - 1) / fd::kFp4PartRows);
    const int part_rows = (int)((rows + parts - 1) / parts);
    fd::Fp4Params f;
    memset(&f, 0, sizeof f);
    fd::Params &p = f.p;
    p.B = (int32_t)B; p.n_q = n_q; p.Hq = (int32_t)Hq; p.Hkv = (int32_t)(c.Hkv * parts);
    p.g = (int32_t)g; p.d = (int32_t)c.d; p.cap = c.cap; p.rows = part_rows;
    p.mode = block_table ? fd::kPaged : fd::kDense;
    p.causal = causal; p.out_f32 = out->dtype == FD_F32;
    p.tile = fd::fp4_tile_tokens((int)c.d, part_rows);
    p.scale_log2 = (float)((double)scale * k_global * 1.4426950408889634);
    p.nseg = B * p.Hkv;
    p.q = static_cast<const uint16_t *>(q->data);
    p.k = k_cache->data; p.v = v_cache->data;
    f.ks = static_cast<const uint8_t *>(k_scale->data);
    f.vs = static_cast<const uint8_t *>(v_scale->data);
    for (int i = 0; i < 4; ++i) {
        p.qs[i] = q->stride[i]; p.os[i] = out->stride[i];
        p.ks[i] = k_cache->stride[i]; p.vs[i] = v_cache->stride[i];
    }
    for (int i = 0; i < 3; ++i) { f.kss[i] = k_scale->stride[i]; f.vss[i] = v_scale->stride[i]; }
    p.kv_lengths = kv_lengths;
    p.block_table = block_table;
    p.page_size = c.page_size; p.page_shift = c.page_shift; p.max_pages = c.max_pages;
    p.num_pages = c.lead;
    p.out = out->data;
    p.counters = ws->counters; p.status = ws->status; p.partials = ws->partials;
    f.v_global = v_global; f.parts = parts; f.all_rows = (int32_t)rows;
    f.groups = ws->groups;
    f.q_aligned8 = reinterpret_cast<uintptr_t>(q->data) % 8 == 0 && q->stride[0] % 4 == 0 &&
                   q->stride[1] % 4 == 0 && q->stride[2] % 4 == 0;
    p.seg_units = fd::fp4_seg_units(p.tile);
    // work units are counted in 32 bits on the device
    if (p.nseg * (fd::ceil_div(c.cap, p.tile) + p.seg_units) >= ((int64_t)1 << 31)) return FD_ERR_UNSUPPORTED;

    int32_t G = opts->num_ctas < 65535 ? opts->num_ctas : 65535;
    if (G == 0) {
        const int sms = fd::sm_count_current();
        if (sms <= 0) return FD_ERR_CUDA;
        const int64_t most = p.nseg * (fd::ceil_div(c.cap, p.tile) + p.seg_units);
        const int64_t want = (int64_t)sms * fd::fp4_blocks_per_sm(part_rows);
        G = (int32_t)(want < most ? want : most);
    }
    if (p.nseg > ws->max_segments || part_rows > ws->max_rows || c.d > ws->head_dim ||
        G > ws->max_ctas ||
        (size_t)(p.nseg + G) * (size_t)fd::slot_floats(part_rows, c.d) > ws->partial_floats)
        return FD_ERR_WORKSPACE;
    const std::lock_guard<std::mutex> turn(ws->turn);
    return status_of(fd::launch_fp4_decode(f, G, static_cast<cudaStream_t>(opts->stream)));
}

int fd_append_fp4(const fd_tensor *k_new, const fd_tensor *v_new, const int32_t *new_lengths,
                  const fd_tensor *k_cache, const fd_tensor *v_cache, const fd_tensor *k_scale,
                  const fd_tensor *v_scale, float k_global, float v_global,
                  const int32_t *block_table, int32_t max_pages, const int32_t *kv_lengths,
                  int32_t *lengths_out, const fd_opts *opts) {
    int rc;
    if ((rc = check_tensor(k_new, 4))) return rc;
    Cache c;
    if ((rc = check_cache(k_cache, v_cache, k_scale, v_scale, k_global, v_global, block_table,
                          max_pages, &c)))
        return rc;
    const int64_t B = k_new->shape[0], n = k_new->shape[1];
    if (B < 1 || B > (1 << 24) || n < 1 || n > INT32_MAX || (!block_table && c.lead != B))
        return FD_ERR_ARG;
    if ((rc = check_rows(k_new, B, n, c)) || (rc = check_rows(v_new, B, n, c))) return rc;
    if (k_new->dtype != FD_BF16 || v_new->dtype != FD_BF16 || !kv_lengths) return FD_ERR_ARG;
    // lengths_out is kv_lengths, or apart from it and from new_lengths
    const auto apart = [&](const int32_t *a) {
        return !a || !lengths_out || lengths_out + B <= a || a + B <= lengths_out;
    };
    if ((lengths_out != kv_lengths && !apart(kv_lengths)) || !apart(new_lengths)) return FD_ERR_ARG;
    if ((rc = check_opts(opts))) return rc;
    fd::Fp4Rows p;
    memset(&p, 0, sizeof p);
    fill_rows(&p, k_cache, v_cache, k_scale, v_scale, c, k_global, v_global, block_table);
    p.B = (int32_t)B; p.n = (int32_t)n;
    p.lengths = kv_lengths; p.status = opts->ws->status;
    p.k_new = static_cast<const uint16_t *>(k_new->data);
    p.v_new = static_cast<const uint16_t *>(v_new->data);
    for (int i = 0; i < 3; ++i) { p.kns[i] = k_new->stride[i]; p.vns[i] = v_new->stride[i]; }
    p.aligned32 = aligned32(k_new) && aligned32(v_new);
    p.new_lengths = new_lengths;
    p.lengths_out = lengths_out;
    p.grid = lengths_out == kv_lengths ? opts->ws->status + 34 : nullptr;
    return status_of(fd::launch_fp4_append(p, static_cast<cudaStream_t>(opts->stream)));
}

int fd_read_fp4(const fd_tensor *k_cache, const fd_tensor *v_cache, const fd_tensor *k_scale,
                const fd_tensor *v_scale, float k_global, float v_global,
                const int32_t *block_table, int32_t max_pages, const int32_t *start,
                const int32_t *kv_lengths, const fd_tensor *k_out, const fd_tensor *v_out,
                const fd_opts *opts) {
    int rc;
    if ((rc = check_tensor(k_out, 4))) return rc;
    Cache c;
    if ((rc = check_cache(k_cache, v_cache, k_scale, v_scale, k_global, v_global, block_table,
                          max_pages, &c)))
        return rc;
    const int64_t B = k_out->shape[0], n = k_out->shape[1];
    if (B < 1 || B > (1 << 24) || n < 1 || n > INT32_MAX || (!block_table && c.lead != B))
        return FD_ERR_ARG;
    if ((rc = check_rows(k_out, B, n, c)) || (rc = check_rows(v_out, B, n, c))) return rc;
    if ((k_out->dtype != FD_BF16 && k_out->dtype != FD_F32) || v_out->dtype != k_out->dtype ||
        !kv_lengths)
        return FD_ERR_ARG;
    if ((rc = check_opts(opts))) return rc;
    fd::Fp4Rows p;
    memset(&p, 0, sizeof p);
    fill_rows(&p, k_cache, v_cache, k_scale, v_scale, c, k_global, v_global, block_table);
    p.B = (int32_t)B; p.n = (int32_t)n;
    p.lengths = kv_lengths; p.status = opts->ws->status;
    p.start = start;
    p.k_out = k_out->data; p.v_out = v_out->data;
    for (int i = 0; i < 3; ++i) { p.kos[i] = k_out->stride[i]; p.vos[i] = v_out->stride[i]; }
    p.out_f32 = k_out->dtype == FD_F32;
    p.aligned32 = aligned32(k_out) && aligned32(v_out);
    return status_of(fd::launch_fp4_read(p, static_cast<cudaStream_t>(opts->stream)));
}

size_t fd_pages_scratch_bytes(int64_t num_pages) {
    if (num_pages < 1 || num_pages > (1 << 30)) return 0;
    return (size_t)fd::pages_scratch_words(num_pages) * 4;
}

int fd_pages_reserve(int32_t *block_table, int32_t B, int32_t max_pages,
                     const int32_t *kv_lengths, const int32_t *n_new, int32_t n_each,
                     int32_t page_size, int32_t *refs, int32_t num_pages, int32_t *pairs,
                     int32_t *count, const fd_opts *opts) {
    fd::Books k;
    const int rc = check_books(&k, block_table, B, max_pages, const_cast<int32_t *>(kv_lengths),
                               page_size, refs, num_pages, opts);
    if (rc) return rc;
    if (!pairs || !count || (!n_new && n_each < 0)) return FD_ERR_ARG;
    if ((size_t)fd::pages_scratch_words(num_pages) > opts->ws->partial_floats) return FD_ERR_WORKSPACE;
    const std::lock_guard<std::mutex> turn(opts->ws->turn);
    return status_of(fd::launch_pages_reserve(k, n_new, n_each, pairs, count,
                                              reinterpret_cast<int32_t *>(opts->ws->partials),
                                              static_cast<cudaStream_t>(opts->stream)));
}

int fd_pages_fork(int32_t *block_table, int32_t B, int32_t max_pages, int32_t *kv_lengths,
                  int32_t page_size, int32_t *refs, int32_t num_pages, const int32_t *src,
                  const int32_t *dst, const int32_t *lengths, int32_t n, const fd_opts *opts) {
    fd::Books k;
    const int rc = check_books(&k, block_table, B, max_pages, kv_lengths, page_size, refs,
                               num_pages, opts);
    if (rc) return rc;
    if (n < 0 || (n > 0 && (!src || !dst))) return FD_ERR_ARG;
    if (n == 0) return FD_OK;
    return status_of(fd::launch_pages_fork(k, src, dst, lengths, n,
                                           static_cast<cudaStream_t>(opts->stream)));
}

int fd_pages_reorder(int32_t *block_table, int32_t B, int32_t max_pages, int32_t *kv_lengths,
                     int32_t page_size, int32_t *refs, int32_t num_pages, const int32_t *src,
                     const fd_opts *opts) {
    if (!src) return FD_ERR_ARG;
    if (B > fd::kReorderRows) return FD_ERR_UNSUPPORTED;
    fd::Books k;
    const int rc = check_books(&k, block_table, B, max_pages, kv_lengths, page_size, refs,
                               num_pages, opts);
    if (rc) return rc;
    return status_of(fd::launch_pages_reorder(k, src, opts->ws->status + 34,
                                              static_cast<cudaStream_t>(opts->stream)));
}

int fd_pages_free(int32_t *block_table, int32_t B, int32_t max_pages, int32_t *kv_lengths,
                  int32_t page_size, int32_t *refs, int32_t num_pages, const int32_t *seqs,
                  const int32_t *lengths, int32_t n, const fd_opts *opts) {
    fd::Books k;
    const int rc = check_books(&k, block_table, B, max_pages, kv_lengths, page_size, refs,
                               num_pages, opts);
    if (rc) return rc;
    if (n < 0 || (n > 0 && !seqs && n != B)) return FD_ERR_ARG;
    if (n == 0) return FD_OK;
    return status_of(fd::launch_pages_free(k, seqs, lengths, n,
                                           static_cast<cudaStream_t>(opts->stream)));
}

int fd_pages_compact(int32_t *block_table, int32_t B, int32_t max_pages, int32_t *refs,
                     int32_t num_pages, int32_t *pairs, int32_t *count, const fd_opts *opts) {
    fd::Books k;
    // lengths and page size play no part
    const int rc = check_books(&k, block_table, B, max_pages, block_table, 1, refs, num_pages, opts);
    if (rc) return rc;
    if (!pairs || !count) return FD_ERR_ARG;
    if ((size_t)fd::pages_scratch_words(num_pages) > opts->ws->partial_floats) return FD_ERR_WORKSPACE;
    const std::lock_guard<std::mutex> turn(opts->ws->turn);
    return status_of(fd::launch_pages_compact(k, pairs, count,
                                              reinterpret_cast<int32_t *>(opts->ws->partials),
                                              static_cast<cudaStream_t>(opts->stream)));
}

int fd_pages_copy(const fd_tensor *pools, int32_t n_pools, const int32_t *pairs,
                  const int32_t *count, int32_t max_pairs, const fd_opts *opts) {
    if (!pools || n_pools < 1 || n_pools > fd::kMaxPools || !pairs || !count || max_pairs < 1)
        return FD_ERR_ARG;
    fd::Pools q;
    memset(&q, 0, sizeof q);
    q.n = n_pools;
    int64_t units = 0;
    for (int i = 0; i < n_pools; ++i) {
        const fd_tensor &t = pools[i];
        if (t.ndim < 1 || t.ndim > 4) return FD_ERR_ARG;
        const int rc = check_tensor(&t, t.ndim);
        if (rc) return rc;
        if (t.shape[0] != pools[0].shape[0] || t.shape[0] < 1 || t.shape[0] > (1 << 30)) return FD_ERR_ARG;
        // the page's elements fill [0, elems): taken by increasing stride, each
        // dimension of more than one steps by what those before it fill
        int64_t elems = 1;
        bool left[4] = {true, true, true, true};
        for (int j = 1; j < t.ndim; ++j) {
            if (t.shape[j] < 1) return FD_ERR_ARG;
            left[j] = t.shape[j] > 1;
        }
        for (;;) {
            int next = 0;
            for (int j = 1; j < t.ndim; ++j)
                if (left[j] && (next == 0 || t.stride[j] < t.stride[next])) next = j;
            if (next == 0) break;
            if (t.stride[next] != elems) return FD_ERR_ARG;
            elems *= t.shape[next];
            left[next] = false;
        }
        if (t.shape[0] > 1 && t.stride[0] < elems) return FD_ERR_ARG;
        q.base[i] = static_cast<uint8_t *>(t.data);
        q.step[i] = t.stride[0] * esize(t.dtype);
        q.bytes[i] = elems * esize(t.dtype);
        q.units[i] = (int32_t)units;
        units += fd::ceil_div(q.bytes[i], fd::pages_unit_bytes());
        if (units > INT32_MAX) return FD_ERR_UNSUPPORTED;
    }
    q.units[n_pools] = (int32_t)units;
    const int rc = check_opts(opts);
    if (rc) return rc;
    const int sms = fd::sm_count_current();
    if (sms <= 0) return FD_ERR_CUDA;
    return status_of(fd::launch_pages_copy(q, pairs, count, max_pairs, (int)pools[0].shape[0],
                                           opts->ws->status, sms,
                                           static_cast<cudaStream_t>(opts->stream)));
}

}  // extern "C"
