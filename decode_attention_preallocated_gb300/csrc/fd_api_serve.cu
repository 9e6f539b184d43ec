// fd_api_serve.cu -- the C ABI of the calls around decode (declared in
// include/fd.h): rows appended to a bf16 or int8 cache, attention of a chunk of
// new tokens, beam selection.  As in fd_api.cu every check runs before the
// first CUDA call, and nothing allocates, frees, synchronises or reads device
// data.
#include <cuda_runtime.h>

#include <math.h>
#include <stdint.h>
#include <string.h>

#include "fd.h"
#include "fd_api.h"
#include "fd_prefill.h"
#include "fd_serve.h"

namespace {

using fd::aligned16;
using fd::check_tensor;
using fd::esize;

// What every call here wants of opts; `any_kernel`: a kernel may be chosen.
int check_opts(const fd_opts *o, bool any_kernel) {
    if (!o || o->reserved[0] || o->reserved[1] || o->num_ctas < 0 || o->wait_limit_us < 0 ||
        o->wait_limit_us > 2000000)
        return FD_ERR_ARG;
    if (o->kernel != FD_KERNEL_AUTO && !(any_kernel && (o->kernel == FD_KERNEL_SIMT || o->kernel == FD_KERNEL_TC)))
        return FD_ERR_ARG;
    return o->ws ? FD_OK : FD_ERR_WORKSPACE;
}

bool overlap(const void *a, size_t bytes_a, const void *b, size_t bytes_b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + bytes_b && y < x + bytes_a;
}

int status_of(int rc) { return rc == 0 ? FD_OK : (rc == -2 ? FD_ERR_UNSUPPORTED : FD_ERR_CUDA); }

int check_cache(const fd_tensor *k, const fd_tensor *v, const fd_tensor *ks, const fd_tensor *vs,
                const int32_t *table, int32_t max_pages, fd::KvCache *c) {
    int rc;
    if ((rc = check_tensor(k, 4)) || (rc = check_tensor(v, 4))) return rc;
    if ((k->dtype != FD_BF16 && k->dtype != FD_I8) || v->dtype != k->dtype) return FD_ERR_ARG;
    memset(c, 0, sizeof *c);
    c->int8 = k->dtype == FD_I8;
    if (!c->int8 && (ks || vs)) return FD_ERR_ARG;
    if (c->int8 && ((rc = check_tensor(ks, 3)) || (rc = check_tensor(vs, 3)))) return rc;
    if (c->int8 && (ks->dtype != FD_F32 || vs->dtype != FD_F32)) return FD_ERR_ARG;
    for (int i = 0; i < 4; ++i) {
        if (v->shape[i] != k->shape[i]) return FD_ERR_ARG;
        if (c->int8 && i < 3 && (ks->shape[i] != k->shape[i] || vs->shape[i] != k->shape[i])) return FD_ERR_ARG;
    }
    if (k->shape[0] < 1 || k->shape[1] < 1 || k->shape[2] < 1 || k->shape[1] > 4096) return FD_ERR_ARG;
    if (k->shape[3] != 128 && k->shape[3] != 256) return FD_ERR_UNSUPPORTED;
    if (k->shape[0] > (1 << 30) || k->shape[2] > INT32_MAX) return FD_ERR_UNSUPPORTED;
    if (k->stride[3] != 1 || v->stride[3] != 1) return FD_ERR_ARG;
    if (!aligned16(k->data) || !aligned16(v->data)) return FD_ERR_ALIGN;
    const int es = esize(k->dtype);
    for (int i = 0; i < 3; ++i)
        if (k->stride[i] * es % 16 || v->stride[i] * es % 16) return FD_ERR_ALIGN;
    c->k = k->data; c->v = v->data;
    c->lead = k->shape[0]; c->Hkv = (int32_t)k->shape[1]; c->d = (int32_t)k->shape[3];
    for (int i = 0; i < 3; ++i) {
        c->ks[i] = k->stride[i]; c->vs[i] = v->stride[i];
        if (c->int8) { c->kss[i] = ks->stride[i]; c->vss[i] = vs->stride[i]; }
    }
    if (c->int8) {
        if (reinterpret_cast<uintptr_t>(ks->data) % 4 || reinterpret_cast<uintptr_t>(vs->data) % 4) return FD_ERR_ALIGN;
        c->k_scale = static_cast<float *>(ks->data);
        c->v_scale = static_cast<float *>(vs->data);
    }
    c->page_shift = -1;
    c->cap = k->shape[2];
    if (table) {
        if (max_pages < 1) return FD_ERR_ARG;
        c->cap *= max_pages;
        c->block_table = table;
        c->max_pages = max_pages;
        c->page_size = (int32_t)k->shape[2];
        for (int sh = 0; sh < 31; ++sh)
            if (((int64_t)1 << sh) == k->shape[2]) c->page_shift = sh;
    } else if (max_pages != 0) {
        return FD_ERR_ARG;
    }
    return c->cap < ((int64_t)1 << 31) ? FD_OK : FD_ERR_UNSUPPORTED;
}

// bf16 rows [B, n, H, d]: 16-byte aligned, innermost dense.
int check_rows(const fd_tensor *t, int64_t B, int64_t n, int64_t H, int64_t d) {
    const int rc = check_tensor(t, 4);
    if (rc) return rc;
    if (t->dtype != FD_BF16 || t->shape[0] != B || t->shape[1] != n || t->shape[2] != H || t->shape[3] != d ||
        t->stride[3] != 1)
        return FD_ERR_ARG;
    if (!aligned16(t->data)) return FD_ERR_ALIGN;
    for (int i = 0; i < 3; ++i)
        if (t->stride[i] % 8) return FD_ERR_ALIGN;
    return FD_OK;
}

// B sequences of n tokens, whose products are counted in 32 bits.
int check_tokens(int64_t B, int64_t n, const fd::KvCache &c) {
    if (B < 1 || n < 1 || (!c.block_table && c.lead != B)) return FD_ERR_ARG;
    return B <= (1 << 24) && n <= (1 << 24) && B * n < ((int64_t)1 << 31) ? FD_OK : FD_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

int fd_append(const fd_tensor *k_new, const fd_tensor *v_new, const int32_t *new_lengths,
              const fd_tensor *q, const fd_tensor *q_out, const fd_tensor *rope,
              int32_t interleaved, const fd_tensor *k_cache, const fd_tensor *v_cache,
              const fd_tensor *k_scale, const fd_tensor *v_scale, const int32_t *block_table,
              int32_t max_pages, const int32_t *kv_lengths, int32_t *lengths_out,
              const fd_opts *opts) {
    int rc;
    if ((rc = check_tensor(k_new, 4))) return rc;
    fd::RowsParams p;
    memset(&p, 0, sizeof p);
    if ((rc = check_cache(k_cache, v_cache, k_scale, v_scale, block_table, max_pages, &p.c))) return rc;
    const int64_t B = k_new->shape[0], n = k_new->shape[1];
    if ((rc = check_tokens(B, n, p.c))) return rc;
    if ((rc = check_rows(k_new, B, n, p.c.Hkv, p.c.d)) || (rc = check_rows(v_new, B, n, p.c.Hkv, p.c.d))) return rc;
    if (!kv_lengths || !q != !q_out || (interleaved != 0 && interleaved != 1)) return FD_ERR_ARG;
    if (q) {
        if ((rc = check_tensor(q, 4))) return rc;
        const int64_t Hq = q->shape[2];
        if (Hq < 1 || Hq > 4096) return FD_ERR_ARG;
        if ((rc = check_rows(q, B, n, Hq, p.c.d)) || (rc = check_rows(q_out, B, n, Hq, p.c.d))) return rc;
        if (q_out->data == q->data)
            for (int i = 0; i < 3; ++i)
                if (q->shape[i] > 1 && q_out->stride[i] != q->stride[i]) return FD_ERR_ARG;
        p.Hq = (int32_t)Hq;
        p.q = static_cast<const uint16_t *>(q->data);
        p.q_out = static_cast<uint16_t *>(q_out->data);
        for (int i = 0; i < 3; ++i) { p.qs[i] = q->stride[i]; p.qos[i] = q_out->stride[i]; }
    }
    if (rope) {
        if ((rc = check_tensor(rope, 2))) return rc;
        const int64_t r = rope->shape[1];
        if (rope->dtype != FD_F32 || rope->stride[1] != 1 || rope->shape[0] < 1 || r < 1 || r > p.c.d) return FD_ERR_ARG;
        if (r % 16) return FD_ERR_UNSUPPORTED;
        if (!aligned16(rope->data) || rope->stride[0] % 4) return FD_ERR_ALIGN;
        p.r = (int32_t)r; p.interleaved = interleaved;
        p.rope = static_cast<const float *>(rope->data);
        p.rope_stride = rope->stride[0];
        p.positions = rope->shape[0];
    }
    // lengths_out is kv_lengths, or apart from it and from new_lengths
    const auto apart = [&](const int32_t *a) {
        return !a || !lengths_out || lengths_out + B <= a || a + B <= lengths_out;
    };
    if ((lengths_out != kv_lengths && !apart(kv_lengths)) || !apart(new_lengths)) return FD_ERR_ARG;
    if ((rc = check_opts(opts, false))) return rc;
    p.B = (int32_t)B; p.n = (int32_t)n;
    p.k_new = static_cast<const uint16_t *>(k_new->data);
    p.v_new = static_cast<const uint16_t *>(v_new->data);
    for (int i = 0; i < 3; ++i) { p.kns[i] = k_new->stride[i]; p.vns[i] = v_new->stride[i]; }
    p.new_lengths = new_lengths; p.lengths = kv_lengths; p.lengths_out = lengths_out;
    p.status = opts->ws->status;
    p.grid = lengths_out == kv_lengths ? opts->ws->status + 34 : nullptr;
    return status_of(fd::launch_append_rows(p, static_cast<cudaStream_t>(opts->stream)));
}

size_t fd_prefill_scratch_bytes(int32_t num_ctas, int32_t head_dim) {
    if (num_ctas < 0 || num_ctas > 65535 || (head_dim != 128 && head_dim != 256)) return 0;
    if (num_ctas == 0) num_ctas = fd::sm_count_current();
    return (size_t)num_ctas * 2 * (size_t)fd::prefill_slot_floats(head_dim) * 4;
}

int fd_prefill(const fd_tensor *q, const fd_tensor *k_cache, const fd_tensor *v_cache,
               const fd_tensor *k_scale, const fd_tensor *v_scale, const int32_t *block_table,
               int32_t max_pages, const int32_t *kv_lengths, const int32_t *new_lengths,
               int32_t causal, float scale, const fd_tensor *out, const fd_opts *opts) {
    int rc;
    if ((rc = check_tensor(q, 4))) return rc;
    fd::PrefillParams p;
    memset(&p, 0, sizeof p);
    if ((rc = check_cache(k_cache, v_cache, k_scale, v_scale, block_table, max_pages, &p.c))) return rc;
    const int64_t B = q->shape[0], n = q->shape[1], Hq = q->shape[2];
    if ((rc = check_tokens(B, n, p.c))) return rc;
    if (Hq < 1 || Hq % p.c.Hkv) return FD_ERR_ARG;
    if ((rc = check_rows(q, B, n, Hq, p.c.d)) || (rc = check_rows(out, B, n, Hq, p.c.d))) return rc;
    if (Hq / p.c.Hkv > 128) return FD_ERR_UNSUPPORTED;
    if (!kv_lengths || (causal != 0 && causal != 1) || !isfinite(scale)) return FD_ERR_ARG;
    if ((rc = check_opts(opts, true))) return rc;
    p.B = (int32_t)B; p.n = (int32_t)n; p.Hq = (int32_t)Hq; p.g = (int32_t)(Hq / p.c.Hkv);
    p.causal = causal;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);
    p.q = static_cast<const uint16_t *>(q->data);
    p.out = static_cast<uint16_t *>(out->data);
    for (int i = 0; i < 3; ++i) { p.qs[i] = q->stride[i]; p.os[i] = out->stride[i]; }
    p.lengths = kv_lengths; p.new_lengths = new_lengths;
    p.status = opts->ws->status; p.partials = opts->ws->partials;
    p.wait_rounds = opts->wait_limit_us > 0 ? opts->wait_limit_us : (int32_t)(fd::kDefaultWaitNs / 1000);
    const cudaStream_t st = static_cast<cudaStream_t>(opts->stream);
    if (opts->kernel != FD_KERNEL_SIMT && fd::prefill_tc_supports(p)) {
        int32_t G = opts->num_ctas < 65535 ? opts->num_ctas : 65535;
        if (G == 0) G = fd::sm_count_current();
        if (G <= 0) return FD_ERR_CUDA;
        if (fd_prefill_scratch_bytes(G, p.c.d) > opts->ws->partial_floats * 4) return FD_ERR_WORKSPACE;
        const std::lock_guard<std::mutex> turn(opts->ws->turn);
        rc = fd::launch_prefill_tc(p, G, st);
        if (rc != -2) return status_of(rc);
    }
    if (opts->kernel == FD_KERNEL_TC) return FD_ERR_UNSUPPORTED;
    return status_of(fd::launch_prefill_simple(p, st));
}

size_t fd_beam_scratch_bytes(int64_t B, int32_t K, int64_t V, int32_t n_out) {
    if (B < 1 || B > (1 << 24) || K < 1 || K > 128 || V < 1 || V >= (1 << 24) || n_out < 1 || n_out > 64) return 0;
    return (size_t)fd::beam_scratch_bytes(B, K, V, n_out);
}

int fd_beam_select(const fd_tensor *logits, const float *scores, const int32_t *finished,
                   int32_t end_token, int32_t n_out, float *scores_out, int32_t *beams_out,
                   int32_t *tokens_out, const fd_opts *opts) {
    int rc;
    if ((rc = check_tensor(logits, 3))) return rc;
    if ((logits->dtype != FD_BF16 && logits->dtype != FD_F32) || logits->stride[2] != 1) return FD_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(logits->data) % esize(logits->dtype)) return FD_ERR_ALIGN;
    const int64_t B = logits->shape[0], K = logits->shape[1], V = logits->shape[2];
    if (B < 1 || K < 1 || V < 1 || n_out < 1 || !scores || !scores_out || !beams_out || !tokens_out) return FD_ERR_ARG;
    if (B > (1 << 24) || K > 128 || V >= (1 << 24) || n_out > 64) return FD_ERR_UNSUPPORTED;
    if (finished && (end_token < 0 || end_token >= V)) return FD_ERR_ARG;
    if ((rc = check_opts(opts, false))) return rc;
    // a request's winners are written while its scores are read
    const void *const outs[3] = {scores_out, beams_out, tokens_out};
    const size_t out_bytes = (size_t)(B * n_out) * 4, in_bytes = (size_t)(B * K) * 4;
    for (int i = 0; i < 3; ++i)
        if (overlap(outs[i], out_bytes, scores, in_bytes) || overlap(outs[i], out_bytes, finished, in_bytes) ||
            overlap(outs[i], out_bytes, outs[(i + 1) % 3], out_bytes))
            return FD_ERR_ARG;
    fd_workspace *ws = opts->ws;
    if ((size_t)fd::beam_scratch_bytes(B, (int)K, V, n_out) > ws->partial_floats * 4 || B > ws->max_segments)
        return FD_ERR_WORKSPACE;
    fd::BeamParams p;
    memset(&p, 0, sizeof p);
    p.logits = logits->data;
    p.ls[0] = logits->stride[0]; p.ls[1] = logits->stride[1];
    p.bf16 = logits->dtype == FD_BF16;
    p.B = (int32_t)B; p.K = (int32_t)K; p.V = (int32_t)V; p.n_out = n_out;
    p.scores = scores; p.finished = finished; p.end_token = end_token;
    p.scores_out = scores_out; p.beams_out = beams_out; p.tokens_out = tokens_out;
    p.scratch = reinterpret_cast<char *>(ws->partials);
    p.tickets = ws->counters;
    const std::lock_guard<std::mutex> turn(ws->turn);
    return status_of(fd::launch_beam_select(p, static_cast<cudaStream_t>(opts->stream)));
}

}  // extern "C"
