// C entry points of the attention operators: argument checks, then dispatch.
// The contract of every function is in include/dsc_attn.h.
#include <math.h>

#include <initializer_list>

#include "attn.cuh"

namespace dsc {
namespace {

dsc_status aligned(std::initializer_list<const void *> ptrs, uintptr_t to = 16) {
    for (const void *q : ptrs)
        if (!q) return DSC_ERR_INVALID_ARG;
    for (const void *q : ptrs)
        if (reinterpret_cast<uintptr_t>(q) & (to - 1)) return DSC_ERR_MISALIGNED;
    return DSC_OK;
}

dsc_status check_heads(int64_t T, int64_t Hq, int64_t Hkv, int64_t d, int dtype) {
    if (T < 1 || Hq < 1 || Hkv < 1 || d < 1 || Hq % Hkv) return DSC_ERR_INVALID_ARG;
    if (dtype != DSC_F32 && dtype != DSC_BF16) return DSC_ERR_INVALID_ARG;
    if (d % 8 || d > 128) return DSC_ERR_UNSUPPORTED;
    if (T > (int64_t)1 << 30 || Hq > 1024 || T * Hq >= (int64_t)1 << 38) return DSC_ERR_UNSUPPORTED;
    return DSC_OK;
}

// A row stride covers the row and keeps rows at 16-byte boundaries.
dsc_status check_stride(int64_t stride, int64_t width, int dtype) {
    if (stride < width || stride > (int64_t)1 << 38) return DSC_ERR_INVALID_ARG;
    return stride % (dtype == DSC_BF16 ? 8 : 4) ? DSC_ERR_MISALIGNED : DSC_OK;
}

dsc_status check_docs(const int32_t *cu, int64_t n_docs) {
    if (!cu || n_docs < 1) return DSC_ERR_INVALID_ARG;
    if (n_docs > (int64_t)1 << 24) return DSC_ERR_UNSUPPORTED;
    return aligned({cu}, 4);
}

dsc_status check_attn(const dsc_attn_problem *p) {
    if (!p) return DSC_ERR_INVALID_ARG;
    dsc_status s = check_heads(p->T, p->Hq, p->Hkv, p->d, p->dtype);
    if (s == DSC_OK && !(p->scale > 0.f && isfinite(p->scale))) s = DSC_ERR_INVALID_ARG;
    if (s == DSC_OK) s = check_stride(p->q_stride, p->Hq * p->d, p->dtype);
    return s;
}

dsc_status check_attn_kv(const dsc_attn_problem *p) {
    dsc_status s = check_attn(p);
    if (s == DSC_OK) s = check_stride(p->k_stride, p->Hkv * p->d, p->dtype);
    if (s == DSC_OK) s = check_stride(p->v_stride, p->Hkv * p->d, p->dtype);
    return s;
}

dsc_status check_cache(const dsc_paged_cache *c) {
    if (!c || c->n_pages < 1 || c->page < 1 || c->max_pages < 1) return DSC_ERR_INVALID_ARG;
    const int64_t most = (int64_t)1 << 30;
    if (c->n_pages > INT32_MAX || c->page > most || c->max_pages > most / c->page) return DSC_ERR_UNSUPPORTED;
    return DSC_OK;
}

dsc_status check_rope(const dsc_rope_problem *p, const float *inv_freq) {
    if (!p) return DSC_ERR_INVALID_ARG;
    dsc_status s = check_heads(p->T, p->Hq, p->Hkv, p->d, p->dtype);
    if (s != DSC_OK) return s;
    if (p->rot < 0 || p->rot > p->d || p->rot % 2 || (p->interleaved != 0 && p->interleaved != 1)) return DSC_ERR_INVALID_ARG;
    if (p->rot && (s = aligned({inv_freq}, 4)) != DSC_OK) return s;
    return check_stride(p->k_stride, p->Hkv * p->d, p->dtype);
}

Ctx ctx(void *stream) {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = 148;
    }
    return Ctx{static_cast<cudaStream_t>(stream), n};
}

dsc_status done(cudaError_t e) { return e == cudaSuccess ? DSC_OK : DSC_ERR_CUDA; }

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

AttnArgs attn_args(const dsc_attn_problem &p) {
    AttnArgs a{};
    a.T = p.T;
    a.Hq = (int)p.Hq; a.Hkv = (int)p.Hkv; a.d = (int)p.d; a.group = (int)(p.Hq / p.Hkv);
    a.qs = p.q_stride; a.ks = p.k_stride; a.vs = p.v_stride;
    a.scale = p.scale;
    return a;
}

// Rows of a forward and of a backward tile.
int fwd_rows(const dsc_attn_problem &p) { return p.dtype == DSC_BF16 ? attn_fwd_tc_rows((int)(p.Hq / p.Hkv)) : SIMT_ROWS; }

int bwd_rows(const dsc_attn_problem &p) { return p.dtype == DSC_BF16 ? ATTN_TC_BWD_ROWS : SIMT_ROWS; }

// The tensor-core kernels make short lists themselves, where every block has
// two items at most.  (Beyond that the items are dealt out in turn instead of
// drawn as blocks get free, and the balance is worth more than the launch:
// forward and backward of 5003 tokens, 14/2 heads, 123 us against 113; three
// prompts of 300 tokens in all 9.6 us against 11.5, replayed from a graph.)
bool inline_list(const dsc_attn_problem &p, int64_t n_docs, int rows) {
    const int64_t tiles = attn_max_tiles(p.T, n_docs, rows);
    return p.dtype == DSC_BF16 && tiles <= INLINE_TILES && tiles * p.Hq <= 2 * ctx(nullptr).sms;
}
size_t list_bytes(const dsc_attn_problem &p, int64_t n_docs, int rows) {
    return inline_list(p, n_docs, rows) ? 0 : up256(attn_list_bytes(p.T, n_docs, rows));
}

// Bytes of q-like and k-like tensors that a kernel reads again and again.
size_t input_bytes(const dsc_attn_problem &p, int q_like, int k_like) {
    return (size_t)p.T * (size_t)(q_like * p.Hq + k_like * p.Hkv) * (size_t)p.d * (p.dtype == DSC_BF16 ? 2 : 4);
}

size_t delta_bytes(const dsc_attn_problem &p) { return (size_t)p.Hq * (size_t)p.T * sizeof(float); }

TileList list_at(void *ws) {
    int *count = static_cast<int *>(ws);
    return TileList{count, count + 1, reinterpret_cast<const AttnTile *>(count + 4)};
}

dsc_status rope(const dsc_rope_problem *p, const int32_t *cu, int64_t n_docs, const void *q, const void *k,
                const float *inv_freq, void *q_out, void *k_out, float sign, void *stream) {
    dsc_status s = check_rope(p, inv_freq);
    if (s == DSC_OK) s = check_stride(p->q_stride, p->Hq * p->d, p->dtype);
    if (s == DSC_OK) s = check_docs(cu, n_docs);
    if (s == DSC_OK) s = aligned({q, k, q_out, k_out});
    if (s != DSC_OK) return s;
    RopeArgs a{};
    a.T = p->T;
    a.Hq = (int)p->Hq; a.Hkv = (int)p->Hkv; a.d = (int)p->d; a.rot = (int)p->rot;
    a.qs = p->q_stride; a.ks = p->k_stride;
    a.sign = sign;
    a.cu = cu; a.n_seqs = n_docs;
    a.inv_freq = inv_freq;
    a.q = q; a.k = k; a.q_out = q_out; a.k_out = k_out;
    return done(launch_rope(ctx(stream), p->dtype, p->interleaved, a));
}

}  // namespace
}  // namespace dsc

using namespace dsc;

extern "C" {

size_t dsc_fwd_attn_varlen_workspace_bytes(const dsc_attn_problem *p, int64_t n_docs) {
    if (check_attn_kv(p) != DSC_OK || n_docs < 1 || n_docs > (int64_t)1 << 24) return 0;
    return list_bytes(*p, n_docs, fwd_rows(*p));
}

dsc_status dsc_fwd_attn_varlen(const dsc_attn_problem *p, const int32_t *cu_seqlens, int64_t n_docs, const void *q,
                               const void *k, const void *v, void *o, float *lse, void *workspace,
                               size_t workspace_bytes, void *stream) {
    dsc_status s = check_attn_kv(p);
    if (s == DSC_OK) s = check_docs(cu_seqlens, n_docs);
    if (s == DSC_OK) s = aligned({q, k, v, o, lse});
    if (s != DSC_OK) return s;
    const int rows = fwd_rows(*p);
    const size_t need = list_bytes(*p, n_docs, rows);
    if (need && (s = aligned({workspace})) != DSC_OK) return s;
    if (workspace_bytes < need) return DSC_ERR_INVALID_ARG;
    const Ctx c = ctx(stream);
    AttnArgs a = attn_args(*p);
    a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
    const int64_t tiles = attn_max_tiles(p->T, n_docs, rows);
    if (tiles * p->Hq > INT32_MAX - (1 << 20)) return DSC_ERR_UNSUPPORTED;  // items, counted a little past their end
    if (need) {
        a.list = list_at(workspace);
        const cudaError_t e = launch_attn_tiles(c, cu_seqlens, n_docs, p->T, rows, input_bytes(*p, 1, 2), workspace, nullptr);
        if (e != cudaSuccess) return done(e);
    } else {
        a.cu = cu_seqlens;
        a.n_docs = (int)n_docs;
    }
    return done(p->dtype == DSC_BF16 ? launch_attn_fwd_tc(c, a, tiles) : launch_attn_fwd_simt(c, a, tiles));
}

// Backward workspace: the tile lists of dq (longest query tiles first) and of
// dk, dv (longest key tiles first), delta [Hq, T], and the parts of dk and dv
// where several blocks share a group.
size_t dsc_bwd_attn_varlen_workspace_bytes(const dsc_attn_problem *p, int64_t n_docs) {
    if (check_attn_kv(p) != DSC_OK || n_docs < 1 || n_docs > (int64_t)1 << 24) return 0;
    const int splits = attn_dkv_splits(p->T, bwd_rows(*p), (int)p->Hkv, (int)(p->Hq / p->Hkv), ctx(nullptr).sms);
    const size_t parts = splits > 1 ? 2 * (size_t)splits * (size_t)(p->T * p->Hkv * p->d) * sizeof(float) : 0;
    return 2 * list_bytes(*p, n_docs, bwd_rows(*p)) + up256(delta_bytes(*p)) + parts;
}

dsc_status dsc_bwd_attn_varlen(const dsc_attn_problem *p, const int32_t *cu_seqlens, int64_t n_docs, const void *q,
                               const void *k, const void *v, const void *o, const float *lse, const void *dout,
                               void *dq, int64_t dq_stride, void *dk, int64_t dk_stride, void *dv, int64_t dv_stride,
                               void *workspace, size_t workspace_bytes, void *stream) {
    dsc_status s = check_attn_kv(p);
    if (s == DSC_OK) s = check_docs(cu_seqlens, n_docs);
    if (s == DSC_OK) s = check_stride(dq_stride, p->Hq * p->d, p->dtype);
    if (s == DSC_OK) s = check_stride(dk_stride, p->Hkv * p->d, p->dtype);
    if (s == DSC_OK) s = check_stride(dv_stride, p->Hkv * p->d, p->dtype);
    if (s == DSC_OK) s = aligned({q, k, v, o, lse, dout, dq, dk, dv, workspace});
    if (s != DSC_OK) return s;
    if (workspace_bytes < dsc_bwd_attn_varlen_workspace_bytes(p, n_docs)) return DSC_ERR_INVALID_ARG;
    const Ctx c = ctx(stream);
    AttnArgs a = attn_args(*p);
    a.q = q; a.k = k; a.v = v; a.dout = dout;
    a.lse = const_cast<float *>(lse);
    a.dq = dq; a.dk = dk; a.dv = dv;
    a.dqs = dq_stride; a.dks = dk_stride; a.dvs = dv_stride;
    const bool bf = p->dtype == DSC_BF16;
    const int rows = bwd_rows(*p);
    const size_t lb = list_bytes(*p, n_docs, rows);
    const int64_t tiles = attn_max_tiles(p->T, n_docs, rows);
    if (tiles * p->Hq > INT32_MAX - (1 << 20)) return DSC_ERR_UNSUPPORTED;  // items, counted a little past their end
    char *w = static_cast<char *>(workspace);
    float *delta = reinterpret_cast<float *>(w + 2 * lb);
    a.delta = delta;
    a.nsplit = attn_dkv_splits(p->T, rows, a.Hkv, a.group, c.sms);
    if (a.nsplit > 1) {
        a.kpart = reinterpret_cast<float *>(w + 2 * lb + up256(delta_bytes(*p)));
        a.vpart = a.kpart + (size_t)a.nsplit * (size_t)(p->T * p->Hkv * p->d);
    }
    cudaError_t e = cudaSuccess;
    if (lb) {
        e = launch_attn_tiles(c, cu_seqlens, n_docs, p->T, rows, input_bytes(*p, 2, 2), w, w + lb);
    } else {
        a.cu = cu_seqlens;
        a.n_docs = (int)n_docs;
    }
    const TileList rising = list_at(w), falling = list_at(w + lb);
    if (bf) {  // dq first: it makes delta, from the probabilities
        a.list = rising;
        if (e == cudaSuccess) e = launch_attn_dq_tc(c, a, tiles);
        a.list = falling;
        if (e == cudaSuccess) e = launch_attn_dkv_tc(c, a, tiles);
    } else {
        if (e == cudaSuccess)
            e = launch_attn_delta(c, p->T, a.Hq, a.d, static_cast<const float *>(o), static_cast<const float *>(dout), delta);
        // dk, dv first: 187 us against 197 the other way round (1500 tokens, 8/4 heads of 64)
        a.list = falling;
        if (e == cudaSuccess) e = launch_attn_dkv_simt(c, a, tiles);
        a.list = rising;
        if (e == cudaSuccess) e = launch_attn_dq_simt(c, a, tiles);
    }
    return done(e);
}

dsc_status dsc_selftest_attn_timeout(void *stream) { return done(launch_feed_selftest(static_cast<cudaStream_t>(stream))); }

dsc_status dsc_fwd_rope_varlen(const dsc_rope_problem *p, const int32_t *cu_seqlens, int64_t n_docs, const void *q,
                               const void *k, const float *inv_freq, void *q_out, void *k_out, void *stream) {
    return rope(p, cu_seqlens, n_docs, q, k, inv_freq, q_out, k_out, 1.f, stream);
}

dsc_status dsc_bwd_rope_varlen(const dsc_rope_problem *p, const int32_t *cu_seqlens, int64_t n_docs, const void *dq,
                               const void *dk, const float *inv_freq, void *dq_out, void *dk_out, void *stream) {
    return rope(p, cu_seqlens, n_docs, dq, dk, inv_freq, dq_out, dk_out, -1.f, stream);
}

dsc_status dsc_kv_append(const dsc_rope_problem *p, const dsc_paged_cache *c, const int32_t *cu_seqlens,
                         int64_t n_seqs, const int32_t *seq_lens, const int32_t *block_table, const void *q,
                         const void *k, const void *v, const float *inv_freq, void *q_out, void *k_out, void *k_cache,
                         void *v_cache, void *stream) {
    dsc_status s = check_rope(p, inv_freq);
    if (s == DSC_OK) s = check_cache(c);
    if (s == DSC_OK && (!q) != (!q_out)) s = DSC_ERR_INVALID_ARG;
    if (s == DSC_OK && q) s = check_stride(p->q_stride, p->Hq * p->d, p->dtype);
    if (s == DSC_OK && q) s = aligned({q, q_out});
    if (s == DSC_OK && k_out) s = aligned({k_out});
    if (s == DSC_OK) s = check_stride(p->v_stride, p->Hkv * p->d, p->dtype);
    if (s == DSC_OK) s = aligned({k, v, k_cache, v_cache});
    if (s == DSC_OK) s = aligned({seq_lens, block_table}, 4);
    if (s == DSC_OK && cu_seqlens) s = check_docs(cu_seqlens, n_seqs);
    if (s == DSC_OK && !cu_seqlens && n_seqs != p->T) s = DSC_ERR_INVALID_ARG;
    if (s != DSC_OK) return s;
    RopeArgs a{};
    a.T = p->T;
    a.Hq = (int)p->Hq; a.Hkv = (int)p->Hkv; a.d = (int)p->d; a.rot = (int)p->rot;
    a.qs = p->q_stride; a.ks = p->k_stride; a.vs = p->v_stride;
    a.sign = 1.f;
    a.cu = cu_seqlens; a.n_seqs = n_seqs;
    a.seq_lens = seq_lens; a.table = block_table;
    a.n_pages = c->n_pages; a.page = c->page; a.max_pages = c->max_pages;
    a.inv_freq = inv_freq;
    a.q = q; a.k = k; a.v = v;
    a.q_out = q_out; a.k_out = k_out; a.k_cache = k_cache; a.v_cache = v_cache;
    return done(launch_rope(ctx(stream), p->dtype, p->interleaved, a));
}

size_t dsc_decode_attn_workspace_bytes(const dsc_attn_problem *p, const dsc_paged_cache *c) {
    if (check_attn(p) != DSC_OK || check_cache(c) != DSC_OK) return 0;
    return decode_attn_ws_bytes(ctx(nullptr), p->dtype, (int)p->d);
}

dsc_status dsc_decode_attn(const dsc_attn_problem *p, const dsc_paged_cache *c, const int32_t *seq_lens,
                           const int32_t *block_table, const void *q, const void *k_cache, const void *v_cache,
                           void *o, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    dsc_status s = check_attn(p);
    if (s == DSC_OK) s = check_cache(c);
    if (s == DSC_OK) s = aligned({q, k_cache, v_cache, o, workspace});
    if (s == DSC_OK) s = aligned({seq_lens, block_table}, 4);
    if (s == DSC_OK && lse) s = aligned({lse}, 4);
    if (s != DSC_OK) return s;
    if (workspace_bytes < dsc_decode_attn_workspace_bytes(p, c)) return DSC_ERR_INVALID_ARG;
    DecodeArgs a{};
    a.B = (int)p->T;
    a.Hq = (int)p->Hq; a.Hkv = (int)p->Hkv; a.d = (int)p->d; a.group = (int)(p->Hq / p->Hkv);
    a.qs = p->q_stride;
    a.n_pages = c->n_pages; a.max_pages = c->max_pages; a.page = (int)c->page;
    a.scale = p->scale;
    a.seq_lens = seq_lens; a.table = block_table;
    a.q = q; a.k = k_cache; a.v = v_cache; a.o = o; a.lse = lse;
    return done(launch_decode_attn(ctx(stream), p->dtype, a, workspace));
}

}  // extern "C"
