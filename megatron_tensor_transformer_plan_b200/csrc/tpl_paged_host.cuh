// Host side of the paged-cache calls: what their arguments have to satisfy,
// their launches and the entry points.  Included by tpl_device.cu after its
// launch helpers.
#pragma once

#include "tpl_paged.cuh"
#include "tpl_paged_decode.cuh"
#include "tpl_paged_prompt.cuh"

namespace tpl {
namespace {

int paged_view(const tpl_plan *p, const tpl_paged_kv *kv, const tpl_paged_batch *b, PagedView *v) {
    if (!p || !kv || !b) return TPL_EINVAL;
    if (!kv->k || !kv->v || !al16(kv->k) || !al16(kv->v) || kv->n_pages < 1 || kv->page_size < 1) return TPL_EINVAL;
    if (b->n_seqs < 0 || b->n_tokens < 0 || (!b->q_start && b->n_tokens != b->n_seqs)) return TPL_EINVAL;
    if (b->n_tokens > 0 && (b->n_seqs == 0 || !b->page_table || !b->kv_len || b->max_pages < 1 ||
                            b->table_stride < b->max_pages))
        return TPL_EINVAL;
    if (((uintptr_t)b->page_table | (uintptr_t)b->kv_len | (uintptr_t)b->q_start) & 3u) return TPL_EINVAL;
    int shift = 4;
    while (shift < 8 && (1 << shift) != kv->page_size) ++shift;
    if ((1 << shift) != kv->page_size) return TPL_EUNSUPPORTED;
    if (((int64_t)p->d.n_kv_heads * kv->n_pages << shift) > 0x7fffffffll) return TPL_EUNSUPPORTED;
    if (((int64_t)b->max_pages << shift) > 0x7fffffffll - 4096) return TPL_EUNSUPPORTED;
    if (b->n_seqs > kPagedMaxSeqs || b->n_tokens > kPagedMaxTokens) return TPL_EUNSUPPORTED;
    v->table = b->page_table;
    v->table_stride = b->table_stride;
    v->kv_len = b->kv_len;
    v->q_start = b->q_start;
    v->max_pages = b->max_pages;
    v->n_pages = kv->n_pages;
    v->page_shift = shift;
    v->n_seqs = b->n_seqs;
    v->n_tokens = b->n_tokens;
    v->nkv = p->d.n_kv_heads;
    v->nkv_s = p->nkv_s;
    return TPL_OK;
}

int check_heads(const tpl_heads *h) {
    if (!h || !h->data || !al16(h->data) || (h->type != TPL_BF16 && h->type != TPL_F32)) return TPL_EINVAL;
    const int64_t per16 = h->type == TPL_F32 ? 4 : 8;
    if (h->token_stride < 0 || h->head_stride < 0 || h->token_stride % per16 || h->head_stride % per16)
        return TPL_EINVAL;
    return TPL_OK;
}

// Rows that are written: no two of them may overlap, and the input they are
// made from may only lie at the very same place.
int check_out_heads(const tpl_heads *o, const tpl_heads *in, int64_t heads, int64_t rows) {
    int rc = check_heads(o);
    if (rc != TPL_OK) return rc;
    if (o->type != in->type) return TPL_EINVAL;
    const int64_t ts = o->token_stride, hs = o->head_stride;
    if ((rows > 1 && ts < 128) || (heads > 1 && hs < 128)) return TPL_EINVAL;
    if (rows > 1 && heads > 1 && (ts - 128) / hs < heads - 1 && (hs - 128) / ts < rows - 1) return TPL_EINVAL;
    if (o->data == in->data && ((rows > 1 && ts != in->token_stride) || (heads > 1 && hs != in->head_stride)))
        return TPL_EINVAL;
    return TPL_OK;
}

int paged_append(const tpl_plan *p, const tpl_paged_kv *kv, const PagedView &view, const tpl_heads *q,
                 const tpl_heads *q_out, const tpl_heads *k, const tpl_heads *v, cudaStream_t st) {
    AppendArgs a;
    std::memset(&a, 0, sizeof(a));
    a.v = view;
    if (q) {
        a.q = q->data;
        a.q_ts = q->token_stride;
        a.q_hs = q->head_stride;
        a.q_out = q_out->data;
        a.qo_ts = q_out->token_stride;
        a.qo_hs = q_out->head_stride;
        a.nq = p->d.n_q_heads;
    }
    a.k = k->data;
    a.k_ts = k->token_stride;
    a.k_hs = k->head_stride;
    a.kv = v->data;
    a.v_ts = v->token_stride;
    a.v_hs = v->head_stride;
    a.kc = static_cast<__nv_bfloat16 *>(kv->k);
    a.vc = static_cast<__nv_bfloat16 *>(kv->v);
    a.rope = p->rope ? 1 : 0;
    for (int e = 0; e < 64; ++e) a.turns[e] = p->rope_theta[e] * 0.15915494309189535;
    const bool f32 = k->type == TPL_F32;
    const int sms = num_sms_current();
    if (sms <= 0) return TPL_ECUDA;
    // A token per CTA, or as many as fill its threads; with few tokens a token's heads are
    // spread over more CTAs, one item per thread, so that it does not wait on one SM: up to 4
    // such CTAs per SM.  Spread and not: 1 token of 64/8 heads in fp32 2.5 and 5.1 us, 32 tokens
    // 2.7 and 5.3, 128 (9 per SM) 4.7 and 5.8, 256 8.2 and 8.8, 512 13.0 and 11.3; 32/8 in bf16,
    // 64 tokens 2.8 and 5.1, 256 (5 per SM) 4.6 and 5.2, 512 6.6 and 5.9.
    const int items = (a.nq + 2 * view.nkv) * (f32 ? 16 : 8);
    const int parts = (items + kAppendThreads - 1) / kAppendThreads;
    const bool spread = (int64_t)view.n_tokens * parts <= 4 * sms;
    a.items_per_cta = spread ? kAppendThreads : items;
    a.tokens_per_cta = spread ? 1 : std::max(1, std::min(kAppendTokens, kAppendItems * kAppendThreads / items));
    const dim3 grid((unsigned)((view.n_tokens + a.tokens_per_cta - 1) / a.tokens_per_cta),
                    (unsigned)((items + a.items_per_cta - 1) / a.items_per_cta));
    auto go = [&](auto *kernel) { return cuda_rc(launch_pdl(kernel, grid, kAppendThreads, 0, st, a)); };
    if (a.tokens_per_cta > 1)
        return f32 ? go(paged_append_kernel<float, true>) : go(paged_append_kernel<__nv_bfloat16, true>);
    return f32 ? go(paged_append_kernel<float, false>) : go(paged_append_kernel<__nv_bfloat16, false>);
}

struct PagedCall {
    const tpl_plan *p;
    const tpl_paged_kv *kv;
    PagedView v;
    const tpl_heads *q;
    void *o;
    float *lse;
    char *ws;
    PagedWs L;
    cudaStream_t st;
};

int paged_call(const tpl_plan *p, const tpl_paged_kv *kv, const PagedView &v, const tpl_heads *q, void *o, float *lse,
               void *ws, size_t ws_bytes, tpl_stream stream, PagedCall *c) {
    int rc = check_heads(q);
    if (rc != TPL_OK) return rc;
    if (!o || !al16(o) || !ws || !al16(ws) || ((uintptr_t)lse & 3u)) return TPL_EINVAL;
    if ((rc = paged_ws_layout(p, v.n_seqs, v.n_tokens, &c->L)) != TPL_OK) return rc;
    if (ws_bytes < c->L.total) return TPL_EWORKSPACE;
    c->p = p;
    c->kv = kv;
    c->v = v;
    c->q = q;
    c->o = o;
    c->lse = lse;
    c->ws = static_cast<char *>(ws);
    c->st = static_cast<cudaStream_t>(stream);
    return TPL_OK;
}

// The pool as rows of 128 values: boxes of 64 dims x the rows of a page (at
// most box_max), or of both halves of the dims one behind the other.
int paged_maps(const PagedCall &c, CUtensorMap *k, CUtensorMap *v, int box_max, bool halves) {
    const uint64_t rows = (uint64_t)c.v.nkv * c.v.n_pages << c.v.page_shift;
    const uint32_t box = (uint32_t)std::min(1 << c.v.page_shift, box_max);
    for (CUtensorMap *m : {k, v}) {
        const void *pool = m == k ? c.kv->k : c.kv->v;
        const int rc = halves ? make_map(m, pool, 64, rows, 256, 64, box, 2, 128, 2) : make_map(m, pool, 128, rows, 256, 64, box);
        if (rc != TPL_OK) return rc;
    }
    return TPL_OK;
}

float paged_scale_log2(const tpl_plan *p) { return 1.4426950408889634f / sqrtf((float)p->d.head_dim); }

bool g_pd_attr[64][2];

template <int GM>
int paged_decode_go(const PagedDecodeArgs &a, int grid, cudaStream_t st) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return TPL_ECUDA;
    if (!g_pd_attr[dev][GM / 8 - 1]) {
        if (cudaFuncSetAttribute(paged_decode_kernel<GM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)PdSmem<GM>::BYTES) != cudaSuccess)
            return TPL_ECUDA;
        g_pd_attr[dev][GM / 8 - 1] = true;
    }
    return cuda_rc(launch_pdl(paged_decode_kernel<GM>, grid, kPdThreads, PdSmem<GM>::BYTES, st, a));
}

// Single tokens over the keys from `base` on; own: the unnormalised results
// into the workspace for the join of a shared prefix.
int paged_decode(const PagedCall &c, int window, int sinks, int base, bool own) {
    const int sms = num_sms_current();
    if (sms <= 0) return TPL_ECUDA;
    PagedDecodeArgs a;
    std::memset(&a, 0, sizeof(a));
    int rc = paged_maps(c, &a.tm_k, &a.tm_v, kPdKeys, true);
    if (rc != TPL_OK) return rc;
    a.v = c.v;
    a.q = c.q->data;
    a.q_f32 = c.q->type == TPL_F32;
    a.q_ts = c.q->token_stride;
    a.q_hs = c.q->head_stride;
    a.nq = c.p->d.n_q_heads;
    a.g = c.p->g;
    a.window = window;
    a.sinks = sinks;
    a.base = base;
    a.scale_log2 = paged_scale_log2(c.p);
    a.part_o = reinterpret_cast<float *>(c.ws + c.L.dec_o);
    a.part_ml = reinterpret_cast<float *>(c.ws + c.L.dec_ml);
    a.tickets = reinterpret_cast<unsigned *>(c.ws + c.L.tickets) + kTicketAttn;
    a.o = c.o;
    a.o_f32 = c.p->f32 ? 1 : 0;
    a.lse = c.lse;
    if (own) {
        a.own_o = reinterpret_cast<float *>(c.ws + c.L.own_o);
        a.own_ml = reinterpret_cast<float *>(c.ws + c.L.own_ml);
        a.ready = reinterpret_cast<const unsigned *>(c.ws + c.L.tickets) + kTicketPagedReady;
    }
    const int grid = std::min(sms, kPagedMaxCtas);
    return a.g <= 8 ? paged_decode_go<8>(a, grid, c.st) : paged_decode_go<16>(a, grid, c.st);
}

bool g_pt_attr[64][2];

template <bool QF32>
int paged_prompt_go(const PagedPromptArgs &a, int grid, cudaStream_t st) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return TPL_ECUDA;
    if (!g_pt_attr[dev][QF32]) {
        if (cudaFuncSetAttribute(paged_prompt_kernel<QF32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)PtSmem<QF32>::BYTES) != cudaSuccess)
            return TPL_ECUDA;
        g_pt_attr[dev][QF32] = true;
    }
    return cuda_rc(launch_pdl(paged_prompt_kernel<QF32>, grid, kPtThreads, PtSmem<QF32>::BYTES, st, a));
}

int paged_prompt_args(const PagedCall &c, PagedPromptArgs *a, int *grid) {
    const int sms = num_sms_current();
    if (sms <= 0) return TPL_ECUDA;
    *grid = std::min(sms, kPagedMaxCtas);
    std::memset(a, 0, sizeof(*a));
    int rc = paged_maps(c, &a->tm_k, &a->tm_v, kPtKeys, false);
    if (rc != TPL_OK) return rc;
    a->v = c.v;
    a->q = c.q->data;
    a->q_ts = c.q->token_stride;
    a->q_hs = c.q->head_stride;
    a->nq = c.p->d.n_q_heads;
    a->g = c.p->g;
    a->tb = 128 / c.p->g;
    a->scale_log2 = paged_scale_log2(c.p);
    a->o = static_cast<__nv_bfloat16 *>(c.o);
    a->lse = c.lse;
    a->part_o = reinterpret_cast<float *>(c.ws + c.L.part_o);
    a->part_ml = reinterpret_cast<float *>(c.ws + c.L.part_ml);
    a->part_rows = c.L.part_rows;
    return TPL_OK;
}

int paged_prompts(const PagedCall &c, int window, int sinks) {
    PagedPromptArgs a;
    int grid = 0;
    int rc = paged_prompt_args(c, &a, &grid);
    if (rc != TPL_OK) return rc;
    a.window = window;
    a.sinks = sinks;
    a.cut = reinterpret_cast<int4 *>(c.ws + c.L.cut);
    rc = c.q->type == TPL_F32 ? paged_prompt_go<true>(a, grid, c.st) : paged_prompt_go<false>(a, grid, c.st);
    if (rc != TPL_OK) return rc;
    const dim3 join((unsigned)grid, (unsigned)(a.part_rows / kPtJoinRows));
    return cuda_rc(launch_pdl(paged_prompt_join_kernel, join, kPtJoinThreads, 0, c.st, a));
}

int paged_shared(const PagedCall &c, int shared) {
    PagedSharedJoinArgs s;
    std::memset(&s, 0, sizeof(s));
    PagedPromptArgs &a = s.p;
    int grid = 0;
    int rc = paged_prompt_args(c, &a, &grid);
    if (rc != TPL_OK) return rc;
    a.shared = shared;
    a.ready = reinterpret_cast<unsigned *>(c.ws + c.L.tickets) + kTicketPagedReady;
    // The CTAs: as many per item as there are, so that no CTA has parts of two (64 sequences,
    // 8192 keys: 16 items, 144 CTAs rather than 148), when there are more CTAs than items.
    const int64_t items = (int64_t)((c.v.n_tokens + 2 * a.tb - 1) / (2 * a.tb)) * c.v.nkv;
    const int64_t U = items * ((shared + kPtKeys - 1) / kPtKeys);
    a.G = (int)std::min<int64_t>(grid, (U + kPtMinTilesPrefix - 1) / kPtMinTilesPrefix);
    if (items <= a.G) a.G = (int)(a.G / items * items);
    s.G = a.G;
    rc = c.q->type == TPL_F32 ? paged_prompt_go<true>(a, grid, c.st) : paged_prompt_go<false>(a, grid, c.st);
    if (rc == TPL_OK) rc = paged_decode(c, 0, 0, shared, true);
    if (rc != TPL_OK) return rc;
    s.own_o = reinterpret_cast<const float *>(c.ws + c.L.own_o);
    s.own_ml = reinterpret_cast<const float *>(c.ws + c.L.own_ml);
    const int64_t rows = (int64_t)c.v.n_tokens * a.nq;
    return cuda_rc(launch_pdl(paged_shared_join_kernel, (unsigned)((rows + kPtJoinRows - 1) / kPtJoinRows), kPtJoinThreads,
                              0, c.st, s));
}

}  // namespace
}  // namespace tpl

using namespace tpl;

extern "C" {

int tpl_paged_append(const tpl_plan *p, const tpl_paged_kv *kv, const tpl_paged_batch *batch, const tpl_heads *q,
                     const tpl_heads *q_out, const tpl_heads *k, const tpl_heads *v, tpl_stream stream) {
    PagedView view;
    int rc = paged_view(p, kv, batch, &view);
    if (rc != TPL_OK || view.n_tokens == 0) return rc;
    if (!q != !q_out || (rc = check_heads(k)) != TPL_OK || (rc = check_heads(v)) != TPL_OK || v->type != k->type)
        return TPL_EINVAL;
    if (q && ((rc = check_heads(q)) != TPL_OK || (rc = check_out_heads(q_out, q, p->d.n_q_heads, view.n_tokens)) != TPL_OK ||
              q->type != k->type))
        return TPL_EINVAL;
    return paged_append(p, kv, view, q, q_out, k, v, static_cast<cudaStream_t>(stream));
}

int tpl_paged_attn(const tpl_plan *p, const tpl_paged_kv *kv, const tpl_paged_batch *batch, const tpl_heads *q,
                   int32_t window, int32_t sinks, void *o, float *lse, void *ws, size_t ws_bytes, tpl_stream stream) {
    PagedView view;
    int rc = paged_view(p, kv, batch, &view);
    if (rc != TPL_OK) return rc;
    if (window < 0 || sinks < 0) return TPL_EINVAL;
    if (view.q_start && p->f32) return TPL_EUNSUPPORTED;
    if (view.n_tokens == 0) return TPL_OK;
    PagedCall c;
    if ((rc = paged_call(p, kv, view, q, o, lse, ws, ws_bytes, stream, &c)) != TPL_OK) return rc;
    return view.q_start ? paged_prompts(c, window, sinks) : paged_decode(c, window, sinks, 0, false);
}

int tpl_paged_attn_shared(const tpl_plan *p, const tpl_paged_kv *kv, const tpl_paged_batch *batch,
                          int64_t shared_len, const tpl_heads *q, void *o, float *lse, void *ws, size_t ws_bytes,
                          tpl_stream stream) {
    PagedView view;
    int rc = paged_view(p, kv, batch, &view);
    if (rc != TPL_OK) return rc;
    if (view.q_start || p->f32) return TPL_EUNSUPPORTED;
    if (view.n_tokens == 0) return TPL_OK;
    if (shared_len < 0 || shared_len % kv->page_size || shared_len > (int64_t)view.max_pages * kv->page_size)
        return TPL_EINVAL;
    PagedCall c;
    if ((rc = paged_call(p, kv, view, q, o, lse, ws, ws_bytes, stream, &c)) != TPL_OK) return rc;
    return shared_len == 0 ? paged_decode(c, 0, 0, 0, false) : paged_shared(c, (int)shared_len);
}

}  // extern "C"
