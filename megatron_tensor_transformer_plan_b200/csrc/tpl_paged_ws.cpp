// The workspace of the paged attention calls.
#include <algorithm>

#include "tpl_paged_ws.h"

namespace tpl {

int paged_ws_layout(const tpl_plan *p, int n_seqs, int n_tokens, PagedWs *w) {
    if (n_seqs <= 0 || n_tokens <= 0) return TPL_EINVAL;
    if (n_seqs > kPagedMaxSeqs || n_tokens > kPagedMaxTokens) return TPL_EUNSUPPORTED;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        size_t o = off;
        off = (off + bytes + 255) / 256 * 256;
        return o;
    };
    const size_t d = (size_t)p->d.head_dim * 4, nq = (size_t)p->d.n_q_heads, g = (size_t)p->g;
    const int tb = 128 / p->g;  // tokens per tile of 128 rows
    w->tickets = take(sizeof(uint32_t) * kTicketSlots);
    w->dec_o = take(2 * kPagedMaxCtas * g * d);
    w->dec_ml = take(2 * kPagedMaxCtas * g * 8);
    w->cut = take(kPagedMaxCtas * 16);
    // prompts: two partials per CTA; a prefix: one per CTA and per item
    w->part_rows = n_tokens <= tb ? 128 : 256;
    const size_t items = (size_t)p->d.n_kv_heads * ((n_seqs + 2 * tb - 1) / (2 * tb));
    const size_t slots = std::max<size_t>(2 * kPagedMaxCtas, items + kPagedMaxCtas);
    w->part_o = take(slots * w->part_rows * d);
    w->part_ml = take(slots * w->part_rows * 8);
    w->own_o = take((size_t)n_seqs * nq * d);
    w->own_ml = take((size_t)n_seqs * nq * 8);
    w->total = off;
    return TPL_OK;
}

}  // namespace tpl

extern "C" int tpl_paged_workspace_size(const tpl_plan *p, int32_t n_seqs, int32_t n_tokens, size_t *out) {
    if (!p || !out) return TPL_EINVAL;
    tpl::PagedWs w;
    int rc = tpl::paged_ws_layout(p, n_seqs, n_tokens, &w);
    if (rc != TPL_OK) return rc;
    *out = w.total;
    return TPL_OK;
}
