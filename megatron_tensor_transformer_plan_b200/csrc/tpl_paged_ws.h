// Sizes of the paged-cache calls and the workspace of their attention.
#pragma once

#include "tpl_internal.h"

namespace tpl {

constexpr int kPagedMaxSeqs = 1024;       // sequences per call
constexpr int kPagedMaxTokens = 1 << 22;  // rows of q per call
constexpr int kPagedMaxCtas = 160;        // CTAs of one paged attention launch at most
constexpr int kTicketPagedReady = kTicketAttn + kPagedMaxCtas;  // behind the paged tickets: the word of pdl_pass_on

// Workspace of the paged attention calls (byte offsets).
struct PagedWs {
    size_t tickets;
    size_t dec_o, dec_ml;    // single tokens: partials of the cut pairs
    size_t cut, part_o, part_ml;  // prompts and prefixes: the cut items and their partials
    size_t own_o, own_ml;    // shared prefixes: what each sequence's own keys give
    int part_rows;           // rows per partial
    size_t total;
};
int paged_ws_layout(const tpl_plan *p, int n_seqs, int n_tokens, PagedWs *w);

}  // namespace tpl
