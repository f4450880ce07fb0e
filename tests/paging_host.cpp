// Host build of the paged cache's index arithmetic (causal_attention_sdpa_b200/csrc/paging.h) for the
// CPU tests.
#include "paging.h"

using namespace gpt_attn;

extern "C" {
// Tiles that a sequence's new tokens visit, in order, into `tiles`; returns their number.
int pg_tiles(int len, int n, int page, int max_pages, int window, int sinks, int tile, int cap_out, int* tiles) {
    const PagedSpan s = paged_span(len, n, page * max_pages, window, sinks, tile);
    for (int i = 0; i < s.n_tiles && i < cap_out; ++i) tiles[i] = s.tile(i);
    return s.n_tiles;
}
// Whether the key's row is read.
int pg_needs(int len, int n, int page, int max_pages, int window, int sinks, int key) {
    return paged_span(len, n, page * max_pages, window, sinks, 64).needs(key, sinks);
}
// Whether node i sees `key`.
int pg_sees(int i, const int* parents, int N, int L, int key, int window, int sinks) {
    int depth[kMaxNodes];
    for (int d = 0; d < N; ++d) {
        depth[d] = 0;
        for (unsigned long long a = paged_ancestors(d, parents) & ~(1ull << d); a; a &= a - 1) ++depth[d];
    }
    const int pos = L + depth[i];
    const unsigned long long vis = paged_visible(paged_ancestors(i, parents), pos, depth, L, window, sinks);
    return (paged_sees(key & ~31, L, paged_lower(pos, window), sinks, vis) >> (key & 31)) & 1;
}
int pg_row(const int* table_row, int key, int page, int n_pages, int Hkv, int h) {
    return paged_row(table_row, key, fast_div(page), n_pages, Hkv, h);
}
int pg_div(int n, int d) { return fast_div(d).div(n); }
int pg_box(int page) { return paged_box(page); }
// Whether a box of n keys from `key` on is read.
int pg_needs_any(int len, int n, int page, int max_pages, int window, int sinks, int key, int box) {
    return paged_span(len, n, page * max_pages, window, sinks, 64).needs_any(key, box, sinks);
}
int pg_differs(int len, int n, int page, int max_pages, int window, int sinks, int key, int n_keys) {
    return paged_span(len, n, page * max_pages, window, sinks, 64).differs(key, n_keys, window);
}
int pg_chunk(int total, int blocks, int least) { return paged_chunk(total, blocks, least); }
}
