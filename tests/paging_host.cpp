// Host build of the paged cache's index arithmetic (causal_attention_sdpa_b200/csrc/paging.h) for the
// CPU tests.
#include "paging.h"

using namespace gpt_attn;

extern "C" {
// Tiles that a sequence's new tokens visit, in order, into `tiles`; returns their number.
int pg_tiles(int len, int n, int page, int max_pages, int window, int sinks, int cap_out, int* tiles) {
    const PagedSpan s = paged_span(len, n, page * max_pages, window, sinks);
    for (int i = 0; i < s.n_tiles && i < cap_out; ++i) tiles[i] = s.tile(i);
    return s.n_tiles;
}
// Whether the key's row is read.
int pg_needs(int len, int n, int page, int max_pages, int window, int sinks, int key) {
    return paged_span(len, n, page * max_pages, window, sinks).needs(key, sinks);
}
// Whether node i sees `key`.
int pg_sees(int i, const int* parents, int N, int L, int key, int window, int sinks) {
    int depth[kMaxNodes];
    for (int d = 0; d < N; ++d) {
        depth[d] = 0;
        for (unsigned long long a = paged_ancestors(d, parents) & ~(1ull << d); a; a &= a - 1) ++depth[d];
    }
    return paged_sees(key, L + depth[i], paged_ancestors(i, parents), depth, L, window, sinks);
}
int pg_row(const int* table_row, int key, int page, int n_pages, int Hkv, int h) {
    return paged_row(table_row, key, page, n_pages, Hkv, h);
}
long long pg_chunk(long long total, int blocks, int least) { return paged_chunk(total, blocks, least); }
}
