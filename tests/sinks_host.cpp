// Host build of the work decomposition with sinks (causal_attention_sdpa_b200/csrc/schedule.h) for
// the CPU tests.
#include "schedule.h"

using namespace gpt_attn;

namespace {
int doc_at(const int* ds, int T, int i) { return ds ? row_doc(i, ds[i < T ? i : T - 1]) : 0; }
int lower_at(const int* ds, int T, int W, int i) { return row_lower(i, W, ds ? ds[i < T ? i : T - 1] : 0); }
FwdSpan span_of(const int* ds, int T, int W, int sinks, int qt) {
    FwdSpan s;
    fwd_key_range_lb(qt, lower_at(ds, T, W, qt * kTile), s.lo, s.hi);
    s.s = s.ns = 0;
    fwd_add_sinks(s, doc_at(ds, T, qt * kTile), sinks);
    return s;
}
}  // namespace

extern "C" {
// Key tiles that block qb visits, in order, into `tiles` (at most cap); for query tile t of the
// block, which of them it uses into use[t * cap ...], and the tiles by its own order into
// own[t * cap ...], counts in n_own[t].  Returns the number of tiles.
int snk_fwd_block(const int* ds, int T, int W, int sinks, int qb, int cap, int* tiles, int* use, int* own, int* n_own) {
    FwdSpan a = span_of(ds, T, W, sinks, 2 * qb), b = span_of(ds, T, W, sinks, 2 * qb + 1);
    fwd_fit_pair(a, b);
    const int n = a.ns + b.hi - a.lo + 1;
    for (int u = 0; u < n && u < cap; ++u) {
        tiles[u] = a.tile(u);
        use[u] = a.has(tiles[u]);
        use[cap + u] = b.has(tiles[u]);
    }
    const FwdSpan* sp[2] = {&a, &b};
    for (int t = 0; t < 2; ++t) {
        n_own[t] = sp[t]->count();
        for (int i = 0; i < n_own[t] && i < cap; ++i) own[t * cap + i] = sp[t]->tile(i);
    }
    return n;
}
int snk_bwd_last(const int* ds, int T, int W, int sinks, int kt) {
    const int n_tiles = (T + kTile - 1) / kTile;
    if (!ds) return bwd_last_query_tile_sinks(kt, n_tiles, W, sinks);
    return bwd_last_query_tile_sinks_lb(
        kt, n_tiles, sinks, [&](int qt) { return lower_at(ds, T, W, qt * kTile); },
        [&](int qt) { return doc_at(ds, T, qt * kTile); });
}
// The cut of the sink tiles: n_s and len; returns the units of a head's sink tiles.
int snk_cut(int BH, int n_cls, int window, int sinks, int* n_s, int* len) {
    const SinkCut c = sink_cut(BH, n_cls, window, sinks, 148);
    *n_s = c.n_s;
    *len = c.len;
    return c.units;
}
void snk_list_item(int u, int BH, int n_cls, int n_s, int len, int tail, int* bh, int* cls, int* piece) {
    list_item_sinks(u, BH, n_cls, make_cut(n_s, len, n_cls), tail, *bh, *cls, *piece);
}
}
