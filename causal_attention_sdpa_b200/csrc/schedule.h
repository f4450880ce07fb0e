// Work decomposition of the attention kernels, as plain integer code: which key tiles a query
// tile sees, which query tiles a key tile reaches, and the order in which the work items of both
// passes go to the SMs.  nvcc compiles it into the kernels and the host launcher; the
// CPU tests compile the same header with a host compiler and check it against brute force.
//
// Visibility follows the masked softmax of the causal attention definition: query i sees key j
// when j <= i and, with a sliding window W > 0, j > i - W.
#pragma once

#if defined(__CUDACC__)
#define GPT_ATTN_HD __host__ __device__ __forceinline__
#else
#define GPT_ATTN_HD inline
#endif

namespace gpt_attn {

constexpr int kTile = 128;           // rows per Q tile and per K/V tile

// Lower bound of the keys query i may see: key j is visible iff row_lower(i, ...) <= j <= i.
// window > 0 keeps the last `window` keys (diagonal included); doc_start_i is the first position
// of the document holding token i (0 when the row is one document).  Document starts are clamped
// to [0, i], so every query sees at least itself whatever the input holds.
GPT_ATTN_HD int row_lower(int i, int window, int doc_start_i) {
    int lo = window > 0 ? i - window + 1 : 0;
    int d = doc_start_i < 0 ? 0 : (doc_start_i > i ? i : doc_start_i);
    if (lo < d) lo = d;
    return lo < 0 ? 0 : lo;
}

// Key tiles [lo, hi] hold every key visible to some query of query tile qt, given the lower
// bound of the tile's first row (lower bounds do not decrease along a row of documents).
GPT_ATTN_HD void fwd_key_range_lb(int qt, int first_row_lower, int& lo, int& hi) {
    hi = qt;
    lo = first_row_lower / kTile;
    if (lo > hi) lo = hi;
}

// Key tiles [lo, hi] hold every key visible to some query of query tile qt.
GPT_ATTN_HD void fwd_key_range(int qt, int window, int& lo, int& hi) {
    hi = qt;
    lo = 0;
    if (window > 0) {
        const int first = qt * kTile - window + 1;
        lo = first > 0 ? first / kTile : 0;
    }
}

// Sink keys: besides its window, query i sees the first `sinks` tokens of its document (of the
// row when it is one document), as far as they come before it.  With d the first position of
// query i's document, key j in [d, i] is visible iff i - j < window or j - d < sinks.

// First position of query i's document, clamped to [0, i].
GPT_ATTN_HD int row_doc(int i, int doc_start_i) { return doc_start_i < 0 ? 0 : (doc_start_i > i ? i : doc_start_i); }

// Key tiles one query tile visits: its sink tiles [s, s + ns), all before lo, then its window's
// tiles [lo, hi].  ns = 0 without sinks.
struct FwdSpan {
    int lo, hi, s, ns;
    GPT_ATTN_HD bool has(int j) const { return (j >= lo && j <= hi) || (j >= s && j < s + ns); }
    GPT_ATTN_HD int count() const { return ns + hi - lo + 1; }
    GPT_ATTN_HD int tile(int i) const { return i < ns ? s + i : lo + (i - ns); }
};

// Adds the sink tiles to query tile `sp` whose first row's document starts at `doc`.  The tile's
// other rows belong to that document or to one that starts inside the tile, whose sinks lie in
// tile hi, so no other tile before lo is needed.
GPT_ATTN_HD void fwd_add_sinks(FwdSpan& sp, int doc, int sinks) {
    sp.s = doc / kTile;
    const int end = (int)(((long long)doc + sinks - 1) / kTile) + 1;
    sp.ns = (end < sp.lo ? end : sp.lo) - sp.s;
    if (sp.ns < 0) sp.ns = 0;
}

// A block of two query tiles a, b visits a's sink tiles, then [a.lo, b.hi].  For document starts
// that increase this covers b's tiles; b is cut to it, so that any contents keep the roles of
// the kernel in step.
GPT_ATTN_HD void fwd_fit_pair(const FwdSpan& a, FwdSpan& b) {
    if (b.lo < a.lo) b.lo = a.lo;
    const int end = b.s + b.ns;
    if (b.s != a.s && b.s < a.lo) b.s = a.lo;
    b.ns = (end < b.lo ? end : b.lo) - b.s;
    if (b.s == a.s && b.s + b.ns > a.s + a.ns && a.s + a.ns < a.lo) b.ns = a.ns;
    if (b.ns < 0) b.ns = 0;
}

// Query tiles that see at least one key of key tile kt: [kt, bwd_last_query_tile(...)].
GPT_ATTN_HD int bwd_last_query_tile(int kt, int n_tiles, int window) {
    if (window <= 0) return n_tiles - 1;
    const long long last = (long long)kt * kTile + kTile - 1 + window - 1;   // last query seeing the tile
    const long long t = last / kTile;
    return t < n_tiles - 1 ? (int)t : n_tiles - 1;
}

// Last query tile that sees key tile kt when rows carry lower bounds (document masks):
// lower_of_tile(qt) is the lower bound of query tile qt's first row.  Lower bounds do not
// decrease along a row, so tile qt > kt sees the key tile iff its first row's bound is at or
// before the tile's last key, and those tiles form a prefix [kt, last].
template <typename LowerOfTile>
GPT_ATTN_HD int bwd_last_query_tile_lb(int kt, int n_tiles, LowerOfTile lower_of_tile) {
    const int kend = kt * kTile + kTile - 1;
    int qt = kt;
    while (qt + 1 < n_tiles && lower_of_tile(qt + 1) <= kend) ++qt;
    return qt;
}

// The same with sinks and without documents: the tiles that hold sinks are seen to the end.
GPT_ATTN_HD int bwd_last_query_tile_sinks(int kt, int n_tiles, int window, int sinks) {
    return kt * kTile < sinks ? n_tiles - 1 : bwd_last_query_tile(kt, n_tiles, window);
}

// The same with sinks and documents.  Query tile qt > kt sees key tile kt iff its first row's
// window reaches it, or that row's document starts at or before the key tile's end and its sinks
// reach past the key tile's start.  As qt grows the document starts of the first rows do not
// decrease, so the tiles that see kt are a prefix [kt, last]: windows give a prefix, and where
// sinks of an earlier document end before kt those of a later one that starts in kt take over
// from kt + 1 on.
template <typename LowerOfTile, typename DocOfTile>
GPT_ATTN_HD int bwd_last_query_tile_sinks_lb(int kt, int n_tiles, int sinks, LowerOfTile lower_of_tile,
                                             DocOfTile doc_of_tile) {
    const int k0 = kt * kTile, kend = k0 + kTile - 1;
    int qt = kt;
    while (qt + 1 < n_tiles) {
        const int d = doc_of_tile(qt + 1);
        if (!(lower_of_tile(qt + 1) <= kend || (d <= kend && (long long)d + sinks > k0))) break;
        ++qt;
    }
    return qt;
}

// Work order of both passes.  Every pass splits into work items of one head each, n_cls of
// them per head (the forward: 256-query blocks; the backward: 128-key tiles), and the items go
// to the SMs in a fixed list order, each SM taking the next item when it is ready for one (the
// forward kernel through cluster launch control, the backward kernel from a counter; the
// forward kernel also has a static order, below).  The
// items of one head should run at the same time, so that what they share (K/V in the forward;
// Q, dO and the dQ accumulator in the backward) is read from HBM once and from L2 by the
// others while it is still there: the list is head-major, each head's items longest first
// (class 0: the last query block in the forward, the first key tile in the backward).  Taken
// that way, though, the list would end with the long items of the last heads while the other
// SMs run dry; so the last `tail` heads go class-major instead (all their class-0 items, then
// all their class-1 items, ...), and the list ends with short items.

// Heads of the class-major tail: enough for the tail to hold two items per SM.
GPT_ATTN_HD int tail_heads(int BH, int n_cls, int sms) {
    const int t = (2 * sms + n_cls - 1) / n_cls;
    return t < BH ? t : BH;
}

// Item i of the list (0 <= i < BH * n_cls) whose last `tail` heads go class-major.  Returns
// head and class.
GPT_ATTN_HD void list_item(int i, int BH, int n_cls, int tail, int& bh, int& cls) {
    const int head_major = (BH - tail) * n_cls;     // items before the tail
    if (i < head_major) {
        bh = i / n_cls;
        cls = i % n_cls;
    } else {
        const int l = i - head_major;
        cls = l / tail;
        bh = BH - tail + l % tail;
    }
}

// Backward with sinks and without documents: n_s of a head's n_cls key tiles hold sinks, hence are seen
// by all later query tiles where the others are seen by a window's worth.  Those are cut into pieces of
// `len` query tiles (n_cls: not cut), each a unit of its own with partial sums of dK and dV that are
// added up afterwards, and their units go first, then the list of the others.  In the plain order the
// last heads' sink tiles started late and ran on alone: 540 against 428 us at B=4 H=6 T=8192 D=128, window
// 1024, 4 sinks, where nothing is cut.
struct SinkCut {
    int n_s, len;
    int most, units;              // most pieces of a tile (1: nothing is cut), and units of a head's sink tiles
    // Pieces of key tile kt.
    GPT_ATTN_HD int pieces(int kt, int n_cls) const { return (n_cls - kt + len - 1) / len; }
};

GPT_ATTN_HD SinkCut make_cut(int n_s, int len, int n_cls) {
    SinkCut c{n_s, len, 1, 0};
    if (n_s > 0) c.most = c.pieces(0, n_cls);
    for (int kt = 0; kt < n_s; ++kt) c.units += c.pieces(kt, n_cls);
    return c;
}

// The cut for a window and sinks (both at least 1): a piece is as long as an SM's share of all units,
// so that a sink tile does not outlast the rest (B=1 H=6 T=8192 D=128, window 512, 4 sinks, both passes: 145 us,
// not cut 300; B=1 H=2 D=64, window 128: 46 and 157),
// and no shorter than the unit of another key tile.
GPT_ATTN_HD SinkCut sink_cut(int BH, int n_cls, int window, int sinks, int sms) {
    const long long holds = ((long long)sinks + kTile - 1) / kTile;
    const int n_s = holds < n_cls ? (int)holds : n_cls;
    const long long reach = ((long long)window + kTile - 2) / kTile + 1;     // query tiles that see a key tile
    const long long all = BH * ((long long)n_s * n_cls + (n_cls - n_s) * (reach < n_cls ? reach : n_cls));
    long long len = (all + sms - 1) / sms;
    if (len < reach) len = reach;
    return make_cut(n_s, len < n_cls ? (int)len : n_cls, n_cls);
}

// Unit u of that order: head, key tile and piece (0 of the tiles that are not cut).
GPT_ATTN_HD void list_item_sinks(int u, int BH, int n_cls, const SinkCut& cut, int tail, int& bh, int& cls, int& piece) {
    const int first = BH * cut.units;
    piece = 0;
    if (u < first) {
        cls = u / BH;
        bh = u % BH;
        if (cut.most <= 1) return;                            // one piece a tile
        for (piece = cls, cls = 0; piece >= cut.pieces(cls, n_cls); ++cls) piece -= cut.pieces(cls, n_cls);
    } else {
        list_item(u - first, BH, n_cls - cut.n_s, tail, bh, cls);
        cls += cut.n_s;
    }
}

// The forward kernel has a second, static order for work that comes in many full rounds: items
// go out in waves of whole heads, heads_per_wave * n_blocks blocks, one per SM, and from one wave
// to the next the block class each block gets rotates, so that over n_blocks waves every block
// runs every class once.  Measured on the GPT-2 shapes this beats taking items on demand when
// the waves make at least kStaticCycles full rotations; with fewer, the partial rotation leaves
// some SMs with much more work than others, and the list above is used instead.
constexpr int kStaticCycles = 4;

// Static forward grid for n_blocks blocks per head: heads_per_wave and n_waves, and whether the
// static order applies at all.
GPT_ATTN_HD bool fwd_static_grid(int sms, int n_blocks, int BH, int& heads_per_wave, int& n_waves) {
    int hpw = sms / n_blocks;
    if (hpw < 1) hpw = 1;
    if (hpw > BH) hpw = BH;
    heads_per_wave = hpw;
    n_waves = (BH + hpw - 1) / hpw;
    return hpw * n_blocks <= sms && n_waves >= kStaticCycles * n_blocks;
}

// Static item of block `cta` in wave k: head bh (or -1 when the wave has none for it) and block
// qb.  Slot s of a wave holds block class s / heads_per_wave (longest first) of head
// s % heads_per_wave; a block's slot moves on by heads_per_wave each wave, so each block keeps
// to the same head position and cycles through the classes, while the blocks of a head run at
// the same time.
GPT_ATTN_HD void fwd_static_item(int heads_per_wave, int n_blocks, int BH, int cta, int k, int& bh, int& qb) {
    const int G = heads_per_wave * n_blocks;
    const int slot = (cta + heads_per_wave * (k % n_blocks)) % G;   // hpw * k mod G cycles with k mod n_blocks
    bh = heads_per_wave * k + slot % heads_per_wave;
    qb = n_blocks - 1 - slot / heads_per_wave;
    if (bh >= BH) bh = -1;
}

// Forward item i: head bh and 256-query block qb (class 0 = the last block, the longest under
// a causal mask).
GPT_ATTN_HD void fwd_item(int i, int BH, int n_blocks, int tail, int& bh, int& qb) {
    int cls;
    list_item(i, BH, n_blocks, tail, bh, cls);
    qb = n_blocks - 1 - cls;
}

// Backward work unit u: head bh, key tile kt (class 0 = key tile 0, seen by the most query
// tiles), and the n_q query tiles [kt, kt + n_q) that see it under a window (no document mask).
GPT_ATTN_HD void bwd_unit(int u, int BH, int n_tiles, int tail, int window, int& bh, int& kt, int& n_q) {
    list_item(u, BH, n_tiles, tail, bh, kt);
    n_q = bwd_last_query_tile(kt, n_tiles, window) - kt + 1;
}

}  // namespace gpt_attn
