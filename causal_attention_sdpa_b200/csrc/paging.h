// Index arithmetic of the paged cache, as plain integer code: which key tiles a sequence's new
// tokens visit, which keys a node of a draft tree sees, and where a position lives.  nvcc compiles
// it into the kernels (paged_ancestors aside, which the tests go by); the CPU tests compile the same
// header with a host compiler and check it against brute force.
#pragma once

#include "schedule.h"

namespace gpt_attn {

constexpr int kPagedBox = 64;         // rows that one load brings at most
constexpr int kMaxNodes = 64;        // new tokens of a sequence in one call (one bit each)

GPT_ATTN_HD int clamp_int(int x, int lo, int hi) { return x < lo ? lo : (x > hi ? hi : x); }

// Division of 0 <= n < 2^31 by a constant d >= 1 as a multiplication and a shift: with l = ceil(log2 d)
// and m = floor(2^(31 + l) / d) + 1, m d = 2^(31 + l) + e with 0 < e <= d <= 2^l, and n m / 2^(31 + l) is
// n / d plus n e / (d 2^(31 + l)) < 1 / d, which does not reach the next whole number.
struct FastDiv {
    unsigned long long m;
    int shift, d;
    GPT_ATTN_HD int div(int n) const { return (int)((unsigned long long)(unsigned)n * m >> shift); }
};

GPT_ATTN_HD FastDiv fast_div(int d) {
    int l = 0;
    while (l < 31 && (1ll << l) < d) ++l;
    FastDiv f;
    f.shift = 31 + l;
    f.m = (1ull << f.shift) / (unsigned)d + 1;
    f.d = d;
    return f;
}

// What the new tokens of one sequence visit: L cached tokens (clamped to the table's capacity), n
// new ones behind them.  The node at depth 0 stands at position L, so with a window the cached
// keys in use are [w_lo, L) and the sinks before them; the new tokens' own keys are [L, end).
// Tiles of `tile` keys: ns sink tiles from 0 on, then [t_lo, t_lo + n_tiles - ns).
struct PagedSpan {
    int L, n, end, w_lo, ns, t_lo, n_tiles;
    GPT_ATTN_HD int tile(int i) const { return i < ns ? i : t_lo + (i - ns); }
    // Whether the key's row has to be read at all.
    GPT_ATTN_HD bool needs(int key, int sinks) const { return key < end && (key >= w_lo || key < sinks); }
    // The same for any of `n` keys from `key` on.
    GPT_ATTN_HD bool needs_any(int key, int n, int sinks) const {
        return key < end && (key + n > w_lo || key < sinks);
    }
    // Whether some node sees one of `n_keys` keys from `key` on that another does not: a new token, or one at
    // the window's lower edge.
    GPT_ATTN_HD bool differs(int key, int n_keys, int window) const {
        return n > 1 && (key + n_keys > L || (window > 0 && key + n_keys > w_lo && key <= L + n - 1 - window));
    }
};

GPT_ATTN_HD PagedSpan paged_span(int len, int n_new, int cap, int window, int sinks, int tile) {
    PagedSpan s;
    s.L = clamp_int(len, 0, cap);
    s.n = n_new;
    s.end = s.L + n_new < cap ? s.L + n_new : cap;
    s.w_lo = window > 0 && s.L - window + 1 > 0 ? s.L - window + 1 : 0;
    s.t_lo = s.w_lo / tile;
    s.ns = (int)(((long long)sinks + tile - 1) / tile);
    if (s.ns > s.t_lo) s.ns = s.t_lo;
    s.n_tiles = s.n > 0 && s.end > 0 ? s.ns + (s.end - 1) / tile - s.t_lo + 1 : 0;
    return s;
}

// A node on its way to its ancestors: those known so far (itself included), and the next one up, -1: none.
struct TreeNode {
    unsigned long long anc;
    int up;
};
// Node n before the first step; a parent that is not before its child counts as the cached context.
GPT_ATTN_HD TreeNode tree_node(int n, int parent) { return TreeNode{1ull << n, parent < n ? parent : -1}; }
// One step of all nodes at once doubles how far each has come: it takes over the ancestors of the node that it
// points at, and points where that one did.
GPT_ATTN_HD TreeNode tree_step(TreeNode x, TreeNode up) {
    return TreeNode{x.anc | (x.up < 0 ? 0 : up.anc), x.up < 0 ? -1 : up.up};
}

// Ancestors (itself included) of node i, parent by parent: what the steps above have to come to.
GPT_ATTN_HD unsigned long long paged_ancestors(int i, const int* parents) {
    unsigned long long m = 1ull << i;
    while (parents[i] >= 0 && parents[i] < i) {
        i = parents[i];
        m |= 1ull << i;
    }
    return m;
}

// New tokens that the node at position `pos` with ancestors `anc` (bit d: new token d, itself included)
// sees; new token d stands at L + depth[d].
GPT_ATTN_HD unsigned long long paged_visible(unsigned long long anc, int pos, const int* depth, int L, int window,
                                             int sinks) {
    if (window <= 0 || pos - L < window) return anc;          // the window reaches back to the first of them
    unsigned long long vis = 0;
    for (int d = 0; d < kMaxNodes; ++d)
        if (((anc >> d) & 1) && (pos - (L + depth[d]) < window || L + depth[d] < sinks)) vis |= 1ull << d;
    return vis;
}

// First position within the window of a node at `pos`.
GPT_ATTN_HD int paged_lower(int pos, int window) { return window > 0 && pos - window + 1 > 0 ? pos - window + 1 : 0; }

// The lowest n bits.
GPT_ATTN_HD unsigned bits_below(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1); }

// Which of the keys [key0, key0 + 32) a node sees: cached ones by their positions, new ones by the
// node's visible ones.
GPT_ATTN_HD unsigned paged_sees(int key0, int L, int lower, int sinks, unsigned long long vis) {
    const int at = L - key0;                                  // the bit of new token 0
    const unsigned cached = bits_below(at) & (~bits_below(lower - key0) | bits_below(sinks - key0));
    if (at >= 32 || at <= -kMaxNodes) return cached;
    return cached | (unsigned)(at >= 0 ? vis << at : vis >> -at);
}

// Row `in_page` of head h of page `entry` of a pool [n_pages, Hkv, page, D], in rows of D; -1 if there is no
// such page.
GPT_ATTN_HD int pool_row(int entry, int in_page, const FastDiv& page, int n_pages, int Hkv, int h) {
    return entry < 0 || entry >= n_pages ? -1 : (entry * Hkv + h) * page.d + in_page;
}

// Row of position `key` of a sequence.
GPT_ATTN_HD int paged_row(const int* table_row, int key, const FastDiv& page, int n_pages, int Hkv, int h) {
    const int j = page.div(key);
    return pool_row(table_row[j], key - j * page.d, page, n_pages, Hkv, h);
}

// Rows of a page that one load brings: the largest power of two that divides the page, up to
// kPagedBox, so that a box begins and ends within a page and within a tile.
GPT_ATTN_HD int paged_box(int page) {
    int box = page & -page;
    return box < kPagedBox ? box : kPagedBox;
}

// The list of all items' tiles and costs is cut into pieces of `chunk`, one to each of `workers` (teams of
// warps), none shorter than `least`.
GPT_ATTN_HD int paged_chunk(int total, int workers, int least) {
    const int c = total / workers + (total % workers > 0);
    return c < least ? least : c;
}

}  // namespace gpt_attn
