// Index arithmetic of the paged cache, as plain integer code: which key tiles a sequence's new
// tokens visit, which keys a node of a draft tree sees, and where a position lives.  nvcc compiles
// it into the kernels; the CPU tests compile the same header with a host compiler and check it
// against brute force.
#pragma once

#include "schedule.h"

namespace gpt_attn {

constexpr int kPagedTile = 64;       // keys per tile of the paged decode kernel
constexpr int kMaxNodes = 64;        // new tokens of a sequence in one call (one bit each)

GPT_ATTN_HD int clamp_int(int x, int lo, int hi) { return x < lo ? lo : (x > hi ? hi : x); }

// What the new tokens of one sequence visit: L cached tokens (clamped to the table's capacity), n
// new ones behind them.  The node at depth 0 stands at position L, so with a window the cached
// keys in use are [w_lo, L) and the sinks before them; the new tokens' own keys are [L, end).
// Tiles of 64 keys: ns sink tiles from 0 on, then [t_lo, t_lo + n_tiles - ns).
struct PagedSpan {
    int L, n, end, w_lo, ns, t_lo, n_tiles;
    GPT_ATTN_HD int tile(int i) const { return i < ns ? i : t_lo + (i - ns); }
    // Whether the key's row has to be read at all.
    GPT_ATTN_HD bool needs(int key, int sinks) const { return key < end && (key >= w_lo || key < sinks); }
};

GPT_ATTN_HD PagedSpan paged_span(int len, int n_new, int cap, int window, int sinks) {
    PagedSpan s;
    s.L = clamp_int(len, 0, cap);
    s.n = n_new;
    s.end = s.L + n_new < cap ? s.L + n_new : cap;
    s.w_lo = window > 0 && s.L - window + 1 > 0 ? s.L - window + 1 : 0;
    s.t_lo = s.w_lo / kPagedTile;
    s.ns = (int)(((long long)sinks + kPagedTile - 1) / kPagedTile);
    if (s.ns > s.t_lo) s.ns = s.t_lo;
    s.n_tiles = s.n > 0 && s.end > 0 ? s.ns + (s.end - 1) / kPagedTile - s.t_lo + 1 : 0;
    return s;
}

// Whether the node at position `pos` with ancestors `anc` (bit d: new token d, itself included)
// sees key `key`; a new token d stands at L + depth[d].
GPT_ATTN_HD bool paged_sees(int key, int pos, unsigned long long anc, const int* depth, int L, int window, int sinks) {
    int x = key;
    if (key >= L) {
        const int d = key - L;
        if (d >= kMaxNodes || !((anc >> d) & 1)) return false;
        x = L + depth[d];
    }
    return window <= 0 || pos - x < window || x < sinks;
}

// Ancestors (itself included) of node i, by its parents; a parent that is not before its child
// counts as the cached context.
GPT_ATTN_HD unsigned long long paged_ancestors(int i, const int* parents) {
    unsigned long long m = 1ull << i;
    while (parents[i] >= 0 && parents[i] < i) {
        i = parents[i];
        m |= 1ull << i;
    }
    return m;
}

// Row of position `key` of a sequence within a pool [n_pages, Hkv, page, D], in rows of D; -1 if
// its page is missing.
GPT_ATTN_HD int paged_row(const int* table_row, int key, int page, int n_pages, int Hkv, int h) {
    const int e = table_row[key / page];
    return e < 0 || e >= n_pages ? -1 : (e * Hkv + h) * page + key % page;
}

// The flattened list of tiles of all items is cut into pieces of `chunk` tiles, one to a block;
// at least `least` to a piece, so that short calls are not scattered.
GPT_ATTN_HD long long paged_chunk(long long total, int blocks, int least) {
    const long long c = (total + blocks - 1) / blocks;
    return c < least ? least : c;
}

}  // namespace gpt_attn
