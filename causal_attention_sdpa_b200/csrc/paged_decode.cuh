// Attention of a sequence's newest tokens over a paged key/value cache: one token, or a tree of
// drafted tokens (each node sees the cached tokens and its own ancestors), with key heads shared by
// groups of query heads, and optionally a window with sinks.
//
// The rows of one item are the N new tokens of the G query heads that share a key head: R = G * N
// rows against the same keys.  A key and a value of D elements (4 D bytes) serve 4 D R flops, R flops a
// byte, so up to some hundred rows HBM bounds the call, and the kernel is built to keep loads in
// flight.  This file has what both kernels share and the one for up to 32 rows; paged_decode_tc.cuh
// has the one for more.
//   - Keys and values come in tiles of 32 KB (128 keys of 64 elements, 64 of 128) through a ring of
//     shared-memory stages.  Producer warps bring them with TMA, in boxes of as many rows as a page
//     lets them be (the largest power of two that divides it, so a tile takes 8 boxes from pages of 16
//     tokens, 128 from odd pages), one lane to a box.  Boxes that nobody sees and missing pages are
//     not read but zero-filled.  A tile's pages are looked up while the tile before it is issued.
//   - All (sequence, key head, row block) items form one list, each as long as its tiles and what it
//     costs besides, cut into equal pieces, one to a team of warps (two teams to an SM): ragged batches
//     and single long sequences fill the GPU alike.  The ring runs on across items.  A piece that holds
//     a whole item writes O and lse; the others leave fp32 partial results, joined by
//     paged_combine_kernel.
//   - Four warps of a team compute: scores and P V on warp-level matrix instructions (16 rows x 16 keys
//     a step; a tcgen05 tile has 128 rows, of which these calls have 1 to 32), the softmax in registers
//     between them.  With up to 16 rows each warp takes a quarter of a tile's keys, else each pair of
//     warps 16 rows and each of them half of the keys; every warp has a softmax state of its own, joined
//     at the end of the item.
// A warp's steps on a tile depend on one another, so their latency counts, not their number: two teams
// share one block because its warps can then have 208 registers each (blocks of one team put five warps
// on an SM sub-partition's registers and spilled).
// Measured on one B200: one token of 16 sequences of 16384 (6 heads of 128) 132 us, 6.1 TB/s; of 64
// sequences of 4096 (12 heads of 64, pages of 16) 133 us, 6.1 TB/s; of 64 up to 1024 32 us, 3.9 TB/s; of
// one of 777 9 us.  Calls on many sequences take some 9 to 13 us more than their bytes at a copy's rate:
// launches, the first loads and the joins.
// Statistics and accumulators are fp32.  The second product takes bf16 inputs.  With up to 16 rows P goes
// into it as two terms, its rounding and what that left out, so that O is as exact as attn_decode.cuh's,
// which keeps P in fp32: an error of O's own rounding alone, 0.0016 of its norm, where one term has 0.0020.
// With up to 8 rows the second terms are the rows of the 16-row tile that the item does not have, and their
// sums are added at its end: no product more, and no exponentials for rows that are not there (one token of
// 64 sequences of up to 1024 31.8 us, where P rounded once and 16 rows' work took 33.2; of 16 of 16384 the
// same).  With products of their own, which 9 to 16 rows have, the second terms cost those calls 7 %; 16
// rows over 16 sequences of 4096 take 40.5 us where one term took 40.0.  More rows would pay 8 to 11 % (8
// rows of 4 heads over 8192: 44.5 against 40.9 us; 13 of 4 under a window of 4096 on the tcgen05 tiles: 75
// against 67), and P is rounded once, as in the forward kernel of the training calls.  P's sum is taken
// before the rounding.
#pragma once

#include "attn_fwd.cuh"
#include "paging.h"

namespace gpt_attn {

constexpr int kPagedTeams = 2;                                // of a block
constexpr int kPagedTeamWarps = 4;
constexpr int kPagedTeam = 32 * kPagedTeamWarps;
constexpr int kPagedThreads = kPagedTeams * kPagedTeam + 128; // and a warpgroup with a producer warp for each team
// What an item costs besides its tiles (its rows in, its states joined, its output), in tiles; pieces are
// cut by tiles and items together, since those with an item's end in them ran on.  It grows with the
// rows: 8 tiles with more than 16 of them (13 drafts over 16 streams, window 4096: 52.9 us, at 1 56.5, at 3
// 54.1; 32 drafts over 8 contexts up to 8192: 43.3, 46.4, 45.1), else 1 (one token of 64 sequences up to
// 1024: 32.2 us, at 3 32.0, at 8 33.4; of one sequence: 8.8, 9.3, 9.3).
constexpr int paged_item_cost(int rows) { return rows > 16 ? 8 : 1; }
// Registers of a thread: 168 at the launch, given up by the producers' warpgroup and taken by the teams.
constexpr int kPagedProducerRegs = 88, kPagedTeamRegs = 208;

struct PagedParams {
    const __nv_bfloat16* q;
    const __nv_bfloat16* k;       // [n_pages, Hkv, page, D]
    const __nv_bfloat16* v;
    const int* table;             // [B, max_pages]
    const int* lens;              // [B] cached tokens
    const int* n_new;             // [B] new tokens, or nullptr: N each
    const int* parents;           // [B, N], or nullptr: each new token's parent is the one before it
    __nv_bfloat16* o;
    float* lse;                   // [B, H, N]
    Strides q_str, o_str;         // [b, h, n, d]
    float* part_o;                // [2 * teams, rows of a row block, D]
    float* part_ml;               // [2 * teams, rows of a row block, 2]
    int* prefix;                  // [B + 1] place of each sequence in the list, then the pieces' length
    int B, H, Hkv, G, N;
    FastDiv by_n;                 // N
    int R, RB;                    // rows of an item, row blocks
    int item_cost;
    FastDiv page;
    int box_log2;                 // log2 of the rows that one load brings
    int max_pages, n_pages, cap;
    int window, sinks;
    float scale_log2;             // |scale| log2 e, of a scale of 0 1
    uint32_t q_keep, q_flip;      // q & keep ^ flip: 0 for a scale of 0, -q for one below 0
    uint64_t timeout_ns;
};

__device__ __forceinline__ int paged_n_new(const PagedParams& p, int b) {
    return p.n_new ? clamp_int(__ldg(p.n_new + b), 0, p.N) : p.N;
}

__device__ __forceinline__ PagedSpan paged_seq_span(const PagedParams& p, int b, int tile) {
    return paged_span(__ldg(p.lens + b), paged_n_new(p, b), p.cap, p.window, p.sinks, tile);
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// c += a b: 16 x 16 rows by 16 x 8 columns, bf16 inputs, fp32 sums
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Whether one of two packed bf16 values is an infinity or NaN.
__device__ __forceinline__ bool not_finite(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// Two packed bf16 values with 0 in place of infinities and NaN.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t w) {
    return ((w & 0x7f80u) == 0x7f80u ? 0u : w & 0xffffu) | ((w & 0x7f800000u) == 0x7f800000u ? 0u : w & 0xffff0000u);
}

// What rounding lo and hi to the two bf16 values in `w` left out, rounded itself: together they hold 16 bits.
__device__ __forceinline__ uint32_t rest_bf16x2(float lo, float hi, uint32_t w) {
    return pack_bf16x2(lo - __uint_as_float(w << 16), hi - __uint_as_float(w & 0xffff0000u));
}

template <int D>
struct PagedCfg {
    static constexpr int kTile = D == 64 ? 128 : 64;              // keys of a tile
    static constexpr int kTileBytes = kTile * D * 2;              // of its keys: 16 KB
    static constexpr int kStages = 3;
};

// Byte offset of 16-byte chunk c of row r in a tile as TMA's 128-byte swizzle lays it out: 64 columns
// of all rows after one another.
template <int kTile>
__device__ __forceinline__ uint32_t paged_at(int r, int c) {
    return (c >> 3) * (kTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// A place in the list: tile t of item (sequence b, key head h, row block rb), number `pos` of the list.
struct PagedAt {
    int b, h, rb, t, pos;
};

// Length of an item of the list.
__device__ __forceinline__ int paged_item(const PagedParams& p, int n_tiles) { return n_tiles + p.item_cost; }

// On to the next tile; false (and nowhere) at the end of the piece.
__device__ __forceinline__ bool paged_step(const PagedParams& p, PagedAt& at, PagedSpan& sp, int tile, int end) {
    ++at.pos;
    if (at.t + 1 == sp.n_tiles) {
        at.pos += p.item_cost;
        if (at.pos >= end) return false;
        at.t = 0;
        if (++at.rb == p.RB) {
            at.rb = 0;
            if (++at.h == p.Hkv) {
                at.h = 0;
                do sp = paged_seq_span(p, ++at.b, tile);
                while (sp.n_tiles == 0);
            }
        }
        return true;
    }
    ++at.t;
    return at.pos < end;
}

// What the computing warps have to know of one tile.
struct PagedTile {
    uint32_t seen[4];             // keys of the tile that some row may see
    int key0;                     // its first key
    int mask;                     // some row may not see some key of the tile
};

// One team's shared memory.
template <int D>
struct PagedTeam {
    using C = PagedCfg<D>;
    alignas(1024) uint8_t kv[C::kStages][2 * C::kTileBytes];      // keys, then values
    PagedTile tile[C::kStages];
    uint64_t bar_full[C::kStages], bar_empty[C::kStages];
    uint64_t bar_join;
    alignas(128) uint8_t q[kPagedTeamWarps][16 * 128];            // 64 columns of each warp's rows, on their way in
    unsigned long long anc[2][kMaxNodes];                         // the tree, of alternate sequences
    int depth[2][kMaxNodes];
    float m[2][kPagedTeamWarps][16], l[2][kPagedTeamWarps][16];
    int odd[2][kPagedTeamWarps];
    PagedAt start;
};

template <int D>
struct PagedSmem {
    PagedTeam<D> team[kPagedTeams];
    int row_head[32], row_node[32];                               // row blocks of up to 32 rows: of each row
    int scan[kPagedThreads / 32];
    int abort;
};

// A team's pass over the values of a tile some rows of which are not to be used: unseen rows are cleared
// and, if `check`, infinities and NaN of the others looked for.  The pass runs a few times a call, so that its
// instructions are waited for: not unrolled, the tcgen05 kernel gains 2 us of 61.  The kernel for up to 32 rows
// takes the same time either way (8 nodes over 16 sequences of 3000: 29.0 and 29.2 us).
template <int D, int kTile, int kUnroll>
__device__ __forceinline__ bool paged_clean(uint8_t* v, const PagedTile& t, int tid, bool check) {
    constexpr int kPerRow = kPagedTeam / kTile, kMine = D / 8 / kPerRow;      // threads to a row, 16-byte chunks of each
    const int key = tid / kPerRow, c0 = tid % kPerRow * kMine;
    bool odd = false;
    if (!((t.seen[key >> 5] >> (key & 31)) & 1)) {
#pragma unroll kUnroll
        for (int c = 0; c < kMine; ++c) *reinterpret_cast<uint4*>(v + paged_at<kTile>(key, c0 + c)) = make_uint4(0u, 0u, 0u, 0u);
    } else if (check) {
#pragma unroll kUnroll
        for (int c = 0; c < kMine; ++c) {
            const uint4 x = *reinterpret_cast<const uint4*>(v + paged_at<kTile>(key, c0 + c));
            odd = odd || not_finite(x.x) || not_finite(x.y) || not_finite(x.z) || not_finite(x.w);
        }
    }
    return odd;
}

// One warp works out the tree of sequence b, two nodes a lane: tree_step for all nodes at once, 6 times for 64.
__device__ __forceinline__ void paged_tree(const PagedParams& p, int b, unsigned long long* anc, int* depth) {
    const int lane = threadIdx.x & 31;
    TreeNode x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int n = lane + 32 * e;
        x[e] = tree_node(n, n < p.N ? __ldg(p.parents + (size_t)b * p.N + n) : -1);
    }
#pragma unroll 1
    for (int step = 1; step < p.N; step *= 2) {
        TreeNode next[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int from = max(x[e].up, 0);
            const unsigned long long a0 = __shfl_sync(0xffffffffu, x[0].anc, from & 31), a1 = __shfl_sync(0xffffffffu, x[1].anc, from & 31);
            const int u0 = __shfl_sync(0xffffffffu, x[0].up, from & 31), u1 = __shfl_sync(0xffffffffu, x[1].up, from & 31);
            next[e] = tree_step(x[e], TreeNode{from < 32 ? a0 : a1, from < 32 ? u0 : u1});
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) x[e] = next[e];
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        anc[lane + 32 * e] = x[e].anc;
        depth[lane + 32 * e] = __popcll(x[e].anc) - 1;
    }
}

// Cuts the list into the teams' pieces.  Team g of block x is number g * blocks + x, so that short lists
// take an SM a piece.  Every thread of the block takes part; the teams' places to start at are written
// where there are any, and read after the call.
struct PagedPiece {
    int chunk, all;               // length of a piece, and of the list
};

template <int kTile, int kThreads>
__device__ __forceinline__ PagedPiece paged_cut(const PagedParams& p, int* scan, PagedAt* start0, PagedAt* start1) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int total = 0, mine = 0, upto = 0;               // lengths of all sequences; of sequence b, and up to its end
    auto count = [&](int base) {
        const int b = base + threadIdx.x;
        const int n_tiles = b < p.B ? paged_seq_span(p, b, kTile).n_tiles : 0;
        mine = upto = n_tiles > 0 ? paged_item(p, n_tiles) * p.Hkv * p.RB : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += y;
        }
        __syncthreads();
        if (lane == 31) scan[warp] = upto;
        __syncthreads();
        upto += total;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            const int x = scan[w];
            if (w < warp) upto += x;
            total += x;
        }
    };
    for (int base = 0; base < p.B; base += kThreads) count(base);
    const int chunk = paged_chunk(total, kPagedTeams * gridDim.x, 1), all = total;
    auto find = [&](int base) {
        const int b = base + threadIdx.x;
        if (b >= p.B) return;
        for (int g = 0; g < kPagedTeams; ++g) {
            const long long begin = (long long)chunk * (g * gridDim.x + blockIdx.x);
            if (begin >= upto - mine && begin < upto) {
                const int len = paged_item(p, paged_seq_span(p, b, kTile).n_tiles), in_b = (int)begin - (upto - mine);
                const int x = in_b / len, in_x = in_b - x * len;              // the item, and the place in it
                (g ? *start1 : *start0) = PagedAt{b, x / p.RB, x % p.RB, max(in_x - p.item_cost, 0),
                                              (int)begin + max(p.item_cost - in_x, 0)};
            }
        }
        if (blockIdx.x == 0) p.prefix[b] = upto - mine;
    };
    if (p.B <= kThreads) {
        find(0);
    } else {
        total = 0;
        for (int base = 0; base < p.B; base += kThreads) {
            count(base);
            find(base);
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.prefix[p.B] = all;
        p.prefix[p.B + 1] = chunk;
    }
    __syncthreads();
    return PagedPiece{chunk, all};
}

// One of the two producer warps of a team, for its keys (which = 0) or values (1): walks the team's
// piece of the list from `at` up to place `end`, one tile a step, through kStages slots at `slots`,
// `stride` bytes apart.  The keys' producer also describes each tile in the ring `tiles` of kRing (and
// arrives on its `tile_full`, if the ring has barriers of its own).  Such a warp issues nearly alone, at 6
// to 8 cycles an instruction and some 80 a load, so instructions count here: one warp for both, with
// integer divisions and the table's entries awaited where they were looked up, bounded the kernel.
template <int D, int kTile, int kStages, int kRing>
__device__ __forceinline__ void paged_produce(const PagedParams& p, const CUtensorMap* tm, int which, PagedAt at, int end,
                                              uint8_t* slots, int stride, uint64_t* bar_full, uint64_t* bar_empty,
                                              PagedTile* tiles, uint64_t* tile_full, const AbortCtl& ac) {
    constexpr int kWords = kTile / 32, kTileBytes = kTile * D * 2;
    const int lane = threadIdx.x & 31;
    PagedSpan sp = paged_seq_span(p, at.b, kTile);
    const int box = 1 << p.box_log2, boxes = kTile >> p.box_log2, past = p.n_pages * p.Hkv * p.page.d;
    const int* table = p.table + (size_t)at.b * p.max_pages;
    // Boxes lane, lane + 32, ... of the current tile: the table's entry (-1: nobody sees the box) and the
    // first row within the page; the head in rows of the pool
    int entry[kWords], in_page[kWords], h = at.h;
    auto look_up = [&](int w) {
        const int j = lane + w * 32, key = sp.tile(at.t) * kTile + (j << p.box_log2);
        entry[w] = -1;
        if (j < boxes && sp.needs_any(key, box, p.sinks)) {
            const int page = p.page.div(key);
            entry[w] = table[page];
            in_page[w] = key - page * p.page.d;
        }
    };
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
        entry[w] = -1;
        in_page[w] = 0;
        if (w * 32 < boxes) look_up(w);
    }
    int i = 0, s = -1;
    uint32_t lap = 0;                                // parity of the stage's last release
    for (bool more = true; more; ++i) {
        if (++s == kStages) {
            s = 0;
            lap ^= 1;
        }
        int row[kWords];
#pragma unroll
        for (int w = 0; w < kWords; ++w)
            if (w * 32 < boxes) row[w] = pool_row(entry[w], in_page[w], p.page, p.n_pages, p.Hkv, h);
        PagedTile d;
        if (which == 0) {
            d.key0 = sp.tile(at.t) * kTile;
            // every node stands at most n - 1 past L, so keys within the window of that position are
            // within everybody's
            d.mask = d.key0 + kTile > sp.L || (p.window > 0 && sp.L + sp.n - 1 - d.key0 >= p.window);
            uint32_t there[kWords];
            bool all = d.key0 >= sp.w_lo && d.key0 + kTile <= sp.end;
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                there[w] = w * 32 < boxes ? __ballot_sync(0xffffffffu, row[w] >= 0) : 0;
                all = all && there[w] == bits_below(boxes - w * 32);
            }
#pragma unroll
            for (int w = 0; w < kWords; ++w) d.seen[w] = 0xffffffffu;
            d.mask |= !all;
            if (!all) {
#pragma unroll
                for (int w = 0; w < kWords; ++w) {
                    const int j = (lane + w * 32) >> p.box_log2;
                    uint32_t of = there[0];
#pragma unroll
                    for (int x = 1; x < kWords; ++x) of = j >> 5 == x ? there[x] : of;
                    d.seen[w] =
                        __ballot_sync(0xffffffffu, ((of >> (j & 31)) & 1) && sp.needs(d.key0 + lane + w * 32, p.sinks));
                }
            }
        }
        // the next tile's pages
        const int b = at.b;
        more = paged_step(p, at, sp, kTile, end);
        if (more) {
            if (at.b != b) table = p.table + (size_t)at.b * p.max_pages;
            h = at.h;
#pragma unroll
            for (int w = 0; w < kWords; ++w)
                if (w * 32 < boxes) look_up(w);
        }
        if (i >= kStages && !warp_wait(&bar_empty[s], lap ^ 1, ac)) break;
        if (which == 0 && debug_skip_load(3, i)) continue;   // debug builds: exercise the abort path
        if (lane == 0) {
            if (which == 0) {
                tiles[i % kRing] = d;
                if (tile_full) mbar_arrive(&tile_full[i % kRing]);
            }
            mbar_arrive_expect_tx(&bar_full[s], kTileBytes);
        }
        __syncwarp();
        uint8_t* dst = slots + s * stride;
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            const int j = lane + w * 32;
            if (w * 32 >= boxes || j >= boxes) continue;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
                tma_load_2d(dst + c * kTile * 128 + (j << p.box_log2) * 128, tm, &bar_full[s], c * 64,
                            row[w] < 0 ? past : row[w]);
        }
    }
    // the copies in flight land before the block's shared memory is given up
    for (int j = max(0, i - kStages); j < i; ++j) mbar_wait_drain(&bar_full[j % kStages], (j / kStages) & 1, p.timeout_ns);
}

// MT: 16-row tiles of an item's rows.  kFold: the item has up to 8 rows, whose second terms of P take the
// place of the tile's other 8.
template <int D, int MT, bool kFold>
__global__ void __launch_bounds__(kPagedThreads, 1)
paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ PagedParams p) {
    using C = PagedCfg<D>;
    constexpr int kStages = C::kStages, kTile = C::kTile;
    constexpr int KS = kPagedTeamWarps / MT;         // warps that share a 16-row tile's keys
    constexpr int kKeys = kTile / KS;                // keys of a warp in a tile
    constexpr int NT = kKeys / 8;
    constexpr int kChunks = D / 8;                   // 16-byte chunks of a row
    constexpr int kRows = 16 * MT;
    static_assert(!kFold || MT == 1, "one tile");
    constexpr bool kTwoTerms = MT == 1 && !kFold;    // P in two bf16 terms, each in products of its own
    constexpr int kE = kFold ? 1 : 2;                // rows of a thread: r_lo, r_lo + 8
    extern __shared__ uint8_t smem_raw[];
    PagedSmem<D>& block = *reinterpret_cast<PagedSmem<D>*>(smem_align1024(smem_raw));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    launch_dependents();
    if (threadIdx.x == 0) {
        for (int g = 0; g < kPagedTeams; ++g) {
            for (int s = 0; s < kStages; ++s) {
                mbar_init(&block.team[g].bar_full[s], 2);          // the two producers
                mbar_init(&block.team[g].bar_empty[s], kPagedTeamWarps);
            }
            mbar_init(&block.team[g].bar_join, kPagedTeamWarps);
        }
        block.abort = 0;
        fence_barrier_init();
    }
    if (threadIdx.x < kRows) {
        block.row_head[threadIdx.x] = p.by_n.div(threadIdx.x);
        block.row_node[threadIdx.x] = threadIdx.x - p.by_n.div(threadIdx.x) * p.N;
    }
    if (!p.parents && threadIdx.x < p.N) {           // one after the other: the same for all sequences
        for (int g = 0; g < kPagedTeams; ++g) {
            block.team[g].anc[0][threadIdx.x] = (2ull << threadIdx.x) - 1;
            block.team[g].depth[0][threadIdx.x] = threadIdx.x;
        }
    }

    const PagedPiece piece = paged_cut<kTile, kPagedThreads>(p, block.scan, &block.team[0].start, &block.team[1].start);

    // warps of team 0, of team 1, then keys' and values' producers of team 0, of team 1
    static_assert(kPagedTeams == 2, "two producers to a team make a warpgroup");
    const int extra = warp - kPagedTeams * kPagedTeamWarps;
    const int g = extra < 0 ? warp / kPagedTeamWarps : extra / 2;
    const int team_no = g * gridDim.x + blockIdx.x;
    const int end = (int)min((long long)piece.all, (long long)piece.chunk * (team_no + 1));
    const bool none = (long long)piece.chunk * team_no >= piece.all || block.team[g].start.pos >= end;
    const AbortCtl ac{&block.abort, p.timeout_ns};
    if (extra >= 0) {
        regs_dec<kPagedProducerRegs>();
        if (!none) {
            PagedTeam<D>& t = block.team[g];
            paged_produce<D, kTile, kStages, kStages>(p, extra & 1 ? &tm_v : &tm_k, extra & 1, t.start, end,
                                                      t.kv[0] + (extra & 1) * C::kTileBytes, 2 * C::kTileBytes, t.bar_full,
                                                      t.bar_empty, t.tile, nullptr, ac);
        }
        return;
    }
    regs_inc<kPagedTeamRegs>();
    if (none) return;
    PagedTeam<D>& sm = block.team[g];
    const int tid = threadIdx.x - g * kPagedTeam, w4 = warp - g * kPagedTeamWarps;

    // state of the current item: two rows per thread (r and r + 8 of the warp's 16)
    const int mt = w4 / KS, ks = w4 % KS;
    const int kb = ks * kKeys;                       // first key of the warp within a tile
    const int r_lo = mt * 16 + (lane >> 2);
    uint32_t qf[D / 16][4];
    float oacc[D / 8][4];
    float m[2], l[2];
    int lower[2];
    unsigned long long vis[2];                       // 0: no such row, or no such node
    int node[2], head[2];                            // node, and head within the group, of the two rows; -1: no row
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        const int r = r_lo + 8 * e, hd = p.by_n.div(r);
        head[e] = r < p.R ? hd : -1;
        node[e] = r - hd * p.N;
    }
    int cur_b = -1, item = 0, tree = 0;
    uint32_t joins = 0, lap = 1;
    int s = -1;
    // a barrier of the team
    auto join = [&]() -> bool {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.bar_join);
        return warp_wait(&sm.bar_join, joins++ & 1, ac);
    };
    PagedAt at = sm.start;
    int first = at.t, part_i = 0;                    // the part's first tile within the item and the piece
    PagedSpan sp = paged_seq_span(p, at.b, kTile);
    // The item's rows, before its first tile is waited for.
    auto set_up = [&]() -> bool {
        // the rows, 16 bytes a lane, before anything that waits
        uint4 raw[D / 64][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = mt * 16 + j * 4 + (lane >> 3), hd = p.by_n.div(r), nd = r - hd * p.N;
            const bool live = r < p.R && nd < sp.n;
            const __nv_bfloat16* src = p.q + at.b * p.q_str.b + (long long)(at.h * p.G + hd) * p.q_str.h + nd * p.q_str.t +
                                       (lane & 7) * 8;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
                raw[c][j] = live ? __ldg(reinterpret_cast<const uint4*>(src + c * 64)) : make_uint4(0u, 0u, 0u, 0u);
        }
        if (p.parents && at.b != cur_b) {
            // The tree of this sequence, by the first warp.  The other buffer may still be read; the one
            // before it is not, since all have passed that tree's join.
            tree ^= cur_b >= 0;
            cur_b = at.b;
            if (w4 == 0) paged_tree(p, at.b, sm.anc[tree], sm.depth[tree]);
            if (!join()) return false;
        }
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = j * 4 + (lane >> 3);
                *reinterpret_cast<uint4*>(sm.q[w4] + r * 128 + (((lane & 7) ^ (r & 7)) << 4)) = raw[c][j];
            }
            __syncwarp();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t(&a)[4] = qf[c * 4 + kk];
                ldmatrix4(a, smem_u32(sm.q[w4]) + (lane & 15) * 128 + (((kk * 2 + (lane >> 4)) ^ (lane & 7)) << 4));
#pragma unroll
                for (int e = 0; e < 4; ++e) a[e] = a[e] & p.q_keep ^ p.q_flip;
            }
        }
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const bool live = head[e] >= 0 && node[e] < sp.n;
            const int pos = sp.L + sm.depth[tree][node[e]];
            lower[e] = paged_lower(pos, p.window);
            vis[e] = live ? paged_visible(sm.anc[tree][node[e]], pos, sm.depth[tree], sp.L, p.window, p.sinks) : 0;
            m[e] = -INFINITY;
            l[e] = 0.f;
        }
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) oacc[n][e] = 0.f;
        return true;
    };
    if (!set_up()) return;

    bool more = true;
    for (int i = 0; more; ++i) {
        if (++s == kStages) s = 0;
        if (s == 0) lap ^= 1;
        if (!warp_wait(&sm.bar_full[s], lap, ac)) return;
        const PagedTile& t = sm.tile[s];

        // ---- scores of this warp's keys
        const uint32_t k_addr = smem_u32(sm.kv[s]), v_addr = k_addr + C::kTileBytes;
        uint8_t* vt = sm.kv[s] + C::kTileBytes;
        float sc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
        {
            const int key = kb + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t at = k_addr + paged_at<kTile>(key, kk * 2 + ((lane >> 3) & 1));
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                    uint32_t b4[4];
                    ldmatrix4(b4, at + n * 8 * 128);
                    mma_16816(sc[n], qf[kk], b4[0], b4[1]);
                    mma_16816(sc[n + 1], qf[kk], b4[2], b4[3]);
                }
            }
        }
        // keys behind the cached tokens, at a window's edge or on missing pages; rows of nodes that
        // do not exist see nothing anywhere, which the end of the item takes care of
        const int mask = t.mask;
        // one token, and keys of each warp's own: a warp goes by its own keys alone
        constexpr bool kOwnKeys = KS == kPagedTeamWarps;
        bool partial = mask;
        if (kOwnKeys && p.N == 1) partial = mask && (~(t.seen[kb / 32] >> (kb & 31)) & bits_below(kKeys)) != 0;
        if (partial) {
            const int key0 = t.key0 + kb;
#pragma unroll
            for (int e = 0; e < kE; ++e)
#pragma unroll
                for (int w = 0; w < (NT + 3) / 4; ++w) {
                    // this lane's keys of the word: bits 0 and 1, 8 and 9, ...
                    const uint32_t see = ((t.seen[kb / 32 + w] >> (kb & 31)) &
                                          paged_sees(key0 + w * 32, sp.L, lower[e], p.sinks, vis[e])) >>
                                         ((lane & 3) * 2);
#pragma unroll
                    for (int n = 0; n < 4 && w * 4 + n < NT; ++n)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            if (!((see >> (n * 8 + x)) & 1)) sc[w * 4 + n][2 * e + x] = -INFINITY;
                }
        }
        // ---- online softmax: rescaled only where a row's maximum grows by more than 2^8.  The scale is
        // above 0 (its sign is q's), so it is applied to the maximum, and to the scores within the exponent.
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            mx[0] = fmaxf(mx[0], fmaxf(sc[n][0], sc[n][1]));
            if constexpr (!kFold) mx[1] = fmaxf(mx[1], fmaxf(sc[n][2], sc[n][3]));
        }
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2)) * p.scale_log2;
        }
        const bool grow0 = mx[0] > m[0] + kLazyRescale, grow1 = !kFold && mx[1] > m[1] + kLazyRescale;
        if (__any_sync(0xffffffffu, grow0 || grow1)) {
            const float a0 = grow0 ? ex2_approx(m[0] - mx[0]) : 1.f;
            const float a1 = kFold ? a0 : (grow1 ? ex2_approx(m[1] - mx[1]) : 1.f);
            if (grow0) m[0] = mx[0];
            if (grow1) m[1] = mx[1];
            l[0] *= a0;
            if constexpr (!kFold) l[1] *= a1;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
                oacc[n][0] *= a0;
                oacc[n][1] *= a0;
                oacc[n][2] *= a1;
                oacc[n][3] *= a1;
            }
        }
        const float mu0 = m[0] == -INFINITY ? 0.f : m[0], mu1 = kFold || m[1] == -INFINITY ? 0.f : m[1];
        uint32_t pf[NT / 2][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float p0 = ex2_approx(fmaf(sc[n][0], p.scale_log2, -mu0)), p1 = ex2_approx(fmaf(sc[n][1], p.scale_log2, -mu0));
            uint32_t(&a)[4] = pf[n / 2];
            const int x = (n & 1) * 2;
            l[0] += p0 + p1;
            a[x] = pack_bf16x2(p0, p1);
            if constexpr (kFold) {
                a[x + 1] = rest_bf16x2(p0, p1, a[x]);
            } else {
                const float p2 = ex2_approx(fmaf(sc[n][2], p.scale_log2, -mu1));
                const float p3 = ex2_approx(fmaf(sc[n][3], p.scale_log2, -mu1));
                l[1] += p2 + p3;
                a[x + 1] = pack_bf16x2(p2, p3);
                sc[n][0] = p0;
                sc[n][1] = p1;
                sc[n][2] = p2;
                sc[n][3] = p3;
            }
        }
        // Rows that came along in a box without being seen may hold anything, and new tokens that are not
        // every node's ancestors infinities and NaN, which must not reach the others through 0 * NaN.
        // The former are cleared; where there are some of the latter, they are added to the rows with
        // P > 0 one by one and then cleared as well.
        if (kOwnKeys && p.N == 1) {
            // only the former
#pragma unroll 1
            for (int c = partial ? lane : kKeys * kChunks; c < kKeys * kChunks; c += 32) {
                const int key = kb + c / kChunks;
                if (!((t.seen[key >> 5] >> (key & 31)) & 1))
                    *reinterpret_cast<uint4*>(vt + paged_at<kTile>(key, c % kChunks)) = make_uint4(0u, 0u, 0u, 0u);
            }
            __syncwarp();
        } else if (mask) {
            uint4* rows = reinterpret_cast<uint4*>(vt);
            bool odd = paged_clean<D, kTile, D / 8>(vt, t, tid, sp.differs(t.key0, kTile, p.window));
            odd = __any_sync(0xffffffffu, odd);
            int(&any)[kPagedTeamWarps] = sm.odd[joins & 1];       // a warp may be a join ahead of the readers
            if (lane == 0) any[w4] = odd;
            if (!join()) return;
            odd = any[0] | any[1] | any[2] | any[3];
            if (odd) {
                // P through the stage's keys, which all warps have read
                __nv_bfloat16(*pw)[kKeys] = reinterpret_cast<__nv_bfloat16(*)[kKeys]>(sm.kv[s]) + w4 * 16;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<uint32_t*>(&pw[(lane >> 2) + 8 * e][n * 8 + (lane & 3) * 2]) =
                            pf[n / 2][(n & 1) * 2 + e];
                __syncwarp();
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
#pragma unroll 1
                    for (int kk = 0; kk < kKeys; ++kk) {
                        const uint32_t w = *reinterpret_cast<const uint32_t*>(vt + paged_at<kTile>(kb + kk, n) + (lane & 3) * 4);
                        if (!not_finite(w)) continue;
                        const float x0 = __uint_as_float(w << 16), x1 = __uint_as_float(w & 0xffff0000u);
#pragma unroll
                        for (int e = 0; e < kE; ++e) {
                            if (__bfloat162float(pw[(lane >> 2) + 8 * e][kk]) == 0.f) continue;
                            if (!isfinite(x0)) oacc[n][2 * e] += x0;
                            if (!isfinite(x1)) oacc[n][2 * e + 1] += x1;
                        }
                    }
                if (!join()) return;
                for (int c = tid; c < kTile * kChunks; c += kPagedTeam) {
                    uint4 x = rows[c];
                    x.x = finite_bf16x2(x.x);
                    x.y = finite_bf16x2(x.y);
                    x.z = finite_bf16x2(x.z);
                    x.w = finite_bf16x2(x.w);
                    rows[c] = x;
                }
                if (!join()) return;
            }
        }
        // ---- O += P V
        {
            const int key = kb + (lane & 15);
#pragma unroll
            for (int kk = 0; kk < NT / 2; ++kk) {
                uint32_t rest[4];
                if constexpr (kTwoTerms) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float* x = &sc[2 * kk + (e >> 1)][(e & 1) * 2];
                        rest[e] = rest_bf16x2(x[0], x[1], pf[kk][e]);
                    }
                }
#pragma unroll
                for (int n = 0; n < D / 16; ++n) {
                    uint32_t b4[4];
                    ldmatrix4_trans(b4, v_addr + paged_at<kTile>(key, n * 2 + (lane >> 4)) + kk * 16 * 128);
                    mma_16816(oacc[2 * n], pf[kk], b4[0], b4[1]);
                    mma_16816(oacc[2 * n + 1], pf[kk], b4[2], b4[3]);
                    if constexpr (kTwoTerms) {
                        mma_16816(oacc[2 * n], rest, b4[0], b4[1]);
                        mma_16816(oacc[2 * n + 1], rest, b4[2], b4[3]);
                    }
                }
            }
        }

        const bool done = at.t == sp.n_tiles - 1;
        if (done || at.pos + 1 >= end) {
            // ---- end of the item (or of this team's part)
            const int b = at.b, h = at.h;
            const bool whole = done && first == 0;
            if constexpr (kFold) {
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    oacc[n][0] += oacc[n][2];
                    oacc[n][1] += oacc[n][3];
                }
            }
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
                if (vis[e] == 0) {                   // a row or node that does not exist sees nothing
                    m[e] = -INFINITY;
                    l[e] = 0.f;
                }
            }
            // a piece has at most two partial items: the one it starts in and the one it ends in
            const size_t part = (2 * (size_t)team_no + (part_i > 0)) * kRows;
            // The warps that share rows join their states through the stage itself, which they
            // have all read by then.  (The statistics alternate between two buffers: a warp may
            // be an item ahead of those that still read the last one's.)
            const int par = item++ & 1;
            if ((lane & 3) == 0) {
#pragma unroll
                for (int e = 0; e < kE; ++e) {
                    sm.m[par][w4][(lane >> 2) + 8 * e] = m[e];
                    sm.l[par][w4][(lane >> 2) + 8 * e] = l[e];
                }
            }
            if (!join()) return;
            float2* state = reinterpret_cast<float2*>(sm.kv[s]);
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                const int r = (lane >> 2) + 8 * e;
                if (vis[e] == 0) continue;
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    state[(w4 * 16 + r) * (D / 2) + ((n * 4 + (lane & 3)) ^ ((r & 3) * 4))] =
                        make_float2(oacc[n][2 * e], oacc[n][2 * e + 1]);
            }
            if (!join()) return;
            for (int at = tid; at < p.R * (D / 4); at += kPagedTeam) {       // R <= kRows: one row block
                const int r = at / (D / 4), c = at % (D / 4);
                const int w0 = (r / 16) * KS, rr = r % 16;
                float M = -INFINITY, sum = 0.f;
#pragma unroll
                for (int w = 0; w < KS; ++w) M = fmaxf(M, sm.m[par][w0 + w][rr]);
                const float mu = M == -INFINITY ? 0.f : M;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < KS; ++w) {
                    const float lw = sm.l[par][w0 + w][rr];
                    if (lw == 0.f) continue;     // a warp whose keys the row does not see wrote nothing of use
                    const float f = ex2_approx(sm.m[par][w0 + w][rr] - mu);
                    sum += lw * f;
                    const float4 y = *reinterpret_cast<const float4*>(state + ((w0 + w) * 16 + rr) * (D / 2) +
                                                                      ((c * 2) ^ ((rr & 3) * 4)));
                    a.x += f * y.x;
                    a.y += f * y.y;
                    a.z += f * y.z;
                    a.w += f * y.w;
                }
                const bool any = sum != 0.f;
                if (whole) {
                    const int hd = h * p.G + block.row_head[r], nd = block.row_node[r];
                    __nv_bfloat16* dst = p.o + b * p.o_str.b + hd * p.o_str.h + nd * p.o_str.t + c * 4;
                    const float inv = any ? 1.f / sum : 0.f;
                    *reinterpret_cast<uint2*>(dst) =
                        make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
                    if (c == 0)
                        p.lse[((size_t)b * p.H + hd) * p.N + nd] =
                            any ? (M + log2f(sum)) * 0.69314718055994531f : -INFINITY;
                } else {
                    *reinterpret_cast<float4*>(p.part_o + (part + r) * D + c * 4) = a;
                    if (c == 0) *reinterpret_cast<float2*>(p.part_ml + (part + r) * 2) = make_float2(M, sum);
                }
            }

            fence_proxy_async_smem();                // what was written into the stage comes before the next copies
        }
        if (mask) fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.bar_empty[s]);
        more = paged_step(p, at, sp, kTile, end);
        if (done && more) {
            first = 0;
            part_i = i + 1;
            if (!set_up()) return;
        }
    }
}

// Joins the parts of the items that more than one block worked on, in the order of the list, and
// writes the rows of sequences that have no tiles.  One warp to a row, a lane to four columns (and,
// with D = 64, the halves of the warp to every other part).  Its blocks may start while the decode
// kernel's last ones run (8.9 against 10.9 us a call of one sequence); the same for the kernels before
// and after gained nothing.
constexpr int kCombineWarps = 4;

template <int D, int kTile, int kRows>
__global__ void __launch_bounds__(32 * kCombineWarps)
paged_combine_kernel(const __grid_constant__ PagedParams p) {
    constexpr int kPerRow = D / 4, kGroups = 32 / kPerRow;
    wait_prerequisites();
    const int x = blockIdx.x % (p.Hkv * p.RB), b = blockIdx.x / (p.Hkv * p.RB);
    const int h = x / p.RB, rb = x - h * p.RB;
    const int lane = threadIdx.x & 31;
    const int r = blockIdx.y * kCombineWarps + (threadIdx.x >> 5);
    const int c = lane % kPerRow, g = lane / kPerRow;
    if (r >= kRows || rb * kRows + r >= p.R) return;
    const int chunk = p.prefix[p.B + 1], in_b = p.prefix[b];
    const int n_tiles = paged_seq_span(p, b, kTile).n_tiles;
    const int first = in_b + x * paged_item(p, n_tiles);          // the item's place in the list
    float M = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (n_tiles > 0) {
        const int from = (first + p.item_cost) / chunk, to = (first + paged_item(p, n_tiles) - 1) / chunk;
        if (from == to) return;                        // one block had the whole item
        auto row_of = [&](int s) { return (2 * (size_t)s + (first > s * chunk)) * kRows + r; };
        for (int s = from + lane; s <= to; s += 32) M = fmaxf(M, p.part_ml[row_of(s) * 2]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        const float mu = M == -INFINITY ? 0.f : M;
        for (int s0 = from; s0 <= to; s0 += 32) {
            const int n = min(32, to - s0 + 1);
            float w = 0.f;
            if (lane < n) {
                const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + row_of(s0 + lane) * 2);
                w = ex2_approx(ml.x - mu);
                l += ml.y == 0.f ? 0.f : w * ml.y;
                if (ml.y == 0.f) w = 0.f;
            }
#pragma unroll 4
            for (int j = 0; j < n; j += kGroups) {
                const float wj = __shfl_sync(0xffffffffu, w, j + g);
                if (j + g < n && wj != 0.f) {          // a part without a visible key may hold anything
                    const float4 a = *reinterpret_cast<const float4*>(p.part_o + row_of(s0 + j + g) * D + c * 4);
                    acc.x += wj * a.x;
                    acc.y += wj * a.y;
                    acc.z += wj * a.z;
                    acc.w += wj * a.w;
                }
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        if (kGroups > 1) {
            acc.x += __shfl_xor_sync(0xffffffffu, acc.x, 16);
            acc.y += __shfl_xor_sync(0xffffffffu, acc.y, 16);
            acc.z += __shfl_xor_sync(0xffffffffu, acc.z, 16);
            acc.w += __shfl_xor_sync(0xffffffffu, acc.w, 16);
        }
    }
    if (g > 0) return;
    const int row = rb * kRows + r, head = h * p.G + row / p.N, node = row % p.N;
    const bool any = l != 0.f;
    const float inv = any ? 1.f / l : 0.f;
    __nv_bfloat16* dst = p.o + b * p.o_str.b + (long long)head * p.o_str.h + node * p.o_str.t + c * 4;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (c == 0) p.lse[((size_t)b * p.H + head) * p.N + node] = any ? (M + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace gpt_attn
