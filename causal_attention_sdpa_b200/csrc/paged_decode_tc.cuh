// The paged decode kernel for items of many rows (trees of drafts, groups of query heads): the same
// list, pieces, teams and producers as in paged_decode.cuh, the products on tcgen05 tiles of 128 rows.
//
// An item's rows, in blocks of up to 128, are the rows of one Q tile in shared memory.  For each tile of
// 64 keys an MMA warp issues S = Q K^T into one of two TMEM buffers, four softmax warps (a thread to a
// row) turn S into P in place, and the MMA warp issues O += P V; S of the next tile is issued before P of
// this one is waited for, so the tensor work hides behind the softmax.  The keys' slot is free once S is
// done, the values' once O is.  Another warp brings the next item's rows in while the last tile of this
// one is in the softmax.
//
// What bounds it: HBM for long items, else what comes before and after the tiles (rows, masks, joining).  A
// tile's softmax takes a warp some 1600 cycles whatever its rows, so what counts is that all rows of an item share one tile, and that the two teams of a block do not wait for one
// another: with 64 rows or fewer only two warps of a team have rows, and the second team's rows are put
// at the other end of its tile, where the other two sub-partitions of the SM read them.
// Measured on one B200: 13 drafts over 16 streams up to 32768 (24 query heads on 6 of 128, window 4096) 52 us,
// 4.0 TB/s; the same without a window over 16 contexts of 16384 167 us, 4.8 TB/s.
//
// Masks are words of 32 keys, as in the other kernel.  Rows that came along in a box unseen are cleared,
// and infinities and NaN of drafts, which other nodes must not see through 0 * NaN, are cleared too and
// noted for each row that does see them (one bit a column), to be added to O at the end.
#pragma once

#include "paged_decode.cuh"

namespace gpt_attn {

constexpr int kPagedTcRows = 128;
constexpr int kPagedTcTile = 64;
constexpr int kPagedTcThreads = 512;     // two teams' softmax warps, the producers, the MMA and row warps
// Registers of a thread: 128 at the launch; 80 for the two warpgroups of producers, MMA and row warps,
// 176 for the softmax's.
constexpr int kPagedTcHelperRegs = 80, kPagedTcSoftmaxRegs = 176;

template <int D>
struct PagedTcTeam {
    static constexpr int kSlots = D == 64 ? 4 : 2;
    static constexpr int kRing = 8;                               // tile descriptions outlive the keys' slot
    static constexpr int kTileBytes = kPagedTcTile * D * 2;
    static constexpr int kQBytes = kPagedTcRows * D * 2;
    alignas(1024) uint8_t k[kSlots][kTileBytes];
    alignas(1024) uint8_t v[kSlots][kTileBytes];
    alignas(1024) uint8_t q[kQBytes];
    PagedTile tile[kRing];
    uint64_t tile_full[kRing];
    uint64_t k_full[kSlots], k_empty[kSlots], v_full[kSlots], v_empty[kSlots];
    uint64_t q_first;             // the first item's rows are in
    uint64_t q_full, q_empty;     // the next item's rows are in; all S of an item are done
    uint64_t s_full[2], p_full[2], o_done[2];                     // of tiles in either S buffer
    uint64_t o_free;              // the item's O has been read
    uint64_t bar_join, bar_drain;
    unsigned long long anc[2][kMaxNodes];                         // the tree, of alternate sequences
    int depth[2][kMaxNodes];
    uint32_t inf[2][kPagedTcTile][D / 32];                        // columns of a key with +inf or NaN, and -inf or NaN
    int odd[2][kPagedTeamWarps];
    PagedAt start;
};

template <int D>
struct PagedTcSmem {
    PagedTcTeam<D> team[kPagedTeams];
    int scan[kPagedTcThreads / 32];
    uint32_t tmem;
    int abort;
};

// The first tile of the item after `at`; false at the end of the piece.
__device__ __forceinline__ bool paged_next_item(const PagedParams& p, PagedAt& at, PagedSpan& sp, int tile, int end) {
    at.pos += sp.n_tiles - 1 - at.t;
    at.t = sp.n_tiles - 1;
    return paged_step(p, at, sp, tile, end);
}

// The rows of item `at` into the Q tile, K-major with the 128-byte swizzle; row r of the block at tile row
// (r + first) % 128.  Warp `part` of `parts` takes every parts-th group of 16 rows.
template <int D>
__device__ __forceinline__ void paged_tc_rows(const PagedParams& p, uint8_t* q, const PagedAt& at, const PagedSpan& sp,
                                              int first, int part, int parts) {
    const int lane = threadIdx.x & 31;
    const int r0 = at.rb * kPagedTcRows, n = min(p.R - r0, kPagedTcRows);
    for (int base = part * 16; base < n; base += parts * 16) {
        uint4 raw[D / 64][4];                        // a row's 64 columns to 8 lanes
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = base + j * 4 + (lane >> 3), hd = p.by_n.div(r0 + r), nd = r0 + r - hd * p.N;
            const bool live = r < n && nd < sp.n;
            const __nv_bfloat16* src = p.q + at.b * p.q_str.b + (long long)(at.h * p.G + hd) * p.q_str.h + nd * p.q_str.t +
                                       (lane & 7) * 8;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
                raw[c][j] = live ? __ldg(reinterpret_cast<const uint4*>(src + c * 64)) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = base + j * 4 + (lane >> 3), row = (r + first) % kPagedTcRows;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                uint4 x = raw[c][j];
                x.x = x.x & p.q_keep ^ p.q_flip;
                x.y = x.y & p.q_keep ^ p.q_flip;
                x.z = x.z & p.q_keep ^ p.q_flip;
                x.w = x.w & p.q_keep ^ p.q_flip;
                *reinterpret_cast<uint4*>(q + c * kPagedTcRows * 128 + row * 128 + (((lane & 7) ^ (row & 7)) << 4)) = x;
            }
        }
    }
    fence_proxy_async_smem();
    __syncwarp();
}

// Row warp: brings in the rows of each item after the first once S of the last one is done.
template <int D>
__device__ __forceinline__ void paged_tc_next_rows(const PagedParams& p, PagedTcTeam<D>& sm, int first, int end,
                                                   const AbortCtl& ac) {
    PagedAt at = sm.start;
    PagedSpan sp = paged_seq_span(p, at.b, kPagedTcTile);
    for (int item = 0; paged_next_item(p, at, sp, kPagedTcTile, end); ++item) {
        if (!warp_wait(&sm.q_empty, item & 1, ac)) return;
        paged_tc_rows<D>(p, sm.q, at, sp, first, 0, 1);
        if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.q_full);
    }
}

// MMA warp (one lane): S of tile u + 1, then O of tile u; at an item's end the other way round, since the
// next item's rows come only once S of the last tile is done.
template <int D>
__device__ __forceinline__ void paged_tc_mma(const PagedParams& p, PagedTcTeam<D>& sm, uint32_t tmem, int end,
                                             const AbortCtl& ac) {
    constexpr int kSlots = PagedTcTeam<D>::kSlots;
    constexpr uint32_t kIdescS = idesc_bf16_f32(128, kPagedTcTile, 0, 0), kIdescO = idesc_bf16_f32(128, D, 0, 1);
    constexpr int kHalf = kPagedTcTile * 128;        // 64 columns of a tile's keys
    const uint32_t col_o = tmem, col_s = tmem + 128;
    PagedAt at = sm.start;
    PagedSpan sp = paged_seq_span(p, at.b, kPagedTcTile);
    int s_item = 0;                                  // items S has begun
    auto issue_s = [&](int u, bool first, bool last) -> bool {
        if (first && !(s_item++ == 0 ? mbar_wait(&sm.q_first, 0, ac) : mbar_wait(&sm.q_full, s_item & 1, ac))) return false;
        const int s = u % kSlots;
        if (!mbar_wait(&sm.k_full[s], (u / kSlots) & 1, ac)) return false;
        if (u >= 2 && !mbar_wait(&sm.o_done[u & 1], ((u >> 1) - 1) & 1, ac)) return false;  // P of tile u - 2 was here
        tc_fence_after();
        const uint32_t q = smem_u32(sm.q), k = smem_u32(sm.k[s]);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(col_s + (u & 1) * kPagedTcTile, sw128_desc(q + (kk >> 2) * (kPagedTcRows * 128) + (kk & 3) * 32, 16, 1024),
                   sw128_desc(k + (kk >> 2) * kHalf + (kk & 3) * 32, 16, 1024), kIdescS, kk > 0);
        mma_commit(&sm.s_full[u & 1]);
        mma_commit(&sm.k_empty[s]);
        if (last) mma_commit(&sm.q_empty);
        return true;
    };
    int o_item = 0;                                  // items O has begun
    auto issue_o = [&](int u, bool first) -> bool {
        const int s = u % kSlots;
        if (!mbar_wait(&sm.v_full[s], (u / kSlots) & 1, ac)) return false;
        if (first && o_item++ > 0 && !mbar_wait(&sm.o_free, o_item & 1, ac)) return false;
        if (!mbar_wait(&sm.p_full[u & 1], (u >> 1) & 1, ac)) return false;
        tc_fence_after();
        const uint32_t v = smem_u32(sm.v[s]);
#pragma unroll
        for (int kk = 0; kk < kPagedTcTile / 16; ++kk)
            mma_ts(col_o, col_s + (u & 1) * kPagedTcTile + kk * 8, sw128_desc(v + kk * 2048, kHalf, 1024), kIdescO,
                   (!first || kk > 0) ? 1u : 0u);
        mma_commit(&sm.o_done[u & 1]);
        mma_commit(&sm.v_empty[s]);
        return true;
    };
    auto last_of = [&]() { return at.t == sp.n_tiles - 1 || at.pos + 1 >= end; };
    bool first = true, last = last_of();
    bool ok = issue_s(0, true, last), more = true;
    for (int u = 0; ok && more; ++u) {
        const bool o_first = first;
        more = paged_step(p, at, sp, kPagedTcTile, end);
        first = last;                                // the next tile begins an item where this one ended
        if (more) last = last_of();
        if (first || !more) {
            ok = issue_o(u, o_first) && (!more || issue_s(u + 1, true, last));
        } else {
            ok = issue_s(u + 1, false, last) && issue_o(u, o_first);
        }
    }
    mma_commit(&sm.bar_drain);
    mbar_wait_drain(&sm.bar_drain, 0, p.timeout_ns);
}

// Softmax warps of team g: thread t has tile row t, which is row (t - 64 g) % 128 of the row block.
template <int D>
__device__ __forceinline__ void paged_tc_softmax(const PagedParams& p, PagedTcTeam<D>& sm, uint32_t tmem, int g, int team_no,
                                                 int end, const AbortCtl& ac) {
    constexpr int kSlots = PagedTcTeam<D>::kSlots, kRing = PagedTcTeam<D>::kRing, kTile = kPagedTcTile;
    const int tid = threadIdx.x - g * kPagedTeam, lane = tid & 31, w4 = tid >> 5;
    const int r_loc = (tid + 64 * g) % kPagedTcRows;
    const uint32_t t_lane = tmem + ((uint32_t)(w4 * 32) << 16), t_s = t_lane + 128;
    PagedAt at = sm.start;
    PagedSpan sp = paged_seq_span(p, at.b, kTile);
    int cur_b = -1, tree = 0, first = at.t, part_u = 0;
    uint32_t joins = 0;
    auto join = [&]() -> bool {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.bar_join);
        return warp_wait(&sm.bar_join, joins++ & 1, ac);
    };
    // this thread's row of the current item
    int head, node, lower;
    bool exists, warp_rows;                          // the row exists; some row of the warp does
    unsigned long long vis;                          // 0: no such row, or no such node
    float m, l;
    uint32_t up[D / 32], down[D / 32];               // columns to which +inf and -inf are to be added
    auto set_up = [&]() -> bool {
        if (p.parents && at.b != cur_b) {
            tree ^= cur_b >= 0;
            cur_b = at.b;
            if (w4 == 0) paged_tree(p, at.b, sm.anc[tree], sm.depth[tree]);
            if (!join()) return false;
        }
        const int r = at.rb * kPagedTcRows + r_loc;
        head = p.by_n.div(r);
        node = r - head * p.N;
        exists = r < p.R;
        warp_rows = __any_sync(0xffffffffu, exists);
        const int pos = sp.L + sm.depth[tree][node];
        lower = paged_lower(pos, p.window);
        vis = exists && node < sp.n ? paged_visible(sm.anc[tree][node], pos, sm.depth[tree], sp.L, p.window, p.sinks) : 0;
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int w = 0; w < D / 32; ++w) up[w] = down[w] = 0;
        return true;
    };
    // the first item's rows: the row warp alone would take them 16 at a time
    paged_tc_rows<D>(p, sm.q, at, sp, 64 * g, w4, kPagedTeamWarps);
    if (lane == 0) mbar_arrive(&sm.q_first);
    if (!set_up()) return;
    bool more = true, begin = true;                  // begin: the item's first tile here
    for (int u = 0; more; ++u) {
        const int buf = u & 1;
        if (!warp_wait(&sm.tile_full[u % kRing], (u / kRing) & 1, ac)) return;
        if (!warp_wait(&sm.s_full[buf], (u >> 1) & 1, ac)) return;
        tc_fence_after();
        const PagedTile& t = sm.tile[u % kRing];
        const int mask = t.mask;
        const uint32_t col_s = t_s + buf * kTile;
        float s[kTile];
        if (warp_rows) {
            uint32_t a[32], b[32];
            tmem_ld32(col_s, a);
            tmem_ld32(col_s + 32, b);
            tmem_wait_ld_regs2(a, b);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                s[e] = __uint_as_float(a[e]);
                s[32 + e] = __uint_as_float(b[e]);
            }
            if (mask) {
                const int key0 = t.key0;
#pragma unroll
                for (int w = 0; w < kTile / 32; ++w) {
                    const uint32_t see = t.seen[w] & paged_sees(key0 + w * 32, sp.L, lower, p.sinks, vis);
#pragma unroll
                    for (int e = 0; e < 32; ++e) s[w * 32 + e] = (see >> e) & 1 ? s[w * 32 + e] : -INFINITY;
                }
            }
            float m0 = fmax3(s[0], s[1], s[2]), m1 = fmax3(s[3], s[4], s[5]);
#pragma unroll
            for (int e = 6; e < kTile - 2; e += 4) {
                m0 = fmax3(m0, s[e], s[e + 1]);
                m1 = fmax3(m1, s[e + 2], s[e + 3]);
            }
            const float mx = fmaxf(fmax3(m0, s[kTile - 2], s[kTile - 1]), m1) * p.scale_log2;
            const bool grow = mx > m + kLazyRescale;
            if (__any_sync(0xffffffffu, grow)) {
                const float alpha = grow ? ex2_approx(m - mx) : 1.f;
                if (grow) m = mx;
                l *= alpha;
                if (!begin) {
                    // O up to the last tile, rescaled in place
                    if (!warp_wait(&sm.o_done[buf ^ 1], ((u - 1) >> 1) & 1, ac)) return;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t x[32];
                        tmem_ld32(t_lane + c * 32, x);
                        tmem_wait_ld_regs(x);
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * alpha);
                        tmem_st32(t_lane + c * 32, x);
                    }
                    tmem_wait_st();
                }
            }
            const float mu = m == -INFINITY ? 0.f : m;
            float l0 = 0.f, l1 = 0.f;
            uint32_t pk[kTile / 2];
#pragma unroll
            for (int e = 0; e < kTile; e += 2) {
                s[e] = ex2_approx(fmaf(s[e], p.scale_log2, -mu));
                s[e + 1] = ex2_approx(fmaf(s[e + 1], p.scale_log2, -mu));
                l0 += s[e];
                l1 += s[e + 1];
                pk[e / 2] = pack_bf16x2(s[e], s[e + 1]);
            }
            l += l0 + l1;
            tmem_st32(col_s, pk);
        }
        if (mask) {
            const int slot = u % kSlots;
            if (!warp_wait(&sm.v_full[slot], (u / kSlots) & 1, ac)) return;
            const bool check = sp.differs(t.key0, kTile, p.window);
            bool odd = paged_clean<D, kTile, 1>(sm.v[slot], t, tid, check);
            if (check) {
                odd = __any_sync(0xffffffffu, odd);
                int(&any)[kPagedTeamWarps] = sm.odd[joins & 1];   // a warp may be a join ahead of the readers
                if (lane == 0) any[w4] = odd;
                if (!join()) return;
                if (any[0] | any[1] | any[2] | any[3]) {
                    // which columns of which keys, then their values cleared
                    for (int x = tid; x < kTile * (D / 32); x += kPagedTeam) {
                        const int key = x % kTile, w = x / kTile;
                        uint32_t plus = 0, minus = 0;
                        for (int c = 0; c < 4; ++c) {
                            uint4* at4 = reinterpret_cast<uint4*>(sm.v[slot] + paged_at<kTile>(key, w * 4 + c));
                            const uint4 y = *at4;
                            const uint32_t y4[4] = {y.x, y.y, y.z, y.w};
                            for (int e = 0; e < 8; ++e) {
                                const uint32_t h = y4[e >> 1] >> (e & 1 ? 16 : 0) & 0xffffu;
                                if ((h & 0x7f80u) != 0x7f80u) continue;
                                plus |= (h != 0xff80u ? 1u : 0u) << (c * 8 + e);
                                minus |= (h != 0x7f80u ? 1u : 0u) << (c * 8 + e);
                            }
                            *at4 = make_uint4(finite_bf16x2(y.x), finite_bf16x2(y.y), finite_bf16x2(y.z), finite_bf16x2(y.w));
                        }
                        sm.inf[0][key][w] = plus;
                        sm.inf[1][key][w] = minus;
                    }
                    unsigned long long has = 0;      // keys with P > 0, as it was rounded
                    if (warp_rows) {
#pragma unroll
                        for (int e = 0; e < kTile; ++e) has |= (unsigned long long)(__float2bfloat16_rn(s[e]) > __nv_bfloat16(0.f)) << e;
                    }
                    if (!join()) return;
                    while (has) {
                        const int key = __ffsll(has) - 1;
                        has &= has - 1;
#pragma unroll
                        for (int w = 0; w < D / 32; ++w) {
                            up[w] |= sm.inf[0][key][w];
                            down[w] |= sm.inf[1][key][w];
                        }
                    }
                    if (!join()) return;             // the table is read before another tile writes it
                }
            }
            fence_proxy_async_smem();
        }
        if (warp_rows) tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&sm.p_full[buf]);

        const bool done = at.t == sp.n_tiles - 1;
        if (done || at.pos + 1 >= end) {
            // ---- end of the item (or of this team's part)
            const bool whole = done && first == 0;
            const size_t row = (2 * (size_t)team_no + (part_u > 0)) * kPagedTcRows + r_loc;
            if (!warp_wait(&sm.o_done[buf], (u >> 1) & 1, ac)) return;
            tc_fence_after();
            if (warp_rows) {
                if (vis == 0) {
                    m = -INFINITY;
                    l = 0.f;
                }
                const bool any = l != 0.f;
                const float inv = whole ? (any ? 1.f / l : 0.f) : 1.f;
                const int hd = at.h * p.G + head;
                __nv_bfloat16* dst = p.o + at.b * p.o_str.b + (long long)hd * p.o_str.h + node * p.o_str.t;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t x[32];
                    tmem_ld32(t_lane + c * 32, x);
                    tmem_wait_ld_regs(x);
                    if (__any_sync(0xffffffffu, (up[c] | down[c]) != 0)) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            float y = __uint_as_float(x[e]);
                            if ((up[c] >> e) & 1) y += INFINITY;
                            if ((down[c] >> e) & 1) y -= INFINITY;
                            x[e] = __float_as_uint(y);
                        }
                    }
                    if (!exists) continue;
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint32_t y[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                y[k] = any ? pack_bf16x2(__uint_as_float(x[e + 2 * k]) * inv, __uint_as_float(x[e + 2 * k + 1]) * inv)
                                           : 0u;
                            *reinterpret_cast<uint4*>(dst + c * 32 + e) = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<uint4*>(p.part_o + row * D + c * 32 + e) =
                                make_uint4(x[e], x[e + 1], x[e + 2], x[e + 3]);
                    }
                }
                if (exists) {
                    if (whole)
                        p.lse[((size_t)at.b * p.H + hd) * p.N + node] = any ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
                    else
                        *reinterpret_cast<float2*>(p.part_ml + row * 2) = make_float2(m, l);
                }
            }
            tc_fence_before();
            mbar_arrive(&sm.o_free);
        }
        more = paged_step(p, at, sp, kTile, end);
        begin = done;
        if (done && more) {
            first = 0;
            part_u = u + 1;
            if (!set_up()) return;
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kPagedTcThreads, 1)
paged_decode_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ PagedParams p) {
    using Team = PagedTcTeam<D>;
    constexpr int kSlots = Team::kSlots;
    constexpr uint32_t kTmemCols = 512;              // a team: O [0, D), S [128, 256)
    extern __shared__ uint8_t smem_raw[];
    PagedTcSmem<D>& block = *reinterpret_cast<PagedTcSmem<D>*>(smem_align1024(smem_raw));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    launch_dependents();
    if (threadIdx.x == 0) {
        for (int g = 0; g < kPagedTeams; ++g) {
            Team& t = block.team[g];
            for (int s = 0; s < kSlots; ++s) {
                mbar_init(&t.k_full[s], 1);
                mbar_init(&t.k_empty[s], 1);
                mbar_init(&t.v_full[s], 1);
                mbar_init(&t.v_empty[s], 1);
            }
            for (int s = 0; s < Team::kRing; ++s) mbar_init(&t.tile_full[s], 1);
            mbar_init(&t.q_first, kPagedTeamWarps);
            mbar_init(&t.q_full, 1);
            mbar_init(&t.q_empty, 1);
            for (int b = 0; b < 2; ++b) {
                mbar_init(&t.s_full[b], 1);
                mbar_init(&t.p_full[b], kPagedTeam);
                mbar_init(&t.o_done[b], 1);
            }
            mbar_init(&t.o_free, kPagedTeam);
            mbar_init(&t.bar_join, kPagedTeamWarps);
            mbar_init(&t.bar_drain, 1);
        }
        block.abort = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (!p.parents && threadIdx.x < p.N) {           // one after the other: the same for all sequences
        for (int g = 0; g < kPagedTeams; ++g) {
            block.team[g].anc[0][threadIdx.x] = (2ull << threadIdx.x) - 1;
            block.team[g].depth[0][threadIdx.x] = threadIdx.x;
        }
    }
    if (warp == 12) {
        tmem_alloc(&block.tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    const PagedPiece piece =
        paged_cut<kPagedTcTile, kPagedTcThreads>(p, block.scan, &block.team[0].start, &block.team[1].start);
    tc_fence_after();
    const uint32_t tmem = block.tmem;
    const AbortCtl ac{&block.abort, p.timeout_ns};
    // warps 0-3 and 4-7: the teams' softmax; 8-11: keys and values of team 0, of team 1; 12, 13: the teams'
    // MMA; 14, 15: the teams' rows
    const int g = warp < 8 ? warp / 4 : (warp < 12 ? (warp - 8) / 2 : warp & 1);
    const int team_no = g * gridDim.x + blockIdx.x;
    const int end = (int)min((long long)piece.all, (long long)piece.chunk * (team_no + 1));
    const bool none = (long long)piece.chunk * team_no >= piece.all || block.team[g].start.pos >= end;
    Team& t = block.team[g];
    if (warp >= 8) {
        regs_dec<kPagedTcHelperRegs>();
        if (none) {
        } else if (warp < 12) {
            const int which = warp & 1;
            paged_produce<D, kPagedTcTile, kSlots, Team::kRing>(p, which ? &tm_v : &tm_k, which, t.start, end,
                                                                which ? t.v[0] : t.k[0], Team::kTileBytes,
                                                                which ? t.v_full : t.k_full, which ? t.v_empty : t.k_empty,
                                                                t.tile, t.tile_full, ac);
        } else if (warp < 14) {
            if (lane == 0) paged_tc_mma<D>(p, t, tmem + g * 256, end, ac);
        } else {
            paged_tc_next_rows<D>(p, t, 64 * g, end, ac);
        }
    } else {
        regs_inc<kPagedTcSoftmaxRegs>();
        if (!none) paged_tc_softmax<D>(p, t, tmem + g * 256, g, team_no, end, ac);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace gpt_attn
