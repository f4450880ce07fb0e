// Attention of a sequence's newest tokens over a paged key/value cache: one token, or a tree of
// drafted tokens (each node sees the cached tokens and its own ancestors), with key heads shared by
// groups of query heads, and optionally a window with sinks.
//
// The rows of one item are the N new tokens of the G query heads that share a key head: R = G * N
// rows against the same keys, in blocks of up to 64.  A key and a value of D elements (4 D bytes)
// serve 4 D R flops, R flops a byte, so up to some hundred rows HBM bounds the call, and the kernel
// is built to keep loads in flight:
//   - A producer warp brings tiles of 64 keys through a ring of shared-memory stages.  A row of a
//     page is D * 2 contiguous bytes wherever the page lies, so 16-byte asynchronous copies by row
//     address serve any page size; rows nobody sees are not read but zero-filled.  A tile's pages are
//     looked up while the tile before it is issued.
//   - All tiles of all (sequence, key head, row block) items form one list, cut into equal pieces,
//     one to a resident block (two to an SM): ragged batches and single long sequences fill the
//     GPU alike.  The ring runs on across items.  A piece that holds a whole item writes O and lse;
//     the others leave fp32 partial results, joined by paged_combine_kernel.
//   - Four warps compute: scores and P V on warp-level matrix instructions (16 rows x 16 keys a step;
//     a tcgen05 tile has 128 rows, of which a call has 1 to 64), the softmax in registers between
//     them.  In a block of 16 rows each warp takes a quarter of a tile's keys, with a softmax state of
//     its own, joined at the end of the item; of 32 rows, each pair of warps 16 rows; of 64 rows, each
//     warp 16 rows and all keys.
// Statistics and accumulators are fp32; P is rounded to bf16 for the second product, as in the
// forward kernel, while its sum is taken before the rounding.
#pragma once

#include "attn_fwd.cuh"
#include "paging.h"

namespace gpt_attn {

constexpr int kPagedComputeWarps = 4;
constexpr int kPagedCompute = 32 * kPagedComputeWarps;
constexpr int kPagedThreads = kPagedCompute + 32;             // and the producer warp
constexpr int kPagedBlocksPerSm = 2;
constexpr int kPagedLeastTiles = 1;      // tiles of a piece at least

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
    float* part_o;                // [2 * blocks, rows of a block, D]
    float* part_ml;               // [2 * blocks, rows of a block, 2]
    long long* prefix;            // [B + 1] first tile of each sequence in the list, then chunk
    int B, H, Hkv, G, N;
    int R, RB;                    // rows of an item, row blocks
    int page, max_pages, n_pages, cap;
    int window, sinks;
    float scale_log2;
    uint64_t timeout_ns;
};

__device__ __forceinline__ int paged_n_new(const PagedParams& p, int b) {
    return p.n_new ? clamp_int(__ldg(p.n_new + b), 0, p.N) : p.N;
}

__device__ __forceinline__ PagedSpan paged_seq_span(const PagedParams& p, int b) {
    return paged_span(__ldg(p.lens + b), paged_n_new(p, b), p.cap, p.window, p.sinks);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    const int bytes = valid ? 16 : 0;       // 0: the 16 bytes are zero-filled, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// Arrives on `bar` once all copies that this thread has issued have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

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
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
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

template <int D>
struct PagedCfg {
    static constexpr int kStages = D == 64 ? 6 : 3;               // of 16 KB (D = 64), 32 KB (D = 128)
    static constexpr int kRowBytes = D * 2;
    static constexpr int kTileBytes = kPagedTile * kRowBytes;
};

// What the computing warps have to know of one tile.
struct PagedTile {
    unsigned long long present;   // keys of the tile that were read
    int b, x;                     // sequence; key head * RB + row block
    int key0, L;
    int n_b;                      // new tokens of the sequence
    int first, last;              // first / last tile of this block's part of the item
    int whole;                    // the block has the whole item
    int mask;                     // some row may not see some key that was read
};

template <int D>
struct PagedSmem {
    using C = PagedCfg<D>;
    alignas(128) uint8_t kv[C::kStages][2 * C::kTileBytes];       // keys, then values
    PagedTile tile[C::kStages];
    uint64_t bar_full[C::kStages], bar_empty[C::kStages];
    uint64_t bar_join;
    unsigned long long anc[kMaxNodes];
    int depth[kMaxNodes];
    int parents[kMaxNodes];
    float m[2][kPagedComputeWarps][16], l[2][kPagedComputeWarps][16];
    __nv_bfloat16 p[kPagedComputeWarps][16 * kPagedTile];
    int odd[2][kPagedComputeWarps];
    long long scan[kPagedThreads / 32];
    long long start_prefix;
    int start_b;
    int abort;
};

// Tiles of the list that sequence b contributes.
__device__ __forceinline__ long long paged_seq_tiles(const PagedParams& p, int b) {
    return (long long)paged_seq_span(p, b).n_tiles * p.Hkv * p.RB;
}

template <int D, int MT>
__global__ void __launch_bounds__(kPagedThreads, kPagedBlocksPerSm)
paged_decode_kernel(const __grid_constant__ PagedParams p) {
    using C = PagedCfg<D>;
    constexpr int kStages = C::kStages;
    constexpr int KS = kPagedComputeWarps / MT;      // warps that share a 16-row tile's keys
    constexpr int NT = kPagedTile / KS / 8;          // 8-key columns of a warp
    constexpr int kChunks = D / 8;                   // 16-byte chunks of a row
    constexpr int kRows = 16 * MT;
    constexpr int kWarps = kPagedThreads / 32;
    extern __shared__ uint8_t smem_raw[];
    PagedSmem<D>& sm = *reinterpret_cast<PagedSmem<D>*>(smem_align1024(smem_raw));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;");

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sm.bar_full[s], 64);          // each producer lane: its copies, and its writes
            mbar_init(&sm.bar_empty[s], kPagedComputeWarps);
        }
        mbar_init(&sm.bar_join, kPagedComputeWarps);
        sm.abort = 0;
        fence_barrier_init();
    }
    if (!p.parents && tid < p.N) {                   // one after the other: the same for all sequences
        sm.anc[tid] = (2ull << tid) - 1;
        sm.depth[tid] = tid;
    }

    // ---- this block's piece of the list
    long long total = 0;
    for (int b = tid; b < p.B; b += kPagedThreads) total += paged_seq_tiles(p, b);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    if (lane == 0) sm.scan[warp] = total;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += sm.scan[w];
    const long long chunk = paged_chunk(total, gridDim.x, kPagedLeastTiles);
    const long long begin = chunk * blockIdx.x;
    const int n_mine = (int)max(0ll, min(chunk, total - begin));
    {
        long long before = 0;
        for (int base = 0; base < p.B; base += kPagedThreads) {
            const int b = base + tid;
            const long long mine = b < p.B ? paged_seq_tiles(p, b) : 0;
            long long inc = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, inc, off);
                if (lane >= off) inc += y;
            }
            __syncthreads();
            if (lane == 31) sm.scan[warp] = inc;
            __syncthreads();
            inc += before;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) inc += sm.scan[w];
                before += sm.scan[w];
            }
            if (b < p.B && begin >= inc - mine && begin < inc) {
                sm.start_b = b;
                sm.start_prefix = inc - mine;
            }
            if (blockIdx.x == 0 && b < p.B) p.prefix[b] = inc - mine;
        }
        if (blockIdx.x == 0 && tid == 0) {
            p.prefix[p.B] = total;
            p.prefix[p.B + 1] = chunk;
        }
        __syncthreads();
    }
    if (n_mine == 0) return;
    const AbortCtl ac{&sm.abort, p.timeout_ns};

    if (warp == kPagedComputeWarps) {
        // ================ producer: walks the piece, one tile a step
        int b = sm.start_b, x, t, first;             // item (b, x), tile t; first: this part's first tile
        PagedSpan sp = paged_seq_span(p, b);
        int n_b = paged_n_new(p, b);
        {
            const long long in_b = begin - sm.start_prefix;
            x = (int)(in_b / sp.n_tiles);
            t = first = (int)(in_b % sp.n_tiles);
        }
        // rows in the pools of this lane's two keys of the current tile
        auto rows_of = [&](int& r0, int& r1) {
            const int key = sp.tile(t) * kPagedTile + lane;
            const int* table = p.table + (size_t)b * p.max_pages;
            r0 = sp.needs(key, p.sinks) ? paged_row(table, key, p.page, p.n_pages, p.Hkv, x / p.RB) : -1;
            r1 = sp.needs(key + 32, p.sinks) ? paged_row(table, key + 32, p.page, p.n_pages, p.Hkv, x / p.RB) : -1;
        };
        int r0, r1;
        rows_of(r0, r1);
        for (int i = 0; i < n_mine; ++i) {
            const int s = i % kStages;
            PagedTile d;
            d.b = b;
            d.x = x;
            d.key0 = sp.tile(t) * kPagedTile;
            d.L = sp.L;
            d.n_b = n_b;
            d.first = t == first;
            d.last = i == n_mine - 1 || t == sp.n_tiles - 1;
            d.whole = first == 0 && t == sp.n_tiles - 1;
            // every node stands at most n - 1 past L, so keys within the window of that position are
            // within everybody's
            d.mask = d.key0 + kPagedTile > sp.L || (p.window > 0 && sp.L + sp.n - 1 - d.key0 >= p.window);
            // the next tile's pages
            int n0 = -1, n1 = -1;
            if (i + 1 < n_mine) {
                if (++t == sp.n_tiles) {
                    t = first = 0;
                    if (++x == p.Hkv * p.RB) {
                        x = 0;
                        do sp = paged_seq_span(p, ++b);
                        while (sp.n_tiles == 0);
                        n_b = sp.n;
                    }
                }
                rows_of(n0, n1);
            }
            if (i >= kStages && !warp_wait(&sm.bar_empty[s], ((i / kStages) - 1) & 1, ac)) break;
            d.present = __ballot_sync(0xffffffffu, r0 >= 0) | (unsigned long long)__ballot_sync(0xffffffffu, r1 >= 0) << 32;
            if (lane == 0) sm.tile[s] = d;
            constexpr int kAtOnce = 32 / kChunks;    // rows a warp copies at once
            const int c = lane % kChunks;
            const uint32_t kd = smem_u32(sm.kv[s]), vd = kd + C::kTileBytes;
            const __nv_bfloat16 *kc = p.k + c * 8, *vc = p.v + c * 8;
#pragma unroll
            for (int j = 0; j < kPagedTile / kAtOnce; ++j) {
                const int r = j * kAtOnce + lane / kChunks;
                const int row = __shfl_sync(0xffffffffu, j < 32 / kAtOnce ? r0 : r1, r & 31);
                const size_t src = (size_t)max(row, 0) * D;
                const uint32_t dst = r * C::kRowBytes + ((c ^ (r & 7)) << 4);
                cp_async16(kd + dst, kc + src, row >= 0);
                cp_async16(vd + dst, vc + src, row >= 0);
            }
            cp_async_arrive(&sm.bar_full[s]);
            mbar_arrive(&sm.bar_full[s]);
            r0 = n0;
            r1 = n1;
        }
        cp_async_wait_all();
        return;
    }

    // ================ computing warps
    // state of the current item: two rows per thread (r and r + 8 of the warp's 16)
    const int mt = warp / KS, ks = warp % KS;
    uint32_t qf[D / 16][4];
    float oacc[D / 8][4];
    float m[2], l[2];
    int pos[2];
    unsigned long long anc[2];
    int cur_b = -1, part_i = 0, item = 0;            // part_i: the part's first tile
    const int r_lo = mt * 16 + (lane >> 2);
    uint32_t joins = 0;
    // a barrier of the computing warps
    auto join = [&]() -> bool {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.bar_join);
        return warp_wait(&sm.bar_join, joins++ & 1, ac);
    };

    for (int i = 0; i < n_mine; ++i) {
        const int s = i % kStages;
        if (!warp_wait(&sm.bar_full[s], (i / kStages) & 1, ac)) return;
        const PagedTile t = sm.tile[s];
        const int h = t.x / p.RB, rb = t.x - h * p.RB;
        if (t.first) {
            part_i = i;
            if (p.parents && t.b != cur_b) {
                // the tree of this sequence
                cur_b = t.b;
                if (!join()) return;                 // the last sequence's is no longer read
                if (tid < p.N) sm.parents[tid] = __ldg(p.parents + (size_t)t.b * p.N + tid);
                if (!join()) return;
                if (tid < p.N) {
                    const unsigned long long a = paged_ancestors(tid, sm.parents);
                    sm.anc[tid] = a;
                    sm.depth[tid] = __popcll(a) - 1;
                }
                if (!join()) return;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = rb * 64 + r_lo + 8 * e;
                const int node = r % p.N;
                const bool live = r < p.R && node < t.n_b;
                anc[e] = live ? sm.anc[node] : 0;
                pos[e] = t.L + sm.depth[node];
                m[e] = -INFINITY;
                l[e] = 0.f;
                const __nv_bfloat16* src = p.q + t.b * p.q_str.b + (long long)(h * p.G + (live ? r / p.N : 0)) * p.q_str.h +
                                           node * p.q_str.t + (lane & 3) * 2;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    qf[kk][e] = live ? *reinterpret_cast<const uint32_t*>(src + kk * 16) : 0u;
                    qf[kk][e + 2] = live ? *reinterpret_cast<const uint32_t*>(src + kk * 16 + 8) : 0u;
                }
            }
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) oacc[n][e] = 0.f;
        }

        // ---- scores of this warp's keys
        const uint8_t* kt = sm.kv[s];
        const uint8_t* vt = sm.kv[s] + C::kTileBytes;
        const int kb = ks * (kPagedTile / KS);        // first key of the warp within the tile
        float sc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
        {
            const int key = kb + (lane & 7) + ((lane >> 4) << 3);
            const uint32_t base = smem_u32(kt) + key * C::kRowBytes;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const int c = kk * 2 + ((lane >> 3) & 1);
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                    uint32_t b4[4];
                    ldmatrix4(b4, base + n * 8 * C::kRowBytes + ((c ^ (key & 7)) << 4));
                    mma_16816(sc[n], qf[kk], b4[0], b4[1]);
                    mma_16816(sc[n + 1], qf[kk], b4[2], b4[3]);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[n][e] *= p.scale_log2;
        // keys behind the cached tokens, at a window's edge or on missing pages; rows of nodes that
        // do not exist see nothing anywhere, which the end of the item takes care of
        if (t.mask || ~t.present) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = kb + n * 8 + (lane & 3) * 2 + (e & 1);
                    const bool see = ((t.present >> key) & 1) && paged_sees(t.key0 + key, pos[e >> 1], anc[e >> 1], sm.depth,
                                                                           t.L, p.window, p.sinks);
                    sc[n][e] = see ? sc[n][e] : -INFINITY;
                }
        }
        // ---- online softmax: rescaled only where a row's maximum grows by more than 2^8
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            mx[0] = fmaxf(mx[0], fmaxf(sc[n][0], sc[n][1]));
            mx[1] = fmaxf(mx[1], fmaxf(sc[n][2], sc[n][3]));
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
        }
        const bool grow0 = mx[0] > m[0] + kLazyRescale, grow1 = mx[1] > m[1] + kLazyRescale;
        if (__any_sync(0xffffffffu, grow0 || grow1)) {
            const float a0 = grow0 ? ex2_approx(m[0] - mx[0]) : 1.f, a1 = grow1 ? ex2_approx(m[1] - mx[1]) : 1.f;
            if (grow0) m[0] = mx[0];
            if (grow1) m[1] = mx[1];
            l[0] *= a0;
            l[1] *= a1;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
                oacc[n][0] *= a0;
                oacc[n][1] *= a0;
                oacc[n][2] *= a1;
                oacc[n][3] *= a1;
            }
        }
        const float mu0 = m[0] == -INFINITY ? 0.f : m[0], mu1 = m[1] == -INFINITY ? 0.f : m[1];
        uint32_t pf[NT / 2][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float p0 = ex2_approx(sc[n][0] - mu0), p1 = ex2_approx(sc[n][1] - mu0);
            const float p2 = ex2_approx(sc[n][2] - mu1), p3 = ex2_approx(sc[n][3] - mu1);
            l[0] += p0 + p1;
            l[1] += p2 + p3;
            pf[n / 2][(n & 1) * 2] = pack_bf16x2(p0, p1);
            pf[n / 2][(n & 1) * 2 + 1] = pack_bf16x2(p2, p3);
        }
        // New tokens that are not every node's ancestors may hold infinities or NaN, which must not
        // reach the others through 0 * NaN.  Where a tile holds some, they are added to the rows with
        // P > 0 one by one and then cleared in the stage.
        if (t.mask && p.N > 1) {
            uint4* rows = reinterpret_cast<uint4*>(sm.kv[s] + C::kTileBytes);
            bool odd = false;
#pragma unroll 4
            for (int c = tid; c < kPagedTile * kChunks; c += kPagedCompute) {
                const uint4 x = rows[c];
                odd = odd || not_finite(x.x) || not_finite(x.y) || not_finite(x.z) || not_finite(x.w);
            }
            odd = __any_sync(0xffffffffu, odd);
            int(&all)[kPagedComputeWarps] = sm.odd[joins & 1];    // a warp may be a join ahead of the readers
            if (lane == 0) all[warp] = odd;
            if (!join()) return;
            odd = all[0] | all[1] | all[2] | all[3];
            if (odd) {
                __nv_bfloat16(*pw)[NT * 8] = reinterpret_cast<__nv_bfloat16(*)[NT * 8]>(sm.p[warp]);
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
                    for (int kk = 0; kk < NT * 8; ++kk) {
                        const int key = kb + kk;
                        const uint32_t w = *reinterpret_cast<const uint32_t*>(
                            vt + key * C::kRowBytes + ((n ^ (key & 7)) << 4) + (lane & 3) * 4);
                        if (!not_finite(w)) continue;
                        const float x0 = __uint_as_float(w << 16), x1 = __uint_as_float(w & 0xffff0000u);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            if (__bfloat162float(pw[(lane >> 2) + 8 * e][kk]) == 0.f) continue;
                            if (!isfinite(x0)) oacc[n][2 * e] += x0;
                            if (!isfinite(x1)) oacc[n][2 * e + 1] += x1;
                        }
                    }
                if (!join()) return;
                for (int c = tid; c < kPagedTile * kChunks; c += kPagedCompute) {
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
            const uint32_t base = smem_u32(vt) + key * C::kRowBytes;
#pragma unroll
            for (int kk = 0; kk < NT / 2; ++kk) {
#pragma unroll
                for (int n = 0; n < D / 16; ++n) {
                    const int c = n * 2 + (lane >> 4);
                    uint32_t b4[4];
                    ldmatrix4_trans(b4, base + kk * 16 * C::kRowBytes + ((c ^ (key & 7)) << 4));
                    mma_16816(oacc[2 * n], pf[kk], b4[0], b4[1]);
                    mma_16816(oacc[2 * n + 1], pf[kk], b4[2], b4[3]);
                }
            }
        }

        if (t.last) {
            // ---- end of the item (or of this block's part)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
                if (anc[e] == 0) {                   // a row or node that does not exist sees nothing
                    m[e] = -INFINITY;
                    l[e] = 0.f;
                }
            }
            // a piece has at most two partial items: the one it starts in and the one it ends in
            const size_t part = (2 * (size_t)blockIdx.x + (part_i > 0)) * kRows;
            auto out_row = [&](int r, int& head, int& node) {
                head = h * p.G + (rb * 64 + r) / p.N;
                node = (rb * 64 + r) % p.N;
                return p.o + t.b * p.o_str.b + (long long)head * p.o_str.h + node * p.o_str.t;
            };
            if constexpr (KS > 1) {
                // The warps that share rows join their states through the stage itself, which they
                // have all read by then.  (The statistics alternate between two buffers: a warp may
                // be an item ahead of those that still read the last one's.)
                const int par = item++ & 1;
                if ((lane & 3) == 0) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        sm.m[par][warp][(lane >> 2) + 8 * e] = m[e];
                        sm.l[par][warp][(lane >> 2) + 8 * e] = l[e];
                    }
                }
                if (!join()) return;
                float2* mine = reinterpret_cast<float2*>(sm.kv[s]) + (size_t)warp * 16 * (D / 2);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = (lane >> 2) + 8 * e;
                    if (anc[e] == 0) continue;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n)
                        mine[r * (D / 2) + ((n * 4 + (lane & 3)) ^ ((r & 3) * 4))] =
                            make_float2(oacc[n][2 * e], oacc[n][2 * e + 1]);
                }
                if (!join()) return;
                const int n_rows = min(p.R - rb * 64, kRows);
                for (int at = tid; at < n_rows * (D / 4); at += kPagedCompute) {
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
                        const float f = ex2_approx(sm.m[par][w0 + w][rr] - mu);
                        sum += lw == 0.f ? 0.f : lw * f;
                        if (lw != 0.f) {             // a warp whose keys the row does not see wrote nothing of use
                            const float4 y = *reinterpret_cast<const float4*>(
                                reinterpret_cast<const float2*>(sm.kv[s]) + (size_t)(w0 + w) * 16 * (D / 2) + rr * (D / 2) +
                                ((c * 2) ^ ((rr & 3) * 4)));
                            a.x += f * y.x;
                            a.y += f * y.y;
                            a.z += f * y.z;
                            a.w += f * y.w;
                        }
                    }
                    const bool any = sum != 0.f;
                    if (t.whole) {
                        int head, node;
                        __nv_bfloat16* dst = out_row(r, head, node) + c * 4;
                        const float inv = any ? 1.f / sum : 0.f;
                        *reinterpret_cast<uint2*>(dst) =
                            make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
                        if (c == 0)
                            p.lse[((size_t)t.b * p.H + head) * p.N + node] =
                                any ? (M + log2f(sum)) * 0.69314718055994531f : -INFINITY;
                    } else {
                        *reinterpret_cast<float4*>(p.part_o + (part + r) * D + c * 4) = a;
                        if (c == 0) *reinterpret_cast<float2*>(p.part_ml + (part + r) * 2) = make_float2(M, sum);
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = r_lo + 8 * e;
                    if (rb * 64 + r >= p.R) continue;
                    const bool any = l[e] != 0.f;
                    if (t.whole) {
                        int head, node;
                        __nv_bfloat16* dst = out_row(r, head, node) + (lane & 3) * 2;
                        const float inv = any ? 1.f / l[e] : 0.f;
#pragma unroll
                        for (int n = 0; n < D / 8; ++n)
                            *reinterpret_cast<uint32_t*>(dst + n * 8) =
                                any ? pack_bf16x2(oacc[n][2 * e] * inv, oacc[n][2 * e + 1] * inv) : 0u;
                        if ((lane & 3) == 0)
                            p.lse[((size_t)t.b * p.H + head) * p.N + node] =
                                any ? (m[e] + log2f(l[e])) * 0.69314718055994531f : -INFINITY;
                    } else {
                        float* dst = p.part_o + (part + r) * D + (lane & 3) * 2;
#pragma unroll
                        for (int n = 0; n < D / 8; ++n)
                            *reinterpret_cast<float2*>(dst + n * 8) = make_float2(oacc[n][2 * e], oacc[n][2 * e + 1]);
                        if ((lane & 3) == 0)
                            *reinterpret_cast<float2*>(p.part_ml + (part + r) * 2) = make_float2(m[e], l[e]);
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.bar_empty[s]);
    }
}

// Joins the parts of the items that more than one block worked on, in the order of the list, and
// writes the rows of sequences that have no tiles.  One warp to a row, a lane to four columns (and,
// with D = 64, the halves of the warp to every other part).  Launched so that its blocks may start
// while the decode kernel's last ones run; they wait for its end first.
constexpr int kCombineWarps = 4;

template <int D, int MT>
__global__ void __launch_bounds__(32 * kCombineWarps)
paged_combine_kernel(const __grid_constant__ PagedParams p) {
    constexpr int kRows = 16 * MT;
    constexpr int kPerRow = D / 4, kGroups = 32 / kPerRow;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int x = blockIdx.x % (p.Hkv * p.RB), b = blockIdx.x / (p.Hkv * p.RB);
    const int h = x / p.RB, rb = x - h * p.RB;
    const int lane = threadIdx.x & 31;
    const int r = blockIdx.y * kCombineWarps + (threadIdx.x >> 5);
    const int c = lane % kPerRow, g = lane / kPerRow;
    if (rb * 64 + r >= p.R) return;
    const long long chunk = p.prefix[p.B + 1], in_b = p.prefix[b];
    const int n_tiles = paged_seq_span(p, b).n_tiles;
    const long long first = in_b + (long long)x * n_tiles;
    float M = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (n_tiles > 0) {
        const int from = (int)(first / chunk), to = (int)((first + n_tiles - 1) / chunk);
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
    const int row = rb * 64 + r, head = h * p.G + row / p.N, node = row % p.N;
    const bool any = l != 0.f;
    const float inv = any ? 1.f / l : 0.f;
    __nv_bfloat16* dst = p.o + b * p.o_str.b + (long long)head * p.o_str.h + node * p.o_str.t + c * 4;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (c == 0) p.lse[((size_t)b * p.H + head) * p.N + node] = any ? (M + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace gpt_attn
