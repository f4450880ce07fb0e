// Attention of a sequence's newest tokens over a paged key/value cache: one token, or a tree of
// drafted tokens (each node sees the cached tokens and its own ancestors), with key heads shared by
// groups of query heads, and optionally a window with sinks.
//
// The rows of one item are the N new tokens of the G query heads that share a key head: R = G * N
// rows against the same keys, in blocks of up to 64.  A key and a value of D elements (4 D bytes)
// serve 4 D R flops, R flops a byte, so up to some hundred rows HBM bounds the call, and the kernel
// is built to keep loads in flight:
//   - Tiles of 64 keys come through a ring of cp.async stages.  A row of a page is D * 2 contiguous
//     bytes wherever the page lies, so 16-byte copies by row address serve any page size; rows
//     nobody sees are not read but zero-filled.  A row's page is looked up one tile before its copy
//     is issued, so no copy waits for the table.
//   - All tiles of all (sequence, key head, row block) items form one list, cut into equal pieces,
//     one to a resident block (two to an SM): ragged batches and single long sequences fill the
//     GPU alike.  A block keeps its ring going across items.  A piece that holds a whole item
//     writes O and lse; the others leave fp32 partial results, merged by paged_combine_kernel.
//   - Scores and P V run on warp-level matrix instructions (16 rows x 16 keys a step), the softmax
//     in registers between them.  A block of 16 rows gives each of its 4 warps a quarter of a
//     tile's keys, with a softmax state of its own, merged at the end of the item; of 32 rows, each
//     pair of warps 16 rows; of 64 rows, each warp 16 rows and all keys.
// Statistics and accumulators are fp32; P is rounded to bf16 for the second product, as in the
// forward kernel, while its sum is taken before the rounding.
#pragma once

#include "attn_fwd.cuh"
#include "paging.h"

namespace gpt_attn {

constexpr int kPagedThreads = 128;
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
};

__device__ __forceinline__ PagedSpan paged_seq_span(const PagedParams& p, int b) {
    const int n = p.n_new ? clamp_int(__ldg(p.n_new + b), 0, p.N) : p.N;
    return paged_span(__ldg(p.lens + b), n, p.cap, p.window, p.sinks);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    const int bytes = valid ? 16 : 0;       // 0: the 16 bytes are zero-filled, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

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

// Two packed bf16 values as finite ones (0 for the others) and two indicators, 1 where the value is
// +inf or NaN (up) and where it is -inf or NaN (down).
__device__ __forceinline__ void split_bf16x2(uint32_t w, uint32_t& fin, uint32_t& up, uint32_t& down) {
    fin = up = down = 0;
#pragma unroll
    for (int s = 0; s < 32; s += 16) {
        const uint32_t x = (w >> s) & 0xffffu;
        const bool ok = (x & 0x7f80u) != 0x7f80u;
        fin |= (ok ? x : 0u) << s;
        up |= (!ok && x != 0xff80u ? 0x3f80u : 0u) << s;
        down |= (!ok && x != 0x7f80u ? 0x3f80u : 0u) << s;
    }
}

template <int D>
struct PagedCfg {
    static constexpr int kStages = D == 64 ? 6 : 3;               // 32 KB stages (D = 128), 16 KB (D = 64)
    static constexpr int kRing = kStages + 1;                     // tile descriptors
    static constexpr int kRowBytes = D * 2;
    static constexpr int kTileBytes = kPagedTile * kRowBytes;
};

// What a block has to know of one tile of its piece.
struct PagedTile {
    int b, x;          // sequence; key head * RB + row block
    int key0;
    int L;
    int first, last;   // first / last tile of this block's part of the item
    int whole;         // the block has the whole item
    int mask;          // some row may not see some key
};

template <int D>
struct PagedSmem {
    using C = PagedCfg<D>;
    alignas(128) uint8_t k[C::kStages][C::kTileBytes];
    alignas(128) uint8_t v[C::kStages][C::kTileBytes];
    alignas(16) float merge[16 * D];
    int row[C::kRing][kPagedTile];       // each key's row in the pools, -1: not read
    PagedTile tile[C::kRing];
    unsigned long long anc[kMaxNodes];
    int depth[kMaxNodes];
    int parents[kMaxNodes];
    float m[4][16], l[4][16];
    long long scan[4];
    long long start_prefix;
    int start_b;
};

// Tiles of the list that sequence b contributes.
__device__ __forceinline__ long long paged_seq_tiles(const PagedParams& p, int b) {
    return (long long)paged_seq_span(p, b).n_tiles * p.Hkv * p.RB;
}

template <int D, int MT>
__global__ void __launch_bounds__(kPagedThreads, kPagedBlocksPerSm)
paged_decode_kernel(const __grid_constant__ PagedParams p) {
    using C = PagedCfg<D>;
    constexpr int KS = 4 / MT;                       // warps that share a 16-row tile's keys
    constexpr int NT = kPagedTile / KS / 8;          // 8-key columns of a warp
    constexpr int kChunks = D / 8;                   // 16-byte chunks of a row
    constexpr int kRows = 16 * MT;
    extern __shared__ uint8_t smem_raw[];
    PagedSmem<D>& sm = *reinterpret_cast<PagedSmem<D>*>(smem_align1024(smem_raw));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int mt = warp / KS, ks = warp % KS;

    // ---- this block's piece of the list
    long long total = 0;
    for (int b = tid; b < p.B; b += kPagedThreads) total += paged_seq_tiles(p, b);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    if (lane == 0) sm.scan[warp] = total;
    __syncthreads();
    total = sm.scan[0] + sm.scan[1] + sm.scan[2] + sm.scan[3];
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
            for (int w = 0; w < warp; ++w) inc += sm.scan[w];
            inc += before;
            if (b < p.B && begin >= inc - mine && begin < inc) {
                sm.start_b = b;
                sm.start_prefix = inc - mine;
            }
            if (blockIdx.x == 0 && b < p.B) p.prefix[b] = inc - mine;
            before += sm.scan[0] + sm.scan[1] + sm.scan[2] + sm.scan[3];
        }
        if (blockIdx.x == 0 && tid == 0) {
            p.prefix[p.B] = total;
            p.prefix[p.B + 1] = chunk;
        }
        __syncthreads();
    }
    if (n_mine == 0) return;

    // ---- walks the piece, one tile per call, writing tile i's descriptor; threads 0..63 return
    // their key's row (the caller stores it once the lookup has landed)
    int it_b = sm.start_b, it_x, it_t, it_first;     // it_first: first tile of the item in this piece
    PagedSpan sp = paged_seq_span(p, it_b);
    {
        const long long in_b = begin - sm.start_prefix;
        it_x = (int)(in_b / sp.n_tiles);
        it_t = it_first = (int)(in_b % sp.n_tiles);
    }
    auto next_tile = [&](int i) -> int {
        const int key0 = sp.tile(it_t) * kPagedTile;
        const int key = key0 + tid;
        int row = -1;
        if (tid < kPagedTile && sp.needs(key, p.sinks))
            row = paged_row(p.table + (size_t)it_b * p.max_pages, key, p.page, p.n_pages, p.Hkv, it_x / p.RB);
        if (tid == 0) {
            PagedTile& d = sm.tile[i % C::kRing];
            d.b = it_b;
            d.x = it_x;
            d.key0 = key0;
            d.L = sp.L;
            d.first = i == 0 || it_t == 0;
            d.last = i == n_mine - 1 || it_t == sp.n_tiles - 1;
            d.whole = it_first == 0 && it_t == sp.n_tiles - 1;
            // every node stands at most n - 1 past L, so keys within the window of that position are
            // within everybody's
            d.mask = key0 + kPagedTile > sp.L || (p.window > 0 && sp.L + sp.n - 1 - key0 >= p.window);
        }
        if (++it_t == sp.n_tiles) {
            it_t = it_first = 0;
            if (++it_x == p.Hkv * p.RB && i + 1 < n_mine) {
                it_x = 0;
                do sp = paged_seq_span(p, ++it_b);
                while (sp.n_tiles == 0);
            }
        }
        return row;
    };
    auto load_tile = [&](int i) {
        const int s = i % C::kStages;
        const int* rows = sm.row[i % C::kRing];
        const int c = tid % kChunks;
        const uint32_t kd = smem_u32(sm.k[s]), vd = smem_u32(sm.v[s]);
#pragma unroll
        for (int r = tid / kChunks; r < kPagedTile; r += kPagedThreads / kChunks) {
            const int row = rows[r];
            const size_t src = (size_t)max(row, 0) * D + c * 8;
            const uint32_t dst = r * C::kRowBytes + ((c ^ (r & 7)) << 4);
            cp_async16(kd + dst, p.k + src, row >= 0);
            cp_async16(vd + dst, p.v + src, row >= 0);
        }
    };
    for (int i = 0; i < C::kStages && i < n_mine; ++i) {
        const int row = next_tile(i);
        if (tid < kPagedTile) sm.row[i % C::kRing][tid] = row;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) {
        if (i < n_mine) load_tile(i);
        cp_async_commit();
    }

    // ---- state of the current item: two rows per thread (r and r + 8 of the warp's 16)
    uint32_t qf[D / 16][4];
    float oacc[D / 8][4];
    float m[2], l[2];
    int pos[2];
    unsigned long long anc[2];
    int row_id[2];
    int cur_b = -1, part_i = 0;                      // part_i: the part's first tile
    const int r_lo = mt * 16 + (lane >> 2);

    for (int i = 0; i < n_mine; ++i) {
        cp_async_wait<C::kStages - 2>();
        __syncthreads();
        if (i + C::kStages - 1 < n_mine) load_tile(i + C::kStages - 1);
        cp_async_commit();
        int ahead = -1;
        const bool more = i + C::kStages < n_mine;
        if (more) ahead = next_tile(i + C::kStages);

        const PagedTile t = sm.tile[i % C::kRing];
        const int h = t.x / p.RB, rb = t.x - h * p.RB;
        if (t.first) {
            part_i = i;
            if (t.b != cur_b) {
                // the tree of this sequence
                cur_b = t.b;
                if (p.parents) {
                    if (tid < p.N) sm.parents[tid] = __ldg(p.parents + (size_t)t.b * p.N + tid);
                    __syncthreads();
                }
                if (tid < p.N) {
                    const unsigned long long a = p.parents ? paged_ancestors(tid, sm.parents)
                                                           : (2ull << tid) - 1;
                    sm.anc[tid] = a;
                    sm.depth[tid] = __popcll(a) - 1;
                }
                __syncthreads();
            }
            const int n_b = p.n_new ? clamp_int(__ldg(p.n_new + t.b), 0, p.N) : p.N;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = rb * 64 + r_lo + 8 * e;
                const int node = r % p.N;
                const bool live = r < p.R && node < n_b;
                row_id[e] = r < p.R ? r : -1;
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
        const int s = i % C::kStages;
        const int kb = ks * (kPagedTile / KS);        // first key of the warp within the tile
        float sc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
        {
            const int key = kb + (lane & 7) + ((lane >> 4) << 3);
            const uint32_t base = smem_u32(sm.k[s]) + key * C::kRowBytes;
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
        if (t.mask || __any_sync(0xffffffffu, sm.row[i % C::kRing][lane] < 0 || sm.row[i % C::kRing][lane + 32] < 0)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int kt = kb + n * 8 + (lane & 3) * 2 + (e & 1);
                    const bool see = sm.row[i % C::kRing][kt] >= 0 &&
                                     paged_sees(t.key0 + kt, pos[e >> 1], anc[e >> 1], sm.depth, t.L, p.window, p.sinks);
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
        // ---- O += P V
        {
            const int key = kb + (lane & 15);
            const uint32_t base = smem_u32(sm.v[s]) + key * C::kRowBytes;
            // New tokens that are not every node's ancestors may hold infinities or NaN, which must
            // not reach the others through 0 * NaN: such a tile takes the path below.
            bool odd = false;
            if (t.mask && p.N > 1) {
                const uint4* rows = reinterpret_cast<const uint4*>(sm.v[s] + kb * C::kRowBytes);
#pragma unroll 4
                for (int c = lane; c < NT * 8 * kChunks; c += 32) {
                    const uint4 x = rows[c];
                    odd = odd || not_finite(x.x) || not_finite(x.y) || not_finite(x.z) || not_finite(x.w);
                }
                odd = __any_sync(0xffffffffu, odd);
            }
            if (!odd) {
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
            } else {
                // The finite values, and how many keys with P > 0 hold +inf or NaN (up) and -inf or
                // NaN (down) in each column.
#pragma unroll
                for (int n = 0; n < D / 16; ++n) {
                    float up[2][4] = {}, down[2][4] = {};
#pragma unroll
                    for (int kk = 0; kk < NT / 2; ++kk) {
                        const int c = n * 2 + (lane >> 4);
                        uint32_t b4[4], ones[4], f4[4], u4[4], d4[4];
                        ldmatrix4_trans(b4, base + kk * 16 * C::kRowBytes + ((c ^ (key & 7)) << 4));
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            split_bf16x2(b4[e], f4[e], u4[e], d4[e]);
                            ones[e] = ((pf[kk][e] & 0xffffu) ? 0x3f80u : 0u) | ((pf[kk][e] >> 16) ? 0x3f800000u : 0u);
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            mma_16816(oacc[2 * n + j], pf[kk], f4[2 * j], f4[2 * j + 1]);
                            mma_16816(up[j], ones, u4[2 * j], u4[2 * j + 1]);
                            mma_16816(down[j], ones, d4[2 * j], d4[2 * j + 1]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (up[j][e] > 0.f) oacc[2 * n + j][e] += INFINITY;
                            if (down[j][e] > 0.f) oacc[2 * n + j][e] -= INFINITY;
                        }
                }
            }
        }
        if (more && tid < kPagedTile) sm.row[(i + C::kStages) % C::kRing][tid] = ahead;

        if (t.last) {
            // ---- end of the item (or of this block's part): the warps that share a row tile merge
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            }
            if constexpr (KS > 1) {
                if ((lane & 3) == 0) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        sm.m[warp][(lane >> 2) + 8 * e] = m[e];
                        sm.l[warp][(lane >> 2) + 8 * e] = l[e];
                    }
                }
                __syncthreads();
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = (lane >> 2) + 8 * e;
                    float M = -INFINITY, lt = 0.f;
#pragma unroll
                    for (int w = 0; w < KS; ++w) M = fmaxf(M, sm.m[mt * KS + w][r]);
                    const float mu = M == -INFINITY ? 0.f : M;
#pragma unroll
                    for (int w = 0; w < KS; ++w) lt += sm.l[mt * KS + w][r] * ex2_approx(sm.m[mt * KS + w][r] - mu);
                    const float f = ex2_approx(m[e] - mu);
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        oacc[n][2 * e] *= f;
                        oacc[n][2 * e + 1] *= f;
                    }
                    m[e] = M;
                    l[e] = lt;
                }
                // The merge buffer holds 16 x D values: 1 / MT of the columns of each row tile at a time.
                constexpr int kPart = D / 8 / MT;
#pragma unroll
                for (int part = 0; part < MT; ++part) {
                    float4* buf = reinterpret_cast<float4*>(sm.merge) + (size_t)mt * kPart * 32 + lane;
#pragma unroll
                    for (int w = KS - 1; w > 0; --w) {
                        if (ks == w) {
#pragma unroll
                            for (int n = 0; n < kPart; ++n) {
                                const float(&a)[4] = oacc[part * kPart + n];
                                buf[n * 32] = make_float4(a[0], a[1], a[2], a[3]);
                            }
                        }
                        __syncthreads();
                        if (ks == w - 1) {
#pragma unroll
                            for (int n = 0; n < kPart; ++n) {
                                const float4 a = buf[n * 32];
                                float(&c)[4] = oacc[part * kPart + n];
                                c[0] += a.x;
                                c[1] += a.y;
                                c[2] += a.z;
                                c[3] += a.w;
                            }
                        }
                    }
                    if (MT > 1) __syncthreads();
                }
            }
            if (ks == 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (row_id[e] < 0) continue;
                    const bool any = l[e] != 0.f && anc[e] != 0;  // a node that does not exist sees nothing
                    if (t.whole) {
                        const int g = row_id[e] / p.N, node = row_id[e] % p.N;
                        const int head = h * p.G + g;
                        __nv_bfloat16* dst = p.o + t.b * p.o_str.b + (long long)head * p.o_str.h + node * p.o_str.t +
                                             (lane & 3) * 2;
                        const float inv = any ? 1.f / l[e] : 0.f;
#pragma unroll
                        for (int n = 0; n < D / 8; ++n)
                            *reinterpret_cast<uint32_t*>(dst + n * 8) =
                                pack_bf16x2(oacc[n][2 * e] * inv, oacc[n][2 * e + 1] * inv);
                        if ((lane & 3) == 0)
                            p.lse[((size_t)t.b * p.H + head) * p.N + node] =
                                any ? (m[e] + log2f(l[e])) * 0.69314718055994531f : -INFINITY;
                    } else {
                        // a piece has at most two partial items: the one it starts in and the one it ends in
                        const size_t pr = (2 * (size_t)blockIdx.x + (part_i > 0)) * kRows + r_lo + 8 * e;
                        float* dst = p.part_o + pr * D + (lane & 3) * 2;
#pragma unroll
                        for (int n = 0; n < D / 8; ++n)
                            *reinterpret_cast<float2*>(dst + n * 8) = make_float2(oacc[n][2 * e], oacc[n][2 * e + 1]);
                        if ((lane & 3) == 0)
                            *reinterpret_cast<float2*>(p.part_ml + pr * 2) = make_float2(any ? m[e] : -INFINITY, any ? l[e] : 0.f);
                    }
                }
            }
        }
    }
}

// Joins the parts of the items that more than one block worked on, in the order of the list, and
// writes the rows of sequences that have no tiles.  A thread takes four columns of a row.
template <int D, int MT>
__global__ void __launch_bounds__(kPagedThreads)
paged_combine_kernel(const __grid_constant__ PagedParams p) {
    constexpr int kRows = 16 * MT;
    constexpr int kPerRow = D / 4;
    const int x = blockIdx.x % (p.Hkv * p.RB), b = blockIdx.x / (p.Hkv * p.RB);
    const int h = x / p.RB, rb = x - h * p.RB;
    const int r = blockIdx.y * (kPagedThreads / kPerRow) + threadIdx.x / kPerRow;
    const int c = threadIdx.x % kPerRow;
    if (rb * 64 + r >= p.R || r >= kRows) return;
    const long long chunk = p.prefix[p.B + 1];
    const int n_tiles = paged_seq_span(p, b).n_tiles;
    const long long first = p.prefix[b] + (long long)x * n_tiles;
    float M = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (n_tiles > 0) {
        const int from = (int)(first / chunk), to = (int)((first + n_tiles - 1) / chunk);
        if (from == to) return;                        // one block had the whole item
        for (int s = from; s <= to; ++s) {
            const size_t pr = (2 * (size_t)s + (first > s * chunk)) * kRows + r;
            const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + pr * 2);
            const float4 a = *reinterpret_cast<const float4*>(p.part_o + pr * D + c * 4);
            const float top = fmaxf(M, ml.x);
            const float mu = top == -INFINITY ? 0.f : top;
            const float w0 = ex2_approx(M - mu), w1 = ex2_approx(ml.x - mu);
            // a part without a visible key has weight 0 and may hold anything
            const float4 y = ml.x == -INFINITY ? make_float4(0.f, 0.f, 0.f, 0.f) : a;
            acc.x = acc.x * w0 + y.x * w1;
            acc.y = acc.y * w0 + y.y * w1;
            acc.z = acc.z * w0 + y.z * w1;
            acc.w = acc.w * w0 + y.w * w1;
            l = l * w0 + ml.y * w1;
            M = top;
        }
    }
    const int row = rb * 64 + r, head = h * p.G + row / p.N, node = row % p.N;
    const bool any = l != 0.f;
    const float inv = any ? 1.f / l : 0.f;
    __nv_bfloat16* dst = p.o + b * p.o_str.b + (long long)head * p.o_str.h + node * p.o_str.t + c * 4;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (c == 0) p.lse[((size_t)b * p.H + head) * p.N + node] = any ? (M + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace gpt_attn
