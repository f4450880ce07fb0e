// The pages of a paged key/value cache: rows of new tokens into them, accepted drafts moved up,
// and the table that says which sequence holds which page (forked, reserved, freed, packed).
//
// A pool is [n_pages, Hkv, page, D] bf16 for keys and one for values; the table [S, M] gives each
// slot's pages in order (-1: none), lens [S] its cached tokens, refs [P] how many slots hold a page.
//
// The moves of rows and pages are bound by HBM (each byte read and written once).  The table work
// is a few thousand integers with dependent steps (count, rank, assign), so latency bounds it: one
// cluster of 8 blocks does all steps of a call in one launch, each block a slice of the slots and of
// the pages, with cluster barriers in place of launches between the steps.  Ranks come from
// ballots, so results do not depend on the order of threads: the lowest free pages go to the lowest
// slots.
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "attn_fwd.cuh"
#include "paging.h"

namespace gpt_attn {

struct PagedPools {
    __nv_bfloat16* k;             // [n_pages, Hkv, page, D]
    __nv_bfloat16* v;
    const int* table;             // [B, max_pages]
    const int* lens;              // [B]
    int n_pages, Hkv, max_pages, cap;
    FastDiv page;
};

// ------------------------------------------------------------------------------- rows of tokens
struct AppendParams {
    PagedPools c;
    const __nv_bfloat16* k_new;   // [b, h, n, d]
    const __nv_bfloat16* v_new;
    Strides k_str, v_str;
    const int* n_new;             // [B] or nullptr: N each
    int N;
    long long chunks;             // B * Hkv * N * D / 8
};

// New token n of sequence b goes to position lens[b] + n.  One thread to 16 bytes of both pools.
template <int D>
__global__ void __launch_bounds__(256) paged_append_kernel(const __grid_constant__ AppendParams p) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= p.chunks) return;
    const int c = (int)(i % (D / 8));
    long long r = i / (D / 8);
    const int n = (int)(r % p.N);
    r /= p.N;
    const int h = (int)(r % p.c.Hkv), b = (int)(r / p.c.Hkv);
    if (p.n_new && n >= __ldg(p.n_new + b)) return;
    const long long at = (long long)clamp_int(__ldg(p.c.lens + b), 0, p.c.cap) + n;
    if (at >= p.c.cap) return;
    const int row = paged_row(p.c.table + (size_t)b * p.c.max_pages, (int)at, p.c.page, p.c.n_pages, p.c.Hkv, h);
    if (row < 0) return;
    const size_t dst = (size_t)row * D + c * 8;
    const uint4 k = __ldg(reinterpret_cast<const uint4*>(p.k_new + b * p.k_str.b + h * p.k_str.h + n * p.k_str.t + c * 8));
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p.v_new + b * p.v_str.b + h * p.v_str.h + n * p.v_str.t + c * 8));
    *reinterpret_cast<uint4*>(p.c.k + dst) = k;
    *reinterpret_cast<uint4*>(p.c.v + dst) = v;
}

struct AcceptParams {
    PagedPools c;
    const int* accepted;          // [B, N] nodes, in the order of the accepted path
    const int* n_accepted;        // [B]
    int N;
};

constexpr int kAcceptThreads = 256;

// Node accepted[b][i] of sequence b moves from position lens[b] + accepted[b][i] to lens[b] + i.
// One block to a (sequence, key head): all rows are read before one is written, so any order of
// nodes is allowed.  Each thread keeps its 16-byte pieces in registers between the two.
template <int D>
__global__ void __launch_bounds__(kAcceptThreads) paged_accept_kernel(const __grid_constant__ AcceptParams p) {
    constexpr int kChunks = D / 8, kAtOnce = kAcceptThreads / kChunks, kKeep = (kMaxNodes + kAtOnce - 1) / kAtOnce;
    const int h = blockIdx.x % p.c.Hkv, b = blockIdx.x / p.c.Hkv;
    const int n = clamp_int(__ldg(p.n_accepted + b), 0, p.N);
    const int L = clamp_int(__ldg(p.c.lens + b), 0, p.c.cap);
    const int* table = p.c.table + (size_t)b * p.c.max_pages;
    const int c = threadIdx.x % kChunks;
    uint4 k[kKeep], v[kKeep];
    int dst[kKeep];
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
        const int i = j * kAtOnce + threadIdx.x / kChunks;
        dst[j] = -1;
        if (i >= n) continue;
        const int node = __ldg(p.accepted + (size_t)b * p.N + i);
        if (node < 0 || node >= p.N || node == i || L + node >= p.c.cap || L + i >= p.c.cap) continue;
        const int src = paged_row(table, L + node, p.c.page, p.c.n_pages, p.c.Hkv, h);
        const int to = paged_row(table, L + i, p.c.page, p.c.n_pages, p.c.Hkv, h);
        if (src < 0 || to < 0) continue;
        dst[j] = to;
        k[j] = *reinterpret_cast<const uint4*>(p.c.k + (size_t)src * D + c * 8);
        v[j] = *reinterpret_cast<const uint4*>(p.c.v + (size_t)src * D + c * 8);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
        if (dst[j] < 0) continue;
        *reinterpret_cast<uint4*>(p.c.k + (size_t)dst[j] * D + c * 8) = k[j];
        *reinterpret_cast<uint4*>(p.c.v + (size_t)dst[j] * D + c * 8) = v[j];
    }
}

// ------------------------------------------------------------------------------- whole pages
struct CopyParams {
    uint4* k;
    uint4* v;
    const int2* pairs;            // (from, to); a pair with a page outside the pool is skipped
    const int* n_pairs;           // device count of pairs in use, or nullptr: max_pairs
    int max_pairs, n_pages;
    int page_chunks;              // 16-byte chunks of a page in one pool
    int units;                    // units of kCopyUnit chunks that a page is cut into
};

constexpr int kCopyThreads = 256;
constexpr int kCopyDeep = 8;                               // loads in flight per thread
constexpr int kCopyUnit = kCopyThreads * kCopyDeep;        // 32 KB
constexpr int kCopyBlocksPerSm = 32;

// Bound by HBM.  Pages are cut into units of 32 KB and blocks take unit after unit, so a few large pages
// and many small ones fill the GPU alike, and a count known only on the device costs little.  Packing
// two pools of 0.5 GB of which half is in use (531 MB read and written) on one B200: 84 us, 6.3 TB/s, of a measured copy's
// 6.5; with 4 loads a thread 94, with as many blocks as are resident (8 to an SM) 88, where the slowest
// block's last unit is waited for.
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ CopyParams p) {
    const int n = p.n_pairs ? clamp_int(__ldg(p.n_pairs), 0, p.max_pairs) : p.max_pairs;
    const long long total = 2LL * n * p.units;
    for (long long u = blockIdx.x; u < total; u += gridDim.x) {
        const int part = (int)(u % p.units);
        const long long w = u / p.units;
        const int2 pair = __ldg(p.pairs + (w >> 1));
        if (pair.x < 0 || pair.x >= p.n_pages || pair.y < 0 || pair.y >= p.n_pages || pair.x == pair.y) continue;
        uint4* pool = (w & 1) ? p.v : p.k;
        const uint4* src = pool + (size_t)pair.x * p.page_chunks;
        uint4* dst = pool + (size_t)pair.y * p.page_chunks;
        const int at = part * kCopyUnit + threadIdx.x;
        uint4 r[kCopyDeep];
#pragma unroll
        for (int i = 0; i < kCopyDeep; ++i)
            if (at + i * kCopyThreads < p.page_chunks) r[i] = src[at + i * kCopyThreads];
#pragma unroll
        for (int i = 0; i < kCopyDeep; ++i)
            if (at + i * kCopyThreads < p.page_chunks) dst[at + i * kCopyThreads] = r[i];
    }
}

// ------------------------------------------------------------------------------- the table
constexpr int kPagesThreads = 1024;
constexpr int kPagesCluster = 8;

struct PagesParams {
    int* table;                   // [S, M]
    int* lens;                    // [S]
    int* refs;                    // [P]
    int S, M, P, page;
    const int* arg;               // fork: parents [S]; reserve: tokens [S]; free: drop [S]
    int* status;                  // [S]
    int2* pairs;                  // fork: [S]; pack: [P / 2]
    int* new_table;               // pack: [S, M]
    int* new_refs;                // pack: [P]
    int* moves;                   // pack: [1]
    int* need;                    // workspace: [S] pages asked for
    int* list;                    // workspace: [P] free pages, or the new place of each page
    int* counts;                  // workspace: [4 * kPagesCluster]
};

// This block's slice [lo, hi) of n things.
__device__ __forceinline__ void cluster_slice(int n, int rank, int& lo, int& hi) {
    const int per = (n + kPagesCluster - 1) / kPagesCluster;
    lo = min((long long)rank * per, (long long)n);
    hi = min(lo + per, n);
}

// Sum of x over the block, and this thread's exclusive prefix.
__device__ __forceinline__ int block_scan(int x, int* scratch, int& before) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += y;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    int base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kPagesThreads / 32; ++w) {
        base += w < warp ? scratch[w] : 0;
        total += scratch[w];
    }
    before = base + inc - x;
    return total;
}

// How many things of this block's slice `is` holds for.
template <typename Pred>
__device__ __forceinline__ int slice_count(int lo, int hi, int* scratch, Pred is) {
    int mine = 0, before;
    for (int i = lo + threadIdx.x; i < hi; i += kPagesThreads) mine += is(i) ? 1 : 0;
    return block_scan(mine, scratch, before);
}

// Calls take(i, k) for the things of the slice that `is` holds for, k counting up from `base` in
// their order.
template <typename Pred, typename Take>
__device__ __forceinline__ void slice_rank(int lo, int hi, int base, int* scratch, Pred is, Take take) {
    for (int at = lo; at < hi; at += kPagesThreads) {
        const int i = at + threadIdx.x;
        const bool mine = i < hi && is(i);
        int before;
        const int n = block_scan(mine ? 1 : 0, scratch, before);
        if (mine) take(i, base + before);
        base += n;
    }
}

__device__ __forceinline__ int sum_before(const int* counts, int rank, int& total) {
    int before = 0;
    total = 0;
#pragma unroll
    for (int r = 0; r < kPagesCluster; ++r) {
        const int c = counts[r];
        before += r < rank ? c : 0;
        total += c;
    }
    return before;
}

__device__ __forceinline__ bool page_held(const PagesParams& p, int e) { return e >= 0 && e < p.P && p.refs[e] > 0; }

// One warp looks slot s over.  Returns the pages it asks for, -1 for a refusal, -2 for nothing asked.
// Fork: parents[s] must be another slot that is not itself asked for, with all its pages in place,
// and s must be empty.  A partial last page is the one page that a fork asks for.
__device__ __forceinline__ int fork_need(const PagesParams& p, int s) {
    const int lane = threadIdx.x & 31;
    const int src = p.arg[s];
    if (src < 0) return -2;
    if (src >= p.S || p.arg[src] >= 0) return -1;
    const int n = p.lens[src];
    bool ok = p.lens[s] == 0 && n >= 0 && n <= (long long)p.M * p.page;
    const int used = ok ? (int)(((long long)n + p.page - 1) / p.page) : 0;
    for (int j = lane; j < p.M; j += 32) {
        ok = ok && p.table[(size_t)s * p.M + j] < 0;
        if (j < used) ok = ok && page_held(p, p.table[(size_t)src * p.M + j]);
    }
    return __all_sync(0xffffffffu, ok) ? (n % p.page != 0) : -1;
}

// Pages that slot s holds: the entries before the first -1.
__device__ __forceinline__ int slot_pages(const PagesParams& p, int s) {
    const int lane = threadIdx.x & 31;
    for (int j = 0; j < p.M; j += 32) {
        const unsigned none = __ballot_sync(0xffffffffu, j + lane >= p.M || p.table[(size_t)s * p.M + j + lane] < 0);
        if (none) return j + __ffs(none) - 1;
    }
    return p.M;
}

// Whether slot s holds a page behind the first -1 of its row, that is past its `held` ones.
__device__ __forceinline__ bool slot_gap(const PagesParams& p, int s, int held) {
    bool page = false;
    for (int j = held + (threadIdx.x & 31); j < p.M; j += 32) page |= p.table[(size_t)s * p.M + j] >= 0;
    return __any_sync(0xffffffffu, page);
}

// Reserve: pages for arg[s] more tokens than lens[s].  They would overwrite the pages behind a gap, which
// nobody could give back then.
__device__ __forceinline__ int reserve_need(const PagesParams& p, int s) {
    const int more = p.arg[s], n = p.lens[s];
    if (more <= 0) return -2;
    if (n < 0 || (long long)n + more > (long long)p.M * p.page) return -1;
    const int held = slot_pages(p, s);
    if (slot_gap(p, s, held)) return -1;
    const int want = (int)(((long long)n + more + p.page - 1) / p.page);
    return want > held ? want - held : 0;
}

// Fork and reserve: every slot's wish, the free pages in order, then each slot's share of them.  A
// slot is served if it asks for no page, or if the wishes up to and including its own fit into the free
// pages.
template <bool kFork>
__global__ void __cluster_dims__(kPagesCluster, 1, 1) __launch_bounds__(kPagesThreads)
pages_take_kernel(const __grid_constant__ PagesParams p) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ int scratch[kPagesThreads / 32];
    const int rank = (int)blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s_lo, s_hi, p_lo, p_hi;
    cluster_slice(p.S, rank, s_lo, s_hi);
    cluster_slice(p.P, rank, p_lo, p_hi);
    auto is_free = [&](int i) { return p.refs[i] <= 0; };

    int asked = 0;                                  // pages asked for by this warp's slots (same in all lanes)
    for (int s = s_lo + warp; s < s_hi; s += kPagesThreads / 32) {
        const int need = kFork ? fork_need(p, s) : reserve_need(p, s);
        if (lane == 0) p.need[s] = need;
        asked += need > 0 ? need : 0;
    }
    int before;
    asked = block_scan(lane == 0 ? asked : 0, scratch, before);
    const int n_free = slice_count(p_lo, p_hi, scratch, is_free);
    if (threadIdx.x == 0) {
        p.counts[rank] = n_free;
        p.counts[kPagesCluster + rank] = asked;
    }
    cluster.sync();

    int total_free, total_asked;
    const int free_base = sum_before(p.counts, rank, total_free);
    int base = sum_before(p.counts + kPagesCluster, rank, total_asked);
    slice_rank(p_lo, p_hi, free_base, scratch, is_free, [&](int i, int k) {
        if (k < total_asked) p.list[k] = i;
    });
    cluster.sync();

    // shares: a slot's first page is list[base + wishes before it]
    for (int at = s_lo; at < s_hi; at += kPagesThreads / 32) {
        const int s = at + warp;
        const int need = s < s_hi ? p.need[s] : -2;
        int first;
        const int n = block_scan(lane == 0 && need > 0 ? need : 0, scratch, first);
        first = base + __shfl_sync(0xffffffffu, first, 0);
        base += n;
        if (s >= s_hi) continue;
        const bool served = need == 0 || (need > 0 && (long long)first + need <= total_free);
        if (lane == 0) p.status[s] = need == -2 ? 0 : (served ? 1 : (need < 0 ? -1 : -2));
        int* row = p.table + (size_t)s * p.M;
        if (kFork) {
            int2 pair = make_int2(-1, -1);
            if (served) {
                const int src = p.arg[s], len = p.lens[src];
                const int* from = p.table + (size_t)src * p.M;
                const int full = len / p.page;
                for (int j = lane; j < full; j += 32) {
                    const int e = from[j];
                    row[j] = e;
                    atomicAdd(p.refs + e, 1);
                }
                if (need > 0) {
                    pair = make_int2(from[full], p.list[first]);
                    if (lane == 0) {
                        row[full] = pair.y;
                        p.refs[pair.y] = 1;
                    }
                }
                if (lane == 0) p.lens[s] = len;
            }
            if (lane == 0) p.pairs[s] = pair;
        } else if (served && need > 0) {
            const int held = slot_pages(p, s);
            for (int j = lane; j < need; j += 32) {
                const int e = p.list[first + j];
                row[held + j] = e;
                p.refs[e] = 1;
            }
        }
    }
}

// One warp to a slot: its pages lose a holder, its row and length are cleared.
__global__ void __launch_bounds__(256) pages_free_kernel(const __grid_constant__ PagesParams p) {
    const int s = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (s >= p.S || p.arg[s] <= 0) return;
    for (int j = lane; j < p.M; j += 32) {
        int* slot = p.table + (size_t)s * p.M + j;
        const int e = *slot;
        // a page that nobody holds stays at 0
        if (e >= 0 && e < p.P && atomicSub(p.refs + e, 1) <= 0) atomicAdd(p.refs + e, 1);
        *slot = -1;
    }
    if (lane == 0) p.lens[s] = 0;
}

// Packing: with n pages in use, the k-th page in use at or past place n goes to the k-th free place
// before n; there are as many of the one as of the other.
__global__ void __cluster_dims__(kPagesCluster, 1, 1) __launch_bounds__(kPagesThreads)
pages_compact_kernel(const __grid_constant__ PagesParams p) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ int scratch[kPagesThreads / 32];
    const int rank = (int)blockIdx.x;
    int lo, hi;
    cluster_slice(p.P, rank, lo, hi);
    const int n_mine = slice_count(lo, hi, scratch, [&](int i) { return p.refs[i] > 0; });
    if (threadIdx.x == 0) p.counts[rank] = n_mine;
    cluster.sync();
    int live;
    sum_before(p.counts, rank, live);
    auto late = [&](int i) { return i >= live && p.refs[i] > 0; };
    auto hole = [&](int i) { return i < live && p.refs[i] <= 0; };
    const int n_late = slice_count(lo, hi, scratch, late), n_hole = slice_count(lo, hi, scratch, hole);
    if (threadIdx.x == 0) {
        p.counts[kPagesCluster + rank] = n_late;
        p.counts[2 * kPagesCluster + rank] = n_hole;
    }
    cluster.sync();
    int moves, holes;
    const int late_base = sum_before(p.counts + kPagesCluster, rank, moves);
    const int hole_base = sum_before(p.counts + 2 * kPagesCluster, rank, holes);
    slice_rank(lo, hi, late_base, scratch, late, [&](int i, int k) { p.pairs[k].x = i; });
    slice_rank(lo, hi, hole_base, scratch, hole, [&](int i, int k) { p.pairs[k].y = i; });
    for (int i = lo + threadIdx.x; i < hi; i += kPagesThreads) {
        p.list[i] = i;
        if (i >= live) p.new_refs[i] = 0;
        else if (p.refs[i] > 0) p.new_refs[i] = p.refs[i];
    }
    for (int k = moves + rank * kPagesThreads + threadIdx.x; k < p.P / 2; k += kPagesCluster * kPagesThreads)
        p.pairs[k] = make_int2(-1, -1);
    if (rank == 0 && threadIdx.x == 0) *p.moves = moves;
    cluster.sync();
    for (int k = rank * kPagesThreads + threadIdx.x; k < moves; k += kPagesCluster * kPagesThreads) {
        const int2 m = p.pairs[k];
        p.list[m.x] = m.y;
        p.new_refs[m.y] = p.refs[m.x];
    }
    cluster.sync();
    const long long n = (long long)p.S * p.M;
    for (long long i = rank * kPagesThreads + threadIdx.x; i < n; i += kPagesCluster * kPagesThreads) {
        const int e = p.table[i];
        p.new_table[i] = e >= 0 && e < p.P ? p.list[e] : -1;
    }
}

}  // namespace gpt_attn
