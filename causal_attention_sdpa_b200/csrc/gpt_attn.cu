// C ABI of the attention library: argument checks, TMA descriptor encoding
// and kernel launches on the caller's stream.  No allocation, no host sync
// (except in gpt_attn_check, which exists to sync).
#include <cuda.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <mutex>
#include <vector>

#include "attn_bwd.cuh"
#include "attn_bwd_d64.cuh"
#include "attn_decode.cuh"
#include "attn_fwd.cuh"
#include "gpt_attn.h"
#include "paged_decode.cuh"
#include "paged_decode_tc.cuh"
#include "pages.cuh"
#include "qk_prologue.cuh"
#include "tmap_cache.h"

extern "C" size_t gpt_attn_bwd_workspace_bytes(int B, int H, int T, int D);
extern "C" size_t gpt_attn_pages_workspace_bytes(int S, int M, int P);

namespace gpt_attn {
namespace {

constexpr uint64_t kDefaultTimeoutNs = 1000ull * 1000ull * 1000ull;   // 1 s per wait

uint64_t wait_timeout_ns() {
    static uint64_t v = []() -> uint64_t {
        const char* s = getenv("GPT_ATTN_WAIT_TIMEOUT_MS");
        if (s && *s) {
            const long long ms = atoll(s);
            if (ms > 0) return (uint64_t)ms * 1000000ull;
        }
        return kDefaultTimeoutNs;
    }();
    return v;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// Encodes the tensor map of `key` (see TmapKind): 128-row boxes whose width is 128 bytes of
// elements (64 bf16 or 32 fp32 columns), 128-byte swizzle (the UMMA canonical 128B-swizzled
// layout), zero fill outside the tensor so ragged tails read as zeros.  bf16 maps are 4-D
// (D, T, H, B) with the tensor's own token, head and batch strides, so any [b, h, t, d] view with
// contiguous d (e.g. the q, k, v columns of a fused [B, T, 3, H, D] projection) is read and
// written in place; the fp32 accumulator map is 3-D (D, T, B*H), contiguous; the maps of cache pools
// are 2-D (D, rows), their boxes as many rows high as a page lets them be.
bool encode_tmap(const TmapKey& key, CUtensorMap* m) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const bool f32 = key.kind == (int)TmapKind::kF32Box32x128, rows = key.kind == (int)TmapKind::kBf16Rows;
    const cuuint64_t esz = f32 ? 4 : 2;
    const cuuint32_t rank = rows ? 2 : (f32 ? 3 : 4);
    cuuint64_t dims[4] = {(cuuint64_t)key.d0, (cuuint64_t)key.d1, (cuuint64_t)key.d2, (cuuint64_t)key.d3};
    cuuint64_t strides[3] = {(cuuint64_t)key.s1 * esz, (cuuint64_t)key.s2 * esz, (cuuint64_t)key.s3 * esz};
    cuuint32_t box[4] = {f32 ? 32u : 64u, rows ? (cuuint32_t)key.d2 : 128u, 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
                    reinterpret_cast<void*>(key.base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

TmapCache<CUtensorMap>& tmap_cache() {
    static TmapCache<CUtensorMap> c;
    return c;
}

bool cached_tmap(CUtensorMap* m, const TmapKey& key) {
    return tmap_cache().get(key, m, [](const TmapKey& k, CUtensorMap* v) { return encode_tmap(k, v); });
}

// bf16 tensor indexed [b, h, t, d] with strides `st`; 64-column x 128-row boxes.
bool make_tmap_bf16(CUtensorMap* m, const void* base, int B, int H, int T, int D, const Strides& st) {
    const TmapKey key{reinterpret_cast<uintptr_t>(base), (int)TmapKind::kBf16Box64x128, D, T, H, B, st.t, st.h, st.b};
    return cached_tmap(m, key);
}

// fp32 dQ accumulator [BH, T, D]; 32-column x 128-row boxes for the bulk reduce-add.
bool make_tmap_f32_acc(CUtensorMap* m, const void* base, int BH, int T, int D) {
    const TmapKey key{reinterpret_cast<uintptr_t>(base), (int)TmapKind::kF32Box32x128, D, T, BH, 1,
                      (long long)D, (long long)T * D, (long long)BH * T * D};
    return cached_tmap(m, key);
}

// A pool of the paged cache as bf16 rows; 64-column x box_rows boxes.
bool make_tmap_rows(CUtensorMap* m, const void* base, int rows, int D, int box_rows) {
    const TmapKey key{reinterpret_cast<uintptr_t>(base), (int)TmapKind::kBf16Rows, D, rows, box_rows, 1, (long long)D, 0, 0};
    return cached_tmap(m, key);
}

// Strides of every tensor of one call.
struct Layout {
    Strides q, k, v, o, dO, dq, dk, dv;
};

Strides contiguous(int H, int T, int D) { return Strides{(long long)H * T * D, (long long)T * D, (long long)D}; }

Layout contiguous_layout(int H, int T, int D) {
    const Strides c = contiguous(H, T, D);
    return Layout{c, c, c, c, c, c, c, c};
}

// From the C ABI's description (nullptr: contiguous [B, H, T, D]).  TMA needs every stride to be
// a multiple of 16 bytes (8 elements).
int make_layout(Layout* L, const gpt_attn_layout* a, int H, int T, int D) {
    *L = contiguous_layout(H, T, D);
    if (!a) return GPT_ATTN_OK;
    const gpt_attn_strides* in[8] = {&a->q, &a->k, &a->v, &a->o, &a->dO, &a->dq, &a->dk, &a->dv};
    Strides* out[8] = {&L->q, &L->k, &L->v, &L->o, &L->dO, &L->dq, &L->dk, &L->dv};
    for (int i = 0; i < 8; ++i) {
        const gpt_attn_strides& x = *in[i];
        if (x.batch < 0 || x.head < 0 || x.token < 0) return GPT_ATTN_ERR_SHAPE;
        if ((x.batch | x.head | x.token) & 7) return GPT_ATTN_ERR_ALIGN;
        *out[i] = Strides{x.batch, x.head, x.token};
    }
    return GPT_ATTN_OK;
}

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

int check_shape(int B, int H, int T, int D) {
    if (B < 1 || H < 1 || T < 1) return GPT_ATTN_ERR_SHAPE;
    if (D != 64 && D != 128) return GPT_ATTN_ERR_UNSUPPORTED_D;
    // Every element index must fit in int64, and the TMA coordinates (T, B*H) in int32.
    const long long bh = (long long)B * H;
    if (bh > 0x7fffffffLL) return GPT_ATTN_ERR_SHAPE;
    const long long tp = ((long long)T + 127) / 128 * 128;
    if (tp > (0x7fffffffffffffffLL / D) / bh) return GPT_ATTN_ERR_SHAPE;
    if ((tp / 128) * bh > 0x7fffffffLL) return GPT_ATTN_ERR_SHAPE;   // grid size
    return GPT_ATTN_OK;
}

template <typename Kern>
bool set_smem(Kern k, size_t bytes) {
    // The attribute is a per-function setting: raise it once per kernel and device (and again only
    // for a larger size) instead of paying a driver call on every launch.
    struct Entry { const void* fn; int dev; size_t bytes; };
    static std::mutex mu;
    static std::vector<Entry> done;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const void* fn = reinterpret_cast<const void*>(k);
    std::lock_guard<std::mutex> g(mu);
    for (auto& e : done)
        if (e.fn == fn && e.dev == dev) {
            if (e.bytes >= bytes) return true;
            if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
                return false;
            e.bytes = bytes;
            return true;
        }
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess) return false;
    done.push_back({fn, dev, bytes});
    return true;
}

// Launches a kernel that may start before the one before it in the stream has ended (it waits for
// that itself, see sm100.cuh).
template <typename... Params, typename... Args>
bool launch_dependent(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st,
                      const Args&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess && cudaGetLastError() == cudaSuccess;
}

int sm_count();

// Kernel-side mask parameters from the C ABI's description (nullptr: plain causal).  Per-head
// windows are copied out of the caller's host array into the kernel parameters.  A window past T acts as one of
// T, so that sums of positions and windows fit an int.
int make_mask(MaskParams* m, const gpt_attn_mask* a, int H, int T) {
    memset(m, 0, sizeof(*m));
    m->H = H;
    if (!a) return GPT_ATTN_OK;
    auto within = [&](int w) { return w <= 0 ? 0 : (w < T ? w : T); };
    m->window = within(a->window);
    m->doc_start = a->doc_start;
    if (a->doc_start && (reinterpret_cast<uintptr_t>(a->doc_start) & 3u)) return GPT_ATTN_ERR_ALIGN;
    if (a->head_windows) {
        if (H > kMaxHeadWindows) return GPT_ATTN_ERR_SHAPE;
        m->head_windows = 1;
        for (int h = 0; h < H; ++h) m->win[h] = within(a->head_windows[h]);
    }
    return GPT_ATTN_OK;
}

// True when every head shares one window and there are no document starts.
bool plain_window(const MaskParams& m) { return !m.head_windows && !m.doc_start; }

// The mask with sinks, every window and the sinks clamped to T (a window of T or more is causal:
// nothing is out of its reach, so sinks add nothing).  Returns false when no head needs sinks.
bool sink_mask(SinkMask* s, const MaskParams& m, int sinks, int H, int T) {
    static_cast<MaskParams&>(*s) = m;
    s->sinks = sinks < T ? sinks : T;
    auto clamp = [&](int w) { return w > 0 && w < T ? w : 0; };
    s->window = clamp(m.window);
    bool any = !m.head_windows && s->window > 0;
    for (int h = 0; m.head_windows && h < H; ++h) any |= (s->win[h] = clamp(m.win[h])) > 0;
    return sinks > 0 && any;
}

MaskParams window_mask(int window, int H, int T) {
    gpt_attn_mask a{window, nullptr, nullptr};
    MaskParams m;
    make_mask(&m, &a, H, T);
    return m;
}

ScoreScale score_scale(float scale) {
    return ScoreScale{scale == 0.f ? FLT_MIN : fabsf(scale) * 1.4426950408889634f, scale < 0.f ? kIdescNegateA : 0u};
}

template <int D>
int launch_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int T, float scale,
               const MaskParams& mask, const Layout& L, cudaStream_t st, const SinkMask* sinks = nullptr) {
    const int BH = B * H;
    CUtensorMap mq, mk, mv, mo;
    if (!make_tmap_bf16(&mq, q, B, H, T, D, L.q) || !make_tmap_bf16(&mk, k, B, H, T, D, L.k) ||
        !make_tmap_bf16(&mv, v, B, H, T, D, L.v) || !make_tmap_bf16(&mo, o, B, H, T, D, L.o))
        return GPT_ATTN_ERR_CUDA;
    FwdParams p;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.o_str = L.o;
    p.H = H;
    p.T = T;
    p.BH = BH;
    p.n_tiles = (T + kTile - 1) / kTile;
    p.n_blocks = (p.n_tiles + 1) / 2;
    const ScoreScale ss = score_scale(scale);
    p.scale_log2 = ss.log2;
    p.score_sign = ss.sign;
    p.timeout_ns = wait_timeout_ns();
    // Work order (schedule.h): static waves with one block per SM when they make enough full
    // rotations (D = 64), else one block per item, the blocks that start taking the items of
    // those that have not through cluster launch control.
    const int sms = sm_count();
    p.tail = tail_heads(BH, p.n_blocks, sms);
    p.static_hpw = 0;
    p.static_waves = 0;
    int hpw, waves;
    const bool stat = D == 64 && fwd_static_grid(sms, p.n_blocks, BH, hpw, waves);
    if (stat) {
        p.static_hpw = hpw;
        p.static_waves = waves;
    }
    const size_t smem = sizeof(FwdSmem<D>) + 1024;
    const unsigned grid = stat ? (unsigned)(hpw * p.n_blocks) : (unsigned)((long long)BH * p.n_blocks);
    if (sinks) {
        if (!set_smem(attn_fwd_kernel<D, SinkMask>, smem)) return GPT_ATTN_ERR_CUDA;
        attn_fwd_kernel<D, SinkMask><<<grid, kFwdThreads, smem, st>>>(mq, mk, mv, mo, p, *sinks);
    } else if (plain_window(mask)) {
        // Causal or one window for every head: the instantiation without per-head or document data.
        if (!set_smem(attn_fwd_kernel<D, WindowMask>, smem)) return GPT_ATTN_ERR_CUDA;
        attn_fwd_kernel<D, WindowMask><<<grid, kFwdThreads, smem, st>>>(mq, mk, mv, mo, p, WindowMask{mask.window});
    } else {
        if (!set_smem(attn_fwd_kernel<D, MaskParams>, smem)) return GPT_ATTN_ERR_CUDA;
        attn_fwd_kernel<D, MaskParams><<<grid, kFwdThreads, smem, st>>>(mq, mk, mv, mo, p, mask);
    }
    return cudaGetLastError() == cudaSuccess ? GPT_ATTN_OK : GPT_ATTN_ERR_CUDA;
}

struct WsLayout {
    float* dq_acc;
    float* lse2;
    float* delta;
    int* lower2;
    int* last_qt;
    int* sched;
    int n_tiles;
    int T_pad;
};

// Workspace: fp32 dQ accumulator [BH, T, D] | lse*log2(e) [BH, T_pad] | Delta [BH, T_pad] |
// row lower bounds [BH, T_pad] and last query tile per key tile [BH, n_tiles] (both used
// with document masks only) | the persistent kernel's work-unit counter.
WsLayout ws_layout(void* ws, int BH, int T, int D) {
    WsLayout w;
    w.n_tiles = (T + kTile - 1) / kTile;
    w.T_pad = w.n_tiles * kTile;
    w.dq_acc = static_cast<float*>(ws);
    w.lse2 = w.dq_acc + (size_t)BH * T * D;
    w.delta = w.lse2 + (size_t)BH * w.T_pad;
    w.lower2 = reinterpret_cast<int*>(w.delta + (size_t)BH * w.T_pad);
    w.last_qt = w.lower2 + (size_t)BH * w.T_pad;
    w.sched = w.last_qt + (size_t)BH * w.n_tiles;
    return w;
}

// The cut of the sink tiles, by the largest of the call's windows (0, or past T: not cut, as the call's
// other heads are as long) and a B200's 148 SMs, so that the workspace can be sized without a device.
SinkCut call_cut(int BH, int T, int window, int sinks) {
    const int n_tiles = (T + kTile - 1) / kTile;
    if (sinks <= 0) return make_cut(0, 1, n_tiles);
    const bool reaches = window <= 0 || window >= T;
    const SinkCut c = sink_cut(BH, n_tiles, reaches ? 1 : window, sinks < T ? sinks : T, 148);
    return reaches ? make_cut(c.n_s, n_tiles, n_tiles) : c;
}
SinkCut launch_cut(int BH, int T, const SinkMask& sinks, const MaskParams& mask) {
    int window = mask.head_windows ? 0 : mask.window;
    for (int h = 0; mask.head_windows && h < mask.H; ++h) window = std::max(window, mask.win[h]);
    return call_cut(BH, T, window, sinks.sinks);
}

// The pieces' sums, behind the rest of the workspace.
size_t sink_part_bytes_of(const SinkCut& c, int BH, int D) {
    return c.most > 1 ? (size_t)BH * c.n_s * c.most * 2 * kTile * D * sizeof(float) : 0;
}
size_t sink_part_bytes(int BH, int T, int D, int window, int sinks) {
    return sink_part_bytes_of(call_cut(BH, T, window, sinks), BH, D);
}
size_t sink_part_at(int BH, int T, int D) { return (gpt_attn_bwd_workspace_bytes(BH, 1, T, D) + 255) / 256 * 256; }
float* sink_part(void* ws, int BH, int T, int D) {
    return reinterpret_cast<float*>(static_cast<char*>(ws) + sink_part_at(BH, T, D));
}

// SM count of the current device, cached per device.  Host threads may call the library at the
// same time: the cache entries are atomics (every thread would store the same value).
int sm_count() {
    static std::atomic<int> counts[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
    int n = counts[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
        counts[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

template <typename Mask>
int launch_bwd_delta(const void* o, const float* lse, const void* dout, int B, int H, int T, int D, void* ws,
                     const Mask& mask, const Layout& L, cudaStream_t st, int exact_rows = 0) {
    const int BH = B * H;
    const WsLayout w = ws_layout(ws, BH, T, D);
    const long long rows = (long long)BH * w.T_pad;
    const int rows_per_block = 256 / (D / 8);
    const unsigned grid = (unsigned)((rows + rows_per_block - 1) / rows_per_block);
    const auto* o16 = static_cast<const __nv_bfloat16*>(o);
    const auto* do16 = static_cast<const __nv_bfloat16*>(dout);
    const bool doc = mask.doc_start != nullptr;
    if (D == 64)
        attn_bwd_prep_kernel<64, Mask><<<grid, 256, 0, st>>>(o16, do16, lse, w.lse2, w.delta, w.dq_acc, w.sched, T,
                                                             w.T_pad, rows, mask, doc ? w.lower2 : nullptr,
                                                             w.last_qt, w.n_tiles, L.o, L.dO, H, exact_rows);
    else
        attn_bwd_prep_kernel<128, Mask><<<grid, 256, 0, st>>>(o16, do16, lse, w.lse2, w.delta, w.dq_acc, w.sched, T,
                                                              w.T_pad, rows, mask, doc ? w.lower2 : nullptr,
                                                              w.last_qt, w.n_tiles, L.o, L.dO, H, exact_rows);
    return cudaGetLastError() == cudaSuccess ? GPT_ATTN_OK : GPT_ATTN_ERR_CUDA;
}

// Rows of each head among which there are some that see few keys: the first ones of each document, hence
// without documents of the head, unless a window with its sinks is as short as that.
int exact_delta_rows(const SinkMask& mask, int H, int T) {
    bool few = mask.doc_start != nullptr;
    for (int h = 0; h < (mask.head_windows ? H : 1); ++h) {
        const int W = mask.head_windows ? mask.win[h] : mask.window;
        few |= W > 0 && (long long)W + mask.sinks <= kExactDelta;
    }
    return few || T < kExactDelta ? T : kExactDelta;
}

// Delta from the keys for those rows; the prep kernel before it has left them out.
int launch_exact_delta(const void* q, const void* k, const void* v, const float* lse, const void* dout, int B, int H,
                       int T, int D, float scale, void* ws, const SinkMask& mask, const Layout& L, cudaStream_t st) {
    const WsLayout w = ws_layout(ws, B * H, T, D);
    DeltaKeys p;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.d_o = static_cast<const __nv_bfloat16*>(dout);
    p.q_str = L.q;
    p.k_str = L.k;
    p.v_str = L.v;
    p.do_str = L.dO;
    p.delta = w.delta;
    p.lse = lse;
    p.BH = B * H;
    p.H = H;
    p.T = T;
    p.T_pad = w.T_pad;
    p.rows = exact_delta_rows(mask, H, T);
    p.scale_log2 = scale * 1.4426950408889634f;
    const dim3 grid((unsigned)(((long long)p.BH * p.rows + 7) / 8));
    return launch_dependent(D == 64 ? attn_exact_delta_kernel<64> : attn_exact_delta_kernel<128>, grid, 256, 0, st, p, mask)
               ? GPT_ATTN_OK
               : GPT_ATTN_ERR_CUDA;
}

template <int D>
int launch_bwd_grads(const void* q, const void* k, const void* v, const void* dout, void* dk, void* dv, int B,
                     int H, int T, float scale, const MaskParams& mask, const Layout& L, void* ws, cudaStream_t st,
                     const SinkMask* sinks = nullptr) {
    const int BH = B * H;
    const WsLayout w = ws_layout(ws, BH, T, D);
    CUtensorMap mq, mk, mv, mdo;
    if (!make_tmap_bf16(&mq, q, B, H, T, D, L.q) || !make_tmap_bf16(&mk, k, B, H, T, D, L.k) ||
        !make_tmap_bf16(&mv, v, B, H, T, D, L.v) || !make_tmap_bf16(&mdo, dout, B, H, T, D, L.dO))
        return GPT_ATTN_ERR_CUDA;
    BwdParams p;
    p.lse2 = w.lse2;
    p.delta = w.delta;
    p.dq_acc = w.dq_acc;
    p.sched = w.sched;
    p.dk = static_cast<__nv_bfloat16*>(dk);
    p.dv = static_cast<__nv_bfloat16*>(dv);
    p.dk_str = L.dk;
    p.dv_str = L.dv;
    p.H = H;
    p.T = T;
    p.T_pad = w.T_pad;
    p.BH = BH;
    p.n_tiles = w.n_tiles;
    p.cut = make_cut(0, 1, w.n_tiles);
    if (sinks && !mask.doc_start) p.cut = launch_cut(BH, T, *sinks, mask);
    p.part = sink_part(ws, BH, T, D);
    p.units = BH * (p.cut.units + w.n_tiles - p.cut.n_s);
    p.tail = tail_heads(BH, std::max(1, w.n_tiles - p.cut.n_s), sm_count());
    p.lower2 = mask.doc_start ? w.lower2 : nullptr;
    p.last_qt = mask.doc_start ? w.last_qt : nullptr;
    const ScoreScale ss = score_scale(scale);
    p.scale_log2 = ss.log2;
    p.score_sign = ss.sign;
    p.scale = scale;
    p.timeout_ns = wait_timeout_ns();
    const int units = p.units;
    const unsigned grid = (unsigned)units;
    if constexpr (D == 64) {
        CUtensorMap mdq, mdk, mdv;
        if (!make_tmap_f32_acc(&mdq, w.dq_acc, BH, T, D) || !make_tmap_bf16(&mdk, dk, B, H, T, D, L.dk) ||
            !make_tmap_bf16(&mdv, dv, B, H, T, D, L.dv))
            return GPT_ATTN_ERR_CUDA;
        const size_t smem = sizeof(Bwd64Smem) + 1024;
        // persistent: one CTA per SM, work units taken from the counter in the workspace
        const unsigned pgrid = (unsigned)(units < sm_count() ? units : sm_count());
        if (sinks && p.cut.most > 1) {
            if (!set_smem(attn_bwd_kernel<CutSinkMask>, smem)) return GPT_ATTN_ERR_CUDA;
            attn_bwd_kernel<CutSinkMask><<<pgrid, kBwd64Threads, smem, st>>>(mq, mk, mv, mdo, mdq, mdk, mdv, p,
                                                                           CutSinkMask{*sinks});
        } else if (sinks) {
            if (!set_smem(attn_bwd_kernel<SinkMask>, smem)) return GPT_ATTN_ERR_CUDA;
            attn_bwd_kernel<SinkMask><<<pgrid, kBwd64Threads, smem, st>>>(mq, mk, mv, mdo, mdq, mdk, mdv, p, *sinks);
        } else if (plain_window(mask)) {
            if (!set_smem(attn_bwd_kernel<WindowMask>, smem)) return GPT_ATTN_ERR_CUDA;
            attn_bwd_kernel<WindowMask><<<pgrid, kBwd64Threads, smem, st>>>(mq, mk, mv, mdo, mdq, mdk, mdv, p,
                                                                          WindowMask{mask.window});
        } else {
            if (!set_smem(attn_bwd_kernel<MaskParams>, smem)) return GPT_ATTN_ERR_CUDA;
            attn_bwd_kernel<MaskParams><<<pgrid, kBwd64Threads, smem, st>>>(mq, mk, mv, mdo, mdq, mdk, mdv, p, mask);
        }
    } else {
        CUtensorMap mdq;
        if (!make_tmap_f32_acc(&mdq, w.dq_acc, BH, T, D)) return GPT_ATTN_ERR_CUDA;
        const size_t smem = sizeof(BwdSmem<D>) + 1024;
        if (sinks && p.cut.most > 1) {
            if (!set_smem(attn_bwd_serial_kernel<D, CutSinkMask>, smem)) return GPT_ATTN_ERR_CUDA;
            attn_bwd_serial_kernel<D, CutSinkMask><<<grid, kBwdThreads, smem, st>>>(mq, mk, mv, mdo, mdq, p,
                                                                                  CutSinkMask{*sinks});
        } else if (sinks) {
            if (!set_smem(attn_bwd_serial_kernel<D, SinkMask>, smem)) return GPT_ATTN_ERR_CUDA;
            attn_bwd_serial_kernel<D, SinkMask><<<grid, kBwdThreads, smem, st>>>(mq, mk, mv, mdo, mdq, p, *sinks);
        } else if (plain_window(mask)) {
            if (!set_smem(attn_bwd_serial_kernel<D, WindowMask>, smem)) return GPT_ATTN_ERR_CUDA;
            attn_bwd_serial_kernel<D, WindowMask><<<grid, kBwdThreads, smem, st>>>(mq, mk, mv, mdo, mdq, p,
                                                                                 WindowMask{mask.window});
        } else {
            if (!set_smem(attn_bwd_serial_kernel<D, MaskParams>, smem)) return GPT_ATTN_ERR_CUDA;
            attn_bwd_serial_kernel<D, MaskParams><<<grid, kBwdThreads, smem, st>>>(mq, mk, mv, mdo, mdq, p, mask);
        }
    }
    if (cudaGetLastError() != cudaSuccess) return GPT_ATTN_ERR_CUDA;
    if (p.cut.most > 1) {
        const dim3 jgrid(2 * kTile * (D / 8) / 256, (unsigned)(BH * p.cut.n_s));
        attn_sink_join_kernel<D><<<jgrid, 256, 0, st>>>(p.part, p.dk, p.dv, L.dk, L.dv, p.cut, w.n_tiles, T, H);
        if (cudaGetLastError() != cudaSuccess) return GPT_ATTN_ERR_CUDA;
    }
    return GPT_ATTN_OK;
}

int launch_dq_convert(void* dq, int B, int H, int T, int D, float scale, void* ws, const Layout& L, cudaStream_t st) {
    const int BH = B * H;
    const WsLayout w = ws_layout(ws, BH, T, D);
    const long long rows = (long long)BH * T;
    const int rows_per_block = 256 / (D / 8);
    const unsigned grid = (unsigned)((rows + rows_per_block - 1) / rows_per_block);
    auto* dq16 = static_cast<__nv_bfloat16*>(dq);
    if (D == 64)
        attn_dq_convert_kernel<64><<<grid, 256, 0, st>>>(w.dq_acc, dq16, rows, scale, T, H, L.dq);
    else
        attn_dq_convert_kernel<128><<<grid, 256, 0, st>>>(w.dq_acc, dq16, rows, scale, T, H, L.dq);
    return cudaGetLastError() == cudaSuccess ? GPT_ATTN_OK : GPT_ATTN_ERR_CUDA;
}

int check_ws(int B, int H, int T, int D, const void* ws, size_t ws_bytes) {
    if (!ws || ws_bytes < gpt_attn_bwd_workspace_bytes(B, H, T, D)) return GPT_ATTN_ERR_WORKSPACE;
    return misaligned(ws) ? GPT_ATTN_ERR_ALIGN : GPT_ATTN_OK;
}

// Decode split: as many splits per head as fit all CTAs on a B200 (148 SMs, kDecodeBlocksPerSm
// resident each) in one wave, at least one, at least 64 keys per split, at most kDecodeMaxChunk.
// A CTA's passes over its keys and values are chains of dependent load rounds, so shorter chunks
// over more CTAs keep more of HBM busy, and a second wave would add a whole chain.  The same
// function sizes the workspace and the launch.
int decode_splits(int BH, int T_max, int window, int* chunk) {
    const int span = (window > 0 && window < T_max) ? window : T_max;   // keys one query can see
    int n = kDecodeBlocksPerSm * 148 / BH;
    const int by_len = (span + 63) / 64;
    if (n > by_len) n = by_len;
    if (n < 1) n = 1;
    if ((span + n - 1) / n > kDecodeMaxChunk) n = (span + kDecodeMaxChunk - 1) / kDecodeMaxChunk;
    *chunk = (span + n - 1) / n;
    return n;
}

int check_decode_shape(int B, int H, int T_max, int D) {
    if (B < 1 || H < 1 || T_max < 1) return GPT_ATTN_ERR_SHAPE;
    if (D != 64 && D != 128) return GPT_ATTN_ERR_UNSUPPORTED_D;
    const long long bh = (long long)B * H;
    if (bh > 0x7fffffffLL) return GPT_ATTN_ERR_SHAPE;                    // grid x
    if ((long long)T_max / 64 + 1 > 65535) return GPT_ATTN_ERR_SHAPE;     // splits on grid y
    if ((long long)T_max > (0x7fffffffffffffffLL / D) / bh) return GPT_ATTN_ERR_SHAPE;
    return GPT_ATTN_OK;
}

template <int D>
int launch_decode(const void* q, const void* k, const void* v, const int* lens, void* o, float* lse, int B, int H,
                  int T_max, float scale, int window, void* ws, cudaStream_t st) {
    DecodeParams p;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.lens = lens;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.H = H;
    p.T_max = T_max;
    p.window = window > 0 ? window : 0;
    p.scale_log2 = scale * 1.4426950408889634f;
    const int BH = B * H;
    p.n_split = decode_splits(BH, T_max, p.window, &p.chunk);
    p.part_o = static_cast<float*>(ws);
    p.part_ml = p.part_o + (size_t)BH * p.n_split * D;
    constexpr int R = kDecodeThreads / (D / 8);
    const size_t smem = (size_t)(p.chunk > R * D ? p.chunk : R * D) * sizeof(float);
    if (!set_smem(attn_decode_split_kernel<D>, smem)) return GPT_ATTN_ERR_CUDA;
    const dim3 grid(BH, p.n_split);
    attn_decode_split_kernel<D><<<grid, kDecodeThreads, smem, st>>>(p);
    if (p.n_split > 1) attn_decode_combine_kernel<D><<<BH, D, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? GPT_ATTN_OK : GPT_ATTN_ERR_CUDA;
}

// Strides of n tensors from the C ABI (nullptr: contiguous [B, H, T, D]); same rules as layouts.
int prologue_strides(Strides* out, const gpt_attn_strides* in, int n, int H, int T, int D) {
    for (int i = 0; i < n; ++i) {
        out[i] = contiguous(H, T, D);
        if (!in) continue;
        const gpt_attn_strides& x = in[i];
        if (x.batch < 0 || x.head < 0 || x.token < 0) return GPT_ATTN_ERR_SHAPE;
        if ((x.batch | x.head | x.token) & 7) return GPT_ATTN_ERR_ALIGN;
        out[i] = Strides{x.batch, x.head, x.token};
    }
    return GPT_ATTN_OK;
}

int launch_prologue(bool backward, const PrologueParams& p, int D, cudaStream_t st) {
    // persistent: 2 blocks per SM for each of q and k, all resident at once (4 x 256 threads of
    // at most 64 registers); a lane group takes a row, or a whole token for token-major inputs
    const long long per_block = kPrologueThreads / (D / 16);
    const long long units = p.token_major ? p.rows / p.H : p.rows;
    const long long need = (units + per_block - 1) / per_block;
    const dim3 grid((unsigned)std::min<long long>(need, 2LL * sm_count()), 2);
    if (p.token_major) {
        if (backward) {
            if (D == 64) qk_prologue_bwd_tok_kernel<64><<<grid, 256, 0, st>>>(p);
            else qk_prologue_bwd_tok_kernel<128><<<grid, 256, 0, st>>>(p);
        } else {
            if (D == 64) qk_prologue_fwd_tok_kernel<64><<<grid, 256, 0, st>>>(p);
            else qk_prologue_fwd_tok_kernel<128><<<grid, 256, 0, st>>>(p);
        }
        return cudaGetLastError() == cudaSuccess ? GPT_ATTN_OK : GPT_ATTN_ERR_CUDA;
    }
    if (backward) {
        if (D == 64) qk_prologue_bwd_kernel<64><<<grid, 256, 0, st>>>(p);
        else qk_prologue_bwd_kernel<128><<<grid, 256, 0, st>>>(p);
    } else {
        if (D == 64) qk_prologue_fwd_kernel<64><<<grid, 256, 0, st>>>(p);
        else qk_prologue_fwd_kernel<128><<<grid, 256, 0, st>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? GPT_ATTN_OK : GPT_ATTN_ERR_CUDA;
}

// A paged cache description, checked: sizes, alignment, and that row numbers fit an int.
int check_cache(PagedPools* c, const gpt_attn_paged_cache* a) {
    if (!a || !a->k_pages || !a->v_pages || !a->table || !a->lens) return GPT_ATTN_ERR_NULL;
    if (a->B < 1 || a->Hkv < 1 || a->n_pages < 1 || a->page < 1 || a->max_pages < 1) return GPT_ATTN_ERR_SHAPE;
    if (a->D != 64 && a->D != 128) return GPT_ATTN_ERR_UNSUPPORTED_D;
    if ((long long)a->max_pages * a->page > (1LL << 30)) return GPT_ATTN_ERR_SHAPE;
    const long long heads = (long long)a->n_pages * a->Hkv;
    if (heads > 0x7fffffffLL || heads * a->page > 0x7fffffffLL) return GPT_ATTN_ERR_SHAPE;
    if ((long long)a->B * a->Hkv > 0x7fffffffLL) return GPT_ATTN_ERR_SHAPE;       // grid x
    if (misaligned(a->k_pages) || misaligned(a->v_pages) || (reinterpret_cast<uintptr_t>(a->table) & 3u) ||
        (reinterpret_cast<uintptr_t>(a->lens) & 3u))
        return GPT_ATTN_ERR_ALIGN;
    c->k = static_cast<__nv_bfloat16*>(a->k_pages);
    c->v = static_cast<__nv_bfloat16*>(a->v_pages);
    c->table = a->table;
    c->lens = a->lens;
    c->n_pages = a->n_pages;
    c->Hkv = a->Hkv;
    c->page = fast_div(a->page);
    c->max_pages = a->max_pages;
    c->cap = a->max_pages * a->page;
    return GPT_ATTN_OK;
}

bool misaligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

// How an item's rows are cut: up to 32 go through the kernel on warp-level products, more through the one on
// tcgen05 tiles of 128 rows.  32 rows over 8 contexts up to 8192 (6 heads of 128): 43.6 against 45.5 us; 52 rows,
// when the former took up to 64, over 16 streams with a window of 4096: 59.5 against 52.5; one row: 32 against 71.
struct PagedShape {
    int R, block, RB;             // rows of an item, of a row block, row blocks
};
PagedShape paged_shape(int H, int Hkv, int N) {
    PagedShape s;
    s.R = H / Hkv * N;
    s.block = s.R <= 16 ? 16 : (s.R <= 32 ? 32 : kPagedTcRows);
    s.RB = (s.R + s.block - 1) / s.block;
    return s;
}

int check_paged_shape(int B, int H, int Hkv, int N, int D) {
    if (B < 1 || H < 1 || Hkv < 1 || N < 1 || N > kMaxNodes || H % Hkv) return GPT_ATTN_ERR_SHAPE;
    if (D != 64 && D != 128) return GPT_ATTN_ERR_UNSUPPORTED_D;
    if ((long long)H / Hkv * N > (1 << 20)) return GPT_ATTN_ERR_SHAPE;
    if ((long long)B * Hkv * paged_shape(H, Hkv, N).RB > 0x7fffffffLL) return GPT_ATTN_ERR_SHAPE;   // grid x
    return GPT_ATTN_OK;
}

// Blocks of the paged decode kernel, one to an SM of a B200 (148), and the teams in them; the
// workspace is sized by them.
constexpr int kPagedBlocks = 148, kPagedAllTeams = kPagedTeams * kPagedBlocks;

template <int D, int kTile, int kRows, typename Kern>
int launch_paged_kernels(Kern kernel, unsigned threads, size_t smem, const PagedParams& p, int grid, cudaStream_t st) {
    CUtensorMap mk, mv;
    const int rows = p.n_pages * p.Hkv * p.page.d, box = 1 << p.box_log2;
    if (!make_tmap_rows(&mk, p.k, rows, D, box) || !make_tmap_rows(&mv, p.v, rows, D, box) || !set_smem(kernel, smem))
        return GPT_ATTN_ERR_CUDA;
    kernel<<<grid, threads, smem, st>>>(mk, mv, p);
    if (cudaGetLastError() != cudaSuccess) return GPT_ATTN_ERR_CUDA;
    const int item_rows = p.R < kRows ? p.R : kRows;
    const dim3 cgrid((unsigned)(p.B * p.Hkv * p.RB), (unsigned)((item_rows + kCombineWarps - 1) / kCombineWarps));
    return launch_dependent(paged_combine_kernel<D, kTile, kRows>, cgrid, 32 * kCombineWarps, 0, st, p) ? GPT_ATTN_OK
                                                                                                        : GPT_ATTN_ERR_CUDA;
}

template <int D>
int launch_paged(const PagedParams& p, int block, int grid, cudaStream_t st) {
    if (block == kPagedTcRows)
        return launch_paged_kernels<D, kPagedTcTile, kPagedTcRows>(paged_decode_tc_kernel<D>, kPagedTcThreads,
                                                                   sizeof(PagedTcSmem<D>) + 1024, p, grid, st);
    constexpr int kTile = PagedCfg<D>::kTile;
    const size_t smem = sizeof(PagedSmem<D>) + 1024;
    // up to 8 rows leave the other half of a 16-row tile to their second terms of P: 31.8 us where products of
    // their own take 34.9 (one token of 64 sequences of up to 1024)
    if (block == 16)
        return launch_paged_kernels<D, kTile, 16>(p.R <= 8 ? paged_decode_kernel<D, 1, true> : paged_decode_kernel<D, 1, false>,
                                                  kPagedThreads, smem, p, grid, st);
    return launch_paged_kernels<D, kTile, 32>(paged_decode_kernel<D, 2, false>, kPagedThreads, smem, p, grid, st);
}

// Strides of n [b, h, n, d] tensors from the C ABI (nullptr: contiguous); as for layouts.
int paged_strides(Strides* out, const gpt_attn_strides* in, const int* heads, int n, int N, int D) {
    for (int i = 0; i < n; ++i) {
        const int sc = prologue_strides(out + i, in ? in + i : nullptr, 1, heads[i], N, D);
        if (sc != GPT_ATTN_OK) return sc;
    }
    return GPT_ATTN_OK;
}

// The table kernels go through slots and pages in steps of up to 8192, so that a place past the last one has
// to fit an int too.
int check_pages(int S, int M, int P) {
    constexpr int kMost = 0x7fffffff - 2 * kPagesCluster * kPagesThreads;
    if (S < 1 || M < 1 || P < 1 || S > kMost || P > kMost) return GPT_ATTN_ERR_SHAPE;
    return (long long)S * M > 0x7fffffffLL ? GPT_ATTN_ERR_SHAPE : GPT_ATTN_OK;
}

// Workspace of the table calls: pages asked for [S] | free pages, or new places [P] | counts.
int pages_params(PagesParams* p, int S, int M, int P, void* ws, size_t ws_bytes) {
    const int sc = check_pages(S, M, P);
    if (sc != GPT_ATTN_OK) return sc;
    if (!ws || ws_bytes < gpt_attn_pages_workspace_bytes(S, M, P)) return GPT_ATTN_ERR_WORKSPACE;
    if (misaligned(ws)) return GPT_ATTN_ERR_ALIGN;
    p->S = S;
    p->M = M;
    p->P = P;
    p->need = static_cast<int*>(ws);
    p->list = p->need + S;
    p->counts = p->list + P;
    return GPT_ATTN_OK;
}

__global__ void debug_wait_kernel(uint64_t timeout_ns) {
    __shared__ uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);   // nothing ever arrives
        abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    const AbortCtl ac{&abort_flag, timeout_ns};
    if (threadIdx.x == 0) (void)mbar_wait(&bar, 0, ac);
    __syncthreads();
}

}  // namespace

// ---------------------------------------------------------------------------
// Built-in scratch for gpt_attn_bwd_noalloc.  A file-scope device array is
// created when the library's module is loaded on a device and lives until the
// process exits, so the entry point below never allocates.  In host code the
// name g_noalloc_scratch is only a host-side shadow symbol, not a device
// address: the device address is looked up with cudaGetSymbolAddress with the
// caller's device current.
constexpr size_t kNoAllocScratchBytes = size_t(32) << 20;   // 32 MiB
__device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

namespace {
// Device address of the scratch array on the current device, or nullptr on a
// CUDA error.  Looked up on every call (a table lookup once the module is
// loaded) rather than cached: after a cudaDeviceReset the module is loaded
// again and the array may live at a different address.
void* noalloc_scratch_current_device() {
    void* ptr = nullptr;
    if (cudaGetSymbolAddress(&ptr, g_noalloc_scratch) != cudaSuccess) return nullptr;
    return ptr;
}
}  // namespace
}  // namespace gpt_attn

using namespace gpt_attn;

extern "C" {

int gpt_attn_fwd_sinks(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int T, int D,
                       float scale, const gpt_attn_mask* mask, int sinks, const gpt_attn_layout* layout,
                       void* stream) {
    if (!q || !k || !v || !o || !lse) return GPT_ATTN_ERR_NULL;
    int sc = check_shape(B, H, T, D);
    if (sc != GPT_ATTN_OK) return sc;
    if (misaligned(q) || misaligned(k) || misaligned(v) || misaligned(o) || misaligned(lse)) return GPT_ATTN_ERR_ALIGN;
    MaskParams m;
    if ((sc = make_mask(&m, mask, H, T)) != GPT_ATTN_OK) return sc;
    Layout L;
    if ((sc = make_layout(&L, layout, H, T, D)) != GPT_ATTN_OK) return sc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    SinkMask sm;
    const SinkMask* sp = sink_mask(&sm, m, sinks, H, T) ? &sm : nullptr;
    return D == 64 ? launch_fwd<64>(q, k, v, o, lse, B, H, T, scale, m, L, st, sp)
                   : launch_fwd<128>(q, k, v, o, lse, B, H, T, scale, m, L, st, sp);
}

int gpt_attn_fwd_ex(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int T, int D,
                    float scale, const gpt_attn_mask* mask, const gpt_attn_layout* layout, void* stream) {
    return gpt_attn_fwd_sinks(q, k, v, o, lse, B, H, T, D, scale, mask, 0, layout, stream);
}

int gpt_attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int T, int D,
                 float scale, int window, void* stream) {
    const gpt_attn_mask m{window, nullptr, nullptr};
    return gpt_attn_fwd_ex(q, k, v, o, lse, B, H, T, D, scale, &m, nullptr, stream);
}

size_t gpt_attn_bwd_workspace_bytes(int B, int H, int T, int D) {
    if (check_shape(B, H, T, D) != GPT_ATTN_OK) return 0;
    const size_t bh = (size_t)B * H;
    const size_t t_pad = ((size_t)T + 127) / 128 * 128;
    return 4 * (bh * T * D + 3 * bh * t_pad + bh * (t_pad / 128)) + 16;
}

int gpt_attn_bwd_delta(const void* o, const float* lse, const void* dO, int B, int H, int T, int D,
                       void* workspace, size_t workspace_bytes, void* stream) {
    if (!o || !lse || !dO) return GPT_ATTN_ERR_NULL;
    int sc = check_shape(B, H, T, D);
    if (sc != GPT_ATTN_OK) return sc;
    if ((sc = check_ws(B, H, T, D, workspace, workspace_bytes)) != GPT_ATTN_OK) return sc;
    if (misaligned(o) || misaligned(lse) || misaligned(dO)) return GPT_ATTN_ERR_ALIGN;
    return launch_bwd_delta(o, lse, dO, B, H, T, D, workspace, window_mask(0, H, T), contiguous_layout(H, T, D),
                            static_cast<cudaStream_t>(stream));
}

int gpt_attn_bwd_grads(const void* q, const void* k, const void* v, const void* dO, void* dk, void* dv, int B,
                       int H, int T, int D, float scale, int window, void* workspace, size_t workspace_bytes,
                       void* stream) {
    if (!q || !k || !v || !dO || !dk || !dv) return GPT_ATTN_ERR_NULL;
    int sc = check_shape(B, H, T, D);
    if (sc != GPT_ATTN_OK) return sc;
    if ((sc = check_ws(B, H, T, D, workspace, workspace_bytes)) != GPT_ATTN_OK) return sc;
    if (misaligned(q) || misaligned(k) || misaligned(v) || misaligned(dO) || misaligned(dk) || misaligned(dv))
        return GPT_ATTN_ERR_ALIGN;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const MaskParams m = window_mask(window, H, T);
    const Layout L = contiguous_layout(H, T, D);
    return D == 64 ? launch_bwd_grads<64>(q, k, v, dO, dk, dv, B, H, T, scale, m, L, workspace, st)
                   : launch_bwd_grads<128>(q, k, v, dO, dk, dv, B, H, T, scale, m, L, workspace, st);
}

int gpt_attn_bwd_dq_convert(void* dq, int B, int H, int T, int D, float scale, void* workspace,
                            size_t workspace_bytes, void* stream) {
    if (!dq) return GPT_ATTN_ERR_NULL;
    int sc = check_shape(B, H, T, D);
    if (sc != GPT_ATTN_OK) return sc;
    if ((sc = check_ws(B, H, T, D, workspace, workspace_bytes)) != GPT_ATTN_OK) return sc;
    if (misaligned(dq)) return GPT_ATTN_ERR_ALIGN;
    return launch_dq_convert(dq, B, H, T, D, scale, workspace, contiguous_layout(H, T, D),
                             static_cast<cudaStream_t>(stream));
}

size_t gpt_attn_bwd_sinks_workspace_bytes(int B, int H, int T, int D, int window, int sinks) {
    const size_t plain = gpt_attn_bwd_workspace_bytes(B, H, T, D);
    const size_t part = plain ? sink_part_bytes(B * H, T, D, window, sinks) : 0;
    return part ? sink_part_at(B * H, T, D) + part : plain;
}

int gpt_attn_bwd_sinks(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                       void* dq, void* dk, void* dv, int B, int H, int T, int D, float scale, const gpt_attn_mask* mask,
                       int sinks, const gpt_attn_layout* layout, void* workspace, size_t workspace_bytes, void* stream) {
    if (!q || !k || !v || !o || !lse || !dO || !dq || !dk || !dv) return GPT_ATTN_ERR_NULL;
    int sc = check_shape(B, H, T, D);
    if (sc != GPT_ATTN_OK) return sc;
    if ((sc = check_ws(B, H, T, D, workspace, workspace_bytes)) != GPT_ATTN_OK) return sc;
    if (misaligned(q) || misaligned(k) || misaligned(v) || misaligned(o) || misaligned(lse) || misaligned(dO) ||
        misaligned(dq) || misaligned(dk) || misaligned(dv))
        return GPT_ATTN_ERR_ALIGN;
    MaskParams m;
    if ((sc = make_mask(&m, mask, H, T)) != GPT_ATTN_OK) return sc;
    Layout L;
    if ((sc = make_layout(&L, layout, H, T, D)) != GPT_ATTN_OK) return sc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    SinkMask sm;
    const SinkMask* sp = sink_mask(&sm, m, sinks, H, T) ? &sm : nullptr;
    if (sp && !m.doc_start) {
        const SinkCut cut = launch_cut(B * H, T, sm, m);
        if (cut.most > 1 && workspace_bytes < sink_part_at(B * H, T, D) + sink_part_bytes_of(cut, B * H, D))
            return GPT_ATTN_ERR_WORKSPACE;
    }
    if (sinks > 0) {
        sc = launch_bwd_delta(o, lse, dO, B, H, T, D, workspace, sm, L, st, exact_delta_rows(sm, H, T));
        if (sc == GPT_ATTN_OK) sc = launch_exact_delta(q, k, v, lse, dO, B, H, T, D, scale, workspace, sm, L, st);
    } else {
        sc = launch_bwd_delta(o, lse, dO, B, H, T, D, workspace, m, L, st);
    }
    if (sc != GPT_ATTN_OK) return sc;
    sc = D == 64 ? launch_bwd_grads<64>(q, k, v, dO, dk, dv, B, H, T, scale, m, L, workspace, st, sp)
                 : launch_bwd_grads<128>(q, k, v, dO, dk, dv, B, H, T, scale, m, L, workspace, st, sp);
    if (sc != GPT_ATTN_OK) return sc;
    return launch_dq_convert(dq, B, H, T, D, scale, workspace, L, st);
}

int gpt_attn_bwd_ex(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                    void* dq, void* dk, void* dv, int B, int H, int T, int D, float scale, const gpt_attn_mask* mask,
                    const gpt_attn_layout* layout, void* workspace, size_t workspace_bytes, void* stream) {
    return gpt_attn_bwd_sinks(q, k, v, o, lse, dO, dq, dk, dv, B, H, T, D, scale, mask, 0, layout, workspace,
                              workspace_bytes, stream);
}

int gpt_attn_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                 void* dq, void* dk, void* dv, int B, int H, int T, int D, float scale, int window, void* workspace,
                 size_t workspace_bytes, void* stream) {
    const gpt_attn_mask m{window, nullptr, nullptr};
    return gpt_attn_bwd_ex(q, k, v, o, lse, dO, dq, dk, dv, B, H, T, D, scale, &m, nullptr, workspace,
                           workspace_bytes, stream);
}

size_t gpt_attn_decode_workspace_bytes(int B, int H, int T_max, int D, int window) {
    if (check_decode_shape(B, H, T_max, D) != GPT_ATTN_OK) return 0;
    int chunk = 0;
    const int n = decode_splits(B * H, T_max, window > 0 ? window : 0, &chunk);
    return n > 1 ? (size_t)B * H * n * (D + 2) * sizeof(float) : 16;
}

int gpt_attn_decode(const void* q, const void* k_cache, const void* v_cache, const int* seq_lens, void* o,
                    float* lse, int B, int H, int T_max, int D, float scale, int window, void* workspace,
                    size_t workspace_bytes, void* stream) {
    if (!q || !k_cache || !v_cache || !seq_lens || !o || !lse) return GPT_ATTN_ERR_NULL;
    const int sc = check_decode_shape(B, H, T_max, D);
    if (sc != GPT_ATTN_OK) return sc;
    const size_t need = gpt_attn_decode_workspace_bytes(B, H, T_max, D, window);
    if (!workspace || workspace_bytes < need) return GPT_ATTN_ERR_WORKSPACE;
    if (misaligned(q) || misaligned(k_cache) || misaligned(v_cache) || misaligned(o) || misaligned(workspace) ||
        (reinterpret_cast<uintptr_t>(lse) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
        return GPT_ATTN_ERR_ALIGN;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return D == 64 ? launch_decode<64>(q, k_cache, v_cache, seq_lens, o, lse, B, H, T_max, scale, window, workspace, st)
                   : launch_decode<128>(q, k_cache, v_cache, seq_lens, o, lse, B, H, T_max, scale, window, workspace,
                                        st);
}

size_t gpt_attn_paged_decode_workspace_bytes(int B, int H, int Hkv, int N, int D) {
    if (check_paged_shape(B, H, Hkv, N, D) != GPT_ATTN_OK) return 0;
    const size_t rows = paged_shape(H, Hkv, N).block;
    return 2 * (size_t)kPagedAllTeams * rows * (D + 2) * sizeof(float) + ((size_t)B + 2) * sizeof(int);
}

int gpt_attn_paged_decode(const void* q, const gpt_attn_paged_cache* cache, const int* n_new, const int* parents,
                          void* o, float* lse, int H, int N, float scale, int window, int sinks,
                          const gpt_attn_strides* strides, void* workspace, size_t workspace_bytes, void* stream) {
    if (!q || !o || !lse) return GPT_ATTN_ERR_NULL;
    PagedPools c;
    int sc = check_cache(&c, cache);
    if (sc != GPT_ATTN_OK) return sc;
    const int B = cache->B, D = cache->D;
    if ((sc = check_paged_shape(B, H, c.Hkv, N, D)) != GPT_ATTN_OK) return sc;
    if (!workspace || workspace_bytes < gpt_attn_paged_decode_workspace_bytes(B, H, c.Hkv, N, D))
        return GPT_ATTN_ERR_WORKSPACE;
    if (misaligned(q) || misaligned(o) || misaligned(workspace) || misaligned4(lse) || misaligned4(n_new) ||
        misaligned4(parents))
        return GPT_ATTN_ERR_ALIGN;
    PagedParams p;
    Strides st[2];
    const int heads[2] = {H, H};
    if ((sc = paged_strides(st, strides, heads, 2, N, D)) != GPT_ATTN_OK) return sc;
    const PagedShape s = paged_shape(H, c.Hkv, N);
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = c.k;
    p.v = c.v;
    p.table = c.table;
    p.lens = c.lens;
    p.n_new = n_new;
    p.parents = parents;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.q_str = st[0];
    p.o_str = st[1];
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = p.part_o + 2 * (size_t)kPagedAllTeams * s.block * D;
    p.prefix = reinterpret_cast<int*>(p.part_ml + 2 * (size_t)kPagedAllTeams * s.block * 2);
    p.B = B;
    p.H = H;
    p.Hkv = c.Hkv;
    p.G = H / c.Hkv;
    p.N = N;
    p.by_n = fast_div(N);
    p.R = s.R;
    p.RB = s.RB;
    p.item_cost = paged_item_cost(s.R);
    p.page = c.page;
    p.box_log2 = 0;
    while ((1 << p.box_log2) < paged_box(c.page.d)) ++p.box_log2;
    p.max_pages = c.max_pages;
    p.n_pages = c.n_pages;
    p.cap = c.cap;
    p.window = window > 0 ? window : 0;
    p.sinks = sinks > 0 && window > 0 ? sinks : 0;
    p.scale_log2 = scale == 0.f ? 1.f : fabsf(scale) * 1.4426950408889634f;
    p.q_keep = scale == 0.f ? 0u : 0xffffffffu;
    p.q_flip = scale < 0.f ? 0x80008000u : 0u;
    p.timeout_ns = wait_timeout_ns();
    // No more blocks than the tables can name tiles; places in the list of them have to fit an int.
    const int tile = s.block == kPagedTcRows || D == 128 ? kPagedTcTile : PagedCfg<64>::kTile;
    const long long items = (long long)B * c.Hkv * s.RB, tiles = (c.cap + tile - 1) / tile + p.item_cost;
    if (items > 0x7fffffffLL / tiles) return GPT_ATTN_ERR_SHAPE;
    const long long most = items * tiles;
    const int grid = (int)(most < kPagedBlocks ? most : kPagedBlocks);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return D == 64 ? launch_paged<64>(p, s.block, grid, cs) : launch_paged<128>(p, s.block, grid, cs);
}

int gpt_attn_paged_append(const gpt_attn_paged_cache* cache, const void* k_new, const void* v_new, int N,
                          const int* n_new, const gpt_attn_strides* strides, void* stream) {
    if (!k_new || !v_new) return GPT_ATTN_ERR_NULL;
    AppendParams p;
    int sc = check_cache(&p.c, cache);
    if (sc != GPT_ATTN_OK) return sc;
    if (N < 1) return GPT_ATTN_ERR_SHAPE;
    if (misaligned(k_new) || misaligned(v_new) || misaligned4(n_new)) return GPT_ATTN_ERR_ALIGN;
    Strides st[2];
    const int heads[2] = {cache->Hkv, cache->Hkv};
    if ((sc = paged_strides(st, strides, heads, 2, N, cache->D)) != GPT_ATTN_OK) return sc;
    p.k_new = static_cast<const __nv_bfloat16*>(k_new);
    p.v_new = static_cast<const __nv_bfloat16*>(v_new);
    p.k_str = st[0];
    p.v_str = st[1];
    p.n_new = n_new;
    p.N = N;
    const long long rows = (long long)cache->B * cache->Hkv;
    if (N > (0x7fffffffLL * 256 / 16) / rows) return GPT_ATTN_ERR_SHAPE;            // grid size
    p.chunks = rows * N * (cache->D / 8);
    const unsigned grid = (unsigned)((p.chunks + 255) / 256);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (cache->D == 64) paged_append_kernel<64><<<grid, 256, 0, cs>>>(p);
    else paged_append_kernel<128><<<grid, 256, 0, cs>>>(p);
    return cudaGetLastError() == cudaSuccess ? GPT_ATTN_OK : GPT_ATTN_ERR_CUDA;
}

int gpt_attn_paged_accept(const gpt_attn_paged_cache* cache, const int* accepted, const int* n_accepted, int N,
                          void* stream) {
    if (!accepted || !n_accepted) return GPT_ATTN_ERR_NULL;
    AcceptParams p;
    const int sc = check_cache(&p.c, cache);
    if (sc != GPT_ATTN_OK) return sc;
    if (N < 1 || N > kMaxNodes) return GPT_ATTN_ERR_SHAPE;
    if (misaligned4(accepted) || misaligned4(n_accepted)) return GPT_ATTN_ERR_ALIGN;
    p.accepted = accepted;
    p.n_accepted = n_accepted;
    p.N = N;
    const unsigned grid = (unsigned)(cache->B * cache->Hkv);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (cache->D == 64) paged_accept_kernel<64><<<grid, kAcceptThreads, 0, cs>>>(p);
    else paged_accept_kernel<128><<<grid, kAcceptThreads, 0, cs>>>(p);
    return cudaGetLastError() == cudaSuccess ? GPT_ATTN_OK : GPT_ATTN_ERR_CUDA;
}

size_t gpt_attn_pages_workspace_bytes(int S, int M, int P) {
    if (check_pages(S, M, P) != GPT_ATTN_OK) return 0;
    return ((size_t)S + P + 4 * kPagesCluster) * sizeof(int);
}

int gpt_attn_pages_reserve(int* table, const int* lens, int* refs, int S, int M, int P, int page, const int* tokens,
                           int* status, void* workspace, size_t workspace_bytes, void* stream) {
    if (!table || !lens || !refs || !tokens || !status) return GPT_ATTN_ERR_NULL;
    PagesParams p{};
    const int sc = pages_params(&p, S, M, P, workspace, workspace_bytes);
    if (sc != GPT_ATTN_OK) return sc;
    if (page < 1) return GPT_ATTN_ERR_SHAPE;
    if (misaligned4(table) || misaligned4(lens) || misaligned4(refs) || misaligned4(tokens) || misaligned4(status))
        return GPT_ATTN_ERR_ALIGN;
    p.table = table;
    p.lens = const_cast<int*>(lens);
    p.refs = refs;
    p.page = page;
    p.arg = tokens;
    p.status = status;
    pages_take_kernel<false><<<kPagesCluster, kPagesThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? GPT_ATTN_OK : GPT_ATTN_ERR_CUDA;
}

int gpt_attn_pages_fork(int* table, int* lens, int* refs, int S, int M, int P, int page, const int* parents,
                        int* status, int* pairs, void* workspace, size_t workspace_bytes, void* stream) {
    if (!table || !lens || !refs || !parents || !status || !pairs) return GPT_ATTN_ERR_NULL;
    PagesParams p{};
    const int sc = pages_params(&p, S, M, P, workspace, workspace_bytes);
    if (sc != GPT_ATTN_OK) return sc;
    if (page < 1) return GPT_ATTN_ERR_SHAPE;
    if (misaligned4(table) || misaligned4(lens) || misaligned4(refs) || misaligned4(parents) || misaligned4(status) ||
        (reinterpret_cast<uintptr_t>(pairs) & 7u))
        return GPT_ATTN_ERR_ALIGN;
    p.table = table;
    p.lens = lens;
    p.refs = refs;
    p.page = page;
    p.arg = parents;
    p.status = status;
    p.pairs = reinterpret_cast<int2*>(pairs);
    pages_take_kernel<true><<<kPagesCluster, kPagesThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? GPT_ATTN_OK : GPT_ATTN_ERR_CUDA;
}

int gpt_attn_pages_free(int* table, int* lens, int* refs, int S, int M, int P, const int* drop, void* stream) {
    if (!table || !lens || !refs || !drop) return GPT_ATTN_ERR_NULL;
    const int sc = check_pages(S, M, P);
    if (sc != GPT_ATTN_OK) return sc;
    if (misaligned4(table) || misaligned4(lens) || misaligned4(refs) || misaligned4(drop)) return GPT_ATTN_ERR_ALIGN;
    PagesParams p{};
    p.table = table;
    p.lens = lens;
    p.refs = refs;
    p.S = S;
    p.M = M;
    p.P = P;
    p.arg = drop;
    pages_free_kernel<<<(unsigned)((S + 7LL) / 8), 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? GPT_ATTN_OK : GPT_ATTN_ERR_CUDA;
}

int gpt_attn_pages_compact(const int* table, const int* refs, int S, int M, int P, int* new_table, int* new_refs,
                           int* pairs, int* moves, void* workspace, size_t workspace_bytes, void* stream) {
    if (!table || !refs || !new_table || !new_refs || (!pairs && P > 1) || !moves) return GPT_ATTN_ERR_NULL;
    PagesParams p{};
    const int sc = pages_params(&p, S, M, P, workspace, workspace_bytes);
    if (sc != GPT_ATTN_OK) return sc;
    if (misaligned4(table) || misaligned4(refs) || misaligned4(new_table) || misaligned4(new_refs) ||
        misaligned4(moves) || (reinterpret_cast<uintptr_t>(pairs) & 7u))
        return GPT_ATTN_ERR_ALIGN;
    p.table = const_cast<int*>(table);
    p.refs = const_cast<int*>(refs);
    p.new_table = new_table;
    p.new_refs = new_refs;
    p.pairs = reinterpret_cast<int2*>(pairs);
    p.moves = moves;
    pages_compact_kernel<<<kPagesCluster, kPagesThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? GPT_ATTN_OK : GPT_ATTN_ERR_CUDA;
}

int gpt_attn_pages_copy(void* k_pages, void* v_pages, int n_pages, int Hkv, int page, int D, const int* pairs,
                        int n_max, const int* n_pairs, void* stream) {
    if (!k_pages || !v_pages || (!pairs && n_max > 0)) return GPT_ATTN_ERR_NULL;
    if (n_pages < 1 || Hkv < 1 || page < 1 || n_max < 0) return GPT_ATTN_ERR_SHAPE;
    if (D != 64 && D != 128) return GPT_ATTN_ERR_UNSUPPORTED_D;
    if ((long long)Hkv * page > 0x7fffffffLL / (D / 8) - kCopyUnit) return GPT_ATTN_ERR_SHAPE;
    if (misaligned(k_pages) || misaligned(v_pages) || (reinterpret_cast<uintptr_t>(pairs) & 7u) ||
        misaligned4(n_pairs))
        return GPT_ATTN_ERR_ALIGN;
    if (n_max == 0) return GPT_ATTN_OK;
    CopyParams p;
    p.k = static_cast<uint4*>(k_pages);
    p.v = static_cast<uint4*>(v_pages);
    p.pairs = reinterpret_cast<const int2*>(pairs);
    p.n_pairs = n_pairs;
    p.max_pairs = n_max;
    p.n_pages = n_pages;
    p.page_chunks = Hkv * page * (D / 8);
    p.units = (p.page_chunks + kCopyUnit - 1) / kCopyUnit;
    const long long most = 2LL * n_max * p.units, blocks = (long long)kCopyBlocksPerSm * sm_count();
    pages_copy_kernel<<<(unsigned)(most < blocks ? most : blocks), kCopyThreads, 0,
                        static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? GPT_ATTN_OK : GPT_ATTN_ERR_CUDA;
}

int gpt_attn_qk_prologue_fwd(const void* q_raw, const void* k_raw, void* q_out, void* k_out, int B, int H, int T,
                             int D, int qk_norm, float rope_base, const gpt_attn_strides* strides, void* stream) {
    if (!q_raw || !k_raw || !q_out || !k_out) return GPT_ATTN_ERR_NULL;
    int sc = check_shape(B, H, T, D);
    if (sc != GPT_ATTN_OK) return sc;
    if (misaligned(q_raw) || misaligned(k_raw) || misaligned(q_out) || misaligned(k_out)) return GPT_ATTN_ERR_ALIGN;
    Strides st[4];
    if ((sc = prologue_strides(st, strides, 4, H, T, D)) != GPT_ATTN_OK) return sc;
    PrologueParams p{};
    p.x[0] = static_cast<const __nv_bfloat16*>(q_raw);
    p.x[1] = static_cast<const __nv_bfloat16*>(k_raw);
    p.out[0] = static_cast<__nv_bfloat16*>(q_out);
    p.out[1] = static_cast<__nv_bfloat16*>(k_out);
    p.xs[0] = st[0], p.xs[1] = st[1], p.outs[0] = st[2], p.outs[1] = st[3];
    p.H = H;
    p.T = T;
    p.rows = (long long)B * H * T;
    p.token_major = st[0].h < st[0].t ? 1 : 0;    // heads of a token adjacent: walk rows token by token
    p.norm = qk_norm ? 1 : 0;
    p.base = rope_base;
    return launch_prologue(false, p, D, static_cast<cudaStream_t>(stream));
}

int gpt_attn_qk_prologue_bwd(const void* q_raw, const void* k_raw, const void* dq_out, const void* dk_out,
                             void* dq_raw, void* dk_raw, int B, int H, int T, int D, int qk_norm, float rope_base,
                             const gpt_attn_strides* strides, void* stream) {
    if (!q_raw || !k_raw || !dq_out || !dk_out || !dq_raw || !dk_raw) return GPT_ATTN_ERR_NULL;
    int sc = check_shape(B, H, T, D);
    if (sc != GPT_ATTN_OK) return sc;
    if (misaligned(q_raw) || misaligned(k_raw) || misaligned(dq_out) || misaligned(dk_out) || misaligned(dq_raw) ||
        misaligned(dk_raw))
        return GPT_ATTN_ERR_ALIGN;
    Strides st[6];
    if ((sc = prologue_strides(st, strides, 6, H, T, D)) != GPT_ATTN_OK) return sc;
    PrologueParams p{};
    p.x[0] = static_cast<const __nv_bfloat16*>(q_raw);
    p.x[1] = static_cast<const __nv_bfloat16*>(k_raw);
    p.dy[0] = static_cast<const __nv_bfloat16*>(dq_out);
    p.dy[1] = static_cast<const __nv_bfloat16*>(dk_out);
    p.out[0] = static_cast<__nv_bfloat16*>(dq_raw);
    p.out[1] = static_cast<__nv_bfloat16*>(dk_raw);
    p.xs[0] = st[0], p.xs[1] = st[1], p.dys[0] = st[2], p.dys[1] = st[3], p.outs[0] = st[4], p.outs[1] = st[5];
    p.H = H;
    p.T = T;
    p.rows = (long long)B * H * T;
    p.token_major = st[0].h < st[0].t ? 1 : 0;    // heads of a token adjacent: walk rows token by token
    p.norm = qk_norm ? 1 : 0;
    p.base = rope_base;
    return launch_prologue(true, p, D, static_cast<cudaStream_t>(stream));
}

int gpt_attn_check(void* stream) {
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return GPT_ATTN_ERR_CUDA;
    int st = 0;
    const int zero = 0;
    if (cudaMemcpyFromSymbol(&st, gpt_attn::g_status, sizeof(int)) != cudaSuccess) return GPT_ATTN_ERR_CUDA;
    if (cudaMemcpyToSymbol(gpt_attn::g_status, &zero, sizeof(int)) != cudaSuccess) return GPT_ATTN_ERR_CUDA;
    if (cudaPeekAtLastError() != cudaSuccess) return GPT_ATTN_ERR_CUDA;
    return st;
}

const char* gpt_attn_status_string(int status) {
    switch (status) {
        case GPT_ATTN_OK: return "ok";
        case GPT_ATTN_ERR_NULL: return "null pointer argument";
        case GPT_ATTN_ERR_SHAPE: return "invalid shape (B, H, T must be >= 1; sizes must fit int64)";
        case GPT_ATTN_ERR_UNSUPPORTED_D: return "unsupported head dimension (D must be 64 or 128)";
        case GPT_ATTN_ERR_ALIGN: return "pointer not 16-byte aligned";
        case GPT_ATTN_ERR_CUDA: return "CUDA error";
        case GPT_ATTN_ERR_TIMEOUT: return "device-side wait timed out";
        case GPT_ATTN_ERR_WORKSPACE: return "workspace missing or too small";
        case GPT_ATTN_ERR_UNAVAILABLE: return "not available in this build";
        case GPT_ATTN_ERR_BOUNDS: return "debug build: a kernel bounds check failed";
        default: return "unknown status";
    }
}

int gpt_attn_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const float* lse,
                         const void* dO, void* dq, void* dk, void* dv, int B, int H, int T, int D, float scale,
                         int window, void* stream) {
    if (!q || !k || !v || !o || !lse || !dO || !dq || !dk || !dv) return GPT_ATTN_ERR_NULL;
    const int sc = check_shape(B, H, T, D);
    if (sc != GPT_ATTN_OK) return sc;
    const size_t need = gpt_attn_bwd_workspace_bytes(B, H, T, D);
    if (need > kNoAllocScratchBytes) return GPT_ATTN_ERR_WORKSPACE;
    void* ws = noalloc_scratch_current_device();
    if (!ws) return GPT_ATTN_ERR_CUDA;
    // The scratch keeps whatever the previous call left; the gpt_attn_bwd stages
    // rewrite every byte they read (dQ accumulator zeroed, row vectors written
    // including padding), so nothing else needs clearing here.
    return gpt_attn_bwd(q, k, v, o, lse, dO, dq, dk, dv, B, H, T, D, scale, window, ws, need, stream);
}

void gpt_attn_tmap_cache_stats(long long* hits, long long* misses, int* entries) {
    long long h = 0, m = 0;
    int u = 0;
    gpt_attn::tmap_cache().stats(&h, &m, &u);
    if (hits) *hits = h;
    if (misses) *misses = m;
    if (entries) *entries = u;
}

int gpt_attn_debug_skip_load(int which) {
#ifdef GPT_ATTN_DEBUG
    if (which < 0 || which > 3) return GPT_ATTN_ERR_SHAPE;
    return cudaMemcpyToSymbol(gpt_attn::g_debug_skip, &which, sizeof(int)) == cudaSuccess ? GPT_ATTN_OK
                                                                                         : GPT_ATTN_ERR_CUDA;
#else
    (void)which;
    return GPT_ATTN_ERR_UNAVAILABLE;
#endif
}

int gpt_attn_debug_wait_timeout(int timeout_us, void* stream) {
    if (timeout_us < 1 || timeout_us > 10 * 1000 * 1000) return GPT_ATTN_ERR_SHAPE;
    gpt_attn::debug_wait_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>((uint64_t)timeout_us * 1000ull);
    return cudaGetLastError() == cudaSuccess ? GPT_ATTN_OK : GPT_ATTN_ERR_CUDA;
}

}  // extern "C"
