"""Sliding-window attention with sinks: the first tokens of a document stay visible past the window.

CPU: the oracle's mask and gradients against brute force and differences; the kernels' choice of
tiles (csrc/schedule.h) against brute force, on valid and on arbitrary document starts; refusals.
GPU: forward and backward against the fp64 definition at the library's parity tolerances."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import causal_attention_sdpa_b200 as ga
from oracle import streaming
from workloads import make_doc_starts, make_inputs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TILE = 128


# ------------------------------------------------------------------------------ oracle
def test_mask_counts():
    m = streaming.sink_mask(9, 3, 2)
    assert m[0].nonzero()[0].tolist() == [0]
    assert m[8].nonzero()[0].tolist() == [0, 1, 6, 7, 8]
    assert m[3].nonzero()[0].tolist() == [0, 1, 2, 3]
    d = streaming.sink_mask(9, 2, 1, [0, 0, 0, 3, 3, 3, 3, 3, 8])
    assert d[6].nonzero()[0].tolist() == [3, 5, 6]
    assert d[8].nonzero()[0].tolist() == [8]
    assert (streaming.sink_mask(9, 0, 5) == np.tril(np.ones((9, 9), dtype=bool))).all()


@pytest.mark.parametrize("W,S", [(2, 1), (3, 4), (1, 2)])
def test_oracle_gradient_is_the_difference_quotient(W, S):
    r = np.random.default_rng(W)
    q, k, v, do = (r.standard_normal((1, 1, 9, 4)) for _ in range(4))
    ds = np.array([[0, 0, 0, 0, 0, 0, 0, 7, 7]])
    grads = streaming.attn_sinks(q, k, v, 0.5, W, S, ds, do)[2:]
    f = lambda: float((streaming.attn_sinks(q, k, v, 0.5, W, S, ds)[0] * do).sum())
    for x, g in zip((q, k, v), grads):
        for at in [(0, 0, 0, 1), (0, 0, 1, 2), (0, 0, 6, 0), (0, 0, 8, 3)]:
            old = x[at]
            x[at] = old + 1e-6
            up = f()
            x[at] = old - 1e-6
            down = f()
            x[at] = old
            assert abs((up - down) / 2e-6 - g[at]) <= 1e-6 * max(1.0, abs(g[at]))


# ------------------------------------------------------------------------------ tiles
@pytest.fixture(scope="module")
def S(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    out = str(tmp_path_factory.mktemp("sinks") / "libsinks_host.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "causal_attention_sdpa_b200", "csrc"),
                    os.path.join(ROOT, "tests", "sinks_host.cpp"), "-o", out], check=True)
    return ctypes.CDLL(out)


def block(S, ds, T, W, sinks, qb):
    cap = 64
    arr = lambda n: (ctypes.c_int * n)()
    tiles, use, own, n_own = arr(cap), arr(2 * cap), arr(2 * cap), arr(2)
    p = None if ds is None else (ctypes.c_int * T)(*[int(x) for x in ds])
    n = S.snk_fwd_block(p, T, W, sinks, qb, cap, tiles, use, own, n_own)
    assert 0 < n <= cap
    return (list(tiles[:n]), [list(use[:n]), list(use[cap:cap + n])],
            [list(own[:n_own[0]]), list(own[cap:cap + n_own[1]])])


def doc_rows(T, seed):
    r = np.random.default_rng(seed)
    row = []
    while len(row) < T:
        row += [len(row)] * int(r.integers(1, 400))
    return np.array(row[:T])


@pytest.mark.parametrize("docs", [None, 1, 2, 3])
@pytest.mark.parametrize("T,W,sinks", [(1, 1, 1), (300, 1, 1), (700, 5, 4), (1000, 128, 129), (1500, 200, 300),
                                       (2000, 1, 700), (1300, 1000, 7), (1537, 129, 1)])
def test_tiles_match_brute_force(S, T, W, sinks, docs):
    ds = None if docs is None else doc_rows(T, docs)
    vis = streaming.sink_mask(T, W, sinks, ds)
    n = -(-T // TILE)
    pad = np.zeros((n * TILE, n * TILE), dtype=bool)
    pad[:T, :T] = vis
    need = pad.reshape(n, TILE, n, TILE).any(axis=(1, 3))          # [query tile, key tile]
    for qb in range((n + 1) // 2):
        tiles, use, own = block(S, ds, T, W, sinks, qb)
        assert tiles == sorted(set(tiles))                          # each tile loaded once
        for t in range(2):
            qt = 2 * qb + t
            assert own[t] == [j for j, u in zip(tiles, use[t]) if u], (qt, tiles, use, own)
            if qt < n:
                assert set(np.nonzero(need[qt])[0]) <= set(own[t]), qt
    for kt in range(n):
        last = S.snk_bwd_last(None if ds is None else (ctypes.c_int * T)(*[int(x) for x in ds]), T, W, sinks, kt)
        seen = np.nonzero(need[:, kt])[0]
        assert last == seen.max(), (kt, last, seen)


def test_any_document_starts_keep_the_roles_in_step(S):
    """Contents that are no document starts give unspecified results, but every role of the forward
    kernel has to go through the same tiles."""
    r = np.random.default_rng(5)
    for _ in range(300):
        T = int(r.integers(1, 1200))
        ds = r.integers(-50, T + 50, size=T)
        W, sinks = int(r.integers(1, 400)), int(r.integers(1, 400))
        for qb in range((-(-T // TILE) + 1) // 2):
            tiles, use, own = block(S, ds, T, W, sinks, qb)
            assert tiles == sorted(set(tiles)) and tiles[0] >= 0
            for t in range(2):
                assert own[t] and own[t] == [j for j, u in zip(tiles, use[t]) if u]
        for kt in range(-(-T // TILE)):
            last = S.snk_bwd_last((ctypes.c_int * T)(*[int(x) for x in ds]), T, W, sinks, kt)
            assert kt <= last < -(-T // TILE)


@pytest.mark.parametrize("BH,n,W,sinks", [(1, 1, 1, 1), (24, 64, 1024, 4), (5, 7, 130, 300), (3, 4, 5, 10 ** 9),
                                          (6, 64, 512, 4), (1, 64, 128, 4), (2, 64, 4000, 500), (100, 9, 128, 200)])
def test_backward_order_takes_each_query_tile_once_and_sink_tiles_first(S, BH, n, W, sinks):
    n_s, length = ctypes.c_int(), ctypes.c_int()
    units = S.snk_cut(BH, n, W, min(sinks, n * TILE), ctypes.byref(n_s), ctypes.byref(length))
    n_s, length = n_s.value, length.value
    assert n_s == min(n, -(-sinks // TILE)) and 1 <= length <= n
    assert length == n or length >= (W + TILE - 2) // TILE + 1      # no shorter than the other tiles' units
    # the longest unit is no longer than another tile's or than an SM's share
    reach = min(n, (W + TILE - 2) // TILE + 1)
    share = -(-BH * (n_s * n + (n - n_s) * reach) // 148)
    assert min(length, n) <= max(reach, share)
    total = BH * (units + n - n_s)
    for tail in {1, BH // 2 + 1, BH}:
        seen = []
        for u in range(total):
            bh, cls, piece = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
            S.snk_list_item(u, BH, n, n_s, length, tail, ctypes.byref(bh), ctypes.byref(cls), ctypes.byref(piece))
            lo = cls.value + piece.value * length
            hi = min(lo + length, n) if cls.value < n_s else cls.value + 1
            assert lo < hi
            seen += [(bh.value, cls.value, q) for q in range(lo, hi)]
            assert (cls.value < n_s) == (u < BH * units)
        want = [(b, c, q) for b in range(BH) for c in range(n) for q in (range(c, n) if c < n_s else [c])]
        assert sorted(seen) == want


# ------------------------------------------------------------------------------ refusals
FAKE = 0x10000


def test_refusals():
    from causal_attention_sdpa_b200 import build
    build.build()
    L, vp = ga.lib(), ctypes.c_void_p
    need = ga.gpt_attn_bwd_sinks_workspace_bytes(1, 2, 300, 64, 100, 4)
    assert need > 0
    assert ga.gpt_attn_bwd_sinks_workspace_bytes(1, 2, 300, 32, 100, 4) == 0
    plain = ga.gpt_attn_bwd_workspace_bytes(1, 2, 300, 64)
    assert need > plain == ga.gpt_attn_bwd_sinks_workspace_bytes(1, 2, 300, 64, 100, 0)
    for window in (0, -1, 300, 2 ** 31 - 1):                        # nothing out of reach: no sinks, nothing cut
        assert ga.gpt_attn_bwd_sinks_workspace_bytes(1, 2, 300, 64, window, 4) == plain
    for window in (1, 128, 1000, 4000):                             # the cut's sums stay small
        for sinks in (1, 300, 2 ** 31 - 1):
            assert ga.gpt_attn_bwd_sinks_workspace_bytes(1, 2, 8192, 128, window, sinks) - \
                ga.gpt_attn_bwd_workspace_bytes(1, 2, 8192, 128) < 64 << 20

    def fwd(ptrs=None, T=300, D=64, sinks=4, m=None, lay=None):
        p = [FAKE] * 5 if ptrs is None else ptrs
        m = ga.GptAttnMask(100, None, None) if m is None else m
        return L.gpt_attn_fwd_sinks(*[vp(x) for x in p], 1, 2, T, D, ctypes.c_float(0.1), ctypes.byref(m), sinks,
                                    lay, vp(0))

    def bwd(ptrs=None, T=300, D=64, ws=FAKE, nbytes=need):
        p = [FAKE] * 9 if ptrs is None else ptrs
        m = ga.GptAttnMask(100, None, None)
        return L.gpt_attn_bwd_sinks(*[vp(x) for x in p], 1, 2, T, D, ctypes.c_float(0.1), ctypes.byref(m), 4, None,
                                    vp(ws), nbytes, vp(0))

    for n, call in ((5, fwd), (9, bwd)):
        for i in range(n):
            p = [FAKE] * n
            p[i] = 0
            assert call(p) == ga.GPT_ATTN_ERR_NULL
            p[i] = FAKE + 8
            assert call(p) == ga.GPT_ATTN_ERR_ALIGN
        assert call(T=0) == ga.GPT_ATTN_ERR_SHAPE
        assert call(D=96) == ga.GPT_ATTN_ERR_UNSUPPORTED_D
    assert bwd(nbytes=need - 1) == ga.GPT_ATTN_ERR_WORKSPACE
    assert bwd(ws=0) == ga.GPT_ATTN_ERR_WORKSPACE
    assert fwd(m=ga.GptAttnMask(100, None, FAKE + 2)) == ga.GPT_ATTN_ERR_ALIGN


def test_binding_refusals_on_the_host():
    q = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ga.gpt_attn_fwd_sinks(q, q, q, window=2, sinks=1)            # not on a GPU


# ------------------------------------------------------------------------------ GPU
TOL_O, TOL_G, TOL_REL, TOL_LSE = 2e-2, 5e-2, 1e-2, 1e-3             # the library's parity tolerances


def close(name, got, want, tol):
    g = got.detach().float().cpu().double().numpy()
    assert np.isfinite(g).all(), name
    # A sink's dK and dV are sums over all later queries, so they can be large, and the output's own
    # rounding, half a bf16 step, is up to 2^-8 of the value: 0.0625 at 16, more than the tolerance.
    over = float((np.abs(g - want) - 2.0 ** -8 * np.abs(want)).max())
    assert over <= tol, (name, over)
    n = float(np.linalg.norm(want))
    if n > 1e-6 * want.size ** 0.5:                                 # W = 1, T = 1: dq, dk are exactly 0
        assert float(np.linalg.norm(g - want)) / n <= TOL_REL, name


def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_attention_sdpa_b200 import build
    build.build()


CASES = [
    # B, H, T, D, window (or one per head), sinks, documents' longest length
    (1, 1, 1, 64, 1, 1, 0), (1, 2, 17, 128, 3, 2, 0), (2, 3, 129, 64, 1, 1, 0), (1, 2, 300, 128, 1, 4, 0),
    (2, 2, 700, 64, 128, 4, 0), (1, 3, 1000, 128, 200, 129, 0), (3, 2, 777, 64, 100, 300, 0),
    (1, 2, 2500, 64, 129, 1, 0), (1, 2, 2100, 128, 256, 7, 0), (1, 2, 513, 64, 60, 10 ** 9, 0),
    (2, 3, 1000, 64, [50, 0, 400], 5, 0), (1, 2, 900, 128, [1, 2 ** 31 - 1], 130, 0),
    (2, 2, 1000, 64, 64, 3, 300), (3, 2, 1111, 128, 100, 7, 600), (2, 2, 1500, 64, 1, 40, 1200),
    (2, 2, 640, 128, [10, 0], 200, 500), (48, 12, 300, 64, 40, 4, 0), (40, 6, 520, 64, 90, 20, 300),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,T,D,W,sinks,docs", CASES, ids=["-".join(map(str, c)).replace(" ", "") for c in CASES])
def test_parity(B, H, T, D, W, sinks, docs):
    gpu()
    q, k, v, do = make_inputs(B, H, T, D, seed=T + D + sinks % 1000)
    ds = make_doc_starts(B, T, 7, docs) if docs else None
    hw = W if isinstance(W, list) else None
    how = dict(window=0 if hw else W, head_windows=hw, sinks=sinks, scale=D ** -0.5,
               doc_start=None if ds is None else torch.as_tensor(ds, dtype=torch.int32).cuda())
    qd, kd, vd, dd = (t.cuda() for t in (q, k, v, do))
    nan = lambda: torch.full_like(qd, float("nan"))
    o, lse = ga.gpt_attn_fwd_sinks(qd, kd, vd, o=nan(), **how)
    got = ga.gpt_attn_bwd_sinks(qd, kd, vd, o, lse, dd, dq=nan(), dk=nan(), dv=nan(), **how)
    assert ga.gpt_attn_check() == ga.GPT_ATTN_OK
    ro, rl, *rg = streaming.attn_sinks(q, k, v, D ** -0.5, W, sinks, None if ds is None else np.asarray(ds), do)
    close("o", o, ro, TOL_O)
    assert float(np.abs(lse.cpu().double().numpy() - rl).max()) <= TOL_LSE
    for n, g, r in zip(("dq", "dk", "dv"), got, rg):
        close(n, g, r, TOL_G)
    # the forward and dk, dv do not depend on the run
    o2, lse2 = ga.gpt_attn_fwd_sinks(qd, kd, vd, **how)
    g2 = ga.gpt_attn_bwd_sinks(qd, kd, vd, o2, lse2, dd, **how)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.equal(got[2], g2[2])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_without_sinks_or_window_it_is_the_plain_call(D):
    gpu()
    q, k, v, do = (t.cuda() for t in make_inputs(2, 3, 700, D, seed=3))
    for kw, plain in ((dict(window=100, sinks=0), dict(window=100)), (dict(window=0, sinks=9), dict(window=0)),
                      (dict(window=700, sinks=9), dict(window=0)),
                      (dict(head_windows=[0, 5, 100], sinks=-1), dict(head_windows=[0, 5, 100]))):
        o, lse = ga.gpt_attn_fwd_sinks(q, k, v, **kw)
        o2, lse2 = ga.gpt_attn_fwd_ex(q, k, v, **plain)
        assert torch.equal(o, o2) and torch.equal(lse, lse2), kw
        g, g2 = ga.gpt_attn_bwd_sinks(q, k, v, o, lse, do, **kw), ga.gpt_attn_bwd_ex(q, k, v, o, lse, do, **plain)
        assert torch.equal(g[2], g2[2]), kw
        if kw["sinks"] <= 0:                                        # with sinks the rows of few keys get another Delta
            assert torch.equal(g[1], g2[1]), kw


@pytest.mark.gpu
@pytest.mark.parametrize("T,W,sinks,docs", [(16, 5, 2, 0), (24, 100, 4, 0), (37, 9, 3, 0), (200, 6, 4, 0), (300, 64, 4, 12)])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_of_few_keys_keep_their_precision(T, W, sinks, docs, D):
    """dQ and dK carry two roundings to bf16, dS's and their own, each uniform within 2^-8 of a value at
    most: a relative norm of up to 2^-8 / 3^0.5 each.  O's rounding, through Delta, must not add a third."""
    gpu()
    B, H = 8, 8
    q, k, v, do = make_inputs(B, H, T, D, seed=T)
    ds = make_doc_starts(B, T, 7, docs) if docs else None
    how = dict(window=W, sinks=sinks, scale=D ** -0.5,
               doc_start=None if ds is None else torch.as_tensor(ds, dtype=torch.int32).cuda())
    a = [t.cuda() for t in (q, k, v)]
    o, lse = ga.gpt_attn_fwd_sinks(*a, **how)
    got = ga.gpt_attn_bwd_sinks(*a, o, lse, do.cuda(), **how)
    want = streaming.attn_sinks(q, k, v, D ** -0.5, W, sinks, None if ds is None else np.asarray(ds), do)[2:]
    for n, g, r in zip(("dq", "dk"), got, want):
        err = float(np.linalg.norm(g.float().cpu().double().numpy() - r) / np.linalg.norm(r))
        assert err <= 2.0 ** -8 * (2 / 3) ** 0.5, (n, err)


@pytest.mark.gpu
@pytest.mark.parametrize("docs", [False, True])
def test_fused_projection_and_autograd(docs):
    """q, k, v out of one projection, O and gradients token-major, through gpt_attention."""
    gpu()
    from causal_attention_sdpa_b200.autograd import gpt_attention
    B, T, H, D, W, S = 2, 600, 3, 64, 70, 5
    g = torch.Generator().manual_seed(4)
    x = torch.randn(B, T, 3, H, D, generator=g).bfloat16()
    do = torch.randn(B, T, H, D, generator=g).bfloat16()
    ds = np.array([[0] * 250 + [250] * 350, [0] * 600]) if docs else None
    leaf = x.cuda().requires_grad_()
    q, k, v = leaf.permute(2, 0, 3, 1, 4).unbind(0)
    o = gpt_attention(q, k, v, window=W, sinks=S, out_layout="bthd",
                      doc_start=torch.as_tensor(ds, dtype=torch.int32).cuda() if docs else None)
    o.backward(do.cuda())
    qh, kh, vh = x.permute(2, 0, 3, 1, 4).unbind(0)
    ro, _, *rg = streaming.attn_sinks(qh, kh, vh, D ** -0.5, W, S, ds, do.transpose(1, 2))
    close("o", o.transpose(1, 2), ro, TOL_O)
    close("grad", leaf.grad.permute(2, 0, 3, 1, 4), np.stack(rg), TOL_G)


@pytest.mark.gpu
def test_captured_and_replayed_on_another_stream():
    gpu()
    q, k, v, do = (t.cuda() for t in make_inputs(1, 4, 900, 64, seed=9))
    kw = dict(window=130, sinks=6)
    bufs = [torch.empty_like(q) for _ in range(4)]
    lse = torch.empty(1, 4, 900, device="cuda")
    ws = torch.empty(ga.gpt_attn_bwd_sinks_workspace_bytes(1, 4, 900, 64, 130, 6), dtype=torch.uint8, device="cuda")

    def step():
        ga.gpt_attn_fwd_sinks(q, k, v, o=bufs[0], lse=lse, **kw)
        ga.gpt_attn_bwd_sinks(q, k, v, bufs[0], lse, do, dq=bufs[1], dk=bufs[2], dv=bufs[3], workspace=ws, **kw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    want = [b.clone() for b in bufs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for b in bufs:
            b.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bufs[0], want[0]) and torch.equal(bufs[2], want[2]) and torch.equal(bufs[3], want[3])
    # dq: the order of its fp32 additions varies, which can turn a rounding: one bf16 step, 2^-7 of a value at most
    assert float((bufs[1].float() - want[1].float()).abs().max()) <= 2 ** -7 * float(want[1].abs().max())
