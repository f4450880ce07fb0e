"""Attention of new and drafted tokens over a paged cache, and the rows of tokens in its pages.

CPU: the oracle against dense causal attention; the kernels' index arithmetic (csrc/paging.h) against
brute force; refusals.  GPU: against the fp64 definition at the library's parity tolerances."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import causal_attention_sdpa_b200 as ga
from oracle import streaming

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def make_cache(B, Hkv, D, page, lens, N, seed, spare=3, extra=0):
    """Pools whose pages are handed out in a random order, with room for N new tokens each; rows that no
    token occupies hold NaN."""
    r = np.random.default_rng(seed)
    M = max(1, -(-(max(lens) + N) // page)) + extra
    held = [-(-(n + N) // page) for n in lens]
    P = sum(held) + spare
    table = np.full((B, M), -1, dtype=np.int32)
    places = list(r.permutation(P))
    k = torch.full((P, Hkv, page, D), float("nan"), dtype=torch.bfloat16)
    v = k.clone()
    g = torch.Generator().manual_seed(seed)
    for b in range(B):
        table[b, :held[b]] = [places.pop() for _ in range(held[b])]
        for j in range(held[b]):
            n = min(page, lens[b] + N - j * page)
            e = int(table[b, j])
            k[e, :, :n] = torch.randn(Hkv, n, D, generator=g).bfloat16()
            v[e, :, :n] = torch.randn(Hkv, n, D, generator=g).bfloat16()
    return k, v, table, np.array(lens, dtype=np.int32)


def random_trees(B, N, seed):
    r = np.random.default_rng(seed)
    return np.array([[-1] + [int(r.integers(max(-1, n - 5), n)) for n in range(1, N)] for _ in range(B)],
                    dtype=np.int32)


# ------------------------------------------------------------------------------ oracle
def test_oracle_is_the_tail_of_causal_attention():
    T, N = 23, 6
    k, v, table, lens = make_cache(1, 1, 8, 5, [T - N], N, 1)
    kk, vv = (streaming.paged_rows(x.double().numpy(), table[0], T)[0][:, 0] for x in (k, v))
    q = np.random.default_rng(2).standard_normal((1, 2, N, 8))
    for W, S in ((0, 0), (4, 2), (1, 0)):
        o, lse = streaming.paged_decode(q, k, v, table, lens, scale=0.4, window=W, sinks=S)
        vis = streaming.sink_mask(T, W, S)[T - N:]
        for h in range(2):
            p, z = streaming.masked_softmax(0.4 * q[0, h] @ kk.T, vis)
            assert np.abs(o[0, h] - p @ vv).max() < 1e-12 and np.abs(lse[0, h] - z).max() < 1e-12


def test_oracle_tree_is_each_path_by_itself():
    k, v, table, lens = make_cache(1, 1, 8, 4, [9], 5, 3)
    q = np.random.default_rng(2).standard_normal((1, 1, 5, 8))
    par = np.array([[-1, 0, 0, 2, -1]])
    o, _ = streaming.paged_decode(q, k, v, table, lens, par, scale=0.4, window=6)
    kk, vv = (streaming.paged_rows(x.double().numpy(), table[0], 14)[0][:, 0] for x in (k, v))
    for n, path in enumerate(([0], [0, 1], [0, 2], [0, 2, 3], [4])):
        rows = list(range(9)) + [9 + x for x in path]
        rows = rows[-6:]                                            # positions within the window
        p = np.exp(0.4 * kk[rows] @ q[0, 0, n])
        assert np.abs(o[0, 0, n] - p @ vv[rows] / p.sum()).max() < 1e-12


# ------------------------------------------------------------------------------ index arithmetic
@pytest.fixture(scope="module")
def S(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    out = str(tmp_path_factory.mktemp("paging") / "libpaging_host.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "causal_attention_sdpa_b200", "csrc"),
                    os.path.join(ROOT, "tests", "paging_host.cpp"), "-o", out], check=True)
    return ctypes.CDLL(out)


def test_tiles_and_visibility_match_brute_force(S):
    r = np.random.default_rng(7)
    for trial in range(250):
        page, M = int(r.choice([1, 3, 16, 64, 100])), int(r.integers(1, 12))
        cap, N = page * M, int(r.integers(1, 65 if trial % 4 == 0 else 12))
        L = int(r.integers(-2, cap + 5))
        W, sinks = (0, 0) if trial % 3 == 0 else (int(r.choice([1, 2, 40, 200, 2 ** 31 - 1])),
                                                  int(r.choice([0, 1, 5, 70, 300, 2 ** 31 - 1])))
        par = random_trees(1, N, trial)[0]
        cpar = (ctypes.c_int * N)(*par.tolist())
        tiles = (ctypes.c_int * 64)()
        tile = 64 << trial % 2
        n_tiles = S.pg_tiles(L, N, page, M, W, sinks, tile, 64, tiles)
        L = min(max(L, 0), cap)
        end = min(L + N, cap)
        read = {x for x in range(end) if S.pg_needs(L, N, page, M, W, sinks, x)}
        got = list(tiles[:n_tiles])
        assert got == sorted(set(got)) and all(0 <= t * tile < end for t in got)
        assert {x // tile for x in read} <= set(got)
        box = S.pg_box(page)
        assert page % box == 0 and 64 % box == 0
        for x in range(0, cap, box):
            assert S.pg_needs_any(L, N, page, M, W, sinks, x, box) == any(y in read for y in range(x, x + box))
        everyone = []
        for n in range(N):
            chain = streaming.ancestors(par, int(n))
            at = L + len(chain) - 1
            seen = [(x, x) for x in range(L)] + [(L + c, L + i) for i, c in enumerate(chain)]
            want = {row for row, x in seen if row < end and (W <= 0 or at - x < W or x < sinks)}
            have = {x for x in read if S.pg_sees(int(n), cpar, N, L, x, W, sinks)}
            assert have == want, (L, N, W, sinks, n)
            everyone.append(want)
        some = set.union(*everyone) - set.intersection(*everyone)
        for x in range(0, cap, 32):
            if some & set(range(x, x + 32)):
                assert S.pg_differs(L, N, page, M, W, sinks, x, 32), (L, N, W, sinks, x)


def test_division_by_multiplication(S):
    r = np.random.default_rng(1)
    top = 2 ** 31 - 1
    for d in [1, 2, 3, 5, 7, 16, 20, 33, 48, 64, 100, 641, 6700417, 2 ** 30, 2 ** 30 + 1, top] + \
            [int(x) for x in r.integers(1, top, 50)]:
        near = [k * d + o for k in (0, 1, 2, top // d // 2, top // d - 1, top // d) for o in (-1, 0, 1)]
        for n in [x for x in near if 0 <= x <= top] + [top] + [int(x) for x in r.integers(0, top, 40)]:
            assert S.pg_div(n, d) == n // d, (n, d)


def test_rows_and_pieces(S):
    row = (ctypes.c_int * 3)(4, -1, 9)
    assert S.pg_row(row, 5, 8, 7, 3, 2) == (4 * 3 + 2) * 8 + 5
    assert S.pg_row(row, 9, 8, 7, 3, 2) == -1                       # no page
    assert S.pg_row(row, 17, 8, 7, 3, 2) == -1                      # outside the pool
    for total, blocks in ((1, 296), (295, 296), (296, 296), (297, 296), (10 ** 9, 296)):
        c = S.pg_chunk(total, blocks, 1)
        assert c * blocks >= total and (c - 1) * blocks < total


# ------------------------------------------------------------------------------ refusals
FAKE = 0x10000


def test_refusals():
    from causal_attention_sdpa_b200 import build
    build.build()
    L, vp = ga.lib(), ctypes.c_void_p
    base = dict(k_pages=FAKE, v_pages=FAKE, table=FAKE, lens=FAKE, B=2, Hkv=2, D=64, n_pages=9, page=16, max_pages=4)
    need = ga.gpt_attn_paged_decode_workspace_bytes(2, 4, 2, 3, 64)
    assert need > 0
    for bad in ((0, 4, 2, 3, 64), (2, 5, 2, 3, 64), (2, 4, 2, 65, 64), (2, 4, 2, 0, 64), (2, 4, 2, 3, 96), (2, 4, 0, 3, 64)):
        assert ga.gpt_attn_paged_decode_workspace_bytes(*bad) == 0

    def decode(q=FAKE, o=FAKE, lse=FAKE, H=4, N=3, ws=FAKE, nbytes=need, st=None, n_new=0, parents=0, **kw):
        c = ga.GptAttnPagedCache(**(base | kw))
        return L.gpt_attn_paged_decode(vp(q), ctypes.byref(c), vp(n_new), vp(parents), vp(o), vp(lse), H, N,
                                       ctypes.c_float(0.1), 0, 0, st, vp(ws), nbytes, vp(0))

    def append(k=FAKE, v=FAKE, N=3, n_new=0, st=None, **kw):
        c = ga.GptAttnPagedCache(**(base | kw))
        return L.gpt_attn_paged_append(ctypes.byref(c), vp(k), vp(v), N, vp(n_new), st, vp(0))

    def accept(a=FAKE, n=FAKE, N=3, **kw):
        c = ga.GptAttnPagedCache(**(base | kw))
        return L.gpt_attn_paged_accept(ctypes.byref(c), vp(a), vp(n), N, vp(0))

    for call in (decode, append, accept):
        for f in ("k_pages", "v_pages", "table", "lens"):
            assert call(**{f: 0}) == ga.GPT_ATTN_ERR_NULL
            assert call(**{f: FAKE + 2}) == ga.GPT_ATTN_ERR_ALIGN
        for f in ("B", "Hkv", "n_pages", "page", "max_pages"):
            assert call(**{f: 0}) == ga.GPT_ATTN_ERR_SHAPE
        assert call(D=32) == ga.GPT_ATTN_ERR_UNSUPPORTED_D
        assert call(N=0) == ga.GPT_ATTN_ERR_SHAPE
        assert call(max_pages=2 ** 20, page=2 ** 11) == ga.GPT_ATTN_ERR_SHAPE
        assert call(n_pages=2 ** 30, page=2) == ga.GPT_ATTN_ERR_SHAPE
    for f in ("q", "o", "lse"):
        assert decode(**{f: 0}) == ga.GPT_ATTN_ERR_NULL
        assert decode(**{f: FAKE + 2}) == ga.GPT_ATTN_ERR_ALIGN
    assert decode(ws=0) == decode(nbytes=need - 1) == ga.GPT_ATTN_ERR_WORKSPACE
    assert decode(H=5) == decode(N=65) == accept(N=65) == ga.GPT_ATTN_ERR_SHAPE
    assert decode(n_new=FAKE + 1) == decode(parents=FAKE + 1) == append(n_new=FAKE + 1) == ga.GPT_ATTN_ERR_ALIGN
    st = (ga.GptAttnStrides * 2)(ga.GptAttnStrides(1024, 64, 60), ga.GptAttnStrides(1024, 64, 64))
    assert decode(st=st) == append(st=st) == ga.GPT_ATTN_ERR_ALIGN
    assert append(k=0) == accept(a=0) == accept(n=0) == ga.GPT_ATTN_ERR_NULL
    assert append(k=FAKE + 8) == accept(a=FAKE + 2) == ga.GPT_ATTN_ERR_ALIGN


def test_binding_refusals_on_the_host():
    k = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16)
    t, n = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        ga.gpt_attn_paged_append(k, k, t, n, k[:1], k[:1])
    with pytest.raises(ValueError):
        ga.gpt_attn_paged_decode(k[:1], k, k, t, n)
    with pytest.raises(ValueError):
        ga.gpt_attn_paged_accept(k, k, t, n, t, n)


# ------------------------------------------------------------------------------ GPU
TOL_O, TOL_REL, TOL_LSE = 2e-2, 1e-2, 1e-3             # the library's parity tolerances


def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_attention_sdpa_b200 import build
    build.build()


def close(o, lse, ro, rl):
    g = o.float().cpu().double().numpy()
    assert np.isfinite(g).all()
    assert float(np.abs(g - ro).max()) <= TOL_O
    n = float(np.linalg.norm(ro))
    assert float(np.linalg.norm(g - ro)) <= TOL_REL * n
    l = lse.cpu().double().numpy()
    assert (np.isneginf(l) == np.isneginf(rl)).all()
    seen = ~np.isneginf(rl)
    assert float(np.abs(l[seen] - rl[seen]).max(initial=0)) <= TOL_LSE


def cuda(*xs):
    return [torch.as_tensor(x).cuda() for x in xs]


CASES = [
    # B, Hkv, G, D, N, page, lens, window, sinks, parents
    (1, 1, 1, 64, 1, 16, [0], 0, 0, False), (1, 12, 1, 64, 1, 64, [777], 0, 0, False),
    (3, 2, 1, 128, 1, 1, [1, 0, 63], 0, 0, False), (4, 2, 3, 64, 1, 7, [64, 65, 127, 128], 0, 0, False),
    (2, 1, 16, 128, 1, 32, [500, 31], 0, 0, False), (2, 2, 17, 64, 1, 32, [500, 31], 0, 0, False),
    (2, 1, 40, 128, 1, 32, [500, 31], 0, 0, False), (2, 1, 3, 64, 33, 20, [333, 7], 0, 0, True),
    (2, 6, 1, 128, 32, 64, [1500, 1000], 0, 0, True), (3, 2, 4, 128, 13, 128, [900, 100, 3], 256, 4, True),
    (2, 2, 8, 64, 64, 16, [100, 700], 0, 0, True), (2, 1, 8, 128, 64, 48, [100, 300], 50, 3, True),
    (2, 2, 1, 64, 64, 16, [0, 5], 0, 0, False), (3, 1, 2, 64, 9, 16, [400, 70, 0], 1, 0, True),
    (3, 1, 2, 64, 9, 16, [400, 70, 0], 3, 1, True), (2, 2, 1, 128, 5, 33, [1000, 200], 64, 130, True),
    (2, 1, 1, 64, 1, 64, [3000, 5], 100, 4, False), (2, 1, 1, 64, 2, 64, [3000, 5], 2 ** 31 - 1, 2 ** 31 - 1, False),
    (40, 8, 1, 64, 1, 16, [(37 * i) % 211 for i in range(40)], 0, 0, False),
    (300, 1, 1, 64, 1, 16, [(53 * i) % 97 for i in range(300)], 0, 0, False),
    (33, 3, 2, 128, 4, 32, [(91 * i) % 400 for i in range(33)], 30, 2, True),
    (900, 1, 1, 64, 1, 16, [(29 * i) % 61 for i in range(900)], 0, 0, False),
    (600, 1, 40, 64, 1, 8, [(29 * i) % 61 for i in range(600)], 20, 1, False),
    (3, 1, 65, 128, 1, 16, [200, 64, 1], 0, 0, False), (2, 2, 5, 64, 26, 24, [400, 130], 60, 3, True),
    (2, 1, 43, 128, 3, 1, [70, 5], 0, 0, True), (1, 2, 11, 64, 64, 2, [77], 0, 0, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hkv,G,D,N,page,lens,W,sinks,tree", CASES, ids=[str(i) for i in range(len(CASES))])
def test_parity(B, Hkv, G, D, N, page, lens, W, sinks, tree):
    gpu()
    k, v, table, ln = make_cache(B, Hkv, D, page, lens, N, seed=N + D)
    g = torch.Generator().manual_seed(3)
    q = torch.randn(B, Hkv * G, N, D, generator=g).bfloat16()
    par = random_trees(B, N, 5) if tree else None
    n_new = None
    if B > 2:
        n_new = np.array([N if b % 3 else (b * 7) % (N + 1) for b in range(B)], dtype=np.int32)
    ro, rl = streaming.paged_decode(q, k, v, table, ln, par, n_new, D ** -0.5, W, sinks)
    kd, vd, td, ld, qd = cuda(k, v, table, ln, q)
    kw = dict(scale=D ** -0.5, window=W, sinks=sinks, parents=None if par is None else torch.as_tensor(par).cuda(),
              n_new=None if n_new is None else torch.as_tensor(n_new).cuda())
    o, lse = ga.gpt_attn_paged_decode(qd, kd, vd, td, ld, o=torch.full_like(qd, float("nan")), **kw)
    close(o, lse, ro, rl)
    o2, lse2 = ga.gpt_attn_paged_decode(qd, kd, vd, td, ld, **kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.gpu
def test_long_sequence_split_over_the_gpu():
    gpu()
    B, Hkv, G, D, N, page = 1, 2, 2, 128, 3, 64
    k, v, table, ln = make_cache(B, Hkv, D, page, [20011], N, seed=1)
    q = torch.randn(B, Hkv * G, N, D, generator=torch.Generator().manual_seed(3)).bfloat16() * 3
    ro, rl = streaming.paged_decode(q, k, v, table, ln, None, None, D ** -0.5)
    o, lse = ga.gpt_attn_paged_decode(*cuda(q, k, v, table, ln))
    close(o, lse, ro, rl)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-3, 3.0])
def test_any_scale(scale):
    gpu()
    k, v, table, ln = make_cache(2, 2, 64, 16, [200, 33], 5, seed=1)
    q = torch.randn(2, 4, 5, 64, generator=torch.Generator().manual_seed(3)).bfloat16()
    par = random_trees(2, 5, 1)
    ro, rl = streaming.paged_decode(q, k, v, table, ln, par, None, scale, 100, 2)
    o, lse = ga.gpt_attn_paged_decode(*cuda(q, k, v, table, ln), scale=scale, window=100, sinks=2,
                                      parents=torch.as_tensor(par).cuda())
    close(o, lse, ro, rl)


@pytest.mark.gpu
@pytest.mark.parametrize("G,N", [(1, 1), (2, 9), (5, 20)])
def test_bad_pages_lengths_and_parents(G, N):
    """Entries outside the pool are missing pages, lengths are clamped, parents not below a node are the
    context; nothing is read outside the pools."""
    gpu()
    B, Hkv, D, page = 5, 2, 64, 16
    k, v, table, ln = make_cache(B, Hkv, D, page, [100, 90, 80, 30, 0], N, seed=2, extra=1)
    P, M = k.shape[0], table.shape[1]
    table[0, 2], table[0, 4], table[1, :] = -7, P, -1
    table[2, 0], table[2, 1] = 2 ** 31 - 1, -2 ** 31
    ln[3], ln[4] = 2 ** 31 - 1, -5
    table[3, table[3] < 0] = 0
    k, v = torch.nan_to_num(k), torch.nan_to_num(v)
    par = random_trees(B, N, 1)
    par[:, -1], par[0, 0] = N, 5
    par[1, N // 2] = N // 2
    q = torch.randn(B, Hkv * G, N, D, generator=torch.Generator().manual_seed(3)).bfloat16()
    n_new = np.array([N, 2 ** 31 - 1, N, N, -3], dtype=np.int32)
    for W, S in ((0, 0), (20, 3)):
        ro, rl = streaming.paged_decode(q, k, v, table, ln, par, n_new, 0.125, W, S)
        a = cuda(q, k, v, table, ln)
        o, lse = ga.gpt_attn_paged_decode(*a, parents=torch.as_tensor(par).cuda(), n_new=torch.as_tensor(n_new).cuda(),
                                          scale=0.125, window=W, sinks=S)
        close(o, lse, ro, rl)
    # appending and accepting skip them too
    kn = torch.randn(B, Hkv, N, D, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    kd, vd, td, ld = cuda(k, v, table, ln)
    ga.gpt_attn_paged_append(kd, vd, td, ld, kn, kn, n_new=torch.as_tensor(n_new).cuda())
    want = k.clone()
    for b in range(B):
        L = min(max(int(ln[b]), 0), M * page)
        for n in range(min(max(int(n_new[b]), 0), N)):
            if L + n < M * page and 0 <= table[b, (L + n) // page] < P:
                want[table[b, (L + n) // page], :, (L + n) % page] = kn[b, :, n].cpu()
    assert torch.equal(kd.cpu(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("D,G,N", [(64, 1, 6), (128, 1, 20), (64, 3, 40), (128, 8, 8)])
def test_what_a_node_does_not_see_does_not_reach_it(D, G, N):
    """Drafts full of infinities and NaN change only the nodes that continue them, which become NaN or
    infinite as the sum does."""
    gpu()
    k, v, table, ln = make_cache(2, 2, D, 16, [100, 41], N, seed=5)
    q = torch.randn(2, 2 * G, N, D, generator=torch.Generator().manual_seed(3)).bfloat16()
    par = random_trees(2, N, 9)
    par[:, 3] = -1                                                  # node 3 and what continues it
    par[:, 5] = 2
    a = cuda(q, k, v, table, ln)
    kw = dict(parents=torch.as_tensor(par).cuda(), window=60, sinks=2)
    o, lse = ga.gpt_attn_paged_decode(*a, **kw)
    for b in range(2):
        at = int(ln[b]) + 3
        e = int(table[b, at // 16])
        a[2][e, :, at % 16, 0::4] = float("inf")
        a[2][e, :, at % 16, 1::4] = float("-inf")
        a[2][e, :, at % 16, 2::4] = float("nan")
    o2, lse2 = ga.gpt_attn_paged_decode(*a, **kw)
    for b in range(2):
        for n in range(N):
            if 3 in streaming.ancestors(par[b], n):
                assert torch.isposinf(o2[b, :, n, 0::4]).all() and torch.isneginf(o2[b, :, n, 1::4]).all()
                assert torch.isnan(o2[b, :, n, 2::4]).all()
                assert torch.equal(o2[b, :, n, 3::4], o[b, :, n, 3::4])
            else:
                assert torch.equal(o2[b, :, n], o[b, :, n]), (b, n)
    assert torch.equal(lse, lse2)
    # the same for keys
    a = cuda(q, k, v, table, ln)
    for b in range(2):
        at = int(ln[b]) + 3
        a[1][int(table[b, at // 16]), :, at % 16] = float("nan")
    o2, _ = ga.gpt_attn_paged_decode(*a, **kw)
    for b in range(2):
        for n in range(N):
            if 3 in streaming.ancestors(par[b], n):
                assert torch.isnan(o2[b, :, n]).all()
            else:
                assert torch.equal(o2[b, :, n], o[b, :, n]), (b, n)


@pytest.mark.gpu
@pytest.mark.parametrize("G,N", [(1, 1), (2, 9), (9, 5), (3, 50)])
def test_nothing_new_and_nothing_cached(G, N):
    gpu()
    k, v, table, ln = make_cache(3, 2, 64, 16, [0, 40, 7], N, seed=2)
    q = torch.randn(3, 2 * G, N, 64).bfloat16()
    a = cuda(q, k, v, table, ln)
    nan = lambda: dict(o=torch.full_like(a[0], float("nan")), lse=torch.full((3, 2 * G, N), float("nan"), device="cuda"))
    for n_new in ([0, 0, 0], [-1, 0, -2 ** 31], [0, min(N, 2), 0]):
        o, lse = ga.gpt_attn_paged_decode(*a, n_new=torch.tensor(n_new, dtype=torch.int32, device="cuda"), **nan())
        ro, rl = streaming.paged_decode(q, k, v, table, ln, None, n_new, 0.125)
        close(o, lse, ro, rl)
    t = torch.full_like(a[3], -1)                                   # no page anywhere
    o, lse = ga.gpt_attn_paged_decode(*a[:3], t, a[4], **nan())
    assert (o == 0).all() and torch.isneginf(lse).all()


@pytest.mark.gpu
@pytest.mark.parametrize("G", [2, 7])
def test_append_decode_accept_as_a_user_runs_them(G):
    """A speculative loop over strided projections and a captured graph, against dense causal attention."""
    gpu()
    B, Hkv, D, page, N = 3, 2, 64, 16, 5
    H, M = Hkv * G, 12
    g = torch.Generator().manual_seed(1)
    P = B * M + 2
    table = torch.randperm(P, generator=g)[:B * M].view(B, M).int().cuda()
    kd = torch.full((P, Hkv, page, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vd = kd.clone()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    hist = [([], []) for _ in range(B)]
    par = torch.tensor([[-1, 0, 0, 2, 3], [-1, -1, 1, 2, 0], [-1, 0, 1, 2, 3]], dtype=torch.int32, device="cuda")
    acc = torch.tensor([[0, 2, 3, 0, 0], [1, 2, 3, 0, 0], [0, 0, 0, 0, 0]], dtype=torch.int32, device="cuda")
    n_acc = torch.tensor([3, 2, 0], dtype=torch.int32, device="cuda")
    # q, k, v columns of one projection [B, N, H + 2 Hkv, D], O token-major
    x = torch.empty(B, N, H + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")
    q, kn, vn = x.transpose(1, 2).split([H, Hkv, Hkv], 1)
    o = torch.empty(B, N, H, D, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    lse = torch.empty(B, H, N, device="cuda")
    ws = torch.empty(ga.gpt_attn_paged_decode_workspace_bytes(B, H, Hkv, N, D), dtype=torch.uint8, device="cuda")

    def step():
        ga.gpt_attn_paged_append(kd, vd, table, lens, kn, vn)
        ga.gpt_attn_paged_decode(q, kd, vd, table, lens, parents=par, o=o, lse=lse, workspace=ws)
        ga.gpt_attn_paged_accept(kd, vd, table, lens, acc, n_acc)
        lens.add_(n_acc)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x.zero_()
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lens.zero_()
    for t in range(8):
        x.copy_(torch.randn(x.shape, generator=g).bfloat16())
        L = lens.cpu().tolist()
        graph.replay()
        xs = x.cpu().double().numpy()
        got = o.float().cpu().double().numpy()
        for b in range(B):
            ks, vs = hist[b]
            assert len(ks) == L[b]
            for n in range(N):
                path = streaming.ancestors(par[b].tolist(), n)
                kk = np.array(ks + [xs[b, c, H:H + Hkv] for c in path])
                vv = np.array(vs + [xs[b, c, H + Hkv:] for c in path])
                for h in range(H):
                    p, _ = streaming.masked_softmax(D ** -0.5 * kk[:, h // G] @ xs[b, n, h], np.ones(len(kk), dtype=bool))
                    assert np.abs(got[b, h, n] - p @ vv[:, h // G]).max() <= TOL_O
            for c in acc[b, :n_acc[b]].tolist():
                ks.append(xs[b, c, H:H + Hkv])
                vs.append(xs[b, c, H + Hkv:])


@pytest.mark.gpu
@pytest.mark.parametrize("N", [2, 40])
def test_pools_past_four_gigabytes(N):
    """The same sequences in a small pool and at the far end of one of 4.4 GB: equal results."""
    gpu()
    Hkv, D, page, far = 8, 128, 64, 33500
    k, v, table, ln = make_cache(2, Hkv, D, page, [200, 70], N, seed=5)
    P = k.shape[0]
    q = torch.randn(2, Hkv, N, D, generator=torch.Generator().manual_seed(3)).bfloat16()
    qd, kd, vd, td, ld = cuda(q, k, v, table, ln)
    kn = torch.randn(2, Hkv, N, D, device="cuda").bfloat16()
    acc = torch.tensor([[N - 1] + [0] * (N - 1), list(range(N - 1, -1, -1))], dtype=torch.int32, device="cuda")
    n_acc = torch.tensor([1, N], dtype=torch.int32, device="cuda")
    kb, vb = (torch.empty(far, Hkv, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert kb.numel() * 2 > 2 ** 32
    kb[far - P:], vb[far - P:] = kd, vd
    tb = torch.where(td >= 0, td + far - P, td)
    pairs = torch.tensor([[0, P - 1]], dtype=torch.int32, device="cuda")
    got = []
    for kk, vv, tt, off in ((kd, vd, td, 0), (kb, vb, tb, far - P)):
        ga.gpt_attn_paged_append(kk, vv, tt, ld, kn, kn)
        got.append(list(ga.gpt_attn_paged_decode(qd, kk, vv, tt, ld)))
        ga.gpt_attn_paged_accept(kk, vv, tt, ld, acc, n_acc)
        ga.gpt_attn_pages_copy(kk, vv, pairs + off)
        got[-1] += [kk[off:].nan_to_num(9), vv[off:].nan_to_num(9)]
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_memory_taken_for_a_call_on_another_stream_is_kept():
    """Outputs and workspaces that the binding allocates are not handed out again while the call waits on
    its own stream."""
    gpu()
    k, v, table, ln = make_cache(1, 2, 128, 64, [6000], 40, seed=5)
    q = torch.randn(1, 2, 40, 128, generator=torch.Generator().manual_seed(3)).bfloat16()
    a = cuda(q, k, v, table, ln)
    x = torch.randn(1, 2, 2000, 128, device="cuda").bfloat16()
    o0, lse0 = ga.gpt_attn_paged_decode(*a)
    f0, l0 = ga.gpt_attn_fwd_sinks(x, x, x, window=100, sinks=4)
    want = [o0.clone(), ga.gpt_attn_bwd_sinks(x, x, x, f0, l0, x, window=100, sinks=4)[2].clone()]
    torch.cuda.synchronize()
    for raw in (False, True):
        s = torch.cuda.Stream()
        arg = s.cuda_stream if raw else s
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)                           # some 10 ms before the calls run
        got = []
        for _ in range(4):
            o, lse = ga.gpt_attn_paged_decode(*a, stream=arg)
            dv = ga.gpt_attn_bwd_sinks(x, x, x, f0, l0, x, window=100, sinks=4, stream=arg)[2]
            got.append((o, dv))
            for n in (2 ** 12, 2 ** 16, 2 ** 20, 2 ** 22, 2 ** 24):  # the current stream overwrites what it gets
                torch.full((n,), float("nan"), device="cuda")
        torch.cuda.synchronize()
        for o, dv in got:
            assert torch.equal(o, want[0]) and torch.equal(dv, want[1])


@pytest.mark.gpu
def test_accept_any_order_and_repeats():
    gpu()
    k, v, table, ln = make_cache(2, 3, 128, 16, [30, 5], 64, seed=5)
    r = np.random.default_rng(1)
    acc = np.stack([r.permutation(64), r.integers(-1, 66, 64)]).astype(np.int32)
    n_acc = np.array([64, 41], dtype=np.int32)
    kd, vd, td, ld, ad, nd = cuda(k, v, table, ln, acc, n_acc)
    ga.gpt_attn_paged_accept(kd, vd, td, ld, ad, nd)
    for got, was in ((kd.cpu(), k), (vd.cpu(), v)):
        want = was.clone()
        at = lambda b, x: (int(table[b, x // 16]), slice(None), x % 16)
        for b in range(2):
            for i in range(n_acc[b]):
                if 0 <= acc[b, i] < 64:
                    want[at(b, ln[b] + i)] = was[at(b, ln[b] + acc[b, i])]
        assert torch.equal(got.nan_to_num(9), want.nan_to_num(9))


@pytest.mark.gpu
def test_binding_refusals():
    gpu()
    k, v, table, ln = make_cache(2, 2, 64, 16, [30, 5], 2, seed=5)
    kd, vd, td, ld = cuda(k, v, table, ln)
    q = torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16, device="cuda")
    dec = ga.gpt_attn_paged_decode
    for bad in (dict(q=q.float()), dict(q=q[:1]), dict(q=q[..., :32]), dict(v_pages=vd[:-1]), dict(k_pages=kd.half()),
                dict(table=td.long()), dict(table=td.t().contiguous().t()), dict(lens=ld[:1]), dict(lens=ld.cpu()),
                dict(parents=torch.zeros(2, 3, dtype=torch.int32, device="cuda")),
                dict(n_new=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(o=q[:, :2]),
                dict(lse=torch.zeros(2, 4, 2, dtype=torch.float64, device="cuda")),
                dict(workspace=torch.zeros(4096, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            dec(**(dict(q=q, k_pages=kd, v_pages=vd, table=td, lens=ld) | bad))
    with pytest.raises(ga.GptAttnError):
        dec(q[:, :3], kd, vd, td, ld)                               # 3 query heads on 2 key heads
    with pytest.raises(ga.GptAttnError):
        dec(q, kd, vd, td, ld, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
