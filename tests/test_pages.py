"""Reserving, forking, freeing, packing and copying the pages of a paged cache, against the plain
definitions in oracle/streaming.py.  Everything is whole numbers and copies, so results are equal."""
import ctypes

import numpy as np
import pytest
import torch

import causal_attention_sdpa_b200 as ga
from oracle import streaming


def state(S, M, P, page, seed, share=0.5):
    """A consistent state: some slots filled, pages in a random order."""
    r = np.random.default_rng(seed)
    table = np.full((S, M), -1, dtype=np.int32)
    lens, refs = np.zeros(S, dtype=np.int32), np.zeros(P, dtype=np.int32)
    places = list(r.permutation(P))
    for s in r.permutation(S)[:max(1, round(S * share))]:
        n = int(r.integers(0, M * page + 1))
        held = -(-n // page)
        if held + 1 > len(places):
            break
        table[s, :held] = [places.pop() for _ in range(held)]
        refs[table[s, :held]] = 1
        lens[s] = n
    return table, lens, refs


# ------------------------------------------------------------------------------ oracle
def test_oracle_fork_free_compact_by_hand():
    table = np.array([[3, 1, -1], [-1, -1, -1], [-1, -1, -1]], dtype=np.int32)
    lens, refs = np.array([6, 0, 0], dtype=np.int32), np.array([0, 1, 0, 1, 0], dtype=np.int32)
    t, n, r, status, pairs = streaming.pages_fork(table, lens, refs, 4, [-1, 0, 0])
    assert t.tolist() == [[3, 1, -1], [3, 0, -1], [3, 2, -1]] and n.tolist() == [6, 6, 6]
    assert r.tolist() == [1, 1, 1, 3, 0] and status == [0, 1, 1] and pairs == [(-1, -1), (1, 0), (1, 2)]
    t, n, r = streaming.pages_free(t, n, r, [1, 0, 1])
    assert t[1].tolist() == [3, 0, -1] and r.tolist() == [1, 0, 0, 1, 0] and n.tolist() == [0, 6, 0]
    t, r, moves = streaming.pages_compact(t, r)
    assert t[1].tolist() == [1, 0, -1] and r.tolist() == [1, 1, 0, 0, 0] and moves == [(3, 1)]
    t, r, status = streaming.pages_reserve(t, n, r, 4, [9, 3, 100])
    assert status == [1, -2, -1] and t.tolist() == [[2, 3, 4], [1, 0, -1], [-1, -1, -1]] and r.tolist() == [1] * 5


# ------------------------------------------------------------------------------ refusals
FAKE = 0x10000


def test_refusals():
    from causal_attention_sdpa_b200 import build
    build.build()
    L, vp = ga.lib(), ctypes.c_void_p
    need = ga.gpt_attn_pages_workspace_bytes(4, 3, 9)
    assert need > 0
    assert ga.gpt_attn_pages_workspace_bytes(0, 3, 9) == ga.gpt_attn_pages_workspace_bytes(2 ** 20, 2 ** 11, 9) == 0

    def call(name, n, tail, p=None, S=4, M=3, P=9, page=16, ws=FAKE, nbytes=need):
        p = [FAKE] * n if p is None else p
        v = [vp(x) for x in p]
        f = getattr(L, "gpt_attn_pages_" + name)
        if name == "compact":
            return f(v[0], v[1], S, M, P, *v[2:], vp(ws), nbytes, vp(0))
        if name == "free":
            return f(*v[:3], S, M, P, v[3], vp(0))
        return f(*v[:3], S, M, P, page, *v[3:], vp(ws), nbytes, vp(0))

    for name, n in (("reserve", 5), ("fork", 6), ("free", 4), ("compact", 6)):
        for i in range(n):
            p = [FAKE] * n
            p[i] = 0
            assert call(name, n, 0, p) == ga.GPT_ATTN_ERR_NULL
            p[i] = FAKE + 2
            assert call(name, n, 0, p) == ga.GPT_ATTN_ERR_ALIGN
        for kw in (dict(S=0), dict(M=0), dict(P=0), dict(S=2 ** 20, M=2 ** 11)):
            assert call(name, n, 0, **kw) == ga.GPT_ATTN_ERR_SHAPE
        if name != "free":
            assert call(name, n, 0, nbytes=need - 1) == call(name, n, 0, ws=0) == ga.GPT_ATTN_ERR_WORKSPACE
    assert call("fork", 6, 0, page=0) == call("reserve", 5, 0, page=0) == ga.GPT_ATTN_ERR_SHAPE

    def copy(k=FAKE, v=FAKE, P=9, Hkv=2, page=16, D=64, pairs=FAKE, n=3, cnt=0):
        return L.gpt_attn_pages_copy(vp(k), vp(v), P, Hkv, page, D, vp(pairs), n, vp(cnt), vp(0))

    assert copy(k=0) == copy(v=0) == copy(pairs=0) == ga.GPT_ATTN_ERR_NULL
    assert copy(k=FAKE + 8) == copy(pairs=FAKE + 4) == copy(cnt=FAKE + 2) == ga.GPT_ATTN_ERR_ALIGN
    assert copy(P=0) == copy(Hkv=0) == copy(page=0) == copy(n=-1) == copy(Hkv=2 ** 20, page=2 ** 11) == \
        ga.GPT_ATTN_ERR_SHAPE
    assert copy(D=80) == ga.GPT_ATTN_ERR_UNSUPPORTED_D
    assert copy(n=0) == ga.GPT_ATTN_OK                              # nothing to do: nothing is launched


def test_binding_refusals_on_the_host():
    t, r = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(9, dtype=torch.int32)
    with pytest.raises(ValueError):
        ga.gpt_attn_pages_compact(t, r)
    with pytest.raises(ValueError):
        ga.gpt_attn_pages_free(t, r[:2], r, r[:2])
    with pytest.raises(ValueError):
        ga.gpt_attn_pages_copy(torch.zeros(2, 1, 4, 64), torch.zeros(2, 1, 4, 64), t[:, :2])


# ------------------------------------------------------------------------------ GPU
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_attention_sdpa_b200 import build
    build.build()


def same(got, want):
    assert np.array_equal(got.cpu().numpy(), np.asarray(want, dtype=np.int32))


def cuda(*xs):
    return [torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda() for x in xs]


SHAPES = [(1, 1, 1, 16), (2, 1, 3, 1), (5, 3, 20, 4), (16, 12, 150, 64), (33, 40, 700, 7), (300, 8, 1500, 16),
          (1000, 5, 9001, 3), (7, 100, 40000, 64), (40, 8, 60, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("S,M,P,page", SHAPES)
def test_fork_and_free(S, M, P, page):
    gpu()
    table, lens, refs = state(S, M, P, page, seed=S + P)
    r = np.random.default_rng(S)
    empty = (lens == 0) & (table < 0).all(1)
    parents = np.where(empty & (r.random(S) < 0.8), r.integers(0, S, S), -1)
    # parents that are not there, themselves asked for, or asked of a slot that holds tokens
    parents[r.random(S) < 0.1] = S + 3
    parents[r.random(S) < 0.1] = r.integers(0, S)
    t, n, rf, par = cuda(table, lens, refs, parents)
    status, pairs = ga.gpt_attn_pages_fork(t, n, rf, page, par)
    wt, wn, wr, ws, wp = streaming.pages_fork(table, lens, refs, page, parents)
    for g, w in ((t, wt), (n, wn), (rf, wr), (status, ws), (pairs, wp)):
        same(g, w)
    drop = (r.random(S) < 0.5).astype(np.int32)
    ga.gpt_attn_pages_free(t, n, rf, cuda(drop)[0])
    for g, w in zip((t, n, rf), streaming.pages_free(wt, wn, wr, drop)):
        same(g, w)


@pytest.mark.gpu
@pytest.mark.parametrize("S,M,P,page", SHAPES)
def test_reserve(S, M, P, page):
    gpu()
    table, lens, refs = state(S, M, P, page, seed=S * P)
    r = np.random.default_rng(S)
    tokens = np.where(r.random(S) < 0.7, r.integers(-2, max(2, M * page // 2), S), 2 ** 31 - 1)
    t, n, rf, tok = cuda(table, lens, refs, tokens)
    status = ga.gpt_attn_pages_reserve(t, n, rf, page, tok)
    wt, wr, ws = streaming.pages_reserve(table, lens, refs, page, tokens)
    for g, w in ((t, wt), (rf, wr), (status, ws), (n, lens)):
        same(g, w)


@pytest.mark.gpu
@pytest.mark.parametrize("S,M,P,page", SHAPES)
@pytest.mark.parametrize("share", [0.0, 0.3, 1.0])
def test_compact(S, M, P, page, share):
    gpu()
    table, lens, refs = state(S, M, P, page, seed=S + P, share=share)
    if share == 0.0:
        table[:], lens[:], refs[:] = -1, 0, 0
    table[-1, -1] = P + 5                                           # no page of the pool
    t, rf = cuda(table, refs)
    nt, nr, pairs, moves = ga.gpt_attn_pages_compact(t, rf)
    wt, wr, wm = streaming.pages_compact(table, refs)
    for g, w in ((nt, wt), (nr, wr), (t, table), (rf, refs), (moves, [len(wm)])):
        same(g, w)
    same(pairs, wm + [(-1, -1)] * (P // 2 - len(wm)) if P > 1 else np.zeros((0, 2)))


@pytest.mark.gpu
def test_fork_refuses_what_is_not_whole():
    """Missing pages, pages nobody holds, lengths the row cannot have: the slot stays as it was."""
    gpu()
    table = np.array([[0, 1], [-1, 3], [9, 5], [4, -1], [6, 7], [2, 2], [-1, -1], [-1, 0], [-1, -1], [-1, -1],
                      [-1, -1], [-1, -1]], dtype=np.int32)
    lens = np.array([8, 8, 8, 9, -1, 4, 0, 0, 0, 3, 0, 0], dtype=np.int32)
    refs = np.array([1, 1, 0, 1, 1, 1, 1, 1, 1], dtype=np.int32)
    for src in (0, 1, 2, 3, 4, 5, 8, 2 ** 31 - 1):
        parents = np.full(12, -1, dtype=np.int32)
        parents[[6, 7, 8, 9, 10]] = src
        parents[11] = 11
        t, n, rf, par = cuda(table, lens, refs, parents)
        status, pairs = ga.gpt_attn_pages_fork(t, n, rf, 4, par)
        for g, w in zip((t, n, rf, status, pairs), streaming.pages_fork(table, lens, refs, 4, parents.tolist())):
            same(g, w)


@pytest.mark.gpu
@pytest.mark.parametrize("P,Hkv,page,D,n", [(1, 1, 1, 64, 1), (40, 3, 7, 64, 12), (300, 12, 64, 64, 140),
                                            (64, 5, 33, 128, 30), (2000, 1, 1, 128, 900), (24, 8, 1024, 128, 11)])
def test_copy(P, Hkv, page, D, n):
    gpu()
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(P, Hkv, page, D, device="cuda", generator=g).bfloat16() for _ in range(2))
    r = np.random.default_rng(2)
    order = r.permutation(P)
    to, src = order[:n], order[n:] if P > 1 else order
    pairs = np.stack([r.choice(src, n), to], 1).astype(np.int32)
    pairs[::5, 0] = -1
    pairs[3::7] = [P, 0]
    pairs[4::9, 1] = -2 ** 31
    p = torch.as_tensor(pairs).cuda()
    for cnt in (None, n // 2, 0, -4, n + 100):
        kd, vd = k.clone(), v.clone()
        ga.gpt_attn_pages_copy(kd, vd, p, n_pairs=None if cnt is None else cuda([cnt])[0])
        wk, wv = k.clone(), v.clone()
        for a, b in pairs[:n if cnt is None else max(0, cnt)].tolist():
            if 0 <= a < P and 0 <= b < P:
                wk[b], wv[b] = k[a], v[a]
        assert torch.equal(kd, wk) and torch.equal(vd, wv)
    ga.gpt_attn_pages_copy(k, v, p[:0])


@pytest.mark.gpu
def test_a_service_forks_grows_and_packs():
    """Prompts, beams, growth, ends and packing together, captured and replayed on one workspace, while
    the attention over the cache keeps its results."""
    gpu()
    S, M, P, page, H, D = 8, 6, 50, 16, 2, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.full((P, H, page, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.full((S, M), -1, dtype=torch.int32, device="cuda")
    lens, refs = torch.zeros(S, dtype=torch.int32, device="cuda"), torch.zeros(P, dtype=torch.int32, device="cuda")
    tokens, n_new, parents, drop = (torch.zeros(S, dtype=torch.int32, device="cuda") for _ in range(4))
    status, pairs = torch.zeros(S, dtype=torch.int32, device="cuda"), torch.zeros(S, 2, dtype=torch.int32, device="cuda")
    kn, vn = (torch.zeros(S, H, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.empty(ga.gpt_attn_pages_workspace_bytes(S, M, P), dtype=torch.uint8, device="cuda")

    def step():
        ga.gpt_attn_pages_free(table, lens, refs, drop)
        ga.gpt_attn_pages_fork(table, lens, refs, page, parents, status=status, pairs=pairs, workspace=ws)
        ga.gpt_attn_pages_copy(k, v, pairs)
        ga.gpt_attn_pages_reserve(table, lens, refs, page, n_new, status=tokens, workspace=ws)
        ga.gpt_attn_paged_append(k, v, table, lens, kn, vn, n_new=n_new)
        lens.add_(n_new)

    parents.fill_(-1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    hist = [[] for _ in range(S)]
    r = np.random.default_rng(3)
    for t in range(90):
        d, par = np.zeros(S, dtype=np.int32), np.full(S, -1, dtype=np.int32)
        for s_ in range(S):
            if hist[s_] and (r.random() < 0.05 or len(hist[s_]) == M * page):
                d[s_], hist[s_] = 1, []
        alive = [s_ for s_ in range(S) if hist[s_]]
        for s_ in range(S):
            if not hist[s_] and alive and r.random() < 0.3:
                par[s_] = r.choice(alive)
        for s_ in range(S):
            if par[s_] >= 0:
                hist[s_] = list(hist[par[s_]])
        more = np.array([1 if hist[s_] or s_ < 2 else 0 for s_ in range(S)], dtype=np.int32)
        for dst, src in ((drop, d), (parents, par), (n_new, more)):
            dst.copy_(torch.as_tensor(src))
        kn.copy_(torch.randn(kn.shape, device="cuda", generator=g))
        vn.copy_(torch.randn(vn.shape, device="cuda", generator=g))
        graph.replay()
        assert (status.cpu().numpy() == (par >= 0)).all() and (tokens.cpu().numpy() == more).all()
        for s_ in range(S):
            if more[s_]:
                hist[s_].append((kn[s_, :, 0].clone(), vn[s_, :, 0].clone()))
        if t % 30 == 20:
            n_table, n_refs, moves, n = ga.gpt_attn_pages_compact(table, refs, workspace=ws)
            ga.gpt_attn_pages_copy(k, v, moves, n_pairs=n)
            table.copy_(n_table)
            refs.copy_(n_refs)
            used = int((refs > 0).sum())
            assert (refs[:used] > 0).all() and int(table.max()) < used
    q = torch.randn(S, H, 1, D, device="cuda", generator=g).bfloat16()
    assert lens.tolist() == [len(x) for x in hist]
    # the newest token is in the pages already: the cache ends before it
    o, _ = ga.gpt_attn_paged_decode(q, k, v, table, (lens - 1).clamp(min=0), n_new=(lens > 0).int())
    for s_ in range(S):
        if not hist[s_]:
            assert (o[s_] == 0).all()
            continue
        kk, vv = (torch.stack([x[i] for x in hist[s_]], 1).double() for i in range(2))
        p = torch.softmax((kk @ q[s_, :, 0, :, None].double()).squeeze(-1) * D ** -0.5, -1)
        want = (p[:, None] @ vv)
        assert float((o[s_].double() - want).abs().max()) <= 2e-2


@pytest.mark.gpu
def test_binding_refusals():
    gpu()
    table, lens, refs = state(4, 3, 20, 16, 1)
    t, n, r = cuda(table, lens, refs)
    z = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (dict(table=t.long()), dict(lens=n[:3]), dict(refs=r.cpu()), dict(parents=z[:2]), dict(status=z.float()),
                dict(pairs=torch.zeros(4, 3, dtype=torch.int32, device="cuda")), dict(table=t[:, ::2]),
                dict(workspace=torch.zeros(4096, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            ga.gpt_attn_pages_fork(**(dict(table=t, lens=n, refs=r, page=16, parents=z) | bad))
    with pytest.raises(ga.GptAttnError):
        ga.gpt_attn_pages_fork(t, n, r, 0, z)
    with pytest.raises(ga.GptAttnError):
        ga.gpt_attn_pages_reserve(t, n, r, 16, z, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
