"""Reserving and forking when free pages are few."""
import numpy as np
import pytest
import torch

import causal_attention_sdpa_b200 as ga
from oracle import streaming

# Pages of 4 tokens, all seven held but none free, or one free.  Slots 0 and 3 end on a page's border, 1 and 2
# have room in their last page, 4 and 5 are empty.
TABLE = np.array([[0, 1, -1], [2, -1, -1], [3, 4, -1], [5, -1, -1], [-1, -1, -1], [-1, -1, -1]], dtype=np.int32)
LENS = np.array([8, 2, 7, 4, 0, 0], dtype=np.int32)
RESERVE = [  # free pages, tokens, status, pages given
    (0, [1, 2, 1, 0, 0, 0], [-2, 1, 1, 0, 0, 0], {}),
    (0, [0, 2, 2, 1, 1, -1], [0, 1, -2, -2, -2, 0], {}),
    (1, [9, 1, 1, 1, 0, 4], [-1, 1, 1, 1, 0, -2], {3: [6]}),
    (1, [5, 2, 1, 1, 0, 0], [-1, 1, 1, 1, 0, 0], {3: [6]}),
    (1, [4, 2, 1, 1, 3, 0], [1, 1, 1, -2, -2, 0], {0: [6]}),
]
FORK = [  # free pages, parents, status
    (0, [-1, -1, -1, -1, 0, 3], [0, 0, 0, 0, 1, 1]),
    (0, [-1, -1, -1, -1, 1, 3], [0, 0, 0, 0, -2, 1]),
    (1, [-1, -1, -1, -1, 1, 2], [0, 0, 0, 0, 1, -2]),
]


def refs_of(free):
    refs = np.array([1] * 6 + [2] * (1 - free) + [0] * free, dtype=np.int32)
    return refs


def row_of(s, more):
    r = [e for e in TABLE[s].tolist() if e >= 0] + more
    return r + [-1] * (3 - len(r))


@pytest.mark.parametrize("free,tokens,status,given", RESERVE)
def test_oracle_reserve_by_hand(free, tokens, status, given):
    t, r, st = streaming.pages_reserve(TABLE, LENS, refs_of(free), 4, tokens)
    assert st == status
    assert t.tolist() == [row_of(s, given.get(s, [])) for s in range(6)]


@pytest.mark.parametrize("free,parents,status", FORK)
def test_oracle_fork_by_hand(free, parents, status):
    t, n, r, st, pairs = streaming.pages_fork(TABLE, LENS, refs_of(free), 4, parents)
    assert st == status
    for s, src in enumerate(parents):
        if status[s] == 1 and LENS[src] % 4 == 0:
            assert t[s].tolist() == TABLE[src].tolist() and n[s] == LENS[src]


def cuda(*xs):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_attention_sdpa_b200 import build
    build.build()
    return [torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda() for x in xs]


def same(got, want):
    assert np.array_equal(got.cpu().numpy(), np.asarray(want, dtype=np.int32))


@pytest.mark.gpu
@pytest.mark.parametrize("free,tokens,status,given", RESERVE)
def test_reserve(free, tokens, status, given):
    """What a slot's own pages hold is not refused for lack of pages that another one asks for."""
    t, n, r, tok = cuda(TABLE, LENS, refs_of(free), tokens)
    same(ga.gpt_attn_pages_reserve(t, n, r, 4, tok), status)
    same(t, [row_of(s, given.get(s, [])) for s in range(6)])
    same(r, streaming.pages_reserve(TABLE, LENS, refs_of(free), 4, tokens)[1])


@pytest.mark.gpu
@pytest.mark.parametrize("free,parents,status", FORK)
def test_fork(free, parents, status):
    t, n, r, par = cuda(TABLE, LENS, refs_of(free), parents)
    st, pairs = ga.gpt_attn_pages_fork(t, n, r, 4, par)
    same(st, status)
    for g, w in zip((t, n, r, st, pairs), streaming.pages_fork(TABLE, LENS, refs_of(free), 4, parents)):
        same(g, w)


@pytest.mark.gpu
@pytest.mark.parametrize("S,M,page", [(5, 3, 4), (70, 40, 7), (300, 8, 16)])
def test_a_full_pool_against_the_plain_definition(S, M, page):
    """Every page held: whatever asks for none is served, whatever asks for one is not."""
    r = np.random.default_rng(S)
    lens = r.integers(1, M * page + 1, S).astype(np.int32)
    lens[::3] = lens[::3] // page * page
    lens[::7] = 0
    held = -(-lens // page)
    places = r.permutation(int(held.sum()))
    table, at = np.full((S, M), -1, dtype=np.int32), 0
    for s in range(S):
        table[s, :held[s]] = places[at:at + held[s]]
        at += held[s]
    refs = np.ones(len(places), dtype=np.int32)
    tokens = r.integers(0, page, S)
    t, n, rf, tok = cuda(table, lens, refs, tokens)
    status = ga.gpt_attn_pages_reserve(t, n, rf, page, tok)
    wt, wr, ws = streaming.pages_reserve(table, lens, refs, page, tokens)
    assert S < 50 or (1 in ws and -2 in ws)
    for g, w in ((t, wt), (rf, wr), (status, ws)):
        same(g, w)
    parents = np.where(lens == 0, r.integers(0, S, S), -1)
    t, n, rf, par = cuda(table, lens, refs, parents)
    got = ga.gpt_attn_pages_fork(t, n, rf, page, par)
    for g, w in zip((t, n, rf, *got), streaming.pages_fork(table, lens, refs, page, parents)):
        same(g, w)
