"""Reserving for rows of the table that have a page behind a missing one: refused, and left as they are."""
import numpy as np
import pytest
import torch

import causal_attention_sdpa_b200 as ga
from oracle import streaming


def state(M):
    """Slots of M pages of 4 tokens: whole, with the first, a middle or the last entry missing before a page."""
    table = np.full((6, M), -1, dtype=np.int32)
    held = [2, M - 2, M - 2, M - 2, 1, 0]
    at = 0
    for s, n in enumerate(held):
        table[s, :n] = range(at, at + n)
        at += n
    table[1, 0] = -1                                # what a window left behind
    table[2, (M - 2) // 2] = -1
    table[3, M - 3], table[3, M - 1] = -1, table[3, M - 3]
    refs = np.zeros(at + 3 * M, dtype=np.int32)
    refs[table[table >= 0]] = 1
    return table, np.array([7, 4 * (M - 2), 4 * (M - 2) - 3, 4 * (M - 2), 4, 0], dtype=np.int32), refs


@pytest.mark.parametrize("M", [4, 33, 70, 200])
def test_oracle(M):
    table, lens, refs = state(M)
    t, r, status = streaming.pages_reserve(table, lens, refs, 4, [3, 1, 1, 4, 5, 0])
    whole = M == 4                                  # slot 2 has two pages then, the second of which is missing
    assert status == [1, -1, 1 if whole else -1, -1, 1, 0]
    assert (t[0, :3] >= 0).all() and (t[4, :3] >= 0).all()
    for s in (1, 3) if whole else (1, 2, 3):
        assert (t[s] == table[s]).all()
    assert int((r > 0).sum()) == int((refs > 0).sum()) + 3 + whole


@pytest.mark.gpu
@pytest.mark.parametrize("M", [4, 33, 70, 200])
def test_reserve(M):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_attention_sdpa_b200 import build
    build.build()
    table, lens, refs = state(M)
    for tokens in ([3, 1, 1, 4, 5, 0], [0, 0, 2, 0, 0, 9], [1, 8, 11, 8, 4 * M - 4, 4 * M]):
        t, n, r, tok = (torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda() for x in (table, lens, refs, tokens))
        status = ga.gpt_attn_pages_reserve(t, n, r, 4, tok)
        for g, w in zip((t, r, status), streaming.pages_reserve(table, lens, refs, 4, tokens)):
            assert np.array_equal(g.cpu().numpy(), np.asarray(w, dtype=np.int32))
