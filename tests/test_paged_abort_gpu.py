"""The paged decode kernels' own abort path, exercised without a fault (debug build).

The producers of block 0 are told to skip the first tile of keys: no copy, no arrival and no description of
the tile, so nothing is in flight for it.  The waits of the other roles (the warps that compute, the one
that issues products, the one that brings rows in) run out, all roles leave their loops, the producers wait
for the copies they did issue, TMEM is released, and gpt_attn_check reports GPT_ATTN_ERR_TIMEOUT.  The same
process then computes correct results."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import sys
sys.path[:0] = [ROOT, ROOT + "/tests"]
import torch
import causal_attention_sdpa_b200 as ga
from causal_attention_sdpa_b200 import build
from oracle import streaming
from test_paged import close, cuda, make_cache, random_trees

ga.LIB_PATH = build.build(debug=True)
L = ga.lib()


def run(D, G, N, lens, parity):
    k, v, table, ln = make_cache(len(lens), 2, D, 16, lens, N, seed=N)
    q = torch.randn(len(lens), 2 * G, N, D, generator=torch.Generator().manual_seed(3)).bfloat16()
    par = random_trees(len(lens), N, 5) if N > 1 else None
    o, lse = ga.gpt_attn_paged_decode(*cuda(q, k, v, table, ln), parents=None if par is None else torch.as_tensor(par).cuda())
    status = ga.gpt_attn_check()
    if parity:
        assert status == ga.GPT_ATTN_OK
        close(o, lse, *streaming.paged_decode(q, k, v, table, ln, par, None, D ** -0.5))
    return status


SHAPES = [(64, 1, 1), (128, 3, 1), (64, 3, 7), (128, 2, 12), (64, 4, 12), (128, 8, 20)]
assert ga.gpt_attn_check() == ga.GPT_ATTN_OK
for D, G, N in SHAPES:                              # the debug build's checks stay quiet on valid work
    run(D, G, N, [700, 3, 90], True)
for D, G, N in SHAPES:
    assert L.gpt_attn_debug_skip_load(3) == ga.GPT_ATTN_OK
    # long enough a list for block 0 to have tiles in its piece, behind what an item counts besides them
    assert run(D, G, N, [3000] * 64, False) == ga.GPT_ATTN_ERR_TIMEOUT, (D, G, N)
    assert L.gpt_attn_debug_skip_load(0) == ga.GPT_ATTN_OK
    run(D, G, N, [300, 0, 900], True)               # same process, after the aborted launch
assert L.gpt_attn_debug_skip_load(4) == ga.GPT_ATTN_ERR_SHAPE
print("ABORT_PATH_OK")
'''


@pytest.mark.gpu
def test_skipped_keys_time_out_and_the_context_survives():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    env = dict(os.environ, GPT_ATTN_WAIT_TIMEOUT_MS="200")
    r = subprocess.run([sys.executable, "-c", f"ROOT = {ROOT!r}\n" + CHILD], env=env, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0 and "ABORT_PATH_OK" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
