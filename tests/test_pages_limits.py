"""The largest numbers of slots and pages: the table kernels' places fit an int, or the call is refused."""
import ctypes

import causal_attention_sdpa_b200 as ga

FAKE = 0x10000
STEP = 8 * 1024                                     # slots or pages that a step of the cluster goes through


def test_slices_of_the_largest_pool_fit_an_int():
    """The kernels' slices and steps, on whole numbers without a limit."""
    for n in (1, 7, 8, 9, 8191, 8193, 2 ** 31 - 2 ** 15):
        per = (n + 7) // 8
        assert per * 7 < 2 ** 31 and per * 8 < 2 ** 31
        for rank in range(8):
            lo = min(rank * per, n)
            hi = min(lo + per, n)
            assert hi + STEP < 2 ** 31


def test_refusals():
    from causal_attention_sdpa_b200 import build
    build.build()
    L, vp = ga.lib(), ctypes.c_void_p
    most = 2 ** 31 - 2 ** 15
    assert ga.gpt_attn_pages_workspace_bytes(1, 1, most) > most
    assert ga.gpt_attn_pages_workspace_bytes(most, 1, 1) > most
    for S, P in ((1, most + 2 ** 15 - 1), (most + 2 ** 15 - 1, 1), (1, most + 2 ** 15 - 512), (1, most + 2 ** 15 - 9000)):
        assert ga.gpt_attn_pages_workspace_bytes(S, 1, P) == 0
        p, big = vp(FAKE), 2 ** 62
        for rc in (L.gpt_attn_pages_reserve(p, p, p, S, 1, P, 16, p, p, p, big, vp(0)),
                   L.gpt_attn_pages_fork(p, p, p, S, 1, P, 16, p, p, p, p, big, vp(0)),
                   L.gpt_attn_pages_free(p, p, p, S, 1, P, p, vp(0)),
                   L.gpt_attn_pages_compact(p, p, S, 1, P, p, p, p, p, p, big, vp(0))):
            assert rc == ga.GPT_ATTN_ERR_SHAPE
