"""Windows, sinks and sizes past the range of a C int: they act as large as they are, or are refused."""
import pytest
import torch

import causal_attention_sdpa_b200 as ga
from workloads import make_inputs

TOP = 2 ** 31 - 1
PAST = [2 ** 31, 2 ** 32 + 3, 2 ** 40]


def built():
    from causal_attention_sdpa_b200 import build
    build.build()


def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    built()


@pytest.mark.parametrize("x", PAST)
def test_masks_and_workspaces_on_the_host(x):
    built()
    assert ga._sinks_mask(2, x, None, None)[0].window == TOP
    m, hw = ga._mask(2, -x, [x, 5])
    assert m.window < 0 and list(hw) == [TOP, 5]
    ws = ga.gpt_attn_bwd_sinks_workspace_bytes
    assert ws(1, 2, 8192, 128, 100, x) == ws(1, 2, 8192, 128, 100, TOP) > ws(1, 2, 8192, 128, 100, 0)
    assert ws(1, 2, 8192, 128, x, 4) == ws(1, 2, 8192, 128, TOP, 4)
    one = dict(B=1, H=2, T=8192, D=64)
    for n in one:
        assert ga.gpt_attn_bwd_workspace_bytes(**one | {n: one[n] + 2 ** 32}) == 0
        assert ws(**one | {n: one[n] + 2 ** 32}, window=100, sinks=4) == 0
        assert ws(**one | {n: one[n] - 2 ** 32}, window=100, sinks=4) == 0
    assert ga.gpt_attn_bwd_workspace_bytes(**one) > 0
    cases = ((ga.gpt_attn_paged_decode_workspace_bytes, (2, 4, 2, 3, 64)), (ga.gpt_attn_pages_workspace_bytes, (4, 3, 9)),
             (ga.gpt_attn_decode_workspace_bytes, (2, 3, 500, 64)))
    for f, a in cases:
        assert f(*a) > 0
        for i in range(len(a)):
            assert f(*a[:i], a[i] + 2 ** 32, *a[i + 1:]) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("x", PAST)
def test_windows_and_sinks_past_an_int(x):
    gpu()
    q, k, v, do = (t.cuda() for t in make_inputs(1, 2, 500, 64, seed=1))
    for kw in (dict(window=30, sinks=x), dict(window=x, sinks=3), dict(head_windows=[20, x], sinks=3),
               dict(head_windows=[20, 30], sinks=x)):
        low = {n: [min(y, TOP) for y in z] if isinstance(z, list) else min(z, TOP) for n, z in kw.items()}
        o, lse = ga.gpt_attn_fwd_sinks(q, k, v, **kw)
        o2, lse2 = ga.gpt_attn_fwd_sinks(q, k, v, **low)
        assert torch.equal(o, o2) and torch.equal(lse, lse2), kw
        g, g2 = ga.gpt_attn_bwd_sinks(q, k, v, o, lse, do, **kw), ga.gpt_attn_bwd_sinks(q, k, v, o, lse, do, **low)
        assert torch.equal(g[1], g2[1]) and torch.equal(g[2], g2[2]), kw
    assert torch.equal(ga.gpt_attn_fwd(q, k, v, window=x)[0], ga.gpt_attn_fwd(q, k, v)[0])
    assert torch.equal(ga.gpt_attn_fwd_ex(q, k, v, head_windows=[x, 9])[0], ga.gpt_attn_fwd_ex(q, k, v, head_windows=[0, 9])[0])
    kp = k.view(1, 2, 500, 64)[:, :, :480].reshape(1, 2, 30, 16, 64).permute(2, 0, 1, 3, 4).reshape(30, 2, 16, 64).contiguous()
    table = torch.arange(30, dtype=torch.int32, device="cuda").view(1, 30)
    lens = torch.tensor([470], dtype=torch.int32, device="cuda")
    dec = lambda **kw: ga.gpt_attn_paged_decode(q[:, :, :3], kp, kp, table, lens, **kw)[0]
    assert torch.equal(dec(window=x, sinks=2), dec(window=TOP, sinks=2))
    assert torch.equal(dec(window=40, sinks=x), dec(window=40, sinks=TOP))
    one = lambda w: ga.gpt_attn_decode(q[:, :, 0].contiguous(), k, v, lens, window=w)[0]
    assert torch.equal(one(x), one(0))


@pytest.mark.gpu
def test_page_sizes_past_an_int_are_refused():
    gpu()
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    for page in (2 ** 31, 2 ** 32 + 16, -2 ** 32 + 16):
        with pytest.raises(ValueError):
            ga.gpt_attn_pages_reserve(z(2, 3) - 1, z(2), z(9), page, z(2))
        with pytest.raises(ValueError):
            ga.gpt_attn_pages_fork(z(2, 3) - 1, z(2), z(9), page, z(2) - 1)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("x", [500, 501, 2 ** 30, TOP - 1, TOP, 2 ** 31, 2 ** 40])
def test_backward_with_windows_past_the_row(x, D):
    """Positions and such windows add up past an int, so they are cut to the row's length first."""
    gpu()
    q, k, v, do = (t.cuda() for t in make_inputs(2, 2, 500, D, seed=1))
    o, lse = ga.gpt_attn_fwd(q, k, v, window=x)
    o2, lse2 = ga.gpt_attn_fwd(q, k, v)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    g, g2 = ga.gpt_attn_bwd(q, k, v, o, lse, do, window=x), ga.gpt_attn_bwd(q, k, v, o, lse, do)
    assert torch.equal(g[1], g2[1]) and torch.equal(g[2], g2[2])
    kw, low = dict(head_windows=[x, 60], doc_start=None), dict(head_windows=[0, 60], doc_start=None)
    for _ in range(2):
        o, lse = ga.gpt_attn_fwd_ex(q, k, v, **kw)
        assert torch.equal(o, ga.gpt_attn_fwd_ex(q, k, v, **low)[0])
        g, g2 = ga.gpt_attn_bwd_ex(q, k, v, o, lse, do, **kw), ga.gpt_attn_bwd_ex(q, k, v, o, lse, do, **low)
        assert torch.equal(g[1], g2[1]) and torch.equal(g[2], g2[2])
        kw["doc_start"] = low["doc_start"] = torch.tensor([[0] * 130 + [130] * 370] * 2, dtype=torch.int32, device="cuda")
