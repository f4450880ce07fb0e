"""Training attention with scales of either sign and of 0, through the plain, windowed, masked and sinks calls."""
import numpy as np
import pytest
import torch

import causal_attention_sdpa_b200 as ga
from oracle import streaming
from workloads import make_doc_starts, make_inputs

pytestmark = pytest.mark.gpu
TOL_O, TOL_REL, TOL_LSE = 2e-2, 1e-2, 1e-3                          # the library's parity tolerances


@pytest.fixture(autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_attention_sdpa_b200 import build
    build.build()


def roundings(q, k, v, do, scale, windows, sinks, ds):
    """Most that the roundings to bf16 can put into (o, dq, dk, dv), each half a step, 2^-8 of a value at
    most, to which a quarter is added for the fp32 sums.  P is rounded for P V and P^T dO, dS for the other
    two products, O for Delta = dO . O, which dS = P (dP - Delta) takes over with the weight P, and each
    result once.  The library's absolute 5e-2 is for a scale of D^-1/2 and a softmax as flat as that: at
    -0.3 and D = 128 dK itself is 3.4 times as large, and so are the roundings behind it."""
    q, k, v, do = (x.double().numpy() for x in (q, k, v, do))
    B, H, T, _ = q.shape
    h = 2.0 ** -8 * 1.25
    out = [np.empty_like(q) for _ in range(4)]
    for b in range(B):
        for x in range(H):
            vis = streaming.sink_mask(T, windows if isinstance(windows, int) else windows[x], sinks,
                                      None if ds is None else ds[b])
            p, _ = streaming.masked_softmax(scale * q[b, x] @ k[b, x].T, vis)
            o, dp = p @ v[b, x], do[b, x] @ v[b, x].T
            d = p * (dp - (p * dp).sum(-1, keepdims=True))
            off = h * np.abs(d) + p * (h * np.abs(do[b, x] * o).sum(-1, keepdims=True))
            out[0][b, x] = h * (np.abs(o) + p @ np.abs(v[b, x]))
            out[1][b, x] = abs(scale) * (h * np.abs(d @ k[b, x]) + off @ np.abs(k[b, x]))
            out[2][b, x] = abs(scale) * (h * np.abs(d.T @ q[b, x]) + off.T @ np.abs(q[b, x]))
            out[3][b, x] = h * (np.abs(p.T @ do[b, x]) + p.T @ np.abs(do[b, x]))
    return out


def close(name, got, want, bound):
    g = got.float().cpu().double().numpy()
    assert np.isfinite(g).all(), name
    assert float((np.abs(g - want) - bound).max()) <= 1e-6, name
    n = float(np.linalg.norm(want))
    if n > 1e-6 * want.size ** 0.5:                                 # a scale of 0: dq and dk are exactly 0
        assert float(np.linalg.norm(g - want)) / n <= TOL_REL, name


CASES = [  # T, window (or one per head), sinks, documents' longest length
    (300, 0, 0, 0), (300, 70, 0, 0), (700, [50, 0], 0, 0), (400, 0, 0, 150), (1, 3, 2, 0), (700, 100, 4, 0),
    (520, 130, 140, 0), (700, 60, 3, 300), (300, [40, 0], 5, 0),
]


@pytest.mark.parametrize("scale", [0.0, -0.0, -0.3, -1e-3, 0.2, 1e-38])
@pytest.mark.parametrize("T,W,sinks,docs", CASES, ids=["-".join(map(str, c)).replace(" ", "") for c in CASES])
@pytest.mark.parametrize("D", [64, 128])
def test_parity(T, W, sinks, docs, D, scale):
    B, H = 2, 2
    q, k, v, do = make_inputs(B, H, T, D, seed=T + D)
    ds = make_doc_starts(B, T, 7, docs) if docs else None
    hw = W if isinstance(W, list) else None
    how = dict(window=0 if hw else W, head_windows=hw, scale=scale,
               doc_start=None if ds is None else torch.as_tensor(ds, dtype=torch.int32).cuda())
    a = [t.cuda() for t in (q, k, v)]
    if sinks:
        o, lse = ga.gpt_attn_fwd_sinks(*a, sinks=sinks, **how)
        got = ga.gpt_attn_bwd_sinks(*a, o, lse, do.cuda(), sinks=sinks, **how)
    elif hw or docs:
        o, lse = ga.gpt_attn_fwd_ex(*a, **how)
        got = ga.gpt_attn_bwd_ex(*a, o, lse, do.cuda(), **how)
    else:
        o, lse = ga.gpt_attn_fwd(*a, scale=scale, window=W)
        got = ga.gpt_attn_bwd(*a, o, lse, do.cuda(), scale=scale, window=W)
    assert ga.gpt_attn_check() == ga.GPT_ATTN_OK
    ro, rl, *rg = streaming.attn_sinks(q, k, v, scale, W, sinks, None if ds is None else np.asarray(ds), do)
    bounds = roundings(q, k, v, do, scale, W, sinks, None if ds is None else np.asarray(ds))
    assert float(np.abs(lse.cpu().double().numpy() - rl).max()) <= TOL_LSE
    for n, g, r, b in zip(("o", "dq", "dk", "dv"), (o, *got), (ro, *rg), bounds):
        close(n, g, r, b)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sinks", [0, 5])
def test_a_negative_scale_is_negated_queries(D, sinks):
    q, k, v, do = (t.cuda() for t in make_inputs(2, 3, 700, D, seed=4))
    kw = dict(window=90, sinks=sinks)
    o, lse = ga.gpt_attn_fwd_sinks(q, k, v, scale=-0.2, **kw)
    o2, lse2 = ga.gpt_attn_fwd_sinks(-q, k, v, scale=0.2, **kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    g = ga.gpt_attn_bwd_sinks(q, k, v, o, lse, do, scale=-0.2, **kw)
    g2 = ga.gpt_attn_bwd_sinks(-q, k, v, o, lse, do, scale=0.2, **kw)
    assert torch.equal(g[1], g2[1]) and torch.equal(g[2], g2[2])
    # dq: the order of its fp32 additions varies, which can turn a rounding: one bf16 step, 2^-7 of a value at most
    assert float((g[0].float() + g2[0].float()).abs().max()) <= 2 ** -7 * float(g[0].abs().max())


def test_one_token_over_a_cache():
    B, H, T, D = 2, 3, 500, 64
    q, k, v, _ = make_inputs(B, H, T, D, seed=2)
    n = torch.tensor([500, 33], dtype=torch.int32)
    for scale in (0.0, -0.3):
        o, lse = ga.gpt_attn_decode(q[:, :, 0].contiguous().cuda(), k.cuda(), v.cuda(), n.cuda(), scale=scale)
        for b in range(B):
            for h in range(H):
                m = int(n[b])
                p, z = streaming.masked_softmax(scale * k[b, h, :m].double().numpy() @ q[b, h, 0].double().numpy(),
                                                np.ones(m, dtype=bool))
                assert np.abs(o[b, h].float().cpu().double().numpy() - p @ v[b, h, :m].double().numpy()).max() <= TOL_O
                assert abs(float(lse[b, h]) - float(z)) <= TOL_LSE
