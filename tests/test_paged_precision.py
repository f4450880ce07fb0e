"""How exact the paged attention of up to 16 rows a key head is: its only rounding to 16 bits is that of O."""
import numpy as np
import pytest
import torch

import causal_attention_sdpa_b200 as ga
from oracle import streaming
from test_paged import cuda, make_cache, random_trees


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,N,lens,W", [(1, 1, [3, 9, 30, 1, 70, 17], 0), (4, 1, [5, 12, 2, 40], 0), (16, 1, [7, 20], 0),
                                        (1, 16, [4, 11, 2], 0), (2, 8, [6, 25], 10), (1, 5, [300, 1000, 4], 9),
                                        (3, 5, [129, 5], 0), (8, 1, [700, 5, 33], 0), (9, 1, [700, 5, 33], 0),
                                        (1, 8, [60, 2], 30), (1, 9, [60, 2], 30)])
def test_one_rounding(G, N, lens, W, D):
    """P enters the second product in two bf16 terms.  Each is off by 2^-8 of what it rounds at most, so P
    is by 2^-16; scores are fp32 sums of up to 128 products, which with the exponential leaves P off by less
    than 2^-13 of itself at these sizes (128 2^-24 sum |q k| scale is 2^-14), and l by the same.  O is then off
    by 2^-12 of sum P |v| / l before its rounding, half a step, 2^-8 of it at most.  P in one term would add up to
    2^-8 of the former."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_attention_sdpa_b200 import build
    build.build()
    Hkv = 8
    k, v, table, ln = make_cache(len(lens), Hkv, D, 16, lens, N, seed=D + N)
    q = torch.randn(len(lens), Hkv * G, N, D, generator=torch.Generator().manual_seed(3)).bfloat16()
    par = random_trees(len(lens), N, 5) if N > 1 else None
    tree = None if par is None else torch.as_tensor(par).cuda()
    o, lse = ga.gpt_attn_paged_decode(*cuda(q, k, v, table, ln), parents=tree, window=W, sinks=2 if W else 0)
    assert ga.gpt_attn_check() == ga.GPT_ATTN_OK
    args = (table, ln, par, None, D ** -0.5, W, 2 if W else 0)
    want, wl = streaming.paged_decode(q, k, v, *args)
    weight, _ = streaming.paged_decode(q, k, v.abs(), *args)        # sum P |v| / l
    over = np.abs(o.float().cpu().double().numpy() - want) - 2.0 ** -8 * np.abs(want) - 2.0 ** -12 * weight
    assert float(over.max()) <= 0
    assert float(np.abs(lse.cpu().double().numpy() - wl).max()) <= 2.0 ** -13
