"""Inputs and gradients that repeat along heads or rows of a batch (stride 0), as expand and reductions leave them."""
import pytest
import torch

import causal_attention_sdpa_b200 as ga
from workloads import make_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_attention_sdpa_b200 import build
    build.build()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kw", [dict(), dict(window=60), dict(window=60, sinks=5)], ids=["causal", "window", "sinks"])
@pytest.mark.parametrize("dims", [(2, 1), (1, 3)], ids=["heads", "batch"])
def test_shared_keys_and_values(D, kw, dims):
    """Keys and values of one head (or one row) for all: the same as with copies, and their gradients summed."""
    from causal_attention_sdpa_b200.autograd import gpt_attention
    B, H, T = 2, 3, 300
    q, k, v, do = (t.cuda() for t in make_inputs(B, H, T, D, seed=3))
    k, v = k[:dims[0], :dims[1]].contiguous(), v[:dims[0], :dims[1]].contiguous()
    out = []
    for copy in (False, True):
        leaves = [t.clone().requires_grad_() for t in (q, k, v)]
        wide = [t.expand(B, H, T, D) for t in leaves]
        assert 0 in wide[1].stride()
        if copy:
            wide = [t.contiguous() for t in wide]
        o = gpt_attention(*wide, **kw)
        o.backward(do)
        out.append((o.detach(), *(t.grad for t in leaves)))
    assert ga.gpt_attn_check() == ga.GPT_ATTN_OK
    for i in (0, 2, 3):
        assert torch.equal(out[0][i], out[1][i])
    # dq: the order of its fp32 additions varies, which can turn a rounding: one bf16 step, 2^-7 of a value at most
    assert float((out[0][1].float() - out[1][1].float()).abs().max()) <= 2 ** -7 * float(out[1][1].abs().max())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kw", [dict(), dict(window=60, sinks=5)], ids=["causal", "sinks"])
@pytest.mark.parametrize("dim", [0, 1, 2])
def test_gradients_that_repeat(D, kw, dim):
    """The gradient of a mean over rows, heads or tokens comes with a stride of 0."""
    from causal_attention_sdpa_b200.autograd import gpt_attention
    q, k, v, do = (t.cuda() for t in make_inputs(2, 3, 300, D, seed=3))
    w = do.sum(dim)
    out = []
    for copy in (False, True):
        leaves = [t.clone().requires_grad_() for t in (q, k, v)]
        o = gpt_attention(*leaves, **kw)
        g = w.unsqueeze(dim).expand_as(o)
        o.backward(g.contiguous() if copy else g)
        out.append([t.grad for t in leaves])
    assert ga.gpt_attn_check() == ga.GPT_ATTN_OK
    assert torch.equal(out[0][1], out[1][1]) and torch.equal(out[0][2], out[1][2])
    assert float((out[0][0].float() - out[1][0].float()).abs().max()) <= 2 ** -7 * float(out[1][0].abs().max())


def test_paged_calls():
    """New rows and queries that repeat along heads."""
    B, H, N, D, page = 2, 4, 3, 64, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()
    k, v = rnd(20, H, page, D), rnd(20, H, page, D)
    table = torch.randperm(20, device="cuda", generator=g)[:16].view(2, 8).int()
    lens = torch.tensor([100, 37], dtype=torch.int32, device="cuda")
    kn, q = rnd(B, 1, N, D).expand(B, H, N, D), rnd(B, 1, N, D).expand(B, H, N, D)
    out = []
    for f in (lambda t: t, lambda t: t.contiguous()):
        a, b = k.clone(), v.clone()
        ga.gpt_attn_paged_append(a, b, table, lens, f(kn), f(kn))
        out.append((a, b, *ga.gpt_attn_paged_decode(f(q), a, b, table, lens)))
    for x, y in zip(*out):
        assert torch.equal(x, y)


def odd(t, dim):
    """t with a stride of no use to anyone in its dimension of size 1."""
    assert t.shape[dim] == 1
    st = list(t.stride())
    st[dim] = t.numel() + 3
    return t.as_strided(t.shape, st)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape,dim", [((1, 3, 300), 0), ((2, 1, 300), 1), ((2, 3, 1), 2)], ids=["B1", "H1", "T1"])
def test_strides_of_dimensions_of_size_one(D, shape, dim):
    """They are never stepped along, so any will do, beside tensors that are not contiguous too."""
    B, H, T = shape
    q, k, v, do = (t.cuda() for t in make_inputs(B, H, T, D, seed=3))
    major = lambda: torch.full((B, T, H, D), float("nan"), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    for kw in (dict(), dict(window=60, sinks=5)):
        fwd, bwd = (ga.gpt_attn_fwd_sinks, ga.gpt_attn_bwd_sinks) if kw else (ga.gpt_attn_fwd_ex, ga.gpt_attn_bwd_ex)
        o, lse = fwd(q, k, v, **kw)
        want = bwd(q, k, v, o, lse, do, **kw)
        x = [odd(t, dim) for t in (q, k, v, o, do)]
        got, l2 = fwd(*x[:3], o=odd(major(), dim), **kw)
        assert torch.equal(got, o) and torch.equal(l2, lse)
        g = bwd(*x[:4], lse, x[4], dq=major(), dk=odd(major(), dim), dv=odd(torch.empty_like(q), dim), **kw)
        assert torch.equal(g[1], want[1]) and torch.equal(g[2], want[2])
    assert ga.gpt_attn_check() == ga.GPT_ATTN_OK


def test_prologue_strides_of_dimensions_of_size_one():
    q, k, _, _ = (t.cuda() for t in make_inputs(1, 3, 300, 64, seed=3))
    for a, b in zip(ga.gpt_attn_qk_prologue_fwd(odd(q, 0), odd(k, 0)), ga.gpt_attn_qk_prologue_fwd(q, k)):
        assert torch.equal(a, b)
