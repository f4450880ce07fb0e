"""Memory that the Python functions take for a call on another stream than the current one: results, and
workspaces that are given back when the function returns."""
import numpy as np
import pytest
import torch

import causal_attention_sdpa_b200 as ga

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def inputs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_attention_sdpa_b200 import build
    build.build()
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()
    S, M, P, page, N = 6, 8, 60, 16, 5
    order = torch.randperm(P, generator=g)[:S * 4].view(S, 4).int()
    table = torch.cat([order, torch.full((S, M - 4), -1, dtype=torch.int32)], 1)
    refs = torch.zeros(P, dtype=torch.int32)
    refs[order.flatten().long()] = 1
    table[5], refs[order[5].long()] = -1, 0
    s = dict(x=rnd(1, 2, 900, 64), q=rnd(S, 4, N, 64), k=rnd(P, 2, page, 64), v=rnd(P, 2, page, 64), table=table.cuda(),
             refs=refs.cuda(), lens=torch.tensor([50, 64, 33, 49, 59, 0], dtype=torch.int32).cuda(),
             more=torch.tensor([9, 1, 0, 40, 2, 0], dtype=torch.int32).cuda(),
             parents=torch.tensor([-1, -1, -1, -1, -1, 0], dtype=torch.int32).cuda(), page=page,
             cached=torch.tensor([45, 59, 28, 44, 54, 0], dtype=torch.int32).cuda(), dq=rnd(1, 2, 900, 64),
             one=rnd(1, 2, 64), at=torch.tensor([733], dtype=torch.int32).cuda())
    s["o"], s["lse"] = ga.gpt_attn_fwd_sinks(s["x"], s["x"], s["x"], window=100, sinks=4)
    s["xs"] = [s["x"]] * 3
    s["causal"] = [s["x"]] * 3 + list(ga.gpt_attn_fwd(*s["xs"])) + [s["x"]]
    torch.cuda.synchronize()
    return s


def _state(s):
    return s["table"].clone(), s["lens"].clone(), s["refs"].clone()


CALLS = {
    "fwd_sinks": lambda s, st: ga.gpt_attn_fwd_sinks(s["x"], s["x"], s["x"], window=100, sinks=4, stream=st),
    "bwd_sinks": lambda s, st: ga.gpt_attn_bwd_sinks(s["x"], s["x"], s["x"], s["o"], s["lse"], s["x"], window=100, sinks=4,
                                                     stream=st),
    "bwd_sinks_dq": lambda s, st: ga.gpt_attn_bwd_sinks(s["x"], s["x"], s["x"], s["o"], s["lse"], s["x"], window=100,
                                                        sinks=4, dq=s["dq"], stream=st),
    "decode": lambda s, st: ga.gpt_attn_paged_decode(s["q"], s["k"], s["v"], s["table"], s["cached"], stream=st),
    "reserve": lambda s, st: (ga.gpt_attn_pages_reserve(s["table"], s["lens"], s["refs"], s["page"], s["more"], stream=st),),
    "fork": lambda s, st: ga.gpt_attn_pages_fork(s["table"], s["lens"], s["refs"], s["page"], s["parents"], stream=st),
    "compact": lambda s, st: ga.gpt_attn_pages_compact(s["table"], s["refs"], stream=st),
    "fwd": lambda s, st: ga.gpt_attn_fwd(*s["xs"], stream=st),
    "fwd_ex": lambda s, st: ga.gpt_attn_fwd_ex(*s["xs"], head_windows=[0, 70], stream=st),
    "bwd": lambda s, st: ga.gpt_attn_bwd(*s["causal"], stream=st),
    "bwd_ex": lambda s, st: ga.gpt_attn_bwd_ex(*s["causal"], stream=st),
    "bwd_noalloc": lambda s, st: ga.gpt_attn_bwd_noalloc(*s["causal"], stream=st),
    "delta": lambda s, st: (ga.gpt_attn_bwd_delta(s["o"], s["lse"], s["x"], None, stream=st),),
    "cache_decode": lambda s, st: ga.gpt_attn_decode(s["one"], s["x"], s["x"], s["at"], stream=st),
    "prologue": lambda s, st: ga.gpt_attn_qk_prologue_fwd(s["x"], s["x"], stream=st),
    "prologue_bwd": lambda s, st: ga.gpt_attn_qk_prologue_bwd(*s["xs"], s["x"], stream=st),
}


@pytest.fixture()
def taken(monkeypatch, inputs):
    """The calls without their kernels; address and size of all memory that they take."""
    seen = []

    def watch(name):
        make = getattr(torch, name)

        def made(*a, **kw):
            t = make(*a, **kw)
            seen.append((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()))
            return t
        monkeypatch.setattr(torch, name, made)

    watch("empty")
    watch("empty_like")
    monkeypatch.setattr(ga, "_launch", lambda *a: None)
    real = ga.lib()

    class Lib:
        def __getattr__(self, name):
            return getattr(real, name) if name.endswith("_bytes") else lambda *a: ga.GPT_ATTN_OK
    monkeypatch.setattr(ga, "lib", Lib)
    return seen


def overlap(a, b):
    return any(x[0] < y[1] and y[0] < x[1] for x in a for y in b)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", sorted(CALLS))
def test_memory_comes_from_the_stream_of_the_call(inputs, taken, name, raw):
    """What the current stream gave back, its kernels perhaps still on their way, is not what a call on
    another stream writes."""
    torch.cuda.synchronize()
    CALLS[name](inputs, None)
    before = list(taken)
    assert before
    taken.clear()
    s = torch.cuda.Stream()
    CALLS[name](inputs, s.cuda_stream if raw else s)
    assert len(taken) == len(before) and not overlap(taken, before)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_memory_of_a_call_is_not_handed_out_while_it_waits(inputs, taken, name):
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)                           # some 10 ms before the call would run
    CALLS[name](inputs, s)                                      # results and workspace are dropped
    mine = list(taken)
    taken.clear()
    held = [torch.empty(b - a, dtype=torch.uint8, device="cuda") for a, b in mine for _ in range(3)]
    assert len(taken) == len(held) > 0 and not overlap(taken, mine)
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", sorted(CALLS))
def test_results_in_use_on_the_current_stream_are_kept(inputs, taken, name):
    """A result that is dropped while the current stream still has to read it is not written by the next
    call on the other stream."""
    s = torch.cuda.Stream()
    CALLS[name](inputs, s)
    torch.cuda.synchronize()
    taken.clear()
    out = CALLS[name](inputs, s)
    torch.cuda._sleep(20_000_000)
    mine = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in out if t.numel()]
    used = [t.clone() for t in out]                             # queued on the current stream
    del out
    taken.clear()
    CALLS[name](inputs, s)
    assert len(taken) > 0 and not overlap(taken, mine)
    torch.cuda.synchronize()
    del used


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", sorted(set(CALLS) - {"delta"}))       # delta's workspace has parts that nobody writes
def test_work_queued_on_the_current_stream_does_not_reach_the_call(inputs, name, raw):
    """The current stream is late with writing memory that was given back there; the call's stream is idle."""
    def run(st):
        own = dict(inputs)
        own["table"], own["lens"], own["refs"] = _state(inputs)
        torch.cuda.synchronize()
        out = CALLS[name](own, st)
        return out, own

    out, own = run(None)
    torch.cuda.synchronize()
    want = [t.clone() for t in (*out, own["table"], own["lens"], own["refs"])]
    sizes = {t.numel() * t.element_size() for t in out} | {2 ** n for n in range(9, 25)}
    del out, own
    s = torch.cuda.Stream()
    arg = s.cuda_stream if raw else s
    CALLS[name](dict(inputs, **dict(zip(("table", "lens", "refs"), _state(inputs)))), arg)      # first use of the stream
    own = dict(inputs)
    own["table"], own["lens"], own["refs"] = _state(inputs)
    spent = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes if n]
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    for t in spent:
        t.fill_(0x7f)
    del t, spent
    out = CALLS[name](own, arg)
    torch.cuda.synchronize()
    for a, b in zip((*out, own["table"], own["lens"], own["refs"]), want):
        if name.startswith("bwd") and a is out[0]:
            # dq: the order of its fp32 additions varies, which can turn a rounding: one bf16 step, 2^-7 of a value at most
            assert float((a.float() - b.float()).abs().max()) <= 2 ** -7 * float(b.abs().max())
        else:
            assert torch.equal(a, b)
    assert ga.gpt_attn_check() == ga.GPT_ATTN_OK


def test_the_streams_that_have_fixed_handles(inputs):
    """0 and 1 are the legacy default stream."""
    want = CALLS["fwd_sinks"](inputs, None)
    for h in (0, 1):
        got = CALLS["fwd_sinks"](inputs, h)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert np.isfinite(want[0].float().cpu().numpy()).all()


@pytest.mark.parametrize("name", sorted(set(CALLS) - {"bwd_noalloc", "delta"}))
def test_captured_on_a_stream_that_joins_the_capture(inputs, name):
    """A call on a second stream of a captured graph: its memory belongs to the graph and is right on replay."""
    names = ("table", "lens", "refs")
    own = dict(inputs, **dict(zip(names, _state(inputs))))
    out = CALLS[name](own, None)
    torch.cuda.synchronize()
    want = [t.clone() for t in (*out, *(own[n] for n in names))]
    del out
    s = torch.cuda.Stream()
    CALLS[name](dict(inputs, **dict(zip(names, _state(inputs)))), s)            # first use, outside of the capture
    own = dict(inputs, **dict(zip(names, _state(inputs))))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        for n in names:
            own[n].copy_(inputs[n])
        s.wait_stream(torch.cuda.current_stream())
        out = CALLS[name](own, s)
        torch.cuda.current_stream().wait_stream(s)
        got = [t.clone() for t in (*out, *(own[n] for n in names))]
        del out
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            if name.startswith("bwd") and i == 0:   # dq: one bf16 step, as above
                assert float((a.float() - b.float()).abs().max()) <= 2 ** -7 * float(b.abs().max())
            else:
                assert torch.equal(a, b), (name, i)
