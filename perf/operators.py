"""Cases, inputs and plain forms of the streaming and paged-cache operators, for measurements.

Three families, each used next to what the library already does for a causal model:

  sinks     training attention with a sliding window and a few first tokens that stay visible:
            query i sees key j iff j <= i, j is in i's document (which starts at a_i), and
            i - j < W or j - a_i < S.  Forward (O, lse) or forward and backward (dQ, dK, dV).
  decode    attention of the newest tokens over a paged cache: one token, or a tree of drafted
            tokens given by each node's parent.  Node n of a sequence with L cached tokens stands
            at position p_n = L + depth(n); it sees the cached tokens and its own ancestors
            (itself included), under a window and sinks the tokens at a position x with
            p_n - x < W or x < S.  With "step" a pass is a whole speculative step of one layer:
            the drafts' rows go into the pages, the tree attends, the accepted path's rows move up.
  pages     the pages themselves: forking sequences (full pages shared, the last partial page
            copied to the lowest free page) and freeing them again; packing the pages in use into
            the lowest places.

`own = False` computes the plain forms with elementary torch operations in 32 bits;
`own = True` calls the library.
"""
import math
import random

import numpy as np
import torch

own = False


# ------------------------------------------------------------------------------------- cases
def _sinks(name, B, H, T, D, window, sinks, docs=False, fused=False, train=True):
    c = dict(kind="sinks", B=B, H=H, T=T, D=D, window=window, sinks=sinks, docs=docs, fused=fused, train=train)
    return dict(c, name=name) if name else c


def _decode(name, B, H, Hkv, D, N, ctx, page, window=0, sinks=0, step=False):
    c = dict(kind="decode", B=B, H=H, Hkv=Hkv, D=D, N=N, ctx=ctx, page=page, window=window, sinks=sinks, step=step)
    return dict(c, name=name) if name else c


def _pages(name, op, slots, Hkv, D, ctx, page, share):
    c = dict(kind="pages", op=op, slots=slots, Hkv=Hkv, D=D, ctx=ctx, page=page, share=share)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the character model's attention (6 heads of 64, 256 tokens), one row: latency
        _sinks("sinks-char", 1, 6, 256, 64, 64, 4),
        # a GPT-2 124M micro-batch, q, k, v read from the fused projection, O written token-major
        _sinks("sinks-gpt2", 8, 12, 1024, 64, 256, 4, fused=True),
        # the long-context workload's shape and window
        _sinks("sinks-long", 4, 6, 8192, 128, 1024, 4),
        # packed documents of an odd length, evaluation only
        _sinks("sinks-docs", 3, 5, 1777, 128, 300, 7, docs=True, train=False),
        # one token of one sequence, GPT-2 124M heads: the smallest serving call
        _decode("token-one", 1, 12, 12, 64, 1, 777, 64),
        # one token of each of 64 ragged sequences, small pages
        _decode("token-batch", 64, 12, 12, 64, 1, 1024, 16),
        # a speculative step with trees of 32 drafts over long contexts
        _decode("tree-step", 8, 6, 6, 128, 32, 8192, 64, step=True),
        # four query heads to a key head, window and sinks, a very long stream, an odd tree
        _decode("tree-window", 16, 24, 6, 128, 13, 32768, 128, window=4096, sinks=4),
        # beams of one prompt
        _pages("fork-beams", "fork", 16, 12, 64, 700, 64, 0.5),
        # 256 sequences in the cache, half of them forked at once
        _pages("fork-batch", "fork", 256, 12, 64, 1024, 64, 0.5),
        # a few sequences gone, pages packed
        _pages("compact-few", "compact", 16, 6, 64, 256, 16, 0.75),
        # a large pool with holes all over
        _pages("compact-batch", "compact", 256, 6, 128, 2048, 64, 0.5),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["sinks", "sinks", "decode", "decode", "pages"])
    if kind == "sinks":
        T, D, H = _log(rng, 16, 8192), rng.choice([64, 128]), rng.randint(1, 20)
        B = _log(rng, 1, 64)
        while B > 1 and B * H * T * T * D > 24 * 8192 * 8192 * 128 * 0.9:
            B -= 1
        while H > 1 and B * H * T * T * D > 24 * 8192 * 8192 * 128 * 0.9:
            H -= 1
        return _sinks(None, B, H, T, D, _log(rng, 8, 2048), _log(rng, 1, 128), docs=rng.random() < 0.4,
                      fused=rng.random() < 0.4, train=rng.random() < 0.7)
    if kind == "decode":
        Hkv, G, D = rng.choice([1, 2, 4, 6, 8, 12, 20]), rng.choice([1, 1, 1, 2, 3, 4, 8]), rng.choice([64, 128])
        N = rng.choice([1, 1, 1, rng.randint(2, 8), rng.randint(9, 64)])
        ctx, B = _log(rng, 1, 32768), _log(rng, 1, 96)
        while B > 1 and (B * Hkv * ctx * D > 16 * 6 * 32768 * 128 * 0.9 or B * Hkv * G * N * ctx > 2 ** 28):
            B = B * 7 // 8
        far = rng.random() < 0.4
        return _decode(None, B, Hkv * G, Hkv, D, N, ctx, rng.choice([16, 32, 64, 128]),
                       window=_log(rng, 1, 8192) if far else 0, sinks=rng.randint(0, 16) if far else 0,
                       step=N > 1 and rng.random() < 0.5)
    return _pages(None, rng.choice(["fork", "compact"]), _log(rng, 4, 200), rng.choice([1, 6, 12]),
                  rng.choice([64, 128]), _log(rng, 16, 1024), rng.choice([16, 32, 64]),
                  rng.choice([0.25, 0.5, 0.75]))


# ------------------------------------------------------------------------------------ inputs
def _doc_starts(c):
    """First position of each token's document, [B, T]: lengths uniform up to about a third of a row."""
    r = random.Random(31 * c["T"] + c["B"])
    rows = []
    for _ in range(c["B"]):
        row = []
        while len(row) < c["T"]:
            row += [len(row)] * min(r.randint(1, max(1, c["T"] // 3)), c["T"] - len(row))
        rows.append(row)
    return np.array(rows, dtype=np.int32)


def _lengths(c):
    """Cached tokens of each sequence, ragged; the first one is as long as the case says."""
    r = random.Random(17 * c["ctx"] + 3)
    n = c.get("B") or c["slots"]
    return [c["ctx"]] + [r.randint(max(1, c["ctx"] // 4), c["ctx"]) for _ in range(n - 1)]


def _trees(c, r):
    """Parents of each node (-1: the cached context), random trees in which a node's parent comes before it."""
    return [[-1] + [r.randint(max(-1, n - 6), n - 1) for n in range(1, c["N"])] for _ in range(c["B"])]


def _prepare_sinks(c, g):
    B, H, T, D = c["B"], c["H"], c["T"], c["D"]
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()  # noqa: E731
    s = {"c": c, "scale": 1 / math.sqrt(D), "doc": torch.from_numpy(_doc_starts(c)).cuda() if c["docs"] else None}
    if c["fused"]:
        s["q"], s["k"], s["v"] = rnd(B, T, 3, H, D).permute(2, 0, 3, 1, 4).unbind(0)
        s["do"] = rnd(B, T, H, D).transpose(1, 2)
    else:
        s["q"], s["k"], s["v"], s["do"] = (rnd(B, H, T, D) for _ in range(4))
    return s


def _prepare_decode(c, g, r):
    B, H, Hkv, D, N, page = c["B"], c["H"], c["Hkv"], c["D"], c["N"], c["page"]
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()  # noqa: E731
    lens = _lengths(c)
    slots = -(-(max(lens) + N) // page)
    table = np.full((B, slots), -1, dtype=np.int32)
    held = [-(-(n + N) // page) for n in lens]
    places = list(range(sum(held) + 3))  # a few pages stay unused
    r.shuffle(places)
    for b in range(B):
        table[b, :held[b]] = [places.pop() for _ in range(held[b])]
    pool = sum(held) + 3
    s = {"c": c, "scale": 1 / math.sqrt(D), "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
         "table": torch.from_numpy(table).cuda(), "q": rnd(B, H, N, D), "k_pages": rnd(pool, Hkv, page, D),
         "v_pages": rnd(pool, Hkv, page, D)}
    trees = _trees(c, r)
    s["parents"] = torch.tensor(trees, dtype=torch.int32, device="cuda") if N > 1 else None
    if c["step"]:
        s["k_new"], s["v_new"] = rnd(B, Hkv, N, D), rnd(B, Hkv, N, D)
        paths = []
        for t in trees:  # the path from the context to a random node is the one accepted
            n, path = r.randrange(N), []
            while n >= 0:
                path, n = [n] + path, t[n]
            paths.append(path)
        s["accepted"] = torch.tensor([p + [0] * (N - len(p)) for p in paths], dtype=torch.int32, device="cuda")
        s["n_accepted"] = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
    return s


def _prepare_pages(c, g, r):
    S, page = c["slots"], c["page"]
    lens, held = _lengths(c), []
    per = -(-c["ctx"] // page)
    table = np.full((S, per), -1, dtype=np.int32)
    keep = round(c["share"] * S)
    live = sorted(random.Random(S + c["ctx"]).sample(range(S), max(1, min(S - 1, keep))))  # by the case: sizes do not go by the seed
    if c["op"] == "fork":  # the slots that are not live are the empty ones that the forks go to
        pool = sum(-(-lens[s] // page) for s in live) + S + 3
        owners = live
    else:  # all slots were filled, then some were freed: holes all over
        pool = sum(-(-n // page) for n in lens)
        owners = range(S)
    places = list(range(pool))
    r.shuffle(places)
    refs = np.zeros(pool, dtype=np.int32)
    for s in owners:
        held = -(-lens[s] // page)
        mine = [places.pop() for _ in range(held)]
        if s in live:
            table[s, :held] = mine
            refs[mine] = 1
    lens = [n if s in live else 0 for s, n in enumerate(lens)]
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()  # noqa: E731
    s = {"c": c, "table": torch.from_numpy(table).cuda(), "refs": torch.from_numpy(refs).cuda(),
         "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
         "k_pages": rnd(pool, c["Hkv"], page, c["D"]), "v_pages": rnd(pool, c["Hkv"], page, c["D"])}
    if c["op"] == "fork":
        parents = [-1 if n in live else r.choice(live) for n in range(S)]
        s["parents"] = torch.tensor(parents, dtype=torch.int32, device="cuda")
        s["drop"] = (s["parents"] >= 0).int()
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["kind"] == "sinks":
        return _prepare_sinks(case, g)
    return (_prepare_decode if case["kind"] == "decode" else _prepare_pages)(case, g, random.Random(seed))


# -------------------------------------------------------------------------------- plain forms
def _sinks_plain(s):
    c = s["c"]
    T = c["T"]
    i = torch.arange(T, device="cuda", dtype=torch.int32)
    a = s["doc"][:, None, :, None] if s["doc"] is not None else 0
    qi, kj = i[:, None], i[None, :]
    near = (qi - kj < c["window"]) | (kj - a < c["sinks"])
    blocked = ~((kj <= qi) & (kj >= a) & near)
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    x = (q @ k.transpose(-1, -2)).mul_(s["scale"]).masked_fill_(blocked, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    lse = (m + z.log()).squeeze(-1)
    p.div_(z)
    o = p @ v
    if not c["train"]:
        return {"o": o.bfloat16(), "lse": lse}
    do = s["do"].float()
    dv = p.transpose(-1, -2) @ do
    delta = (do * o).sum(-1, keepdim=True)
    ds = (do @ v.transpose(-1, -2)).sub_(delta).mul_(p).mul_(s["scale"])
    dq, dk = ds @ k, ds.transpose(-1, -2) @ q
    return {"o": o.bfloat16(), "lse": lse, "dq": dq.bfloat16(), "dk": dk.bfloat16(), "dv": dv.bfloat16()}


def _places(s, at):
    """Page and row of positions `at` [B, n] of each sequence."""
    page = s["c"]["page"]
    return s["table"].long().gather(1, at // page).clamp(min=0), at % page


def _append_plain(s):
    n = torch.arange(s["c"]["N"], device="cuda")
    page, row = _places(s, s["lens"].long()[:, None] + n)
    s["k_pages"][page, :, row] = s["k_new"].transpose(1, 2)
    s["v_pages"][page, :, row] = s["v_new"].transpose(1, 2)


def _accept_plain(s):
    n = torch.arange(s["c"]["N"], device="cuda")
    page, row = _places(s, s["lens"].long()[:, None] + s["accepted"].long())
    k, v = s["k_pages"][page, :, row], s["v_pages"][page, :, row]
    page, row = _places(s, s["lens"].long()[:, None] + n)
    mine = n < s["n_accepted"][:, None]
    s["k_pages"][page[mine], :, row[mine]] = k[mine]
    s["v_pages"][page[mine], :, row[mine]] = v[mine]


def _attend_plain(s):
    c = s["c"]
    B, H, Hkv, N, D = c["B"], c["H"], c["Hkv"], c["N"], c["D"]
    t = torch.arange(s["table"].shape[1] * c["page"], device="cuda")
    page, row = _places(s, t.expand(B, -1))
    k, v = (s[n][page, :, row].permute(0, 2, 1, 3).float() for n in ("k_pages", "v_pages"))
    sees = torch.eye(N, device="cuda").expand(B, N, N)
    if s["parents"] is not None:
        up = (s["parents"][:, :, None] == torch.arange(N, device="cuda")).float()
        sees = torch.matrix_power(sees + up, N) > 0
    sees = sees.bool()
    depth = sees.sum(-1) - 1
    L = s["lens"].long()[:, None]
    d = t - L
    drafted = (d >= 0) & (d < N)
    d = d.clamp(0, N - 1)
    vis = torch.where(drafted[:, None], sees.gather(2, d[:, None].expand(B, N, -1)), (t < L)[:, None])
    if c["window"] > 0:
        x = torch.where(drafted, L + depth.gather(1, d), t)[:, None]
        vis = vis & (((L + depth)[:, :, None] - x < c["window"]) | (x < c["sinks"]))
    q = s["q"].float().view(B, Hkv, H // Hkv, N, D).flatten(2, 3)
    x = (q @ k.transpose(-1, -2)) * s["scale"]
    x = x.view(B, Hkv, H // Hkv, N, -1).masked_fill(~vis[:, None, None], -math.inf).view_as(x)
    m = x.amax(-1, keepdim=True)
    p = (x - m).exp()
    z = p.sum(-1, keepdim=True)
    o = ((p @ v) / z).view(B, H, N, D)
    return {"o": o.bfloat16(), "lse": (m + z.log()).view(B, H, N)}


def _fork_plain(s):
    table, lens, refs, page = s["table"], s["lens"], s["refs"], s["c"]["page"]
    src = s["parents"].long().clamp(min=0)
    asked = s["parents"] >= 0
    n = torch.where(asked, lens[src], 0)
    full = (n // page)[:, None]
    j = torch.arange(table.shape[1], device="cuda")
    rows = torch.where(asked[:, None] & (j < full), table[src], -1)
    partial = asked & (n % page > 0)
    old = table[src].gather(1, full.long().clamp(max=table.shape[1] - 1)).squeeze(1)
    free = torch.argsort((refs > 0).int(), stable=True)  # the free pages first, lowest first
    new = free[(partial.cumsum(0) - 1).clamp(min=0)].int()
    pairs = torch.where(partial[:, None], torch.stack([old, new], 1), -1)
    rows = torch.where(partial[:, None] & (j == full), new[:, None], rows)
    shared = torch.where(rows >= 0, rows, refs.numel()).long().flatten()
    refs += torch.zeros(refs.numel() + 1, dtype=torch.int32, device="cuda").index_add_(
        0, shared, torch.ones_like(shared, dtype=torch.int32))[:-1]
    table.copy_(torch.where(asked[:, None], rows, table))
    lens.copy_(torch.where(asked, n, lens))
    return asked.int(), pairs


def _free_plain(s):
    gone = s["drop"] > 0
    rows = torch.where(gone[:, None] & (s["table"] >= 0), s["table"], s["refs"].numel()).long().flatten()
    s["refs"] -= torch.zeros(s["refs"].numel() + 1, dtype=torch.int32, device="cuda").index_add_(
        0, rows, torch.ones_like(rows, dtype=torch.int32))[:-1]
    s["table"].masked_fill_(gone[:, None], -1)
    s["lens"].masked_fill_(gone, 0)


def _copy_plain(s, pairs):
    old, new = pairs[pairs[:, 0] >= 0].long().unbind(1)
    s["k_pages"][new] = s["k_pages"][old]
    s["v_pages"][new] = s["v_pages"][old]


def _compact_plain(s):
    table, refs = s["table"], s["refs"]
    P = refs.numel()
    p = torch.arange(P, device="cuda")
    live = refs > 0
    n = live.sum()
    late, hole = live & (p >= n), ~live & (p < n)
    moves = late.sum()
    olds = torch.argsort((~late).int(), stable=True)[: P // 2]  # the late pages first, lowest first
    news = torch.argsort((~hole).int(), stable=True)[: P // 2]
    valid = p[: P // 2] < moves
    pairs = torch.where(valid[:, None], torch.stack([olds, news], 1), -1).int()
    to = p.clone()
    to[olds] = torch.where(valid, news, to[olds])
    new_table = torch.where(table >= 0, to[table.long().clamp(min=0)], -1).int()
    new_refs = torch.zeros_like(refs)
    new_refs[to[live]] = refs[live]
    return new_table, new_refs, pairs, moves.int().view(1)


# ---------------------------------------------------------------------------------- the passes
def _run_sinks(s):
    if not own:
        return _sinks_plain(s)
    import causal_attention_sdpa_b200 as ga
    c = s["c"]
    B, H, T, D = c["B"], c["H"], c["T"], c["D"]
    how = dict(scale=s["scale"], window=c["window"], sinks=c["sinks"], doc_start=s["doc"])
    o = torch.empty_like(s["do"])
    o, lse = ga.gpt_attn_fwd_sinks(s["q"], s["k"], s["v"], o=o, **how)
    if not c["train"]:
        return {"o": o, "lse": lse}
    if "ws" not in s:
        s["ws"] = torch.empty(ga.gpt_attn_bwd_sinks_workspace_bytes(B, H, T, D, c["window"], c["sinks"]),
                              dtype=torch.uint8, device="cuda")
    d = [None] * 3
    if c["fused"]:
        d = torch.empty(B, T, 3, H, D, dtype=torch.bfloat16, device="cuda").permute(2, 0, 3, 1, 4).unbind(0)
    dq, dk, dv = ga.gpt_attn_bwd_sinks(s["q"], s["k"], s["v"], o, lse, s["do"], dq=d[0], dk=d[1], dv=d[2],
                                       workspace=s["ws"], **how)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _run_decode(s):
    c = s["c"]
    if own:
        import causal_attention_sdpa_b200 as ga
        cache = (s["k_pages"], s["v_pages"], s["table"], s["lens"])
        if "ws" not in s:
            s["ws"] = torch.empty(ga.gpt_attn_paged_decode_workspace_bytes(c["B"], c["H"], c["Hkv"], c["N"], c["D"]),
                                  dtype=torch.uint8, device="cuda")
    if c["step"]:
        ga.gpt_attn_paged_append(*cache, s["k_new"], s["v_new"]) if own else _append_plain(s)
    if own:
        o, lse = ga.gpt_attn_paged_decode(s["q"], *cache, parents=s["parents"], scale=s["scale"],
                                          window=c["window"], sinks=c["sinks"], workspace=s["ws"])
        out = {"o": o, "lse": lse}
    else:
        out = _attend_plain(s)
    if c["step"]:
        ga.gpt_attn_paged_accept(*cache, s["accepted"], s["n_accepted"]) if own else _accept_plain(s)
        out |= {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    return out


def _run_pages(s):
    c = s["c"]
    if own:
        import causal_attention_sdpa_b200 as ga
        if "ws" not in s:
            s["ws"] = torch.empty(ga.gpt_attn_pages_workspace_bytes(*s["table"].shape, s["refs"].numel()),
                                  dtype=torch.uint8, device="cuda")
    pools = {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if c["op"] == "fork":
        if own:
            status, pairs = ga.gpt_attn_pages_fork(s["table"], s["lens"], s["refs"], c["page"], s["parents"],
                                                   workspace=s["ws"])
            ga.gpt_attn_pages_copy(s["k_pages"], s["v_pages"], pairs)
        else:
            status, pairs = _fork_plain(s)
            _copy_plain(s, pairs)
        table, refs, lens = s["table"].clone(), s["refs"].clone(), s["lens"].clone()
        ga.gpt_attn_pages_free(s["table"], s["lens"], s["refs"], s["drop"]) if own else _free_plain(s)
        return {"status": status, "pairs": pairs, "forked": (table, refs, lens),
                "freed": (s["table"], s["refs"], s["lens"])} | pools
    if own:
        table, refs, pairs, moves = ga.gpt_attn_pages_compact(s["table"], s["refs"], workspace=s["ws"])
        ga.gpt_attn_pages_copy(s["k_pages"], s["v_pages"], pairs, n_pairs=moves)
    else:
        table, refs, pairs, moves = _compact_plain(s)
        _copy_plain(s, pairs)
    return {"table": table, "refs": refs, "pairs": pairs, "moves": moves} | pools


def run(state):
    return {"sinks": _run_sinks, "decode": _run_decode, "pages": _run_pages}[state["c"]["kind"]](state)


# ---------------------------------------------------------------------- what a pass cannot do without
def _work_sinks(c):
    B, H, T, D = c["B"], c["H"], c["T"], c["D"]
    i = np.arange(T, dtype=np.int64)
    a = _doc_starts(c).astype(np.int64) if c["docs"] else np.zeros((B, 1), dtype=np.int64)
    span = i - a + 1
    pairs = H * int(np.minimum(span, np.minimum(span, c["window"]) + c["sinks"]).sum())
    rows = B * H * T
    if c["train"]:
        return {"bytes": rows * (4 * D * 2 + 4 * D * 2 + 4), "flops": 14 * D * pairs}
    return {"bytes": rows * (3 * D * 2 + D * 2 + 4), "flops": 4 * D * pairs}


def _work_decode(c):
    B, H, Hkv, D, N = c["B"], c["H"], c["Hkv"], c["D"], c["N"]
    seen = [min(n, c["window"] + c["sinks"]) if c["window"] > 0 else n for n in _lengths(c)]
    keys = sum(seen) + B * N
    b = keys * Hkv * D * 4 + B * H * N * (4 * D + 4)
    if c["step"]:  # the drafts' rows are read and written; the few that move up are not counted
        b += B * N * Hkv * D * 8
    return {"bytes": b, "flops": 4 * D * H * N * (sum(seen) + B * N / 2)}


def _work_pages(c):
    S, page = c["slots"], c["page"]
    held = [-(-n // page) for n in _lengths(c)]
    meta = 4 * (S * -(-c["ctx"] // page) + sum(held))
    live = c["share"] * sum(held)
    if c["op"] == "fork":  # one partial page to a fork, nearly always
        moved = round((1 - c["share"]) * S)
        meta *= 4
    else:  # live pages whose place is past the last one that stays
        moved = (1 - c["share"]) * live
        meta *= 2
    return {"bytes": meta + moved * c["Hkv"] * page * c["D"] * 2 * 2 * 2, "flops": 0}


def work(case):
    return {"sinks": _work_sinks, "decode": _work_decode, "pages": _work_pages}[case["kind"]](case)


# ---------------------------------------------------------------------------- the definition in 64 bits
def _exact_sinks(c, s):
    """Head by head: the masked softmax in 64 bits, its gradients by automatic differentiation."""
    B, H, T = c["B"], c["H"], c["T"]
    names = ("o", "lse", "dq", "dk", "dv") if c["train"] else ("o", "lse")
    out = {n: torch.empty((B, H, T) if n == "lse" else (B, H, T, c["D"]), dtype=torch.float64, device="cuda")
           for n in names}
    starts = _doc_starts(c) if c["docs"] else np.zeros((B, T), dtype=np.int32)
    for b in range(B):
        first = torch.tensor(starts[b], device="cuda").long()
        pos = torch.arange(T, device="cuda") - first
        away = torch.arange(T, device="cuda")[:, None] - torch.arange(T, device="cuda")[None]
        ok = (away >= 0) & (first[:, None] == first[None]) & ((away < c["window"]) | (pos[None] < c["sinks"]))
        for h in range(H):
            q, k, v = (s[n][b, h].double().requires_grad_() for n in ("q", "k", "v"))
            x = torch.where(ok, q @ k.T * s["scale"], -math.inf)
            lse = torch.logsumexp(x, -1)
            o = torch.exp(x - lse[:, None]) @ v
            out["o"][b, h], out["lse"][b, h] = o.detach(), lse.detach()
            if c["train"]:
                grads = torch.autograd.grad(o, (q, k, v), s["do"][b, h].double())
                out["dq"][b, h], out["dk"][b, h], out["dv"][b, h] = grads
    return out


def _exact_decode(c, s):
    """Sequence by sequence over its rows in order, the visible tokens of each node as a list."""
    B, H, Hkv, N, page = c["B"], c["H"], c["Hkv"], c["N"], c["page"]
    o = torch.empty((B, H, N, c["D"]), dtype=torch.float64, device="cuda")
    lse = torch.empty((B, H, N), dtype=torch.float64, device="cuda")
    parents = s["parents"].tolist() if s["parents"] is not None else [[-1]] * B
    table, lens = s["table"].tolist(), s["lens"].tolist()
    for b in range(B):
        L = lens[b]
        mine = table[b][: -(-(L + N) // page)]
        k, v = (s[n][mine].transpose(0, 1).flatten(1, 2)[:, : L + N].double() for n in ("k_pages", "v_pages"))
        if c["step"]:
            k[:, L:], v[:, L:] = s["k_new"][b].double(), s["v_new"][b].double()
        chains = []
        for n in range(N):
            chains.append((chains[parents[b][n]] if parents[b][n] >= 0 else []) + [n])
        for n in range(N):
            at = L + len(chains[n]) - 1
            pos = torch.cat([torch.arange(L), torch.arange(L, at + 1)]).cuda()
            ids = torch.tensor(list(range(L)) + [L + x for x in chains[n]], device="cuda")
            if c["window"] > 0:
                ids = ids[(pos > at - c["window"]) | (pos < c["sinks"])]
            kk = k[:, ids].repeat_interleave(H // Hkv, 0)
            vv = v[:, ids].repeat_interleave(H // Hkv, 0)
            x = (kk @ s["q"][b, :, n].double()[:, :, None]).squeeze(-1) * s["scale"]
            lse[b, :, n] = torch.logsumexp(x, -1)
            o[b, :, n] = (torch.softmax(x, -1)[:, None] @ vv).squeeze(1)
    out = {"o": o, "lse": lse}
    return out | {"k_pages": None, "v_pages": None} if c["step"] else out


def exact(case, seed):
    if case["kind"] == "pages":
        return None  # copied values and whole numbers: nothing is computed
    s = prepare(case, seed)
    return (_exact_sinks if case["kind"] == "sinks" else _exact_decode)(case, s)
