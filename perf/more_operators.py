"""What stands round the products of a decoder layer, and beams over shared pages, as cases that can be timed.

    norm      the norm after a block, its gate and the residual add, and the norm before the next block, in one
    route     the router's choice: scores, a bias for balance, groups, top-k and its weights, as the expert products
              take them
    beam      the best continuations over beams and vocabulary
    reorder   the cache's sequences become copies of those that their beams continue
    shared    attention of a batch whose sequences share the first pages of the paged 8-bit cache

`own` selects the side: False computes in elementary torch operations, True calls the package.
"""
import math

import torch

own = False

BLOCK = 64        # tokens in a page of the cache, and in the block that shares a scale


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # between two blocks of one decode step, norms on both sides: latency
        dict(name="norm-step", op="norm", rows=1, n=3840, x="f32", y="f32", post=True, gate="none", scale=1.0,
             residual=1.0, offset=1.0),
        # a prompt batch through the same place, with a gate for each channel and a scaled residual
        dict(name="norm-prompt", op="norm", rows=8191, n=3840, x="f32", y="f32", post=True, gate="channel", scale=0.5,
             residual=0.9, offset=0.0),
        # one token's top 8 of 128 experts: latency
        dict(name="route-step", op="route", tokens=1, experts=128, topk=8, logits="f32", score="softmax", bias=False,
             groups=1, group_topk=1, group_best=1, renorm=True, scale=1.0),
        # a prompt batch over 256 experts in 8 groups of which 4 stay, scores of their own with a bias for balance
        dict(name="route-prompt", op="route", tokens=8201, experts=256, topk=8, logits="f32", score="sigmoid",
             bias=True, groups=8, group_topk=4, group_best=2, renorm=True, scale=2.5),
        # the first step of four beams: one of them lives, the others have no score yet
        dict(name="beam-first", op="beam", batch=1, beams=4, vocab=128256, n=8, logits="bf16", dead=3, ended=0),
        # a step of a serving batch in the middle of its beams, some of them at their end
        dict(name="beam-batch", op="beam", batch=24, beams=8, vocab=262144, n=8, logits="bf16", dead=0, ended=1),
        # an odd vocabulary in 32 bits, twice as many candidates as beams
        dict(name="beam-wide", op="beam", batch=6, beams=5, vocab=50257, n=10, logits="f32", dead=0, ended=0),
        # four beams of one request in their own slots
        dict(name="reorder-step", op="reorder", groups=1, beams=4, held=1000, width=64, place="same"),
        # a serving batch with room for 64 thousand tokens each, into the other half of the slots
        dict(name="reorder-batch", op="reorder", groups=40, beams=8, held=30011, width=1024, place="other"),
        # sixteen samples of one prompt, one step
        dict(name="shared-step", op="shared", groups=1, each=16, prefix=4003, tail=150, new=1, idle=0, q_heads=24,
             kv_heads=8, dim=128),
        # a serving step: five prompts of up to 20000 tokens with 24 continuations each, wide heads
        dict(name="shared-batch", op="shared", groups=5, each=24, prefix=20011, tail=600, new=1, idle=1, q_heads=16,
             kv_heads=8, dim=256),
        # questions of up to 512 tokens behind one long document
        dict(name="shared-prompt", op="shared", groups=1, each=6, prefix=12040, tail=0, new=512, idle=0, q_heads=24,
             kv_heads=8, dim=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "route", "route", "beam", "beam", "reorder", "shared", "shared", "shared"])
    if op == "norm":
        n = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            n = -(-n // 64) * 64
        rows = _log(rng, 1, max(1, 8191 * 3840 // n))
        return dict(op="norm", rows=min(rows, 60000), n=n, x=rng.choice(["f32", "f32", "bf16"]),
                    y=rng.choice(["f32", "bf16"]), post=rng.random() < 0.6,
                    gate=rng.choice(["none", "none", "channel", "row"]), scale=rng.choice([1.0, 0.25, 1.4]),
                    residual=rng.choice([1.0, 1.0, 0.8]), offset=rng.choice([0.0, 1.0]))
    if op == "route":
        experts = rng.choice([8, 16, 60, 64, 128, 160, 256, 384])
        topk = min(experts // 2, rng.choice([1, 2, 4, 6, 8, 10]))
        groups = rng.choice([1, 1, 4, 8]) if experts % 8 == 0 and experts >= 64 else 1
        keep = groups if groups == 1 else rng.choice([groups // 2, groups - 1])
        while keep * (experts // groups) < topk:
            keep += 1
        return dict(op="route", tokens=_log(rng, 1, 8201 * 136 // (experts // 2 + topk)), experts=experts, topk=topk,
                    logits=rng.choice(["f32", "bf16"]), score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, group_topk=keep, group_best=rng.choice([1, 2]),
                    renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]))
    if op == "beam":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 16])
        vocab = rng.choice([32000, 50257, 100352, 128256, 151936, 262144, _log(rng, 1000, 200000)])
        kind = rng.choice(["first", "mid", "mid", "ended"])
        batch = _log(rng, 1, max(1, 24 * 8 * 262144 // 2 // (beams * vocab)))
        return dict(op="beam", batch=batch, beams=beams, vocab=vocab, n=beams if kind == "ended" else 2 * beams,
                    logits=rng.choice(["f32", "bf16"]), dead=beams - 1 if kind == "first" else 0,
                    ended=1 if kind == "ended" and beams > 1 else 0)
    if op == "reorder":
        beams = rng.choice([2, 3, 4, 5, 8, 16])
        width = _log(rng, 4, 1024)
        return dict(op="reorder", groups=_log(rng, 1, 320 // beams), beams=beams,
                    held=_log(rng, 1, (width - 1) * BLOCK), width=width, place=rng.choice(["same", "other"]))
    dim = rng.choice([64, 128, 256])
    q_heads, kv_heads = rng.choice([(24, 8), (16, 8), (32, 8), (8, 8), (12, 1)])
    groups = rng.choice([1, 1, 2, 5])
    form = rng.choice(["step", "step", "verify", "prompt"])
    if form == "prompt":
        each, new, prefix, tail = rng.randint(2, 4), _log(rng, 13, 400), _log(rng, 64, 5000), _log(rng, 1, 200)
        groups = min(groups, 2)
    else:
        each = _log(rng, 2, 48)
        new = 1 if form == "step" else rng.randint(2, 6)
        prefix, tail = _log(rng, 40, 20000), _log(rng, 1, 1200)
    return dict(op="shared", groups=groups, each=each, prefix=prefix, tail=tail, new=new,
                idle=rng.choice([0, 1]) if each > 3 else 0, q_heads=q_heads, kv_heads=kv_heads, dim=dim)


def _size(dtype):
    return 4 if dtype == "f32" else 2


def _type(dtype):
    return torch.float32 if dtype == "f32" else torch.bfloat16


def _pages(tokens):
    return -(-tokens // BLOCK)


def _shape(case):
    """Of a shared case: tokens of each group's prefix, and (own tokens behind the shared pages, new rows) of every
    sequence, group by group.  The first group has the case's own numbers, the others less; the last `idle` sequences
    of a group hold nothing (their row stays, and sees nothing)."""
    prefix, seqs = [], []
    for g in range(case["groups"]):
        f = 1.0 if g == 0 else 0.3 + 0.7 * ((g * 0.6180339887498949) % 1.0)
        prefix.append(max(1, int(case["prefix"] * f)))
        row = []
        for b in range(case["each"]):
            f = 1.0 if b == 0 else 0.25 + 0.75 * (((g + b) * 0.6180339887498949) % 1.0)
            new = max(1, int(case["new"] * f))
            row.append((prefix[g] % BLOCK + int(case["tail"] * f) + new, new))
        for b in range(case["each"] - case["idle"], case["each"]):
            row[b] = (0, 1)
        seqs.append(row)
    return prefix, seqs


def work(case):
    op = case["op"]
    if op == "norm":
        e = case["rows"] * case["n"]
        per = 2 * _size(case["x"]) + _size(case["y"]) + 2 + (2 if case["gate"] == "row" else 0)
        vectors = (1 + case["post"] + (case["gate"] == "channel")) * 2 * case["n"]
        return {"bytes": e * per + vectors, "flops": 12 * e}
    if op == "route":
        e = case["tokens"] * case["experts"]
        return {"bytes": e * _size(case["logits"]) + 8 * case["tokens"] * case["topk"] + 4 * case["experts"] * case["bias"],
                "flops": 6 * e}
    if op == "beam":
        rows = case["batch"] * (case["beams"] - max(case["dead"], case["ended"]))
        return {"bytes": rows * case["vocab"] * _size(case["logits"]) + 12 * case["batch"] * case["n"],
                "flops": 4 * rows * case["vocab"]}
    if op == "reorder":
        n = case["groups"] * case["beams"]
        return {"bytes": 8 * n * case["width"] + 16 * n + 4 * n * _pages(case["held"]), "flops": 0}
    prefix, seqs = _shape(case)
    row = case["kv_heads"] * case["dim"]
    nbytes = flops = 0
    for p, group in zip(prefix, seqs):
        pages, rows = p // BLOCK, 0
        for own_tokens, new in group:
            rows += new if own_tokens else 0
            nbytes += own_tokens * row * 2 + 8 * _pages(own_tokens) * case["kv_heads"]
            nbytes += 4 * new * case["q_heads"] * case["dim"]
            seen = sum(own_tokens - new + 1 + i for i in range(new)) if own_tokens else 0
            flops += 4 * seen * case["q_heads"] * case["dim"]
        nbytes += pages * (BLOCK * row * 2 + 8 * case["kv_heads"])
        flops += 4 * rows * pages * BLOCK * case["q_heads"] * case["dim"]
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed(seed * 1000003 + salt)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _norm_inputs(case, seed):
    """A residual stream with a few large channels, a block's output, and weights as training leaves them."""
    g = _gen(seed, 11)
    rows, n = case["rows"], case["n"]
    x = _normal(g, rows, n)
    x *= torch.where(torch.rand(n, generator=g, device="cuda") < 0.01, 30.0, 1.0) * torch.exp(0.5 * _normal(g, rows, 1))
    y = _normal(g, rows, n).mul_(torch.exp(0.7 * _normal(g, n)))
    weight = lambda: (1.0 - case["offset"] + 0.3 * _normal(g, n)).to(torch.bfloat16)
    d = dict(x=x.to(_type(case["x"])), y=y.to(_type(case["y"])), pre=weight(),
             post=weight() if case["post"] else None, gate=None)
    if case["gate"] == "channel":
        d["gate"] = _normal(g, n).to(torch.bfloat16)
    elif case["gate"] == "row":
        d["gate"] = _normal(g, rows, n).to(torch.bfloat16)
    return d


def _route_inputs(case, seed):
    """Logits of a router: some experts are liked more than others by every token."""
    g = _gen(seed, 12)
    logits = 1.3 * _normal(g, case["tokens"], case["experts"]) + 0.5 * _normal(g, case["experts"])
    bias = 0.05 * _normal(g, case["experts"]) if case["bias"] else None
    return logits.to(_type(case["logits"])), bias


def _beam_inputs(case, seed):
    """Logits of a language model: a broad bulk, and for each row some tokens far above it."""
    g = _gen(seed, 13)
    rows, vocab = case["batch"] * case["beams"], case["vocab"]
    logits = _normal(g, rows, vocab).mul_(2.0)
    up = torch.randint(0, vocab, (rows, 40), generator=g, device="cuda")
    logits.scatter_add_(1, up, 6.0 + 4.0 * torch.rand(rows, 40, generator=g, device="cuda"))
    scores = -20.0 + 6.0 * torch.rand(case["batch"], case["beams"], generator=g, device="cuda")
    if case["dead"]:
        scores[:, case["beams"] - case["dead"]:] = -math.inf
    done = None
    if case["ended"]:
        done = torch.zeros(case["batch"], case["beams"], dtype=torch.uint8, device="cuda")
        done.scatter_(1, torch.randint(0, case["beams"], (case["batch"], case["ended"]), generator=g, device="cuda"), 1)
    return logits.to(_type(case["logits"])), scores, done, 2 if case["ended"] else -1


def _reorder_inputs(case, seed):
    """Tables whose beams share their first pages, lens, refs, and parents.  In their own slots the beams that go on
    stay where they are and the others become copies of them; into other slots parents are free."""
    g = torch.Generator().manual_seed(seed * 7919 + 14)
    groups, beams, width = case["groups"], case["beams"], case["width"]
    slots = groups * beams * (2 if case["place"] == "other" else 1)
    perm = torch.randperm(slots, generator=g)
    seqs = perm[:groups * beams].view(groups, beams)
    dst = perm[groups * beams:].view(groups, beams) if case["place"] == "other" else seqs
    table = torch.full((slots, width), -1, dtype=torch.int32)
    lens = torch.zeros(slots, dtype=torch.int32)
    used = _pages(case["held"])
    common = used * 3 // 4
    pages = groups * (common + beams * (used - common)) + 3
    numbers = torch.randperm(pages, generator=g).to(torch.int32)
    at = 0
    for r in range(groups):
        first = numbers[at:at + common]
        at += common
        for b in range(beams):
            table[seqs[r, b], :common] = first
            table[seqs[r, b], common:used] = numbers[at:at + used - common]
            at += used - common
            lens[seqs[r, b]] = case["held"] - (b % 3 if case["held"] > 64 and case["held"] % 64 > 3 else 0)
    refs = torch.zeros(pages, dtype=torch.int32)
    flat = table[table >= 0].long()
    refs.index_add_(0, flat, torch.ones(len(flat), dtype=torch.int32))
    parent = torch.randint(0, beams, (groups, beams), generator=g)
    if case["place"] == "same":
        goes_on = torch.zeros(groups, beams, dtype=torch.bool).scatter_(1, parent, True)
        parent = torch.where(goes_on, torch.arange(beams).expand(groups, beams), parent)
    return pages, table, lens, refs, seqs.to(torch.int32), dst.to(torch.int32), parent.to(torch.int32)


def _rows(g, tokens, heads, dim, spread):
    """Rows as a projection gives them: heads and channels of their own size, a few channels far larger, and tokens
    that differ in size."""
    ch = torch.exp(0.4 * _normal(g, heads, dim))
    ch = torch.where(torch.rand(heads, dim, generator=g, device="cuda") < 0.02, ch * spread, ch)
    return _normal(g, tokens, heads, dim) * ch * torch.exp(0.3 * _normal(g, tokens, 1, 1))


def _held(x):
    """Rows of one sequence from a page's beginning on as e4m3 codes [pages, 64, heads, dim] and the smallest
    power-of-two scale [pages, heads] that holds each block."""
    n = x.shape[0]
    pad = torch.zeros((_pages(n) * BLOCK, *x.shape[1:]), device="cuda")
    pad[:n] = x
    pad = pad.view(-1, BLOCK, *x.shape[1:])
    m, e = torch.frexp(pad.abs().amax(dim=(1, 3)))
    scale = torch.exp2(torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-100).float())   # 448 = 0.875 * 2^9
    return (pad / scale[:, None, :, None]).to(torch.float8_e4m3fn), scale


def _shared_inputs(case, seed):
    """q, and per side (keys, values) the held blocks of each group's shared pages and of each sequence's own."""
    prefix, seqs = _shape(case)
    g = _gen(seed, 15)
    rows = sum(new for group in seqs for _, new in group)
    q = (0.8 * _normal(g, rows, case["q_heads"], case["dim"])).to(torch.bfloat16)
    common, private = [], []
    for p, group in zip(prefix, seqs):
        common.append([_held(_rows(g, p // BLOCK * BLOCK, case["kv_heads"], case["dim"], s)) for s in (5.0, 2.0)])
        tokens = sum(t for t, _ in group)
        both = [_rows(g, tokens, case["kv_heads"], case["dim"], s) for s in (5.0, 2.0)]
        at = 0
        for t, _ in group:
            private.append([_held(x[at:at + t]) for x in both])
            at += t
    return q, common, private


def _values(held, tokens):
    """The values that held blocks stand for, float32 [tokens, heads, dim]."""
    codes, scale = held
    return (codes.float() * scale[:, None, :, None]).flatten(0, 1)[:tokens]


def prepare(case, seed):
    st = dict(case=case)
    op = case["op"]
    if op == "norm":
        st.update(_norm_inputs(case, seed))
    elif op == "route":
        st["logits"], st["bias"] = _route_inputs(case, seed)
    elif op == "beam":
        st["logits"], st["scores"], st["done"], st["eos"] = _beam_inputs(case, seed)
        if own:
            import decode_gemv_tensor_gb300 as dgt
            st["ws"] = dgt.beam_workspace(case["batch"], case["beams"], case["vocab"], case["n"])
    elif op == "reorder":
        pages, table, lens, refs, seqs, dst, parent = _reorder_inputs(case, seed)
        st.update(seqs=seqs.cuda(), dst=dst.cuda(), parent=parent.cuda())
        if own:
            import decode_gemv_tensor_gb300 as dgt
            cache = dgt.KvCache(1, pages, 1, 64, max_seqs=table.shape[0], max_pages=table.shape[1])
            for x, y in ((cache.table, table), (cache.lens, lens), (cache.refs, refs)):
                x.copy_(y)
            st["cache"] = cache
        else:
            st.update(table=table.cuda(), lens=lens.cuda(), refs=refs.cuda())
    else:
        _prepare_shared(st, seed)
    return st


def _prepare_shared(st, seed):
    case = st["case"]
    prefix, seqs = _shape(case)
    q, common, private = _shared_inputs(case, seed)
    st.update(q=q, prefix=prefix, seqs=seqs)
    if not own:
        st.update(common=common, private=private)
        return
    import decode_gemv_tensor_gb300 as dgt
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    flat = [s for group in seqs for s in group]
    width = max(p // BLOCK + _pages(t) for p, group in zip(prefix, seqs) for t, _ in group) + 1
    pages = sum(_pages(p) for p in prefix) + sum(_pages(t) for t, _ in flat) + 4
    groups, each = case["groups"], case["each"]
    cache = dgt.KvCache(1, pages, case["kv_heads"], case["dim"], max_seqs=groups * (each + 1), max_pages=width)
    # slots 0..groups-1 hold the prompts, those behind them the continuations
    parents = i32(list(range(groups)))
    dgt.kv_reserve(cache, parents, i32(prefix))
    for g, p in enumerate(prefix):
        if p >= BLOCK:
            k, v = (_values(x, p // BLOCK * BLOCK).to(torch.bfloat16) for x in common[g])
            dgt.kv_append(cache, 0, k, v, i32([g]), i32([0]), cu=i32([0, len(k)]))
        for b in range(each):
            at = g * each + b
            t = flat[at][0]
            if t:
                slot = i32([groups + at])
                dgt.kv_fork(cache, i32([g]), slot)
                dgt.kv_reserve(cache, slot, i32([t - p % BLOCK]))
                k, v = (_values(x, t).to(torch.bfloat16) for x in private[at])
                dgt.kv_append(cache, 0, k, v, slot, i32([p // BLOCK * BLOCK]), cu=i32([0, t]))
    cu = [0]
    for _, new in flat:
        cu.append(cu[-1] + new)
    st.update(cache=cache, parents=parents, slots=i32([groups + i for i in range(len(flat))]), shared=i32(prefix),
              groups=i32([g * each for g in range(groups + 1)]), cu=None if cu[-1] == len(flat) else i32(cu))
    st["ws"] = dgt.kv_attention_shared_workspace(cache, case["q_heads"], groups, len(flat), cu[-1])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    return (_own if own else _plain)[st["case"]["op"]](st)


def _own_norm(st):
    import decode_gemv_tensor_gb300 as dgt
    c = st["case"]
    return dgt.block_norm(st["x"], st["y"], pre=st["pre"], post=st["post"], gate=st["gate"], scale=c["scale"],
                          residual=c["residual"], offset=c["offset"], eps=1e-6)


def _own_route(st):
    import decode_gemv_tensor_gb300 as dgt
    c = st["case"]
    return dgt.route(st["logits"], c["topk"], score=c["score"], bias=st["bias"], groups=c["groups"],
                     group_topk=c["group_topk"], group_best=c["group_best"], renorm=c["renorm"], scale=c["scale"])


def _own_beam(st):
    import decode_gemv_tensor_gb300 as dgt
    return dgt.beam_select(st["logits"], st["scores"], st["case"]["n"], eos=st["eos"], done=st["done"], ws=st["ws"])


def _own_reorder(st):
    import decode_gemv_tensor_gb300 as dgt
    cache = st["cache"]
    dgt.kv_reorder(cache, st["seqs"], st["parent"], dst=st["dst"])
    return [cache.table, cache.lens, cache.refs]


def _own_shared(st):
    import decode_gemv_tensor_gb300 as dgt
    return dgt.kv_attention_shared(st["cache"], 0, st["q"], st["slots"], st["parents"], st["shared"],
                                   groups=st["groups"], cu=st["cu"], ws=st["ws"])


def _plain_norm(st):
    c = st["case"]

    def normed(u, w):
        return u * torch.rsqrt((u * u).mean(-1, keepdim=True) + 1e-6) * (c["offset"] + w.float())

    u = st["y"].float()
    if st["post"] is not None:
        u = normed(u, st["post"])
    if st["gate"] is not None:
        u = u * st["gate"].float()
    x = c["residual"] * st["x"].float() + c["scale"] * u
    return [x.to(st["x"].dtype), normed(x, st["pre"]).to(torch.bfloat16)]


def _best_first(x):
    """Indices in descending order, the lowest first among equals."""
    return torch.sort(x, dim=-1, descending=True, stable=True)[1]


def _plain_route(st):
    # 64 bits: a choice next to its border decides which expert is taken
    c = st["case"]
    x = st["logits"].double()
    if c["score"] == "softmax":
        e = torch.exp(x - x.amax(-1, keepdim=True))
        s = e / e.sum(-1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-x))
    choice = x if st["bias"] is None else s + st["bias"].double()
    if c["groups"] > 1:
        per = c["experts"] // c["groups"]
        by = (s if st["bias"] is None else choice).view(-1, c["groups"], per)
        by = by.topk(min(per, c["group_best"]), dim=-1)[0].sum(-1)
        keep = torch.zeros_like(by, dtype=torch.bool)
        keep.scatter_(1, _best_first(by)[:, :c["group_topk"]], True)
        choice = torch.where(keep.repeat_interleave(per, 1), choice, -math.inf)
    ids = _best_first(choice)[:, :c["topk"]]
    p = s.gather(1, ids)
    if c["renorm"]:
        p = p / p.sum(-1, keepdim=True)
    return [ids.int(), (p * c["scale"]).float()]


def _plain_beam(st):
    c = st["case"]
    rows, vocab, n = c["batch"] * c["beams"], c["vocab"], c["n"]
    x = st["logits"].float() + 0.0
    top = x.amax(-1, keepdim=True)
    # 64 bits: the sums decide between candidates of different beams
    lse = top.double() + torch.log(torch.exp((x - top).double()).sum(-1, keepdim=True))
    # one whole number for each candidate of a beam: its logit's order, then the lowest token first
    bits = x.view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    key = order * 2 ** 32 + (2 ** 32 - 1 - torch.arange(vocab, device="cuda"))
    token = 2 ** 32 - 1 - (key.topk(n, dim=-1)[0] & (2 ** 32 - 1))
    total = st["scores"].double().view(rows, 1) + (x.gather(1, token).double() - lse)
    if st["done"] is not None:
        done = st["done"].view(rows, 1) != 0
        first = torch.arange(n, device="cuda") == 0
        total = torch.where(done, torch.where(first, st["scores"].double().view(rows, 1), -math.inf), total)
        token = torch.where(done, st["eos"], token)
    total, token = total.view(c["batch"], -1), token.view(c["batch"], -1)
    pick = _best_first(total)[:, :n]
    out = [(pick // n).int(), token.gather(1, pick).int(), total.gather(1, pick).float()]
    if st["done"] is not None:
        out.append(((st["done"].gather(1, pick // n) != 0) | (out[1] == st["eos"])).to(torch.uint8))
    return out


def _plain_reorder(st):
    table, lens, refs = st["table"], st["lens"], st["refs"]
    src = st["seqs"].gather(1, st["parent"].long()).flatten().long()
    dst = st["dst"].flatten().long()
    for rows, sign in ((table[dst], -1), (table[src], 1)):
        pages = rows.flatten().long()
        refs.index_add_(0, pages.clamp(min=0), torch.where(pages >= 0, sign, 0).int())
    table[dst], lens[dst] = table[src], lens[src]
    return [table, lens, refs]


def _plain_shared(st):
    c = st["case"]
    hk, d = c["kv_heads"], c["dim"]
    group = c["q_heads"] // hk
    out, at, seq = [], 0, 0
    for g, p in enumerate(st["prefix"]):
        kp, vp = (_values(x, p // BLOCK * BLOCK) for x in st["common"][g])
        for t, n in st["seqs"][g]:
            q = st["q"][at:at + n].float()
            at += n
            if t == 0:
                out.append(torch.zeros_like(q))
                seq += 1
                continue
            k, v = (torch.cat([a, _values(b, t)]) for a, b in zip((kp, vp), st["private"][seq]))
            seq += 1
            q = q.view(n, hk, group, d).permute(1, 2, 0, 3)               # [hk, group, n, d]
            s = torch.matmul(q, k.permute(1, 2, 0)[:, None]) * (1.0 / math.sqrt(d))
            if n > 1:
                total = k.shape[0]
                ahead = torch.arange(total, device="cuda") > torch.arange(total - n, total, device="cuda")[:, None]
                s = torch.where(ahead, -math.inf, s)
            e = torch.exp(s - s.amax(-1, keepdim=True))
            y = torch.matmul(e, v.permute(1, 0, 2)[:, None]) / e.sum(-1, keepdim=True)
            out.append(y.permute(2, 0, 1, 3).reshape(n, c["q_heads"], d))
    return torch.cat(out).to(torch.bfloat16)


_own = dict(norm=_own_norm, route=_own_route, beam=_own_beam, reorder=_own_reorder, shared=_own_shared)
_plain = dict(norm=_plain_norm, route=_plain_route, beam=_plain_beam, reorder=_plain_reorder, shared=_plain_shared)


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    return dict(norm=_exact_norm, route=_exact_route, beam=_exact_beam, reorder=_exact_reorder,
                shared=_exact_shared)[case["op"]](case, seed)


def _exact_norm(case, seed):
    d = {k: None if v is None else v.double() for k, v in _norm_inputs(case, seed).items()}
    n = case["n"]
    u = d["y"]
    if case["post"]:
        u = u / torch.sqrt(torch.linalg.vecdot(u, u)[:, None] / n + 1e-6) * (d["post"] + case["offset"])
    if case["gate"] != "none":
        u = u * d["gate"]
    x = d["x"] * case["residual"] + u * case["scale"]
    return [x, x / torch.sqrt(torch.linalg.vecdot(x, x)[:, None] / n + 1e-6) * (d["pre"] + case["offset"])]


def _exact_route(case, seed):
    logits, bias = _route_inputs(case, seed)
    x = logits.double()
    s = torch.softmax(x, -1) if case["score"] == "softmax" else torch.sigmoid(x)
    experts, per = case["experts"], case["experts"] // case["groups"]
    rank = s + bias.double() if case["bias"] else s
    order = rank if case["bias"] else x
    open_ = torch.ones_like(x, dtype=torch.bool)
    if case["groups"] > 1:
        two = rank.view(-1, case["groups"], per).sort(-1)[0][..., -case["group_best"]:].sum(-1)
        left = two.clone()
        open_ = torch.zeros_like(open_)
        for _ in range(case["group_topk"]):
            best = left.amax(-1, keepdim=True)
            g = torch.where(left == best, torch.arange(case["groups"], device="cuda"), case["groups"]).amin(-1, keepdim=True)
            left.scatter_(1, g, -math.inf)
            open_ |= torch.arange(experts, device="cuda") // per == g
    order = torch.where(open_, order, -math.inf)
    ids = []
    for _ in range(case["topk"]):
        best = order.amax(-1, keepdim=True)
        i = torch.where(order == best, torch.arange(experts, device="cuda"), experts).amin(-1, keepdim=True)
        order = order.scatter(1, i, -math.inf)
        ids.append(i)
    ids = torch.cat(ids, 1)
    p = torch.take_along_dim(s, ids, 1)
    if case["renorm"]:
        p = p / p.sum(1, keepdim=True)
    return [ids.int(), p * case["scale"]]


def _exact_beam(case, seed):
    logits, scores, done, eos = _beam_inputs(case, seed)
    beams, vocab = case["beams"], case["vocab"]
    out = [[], [], [], []]
    for b in range(case["batch"]):
        x = logits[b * beams:(b + 1) * beams].double()
        total = scores[b].double()[:, None] + torch.log_softmax(x, -1)
        if case["ended"]:
            for i in torch.nonzero(done[b])[:, 0].tolist():
                total[i] = -math.inf
                total[i, eos] = scores[b, i].double()
        total = total.flatten()
        value = total.topk(case["n"])[0]
        at = torch.nonzero(total >= value[-1])[:, 0]                      # all that could be taken, lowest first
        at = at[torch.sort(total[at], descending=True, stable=True)[1]][:case["n"]]
        out[0].append(at // vocab)
        out[1].append(at % vocab)
        out[2].append(total[at])
        if case["ended"]:
            out[3].append((done[b][at // vocab] != 0) | (at % vocab == eos))
    types = (torch.int32, torch.int32, torch.float64, torch.uint8)
    return [torch.stack(x).to(t) for x, t in zip(out, types) if x]


def _exact_reorder(case, seed):
    pages, table, lens, refs, seqs, dst, parent = _reorder_inputs(case, seed)
    rows, length = table.tolist(), lens.tolist()
    new, new_length = [list(r) for r in rows], list(length)
    for s, d, p in zip(seqs.tolist(), dst.tolist(), parent.tolist()):
        for i, slot in enumerate(d):
            new[slot], new_length[slot] = rows[s[p[i]]], length[s[p[i]]]
    table = torch.tensor(new, dtype=torch.int32)
    count = torch.bincount(table[table >= 0].long(), minlength=pages)
    return [table.cuda(), torch.tensor(new_length, dtype=torch.int32).cuda(), count.int().cuda()]


def _exact_shared(case, seed):
    prefix, seqs = _shape(case)
    q, common, private = _shared_inputs(case, seed)
    q, group = q.double(), case["q_heads"] // case["kv_heads"]
    value = lambda held: torch.einsum("pthd,ph->pthd", held[0].double(), held[1].double()).flatten(0, 1)
    out = torch.zeros_like(q)
    at = seq = 0
    for g in range(case["groups"]):
        front = [value(x) for x in common[g]]
        for t, n in seqs[g]:
            rows = slice(at, at + n)
            at += n
            if t:
                k, v = (torch.cat([f, value(x)[:t]]) for f, x in zip(front, private[seq]))
                i = torch.arange(len(k) - n, len(k), device="cuda").view(-1, 1)
                hidden = torch.arange(len(k), device="cuda").view(1, -1) > i
                for h in range(case["q_heads"]):
                    w = q[rows, h] @ k[:, h // group].T / math.sqrt(case["dim"])
                    out[rows, h] = torch.softmax(w.masked_fill(hidden, -math.inf), -1) @ v[:, h // group]
            seq += 1
    return out
