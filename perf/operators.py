"""The serving operators between the products of a decoder layer, as cases that can be timed.

Four operators work on one store of keys and values, the paged 8-bit cache:

    rotate   rotary positions (one axis for text; time, height, width for images and video) on q and k
    append   new keys and values quantised into the cache: e4m3 codes, one power-of-two scale for each
             block of 64 tokens and head
    attend   attention over that cache, grouped-query, causal, optionally a sliding window with first
             tokens that stay visible
    pages    forking sequences, reserving their next pages (copy on write), copying and freeing pages

`own` selects the side: False computes in elementary torch operations, True calls the package.
"""
import math

import torch

own = False

BLOCK = 64        # tokens in a page, and in the block that shares a scale
E_MIN = -100      # smallest exponent of a scale (a block of zeros has it)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of the 24/8-head stack: latency, at a far position
        dict(name="rotate-step", op="rotate", tokens=1, q_heads=24, kv_heads=8, dim=128, rot=128, axes=1,
             interleaved=False, far=131071),
        # a clip's patches at time, height and width, rotated in a prompt batch; an odd count
        dict(name="rotate-video", op="rotate", tokens=12873, q_heads=16, kv_heads=8, dim=128, rot=128, axes=3,
             interleaved=False, far=4096),
        # a decode step's new token of each of sixteen sequences
        dict(name="append-step", op="append", batch=16, new=1, held=3900, kv_heads=8, dim=128),
        # three prompts that arrive together, the first pages of one of them already there
        dict(name="append-prompt", op="append", batch=3, new=3001, held=130, kv_heads=8, dim=256),
        # one user's step early in a conversation: latency
        dict(name="attend-step-short", op="attend", batch=1, new=1, held=777, idle=0, q_heads=24, kv_heads=8,
             dim=128, window=0, sinks=0),
        # a serving step over sequences of all lengths, two slots of the batch idle
        dict(name="attend-step-batch", op="attend", batch=48, new=1, held=6007, idle=2, q_heads=24, kv_heads=8,
             dim=128, window=0, sinks=0),
        # two very long contexts, wide heads
        dict(name="attend-step-long", op="attend", batch=2, new=1, held=131071, idle=0, q_heads=16, kv_heads=8,
             dim=256, window=0, sinks=0),
        # long chats under a sliding window with four first tokens kept
        dict(name="attend-step-window", op="attend", batch=24, new=1, held=12345, idle=0, q_heads=24, kv_heads=8,
             dim=128, window=1024, sinks=4),
        # five drafted tokens of each sequence checked at once, narrow heads
        dict(name="attend-verify", op="attend", batch=8, new=5, held=8003, idle=0, q_heads=32, kv_heads=8, dim=64,
             window=0, sinks=0),
        # the second part of two long prompts
        dict(name="attend-prompt", op="attend", batch=2, new=2048, held=5000, idle=0, q_heads=24, kv_heads=8,
             dim=128, window=0, sinks=0),
        # eight continuations of one prompt, over all layers of a small stack: shared pages, private tails
        dict(name="pages-fork", op="fork", layers=28, forks=8, held=3001, kv_heads=8, dim=128),
        # a defragmenting move of pages over all layers
        dict(name="pages-move", op="move", layers=28, moves=160, kv_heads=8, dim=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "append", "attend", "attend", "attend", "pages"])
    if op == "rotate":
        dim = rng.choice([64, 128, 256])
        axes = rng.choice([1, 3])
        q_heads, kv_heads = rng.choice([(24, 8), (16, 8), (32, 8), (8, 1)])
        return dict(op="rotate", tokens=_log(rng, 1, 12000 * 128 // dim), q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim // 2]), axes=axes, interleaved=rng.random() < 0.4,
                    far=_log(rng, 64, 4000000))
    if op == "append":
        dim = rng.choice([64, 128, 256])
        batch = _log(rng, 1, 64)
        return dict(op="append", batch=batch, new=_log(rng, 1, max(1, 8000 // batch)),
                    held=_log(rng, 1, 4000), kv_heads=rng.choice([1, 4, 8]), dim=dim)
    if op == "attend":
        dim = rng.choice([64, 128, 256])
        q_heads, kv_heads = rng.choice([(24, 8), (16, 8), (32, 8), (8, 8), (12, 1)])
        form = rng.choice(["step", "step", "verify", "prompt"])
        window, sinks = (0, 0) if rng.random() < 0.6 else (_log(rng, 16, 4096), rng.choice([0, 1, 4, 16]))
        if form == "step":
            batch = _log(rng, 1, 96)
            new, held = 1, _log(rng, 1, min(131071, 260000 // batch))
        elif form == "verify":
            batch = _log(rng, 1, 32)
            new = rng.randint(2, 12)
            held = _log(rng, 1, 130000 // batch)
        else:
            batch = rng.randint(1, 4)
            new = _log(rng, 13, 2048 // batch)
            held = _log(rng, 1, 6000)
        return dict(op="attend", batch=batch, new=new, held=held, idle=rng.choice([0, 1]) if batch > 4 else 0,
                    q_heads=q_heads, kv_heads=kv_heads, dim=dim, window=window, sinks=sinks)
    dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([2, 4, 8])
    if rng.random() < 0.5:
        return dict(op="fork", layers=_log(rng, 1, 28), forks=_log(rng, 1, 24), held=_log(rng, 1, 6000),
                    kv_heads=kv_heads, dim=dim)
    return dict(op="move", layers=_log(rng, 1, 28), moves=_log(rng, 1, 160 * 128 // dim), kv_heads=kv_heads, dim=dim)


def _counts(case):
    """(held, new) tokens of each sequence: the first has the case's own numbers, the others between a quarter
    and all of them; the last `idle` slots hold nothing (new rows stay, and see nothing)."""
    held, new = [], []
    for b in range(case["batch"]):
        f = 1.0 if b == 0 else 0.25 + 0.75 * ((b * 0.6180339887498949) % 1.0)
        held.append(max(1, int(case["held"] * f)))
        new.append(max(1, int(case["new"] * f)))
    for b in range(case["batch"] - case.get("idle", 0), case["batch"]):
        held[b], new[b] = 0, 1
    return held, new


def _cu(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


def _pages(tokens):
    return -(-tokens // BLOCK)


def _total(case):
    """Tokens of each sequence once its new ones are in the cache (none for idle slots)."""
    held, new = _counts(case)
    idle = case.get("idle", 0)
    return [0 if b >= case["batch"] - idle else h + n for b, (h, n) in enumerate(zip(held, new))]


def _span(pos, window, sinks):
    """How many positions a row at `pos` sees, and (first of the window, sinks before it)."""
    lo = max(0, pos - window + 1) if window else 0
    return lo, min(sinks, lo)


def work(case):
    op = case["op"]
    if op == "rotate":
        n = case["tokens"] * (case["q_heads"] + case["kv_heads"])
        return {"bytes": n * case["dim"] * 4 + 4 * case["axes"] * case["tokens"], "flops": n * case["rot"] * 3}
    if op == "append":
        held, new = _counts(case)
        row = case["kv_heads"] * case["dim"] * 2
        t = sum(new)
        back = sum(h + n - h // BLOCK * BLOCK for h, n in zip(held, new))
        blocks = sum(_pages(h + n) - h // BLOCK for h, n in zip(held, new))
        return {"bytes": row * (t * 2 + t + back * 2) + 8 * case["kv_heads"] * blocks, "flops": row * t * 2}
    if op == "attend":
        _, new = _counts(case)
        keys = pairs = blocks = 0
        for n, total in zip(new, _total(case)):
            if not total:
                continue
            first = total - n
            lo, s = _span(first, case["window"], case["sinks"])
            seen = total - lo + s
            keys += seen
            blocks += _pages(seen)
            for pos in range(first, total):
                lo, s = _span(pos, case["window"], case["sinks"])
                pairs += pos + 1 - lo + s
        rows = sum(new) * case["q_heads"] * case["dim"]
        return {"bytes": keys * case["kv_heads"] * case["dim"] * 2 + 8 * blocks * case["kv_heads"] + 4 * rows,
                "flops": 4 * pairs * case["q_heads"] * case["dim"]}
    page = case["layers"] * case["kv_heads"] * (BLOCK * case["dim"] * 2 + 8)
    n = case["moves"] if op == "move" else (case["forks"] if case["held"] % BLOCK else 0)
    t = 0 if op == "move" else 4 * (case["forks"] + 1) * _pages(case["held"] + 1)
    return {"bytes": 2 * n * page + t + 8 * n, "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed(seed * 1000003 + salt)


def _bf16_rows(g, tokens, heads, dim, spread):
    """Rows as a projection gives them: heads and channels of their own size, a few channels far larger, and
    tokens that differ in size."""
    x = torch.randn(tokens, heads, dim, generator=g, device="cuda")
    ch = torch.exp(0.4 * torch.randn(heads, dim, generator=g, device="cuda"))
    big = torch.rand(heads, dim, generator=g, device="cuda") < 0.02
    ch = torch.where(big, ch * spread, ch)
    tok = torch.exp(0.3 * torch.randn(tokens, 1, 1, generator=g, device="cuda"))
    return (x * ch * tok).to(torch.bfloat16)


def _kv_rows(case, seed):
    tokens = sum(_total(case))
    g = _gen(seed, 1)
    k = _bf16_rows(g, tokens, case["kv_heads"], case["dim"], 5.0)
    v = _bf16_rows(g, tokens, case["kv_heads"], case["dim"], 2.0)
    return k, v


def _q_rows(case, seed):
    _, new = _counts(case)
    g = _gen(seed, 2)
    return (0.8 * torch.randn(sum(new), case["q_heads"], case["dim"], generator=g, device="cuda")).to(torch.bfloat16)


def _table(case, seed):
    """Page numbers as a pool in use gives them: scattered.  [batch, pages of the longest], -1 past the end."""
    totals = _total(case)
    n = sum(_pages(t) for t in totals)
    g = torch.Generator().manual_seed(seed * 7919 + 3)
    perm = torch.randperm(n + 5, generator=g, dtype=torch.int64)[:n].to(torch.int32)
    width = max(1, max(_pages(t) for t in totals))
    table = torch.full((case["batch"], width), -1, dtype=torch.int32)
    at = 0
    for b, t in enumerate(totals):
        table[b, :_pages(t)] = perm[at:at + _pages(t)]
        at += _pages(t)
    return table, n + 5


def _rotate_inputs(case, seed):
    g = _gen(seed, 4)
    width = (case["q_heads"] + 2 * case["kv_heads"]) * case["dim"]
    qkv = torch.randn(case["tokens"], width, generator=g, device="cuda").to(torch.bfloat16)
    t, far = case["tokens"], case["far"]
    if case["axes"] == 1:
        pos = torch.arange(max(0, far - t + 1), max(0, far - t + 1) + t, dtype=torch.int32, device="cuda").view(1, t)
    else:
        w = max(1, int(round((t * 1.7) ** (1 / 3))))
        i = torch.arange(t, dtype=torch.int32, device="cuda")
        pos = torch.stack([far + i // (w * w), i // w % w, i % w]).to(torch.int32)
    return qkv, pos


def _sections(case):
    """Pairs of each axis: a quarter for time, the rest for height and width."""
    half = case["rot"] // 2
    if case["axes"] == 1:
        return [half]
    s = half // 4
    return [half - 2 * ((half - s) // 2)] + [(half - s) // 2] * 2


def _page_inputs(case, seed):
    """The raw bytes of a pool: pages are copied as they are."""
    held = case.get("held", 0)
    used = _pages(held) if case["op"] == "fork" else 2 * case["moves"]
    pages = used + (2 * case["forks"] + 3 if case["op"] == "fork" else 3)
    g = _gen(seed, 5)
    shape = (case["layers"], pages, case["kv_heads"])
    k = torch.randint(0, 120, (*shape, BLOCK * case["dim"]), generator=g, device="cuda", dtype=torch.uint8)
    v = torch.randint(0, 120, (*shape, BLOCK * case["dim"]), generator=g, device="cuda", dtype=torch.uint8)
    ks = torch.exp2(torch.randint(-8, 2, shape, generator=g, device="cuda").float())
    vs = torch.exp2(torch.randint(-8, 2, shape, generator=g, device="cuda").float())
    c = torch.Generator().manual_seed(seed * 7919 + 6)
    perm = torch.randperm(pages, generator=c, dtype=torch.int64).to(torch.int32)
    return pages, k, v, ks, vs, perm


def prepare(case, seed):
    op = case["op"]
    if op == "rotate":
        return _prepare_rotate(case, seed)
    if op in ("append", "attend"):
        return _prepare_tokens(case, seed)
    return _prepare_pages(case, seed)


def _prepare_rotate(case, seed):
    qkv, pos = _rotate_inputs(case, seed)
    st = dict(case=case, qkv=qkv, pos=pos)
    if own:
        import decode_gemv_tensor_gb300 as dgt
        st["rotary"] = dgt.Rotary(case["rot"], base=500000.0, sections=_sections(case),
                                  interleaved=case["interleaved"])
    else:
        half = case["rot"] // 2
        i = torch.arange(half, dtype=torch.float64, device="cuda")
        st["freq"] = torch.exp(i * (-2.0 / case["rot"] * math.log(500000.0)))
        st["axis"] = torch.repeat_interleave(torch.arange(case["axes"]), torch.tensor(_sections(case))).cuda()
    return st


def _prepare_tokens(case, seed):
    held, new = _counts(case)
    totals = _total(case)
    k, v = _kv_rows(case, seed)
    table, pages = _table(case, seed)
    # an append finds the tokens before its own in the cache; attention finds all of them
    first = held if case["op"] == "append" else totals
    cu_all = _cu(totals)
    idx = torch.cat([torch.arange(cu_all[b], cu_all[b] + first[b]) for b in range(case["batch"])]).cuda()
    st = dict(case=case, held=held, new=new, totals=totals)
    if own:
        import decode_gemv_tensor_gb300 as dgt
        cache = dgt.KvCache(1, pages, case["kv_heads"], case["dim"], max_seqs=case["batch"],
                            max_pages=table.shape[1])
        cache.table.copy_(table)
        cache.lens.copy_(torch.tensor(totals, dtype=torch.int32))
        cache.refs[table[table >= 0].long().cuda()] = 1
        seqs = torch.arange(case["batch"], dtype=torch.int32, device="cuda")
        dgt.kv_append(cache, 0, k[idx], v[idx], seqs, torch.zeros_like(seqs),
                      cu=torch.tensor(_cu(first), dtype=torch.int32, device="cuda"))
        st.update(cache=cache, seqs=seqs)
    else:
        codes = torch.zeros((2, pages, BLOCK, case["kv_heads"], case["dim"]), dtype=torch.uint8, device="cuda")
        scale = torch.zeros((2, pages, case["kv_heads"]), device="cuda")
        st.update(codes=codes, scale=scale, table=table.cuda().long())
        cu = _cu(first)
        for b in range(case["batch"]):
            _plain_append(st, b, 0, [x[idx[cu[b]:cu[b + 1]]] for x in (k, v)])
    if case["op"] == "append":
        idx = torch.cat([torch.arange(cu_all[b] + held[b], cu_all[b + 1]) for b in range(case["batch"])]).cuda()
        st.update(k=k[idx], v=v[idx], cu=_cu(new))
        if own:
            back = [h // BLOCK * BLOCK for h in held]
            i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
            st.update(start=i32(held), cu=None if max(new) == 1 else i32(_cu(new)), back=i32(back),
                      cu_back=i32(_cu([t - s for t, s in zip(totals, back)])),
                      n_back=sum(totals) - sum(back))
    else:
        st["q"] = _q_rows(case, seed)
        if own:
            st["cu"] = None if max(new) == 1 else torch.tensor(_cu(new), dtype=torch.int32, device="cuda")
            st["ws"] = dgt.kv_attention_workspace(st["cache"], case["q_heads"], case["batch"], sum(new))
    return st


def _prepare_pages(case, seed):
    pages, k, v, ks, vs, perm = _page_inputs(case, seed)
    if case["op"] == "move":
        n = case["moves"]
        src, dst = perm[:n].cuda(), perm[n:2 * n].cuda()
    seqs = case.get("forks", 0) + 1
    width = _pages(case.get("held", 0) + 1)
    if own:
        import decode_gemv_tensor_gb300 as dgt
        cache = dgt.KvCache(case["layers"], pages, case["kv_heads"], case["dim"], max_seqs=seqs, max_pages=width)
        for name, x in (("k", k), ("v", v), ("k_scale", ks), ("v_scale", vs)):
            getattr(cache, name).copy_(x)
        st = dict(case=case, cache=cache)
        table, refs, lens = cache.table, cache.refs, cache.lens
    else:
        table = torch.full((seqs, width), -1, dtype=torch.int32, device="cuda")
        refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        st = dict(case=case, k=k, v=v, ks=ks, vs=vs, table=table, refs=refs, lens=lens)
    if case["op"] == "move":
        st.update(src=src, dst=dst)
    else:
        n = _pages(case["held"])
        table[0, :n] = perm[:n].cuda()
        refs[perm[:n].long().cuda()] = 1
        lens[0] = case["held"]
        st["parent"] = torch.zeros(case["forks"], dtype=torch.int32, device="cuda")
        st["children"] = torch.arange(1, case["forks"] + 1, dtype=torch.int32, device="cuda")
        st["ones"] = torch.ones(case["forks"], dtype=torch.int32, device="cuda")
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    return (_own if own else _plain)[st["case"]["op"]](st)


def _own_rotate(st):
    import decode_gemv_tensor_gb300 as dgt
    c, qkv = st["case"], st["qkv"]
    nq, nk = c["q_heads"] * c["dim"], c["kv_heads"] * c["dim"]
    q = qkv[:, :nq].view(-1, c["q_heads"], c["dim"])
    k = qkv[:, nq:nq + nk].view(-1, c["kv_heads"], c["dim"])
    return dgt.rotate(st["rotary"], q, st["pos"], k=k)


def _own_append(st):
    import decode_gemv_tensor_gb300 as dgt
    dgt.kv_append(st["cache"], 0, st["k"], st["v"], st["seqs"], st["start"], cu=st["cu"])
    return dgt.kv_read(st["cache"], 0, st["seqs"], st["back"], st["cu_back"], st["n_back"])


def _own_attend(st):
    import decode_gemv_tensor_gb300 as dgt
    c = st["case"]
    return dgt.kv_attention(st["cache"], 0, st["q"], st["seqs"], cu=st["cu"], window=c["window"], sinks=c["sinks"],
                            ws=st["ws"])


def _own_fork(st):
    import decode_gemv_tensor_gb300 as dgt
    cache = st["cache"]
    dgt.kv_fork(cache, st["parent"], st["children"])
    start = dgt.kv_reserve(cache, st["children"], st["ones"])
    out = [start, cache.table.clone(), cache.refs.clone(), cache.lens.clone()]
    dgt.kv_free(cache, st["children"])
    return out + [cache.k, cache.v, cache.k_scale, cache.v_scale]


def _own_move(st):
    import decode_gemv_tensor_gb300 as dgt
    cache = st["cache"]
    dgt.kv_copy_pages(cache, st["src"], st["dst"])
    return [cache.k, cache.v, cache.k_scale, cache.v_scale]


def _plain_rotate(st):
    c, qkv = st["case"], st["qkv"]
    nq, nk = c["q_heads"] * c["dim"], c["kv_heads"] * c["dim"]
    half = c["rot"] // 2
    angle = st["pos"].double()[st["axis"]].T * st["freq"]            # [tokens, half]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    out = []
    for x in (qkv[:, :nq].view(-1, c["q_heads"], c["dim"]), qkv[:, nq:nq + nk].view(-1, c["kv_heads"], c["dim"])):
        x = x.float()
        if c["interleaved"]:
            a, b = x[..., 0:c["rot"]:2], x[..., 1:c["rot"]:2]
        else:
            a, b = x[..., :half], x[..., half:c["rot"]]
        ra, rb = a * cos - b * sin, b * cos + a * sin
        r = torch.stack([ra, rb], -1).flatten(-2) if c["interleaved"] else torch.cat([ra, rb], -1)
        out.append(torch.cat([r, x[..., c["rot"]:]], -1).to(torch.bfloat16))
    return out


def _scale_exp(amax):
    """Smallest e with amax <= 448 * 2^e, at least E_MIN (448 = 0.875 * 2^9 is the largest e4m3 value)."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, E_MIN).clamp(min=E_MIN)


def _plain_append(st, b, start, rows):
    """Tokens start.. of sequence b from bf16 rows (keys, values), block by block.  A block that already holds
    tokens keeps its scale unless the new ones need a larger one; then its codes are rounded to the new scale."""
    n = rows[0].shape[0]
    if n == 0:
        return
    b0, b1 = start // BLOCK, _pages(start + n)
    page = st["table"][b, b0:b1]
    old = start - b0 * BLOCK
    for side, x in enumerate(rows):
        new = torch.zeros(((b1 - b0) * BLOCK, *x.shape[1:]), device="cuda")
        new[old:old + n] = x.float()
        new = new.view(b1 - b0, BLOCK, *x.shape[1:])
        e = _scale_exp(new.abs().amax(dim=(1, 3)))                    # [blocks, heads]
        if old:
            was = st["scale"][side, page[0]]
            e[0] = torch.maximum(e[0], torch.frexp(was)[1] - 1)
            new[0, :old] = st["codes"][side, page[0], :old].view(torch.float8_e4m3fn).float() * was[:, None]
        s = torch.exp2(e.float())
        st["codes"][side, page] = (new / s[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        st["scale"][side, page] = s


def _plain_values(st, side, b, first, total):
    """Tokens [first, total) of sequence b as the values that their codes stand for (float32)."""
    page = st["table"][b, first // BLOCK:_pages(total)]
    x = st["codes"][side][page].view(torch.float8_e4m3fn).float() * st["scale"][side][page][:, None, :, None]
    return x.flatten(0, 1)[first % BLOCK:][:total - first]


def _plain_append_run(st):
    cu = st["cu"]
    out = [[], []]
    for b in range(st["case"]["batch"]):
        _plain_append(st, b, st["held"][b], [x[cu[b]:cu[b + 1]] for x in (st["k"], st["v"])])
        for side in (0, 1):
            out[side].append(_plain_values(st, side, b, st["held"][b] // BLOCK * BLOCK, st["totals"][b]))
    return [torch.cat(x).to(torch.bfloat16) for x in out]


def _visible(first, total, window, sinks, key0):
    """[rows, keys] truth table: rows at positions first..total-1, keys at key0..total-1."""
    i = torch.arange(first, total, device="cuda")[:, None]
    j = torch.arange(key0, total, device="cuda")[None]
    see = j <= i
    if window:
        see = see & ((j > i - window) | (j < sinks))
    return see


def _plain_attend(st):
    c = st["case"]
    hk, d = c["kv_heads"], c["dim"]
    group = c["q_heads"] // hk
    out, at = [], 0
    for b in range(c["batch"]):
        n, total = st["new"][b], st["totals"][b]
        q = st["q"][at:at + n].float()
        at += n
        if total == 0:
            out.append(torch.zeros_like(q))
            continue
        first = total - n
        # keys before the first row's window are only looked at where they stay visible
        lo = _span(first, c["window"], c["sinks"])[0] // BLOCK * BLOCK
        s = min(c["sinks"], lo) if c["window"] else 0
        k, v = (_plain_values(st, side, b, lo, total) for side in (0, 1))
        see = _visible(first, total, c["window"], c["sinks"], lo)
        if s:
            k, v = (torch.cat([_plain_values(st, side, b, 0, s), x]) for side, x in ((0, k), (1, v)))
            see = torch.cat([torch.ones((n, s), dtype=torch.bool, device="cuda"), see], 1)
        q = q.view(n, hk, group, d).permute(1, 2, 0, 3)                # [hk, group, n, d]
        t = torch.matmul(q, k.permute(1, 2, 0)[:, None]) * (1.0 / math.sqrt(d))
        t = torch.where(see, t, -math.inf)
        p = torch.exp(t - t.amax(-1, keepdim=True))
        y = torch.matmul(p, v.permute(1, 0, 2)[:, None]) / p.sum(-1, keepdim=True)
        out.append(y.permute(2, 0, 1, 3).reshape(n, c["q_heads"], d))
    return torch.cat(out).to(torch.bfloat16)


def _plain_fork(st):
    table, refs, lens = st["table"], st["refs"], st["lens"]
    kids = st["children"].long()
    # fork: the children share the parent's pages
    table[kids] = table[st["parent"].long()]
    lens[kids] = lens[st["parent"].long()]
    shared = table[0][table[0] >= 0].long()
    refs[shared] += len(kids)
    # reserve one token each: a shared partial page is copied, a full one is followed by a fresh page
    held = st["case"]["held"]
    last = held // BLOCK
    free = torch.nonzero(refs == 0)[:len(kids), 0]
    if held % BLOCK:
        old = table[kids, last].long()
        for x in (st["k"], st["v"], st["ks"], st["vs"]):
            x[:, free] = x[:, old]
        refs[old[0]] -= len(kids)
    table[kids, last] = free.int()
    refs[free] = 1
    start = lens[kids]
    lens[kids] = start + 1
    out = [start, table.clone(), refs.clone(), lens.clone()]
    # free the children again
    refs[shared] -= len(kids)
    if held % BLOCK:
        refs[old[0]] += len(kids)
    refs[free] = 0
    table[kids] = -1
    lens[kids] = 0
    return out + [st["k"], st["v"], st["ks"], st["vs"]]


def _plain_move(st):
    src, dst = st["src"].long(), st["dst"].long()
    out = [st["k"], st["v"], st["ks"], st["vs"]]
    for x in out:
        x[:, dst] = x[:, src]
    return out


_own = dict(rotate=_own_rotate, append=_own_append, attend=_own_attend, fork=_own_fork, move=_own_move)
_plain = dict(rotate=_plain_rotate, append=_plain_append_run, attend=_plain_attend, fork=_plain_fork,
              move=_plain_move)


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    return dict(rotate=_exact_rotate, append=_exact_append, attend=_exact_attend, fork=_exact_fork,
                move=_exact_move)[case["op"]](case, seed)


def _exact_rotate(case, seed):
    qkv, pos = _rotate_inputs(case, seed)
    d, rot, half = case["dim"], case["rot"], case["rot"] // 2
    x = qkv.double().view(case["tokens"], -1, d)[:, :case["q_heads"] + case["kv_heads"]]
    y = x.clone()
    pair, axis = 0, 0
    for axis, count in enumerate(_sections(case)):
        for _ in range(count):
            a = pos[axis].double() * 500000.0 ** (-2.0 * pair / rot)
            turn = torch.polar(torch.ones_like(a), a)[:, None]
            i, j = (2 * pair, 2 * pair + 1) if case["interleaved"] else (pair, pair + half)
            z = torch.complex(x[..., i], x[..., j]) * turn
            y[..., i], y[..., j] = z.real, z.imag
            pair += 1
    return [y[:, :case["q_heads"]], y[:, case["q_heads"]:]]


def _exact_e4m3(x):
    """To the nearest e4m3 value, ties to even: three fraction bits, the smallest step 2^-9."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_blocks(x, held):
    """Values of one sequence's rows x [tokens, heads, dim] after an append of the first `held` (when any) and one
    of the rest: each block takes the smallest power-of-two scale that holds it, and never a smaller one."""
    x = x.double()
    out = torch.zeros_like(x)
    for t in range(0, x.shape[0], BLOCK):
        blk = x[t:t + BLOCK]
        cut = min(max(held - t, 0), blk.shape[0])
        s = torch.full((x.shape[1], 1), 2.0 ** E_MIN, dtype=torch.float64, device="cuda")
        val = blk[:0]
        for part in (blk[:cut], blk[cut:]):
            if part.shape[0]:
                top = part.abs().amax(dim=(0, 2))[:, None]
                e = torch.ceil(torch.log2((top / 448.0).clamp(min=2.0 ** -140)))
                e = torch.where(448.0 * torch.exp2(e - 1) >= top, e - 1, e)
                s = torch.maximum(s, torch.exp2(e))
                val = _exact_e4m3(torch.cat([val, part]) / s) * s
        out[t:t + blk.shape[0]] = val
    return out


def _exact_blocks_at_once(x):
    """_exact_blocks for one append of everything, all blocks together."""
    n = x.shape[0]
    pad = torch.zeros((_pages(n) * BLOCK, *x.shape[1:]), dtype=torch.float64, device="cuda")
    pad[:n] = x
    pad = pad.view(-1, BLOCK, *x.shape[1:])
    top = pad.abs().amax(dim=(1, 3), keepdim=True)
    e = torch.ceil(torch.log2((top / 448.0).clamp(min=2.0 ** -140)))
    e = torch.where(448.0 * torch.exp2(e - 1) >= top, e - 1, e).clamp(min=E_MIN)
    s = torch.exp2(e)
    return (_exact_e4m3(pad / s) * s).flatten(0, 1)[:n]


def _exact_append(case, seed):
    held, _ = _counts(case)
    cu = _cu(_total(case))
    out = []
    for x in _kv_rows(case, seed):
        parts = []
        for b in range(case["batch"]):
            t0 = held[b] // BLOCK * BLOCK
            parts.append(_exact_blocks(x[cu[b] + t0:cu[b + 1]], held[b] - t0))
        out.append(torch.cat(parts))
    return out


def _exact_attend(case, seed):
    k, v = _kv_rows(case, seed)
    q = _q_rows(case, seed).double()
    _, new = _counts(case)
    totals = _total(case)
    cu, group = _cu(totals), case["q_heads"] // case["kv_heads"]
    out = torch.zeros_like(q)
    at = 0
    for b in range(case["batch"]):
        n, total = new[b], totals[b]
        rows = slice(at, at + n)
        at += n
        if not total:
            continue
        kb, vb = (_exact_blocks_at_once(x[cu[b]:cu[b + 1]]) for x in (k, v))
        i = torch.arange(total - n, total, device="cuda").view(-1, 1)
        j = torch.arange(total, device="cuda").view(1, -1)
        hidden = j > i
        if case["window"]:
            hidden |= (j <= i - case["window"]) & (j >= case["sinks"])
        for h in range(case["q_heads"]):
            t = q[rows, h] @ kb[:, h // group].T / math.sqrt(case["dim"])
            out[rows, h] = torch.softmax(t.masked_fill(hidden, -math.inf), -1) @ vb[:, h // group]
    return out


def _exact_fork(case, seed):
    pages, k, v, ks, vs, perm = _page_inputs(case, seed)
    held, forks = case["held"], case["forks"]
    own_pages = perm[:_pages(held)].tolist()
    refs = [0] * pages
    for p in own_pages:
        refs[p] = 1 + forks
    width = _pages(held + 1)
    rows = [own_pages + [-1] * (width - len(own_pages))]
    for _ in range(forks):
        row = list(rows[0])
        page = refs.index(0)
        refs[page] = 1
        if held % BLOCK:
            old = row[held // BLOCK]
            refs[old] -= 1
            for x in (k, v, ks, vs):
                x[:, page] = x[:, old]
        row[held // BLOCK] = page
        rows.append(row)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    return [i32([held] * forks), i32(rows), i32(refs), i32([held] + [held + 1] * forks), k, v, ks, vs]


def _exact_move(case, seed):
    _, k, v, ks, vs, perm = _page_inputs(case, seed)
    n = case["moves"]
    out = [k, v, ks, vs]
    for x in out:
        for i in range(n):
            x[:, perm[n + i]] = x[:, perm[i]]
    return out
