"""beam_select and kv_reorder against plain implementations: totals in 64 bits,
tables by lists."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import decode_gemv_tensor_gb300 as dgt  # noqa: E402

pytestmark = pytest.mark.gpu
INF = float("inf")
F32, BF16 = torch.float32, torch.bfloat16


def log_sum(x):
    """log sum e^x of each row, rounded once: rows of the same numbers in any order have the same."""
    out = []
    for row in x.cpu().sort(-1)[0].numpy():
        m = float(row[-1])
        out.append(m + math.log(math.fsum(np.exp(row - m))) if math.isfinite(m) else m)
    return torch.tensor(out, dtype=torch.float64, device=x.device)[:, None]


def reference(logits, scores, n, eos=-1, done=None):
    batch, beams = scores.shape
    vocab = logits.shape[1]
    out = []
    for e in range(batch):
        x = logits[e * beams:(e + 1) * beams].double()
        total = scores[e].double()[:, None] + (x - log_sum(x))
        bad = ~scores[e].isfinite() | x.isnan().any(1) | (x == INF).any(1)
        total = torch.where(bad[:, None] | total.isnan(), -INF, total)
        if done is not None:
            for b in range(beams):
                if done[e, b]:
                    total[b] = -INF
                    if bool(scores[e, b].isfinite()):
                        total[b, eos] = scores[e, b].double()
        total = total.flatten()
        k = min(n, total.numel())
        at = torch.nonzero(total >= total.topk(k)[0][-1])[:, 0]
        at = at[torch.sort(total[at], descending=True, stable=True)[1]][:n]
        at = at[total[at] > -INF]
        p = torch.full((4, n), -1.0, dtype=torch.float64, device=x.device)
        p[2], p[3] = -INF, 0
        p[0, :len(at)], p[1, :len(at)], p[2, :len(at)] = at // vocab, at % vocab, total[at]
        if done is not None:
            p[3, :len(at)] = ((done[e][at // vocab] != 0) | (at % vocab == eos)).double()
        out.append(p)
    return torch.stack(out, 1)


def check(logits, scores, n, eos=-1, done=None, **kw):
    """A total is off by the sum of fp32 terms, below 2^-18, and one rounding."""
    got = dgt.beam_select(logits, scores, n, eos=eos, done=done, **kw)
    want = reference(logits, scores, n, eos, done)
    assert torch.equal(got[0].double(), want[0]) and torch.equal(got[1].double(), want[1])
    same = (got[2].double() == want[2]) | ((got[2].double() - want[2]).abs() <= 2.0 ** -18 + want[2].abs() * 2.0 ** -24)
    assert bool(same.all())
    if done is not None:
        assert torch.equal(got[3].double(), want[3])
    return got


def inputs(batch, beams, vocab, dtype=F32, seed=0, spread=3.0):
    g = torch.Generator("cuda").manual_seed(seed)
    x = (spread * torch.randn(batch * beams, vocab, device="cuda", generator=g)).to(dtype)
    return x, -20 * torch.rand(batch, beams, device="cuda", generator=g)


@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 255, 1000, 4096, 8191, 8193, 32000, 50257, 128256])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_vocabularies(vocab, dtype):
    for batch, beams, n in ((1, 1, 1), (1, 4, 8), (3, 5, 10), (2, 3, 64)):
        x, s = inputs(batch, beams, vocab, dtype, vocab + n)
        check(x, s, n)


@pytest.mark.parametrize("batch,beams,n", [(1, 1, 64), (1, 64, 32), (1, 32, 64), (2, 16, 16), (40, 8, 8), (150, 8, 16),
                                           (700, 1, 2), (5, 2, 1), (1, 2, 33)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_batches(batch, beams, n, dtype):
    x, s = inputs(batch, beams, 9001, dtype, batch)
    check(x, s, n)


def test_large_rows_in_few_segments():
    x, s = inputs(100, 8, 40000, BF16, 3)
    check(x, s, 16)
    x, s = inputs(2, 2, 400000, F32, 4)
    check(x, s, 64)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [300, 30011])
def test_orders_that_fill_the_list(dtype, vocab):
    """Ever greater logits, equal ones, and runs of them: every element passes the threshold of those before it."""
    up = torch.arange(vocab, device="cuda", dtype=torch.float64)
    rows = [up * 1e-3, -up * 1e-3, torch.zeros_like(up), (up // 1000), -(up // 1000), up % 7, (up * 7919) % vocab * 1e-3,
            torch.where(up == vocab - 1, 5.0, 0.0)]
    x = torch.stack(rows).to(dtype)
    s = torch.full((1, 8), -1.0, device="cuda")
    for n in (1, 8, 64):
        check(x, s, n)                     # beams against one another
        check(x, s.view(8, 1), n)          # and alone


def test_equal_rows_are_equal_beams():
    """Two beams with one row and one score: every candidate ties, the lower beam and token come first."""
    x, _ = inputs(1, 1, 50257, BF16, 1)
    x = x.repeat(4, 1)
    check(x, torch.full((1, 4), -3.0, device="cuda"), 16)
    check(x.float(), torch.full((2, 2), -3.0, device="cuda"), 9)


@pytest.mark.parametrize("dtype,vocab", [(F32, 50257), (BF16, 128256)])
def test_totals_that_differ_by_less_than_fp32_sums_can_tell(dtype, vocab):
    """Scores that put the best of one beam next to the best of another, closer than sums of fp32 terms are."""
    for seed in range(12):
        x, _ = inputs(1, 3, vocab, dtype, seed)
        top = (x.double() - torch.logsumexp(x.double(), -1, keepdim=True)).amax(-1)
        s = (-30.0 - top).float().view(1, 3)
        gaps = (s.double().view(-1) + top)
        gaps = (gaps[:, None] - gaps[None]).abs()[[0, 0, 1], [1, 2, 2]]
        assert float(gaps.max()) < 2e-5 and float(gaps.min()) > 2.0 ** -28
        check(x, s, 6)


def test_beams_without_scores_or_at_their_end():
    x, s = inputs(4, 4, 20000, BF16, 8)
    s[0, 1:] = -INF                           # a first step
    s[1] = -INF                               # an entry without beams
    s[2, 0] = float("nan")
    s[2, 1] = INF
    check(x, s, 8)
    done = torch.zeros(4, 4, dtype=torch.uint8, device="cuda")
    done[0, 0] = done[2, 2] = done[3, 1] = 1
    done[3, 2] = 255
    s[3] = torch.tensor([-5.0, -4.0, -100.0, -6.0], device="cuda")
    for n in (1, 4, 8):
        check(x, s, n, eos=7, done=done)
    done[:] = 1
    got = check(x, s, 8, eos=19999, done=done)
    assert bool((got[0][:, 4:] == -1).all())


def test_masked_and_infinite_logits():
    x, s = inputs(2, 3, 9000, F32, 2)
    x[0, 10:] = -INF                          # ten candidates left
    x[1] = -INF                               # none
    x[2, ::2] = -INF
    check(x, s, 64)
    x[0, 3] = INF
    x[2, 8999] = float("nan")
    x[4, 0] = float("nan")
    check(x, s, 16)
    x[:] = -INF
    got = check(x, s, 5)
    assert bool((got[1] == -1).all()) and bool((got[2] == -INF).all())
    x[:] = torch.finfo(F32).min
    check(x, s, 4)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("mask", [-1e4, -1e9, -1.1e9, -3e12, -1e20, -1e30, -3e38])
def test_masks_of_any_size(dtype, mask):
    """Rows whose beginning, end or most is masked by a finite number, and one that is masked throughout."""
    x, s = inputs(3, 4, 20011, dtype, 31)
    x[0, :9000] = x[1, 5:] = x[2, ::2] = x[4, 10001:] = x[5] = mask
    x[6, torch.arange(20011, device="cuda") % 1024 < 1000] = mask
    x[7, :-1] = mask
    check(x, s, 9)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [1e3, 1e5, 1e8, 1e9, 1e10, 1e16, 1e30])
def test_logits_of_any_size(dtype, size):
    x, s = inputs(2, 3, 9001, dtype, 32)
    x[::2] = (x[::2].double() * size).to(dtype)
    check(x, s, 9)
    y = torch.arange(9001, device="cuda", dtype=torch.float64) - 4500.0
    check((y * size / 100).to(dtype)[None].repeat(2, 1), s[:1, :2].contiguous(), 5)
    check((size - y.abs() * 5).to(dtype)[None], s[:1, :1].contiguous(), 5)    # near one another


@pytest.mark.parametrize("vocab", [40, 3000])
def test_totals_that_are_equal_in_64_bits(vocab):
    """Within a beam the greater logit is first all the same, whichever way the candidates are found."""
    x = inputs(4, 1, vocab, F32, 33)[0] * 1e-30
    got = dgt.beam_select(x, torch.full((2, 2), -3.0, device="cuda"), 30)
    for e in range(2):
        order = torch.sort(x[2 * e], descending=True, stable=True)[1][:30]
        assert torch.equal(got[1][e].long(), order) and not bool(got[0][e].any())


def test_strides_and_offsets():
    wide = torch.randn(6, 10007, device="cuda").bfloat16()
    s = -torch.rand(2, 3, device="cuda")
    for a, b in ((0, 10007), (1, 10007), (3, 5003), (8, 10000), (5, 12)):
        check(wide[:, a:b], s, 4)
        check(wide.float()[:, a:b], s, 4)
    check(wide[::2, 7:9000], s[:1], 4)


def test_one_workspace_for_calls_of_all_sizes():
    ws = dgt.beam_workspace(64, 8, 128256, 16)
    for batch, beams, vocab, n in ((64, 8, 3000, 16), (1, 4, 128256, 8), (64, 8, 1000, 8), (3, 2, 50257, 4), (1, 4, 128256, 8)):
        x, s = inputs(batch, beams, vocab, BF16, batch)
        check(x, s, n, ws=ws)


def test_given_outputs_stream_and_graph():
    x, s = inputs(3, 4, 30000, BF16, 5)
    want = dgt.beam_select(x, s, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dgt.beam_select(x, s, 8, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = [torch.empty_like(t) for t in want]
    ws = dgt.beam_workspace(3, 4, 30000, 8)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dgt.beam_select(x, s, 8, parent=out[0], token=out[1], total=out[2], ws=ws)
    for seed in (6, 7):
        y, t = inputs(3, 4, 30000, BF16, seed)
        x.copy_(y), s.copy_(t)
        g.replay()
        w = dgt.beam_select(y, t, 8)
        assert all(torch.equal(a, b) for a, b in zip(out, w))


def test_refusals():
    x, s = inputs(2, 2, 100)
    bad = [dict(scores=s[:1]), dict(scores=s.double()), dict(scores=s.view(-1)), dict(n=0),
           dict(done=torch.zeros(2, 2, device="cuda")), dict(done_out=torch.zeros(2, 4, dtype=torch.uint8, device="cuda")),
           dict(parent=torch.zeros(2, 4, device="cuda")), dict(total=torch.zeros(2, 3, device="cuda"))]
    for kw in bad:
        with pytest.raises(ValueError):
            dgt.beam_select(x, **{"scores": s, "n": 4, **kw})
    with pytest.raises(ValueError):
        dgt.beam_select(x.half(), s, 4)
    for kw in (dict(n=65), dict(n=4, done=torch.zeros(2, 2, dtype=torch.uint8, device="cuda")),
               dict(n=4, ws=torch.zeros(256, dtype=torch.uint8, device="cuda")), dict(n=2, total=s)):
        with pytest.raises(dgt.DgtError):
            dgt.beam_select(x, s, **kw)


def test_two_calls_at_a_time():
    """On two streams, a workspace each."""
    runs = []
    for seed in (1, 2):
        x, s = inputs(8, 4, 60000, BF16, seed)
        runs.append((x, s, dgt.beam_select(x, s, 8), dgt.beam_workspace(8, 4, 60000, 8), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for x, s, _, ws, stream in runs:
            got.append(dgt.beam_select(x, s, 8, ws=ws, stream=stream))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, runs[i % 2][2]))


def test_few_blocks_and_many_choices():
    """Rows of a few blocks of 1 KB: fewer than the choices, and as many as the warps."""
    for vocab, beams, n in ((100, 2, 64), (513, 1, 16), (1500, 1, 64), (3001, 2, 33), (4100, 4, 16), (2000, 32, 64)):
        for dt in (F32, BF16):
            x, s = inputs(2, beams, vocab, dt, vocab)
            check(x, s, n)


# ---- kv_reorder
def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def cache_of(rows, lens, pages=None):
    width = len(rows[0])
    pages = pages or max(max(r) for r in rows) + 3
    c = dgt.KvCache(1, pages, 1, 64, max_seqs=len(rows), max_pages=width)
    c.table.copy_(torch.tensor(rows, dtype=torch.int32))
    c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    c.refs.copy_(refs_of(c))
    return c


def refs_of(c):
    t = c.table.flatten().long()
    return torch.bincount(t[t >= 0], minlength=c.pages).int()


def reorder_reference(rows, lens, seqs, parent, dst):
    new, nl = [list(r) for r in rows], list(lens)
    for s, p, d in zip(seqs, parent, dst):
        for j in range(len(s)):
            new[d[j]] = [-1] * len(rows[0]) if p[j] < 0 else rows[s[p[j]]]
            nl[d[j]] = 0 if p[j] < 0 else lens[s[p[j]]]
    return new, nl


@pytest.mark.parametrize("groups,beams,width", [(1, 1, 1), (1, 4, 5), (3, 2, 33), (2, 5, 64), (7, 8, 100), (1, 40, 31),
                                                (64, 16, 40), (128, 8, 300)])
@pytest.mark.parametrize("other", [False, True])
def test_reorder(groups, beams, width, other):
    g = torch.Generator().manual_seed(groups * 1000 + width)
    n = groups * beams
    slots = n * (2 if other else 1) + 2
    perm = torch.randperm(slots, generator=g).tolist()
    seqs = [perm[i * beams:(i + 1) * beams] for i in range(groups)]
    dst = [perm[n + i * beams:n + (i + 1) * beams] for i in range(groups)] if other else seqs
    used = torch.randint(0, width + 1, (slots,), generator=g).tolist()
    page = torch.randint(0, slots * width // 2 + 1, (slots, width), generator=g).tolist()
    rows = [[page[s][i] if i < used[s] else -1 for i in range(width)] for s in range(slots)]
    lens = [max(0, u * 64 - s % 64) for s, u in enumerate(used)]
    parent = torch.randint(-1, beams, (groups, beams), generator=g).tolist()
    c = cache_of(rows, lens, slots * width)
    st = i32(0)
    dgt.kv_reorder(c, i32(*seqs), i32(*parent), dst=i32(*dst) if other else None, status=st)
    new, nl = reorder_reference(rows, lens, seqs, parent, dst)
    assert c.table.tolist() == new and c.lens.tolist() == nl
    assert torch.equal(c.refs, refs_of(c)) and dgt.read_status(st) == 0


def test_reorder_over_groups_that_read_one_another():
    """All at once: targets that other groups read still give what they were."""
    rows = [[i * 2, i * 2 + 1] for i in range(6)]
    lens = [10 + i for i in range(6)]
    seqs, dst, parent = ((0, 1, 2), (3, 4, 5)), ((3, 4, 5), (0, 1, 2)), ((1, 1, 0), (2, -1, 0))
    c = cache_of(rows, lens)
    st = i32(0)
    dgt.kv_reorder(c, i32(*seqs), i32(*parent), dst=i32(*dst), status=st)
    new, nl = reorder_reference(rows, lens, seqs, parent, dst)
    assert c.table.tolist() == new and c.lens.tolist() == nl
    assert torch.equal(c.refs, refs_of(c)) and dgt.read_status(st) == 0


def test_reorder_skips_what_it_cannot_do():
    rows = [[0, 1, -1], [2, -1, -1], [3, 4, 5], [6, -1, -1]]
    lens = [100, 5, 190, 64]
    for seqs, parent, dst, done in (((0, 1, 2, 3), (1, 4, -2, 0), None, {0: 1, 3: 0}),          # parents out of range
                                    ((0, 9, 2, -1), (1, 0, 2, 3), (0, 1, 2, 3), {1: 0, 2: 2}),  # slots out of range
                                    ((0, 1, 2, 3), (3, 2, 1, 0), (0, 1, 1, 7), {0: 3})):        # a target twice, one too high
        c = cache_of(rows, lens)
        st = i32(0)
        dgt.kv_reorder(c, i32(*seqs), i32(*parent), dst=None if dst is None else i32(*dst), status=st)
        want = [rows[done.get(i, i)] for i in range(4)]
        assert c.table.tolist() == want and c.lens.tolist() == [lens[done.get(i, i)] for i in range(4)]
        assert torch.equal(c.refs, refs_of(c)) and dgt.read_status(st) == -1


def test_reorder_then_reserve_copies_what_is_shared():
    """Beams over one prompt: after a reorder the next reserve gives every beam a last page of its own."""
    c = dgt.KvCache(2, 40, 2, 64, max_seqs=5, max_pages=6)
    st = i32(0)
    g = torch.Generator("cuda").manual_seed(0)
    r = lambda n: torch.randn(n, 2, 64, device="cuda", generator=g).bfloat16()
    dgt.kv_reserve(c, i32(0), i32(100), status=st)
    rows = {}
    for l in range(2):
        k = r(100)
        rows[l] = k
        dgt.kv_append(c, l, k, k, i32(0), i32(0), cu=i32(0, 100), status=st)
    beams = i32(1, 2, 3, 4)
    dgt.kv_fork(c, i32(0, 0, 0, 0), beams, status=st)
    texts = [[] for _ in range(4)]
    for step in range(40):
        start = dgt.kv_reserve(c, beams, i32(1, 1, 1, 1), status=st)
        # each beam's token is its own constant, exact in e4m3
        tok = torch.randint(1, 8, (4,), generator=g, device="cuda")
        for l in range(2):
            x = tok.view(4, 1, 1).expand(4, 2, 64).bfloat16().contiguous()
            dgt.kv_append(c, l, x, x, beams, start, status=st)
        for b in range(4):
            texts[b] = texts[b] + [int(tok[b])]
        parent = torch.randint(0, 4, (1, 4), generator=g, device="cuda", dtype=torch.int32)
        dgt.kv_reorder(c, beams.view(1, 4), parent, status=st)
        texts = [texts[p] for p in parent[0].tolist()]
        assert torch.equal(c.refs, refs_of(c))
    assert dgt.read_status(st) == 0
    for l in range(2):
        k, v = dgt.kv_read(c, l, beams, i32(0, 0, 0, 0), i32(0, 140, 280, 420, 560), 560)
        k = k.view(4, 140, 2, 64)
        assert float((k[:, :64].float() - rows[l][:64].float()).abs().max()) < 0.25
        for b in range(4):
            got = k[b, 100:, 0, 0].float()
            assert torch.equal(got.round(), torch.tensor(texts[b], device="cuda").float())


def test_reorder_in_a_graph_and_on_a_stream():
    rows = [[0, 1], [2, -1], [3, 4]]
    c = cache_of(rows, [100, 5, 120])
    seqs, parent = i32(0, 1, 2).view(1, 3), i32(1, 0, 2).view(1, 3)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dgt.kv_reorder(c, seqs, parent)
    for _ in range(3):
        g.replay()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dgt.kv_reorder(c, seqs, parent, stream=s)
    s.synchronize()
    assert c.table.tolist() == rows and torch.equal(c.refs, refs_of(c))
    with pytest.raises(ValueError):
        dgt.kv_reorder(c, seqs, parent[:, :2])
