"""Attention of sequences that share their first pages, against 64 bits.

Tolerances as for the attention itself (test_gpu_kv_attention): of an output
2^-8 of it, and 2^-10 of the weighted mean of |v|, which covers both parts'
weights and leaves 2^-12 for the factors that join them; of the lse dim * 2^-24
of the largest sum of |q||k| and 2^-17 (two logarithms).

A row whose weights are nearly all one token's has outputs that are far below
its largest |v|, where that token's value is 0.  What such an output is made of
are weights that the kernels hold no better than they say: weight times value
scale to 2^-29 of the row's largest such product.  A value is at most 448 of
its page's scale and a page's scale at most 1/224 of its largest value, so each
of the tokens that a row sees may be off by 2^-30 * 448 / 224 = 2^-29 of the
largest |v|: that times their number is allowed as well."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import decode_gemv_tensor_gb300 as dgt  # noqa: E402

INF = float("inf")


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def cu_of(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


class Forks:
    """Prompts in slots of their own, and for each a group of sequences forked from it: own = tokens of each sequence
    behind the prompt (None: an idle one)."""

    def __init__(self, prompts, own, hk, dim, layers=1, seed=0, spread=1.0, max_pages=None):
        g = torch.Generator("cuda").manual_seed(seed)
        self.g, self.hk, self.dim, self.layer = g, hk, dim, layers - 1
        count = sum(len(o) for o in own)
        pages = sum(-(-p // 64) for p in prompts) + sum(-(-(64 + n) // 64) + 1 for o in own for n in o if n is not None) + 2
        width = max_pages or max(-(-(p + (n or 0)) // 64) for p, o in zip(prompts, own) for n in o) + 2
        c = self.c = dgt.KvCache(layers, pages, hk, dim, max_seqs=len(prompts) + count, max_pages=width)
        st = i32(0)

        def rows(n):
            size = torch.exp2(spread * torch.randn(n, hk, 1, generator=g, device="cuda"))
            return [(torch.randn(n, hk, dim, generator=g, device="cuda") * size).bfloat16() for _ in range(2)]

        self.prompts, self.slots, self.kv, self.lens = prompts, [], [], []
        at = len(prompts)
        for i, (p, o) in enumerate(zip(prompts, own)):
            if p:
                dgt.kv_reserve(c, i32(i), i32(p), status=st)
                dgt.kv_append(c, self.layer, *rows(p), i32(i), i32(0), cu=i32(0, p), status=st)
            for n in o:
                self.slots.append(at)
                if n is None:
                    self.kv.append(None)
                    self.lens.append(0)
                else:
                    dgt.kv_fork(c, i32(i), i32(at), status=st)
                    if n:
                        start = dgt.kv_reserve(c, i32(at), i32(n), status=st)
                        dgt.kv_append(c, self.layer, *rows(n), i32(at), start, cu=i32(0, n), status=st)
                    total = p + n
                    self.lens.append(total)
                    self.kv.append([x.double() for x in dgt.kv_read(c, self.layer, i32(at), i32(0), i32(0, total), total)])
                at += 1
        assert dgt.read_status(st) == 0
        self.groups = cu_of([len(o) for o in own])

    def q(self, rows, hq):
        return torch.randn(rows, hq, self.dim, generator=self.g, device="cuda").bfloat16()

    def call(self, q, counts, shared=None, always=True, **kw):
        one = all(n == 1 for n in counts)
        many = len(self.prompts) > 1
        return dgt.kv_attention_shared(self.c, self.layer, q, i32(*self.slots), i32(*range(len(self.prompts))),
                                       i32(*(shared or self.prompts)), groups=i32(*self.groups) if many else None,
                                       cu=None if one else i32(*cu_of(counts)), always=always, **kw)

    def check(self, q, counts, shared=None, scale=None, **kw):
        st = i32(0)
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        out = self.call(q, counts, shared, scale=scale, lse=lse, status=st, **kw)
        assert dgt.read_status(st) == 0
        sc = self.dim ** -0.5 if scale is None else scale
        rep = q.shape[1] // self.hk
        cu = cu_of(counts)
        for b, n in enumerate(counts):
            y, z = out[cu[b]:cu[b + 1]].double(), lse[cu[b]:cu[b + 1]].double()
            if self.kv[b] is None:
                assert not bool(y.any()) and bool((z == -INF).all())
                continue
            k, v = (x.repeat_interleave(rep, 1) for x in self.kv[b])
            qq = q[cu[b]:cu[b + 1]].double()
            t = torch.einsum("nhd,thd->hnt", qq, k) * sc
            size = torch.einsum("nhd,thd->hnt", qq.abs(), k.abs()) * abs(sc)
            total = self.lens[b]
            ahead = torch.arange(total, device="cuda") > torch.arange(total - n, total, device="cuda")[:, None]
            t, size = t.masked_fill(ahead, -INF), size.masked_fill(ahead, 0.0)
            w = torch.softmax(t, -1)
            ref = torch.einsum("hnt,thd->nhd", w, v)
            mag = torch.einsum("hnt,thd->nhd", w, v.abs())
            lost = total * 2.0 ** -29 * v.abs().amax((0, 2))[None, :, None]
            assert bool(((y - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -10 * mag + lost).all()), b
            want = torch.logsumexp(t, -1).T
            assert bool(((z - want).abs() <= self.dim * 2.0 ** -24 * size.amax(-1).T + 2.0 ** -17).all()), b
        return out


HEADS = [(24, 8, 128), (16, 8, 256), (32, 8, 64), (1, 1, 64), (5, 1, 128), (40, 2, 128), (33, 1, 256), (64, 1, 64)]


@pytest.mark.parametrize("hq,hk,dim", HEADS)
@pytest.mark.parametrize("prompt", [1, 63, 64, 65, 128, 1000])
def test_one_group(hq, hk, dim, prompt):
    f = Forks([prompt], [[1, 3, 70, 200, 1]], hk, dim, seed=prompt + hq)
    f.check(f.q(5, hq), [1] * 5)


@pytest.mark.parametrize("hq,hk,dim", HEADS[:4])
def test_groups_of_all_sizes_with_idle_sequences(hq, hk, dim):
    own = [[1], [5, None, 64, 1], [None], [700, 2], [1] * 20, [65, 63, 64]]
    f = Forks([3000, 130, 500, 64, 777, 10], own, hk, dim, layers=2, seed=dim)
    f.check(f.q(sum(map(len, own)), hq), [1] * sum(map(len, own)))


@pytest.mark.parametrize("hq,hk,dim", HEADS[:6])
@pytest.mark.parametrize("new", [2, 5, 30])
def test_several_rows_a_sequence(hq, hk, dim, new):
    own = [[new, new + 10, None, new + 100], [new + 64]]
    counts = [new, 1, 1, new, max(1, new - 1)]
    f = Forks([1500, 200], own, hk, dim, seed=new)
    f.check(f.q(sum(counts), hq), counts)


@pytest.mark.parametrize("hq,hk,dim", [(24, 8, 128), (16, 8, 256), (8, 8, 64), (12, 1, 128)])
def test_prompts_behind_a_shared_document(hq, hk, dim):
    counts = [300, 513, 64]
    f = Forks([2100], [counts], hk, dim, seed=7)
    f.check(f.q(sum(counts), hq), counts)


def test_many_sequences_of_one_prompt():
    f = Forks([4000], [[1 + i % 90 for i in range(200)]], 2, 128, seed=3)
    f.check(f.q(200, 12), [1] * 200)


def test_many_small_groups():
    own = [[1, 1 + g % 70] for g in range(150)]
    f = Forks([64 * (1 + g % 3) + g % 5 for g in range(150)], own, 1, 64, seed=5)
    f.check(f.q(300, 4), [1] * 300)


@pytest.mark.parametrize("hq,hk,dim", [(24, 8, 128), (16, 8, 256), (32, 8, 64)])
def test_shared_by_itself_where_it_pays(hq, hk, dim):
    """Without `always`: groups that are worth it beside one that is not, and in a cache whose tables could hold more
    than any of them has."""
    own = [[1 + i % 70 for i in range(70)], [2, 1], [1] * 60]
    f = Forks([9000, 300, 8100], own, hk, dim, seed=dim + 1, max_pages=400)
    f.check(f.q(132, hq), [1] * 132, always=False)
    few = Forks([500], [[1, 20, 3]], hk, dim, seed=dim + 2, max_pages=4000)
    few.check(few.q(3, hq), [1] * 3, always=False)


def test_fewer_shared_tokens_than_there_are():
    f = Forks([1000], [[1, 80, 20]], 4, 128, seed=1)
    for shared in (0, 1, 63, 64, 500, 999, 1000):
        f.check(f.q(3, 8), [1] * 3, shared=[shared])


def test_scales_of_the_scores():
    f = Forks([640], [[1, 40, 7]], 2, 64, seed=2)
    q = f.q(3, 8)
    for scale in (0.0, 1.0, -0.3, 2.0):
        f.check(q, [1] * 3, scale=scale)


def test_values_of_very_different_size_before_and_behind():
    """A tail whose scores dwarf the prompt's, and the other way round: one part's weight vanishes, no NaN."""
    f = Forks([256], [[64, 64]], 1, 64, seed=4, spread=0.0)
    q = f.q(2, 4)
    f.check(q, [1, 1], scale=40.0)
    f.check(q, [1, 1], scale=-40.0)


@pytest.mark.parametrize("hq,hk,dim", HEADS[:3])
def test_the_same_as_the_attention_that_shares_nothing(hq, hk, dim):
    f = Forks([900], [[3] * 7], hk, dim, seed=9)
    q = f.q(7, hq)
    a, b = f.call(q, [1] * 7), dgt.kv_attention(f.c, 0, q, i32(*f.slots))
    # each is within 2^-8 of itself and 2^-10 of the mean of |v| of the same value
    mag = torch.stack([kv[1].abs().mean(0).repeat_interleave(hq // hk, 0) for kv in f.kv])
    assert bool(((a.double() - b.double()).abs() <= 2.0 ** -7 * b.double().abs() * 1.01 + 2.0 ** -7 * mag).all())
    assert torch.equal(a, f.call(q, [1] * 7))


def test_strided_queries_and_given_outputs():
    f = Forks([300], [[1, 20, 5]], 2, 128, seed=6)
    wide = torch.randn(3, 8 + 4, 128, device="cuda").bfloat16()
    q = wide[:, :8]
    out = torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    ws = dgt.kv_attention_shared_workspace(f.c, 8, 1, 3, 3)
    got = f.check(q, [1] * 3, out=out, ws=ws)
    assert got is out and torch.equal(out, f.call(q.contiguous(), [1] * 3, ws=ws))


def test_one_workspace_for_calls_of_all_sizes():
    big = Forks([2000, 100], [[1] * 30, [9, 2]], 4, 128, seed=8)
    ws = dgt.kv_attention_shared_workspace(big.c, 16, 2, 32, 500)
    small = Forks([70], [[1, 2]], 4, 128, seed=9)
    for _ in range(2):
        big.check(big.q(32, 16), [1] * 32, ws=ws)
        small.check(small.q(2, 8), [1, 1], ws=ws)


def test_rows_that_are_not_finite():
    f = Forks([200], [[1, 5, 9]], 2, 64, seed=11)
    q = f.q(3, 4)
    q[1, 2, 7] = float("nan")
    q[2, 0, 0] = INF
    y = f.call(q, [1] * 3)
    bad = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    bad[1, 2] = bad[2, 0] = True
    assert torch.equal(y.isnan().all(-1), bad) and torch.equal(y.isnan().any(-1), bad)


def test_a_poisoned_page_reaches_only_who_sees_it():
    f = Forks([130], [[70, 5]], 1, 64, seed=12)
    # an own page of the first sequence
    f.c.v_scale[0, int(f.c.table[f.slots[0], 3])] = float("nan")
    y = f.call(f.q(2, 2), [1, 1])
    assert bool(y[0].isnan().all()) and not bool(y[1].isnan().any())
    f.c.v_scale[0, int(f.c.table[0, 0])] = float("nan")
    assert bool(f.call(f.q(2, 2), [1, 1]).isnan().all())


def test_what_the_device_reports():
    f = Forks([300, 200], [[1, 4], [2, 3]], 2, 64, seed=13)
    q = f.q(4, 4)
    good = f.call(q, [1] * 4)

    def call(seqs=f.slots, prefix=(0, 1), shared=(300, 200), groups=(0, 2, 4)):
        st = i32(0)
        y = dgt.kv_attention_shared(f.c, 0, q, i32(*seqs), i32(*prefix), i32(*shared), groups=i32(*groups), status=st,
                                    always=True)
        return y, dgt.read_status(st)

    y, st = call()
    assert st == 0 and torch.equal(y, good)
    # more shared tokens than the second prefix holds, prefixes that are no sequences: the first group stays
    for kw in (dict(shared=(300, 201)), dict(shared=(300, -1)), dict(prefix=(0, 99)), dict(prefix=(0, -1))):
        y, st = call(**kw)
        assert st == -1 and torch.equal(y[:2], good[:2])
    # a sequence that is none, and one whose new row is inside the shared pages
    y, st = call(seqs=(f.slots[0], 77, f.slots[2], f.slots[3]))
    assert st == -1 and not bool(y[1].any())
    assert torch.equal(y[0], good[0])
    f.c.lens[f.slots[1]] = 256
    y, st = call()
    assert st == -1 and not bool(y[1].any()) and torch.equal(y[2:], good[2:])
    f.c.lens[f.slots[1]] = 304
    # groups that run past the batch, or leave entries out
    for groups in ((0, 2, 9), (0, 2, -5), (1, 2, 4), (0, 2, 3)):
        y, st = call(groups=groups)
        assert st == -1 and torch.equal(y[1], good[1])


def test_a_wait_that_runs_out_is_reported():
    for new in (1, 40):
        f = Forks([1000], [[new, new]], 2, 128, seed=14)
        q, st = f.q(2 * new, 16), i32(0)
        f.call(q, [new] * 2, status=st, test_wait_polls=0)
        torch.cuda.synchronize()
        assert dgt.read_status(st) in (0, -5)
        f.check(q, [new] * 2)


def test_a_stream_and_a_graph_that_follows_the_lengths():
    f = Forks([400], [[1, 1, 1]], 2, 128, seed=15, max_pages=12)
    q = f.q(3, 8)
    want = f.call(q, [1] * 3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = f.call(q, [1] * 3, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    seqs, ones = i32(*f.slots), i32(1, 1, 1)
    ws = dgt.kv_attention_shared_workspace(f.c, 8, 1, 3, 3)
    k, v = (torch.randn(3, 2, 128, device="cuda").bfloat16() for _ in range(2))
    out = torch.empty_like(q)
    prefix, shared = i32(0), i32(400)
    start = i32(0, 0, 0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dgt.kv_reserve(f.c, seqs, ones, start=start)
        dgt.kv_append(f.c, 0, k, v, seqs, start)
        dgt.kv_attention_shared(f.c, 0, q, seqs, prefix, shared, out=out, ws=ws, always=True)
    for _ in range(70):
        g.replay()
    f.lens = [471] * 3
    f.kv = [[x.double() for x in dgt.kv_read(f.c, 0, i32(s), i32(0), i32(0, 471), 471)] for s in f.slots]
    assert torch.equal(f.check(q, [1] * 3), out)


def test_empty_calls_and_refusals():
    f = Forks([100], [[1, 2]], 2, 64, seed=16)
    q = f.q(2, 4)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert dgt.kv_attention_shared(f.c, 0, q[:0], none, i32(0), i32(100)).shape == (0, 4, 64)
    a = (f.c, 0, q, i32(*f.slots), i32(0), i32(100))
    with pytest.raises(ValueError):
        dgt.kv_attention_shared(*a[:4], i32(0, 0), i32(100, 100))
    with pytest.raises(ValueError):
        dgt.kv_attention_shared(*a[:4], i32(0, 0), i32(100))
    with pytest.raises(ValueError):
        dgt.kv_attention_shared(*a, groups=i32(0, 1, 2))
    with pytest.raises(ValueError):
        dgt.kv_attention_shared(f.c, 0, f.q(2, 4)[:, :, :32].contiguous(), *a[3:])
    with pytest.raises(ValueError):
        dgt.kv_attention_shared(*a, out=q.float())
    for kw in (dict(ws=torch.zeros(256, dtype=torch.uint8, device="cuda")),):
        with pytest.raises(dgt.DgtError):
            dgt.kv_attention_shared(*a, **kw)
    with pytest.raises(dgt.DgtError):
        dgt.kv_attention_shared(f.c, 1, *a[2:])
