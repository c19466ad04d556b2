"""Attention over the paged 8-bit cache against 64 bits.

Tolerance of an output element: the bf16 rounding, 2^-8 of it, and of the
weighted mean of |v|: 2^-11 for the weights' fp16 rounding and as much again
for what the scores' fp32 sums (dim * 2^-24 of the largest sum of |q||k|, here
below 60) and the exponential leave in the weights and their sum.  The lse:
those sums' worst case, dim * 2^-24 of the largest sum of |q||k|, and 2^-18."""
import numpy as np
import pytest

import kv_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def dgt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import decode_gemv_tensor_gb300 as d
    d.lib()
    return d


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def f64(t):
    return t.double().cpu().numpy()


def rand(g, *shape, scale=1.0):
    return torch.from_numpy((scale * g.normal(size=shape)).astype(np.float32)).cuda().bfloat16()


class Setup:
    """Sequences of the given lengths in scattered pages, filled with random keys and values."""

    def __init__(self, dgt, g, lens, kv_heads, dim, layers=1, spread=1.0, seqs=None):
        self.dgt, self.lens = dgt, lens
        need = [-(-n // 64) for n in lens]
        self.seqs = list(range(len(lens))) if seqs is None else seqs
        c = dgt.KvCache(layers, sum(need) + 2, kv_heads, dim, max_seqs=max(self.seqs + [0]) + 1,
                        max_pages=max(need + [1]) + 1)
        perm = g.permutation(sum(need) + 2)
        at = 0
        self.kv = []
        for s, n, m in zip(self.seqs, lens, need):
            c.table[s, :m] = i32(perm[at:at + m].tolist())
            at += m
            c.lens[s] = n
            if n:
                size = np.exp2(spread * g.normal(size=(n, kv_heads, 1)))
                k = torch.from_numpy((g.normal(size=(n, kv_heads, dim)) * size).astype(np.float32)).cuda().bfloat16()
                v = torch.from_numpy((g.normal(size=(n, kv_heads, dim)) * size).astype(np.float32)).cuda().bfloat16()
                dgt.kv_append(c, layers - 1, k, v, i32([s]), i32([0]), cu=i32([0, n]))
                self.kv.append([f64(x) for x in dgt.kv_read(c, layers - 1, i32([s]), i32([0]), i32([0, n]), n)])
            else:
                self.kv.append([np.zeros((0, kv_heads, dim))] * 2)
        self.c, self.layer = c, layers - 1

    def check(self, q, counts, window=0, sinks=0, scale=None, rows=None):
        """Every output row (or the given ones) against the reference."""
        dgt, dim = self.dgt, q.shape[2]
        cu = np.concatenate([[0], np.cumsum(counts)]).astype(int)
        one = all(n == 1 for n in counts)
        st = i32([0])
        lse = torch.full((q.shape[0], q.shape[1]), 7.0, device="cuda")
        out = dgt.kv_attention(self.c, self.layer, q, i32(self.seqs), cu=None if one else i32(cu.tolist()),
                               scale=scale, window=window, sinks=sinks, lse=lse, status=st)
        assert dgt.read_status(st) == 0
        y, z, qq = f64(out), f64(lse), f64(q)
        for b, n in enumerate(counts):
            pick = range(n) if rows is None else [i for i in rows if i < n]
            for i in pick:
                r = cu[b] + i
                first = self.lens[b] - n + i
                if self.lens[b] == 0 or first < 0:
                    assert not y[r].any() and np.isneginf(z[r]).all()
                    continue
                ref, lref, mag, big = R.attention(qq[r:r + 1], *self.kv[b], first, window, sinks,
                                                  dim ** -0.5 if scale is None else scale)
                assert (np.abs(y[r] - ref[0]) <= 2.0 ** -8 * np.abs(ref[0]) + 2.0 ** -10 * mag[0]).all(), (b, i)
                assert (np.abs(z[r] - lref[0]) <= dim * 2.0 ** -24 * big[0] + 2.0 ** -18).all(), (b, i)
        return out


HEADS = [(24, 8, 128), (16, 8, 256), (32, 8, 64), (1, 1, 64), (5, 1, 128), (40, 2, 128), (33, 1, 256), (64, 1, 64)]


@pytest.mark.parametrize("hq,hk,dim", HEADS)
@pytest.mark.parametrize("length", [1, 2, 63, 64, 65, 129, 777])
def test_one_row(dgt, hq, hk, dim, length):
    g = np.random.default_rng(hq + dim + length)
    s = Setup(dgt, g, [length], hk, dim)
    s.check(rand(g, 1, hq, dim), [1])


@pytest.mark.parametrize("hq,hk,dim", HEADS[:5])
def test_a_ragged_batch_with_idle_slots(dgt, hq, hk, dim):
    # slots in another order, other layers beside, empty sequences
    g = np.random.default_rng(dim)
    lens = [300, 0, 1, 64, 1000, 65, 0, 128, 511, 2000]
    s = Setup(dgt, g, lens, hk, dim, layers=2, seqs=[3, 1, 12, 0, 7, 5, 2, 9, 8, 4])
    s.check(rand(g, len(lens), hq, dim), [1] * len(lens))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (64, 0), (63, 64), (100, 4), (128, 70), (640, 16),
                                          (1000, 0), (4096, 4), (7, 2000)])
@pytest.mark.parametrize("hq,hk,dim", HEADS[:3])
def test_window_and_sinks(dgt, window, sinks, hq, hk, dim):
    g = np.random.default_rng(window + sinks)
    lens = [777, 64, 3, 129]
    s = Setup(dgt, g, lens, hk, dim)
    s.check(rand(g, 4, hq, dim), [1] * 4, window, sinks)
    s.check(rand(g, 26, hq, dim), [20, 2, 3, 1], window, sinks)


@pytest.mark.parametrize("hq,hk,dim", HEADS)
@pytest.mark.parametrize("counts,lens", [([5, 5, 1, 3], [100, 5, 64, 70]), ([13], [13]), ([64, 1], [64, 500]),
                                         ([2, 0, 7], [700, 3, 64])])
def test_several_rows(dgt, hq, hk, dim, counts, lens):
    g = np.random.default_rng(sum(counts) + dim)
    s = Setup(dgt, g, lens, hk, dim)
    s.check(rand(g, sum(counts), hq, dim), counts)


@pytest.mark.parametrize("hq,hk,dim", HEADS[:3] + HEADS[4:6])
@pytest.mark.parametrize("counts,lens,window,sinks", [([200, 131], [200, 700], 0, 0), ([300], [1000], 130, 5),
                                                      ([129, 1, 64], [129, 400, 65], 0, 0), ([257], [321], 64, 0)])
def test_prompts(dgt, hq, hk, dim, counts, lens, window, sinks):
    g = np.random.default_rng(sum(counts) + dim)
    s = Setup(dgt, g, lens, hk, dim)
    pick = sorted(set([0, 1, 2, 40, 41, 42, 43, 63, 64, 65, 127, 128, 129, 199, 255, 256, 299] +
                      [c - 1 for c in counts] + [c - 2 for c in counts]) & set(range(300)))
    s.check(rand(g, sum(counts), hq, dim), counts, window, sinks, rows=pick)


def test_more_rows_than_tokens(dgt):
    # rows that stand before the sequence begins see nothing
    g = np.random.default_rng(11)
    s = Setup(dgt, g, [3, 100], 2, 64)
    s.check(rand(g, 12, 4, 64), [8, 4])


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_long_context_is_split_and_joined(dgt, dim):
    g = np.random.default_rng(dim)
    s = Setup(dgt, g, [20011, 5], 2, dim)
    s.check(rand(g, 2, 6, dim), [1, 1])
    s.check(rand(g, 4, 6, dim), [3, 1], 5000, 3)


def test_scores_of_any_size(dgt):
    # queries far larger and smaller than a row's other elements, scores in the hundreds, a flat softmax
    g = np.random.default_rng(4)
    s = Setup(dgt, g, [300], 1, 128)
    q = rand(g, 1, 6, 128)
    q[0, 0] *= 2.0 ** -120
    q[0, 1] *= 2.0 ** -20
    q[0, 2] = 0
    q[0, 3, ::2] *= 2.0 ** -14
    s.check(q, [1])
    s.check(q, [1], scale=0.0)
    big = rand(g, 1, 6, 128, scale=4.0)
    out = f64(dgt.kv_attention(s.c, 0, big, i32([0]), scale=1.0))
    # scores near 100 of sums of |q||k| near 1000: the weights follow the scores' fp32 sums, 2^-24 * 128 of those
    ref, _, mag, sums = R.attention(f64(big), *s.kv[0], 299, 0, 0, 1.0)
    assert (np.abs(out - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + 2.0 ** -16 * sums[..., None]) * mag).all()


def test_value_scales_far_apart(dgt):
    # pages whose values differ by 2^60 between each other, the small ones where the weight is
    g = np.random.default_rng(6)
    c = dgt.KvCache(1, 3, 1, 128, max_seqs=1, max_pages=3)
    c.table[0] = i32([2, 0, 1])
    c.lens[0] = 190
    k, v = rand(g, 190, 1, 128, scale=0.1), rand(g, 190, 1, 128)
    v[:64] *= 2.0 ** 40
    v[64:128] *= 2.0 ** -30
    v[128:] = 0
    dgt.kv_append(c, 0, k, v, i32([0]), i32([0]), cu=i32([0, 190]))
    kv = [f64(x) for x in dgt.kv_read(c, 0, i32([0]), i32([0]), i32([0, 190]), 190)]
    for window in (0, 100, 62):
        q = rand(g, 1, 2, 128)
        ref, _, mag, _ = R.attention(f64(q), *kv, 189, window, 0, 128 ** -0.5)
        y = f64(dgt.kv_attention(c, 0, q, i32([0]), window=window))
        assert (np.abs(y - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * mag).all()


@pytest.mark.parametrize("hq,hk,dim", HEADS[:3])
@pytest.mark.parametrize("longest", [70, 900])
def test_more_sequences_than_are_described_at_a_time(dgt, hq, hk, dim, longest):
    g = np.random.default_rng(longest + dim)
    lens = g.integers(0, longest + 1, size=170).tolist()
    s = Setup(dgt, g, lens, hk, dim)
    s.check(rand(g, 170, hq, dim), [1] * 170)
    s.check(rand(g, 170, hq, dim), [1] * 170, 65, 2)


@pytest.mark.parametrize("hq,hk,dim", HEADS[:3])
def test_more_prompts_than_are_described_at_a_time(dgt, hq, hk, dim):
    # some of them without rows, some without tokens, some with more rows than tokens
    g = np.random.default_rng(dim + 1)
    counts = g.integers(0, 120, size=90).tolist()
    lens = [int(n) + int(x) for n, x in zip(counts, g.integers(-20, 300, size=90))]
    lens = [max(n, 0) for n in lens]
    s = Setup(dgt, g, lens, hk, dim)
    s.check(rand(g, sum(counts), hq, dim), counts, rows=[0, 19, 20, 21, 63, 64, 100])
    s.check(rand(g, sum(counts), hq, dim), counts, 70, 3, rows=[0, 20, 64, 100])


def test_a_prompt_of_many_tiles(dgt):
    g = np.random.default_rng(77)
    s = Setup(dgt, g, [6100], 1, 128)
    q = rand(g, 6000, 3, 128)
    s.check(q, [6000], rows=[0, 85, 86, 2047, 2048, 5461, 5462, 5999])
    s.check(q, [6000], 500, 66, rows=[0, 85, 86, 2047, 2048, 5461, 5462, 5999])


@pytest.mark.parametrize("hq,hk,dim", HEADS[:3])
def test_a_prompt_before_the_sequence_begins(dgt, hq, hk, dim):
    g = np.random.default_rng(dim + 2)
    s = Setup(dgt, g, [3, 100, 0], hk, dim)
    s.check(rand(g, 450, hq, dim), [200, 150, 100])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 100])
def test_a_scale_below_zero(dgt, dim, rows):
    g = np.random.default_rng(dim + rows)
    s = Setup(dgt, g, [300], 2, dim)
    s.check(rand(g, rows, 4, dim), [rows], scale=-0.06)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_prompt_of_queries_of_any_size(dgt, dim):
    # many rows keep a query to 2^-17 of the row's largest element: that, times the sum of |k|, is what a score
    # may be off besides its sums
    g = np.random.default_rng(dim + 5)
    s = Setup(dgt, g, [200], 1, dim)
    q = rand(g, 100, 4, dim)
    q[:, 0] *= 2.0 ** -120
    q[:, 1] *= 2.0 ** 10
    q[:, 2] = 0
    q[:, 3, ::2] *= 2.0 ** -14
    scale = dim ** -0.5 * torch.tensor([1, 2.0 ** -10, 1, 1], dtype=torch.float64)
    for h in range(4):
        part = q[:, h:h + 1].contiguous()
        lse = torch.empty(100, 1, device="cuda")
        out = dgt.kv_attention(s.c, 0, part, i32([0]), cu=i32([0, 100]), scale=float(scale[h]), lse=lse)
        ref, lref, mag, big = R.attention(f64(part), *s.kv[0], 100, 0, 0, float(scale[h]))
        keys = np.abs(s.kv[0][0]).sum(2).max() * float(scale[h])
        off = dim * 2.0 ** -24 * big + 2.0 ** -17 * np.abs(f64(part)).max(2) * keys
        assert (np.abs(f64(lse) - lref) <= off + 2.0 ** -18).all()
        assert (np.abs(f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + 2 * off[..., None]) * mag).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_of_a_prompt_that_are_not_finite(dgt, dim):
    g = np.random.default_rng(dim + 8)
    s = Setup(dgt, g, [230], 1, dim)
    q = rand(g, 100, 4, dim)
    clean = dgt.kv_attention(s.c, 0, q, i32([0]), cu=i32([0, 100]))
    for bad in (float("nan"), float("-inf")):
        p = q.clone()
        p[40, 1, 5] = bad
        got = dgt.kv_attention(s.c, 0, p, i32([0]), cu=i32([0, 100]))
        assert torch.isnan(got[40, 1]).all()
        got[40, 1] = clean[40, 1]
        assert torch.equal(got, clean)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("side", [0, 1])
def test_what_a_row_does_not_see_adds_nothing(dgt, dim, side):
    # a poisoned page: rows that see one of its tokens give NaN, rows that see none are as ever; what stands past
    # the end of a sequence does not count
    g = np.random.default_rng(dim + side)
    s = Setup(dgt, g, [300], 1, dim)
    q = rand(g, 100, 2, dim)                       # positions 200..299
    clean = dgt.kv_attention(s.c, 0, q, i32([0]), cu=i32([0, 100]), window=50, sinks=3)
    page = int(s.c.table[0, 2])                    # positions 128..191
    scale = (s.c.k_scale, s.c.v_scale)[side]
    was = scale[0, page].clone()
    scale[0, page] = float("nan")
    got = dgt.kv_attention(s.c, 0, q, i32([0]), cu=i32([0, 100]), window=50, sinks=3)
    sees = torch.arange(200, 300) - 49 <= 191
    assert torch.isnan(got[sees]).all()
    assert torch.equal(got[~sees], clean[~sees])
    scale[0, page] = was
    # stale tokens behind the end, in the last page: their codes and a page beyond
    tail = int(s.c.table[0, 4])                    # positions 256..319, 44 of them held
    off = [d * 64 + t for d in range(dim) for t in range(44, 64)]
    s.c.v[0, tail, 0, off] = 0x7E
    assert torch.equal(dgt.kv_attention(s.c, 0, q, i32([0]), cu=i32([0, 100]), window=50, sinks=3), clean)


def test_rows_of_q_that_are_not_finite(dgt):
    g = np.random.default_rng(8)
    s = Setup(dgt, g, [130], 1, 64)
    q = rand(g, 1, 4, 64)
    clean = dgt.kv_attention(s.c, 0, q, i32([0]))
    for bad in (float("nan"), float("inf")):
        p = q.clone()
        p[0, 1, 5] = bad
        got = dgt.kv_attention(s.c, 0, p, i32([0]))
        assert torch.isnan(got[0, 1]).all()
        assert torch.equal(got[0, [0, 2, 3]], clean[0, [0, 2, 3]])


def test_strides_streams_graphs_and_repeats(dgt):
    # q as a slice of stacked rows, a stream and a workspace of its own, a captured graph that follows lens,
    # and the same bits every time
    g = np.random.default_rng(9)
    s = Setup(dgt, g, [500, 900], 2, 128)
    wide = rand(g, 2, 10, 128)
    q = wide[:, 2:8]
    ref = dgt.kv_attention(s.c, 0, q.contiguous(), i32([0, 1]))
    ws = dgt.kv_attention_workspace(s.c, 6, 2, 2)
    side = torch.cuda.Stream()
    out = torch.empty_like(ref)
    seqs = i32([0, 1])
    torch.cuda.synchronize()
    for _ in range(3):
        dgt.kv_attention(s.c, 0, q, seqs, out=out, ws=ws, stream=side)
        side.synchronize()
        assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dgt.kv_attention(s.c, 0, q, seqs, out=out, ws=ws)
    for lens in ([500, 900], [1, 64], [0, 899], [500, 900]):
        s.c.lens.copy_(i32(lens))
        want = dgt.kv_attention(s.c, 0, q, seqs)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), lens
    # the same workspace for calls of other sizes
    p = rand(g, 2, 2, 128)
    s.c.lens.copy_(i32([333, 64]))
    want = dgt.kv_attention(s.c, 0, p, i32([1, 0]))
    assert torch.equal(dgt.kv_attention(s.c, 0, p, i32([1, 0]), ws=ws), want)


def test_what_the_device_finds_wrong(dgt):
    g = np.random.default_rng(10)
    s = Setup(dgt, g, [100, 200], 1, 64)
    q = rand(g, 2, 2, 64)
    good = dgt.kv_attention(s.c, 0, q, i32([0, 1]))
    st = i32([0])
    got = dgt.kv_attention(s.c, 0, q, i32([0, 9]), status=st)
    assert dgt.read_status(st) == -1 and torch.equal(got[0], good[0]) and not got[1].any()
    st.zero_()
    s.c.table[1, 1] = -1                       # a page that is not there: its tokens are not seen
    got = dgt.kv_attention(s.c, 0, q, i32([0, 1]), status=st)
    assert dgt.read_status(st) == -1 and torch.equal(got[0], good[0]) and torch.isfinite(got.float()).all()
    st.zero_()
    s.c.lens[1] = 10 ** 6
    got = dgt.kv_attention(s.c, 0, q, i32([0, 1]), status=st)
    assert dgt.read_status(st) == -1 and torch.equal(got[0], good[0])
    for bad in (dict(window=-1), dict(sinks=-1), dict(out=torch.empty(2, 2, 64, device="cuda")),
                dict(lse=torch.empty(3, device="cuda")), dict(cu=i32([0, 2])), dict(q=q.half())):
        kw = dict(q=q, seqs=i32([0, 1]))
        kw.update(bad)
        with pytest.raises(ValueError):
            dgt.kv_attention(s.c, 0, **kw)
    with pytest.raises(dgt.DgtError) as e:
        dgt.kv_attention(s.c, 0, q, i32([0, 1]), ws=torch.zeros(0, dtype=torch.uint8, device="cuda")) \
            if dgt.kv_attention_workspace(s.c, 2, 2, 2).numel() > 256 else dgt.kv_attention(s.c, 1, q, i32([0, 1]))
    assert e.value.code == -1


def test_offsets_past_32_bits(dgt):
    # a cache of more than 2^32 bytes a side: blocks on either side of the border
    pages, dim = 70000, 256
    c = dgt.KvCache(2, pages, 2, dim, max_seqs=1, max_pages=3)
    c.table[0] = i32([69999, 3, 69998])
    c.lens[0] = 150
    g = np.random.default_rng(12)
    k, v, q = rand(g, 150, 2, dim), rand(g, 150, 2, dim), rand(g, 1, 4, dim)
    dgt.kv_append(c, 1, k, v, i32([0]), i32([0]), cu=i32([0, 150]))
    kv = [f64(x) for x in dgt.kv_read(c, 1, i32([0]), i32([0]), i32([0, 150]), 150)]
    side = R.Side(3, 2, dim)
    side.append([0, 1, 2], 0, f64(k))
    assert np.array_equal(kv[0], side.read([0, 1, 2], 0, 150))
    ref, _, mag, _ = R.attention(f64(q), *kv, 149, 0, 0, dim ** -0.5)
    y = f64(dgt.kv_attention(c, 1, q, i32([0])))
    assert (np.abs(y - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * mag).all()
    dgt.kv_copy_pages(c, i32([69998, 3]), i32([5, 69997]))
    c.table[0] = i32([69999, 69997, 5])
    assert torch.equal(dgt.kv_attention(c, 1, q, i32([0])).view(torch.int16).cpu(),
                       torch.from_numpy(y).bfloat16().view(torch.int16))


@pytest.mark.parametrize("polls", [0, 1])
@pytest.mark.parametrize("dim,rows", [(64, 1), (128, 1), (256, 1), (128, 9), (64, 100), (128, 100), (256, 100)])
def test_a_wait_that_runs_out_is_reported(dgt, dim, rows, polls):
    # the test hook: waits give up after `polls` polls, the status says so, and the next call is as ever
    g = np.random.default_rng(dim)
    s = Setup(dgt, g, [3000, 70], 2, dim)
    counts = [rows, 1]
    q, cu = rand(g, rows + 1, 6, dim), i32([0, rows, rows + 1])
    ws = dgt.kv_attention_workspace(s.c, 6, 2, rows + 1)
    want = dgt.kv_attention(s.c, 0, q, i32([0, 1]), cu=cu, ws=ws)
    st = i32([0])
    dgt.kv_attention(s.c, 0, q, i32([0, 1]), cu=cu, ws=ws, status=st, test_wait_polls=polls)
    code = dgt.read_status(st)
    assert code == -5 if polls == 0 else code in (0, -5)
    assert torch.equal(dgt.kv_attention(s.c, 0, q, i32([0, 1]), cu=cu, ws=ws), want)
