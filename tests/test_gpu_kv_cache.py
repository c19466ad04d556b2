"""The paged 8-bit cache on the GPU: append and read against the definition
(every value equal), page operations against a step-by-step pool."""
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


def rows(g, n, heads, dim, log2=0.0):
    x = g.normal(size=(n, heads, dim)) * np.exp2(log2 + 2 * g.normal(size=(n, heads, 1)))
    return torch.from_numpy(x.astype(np.float32)).cuda().bfloat16()


def place(cache, tables, lens):
    """Tables given by hand."""
    for s, t in enumerate(tables):
        cache.table[s, :len(t)] = i32(t)
        cache.refs[torch.tensor(t, dtype=torch.long, device="cuda")] = 1
    cache.lens[:len(lens)] = i32(lens)


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads", [1, 3])
@pytest.mark.parametrize("steps", [[1], [64], [65, 1, 1], [3, 60, 1, 1, 70], [200], [127, 130], [1] * 5 + [59, 64]])
def test_append_and_read_equal_the_definition(dgt, dim, heads, steps):
    # two layers (the other stays as it was), scattered pages, scales that grow from call to call
    g = np.random.default_rng(dim + heads + sum(steps))
    total = sum(steps)
    np_ = -(-total // 64)
    pages = [int(p) for p in g.permutation(np_ + 3)[:np_]]
    c = dgt.KvCache(2, np_ + 3, heads, dim, max_seqs=2, max_pages=np_ + 1)
    place(c, [[], pages], [0, total])
    st = i32([0])
    ref = [R.Side(np_ + 3, heads, dim) for _ in range(2)]
    at = 0
    for i, n in enumerate(steps):
        kv = [rows(g, n, heads, dim, log2=i - 2.0) for _ in range(2)]
        dgt.kv_append(c, 1, *kv, i32([1]), i32([at]), cu=i32([0, n]), status=st)
        for r, x in zip(ref, kv):
            r.append(pages, at, f64(x))
        at += n
    got = dgt.kv_read(c, 1, i32([1]), i32([0]), i32([0, total]), total, status=st)
    assert dgt.read_status(st) == 0
    for x, r in zip(got, ref):
        assert np.array_equal(f64(x), r.read(pages, 0, total))
    # a part of it, beginning inside a page, and every layer at once
    if total > 70:
        part = dgt.kv_read(c, 1, i32([1]), i32([61]), i32([0, total - 61]), total - 61)
        both = dgt.kv_read(c, None, i32([1]), i32([61]), i32([0, total - 61]), total - 61)
        for p, b, r in zip(part, both, ref):
            assert np.array_equal(f64(p), r.read(pages, 61, total - 61))
            assert torch.equal(b[1], p) and not b[0].any()


def test_append_of_a_ragged_batch_with_strides(dgt):
    # entries of no rows, of one, of many; k and v as slices of stacked rows; positions inside pages
    g = np.random.default_rng(77)
    heads, dim = 4, 128
    counts, starts = [1, 0, 130, 1, 64, 7, 0], [63, 5, 10, 0, 64, 60, 0]
    tables, used = [], 0
    for n, s in zip(counts, starts):
        k = -(-(n + s) // 64)
        tables.append(list(range(used, used + k))[::-1])
        used += k
    c = dgt.KvCache(1, used, heads, dim, max_seqs=8, max_pages=5)
    place(c, tables, [0] * 7)
    ref = [R.Side(used, heads, dim) for _ in range(2)]
    order = [6, 2, 0, 1, 4, 5, 3]
    # what the pages held before
    for s in order:
        if starts[s]:
            kv = [rows(g, starts[s], heads, dim) for _ in range(2)]
            dgt.kv_append(c, 0, *kv, i32([s]), i32([0]), cu=i32([0, starts[s]]))
            for r, x in zip(ref, kv):
                r.append(tables[s], 0, f64(x))
    total = sum(counts)
    cu = np.concatenate([[0], np.cumsum([counts[s] for s in order])])
    wide = rows(g, total, 3 * heads, dim, log2=3.0)
    k, v = wide[:, heads:2 * heads], wide[:, 2 * heads:]
    st = i32([0])
    dgt.kv_append(c, 0, k, v, i32(order), i32([starts[s] for s in order]), cu=i32(cu.tolist()), status=st)
    assert dgt.read_status(st) == 0
    for i, s in enumerate(order):
        if counts[s] == 0:
            continue
        for side, (r, x) in enumerate(zip(ref, (k, v))):
            r.append(tables[s], starts[s], f64(x[cu[i]:cu[i + 1]]))
        n = starts[s] + counts[s]
        for x, r in zip(dgt.kv_read(c, 0, i32([s]), i32([0]), i32([0, n]), n), ref):
            assert np.array_equal(f64(x), r.read(tables[s], 0, n)), s


def test_append_one_row_each_over_many_steps(dgt):
    # single tokens, the decode form, past a page's end: the same as the definition step by step
    g = np.random.default_rng(3)
    heads, dim, B, steps = 2, 64, 3, 70
    tables = [[0, 5], [1, 4], [3, 2]]
    c = dgt.KvCache(1, 6, heads, dim, max_seqs=3, max_pages=2)
    place(c, tables, [0] * 3)
    ref = [R.Side(6, heads, dim) for _ in range(2)]
    for t in range(steps):
        kv = [rows(g, B, heads, dim, log2=t / 16) for _ in range(2)]
        dgt.kv_append(c, 0, *kv, i32([2, 0, 1]), i32([t] * 3))
        for r, x in zip(ref, kv):
            for b, s in enumerate([2, 0, 1]):
                r.append(tables[s], t, f64(x[b:b + 1]))
    for s in range(3):
        for x, r in zip(dgt.kv_read(c, 0, i32([s]), i32([0]), i32([0, steps]), steps), ref):
            assert np.array_equal(f64(x), r.read(tables[s], 0, steps))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_special_values(dgt, dim):
    # zeros, subnormals, the largest values, ties, and values that are not finite (poisoned blocks)
    pages = [1, 0]
    c = dgt.KvCache(1, 2, 2, dim, max_seqs=1, max_pages=2)
    place(c, [pages], [128])
    bits = np.zeros((100, 2, dim), np.uint16)
    bits[0, 0, :8] = [0x0001, 0x8001, 0x007F, 0x0080, 0x8000, 0x0000, 0x3F80, 0x3F88]
    bits[1, 0, :4] = [0x3F84, 0x3F8C, 0xBF84, 0x4380]      # halfway between e4m3 neighbours at scale 1
    bits[70:, 1, :] = 0x0040                                # a block of subnormals only
    k = torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)
    big = bits.copy()
    big[2, 0, 5], big[3, 1, 1] = 0x7E80, 0xFE00             # 2^126, -2^125
    v = torch.from_numpy(big.view(np.int16)).cuda().view(torch.bfloat16)
    ref = [R.Side(2, 2, dim) for _ in range(2)]
    dgt.kv_append(c, 0, k, v, i32([0]), i32([0]), cu=i32([0, 100]))
    for r, x in zip(ref, (k, v)):
        r.append(pages, 0, f64(x))
    for x, r in zip(dgt.kv_read(c, 0, i32([0]), i32([0]), i32([0, 100]), 100), ref):
        assert np.array_equal(f64(x), r.read(pages, 0, 100))
    for bad in (float("nan"), float("inf"), -float("inf")):
        k2, v2 = k[:2].clone(), v[:2].clone()
        k2[0, 1, 3] = bad
        dgt.kv_append(c, 0, k2, v2, i32([0]), i32([100]), cu=i32([0, 2]))
        kk, vv = dgt.kv_read(c, 0, i32([0]), i32([0]), i32([0, 102]), 102)
        nan = torch.isnan(kk)
        assert nan[64:, 1].all() and not nan[:64].any() and not nan[:, 0].any() and not torch.isnan(vv).any()
        # finite codes all the same, and a fresh beginning of the page clears it
        code = c.k.view(torch.int8)
        assert not ((code & 127) == 127).any()
        dgt.kv_append(c, 0, k[:3], v[:3], i32([0]), i32([64]), cu=i32([0, 3]))
        assert not torch.isnan(dgt.kv_read(c, 0, i32([0]), i32([64]), i32([0, 3]), 3)[0]).any()
        dgt.kv_append(c, 0, k[:33], v[:33], i32([0]), i32([67]), cu=i32([0, 33]))


def test_what_the_device_finds_wrong(dgt):
    # slots, positions and pages out of range: reported, skipped, and the rest is done
    c = dgt.KvCache(1, 4, 1, 64, max_seqs=3, max_pages=2)
    place(c, [[0, 1], [2]], [0, 0, 0])
    c.table[1, 1] = 99
    one = torch.ones(4, 1, 64, device="cuda", dtype=torch.bfloat16)
    for seqs, start in (([0, 3, 1, 2], [0, 0, 0, 0]), ([0, -1, 1, 2], [0, 0, 1, 5]), ([0, 1, 1, 0], [0, 64, 0, 128]),
                        ([0, 1, 1, 2], [0, -1, 0, 0])):
        st = i32([0])
        c.k.zero_()
        dgt.kv_append(c, 0, one, one, i32(seqs), i32(start), status=st)
        assert dgt.read_status(st) == -1
        st.zero_()
        got = dgt.kv_read(c, 0, i32([0]), i32([0]), None, 1, status=st)
        assert dgt.read_status(st) == 0 and (got[0] == 1).all() and (got[1] == 1).all()
        dgt.kv_read(c, 0, i32(seqs), i32(start), None, 4, status=st)
        assert dgt.read_status(st) == -1
    with pytest.raises(ValueError):
        dgt.kv_append(c, 0, one, one[:3], i32([0, 1, 2, 0]), i32([0] * 4))
    with pytest.raises(ValueError):
        dgt.kv_append(c, 0, one, one, i32([0, 1, 2, 0]), i32([0] * 3))
    with pytest.raises(dgt.DgtError) as e:
        dgt.kv_append(c, 1, one, one, i32([0, 1, 2, 0]), i32([0] * 4))
    assert e.value.code == -1


# ---- pages ------------------------------------------------------------------
def fill(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    for x in (c.k, c.v):
        x.copy_(torch.randint(0, 120, x.shape, generator=g, device="cuda", dtype=torch.uint8))
    for x in (c.k_scale, c.v_scale):
        x.copy_(torch.rand(x.shape, generator=g, device="cuda"))


def contents(c):
    return [x.clone() for x in (c.k, c.v, c.k_scale, c.v_scale)]


def check(c, pool, want, where):
    assert np.array_equal(c.table.cpu().numpy(), pool.table()), where
    assert c.refs.tolist() == pool.refs and c.lens.tolist() == pool.lens, where
    for a, b in zip(contents(c), want):
        assert torch.equal(a, b), where


@pytest.mark.parametrize("layers,heads,dim,n", [(1, 1, 64, 1), (3, 2, 128, 5), (2, 4, 256, 40)])
def test_copy_pages(dgt, layers, heads, dim, n):
    c = dgt.KvCache(layers, 2 * n + 3, heads, dim, max_seqs=1, max_pages=1)
    fill(c, n)
    perm = np.random.default_rng(n).permutation(2 * n + 3)
    src, dst = perm[:n].tolist(), perm[n:2 * n].tolist()
    want = contents(c)
    for x in want:
        x[:, dst] = x[:, src]
    st = i32([0])
    dgt.kv_copy_pages(c, i32(src), i32(dst), status=st)
    assert dgt.read_status(st) == 0
    for a, b in zip(contents(c), want):
        assert torch.equal(a, b)
    # out of range: reported, nothing moved
    dgt.kv_copy_pages(c, i32([0, 2 * n + 3]), i32([2 * n + 3, 1]), status=st)
    assert dgt.read_status(st) == -1
    for a, b in zip(contents(c), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("seed", range(6))
def test_page_operations_step_by_step(dgt, seed):
    # a random history of reserves, forks, frees and compactions; tables, references, lengths and
    # every byte of the pool after each
    g = np.random.default_rng(seed)
    pages, seqs, width = int(g.integers(20, 90)), 9, 12
    c = dgt.KvCache(2, pages, 2, 64, max_seqs=seqs, max_pages=width)
    fill(c, seed)
    pool = R.Pool(pages, seqs, width)
    want = contents(c)
    st = i32([0])
    for step in range(40):
        op = g.choice(["reserve", "reserve", "reserve", "fork", "free", "compact"])
        if op == "reserve":
            n = int(g.integers(1, seqs + 1))
            who = g.permutation(seqs)[:n].tolist()
            cnt = [int(x) for x in g.choice([0, 1, 1, 5, 63, 64, 65, 200], size=n)]
            r = pool.reserve(who, cnt)
            start = dgt.kv_reserve(c, i32(who), i32(cnt), status=st)
            if r is None:
                assert dgt.read_status(st) == -9 and start.tolist() == [-1] * n
                st.zero_()
            else:
                assert start.tolist() == r[0]
                for a, b in r[1]:
                    for x in want:
                        x[:, b] = x[:, a]
        elif op == "fork":
            empty = [s for s in range(seqs) if not pool.rows[s]]
            full = [s for s in range(seqs) if pool.rows[s]]
            if not empty or not full:
                continue
            n = int(g.integers(1, len(empty) + 1))
            src = [int(x) for x in g.choice(full, size=n)]
            for a, b in zip(src, empty):
                pool.fork(a, b)
            dgt.kv_fork(c, i32(src), i32(empty[:n]), status=st)
        elif op == "free":
            who = g.permutation(seqs)[:int(g.integers(1, 3))].tolist()
            for s in who:
                pool.free(s)
            dgt.kv_free(c, i32(who + who[:1]), status=st)     # twice in the list: freed once
        else:
            moves, live = pool.compact()
            n = i32([0])
            dgt.kv_compact(c, live=n, status=st)
            assert n.item() == live
            for a, b in moves:
                for x in want:
                    x[:, b] = x[:, a]
        assert dgt.read_status(st) == 0
        check(c, pool, want, (step, op))


def test_page_operations_with_many_pages_and_sequences(dgt):
    # the free list past one scan step, 1024 sequences in a call, refs in the thousands
    pages, seqs = 9000, 1200
    c = dgt.KvCache(1, pages, 1, 64, max_seqs=seqs, max_pages=17)
    pool = R.Pool(pages, seqs, 17)
    st = i32([0])
    start = dgt.kv_reserve(c, i32([0]), i32([1000]), status=st)
    pool.reserve([0], [1000])
    c.refs[16:4500] = 1                        # pages in other hands
    for p in range(16, 4500):
        pool.refs[p] = 1
    kids = list(range(1, 1024))
    dgt.kv_fork(c, i32([0] * 1023), i32(kids), status=st)
    for s in kids:
        pool.fork(0, s)
    want = contents(c)
    who = kids + [0]
    start = dgt.kv_reserve(c, i32(who), i32([25] * 1024), status=st)   # 1000 + 25: the shared page and one more
    r = pool.reserve(who, [25] * 1024)
    assert start.tolist() == r[0] and dgt.read_status(st) == 0
    for a, b in r[1]:
        for x in want:
            x[:, b] = x[:, a]
    check(c, pool, want, "reserve")
    dgt.kv_free(c, i32(who), status=st)
    for s in who:
        pool.free(s)
    check(c, pool, want, "free")


def test_page_operations_report_what_is_wrong(dgt):
    c = dgt.KvCache(1, 6, 1, 64, max_seqs=4, max_pages=3)
    pool = R.Pool(6, 4, 3)
    st = i32([0])

    def refused(code):
        assert dgt.read_status(st) == code
        st.zero_()
        check(c, pool, want, "unchanged")

    dgt.kv_reserve(c, i32([0, 1]), i32([100, 10]), status=st)
    pool.reserve([0, 1], [100, 10])
    want = contents(c)
    assert dgt.read_status(st) == 0
    for seqs, cnt, code in (([2, 4], [1, 1], -1), ([2, -1], [1, 1], -1), ([2, 2], [1, 1], -1), ([2, 3], [1, -1], -1),
                            ([0], [93], -9), ([2, 3], [128, 128], -9), ([0], [2 ** 31 - 1], -9)):
        assert dgt.kv_reserve(c, i32(seqs), i32(cnt), status=st).tolist() == [-1] * len(seqs)
        refused(code)
    for a, b in ((0, 1), (0, 4), (4, 2), (-1, 2), (0, -1), (2, 2)):
        dgt.kv_fork(c, i32([a]), i32([b]), status=st)
        refused(-1)
    for s in (4, -1):
        dgt.kv_free(c, i32([s]), status=st)
        refused(-1)
    with pytest.raises(dgt.DgtError) as e:
        dgt.kv_reserve(c, torch.zeros(1025, dtype=torch.int32, device="cuda"),
                       torch.zeros(1025, dtype=torch.int32, device="cuda"))
    assert e.value.code == -2
