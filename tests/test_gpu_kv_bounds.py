"""Lists on the device that the cache's kernels find wrong: reported, and
nothing read or written for them."""
import pytest

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


def held_of(c):
    return [x.clone() for x in (c.k, c.v, c.k_scale, c.v_scale)]


@pytest.mark.parametrize("cu,start", [([64, 128], [70]), ([1, 128], [70]), ([-64, 128], [70]), ([128, 128], [200]),
                                      ([64, 66, 128], [70, 0])])
def test_rows_that_do_not_begin_at_the_first(dgt, cu, start):
    # numbers of blocks before the first entry's would reach pages and rows before its own
    c = dgt.KvCache(1, 8, 2, 64, max_seqs=2, max_pages=4)
    c.table[0], c.table[1] = i32([0, 1, 2, 3]), i32([4, 5, 6, 7])
    x = torch.ones(128, 2, 64, device="cuda", dtype=torch.bfloat16)
    st = i32([0])
    seqs = i32(list(range(len(start))))
    before = held_of(c)
    dgt.kv_append(c, 0, x, x, seqs, i32(start), cu=i32(cu), status=st)
    assert dgt.read_status(st) == -1
    for a, b in zip(held_of(c), before):
        assert torch.equal(a, b)
    st.zero_()
    dgt.kv_read(c, 0, seqs, i32(start), i32(cu), 128, status=st)
    assert dgt.read_status(st) == -1
    # the same rows from the first on
    st.zero_()
    dgt.kv_append(c, 0, x, x, i32([0]), i32([70]), cu=i32([0, 128]), status=st)
    k, v = dgt.kv_read(c, 0, i32([0]), i32([70]), i32([0, 128]), 128, status=st)
    assert dgt.read_status(st) == 0 and (k == 1).all() and (v == 1).all()


@pytest.mark.parametrize("held", [70, 128, 200])
def test_an_append_into_a_page_that_others_share(dgt, held):
    # a fork shares every page until kv_reserve has given it a last one of its own
    c = dgt.KvCache(2, 12, 2, 64, max_seqs=3, max_pages=5)
    g = torch.Generator(device="cuda").manual_seed(held)
    x = torch.randn(held, 2, 64, device="cuda", generator=g).bfloat16()
    new = 100 * torch.randn(1, 2, 64, device="cuda", generator=g).bfloat16()
    st = i32([0])
    for l in range(2):
        start = dgt.kv_reserve(c, i32([0]), i32([held]), status=st) if l == 0 else i32([0])
        dgt.kv_append(c, l, x, x, i32([0]), start, cu=i32([0, held]), status=st)
    dgt.kv_fork(c, i32([0]), i32([2]), status=st)
    assert dgt.read_status(st) == 0
    before = held_of(c)
    for seq in (0, 2):                   # over a token that is there
        dgt.kv_append(c, 1, new, new, i32([seq]), i32([held - 1]), status=st)
        assert dgt.read_status(st) == -1
        st.zero_()
    for a, b in zip(held_of(c), before):
        assert torch.equal(a, b)
    start = dgt.kv_reserve(c, i32([2]), i32([1]), status=st)
    dgt.kv_append(c, 1, new, new, i32([2]), start, status=st)
    assert dgt.read_status(st) == 0
    k, _ = dgt.kv_read(c, 1, i32([0, 2]), i32([0, 0]), i32([0, held, 2 * held + 1]), 2 * held + 1, status=st)
    want, _ = dgt.kv_read(c, 0, i32([0]), i32([0]), i32([0, held]), held, status=st)
    assert torch.equal(k[:held], want) and dgt.read_status(st) == 0
    assert ((k[-1].float() - new[0].float()).abs() <= 2.0 ** -4 * new[0].float().abs().amax()).all()


def test_copies_right_behind_what_writes_their_pages(dgt):
    # pages copied back and forth between appends, every kernel launched while the one before may still run
    c = dgt.KvCache(1, 130, 8, 128, max_seqs=1, max_pages=64)
    c.table[0] = torch.arange(64, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    x = [torch.randn(64 * 64, 8, 128, device="cuda", generator=g).bfloat16() for _ in range(2)]
    seq, zero, cu = i32([0]), i32([0]), i32([0, 64 * 64])
    here, there = torch.arange(64, dtype=torch.int32, device="cuda"), torch.arange(64, 128, dtype=torch.int32, device="cuda")
    want = []
    for v in x:
        dgt.kv_append(c, 0, v, v, seq, zero, cu=cu)
        torch.cuda.synchronize()
        want.append((c.k[:, :64].clone(), c.v[:, :64].clone()))
    torch.cuda.synchronize()
    for _ in range(5):
        for i, v in enumerate(x):
            dgt.kv_append(c, 0, v, v, seq, zero, cu=cu)
            dgt.kv_copy_pages(c, here, there)
            dgt.kv_append(c, 0, x[1 - i], x[1 - i], seq, zero, cu=cu)
            got = c.k[:, 64:128].clone(), c.v[:, 64:128].clone()
            dgt.kv_copy_pages(c, there, here)
            back = c.k[:, :64].clone(), c.v[:, :64].clone()
            for a in (got, back):
                assert torch.equal(a[0], want[i][0]) and torch.equal(a[1], want[i][1])
