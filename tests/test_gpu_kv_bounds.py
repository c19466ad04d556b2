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


def held(c):
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
    before = held(c)
    dgt.kv_append(c, 0, x, x, seqs, i32(start), cu=i32(cu), status=st)
    assert dgt.read_status(st) == -1
    for a, b in zip(held(c), before):
        assert torch.equal(a, b)
    st.zero_()
    dgt.kv_read(c, 0, seqs, i32(start), i32(cu), 128, status=st)
    assert dgt.read_status(st) == -1
    # the same rows from the first on
    st.zero_()
    dgt.kv_append(c, 0, x, x, i32([0]), i32([70]), cu=i32([0, 128]), status=st)
    k, v = dgt.kv_read(c, 0, i32([0]), i32([70]), i32([0, 128]), 128, status=st)
    assert dgt.read_status(st) == 0 and (k == 1).all() and (v == 1).all()
