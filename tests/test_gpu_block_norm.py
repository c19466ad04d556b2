"""block_norm against its formula in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
import decode_gemv_tensor_gb300 as dgt  # noqa: E402

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-6


def reference(x, y, pre, post, gate, scale, residual, offset):
    """(x', h, size of what x' adds) in 64 bits."""
    d = lambda t: None if t is None else t.double()
    x, y, pre, post, gate = map(d, (x, y, pre, post, gate))
    r = lambda v: 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
    x1 = residual * x
    size = x1.abs()
    if y is not None:
        u = y
        if post is not None:
            u = u * r(u) * (offset + post)
        if gate is not None:
            u = u * gate
        x1 = x1 + scale * u
        size = size + (scale * u).abs()
    return x1, None if pre is None else x1 * r(x1) * (offset + pre), size


def check(got, want, size, pre, offset):
    """Squares of up to 32768 elements are summed in at most 32 steps a thread and 10 between threads, each off by
    2^-24, so a mean square by 42 2^-24 and r by half of that and 3 2^-24 of its own operations: below 2^-19.  x' adds
    terms that are off by that and four more roundings: 2^-18 of their size.  h takes r(x') and x': the error of a row's
    x' reaches r through a mean, never more than 2^-18 of its size."""
    x1, h = got
    err = size * 2.0 ** -18
    half = 2.0 ** -8 if x1.dtype is BF16 else 2.0 ** -24
    assert bool(((x1.double() - want[0]).abs() <= err + want[0].abs() * half + 1e-38).all())
    if h is None:
        return
    rms = torch.sqrt((want[0] ** 2).mean(-1, keepdim=True) + EPS)
    weight = (offset + pre.double()).abs()
    spread = torch.sqrt((size ** 2).mean(-1, keepdim=True)) / rms * 2.0 ** -18     # relative error of r from x'
    tol = (err / rms * weight + want[1].abs() * (spread + 2.0 ** -18)) * (1 + 2.0 ** -8) + want[1].abs() * 2.0 ** -8
    assert bool(((h.double() - want[1]).abs() <= tol + 1e-38).all())


def inputs(rows, n, xt, yt, gate=None, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)
    x = (r(rows, n) * 3).to(xt)
    y = None if yt is None else r(rows, n).mul(torch.exp(r(n))).to(yt)
    w = lambda: (1 + 0.3 * r(n)).to(BF16)
    gate = {None: None, "channel": r(n).to(BF16), "row": r(rows, n).to(BF16)}[gate]
    return x, y, w(), w(), gate


@pytest.mark.parametrize("n", [1, 7, 8, 31, 64, 250, 256, 264, 1000, 1001, 3840, 4097, 8192, 8200, 16384, 16385, 20000,
                               32761, 32768])
@pytest.mark.parametrize("xt,yt", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
def test_sizes_and_types(n, xt, yt):
    x, y, pre, post, _ = inputs(5, n, xt, yt, seed=n)
    got = dgt.block_norm(x, y, pre=pre, post=post, scale=0.5, residual=0.75, eps=EPS)
    want = reference(x, y, pre, post, None, 0.5, 0.75, 0.0)
    assert got[0].dtype is xt and got[1].dtype is BF16
    check(got, want, want[2], pre, 0.0)


@pytest.mark.parametrize("rows", [1, 2, 3, 33, 1027])
@pytest.mark.parametrize("n", [64, 72, 100, 3840])
@pytest.mark.parametrize("post,gate,offset", [(False, None, 0.0), (True, None, 1.0), (False, "channel", 0.0),
                                              (True, "row", 0.0)])
def test_what_is_left_out(rows, n, post, gate, offset):
    x, y, pre, p, g = inputs(rows, n, F32, F32, gate, seed=rows * n)
    p = p if post else None
    got = dgt.block_norm(x, y, pre=pre, post=p, gate=g, offset=offset, eps=EPS)
    want = reference(x, y, pre, p, g, 1.0, 1.0, offset)
    check(got, want, want[2], pre, offset)


def test_no_block_output_and_no_norm_behind():
    x, y, pre, post, _ = inputs(3, 96, BF16, BF16)
    got = dgt.block_norm(x, pre=pre, residual=0.5, eps=EPS)
    want = reference(x, None, pre, None, None, 1.0, 0.5, 0.0)
    check(got, want, want[2], pre, 0.0)
    got = dgt.block_norm(x, y, post=post, eps=EPS)
    assert got[1] is None
    want = reference(x, y, None, post, None, 1.0, 1.0, 0.0)
    check(got, want, want[2], None, 0.0)


@pytest.mark.parametrize("n", [64, 100, 3840])
def test_in_place_strided_and_one_row(n):
    x, y, pre, post, _ = inputs(9, n, F32, F32)
    want = reference(x, y, pre, post, None, 1.0, 1.0, 0.0)
    for extra in (1, 8):     # rows of a wider tensor, unaligned and aligned
        wide = torch.full((9, n + extra), 7.0, device="cuda")
        wide[:, :n] = x
        yw = torch.zeros(9, 2 * n, device="cuda")
        yw[:, n:] = y
        hw = torch.full((9, n + extra), 7.0, device="cuda", dtype=BF16)
        a, h = dgt.block_norm(wide[:, :n], yw[:, n:], pre=pre, post=post, eps=EPS, x_out=wide[:, :n], h=hw[:, :n])
        assert a.data_ptr() == wide.data_ptr()
        check((a, h), want, want[2], pre, 0.0)
        assert bool((wide[:, n:] == 7).all()) and bool((hw[:, n:] == 7).all())
    one = dgt.block_norm(x[4], y[4], pre=pre, post=post, eps=EPS)
    assert one[0].shape == (n,)
    check([t.view(1, n) for t in one], [t[4:5] for t in want[:2]], want[2][4:5], pre, 0.0)


def test_same_bits_each_time_and_for_each_row_count():
    x, y, pre, post, _ = inputs(300, 3840, F32, F32)
    a = dgt.block_norm(x, y, pre=pre, post=post)
    b = dgt.block_norm(x, y, pre=pre, post=post)
    c = dgt.block_norm(x[7:8], y[7:8], pre=pre, post=post)
    for i in range(2):
        assert torch.equal(a[i], b[i]) and torch.equal(a[i][7:8], c[i])


def test_zeros_infinities_and_nan_stay_in_their_rows():
    x, y, pre, post, _ = inputs(4, 256, F32, F32)
    x[0], y[0] = 0, 0
    y[1, 3] = float("inf")
    x[2, 5] = float("nan")
    x1, h = dgt.block_norm(x, y, pre=pre, post=post, eps=EPS)
    assert bool((x1[0] == 0).all()) and bool((h[0] == 0).all())
    assert bool(h[1].isnan().any()) and bool(h[2].isnan().all())
    want = reference(x[3:], y[3:], pre, post, None, 1.0, 1.0, 0.0)
    check((x1[3:], h[3:]), want, want[2], pre, 0.0)


def test_stream_and_graph():
    x, y, pre, post, _ = inputs(40, 512, F32, F32)
    want = dgt.block_norm(x, y, pre=pre, post=post)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = dgt.block_norm(x, y, pre=pre, post=post, stream=s)
    s.synchronize()
    assert torch.equal(got[1], want[1])
    out, h = torch.empty_like(x), torch.empty_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dgt.block_norm(x, y, pre=pre, post=post, x_out=out, h=h)
    x.mul_(2)
    g.replay()
    assert torch.equal(h, dgt.block_norm(x, y, pre=pre, post=post)[1])


def test_refusals():
    x, y, pre, post, _ = inputs(4, 64, F32, F32)
    bad = [dict(pre=pre.float()), dict(pre=pre[:32]), dict(post=post, y=None), dict(y=y[:2]), dict(y=y.double()),
           dict(x_out=x.bfloat16()), dict(gate=y), dict(h=torch.empty(4, 64, device="cuda")),
           dict(y=y.t().contiguous().t())]
    for kw in bad:
        with pytest.raises(ValueError):
            dgt.block_norm(x, **{"y": y, "pre": pre, **kw})
    with pytest.raises(ValueError):
        dgt.block_norm(x, y, pre=pre, x_out=x[:1].expand(4, 64))
    assert [t.shape for t in dgt.block_norm(x[:0], y[:0], pre=pre)] == [(0, 64), (0, 64)]
