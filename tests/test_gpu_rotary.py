"""Rotary positions against the rotation in 64 bits."""
import numpy as np
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


def reference(x, pos, axis, inv_freq, interleaved):
    """x [tokens, heads, dim] float64, pos [axes, tokens]; (result, bound on its error)."""
    rot = 2 * len(inv_freq)
    half = rot // 2
    angle = pos[axis].astype(np.float64).T * inv_freq          # [tokens, half]
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    ia, ib = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (np.arange(half), np.arange(half, rot))
    y, size = x.copy(), np.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    # the angle: 2^-33 revolutions kept and cut off, the frequency's 53 bits on either side times the position,
    # sincospif's 2 half-steps and fp32 products: together below 2^-21 of |a| + |b|, plus |angle| * 2^-51
    size[..., ia] = size[..., ib] = (np.abs(a) + np.abs(b)) * (2.0 ** -21 + np.abs(angle)[:, None] * 2.0 ** -51)
    return y, size + 2.0 ** -8 * np.abs(y)


CASES = [(1, 24, 8, 128, 128, 1, False), (1, 1, 1, 64, 16, 1, True), (7, 3, 1, 64, 64, 3, False),
         (130, 16, 8, 256, 256, 1, False), (33, 5, 2, 128, 64, 3, True), (65, 4, 4, 256, 128, 2, False),
         (9, 2, 2, 80, 48, 1, False), (3, 1, 1, 1024, 1024, 1, True)]


@pytest.mark.parametrize("tokens,hq,hk,dim,rot,axes,inter", CASES)
@pytest.mark.parametrize("far", [0, 131072, 2 ** 31 - 1, -5])
def test_rotate_matches_64_bits(dgt, tokens, hq, hk, dim, rot, axes, inter, far):
    g = np.random.default_rng(tokens + dim + axes)
    half = rot // 2
    sec = [half // axes] * (axes - 1) + [half - (axes - 1) * (half // axes)]
    axis = np.repeat(np.arange(axes), sec)
    # rows of a stacked projection: q, k and something else beside them
    x = torch.from_numpy(g.normal(size=(tokens, (hq + 2 * hk) * dim)).astype(np.float32)).cuda().bfloat16()
    q, k = x[:, :hq * dim].view(tokens, hq, dim), x[:, hq * dim:(hq + hk) * dim].view(tokens, hk, dim)
    pos = (far - g.integers(0, 3000, size=(axes, tokens))).astype(np.int32)
    r = dgt.Rotary(rot, base=10000.0, sections=sec, interleaved=inter)
    pd = torch.from_numpy(pos).cuda()
    inv = 10000.0 ** (-2.0 * np.arange(half) / rot)
    yq, yk = dgt.rotate(r, q, pd, k=k)
    only, none = dgt.rotate(r, q, pd)
    assert none is None and torch.equal(only.view(torch.int16), yq.view(torch.int16))
    for y, t in ((yq, q), (yk, k)):
        ref, tol = reference(t.double().cpu().numpy(), pos, axis, inv, inter)
        assert (np.abs(y.double().cpu().numpy() - ref) <= tol).all()
        assert torch.equal(y[..., rot:].reshape(-1).view(torch.int16), t[..., rot:].reshape(-1).view(torch.int16))
    # in place, on a stream of its own
    before = x.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    dgt.rotate(r, q, pd, k=k, q_out=q, k_out=k, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(q.reshape(-1).view(torch.int16), yq.reshape(-1).view(torch.int16))
    assert torch.equal(k.reshape(-1).view(torch.int16), yk.reshape(-1).view(torch.int16))
    assert torch.equal(x[:, (hq + hk) * dim:], before[:, (hq + hk) * dim:])


def test_own_frequencies_and_axes(dgt):
    # interleaved axes (time, height, width, time, ...) and scaled frequencies
    g = np.random.default_rng(5)
    inv = 0.25 * 500000.0 ** (-2.0 * np.arange(32) / 64)
    axis = np.arange(32) % 3
    x = torch.from_numpy(g.normal(size=(11, 2, 64)).astype(np.float32)).cuda().bfloat16()
    pos = g.integers(0, 100000, size=(3, 11)).astype(np.int32)
    y, _ = dgt.rotate(dgt.Rotary(64, inv_freq=inv, axis=axis.tolist()), x, torch.from_numpy(pos).cuda())
    ref, tol = reference(x.double().cpu().numpy(), pos, axis, inv, False)
    assert (np.abs(y.double().cpu().numpy() - ref) <= tol).all()


def test_rotate_arguments(dgt):
    x = torch.zeros(4, 2, 64, device="cuda", dtype=torch.bfloat16)
    r = dgt.Rotary(64)
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (dict(pos=pos[:3]), dict(pos=pos.long()), dict(q=x.float()), dict(q=x[..., ::2]),
                dict(k=x[:3]), dict(q_out=x[:3])):
        kw = dict(q=x, pos=pos)
        kw.update(bad)
        with pytest.raises(ValueError):
            dgt.rotate(r, **kw)
    for bad in (dict(sections=[16, 15]), dict(inv_freq=[1.0]), dict(axis=[0] * 31)):
        with pytest.raises(ValueError):
            dgt.Rotary(64, **bad)
    with pytest.raises(dgt.DgtError) as e:
        dgt.rotate(dgt.Rotary(128), x, pos)      # more dimensions than a head has
    assert e.value.code == -2
    y, _ = dgt.rotate(r, x[:0], pos[:0])
    assert y.shape == (0, 2, 64)
