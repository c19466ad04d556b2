"""Rotation of many tokens: the same bits as the tokens one by one, in every
form of the kernel, on both sides of the counts where the form changes."""
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


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("tokens", [2047, 2048, 2049, 2051, 5003])
@pytest.mark.parametrize("hq,hk,dim,rot", [(8, 1, 64, 64), (16, 8, 64, 32), (4, 2, 256, 256), (17, 8, 64, 64),
                                           (24, 8, 128, 128), (3, 0, 80, 48)])
def test_many_tokens_equal_single_ones(dgt, inter, tokens, hq, hk, dim, rot):
    g = np.random.default_rng(tokens + dim)
    x = torch.from_numpy(g.normal(size=(tokens, (hq + hk) * dim)).astype(np.float32)).cuda().bfloat16()
    q, k = x[:, :hq * dim].view(tokens, hq, dim), x[:, hq * dim:].view(tokens, hk, dim) if hk else None
    pos = torch.from_numpy(g.integers(-1000, 200000, size=tokens).astype(np.int32)).cuda()
    r = dgt.Rotary(rot, interleaved=inter)
    yq, yk = dgt.rotate(r, q, pos, k=k)
    bits = lambda t: t.reshape(-1).view(torch.int16)
    # in pieces of fewer tokens than any change of form
    at = 0
    for n in (1, 700, 1, 1000, tokens - 1702):
        for a in range(at, at + n, 1024):
            e = min(a + 1024, at + n)
            pq, pk = dgt.rotate(r, q[a:e], pos[a:e], k=None if k is None else k[a:e])
            assert torch.equal(bits(pq), bits(yq[a:e]))
            if hk:
                assert torch.equal(bits(pk), bits(yk[a:e]))
        at += n
