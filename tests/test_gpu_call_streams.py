"""Calls on a stream of their own while the current stream is busy, without a
workspace or outputs given."""
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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rand(seed, *shape):
    g = np.random.default_rng(seed)
    return torch.from_numpy(g.normal(size=shape).astype(np.float32)).cuda().bfloat16()


def busy(*sizes):
    """The current stream with some ten milliseconds of work before it, and blocks of these sizes that it has
    released and is still to write."""
    torch.cuda.synchronize()
    junk = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda._sleep(20_000_000)
    for x in junk:
        x.fill_(255)


def test_attention_without_a_workspace(dgt):
    # 20011 tokens: parts that the last CTA to arrive joins, by counters in the workspace
    c = dgt.KvCache(1, 320, 2, 128, max_seqs=1, max_pages=320)
    c.table[0] = torch.arange(320, dtype=torch.int32, device="cuda")
    c.lens[0] = 20011
    k, v, q, seqs = rand(1, 20011, 2, 128), rand(2, 20011, 2, 128), rand(3, 1, 6, 128), i32([0])
    dgt.kv_append(c, 0, k, v, seqs, i32([0]), cu=i32([0, 20011]))
    want = dgt.kv_attention(c, 0, q, seqs)
    side = torch.cuda.Stream()
    n = dgt.kv_attention_workspace(c, 6, 1, 1).numel()
    for _ in range(3):
        busy(n)
        got = dgt.kv_attention(c, 0, q, seqs, stream=side)
        other = dgt.kv_attention(c, 0, q, seqs, stream=side)
        side.synchronize()
        assert torch.equal(got, want) and torch.equal(other, want)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(other, want)


def test_outputs_and_temporary_memory(dgt):
    # a product whose workspace and outputs are its own, and the cache's read-back
    W, X = rand(4, 256, 4096), rand(5, 64, 4096)
    want = dgt.gemm_bf16(W, X, plan=dgt.gemm_plan(64, 256, 4096, split_k=4))
    c = dgt.KvCache(1, 40, 2, 128, max_seqs=1, max_pages=40)
    c.table[0] = torch.arange(40, dtype=torch.int32, device="cuda")
    k, v, seqs, cu = rand(6, 2500, 2, 128), rand(7, 2500, 2, 128), i32([0]), i32([0, 2500])
    dgt.kv_append(c, 0, k, v, seqs, i32([0]), cu=cu)
    back = dgt.kv_read(c, 0, seqs, i32([0]), cu, 2500)
    zero, plan = i32([0]), dgt.gemm_plan(64, 256, 4096, split_k=4)
    side = torch.cuda.Stream()
    for _ in range(3):
        busy(64 * 256 * 4, 64 * 256 * 2, 64 * 256 * 4 * 4, 2500 * 2 * 128 * 2, 2500 * 2 * 128 * 2)
        got = dgt.gemm_bf16(W, X, plan=plan, stream=side) + tuple(dgt.kv_read(c, 0, seqs, zero, cu, 2500, stream=side))
        torch.cuda.synchronize()
        for a, b in zip(got, want + tuple(back)):
            assert torch.equal(a, b)


def test_exponent_stats(dgt):
    w = rand(8, 4096, 4096)
    _, _, bits, entropy = dgt.exponent_stats(w)
    busy(1 << 20)
    _, _, b2, e2 = dgt.exponent_stats(w, stream=torch.cuda.Stream())
    assert (b2, e2) == (bits, entropy)
