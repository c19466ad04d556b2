"""Every form of the attention, on both sides of the row counts where the next
one takes over, against 64 bits (tolerances as in test_gpu_kv_attention.py).
The form is read off the size of its workspace."""
import numpy as np
import pytest

from test_gpu_kv_attention import Setup, i32, rand

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def dgt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import decode_gemv_tensor_gb300 as d
    d.lib()
    return d


# dimensions, rows of a kv head that an entry has (the mean, rounded up) -> rows of a tile
FORMS = [(64, 1, 8), (64, 8, 8), (64, 9, 16), (64, 16, 16), (64, 17, 24), (64, 24, 24), (64, 25, 256),
         (128, 8, 8), (128, 9, 16), (128, 16, 16), (128, 17, 256), (256, 8, 8), (256, 9, 128)]


def tile_rows(dgt, s, heads, batch, tokens):
    """From the workspace: 2 tiles of (dim + 4) floats a CTA, on 160 SMs."""
    ws = dgt.kv_attention_workspace(s.c, heads, batch, tokens).numel()
    dim = s.c.head_dim
    got = [rt for rt in (8, 16, 24, 128, 256) for ctas in (1, 2, 3)
           if ws == 2048 + 160 * ctas * 2 * rt * (dim + 4) * 4 and ctas == (1 if rt >= 128 else 3 if dim == 64 and rt == 8 else 2)]
    assert len(got) == 1
    return got[0]


@pytest.mark.parametrize("dim,rows,tile", FORMS)
@pytest.mark.parametrize("length", [30, 64, 777, 5000])
def test_rows_of_one_sequence(dgt, dim, rows, tile, length):
    # one query head a kv head: as many tokens as rows
    g = np.random.default_rng(dim + rows + length)
    s = Setup(dgt, g, [length], 2, dim)
    assert tile_rows(dgt, s, 2, 1, rows) == tile
    s.check(rand(g, rows, 2, dim), [rows])
    s.check(rand(g, rows, 2, dim), [rows], 100, 3)


@pytest.mark.parametrize("hq,hk,dim,counts,tile", [(32, 8, 64, [6, 6, 5, 6], 24), (24, 8, 64, [8, 1, 8, 8, 7], 24),
                                                   (5, 1, 64, [4, 5, 3], 24), (32, 8, 128, [4, 4, 3, 4], 16),
                                                   (16, 8, 256, [4, 3, 4], 8)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 1), (64, 0), (130, 70), (640, 16)])
def test_drafted_rows_of_a_batch(dgt, hq, hk, dim, counts, tile, window, sinks):
    g = np.random.default_rng(sum(counts) + window)
    lens = [777, 8, 640, 65, 2003][:len(counts)]
    s = Setup(dgt, g, lens, hk, dim)
    assert tile_rows(dgt, s, hq, len(counts), sum(counts)) == tile
    s.check(rand(g, sum(counts), hq, dim), counts, window, sinks)


@pytest.mark.parametrize("dim,rows,tile", [f for f in FORMS if f[1] in (8, 16, 24, 25) or f[2] == 128])
def test_more_parts_than_lanes_are_joined(dgt, dim, rows, tile):
    # 1875 pages of one head: 36 parts
    g = np.random.default_rng(dim + rows)
    s = Setup(dgt, g, [120000], 1, dim)
    assert tile_rows(dgt, s, 1, 1, rows) == tile
    s.check(rand(g, rows, 1, dim), [rows], rows=[0, 1, 7, 8, 15, 16, 22, 23, 24])
    s.check(rand(g, rows, 1, dim), [rows], 100000, 70, rows=[0, 7, rows - 1])


@pytest.mark.parametrize("longest", [80, 900])
def test_drafted_rows_of_more_sequences_than_are_described_at_a_time(dgt, longest):
    # 64 dimensions, four query heads a kv head, up to seven rows: tiles of 24, some sequences in two, some with none
    g = np.random.default_rng(longest)
    counts = g.integers(4, 8, size=150).tolist()
    for i in range(0, 150, 9):
        counts[i] = i % 4
    lens = [max(0, int(n)) for n in g.integers(-5, longest, size=150)]
    s = Setup(dgt, g, lens, 2, 64)
    assert tile_rows(dgt, s, 8, 150, sum(counts)) == 24
    s.check(rand(g, sum(counts), 8, 64), counts)
    s.check(rand(g, sum(counts), 8, 64), counts, 65, 2)


@pytest.mark.parametrize("polls", [0, 1])
@pytest.mark.parametrize("dim,rows", [(64, 12), (64, 24), (128, 16)])
def test_a_wait_that_runs_out_is_reported(dgt, dim, rows, polls):
    g = np.random.default_rng(dim + rows)
    s = Setup(dgt, g, [3000, 70], 2, dim)
    q, cu = rand(g, 2 * rows, 2, dim), i32([0, rows, 2 * rows])
    ws = dgt.kv_attention_workspace(s.c, 2, 2, 2 * rows)
    want = dgt.kv_attention(s.c, 0, q, i32([0, 1]), cu=cu, ws=ws)
    st = i32([0])
    dgt.kv_attention(s.c, 0, q, i32([0, 1]), cu=cu, ws=ws, status=st, test_wait_polls=polls)
    code = dgt.read_status(st)
    assert code == -5 if polls == 0 else code in (0, -5)
    assert torch.equal(dgt.kv_attention(s.c, 0, q, i32([0, 1]), cu=cu, ws=ws), want)
