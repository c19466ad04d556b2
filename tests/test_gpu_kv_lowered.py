"""Sequences whose length was lowered (drafted tokens that were not taken):
their later pages are used again, and none is lost.  After every operation a
page's references are the table entries that name it."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

PAGE = 64


@pytest.fixture(scope="module")
def dgt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import decode_gemv_tensor_gb300 as d
    d.lib()
    return d


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Watch:
    """A cache, with the state before an operation against the one after it."""

    def __init__(self, dgt, pages, seqs, width):
        self.dgt, self.st = dgt, i32([0])
        self.c = dgt.KvCache(1, pages, 1, 64, max_seqs=seqs, max_pages=width)
        g = torch.Generator(device="cuda").manual_seed(pages)
        self.c.k.copy_(torch.randint(0, 120, self.c.k.shape, generator=g, device="cuda", dtype=torch.uint8))
        self.look()

    def look(self):
        self.table, self.lens = self.c.table.cpu().numpy().copy(), self.c.lens.cpu().numpy().copy()
        self.refs, self.k = self.c.refs.cpu().numpy().copy(), self.c.k[0, :, 0].cpu().numpy().copy()

    def balanced(self, where):
        t = self.c.table.cpu().numpy()
        want = np.bincount(t[t >= 0].ravel(), minlength=self.c.pages)
        assert np.array_equal(self.c.refs.cpu().numpy(), want), where

    def lower(self, seq, n):
        self.c.lens[seq] = n
        self.look()

    def reserve(self, seqs, counts, where=None):
        """Room for the tokens in pages of their own, what was held still there; the whole list or nothing."""
        start = self.dgt.kv_reserve(self.c, i32(seqs), i32(counts), status=self.st).tolist()
        code = self.dgt.read_status(self.st)
        self.st.zero_()
        before, old, k = self.table, self.lens, self.k
        refs = self.refs
        self.look()
        if code:
            assert code == -9 and start == [-1] * len(seqs), where
            assert np.array_equal(self.table, before) and np.array_equal(self.lens, old), where
            assert np.array_equal(self.refs, refs), where
            return False
        assert start == [old[s] for s in seqs], where
        for s in range(self.c.max_seqs):
            n = old[s] + (counts[seqs.index(s)] if s in seqs else 0)
            assert self.lens[s] == n, where
            for i in range(-(-int(old[s]) // PAGE)):
                assert np.array_equal(self.k[self.table[s, i]], k[before[s, i]]), where
            for i in range(old[s] // PAGE, -(-int(n) // PAGE)) if n > old[s] else ():
                assert self.table[s, i] >= 0 and self.refs[self.table[s, i]] == 1, where
        self.balanced(where)
        return True


def test_pages_behind_a_lowered_length_are_used_again(dgt):
    w = Watch(dgt, 6, 1, 6)
    assert w.reserve([0], [300])                     # five pages
    pages = w.table[0, :5].tolist()
    w.lower(0, 70)
    assert w.reserve([0], [100]) and w.table[0, :5].tolist() == pages       # 170: the third again
    w.lower(0, 64)
    assert w.reserve([0], [300]) and w.table[0, :5].tolist() == pages       # 364: five again, and a sixth
    w.lower(0, 0)
    assert w.reserve([0], [384]) and not w.reserve([0], [1])
    dgt.kv_free(w.c, i32([0]))
    assert not w.c.refs.any() and (w.c.table == -1).all()


def test_pages_behind_a_lowered_length_that_are_shared(dgt):
    # two continuations that share what both have given back: each takes pages of its own, and the shared are free
    w = Watch(dgt, 9, 3, 6)
    assert w.reserve([0], [250])                     # pages 0 to 3
    dgt.kv_fork(w.c, i32([0, 0]), i32([1, 2]))
    w.look()
    for s in (1, 2):
        w.lower(s, 64)
    assert w.reserve([2, 1], [90, 90])
    assert w.refs[:4].tolist() == [3, 1, 1, 3]       # the second and third are given up; all three rows list the others
    w.lower(0, 64)
    assert w.reserve([0], [192])
    for s in (0, 1, 2):
        dgt.kv_free(w.c, i32([s]))
    assert not w.c.refs.any()


def test_entries_that_nobody_holds(dgt):
    # a row with entries that were never counted, and one that names no page
    w = Watch(dgt, 4, 2, 3)
    w.c.table[0] = i32([2, 1, 0])
    dgt.kv_reserve(w.c, i32([1, 0]), i32([100, 64]), status=w.st)
    assert dgt.read_status(w.st) == 0
    t = w.c.table.tolist()
    assert t[1] == [0, 1, -1] and t[0][0] == 2 and w.c.refs.tolist() == [1, 1, 1, 0]
    w.c.table[0, 1] = 4
    w.look()
    assert dgt.kv_reserve(w.c, i32([0]), i32([64]), status=w.st).tolist() == [-1] and dgt.read_status(w.st) == -1
    assert np.array_equal(w.c.table.cpu().numpy(), w.table) and w.c.refs.tolist() == [1, 1, 1, 0]


@pytest.mark.parametrize("seed", range(8))
def test_a_history_with_lowered_lengths(dgt, seed):
    g = np.random.default_rng(seed)
    seqs, width = 7, 9
    w = Watch(dgt, int(g.integers(12, 50)), seqs, width)
    done = 0
    for step in range(60):
        op = g.choice(["reserve", "reserve", "lower", "lower", "fork", "free", "compact"])
        if op == "reserve":
            who = g.permutation(seqs)[:int(g.integers(1, seqs + 1))].tolist()
            done += w.reserve(who, [int(x) for x in g.choice([0, 1, 5, 63, 64, 65, 130], size=len(who))], (step, op))
        elif op == "lower":
            s = int(g.integers(seqs))
            w.lower(s, int(g.integers(0, w.lens[s] + 1)))
        elif op == "fork":
            src = [s for s in range(seqs) if w.lens[s] > 0]
            dst = [s for s in range(seqs) if w.lens[s] == 0 and w.table[s, 0] < 0]
            if src and dst:
                dgt.kv_fork(w.c, i32([int(g.choice(src))] * len(dst[:2])), i32(dst[:2]), status=w.st)
        elif op == "free":
            dgt.kv_free(w.c, i32([int(g.integers(seqs))]), status=w.st)
        else:
            dgt.kv_compact(w.c, status=w.st)
        assert dgt.read_status(w.st) == 0
        w.look()
        w.balanced((step, op))
    assert done > 3
