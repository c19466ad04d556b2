"""What a call allocates for itself belongs to the stream that it works on:
the allocations of a call with a stream of its own, seen through stand-ins for
torch's streams and for the library, so that no device is needed."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")
import decode_gemv_tensor_gb300 as dgt  # noqa: E402


class Allocations:
    """(bytes, stream in effect) of every tensor made, and which were recorded on the current stream."""

    def __init__(self, monkeypatch):
        self.made, self.kept, self.stream = [], [], "current"
        for name in ("empty", "zeros"):
            monkeypatch.setattr(torch, name, self.counted(getattr(torch, name)))
        monkeypatch.setattr(torch.cuda, "stream", self.within)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=0, name="current"))
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: self.kept.append((t.data_ptr(), s.name)),
                            raising=False)

    def counted(self, make):
        def f(*a, **kw):
            t = make(*a, **kw)
            self.made.append((t.numel() * t.element_size(), self.stream))
            return t
        return f

    @contextlib.contextmanager
    def within(self, stream):
        was, self.stream = self.stream, stream
        yield
        self.stream = was


class Library:
    """Every call succeeds; every size is 1000 bytes."""

    def __getattr__(self, name):
        return lambda *a: 1000 if name.endswith("_bytes") else 0


@pytest.fixture
def seen(monkeypatch):
    cache = dgt.KvCache(1, 2, 1, 64, max_seqs=1, max_pages=2, device="cpu")
    monkeypatch.setattr(dgt, "_lib", Library())
    monkeypatch.setattr(dgt, "_heads", lambda x, name: b"")
    monkeypatch.setattr(dgt, "_i32", lambda x, name, n=None: x.data_ptr())
    side = types.SimpleNamespace(cuda_stream=7, name="side")
    return cache, side, Allocations(monkeypatch)


def rows(n, heads):
    return torch.ones(n, heads, 64, dtype=torch.bfloat16)


def test_attention_allocates_its_workspace_on_its_stream(seen):
    cache, side, log = seen
    q, seqs, out = rows(1, 2), torch.ones(1, dtype=torch.int32), rows(1, 2)
    log.made.clear()
    dgt.kv_attention(cache, 0, q, seqs, out=out, stream=side)
    assert log.made == [(1000, side)]


def test_an_attention_workspace_made_for_a_stream(seen):
    cache, side, log = seen
    log.made.clear()
    ws = dgt.kv_attention_workspace(cache, 2, 1, 1, stream=side)
    assert log.made == [(1000, side)] and log.kept == [(ws.data_ptr(), "current")]
