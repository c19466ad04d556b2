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
        self.made, self.kept, self.alive, self.stream = [], [], [], "current"
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
            self.alive.append(t)      # so that no address comes twice
            return t
        return f

    @contextlib.contextmanager
    def within(self, stream):
        was, self.stream = self.stream, stream
        if stream is None:
            self.stream = was
        yield
        self.stream = was


class Library:
    """Every call succeeds; every size is 1000 bytes.  What earlier tests left is freed as ever."""

    def __init__(self):
        self.dgt_packed_free = dgt.lib().dgt_packed_free

    def __getattr__(self, name):
        return lambda *a: 1000 if name.endswith("_bytes") else 0


@pytest.fixture
def seen(monkeypatch):
    cache = dgt.KvCache(1, 2, 1, 64, max_seqs=1, max_pages=2, device="cpu")
    monkeypatch.setattr(dgt, "_lib", Library())
    monkeypatch.setattr(dgt, "_raw_stream", lambda i: 0)
    monkeypatch.setattr(dgt, "_heads", lambda x, name: b"")
    monkeypatch.setattr(dgt, "_i32", lambda x, name, n=None: x.data_ptr())
    side = types.SimpleNamespace(cuda_stream=7, name="side")
    return cache, side, Allocations(monkeypatch)


def rows(n, heads):
    return torch.ones(n, heads, 64, dtype=torch.bfloat16)


def test_attention_allocates_its_workspace_on_its_stream(seen):
    cache, side, log = seen
    q, seqs = rows(1, 2), torch.ones(1, dtype=torch.int32)
    log.made.clear()
    dgt.kv_attention(cache, 0, q, seqs, stream=side)
    assert (1000, side) in log.made and all(s is side for _, s in log.made)


F32, BF16 = torch.float32, torch.bfloat16


def calls(cache):
    """name -> call of a stream: every one allocates outputs, or memory of its own, or both."""
    x, f, ids = torch.ones(128, dtype=BF16), torch.ones(128), torch.ones(2, 2, dtype=torch.int32)
    m, w, g = torch.ones(2, 128, dtype=BF16), torch.ones(128, 128, dtype=BF16), torch.ones(2, 128)
    r4 = types.SimpleNamespace(s=dgt.R4Struct(), sm=x, rows=128, cols=128)
    dev = types.SimpleNamespace(view=dgt.PackedView(rows=128, cols=128), tensors={"sm": x})
    one, r = torch.ones(1, dtype=torch.int32), types.SimpleNamespace(axes=1, ptr=0)
    p = torch.ones(2, 2)
    return {
        "load_r4": lambda s: dgt.load_r4(dev, stream=s),
        "r4_to_bf16": lambda s: dgt.r4_to_bf16(r4, stream=s),
        "gemv": lambda s: dgt.gemv(r4, x, stream=s),
        "gemv_bf16": lambda s: dgt.gemv_bf16(w, x, stream=s),
        "moe_gemv": lambda s: dgt.moe_gemv(r4, 2, ids, p, m, stream=s),
        "moe_gemv_bf16": lambda s: dgt.moe_gemv_bf16(w, 2, ids, p, m, stream=s),
        "moe_gemm": lambda s: dgt.moe_gemm(r4, 2, ids, p, m, stream=s),
        "moe_gemm_bf16": lambda s: dgt.moe_gemm_bf16(w, 2, ids, p, m, stream=s),
        "gemm": lambda s: dgt.gemm(r4, m, stream=s),
        "gemm_bf16": lambda s: dgt.gemm_bf16(w, m, stream=s),
        "gemm_rebuild": lambda s: dgt.gemm_rebuild(r4, m, stream=s),
        "add_rmsnorm": lambda s: dgt.add_rmsnorm(f, x, 1e-5, stream=s),
        "silu_mul": lambda s: dgt.silu_mul(f, f, stream=s),
        "silu_mul_rows": lambda s: dgt.silu_mul_rows(g, stream=s),
        "repeat": lambda s: dgt.repeat(x, 256, stream=s),
        "weighted_sum": lambda s: dgt.weighted_sum(g, f[:2], stream=s),
        "rotate": lambda s: dgt.rotate(r, rows(1, 2), one, k=rows(1, 1), stream=s),
        "kv_read": lambda s: dgt.kv_read(cache, 0, one, one, None, 1, stream=s),
        "kv_attention": lambda s: dgt.kv_attention(cache, 0, rows(1, 2), one, stream=s),
        "kv_reserve": lambda s: dgt.kv_reserve(cache, one, one, stream=s),
    }


NAMES = list(calls(None))


@pytest.mark.parametrize("name", NAMES)
def test_what_a_call_allocates_is_its_streams(seen, name):
    cache, side, log = seen
    call = calls(cache)[name]
    log.made.clear()
    got = call(side)
    assert log.made and all(s is side for _, s in log.made)
    # what it returns may be read by the current stream as well
    if name == "load_r4":
        got = (got.nib, got.esc, got.seg)
    given = {t.data_ptr() for t in (got if isinstance(got, (tuple, list)) else (got,)) if t is not None}
    assert given == {p for p, s in log.kept if s == "current"}
    # without one, the current stream's as ever
    log.made.clear()
    log.kept.clear()
    call(None)
    assert all(s == "current" for _, s in log.made) and not log.kept


def test_an_attention_workspace_made_for_a_stream(seen):
    cache, side, log = seen
    log.made.clear()
    ws = dgt.kv_attention_workspace(cache, 2, 1, 1, stream=side)
    assert log.made == [(1000, side)] and log.kept == [(ws.data_ptr(), "current")]


def test_exponent_stats_reads_its_totals_behind_its_kernels(seen, monkeypatch):
    _, side, log = seen
    read = []
    cpu = torch.Tensor.cpu
    monkeypatch.setattr(torch.Tensor, "cpu", lambda t: read.append(log.stream) or cpu(t))
    dgt.exponent_stats(torch.ones(256, dtype=BF16), stream=side)
    assert read == [side] and all(s is side for _, s in log.made)
