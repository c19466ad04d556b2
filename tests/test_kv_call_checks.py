"""What the Python calls of the cache and the attention refuse themselves,
before the library is called: tensors on the host stand for wrong ones, so no
device is needed."""
import types

import pytest

torch = pytest.importorskip("torch")
import decode_gemv_tensor_gb300 as dgt  # noqa: E402


@pytest.fixture
def kv(monkeypatch):
    """A cache, and a library whose cache calls are counted and succeed (others go through: what earlier tests
    left may be freed meanwhile)."""
    cache = dgt.KvCache(3, 2, 1, 64, max_seqs=1, max_pages=2, device="cpu")
    calls, real = [], dgt.lib()

    class Library:
        def __getattr__(self, name):
            if not name.startswith("dgt_kv_"):
                return getattr(real, name)
            return lambda *a: 1000 if name.endswith("_bytes") else calls.append((name, a)) or 0
    monkeypatch.setattr(dgt, "_lib", Library())
    monkeypatch.setattr(dgt, "_raw_stream", lambda i: 0)
    monkeypatch.setattr(dgt, "_heads", lambda x, name: b"")
    monkeypatch.setattr(dgt, "_i32", lambda x, name, n=None: x.data_ptr())
    return types.SimpleNamespace(cache=cache, calls=calls, one=torch.zeros(1, dtype=torch.int32))


def test_read_of_a_layer_below_zero(kv):
    # the library reads -1 as every layer: the outputs of one layer would not hold that
    for layer in (-1, -2):
        with pytest.raises(ValueError):
            dgt.kv_read(kv.cache, layer, kv.one, kv.one, None, 1)
    assert not kv.calls
    k, v = dgt.kv_read(kv.cache, None, kv.one, kv.one, None, 1)
    assert k.shape == v.shape == (3, 1, 1, 64) and kv.calls[-1][1][1] == -1


class Device:
    """A host tensor that says it is on the device."""

    def __init__(self, *shape, dtype=torch.bfloat16, cuda=True):
        self.t, self.is_cuda = torch.zeros(shape, dtype=dtype), cuda

    def __getattr__(self, name):
        return getattr(self.t, name)


BAD_TENSORS = {
    "out on the host": dict(out=Device(1, 2, 64, cuda=False)),
    "out of another type": dict(out=Device(1, 2, 64, dtype=torch.float16)),
    "out of another shape": dict(out=Device(1, 64, 2)),
    "lse on the host": dict(lse=Device(1, 2, dtype=torch.float32, cuda=False)),
    "lse of another size": dict(lse=Device(1, 1, dtype=torch.float32)),
    "ws on the host": dict(ws=Device(4096, dtype=torch.uint8, cuda=False)),
    "status on the host": dict(status=Device(1, dtype=torch.int32, cuda=False)),
    "status of another type": dict(status=Device(1, dtype=torch.int64)),
    "an empty status": dict(status=Device(0, dtype=torch.int32)),
}


@pytest.mark.parametrize("what", list(BAD_TENSORS))
def test_attention_refuses(kv, what):
    good = dict(out=Device(1, 2, 64), lse=Device(1, 2, dtype=torch.float32), ws=Device(4096, dtype=torch.uint8),
                status=Device(1, dtype=torch.int32))
    dgt.kv_attention(kv.cache, 0, Device(1, 2, 64), kv.one, **good)
    assert len(kv.calls) == 1
    with pytest.raises(ValueError):
        dgt.kv_attention(kv.cache, 0, Device(1, 2, 64), kv.one, **{**good, **BAD_TENSORS[what]})
    assert len(kv.calls) == 1


@pytest.mark.parametrize("bad", [Device(1, dtype=torch.int32, cuda=False), Device(1, dtype=torch.int64)])
def test_every_call_checks_its_status(kv, bad):
    c, one, row = kv.cache, kv.one, Device(1, 1, 64)
    for call in (lambda: dgt.kv_append(c, 0, row, row, one, one, status=bad),
                 lambda: dgt.kv_read(c, 0, one, one, None, 1, status=bad),
                 lambda: dgt.kv_reserve(c, one, one, status=bad), lambda: dgt.kv_fork(c, one, one, status=bad),
                 lambda: dgt.kv_free(c, one, status=bad), lambda: dgt.kv_copy_pages(c, one, one, status=bad),
                 lambda: dgt.kv_compact(c, status=bad)):
        with pytest.raises(ValueError):
            call()
    assert not kv.calls


@pytest.mark.parametrize("size", [2 ** 30, 2 ** 32, 2 ** 32 + 5, 2 ** 40])
def test_a_window_past_every_position_stays_one(kv, size):
    # the library takes 32 bits; from 2^30 on a window is none, and first tokens are all
    dgt.kv_attention(kv.cache, 0, Device(1, 2, 64), kv.one, out=Device(1, 2, 64), ws=Device(4096, dtype=torch.uint8),
                     window=size, sinks=size)
    window, sinks = kv.calls[0][1][8:10]
    assert 2 ** 30 <= window < 2 ** 32 and 2 ** 30 <= sinks < 2 ** 32
