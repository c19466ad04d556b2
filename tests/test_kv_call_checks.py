"""What the Python calls of the cache and the attention refuse themselves,
before the library is called: tensors on the host stand for wrong ones, so no
device is needed."""
import types

import pytest

torch = pytest.importorskip("torch")
import decode_gemv_tensor_gb300 as dgt  # noqa: E402


@pytest.fixture
def kv(monkeypatch):
    """A cache, and a library whose calls are counted and succeed."""
    cache = dgt.KvCache(3, 2, 1, 64, max_seqs=1, max_pages=2, device="cpu")
    calls = []

    class Library:
        def __getattr__(self, name):
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
