"""Rows without an entry to own them are refused, on the host."""
import ctypes as C

import pytest

pytest.importorskip("torch")
import decode_gemv_tensor_gb300 as dgt  # noqa: E402

P = 1 << 20     # an aligned address that nothing reads


def test_rows_of_an_empty_batch():
    lib = dgt.lib()
    c = C.byref(dgt.KvCacheStruct(2, 8, 4, 128, 3, 4, P, P, P, P, P, P, P))
    h = lambda n: C.byref(dgt.HeadsStruct(P, n * 128, 128, n, 0))
    for cu in (None, P):
        assert lib.dgt_kv_append(c, 0, h(4), h(4), 5, P, P, cu, 0, None, None) == -1
        assert lib.dgt_kv_read(c, 0, P, P, cu, 0, 5, P, P, None, None) == -1
        assert lib.dgt_kv_attention(c, 0, h(8), 5, P, cu, 0, 1.0, 0, 0, P, None, P, 1 << 30, None, None) == -1
        assert lib.dgt_kv_append(c, 0, h(4), h(4), 0, P, P, cu, 0, None, None) == 0
        assert lib.dgt_kv_attention(c, 0, h(8), 0, P, cu, 0, 1.0, 0, 0, P, None, P, 1 << 30, None, None) == 0
