"""Refusals of the rotary, cache, attention and page entry points: returned
before any device call, so this machine needs no device."""
import ctypes as C

import pytest

pytest.importorskip("torch")
import decode_gemv_tensor_gb300 as dgt  # noqa: E402

ARG, SHAPE = -1, -2
P = 1 << 20     # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    return dgt.lib()


def cache(**kw):
    f = dict(layers=2, pages=8, kv_heads=4, head_dim=128, max_seqs=3, max_pages=4, k=P, v=P, k_scale=P, v_scale=P,
             refs=P, table=P, lens=P)
    f.update(kw)
    return dgt.KvCacheStruct(*f.values())


def heads(n, data=P, ts=None, hs=128):
    return C.byref(dgt.HeadsStruct(data, n * 128 if ts is None else ts, hs, n, 0))


BAD_CACHES = [(dict(k=None), ARG), (dict(v=None), ARG), (dict(k_scale=None), ARG), (dict(table=None), ARG),
              (dict(k=P + 8), ARG), (dict(v=P + 4), ARG), (dict(head_dim=96), SHAPE), (dict(head_dim=0), SHAPE),
              (dict(head_dim=512), SHAPE), (dict(kv_heads=0), SHAPE), (dict(kv_heads=257), SHAPE),
              (dict(layers=0), SHAPE), (dict(pages=0), SHAPE), (dict(pages=(1 << 22) + 1), SHAPE),
              (dict(max_seqs=0), SHAPE), (dict(max_pages=0), SHAPE)]


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(lib, change, code):
    c = C.byref(cache(**change))
    big = 1 << 30
    assert lib.dgt_kv_append(c, 0, heads(4), heads(4), 1, P, P, None, 1, None, None) == code
    assert lib.dgt_kv_read(c, 0, P, P, None, 1, 1, P, P, None, None) == code
    assert lib.dgt_kv_attention(c, 0, heads(8), 1, P, None, 1, 1.0, 0, 0, P, None, P, big, None, None) == code
    assert lib.dgt_kv_copy_pages(c, P, P, 1, None, None) == code
    assert lib.dgt_kv_fork(c, P, P, 1, None, None) == code
    assert lib.dgt_kv_reserve(c, P, P, 1, P, P, big, None, None) == code
    assert lib.dgt_kv_free(c, P, 1, None, None) == code
    assert lib.dgt_kv_compact(c, None, P, big, None, None) == code


def test_append_refusals(lib):
    c = C.byref(cache())
    call = lambda layer=0, k=heads(4), v=heads(4), t=1, s=P, st=P, cu=None, b=1: lib.dgt_kv_append(
        c, layer, k, v, t, s, st, cu, b, None, None)
    assert call(layer=2) == ARG
    assert call(k=None) == ARG and call(v=None) == ARG and call(s=None) == ARG and call(st=None) == ARG
    assert call(k=heads(3)) == ARG
    assert call(k=heads(4, data=P + 2)) == ARG and call(v=heads(4, ts=516)) == ARG and call(v=heads(4, hs=4)) == ARG
    assert call(t=2) == ARG                       # one row each wants tokens == batch
    assert call(t=(1 << 24) + 1, cu=P) == SHAPE and call(t=65537, b=65537) == SHAPE
    assert call(t=0, b=0) == 0


def test_read_refusals(lib):
    c = C.byref(cache())
    call = lambda layer=0, s=P, f=P, cu=None, b=1, t=1, k=P, v=P: lib.dgt_kv_read(c, layer, s, f, cu, b, t, k, v,
                                                                               None, None)
    assert call(layer=2) == ARG and call(layer=-2) == ARG and call(s=None) == ARG and call(f=None) == ARG
    assert call(k=P + 8) == ARG and call(t=3) == ARG
    assert call(t=0, b=0) == 0 and call(k=None, v=None) == 0


def test_attention_refusals(lib):
    c = C.byref(cache())
    need = int(lib.dgt_kv_attention_workspace_bytes(c, 8, 1, 1))
    call = lambda layer=0, q=heads(8), t=1, s=P, cu=None, b=1, out=P, ws=P, n=need: lib.dgt_kv_attention(
        c, layer, q, t, s, cu, b, 1.0, 0, 0, out, None, ws, n, None, None)
    assert call(layer=2) == ARG and call(q=None) == ARG and call(s=None) == ARG and call(out=None) == ARG
    assert call(out=P + 8) == ARG and call(q=heads(8, data=P + 8)) == ARG and call(q=heads(8, ts=1025)) == ARG
    assert call(q=heads(6)) == SHAPE and call(q=heads(4 * 65)) == SHAPE
    assert call(t=2) == ARG and call(t=(1 << 24) + 1, cu=P) == SHAPE
    if need:
        assert call(n=need - 1) == ARG and call(ws=None) == ARG
    assert call(t=0, b=0) == 0


def test_page_refusals(lib):
    c = C.byref(cache())
    need = int(lib.dgt_kv_pages_workspace_bytes(c))
    assert need >= 4 * (3 * 8 + 1)
    assert lib.dgt_kv_copy_pages(c, None, P, 1, None, None) == ARG
    assert lib.dgt_kv_copy_pages(c, P, None, 1, None, None) == ARG
    assert lib.dgt_kv_copy_pages(c, None, None, 0, None, None) == 0
    assert lib.dgt_kv_fork(c, None, P, 1, None, None) == ARG and lib.dgt_kv_fork(c, P, P, 0, None, None) == 0
    assert lib.dgt_kv_free(c, None, 1, None, None) == ARG and lib.dgt_kv_free(c, None, 0, None, None) == 0
    r = lambda s=P, k=P, n=1, st=P, ws=P, nb=need: lib.dgt_kv_reserve(c, s, k, n, st, ws, nb, None, None)
    assert r(s=None) == ARG and r(k=None) == ARG and r(st=None) == ARG and r(ws=None) == ARG and r(nb=need - 1) == ARG
    assert r(n=1025) == SHAPE and r(n=0) == 0
    assert lib.dgt_kv_compact(c, None, None, need, None, None) == ARG
    assert lib.dgt_kv_compact(c, None, P, need - 1, None, None) == ARG


def test_rotate_refusals(lib):
    rot = lambda dim=128, axes=1, f=P, ax=P: C.byref(dgt.RotaryStruct(dim, axes, 0, 0, f, ax))
    call = lambda r=rot(), q=heads(8), k=None, qo=heads(8), ko=None, d=128, t=1, pos=P: lib.dgt_rotate(
        r, q, k, qo, ko, d, t, pos, None)
    assert call(r=None) == ARG and call(q=None) == ARG and call(qo=None) == ARG and call(pos=None) == ARG
    assert call(r=rot(f=None)) == ARG and call(r=rot(ax=None)) == ARG
    assert call(k=heads(2)) == ARG and call(qo=heads(4)) == ARG and call(q=heads(8, data=P + 8)) == ARG
    assert call(r=rot(dim=144)) == SHAPE and call(r=rot(dim=24)) == SHAPE and call(r=rot(dim=0)) == SHAPE
    assert call(r=rot(axes=0)) == SHAPE and call(r=rot(axes=9)) == SHAPE and call(d=1040) == SHAPE
    assert call(d=120) == SHAPE and call(q=heads(0), qo=heads(0)) == SHAPE and call(t=(1 << 24) + 1) == SHAPE
    assert call(t=0) == 0


def test_rotary_frequencies(lib):
    import math
    import numpy as np
    out = np.zeros(64, np.uint64)
    for base in (10000.0, 500000.0, 1.5):
        assert lib.dgt_rotary_freqs(base, 128, out.ctypes.data) == 0
        for i in range(64):
            f = math.ldexp(base ** (-2 * i / 128) / (2 * math.pi), 64)
            # the nearest integer (a half) to a product of roundings: pow and the division on
            # either side, four half-steps of 2^-53
            assert abs(int(out[i]) - f) <= 0.5 + f * 2.0 ** -51
    for base, dim, code in ((1.0, 128, ARG), (math.inf, 128, ARG), (math.nan, 128, ARG), (1e4, 0, SHAPE),
                            (1e4, 7, SHAPE), (1e4, 1026, SHAPE)):
        assert lib.dgt_rotary_freqs(base, dim, out.ctypes.data) == code
    assert lib.dgt_rotary_freqs(1e4, 128, None) == ARG


def test_status_string_of_a_full_pool(lib):
    assert lib.dgt_status_string(-9) == b"no room left in the cache"
    assert "no room left" in str(dgt.DgtError(-9, "x"))


def test_block_layout_is_a_permutation():
    # the layout that dgt.h documents: every byte of a block is one (token, dimension)
    for dim in (64, 128, 256):
        panel = min(dim, 128)
        seen = set()
        for t in range(64):
            for d in range(dim):
                c = d % panel // 16
                x = t % 8 if dim > 64 else t // 2 % 4
                seen.add(d // panel * 64 * panel + t * panel + ((c ^ x) * 16) + d % 16)
        assert seen == set(range(64 * dim))
        assert {d * 64 + t for d in range(dim) for t in range(64)} == set(range(64 * dim))


def test_attention_flags(lib):
    c = C.byref(cache())
    for flags in (1, 4, 1 << 15):
        assert lib.dgt_kv_attention_ex(c, 0, heads(8), 1, P, None, 1, 1.0, 0, 0, P, None, P, 1 << 30, None, flags,
                                       None) == ARG
