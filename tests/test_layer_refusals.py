"""Refusals of the norm, routing, beam and reorder entry points: returned
before any device call, so this machine needs no device."""
import ctypes as C
import struct

import pytest

torch = pytest.importorskip("torch")
import decode_gemv_tensor_gb300 as dgt  # noqa: E402

ARG, SHAPE = -1, -2
P = 1 << 20     # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    return dgt.lib()


def norm(x=P, x_out=P, y=P, h=P, pre=P, post=0, gate=0, xs=64, xos=64, ys=64, hs=64, gs=0, xf=1, yf=1):
    return dgt._pack_norm(x, x_out, y, h, pre, post, gate, xs, xos, ys, hs, gs, xf, yf)


def test_structs_have_the_header_s_size():
    assert struct.calcsize("=7Q5q2I") == 104 and struct.calcsize("=8IfIQ") == 48


@pytest.mark.parametrize("change,code", [
    (dict(x=0), ARG), (dict(x_out=0, h=0, pre=0), ARG), (dict(pre=0), ARG), (dict(h=0), ARG),
    (dict(y=0, post=P), ARG), (dict(y=0, gate=P), ARG), (dict(xf=2), ARG), (dict(yf=2), ARG),
    (dict(x=P + 2), ARG), (dict(x=P + 1, xf=0, x_out=P), ARG), (dict(y=P + 2), ARG), (dict(h=P + 1), ARG),
    (dict(post=P + 1), ARG)])
def test_block_norm_refuses(lib, change, code):
    assert lib.dgt_block_norm(norm(**change), 1, 64, 1.0, 1.0, 0.0, 1e-5, None) == code


def test_block_norm_sizes(lib):
    call = lambda rows=1, n=64, eps=1e-5: lib.dgt_block_norm(norm(), rows, n, 1.0, 1.0, 0.0, eps, None)
    assert call(n=0) == SHAPE and call(n=32769) == SHAPE and call(rows=(1 << 24) + 1) == SHAPE
    assert call(eps=-1.0) == ARG and call(eps=float("nan")) == ARG
    assert call(rows=0) == 0
    assert lib.dgt_block_norm(None, 1, 64, 1.0, 1.0, 0.0, 1e-5, None) == ARG


def router(experts=64, topk=4, groups=1, group_topk=1, group_best=2, f32=1, sigmoid=0, renorm=1, bias=0):
    return dgt._pack_router(experts, topk, groups, group_topk, group_best, f32, sigmoid, renorm, 1.0, 0, bias)


@pytest.mark.parametrize("change,code", [
    (dict(experts=0), SHAPE), (dict(experts=1025), SHAPE), (dict(topk=0), SHAPE), (dict(topk=33), SHAPE),
    (dict(experts=3), SHAPE), (dict(groups=0), SHAPE), (dict(groups=5), SHAPE), (dict(experts=66, groups=33), SHAPE),
    (dict(groups=4, group_topk=0), SHAPE), (dict(groups=4, group_topk=5), SHAPE),
    (dict(groups=32, group_topk=1, topk=3), SHAPE), (dict(group_best=0), ARG), (dict(group_best=3), ARG),
    (dict(f32=2), ARG), (dict(sigmoid=2), ARG), (dict(renorm=2), ARG), (dict(bias=P + 2), ARG)])
def test_route_refuses(lib, change, code):
    assert lib.dgt_route(router(**change), P, 64, 1, P, P, None) == code


def test_route_pointers_and_sizes(lib):
    call = lambda l=P, t=1, ids=P, p=P, f32=1: lib.dgt_route(router(f32=f32), l, 64, t, ids, p, None)
    assert call(l=None) == ARG and call(ids=None) == ARG and call(p=None) == ARG
    assert call(l=P + 2) == ARG and call(l=P + 1, f32=0) == ARG and call(ids=P + 2) == ARG and call(p=P + 1) == ARG
    assert call(t=(1 << 24) + 1) == SHAPE and call(t=0) == 0
    assert lib.dgt_route(None, P, 64, 1, P, P, None) == ARG


def beam(lib, l=P, f32=0, s=P, done=None, eos=-1, batch=2, beams=4, vocab=1000, n=8, parent=P, token=P, total=4 * P,
         done_out=None, ws=P, short=0):
    need = int(lib.dgt_beam_workspace_bytes(batch, beams, vocab, n))
    return lib.dgt_beam_select(l, f32, vocab, s, done, eos, batch, beams, vocab, n, parent, token, total, done_out, ws,
                               need - short, None)


@pytest.mark.parametrize("change,code", [
    (dict(beams=0), SHAPE), (dict(beams=65), SHAPE), (dict(n=0), SHAPE), (dict(n=65), SHAPE),
    (dict(beams=33, n=63), SHAPE), (dict(vocab=0), SHAPE), (dict(vocab=(1 << 24) + 1), SHAPE),
    (dict(batch=65537), SHAPE), (dict(l=None), ARG), (dict(s=None), ARG), (dict(parent=None), ARG),
    (dict(token=None), ARG), (dict(total=None), ARG), (dict(f32=2), ARG), (dict(l=P + 1), ARG),
    (dict(l=P + 2, f32=1), ARG), (dict(s=P + 2), ARG), (dict(done=P), ARG), (dict(done=P, eos=1000), ARG),
    (dict(done_out=P), ARG), (dict(s=2 * P, total=2 * P), ARG), (dict(done=2 * P, eos=1, done_out=2 * P, total=3 * P), ARG),
    (dict(ws=None), ARG), (dict(ws=P + 64), ARG), (dict(short=1), ARG)])
def test_beam_select_refuses(lib, change, code):
    assert beam(lib, **change) == code


def test_beam_workspace(lib):
    size = lib.dgt_beam_workspace_bytes
    assert size(0, 4, 1000, 8) == 0 and size(1, 0, 1000, 8) == 0 and size(1, 4, 0, 8) == 0 and size(1, 4, 1000, 0) == 0
    assert size(1, 4, 1000, 65) == 0
    assert 0 < size(1, 1, 10, 1) < size(64, 8, 262144, 64)
    assert beam(lib, batch=0) == 0


def test_reorder_refuses(lib):
    c = dgt.KvCacheStruct(2, 8, 4, 128, 3, 4, P, P, P, P, P, P, P)
    call = lambda c=C.byref(c), s=P, p=P, g=1, b=2: lib.dgt_kv_reorder(c, s, p, None, g, b, None, None)
    assert call(s=None) == ARG and call(p=None) == ARG and call(c=None) == ARG
    assert call(g=1025, b=1) == SHAPE and call(g=1 << 31, b=1 << 31) == SHAPE
    assert call(g=0) == 0 and call(b=0) == 0


# ---- the Python calls' own checks (tensors of this machine: every call wants CUDA ones)
def test_calls_want_cuda_tensors():
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError):
        dgt.block_norm(x)
    with pytest.raises(ValueError):
        dgt.route(x, 2)
    with pytest.raises(ValueError):
        dgt.beam_select(x, torch.zeros(1, 2), 2)
    with pytest.raises(ValueError):
        dgt.route(x.long(), 2)
    with pytest.raises(ValueError):
        dgt.beam_select(x.view(2, 8, 8), torch.zeros(1, 2), 2)


def test_shared_attention_refuses(lib):
    def cache(**kw):
        f = dict(layers=2, pages=8, kv_heads=4, head_dim=128, max_seqs=3, max_pages=4, k=P, v=P, k_scale=P, v_scale=P,
                 refs=P, table=P, lens=P)
        f.update(kw)
        return C.byref(dgt.KvCacheStruct(*f.values()))

    def heads(n, data=P, ts=None):
        return C.byref(dgt.HeadsStruct(data, n * 128 if ts is None else ts, 128, n, 0))

    need = int(lib.dgt_kv_attention_shared_workspace_bytes(cache(), 8, 2, 4, 4))
    assert need > 0
    size = lib.dgt_kv_attention_shared_workspace_bytes
    assert size(None, 8, 1, 1, 1) == 0 and size(cache(), 2, 1, 1, 1) == 0 and size(cache(), 8, 0, 1, 1) == 0

    def call(c=None, layer=0, q=heads(8), t=4, s=P, cu=None, b=4, prefix=P, shared=P, at=P, g=2, out=P, ws=P, n=need,
             flags=0):
        return lib.dgt_kv_attention_shared(c or cache(), layer, q, t, s, cu, b, prefix, shared, at, g, 1.0, out, None,
                                           ws, n, None, flags, None)

    assert call(c=cache(head_dim=96)) == SHAPE and call(c=cache(k=None)) == ARG and call(layer=2) == ARG
    assert call(q=None) == ARG and call(s=None) == ARG and call(out=None) == ARG and call(out=P + 8) == ARG
    assert call(prefix=None) == ARG and call(shared=None) == ARG and call(at=None) == ARG and call(g=0) == ARG
    assert call(g=65537) == SHAPE and call(t=5) == ARG and call(t=(1 << 24) + 1, cu=P) == SHAPE
    assert call(q=heads(6)) == SHAPE and call(q=heads(4 * 65)) == SHAPE and call(q=heads(8, ts=1025)) == ARG
    assert call(ws=None) == ARG and call(ws=P + 64) == ARG and call(n=need - 1) == ARG
    assert call(flags=1 << 3) == ARG and call(t=0, b=0) == 0
