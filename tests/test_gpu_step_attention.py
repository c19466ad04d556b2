"""Decode steps with attention over the 8-bit cache: R4 and BF16 weights give
bit-identical steps, a captured step moves on token by token, several steps
agree with a 64-bit restatement, a forked sequence goes its own way, and a full
pool is reported.

Bound against 64 bits: 1e-2 (residual) and 2e-2 (normed output), as for the
step without attention, whose rounding of h, a and m to bf16 between products
they cover.  That h differs by a bf16 step in places makes k and v differ by
2^-9 or so, and a few elements in a hundred then take the neighbouring e4m3
code, a step of 2^-3: so the restatement attends to the cache's own values (the
codes are held to their definition elsewhere), and its own k and v are held to
them by both sides' half a step, 2^-4 each, and the 1e-2."""
import numpy as np
import pytest

import kv_ref as R
import oracle
import synthetic as S

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def dgt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import decode_gemv_tensor_gb300 as d
    d.lib()
    return d


def _dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


HID, NQ, NKV, FFN, DIM = 512, 512, 128, 1024, 64     # 8 query heads, 2 kv heads


def _host(nl, seed):
    shapes = {"q": (NQ, HID), "k": (NKV, HID), "v": (NKV, HID), "o": (HID, NQ), "gate": (FFN, HID), "up": (FFN, HID),
              "down": (HID, FFN)}
    # weights of a size that makes scores of order one
    return [{p: S.weights(*shp, (seed, l, i, 0), sigma=0.05) for i, (p, shp) in enumerate(shapes.items())}
            for l in range(nl)]


def _layers(dgt, host, fused):
    out = []
    for L in host:
        W = dict(L)
        if fused:
            W = {"qkv": np.concatenate([L["q"], L["k"], L["v"]]), "o": L["o"],
                 "gate_up": np.concatenate([L["gate"], L["up"]]), "down": L["down"]}
        out.append(W)
    r4 = [{p: dgt.load_r4(dgt.upload(dgt.pack(w, 2))) for p, w in L.items()} for L in out]
    bf = [{p: _dev(w).view(w.shape) for p, w in L.items()} for L in out]
    return r4, bf


def _gammas(nl, seed):
    g = np.random.default_rng(seed)
    return [S.f32_to_bf16_bits((1 + 0.1 * g.normal(size=HID)).astype(np.float32)) for _ in range(2 * nl + 1)]


def _attention(dgt, depth, window=0, sinks=0, pages=12):
    c = dgt.KvCache(depth, pages, NKV // DIM, DIM, max_seqs=3, max_pages=8)
    return dgt.StepAttention(c, dgt.Rotary(DIM), seq=1, window=window, sinks=sinks)


def _f64(bits):
    return oracle.bf16_to_f64(bits)


def _round(x):
    return _f64(oracle.f64_to_bf16(np.ascontiguousarray(x)))


def _reference(host, gam, xs, depth, window, sinks, cached):
    """Steps on the inputs xs in 64 bits, rounded to bf16 where the step is;
    cached[l]: the keys and values that the step's cache ended up with, token
    by token as they were read after each (list of (k, v))."""
    nl = len(host)
    W = [{p: _f64(w) for p, w in L.items()} for L in host]
    heads, kvh = NQ // DIM, NKV // DIM
    half = DIM // 2
    inv = 10000.0 ** (-2.0 * np.arange(half) / DIM)
    norm = lambda x, g: _round(oracle.rmsnorm_eps_f64(x, g, 1e-5))
    out = []
    for pos, x0 in enumerate(xs):
        x = x0.astype(np.float64).copy()
        c, s = np.cos(pos * inv), np.sin(pos * inv)

        def turn(v):
            v = v.reshape(-1, DIM)
            a, b = v[:, :half], v[:, half:]
            return _round(np.concatenate([a * c - b * s, b * c + a * s], 1))
        for l in range(depth):
            w = W[l % nl]
            h = norm(x, gam[(2 * l) % (2 * nl)])
            q, k, v = (_round(w[p] @ h) for p in ("q", "k", "v"))
            kk, vv = cached[pos][0][l], cached[pos][1][l]
            for c8, y in ((kk[pos], turn(k)), (vv[pos], v.reshape(-1, DIM))):
                assert np.linalg.norm(c8 - y) <= (2 * 2.0 ** -4 + 1e-2) * np.linalg.norm(y)
            a = R.attention(turn(q)[None], kk, vv, pos, window, sinks, DIM ** -0.5)[0]
            x = x + w["o"] @ _round(a.reshape(-1))
            h = norm(x, gam[(2 * l + 1) % (2 * nl)])
            x = x + w["down"] @ _round(oracle.silu_mul_f64(w["gate"] @ h, w["up"] @ h))
        out.append((x, norm(x, gam[-1])))
    return out


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 2)])
def test_steps_twins_graph_and_64_bits(dgt, fused, window, sinks):
    depth, nl, steps = 3, 2, 70          # past a page's end
    host, gam = _host(nl, 701), _gammas(nl, 702)
    r4, bf = _layers(dgt, host, fused)
    gd = [_dev(x) for x in gam]
    g = np.random.default_rng(703)
    xs = [g.normal(size=HID).astype(np.float32) for _ in range(steps)]
    ar, ab, ag = (_attention(dgt, depth, window, sinks) for _ in range(3))
    sr, sb = dgt.DecodeStep(r4, gd, depth=depth, attention=ar), dgt.DecodeStep(bf, gd, depth=depth, attention=ab)
    sg = dgt.DecodeStep(r4, gd, depth=depth, attention=ag)
    sg(torch.from_numpy(xs[0]).cuda())
    dgt.kv_free(ag.cache, ag.seq)        # the captured step begins anew
    sg.capture()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    cached, got = [], []
    for i, x0 in enumerate(xs):
        xd = torch.from_numpy(x0).cuda()
        xr, hr = (t.clone() for t in sr(xd))
        xb, hb = sb(xd)
        assert torch.equal(xr.view(torch.int32), xb.view(torch.int32)) and torch.equal(hr.view(torch.int16), hb.view(torch.int16))
        xg, hg = sg.replay(xd)
        assert torch.equal(xg.view(torch.int32), xr.view(torch.int32)) and torch.equal(hg.view(torch.int16), hr.view(torch.int16))
        got.append((xr.double().cpu().numpy(), hr.double().cpu().numpy()))
        cached.append([t.double().cpu().numpy() for t in
                       dgt.kv_read(ar.cache, None, i32([1]), i32([0]), i32([0, i + 1]), i + 1)])
    ref = _reference(host, gam, xs, depth, window, sinks, cached)
    for i, ((xr, hr), (xo, ho)) in enumerate(zip(got, ref)):
        ex, eh = np.linalg.norm(xr - xo) / np.linalg.norm(xo), np.linalg.norm(hr - ho) / np.linalg.norm(ho)
        assert ex <= 1e-2 and eh <= 2e-2, (i, ex, eh)
    for a in (ar, ab, ag):
        assert a.status.item() == 0 and a.cache.lens.tolist() == [0, steps, 0]


def test_a_forked_sequence_goes_its_own_way(dgt):
    # two continuations of one beginning share its pages until they write, and give what separate sequences give
    depth, nl = 2, 1
    host, gam = _host(nl, 711), _gammas(nl, 712)
    r4, _ = _layers(dgt, host, True)
    gd = [_dev(x) for x in gam]
    g = np.random.default_rng(713)
    x = [torch.from_numpy(g.normal(size=HID).astype(np.float32)).cuda() for _ in range(9)]

    def run(step, xs):
        return [step(v)[0].clone() for v in xs]
    alone = []
    for tail in (x[5:7], x[7:9]):
        a = _attention(dgt, depth)
        alone.append(run(dgt.DecodeStep(r4, gd, depth=depth, attention=a), x[:5] + tail)[-2:])
    a = _attention(dgt, depth)
    step = dgt.DecodeStep(r4, gd, depth=depth, attention=a)
    run(step, x[:5])
    i32 = lambda v: torch.tensor([v], dtype=torch.int32, device="cuda")
    dgt.kv_fork(a.cache, i32(1), i32(2), status=a.status)
    b = dgt.StepAttention(a.cache, a.rotary, seq=2)
    other = dgt.DecodeStep(r4, gd, depth=depth, attention=b)
    got = [run(step, x[5:7]), run(other, x[7:9])]
    for p, q in zip(alone, got):
        for u, v in zip(p, q):
            assert torch.equal(u.view(torch.int32), v.view(torch.int32))
    assert a.cache.refs.sum().item() == 2 and a.cache.lens.tolist() == [0, 7, 7]
    # moved together and on
    dgt.kv_free(a.cache, i32(1))
    dgt.kv_compact(a.cache)
    before = step.attention.status.item()
    y = run(other, [x[0]])[0]
    c = _attention(dgt, depth)
    want = run(dgt.DecodeStep(r4, gd, depth=depth, attention=c), x[:5] + x[7:9] + [x[0]])[-1]
    assert before == 0 and torch.equal(y.view(torch.int32), want.view(torch.int32))


def test_a_full_pool_is_reported_and_the_step_ends(dgt):
    depth, nl = 1, 1
    host, gam = _host(nl, 721), _gammas(nl, 722)
    r4, _ = _layers(dgt, host, False)
    a = _attention(dgt, depth, pages=1)
    step = dgt.DecodeStep(r4, [_dev(x) for x in gam], depth=depth, attention=a)
    x = torch.randn(HID, device="cuda")
    for _ in range(64):
        step(x)
    assert a.status.item() == 0 and a.cache.lens[1] == 64
    step(x)
    assert a.status.item() == -9 and a.cache.lens[1] == 64


def test_step_attention_arguments(dgt):
    host, gam = _host(1, 731), _gammas(1, 732)
    r4, _ = _layers(dgt, host, False)
    gd = [_dev(x) for x in gam]
    with pytest.raises(ValueError):      # more layers than the cache has
        dgt.DecodeStep(r4, gd, depth=3, attention=_attention(dgt, 2))
    c = dgt.KvCache(1, 4, 3, DIM, max_seqs=1, max_pages=2)
    with pytest.raises(ValueError):      # query heads that three kv heads do not divide
        dgt.DecodeStep(r4, gd, attention=dgt.StepAttention(c, dgt.Rotary(DIM)))
    with pytest.raises(ValueError):
        dgt.StepAttention(c, dgt.Rotary(DIM, sections=[16, 16]))


def test_moe_step_with_attention(dgt):
    E, topk, ffn = 4, 2, 256
    shapes = {"q": (NQ, HID), "k": (NKV, HID), "v": (NKV, HID), "o": (HID, NQ), "gate": (E * ffn, HID),
              "up": (E * ffn, HID), "down": (E * HID, ffn)}
    host = [{p: S.weights(*shp, (741, 0, i, 0)) for i, (p, shp) in enumerate(shapes.items())}]
    r4 = [{p: dgt.load_r4(dgt.upload(dgt.pack(w, 2))) for p, w in L.items()} for L in host]
    bf = [{p: _dev(w).view(w.shape) for p, w in L.items()} for L in host]
    gd = [_dev(x) for x in _gammas(1, 742)]
    ids, p = S.routing(1, E, topk, (743, 777, 0, 0))
    routes = [(torch.from_numpy(ids.reshape(-1)).cuda(), torch.from_numpy(p.reshape(-1)).cuda())]
    ar, ab = _attention(dgt, 2), _attention(dgt, 2)
    sr = dgt.MoeDecodeStep(r4, gd, routes, E, depth=2, attention=ar)
    sb = dgt.MoeDecodeStep(bf, gd, routes, E, depth=2, attention=ab)
    plain = dgt.MoeDecodeStep(r4, gd, routes, E, depth=2)
    g = np.random.default_rng(744)
    for i in range(3):
        x = torch.from_numpy(g.normal(size=HID).astype(np.float32)).cuda()
        xr, xb = sr(x)[0].clone(), sb(x)[0].clone()
        assert torch.equal(xr.view(torch.int32), xb.view(torch.int32))
        if i:
            assert not torch.equal(xr, plain(x)[0])
    assert ar.cache.lens.tolist() == [0, 3, 0]
