"""Decode steps with a Router and with norms behind their blocks, and a beam
search that uses the norms, the routing, the shared attention, the selection
and the reordering together.

Bound of a step against 64 bits: 1e-2 (residual) and 2e-2 (normed output), as
for the other steps, whose rounding of h, a and m to bf16 between products they
cover."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import decode_gemv_tensor_gb300 as dgt  # noqa: E402
import synthetic as S  # noqa: E402

BF16 = torch.bfloat16
HID, NQ, NKV, FFN, E, TOPK = 512, 512, 128, 256, 16, 4


def dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(BF16)


def vectors(count, seed, around=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return [(around + 0.2 * torch.randn(HID, device="cuda", generator=g)).to(BF16) for _ in range(count)]


def layers(count, moe, seed):
    k = E if moe else 1
    shapes = {"qkv": (NQ + 2 * NKV, HID), "o": (HID, NQ), "gate_up": (k * 2 * FFN, HID), "down": (k * HID, FFN)}
    host = [{p: S.weights(*s, (seed, l, i, 0), sigma=0.05) for i, (p, s) in enumerate(shapes.items())} for l in range(count)]
    r4 = [{p: dgt.load_r4(dgt.upload(dgt.pack(w, 2))) for p, w in L.items()} for L in host]
    return r4, [{p: dev(w).view(w.shape) for p, w in L.items()} for L in host]


def reference(bf, gammas, x, norms, depth, router=None, eps=1e-5):
    """The step in 64 bits, h, a and m rounded to bf16 where the step does."""
    d = lambda t: t.double()
    b = lambda t: t.to(BF16).double()
    r = lambda v: 1 / torch.sqrt((v * v).mean() + eps)
    normed = lambda v, w: v * r(v) * (norms.offset + d(w))

    def add(j, x, y):
        if norms.post is not None:
            y = normed(y, norms.post[j % len(norms.post)])
        if norms.gate is not None:
            y = y * d(norms.gate[j % len(norms.gate)])
        return norms.residual * x + norms.scale * y

    x, chosen = d(x), []
    for l in range(depth):
        W = {p: d(w) for p, w in bf[l].items()}
        h = b(normed(x, gammas[2 * l]))
        v = b((W["qkv"] @ h)[NQ + NKV:])
        x = add(2 * l, x, W["o"] @ v.repeat(NQ // NKV))
        h = b(normed(x, gammas[2 * l + 1]))
        silu = lambda gu: b(gu[:FFN] / (1 + torch.exp(-gu[:FFN])) * gu[FFN:])
        if router is None:
            y = W["down"] @ silu(W["gate_up"] @ h)
        else:
            s = torch.sigmoid(d(router.weights[l]) @ h)
            ids = torch.sort(s + d(router.bias[l]), descending=True, stable=True)[1][:TOPK]
            p = s[ids] / s[ids].sum() * router.kw["scale"]
            gu, dn = W["gate_up"].view(E, 2 * FFN, HID), W["down"].view(E, HID, FFN)
            y = sum(p[j] * (dn[ids[j]] @ silu(gu[ids[j]] @ h)) for j in range(TOPK))
            chosen.append(ids.int())
        x = add(2 * l + 1, x, y)
    return x, normed(x, gammas[2 * depth]), chosen


def near(got, want, bound):
    return float((got.double() - want).norm() / want.norm()) <= bound


NORMS = [dict(post=4, offset=1.0), dict(post=4, gate=4, scale=0.5, residual=0.75), dict(gate=2), dict()]


@pytest.mark.parametrize("kw", NORMS)
def test_dense_step_with_norms_behind_its_blocks(kw):
    kw = dict(kw)
    around = 1.0 - kw.get("offset", 0.0)
    for name, seed in (("post", 1), ("gate", 2)):
        if name in kw:
            kw[name] = vectors(kw[name], seed, around if name == "post" else 0.5)
    norms = dgt.StepNorms(**kw)
    r4, bf = layers(2, False, 21)
    gammas = vectors(5, 3, around)
    x0 = torch.randn(HID, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    want = reference(bf, gammas, x0, norms, 2)
    outs = []
    for W in (r4, bf):
        step = dgt.DecodeStep(W, gammas, norms=norms)
        x, out = (t.clone() for t in step(x0))
        assert near(x, want[0], 1e-2) and near(out, want[1], 2e-2)
        step.capture()
        assert all(torch.equal(a, b) for a, b in zip(step.replay(x0), (x, out)))
        outs.append((x, out))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    if not kw:
        plain = dgt.DecodeStep(bf, gammas)(x0)      # the same step, its norms' sums in another order
        assert near(outs[0][0], plain[0].double(), 1e-2)


def test_moe_step_routes_by_itself():
    r4, bf = layers(2, True, 22)
    gammas = vectors(5, 5)
    g = torch.Generator("cuda").manual_seed(6)
    weights = [(torch.randn(E, HID, device="cuda", generator=g) * 0.05).to(BF16) for _ in range(2)]
    bias = [0.1 * torch.randn(E, device="cuda", generator=g) for _ in range(2)]
    norms = dgt.StepNorms(post=vectors(4, 7))
    for seed in range(3):
        x0 = torch.randn(HID, device="cuda", generator=g)
        outs = []
        for W in (r4, bf):
            router = dgt.Router(weights, TOPK, score="sigmoid", bias=bias, scale=2.0)
            step = dgt.MoeDecodeStep(W, gammas, router, E, norms=norms)
            x, out = (t.clone() for t in step(x0))
            # the routing of the last layer, from the h that it had
            want = dgt.route(dgt.gemv_bf16(weights[1], step.h)[1].view(1, -1), TOPK, score="sigmoid", bias=bias[1], scale=2.0)
            assert torch.equal(router.ids, want[0]) and torch.equal(router.p, want[1])
            step.capture()
            assert all(torch.equal(a, b) for a, b in zip(step.replay(x0), (x, out)))
            ref = reference(bf, gammas, x0, norms, 2, router)
            if torch.equal(ref[2][-1], router.ids[0]):       # roundings of h may turn a choice next to another
                assert near(x, ref[0], 1e-2) and near(out, ref[1], 2e-2)
            outs.append((x, out))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
        # the same step with that routing given
        fixed = [(router.ids.view(-1).clone(), router.p.view(-1).clone())]
        one = dgt.MoeDecodeStep(bf[1:], gammas[2:], fixed, E, depth=1)
        own = dgt.MoeDecodeStep(bf[1:], gammas[2:], dgt.Router(weights[1:], TOPK, score="sigmoid", bias=bias[1:], scale=2.0),
                                E, depth=1)
        a, b = one(x0)[0].clone(), own(x0)[0].clone()
        if torch.equal(own.routes.ids.view(-1), fixed[0][0]) and torch.equal(own.routes.p.view(-1), fixed[0][1]):
            assert torch.equal(a, b)


def test_a_beam_search_over_shared_pages():
    """One layer: norm, attention over the shared prompt and the beams' own pages, norm, routed experts, norm, logits,
    selection, reordering.  What the cache holds for a beam is its own text's keys; what attention gives is what the
    attention that shares nothing gives; the selection is that of the logits."""
    hid, hq, hk, dim, vocab, beams, batch = 256, 8, 2, 64, 640, 4, 2
    g = torch.Generator("cuda").manual_seed(30)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    emb = r(vocab, hid)
    gam = [(1 + 0.1 * r(hid)).to(BF16) for _ in range(5)]
    Wqkv, Wo = (0.08 * r((hq + 2 * hk) * dim, hid)).to(BF16), (0.08 * r(hid, hq * dim)).to(BF16)
    Wr, Wup, Wdn = (0.1 * r(E, hid)).to(BF16), (0.08 * r(E * 128, hid)).to(BF16), (0.08 * r(E * hid, 128)).to(BF16)
    Wv = (0.3 * r(vocab, hid)).to(BF16)
    cache = dgt.KvCache(1, 64, hk, dim, max_seqs=batch * (beams + 1), max_pages=16)
    st = i32(0)
    prompts = (200, 131)
    keys = [[] for _ in range(batch * beams)]       # of each beam's own tokens, as they were appended
    for e, n in enumerate(prompts):
        start = dgt.kv_reserve(cache, i32(e), i32(n), status=st)
        dgt.kv_append(cache, 0, r(n, hk, dim).to(BF16), r(n, hk, dim).to(BF16), i32(e), start, cu=i32(0, n), status=st)
    seqs = torch.arange(batch, batch * (beams + 1), dtype=torch.int32, device="cuda").view(batch, beams)
    dgt.kv_fork(cache, i32(0, 0, 0, 0, 1, 1, 1, 1), seqs.view(-1), status=st)
    scores = torch.tensor([[0.0] + [-float("inf")] * (beams - 1)] * batch, device="cuda")
    done = torch.zeros(batch, beams, dtype=torch.uint8, device="cuda")
    token = torch.randint(0, vocab, (batch * beams,), generator=g, device="cuda")
    rows, ones = batch * beams, torch.ones(batch * beams, dtype=torch.int32, device="cuda")
    ws, bws = dgt.kv_attention_shared_workspace(cache, hq, batch, rows, rows), dgt.beam_workspace(batch, beams, vocab, beams)
    for step in range(30):
        x = emb[token]
        x, h = dgt.block_norm(x, pre=gam[0])
        qkv = dgt.gemm_bf16(Wqkv, h)[1]
        q, k, v = (t.view(rows, -1, dim) for t in qkv.split([hq * dim, hk * dim, hk * dim], dim=1))
        start = dgt.kv_reserve(cache, seqs.view(-1), ones, status=st)
        dgt.kv_append(cache, 0, k, v, seqs.view(-1), start, status=st)
        for b in range(rows):
            keys[b] = keys[b] + [k[b].float()]
        a = dgt.kv_attention_shared(cache, 0, q, seqs.view(-1), i32(0, 1), i32(*prompts), groups=i32(0, beams, rows), ws=ws,
                                    status=st, always=step % 2 == 0)
        plain = dgt.kv_attention(cache, 0, q, seqs.view(-1), status=st)
        # both are within 2^-8 of the value and 2^-10 of the mean of |v|, here below 1.5
        assert bool(((a.float() - plain.float()).abs() <= 2.0 ** -7 * plain.float().abs() + 2.0 ** -8).all())
        y = dgt.gemm_bf16(Wo, a.view(rows, -1))[0]
        x, h = dgt.block_norm(x, y, post=gam[1], pre=gam[2], x_out=x)
        ids, p = dgt.route(h.float() @ Wr.float().T, 2, score="sigmoid")
        up = dgt.moe_gemv_bf16(Wup, E, ids, None, h, status=st)[0]
        assert dgt.read_status(st) == 0
        m = torch.nn.functional.silu(up).to(BF16).view(rows * 2, 128)
        down = dgt.moe_gemv_bf16(Wdn, E, ids.view(-1, 1), None, m, status=st)[0].view(rows, 2, hid)
        assert dgt.read_status(st) == 0
        x, h = dgt.block_norm(x, (down * p[..., None]).sum(1), post=gam[3], pre=gam[4], x_out=x)
        logits = dgt.gemm_bf16(Wv, h)[0]
        parent, nt, total, nd = dgt.beam_select(logits, scores, beams, eos=7, done=done, ws=bws)
        full = scores.double()[..., None] + torch.log_softmax(logits.double(), -1).view(batch, beams, vocab)
        only = torch.full_like(full, -float("inf"))
        only[..., 7] = scores.double()
        full = torch.where(done[..., None] != 0, only, full)
        best = full.view(batch, -1).topk(beams)[0]
        assert bool(((total.double() - best).abs() <= 2.0 ** -17).all())
        pick = full.gather(1, parent.long()[..., None].expand(-1, -1, vocab)).gather(2, nt.long()[..., None])[..., 0]
        assert bool(((pick - best).abs() <= 2.0 ** -30 * best.abs() + 1e-9).all())
        dgt.kv_reorder(cache, seqs, parent, status=st)
        keys = [keys[e * beams + j] for e in range(batch) for j in parent[e].tolist()]
        scores, done, token = total, nd, nt.view(-1).long()
        assert dgt.read_status(st) == 0
    t = cache.table.flatten().long()
    assert torch.equal(cache.refs, torch.bincount(t[t >= 0], minlength=cache.pages).int())
    for b in range(rows):
        n = len(keys[b])
        got = dgt.kv_read(cache, 0, seqs.view(-1)[b:b + 1], i32(prompts[b // beams]), i32(0, n), n)[0].float()
        want = torch.stack(keys[b])
        # half a step of e4m3, 2^-4, twice where a block's scale grew, and its smallest step, 2^-10 of the block's range
        assert bool(((got - want).abs() <= 2.0 ** -3 * want.abs() + 2.0 ** -8).all())
