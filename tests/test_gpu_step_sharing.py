"""Steps that share a StepAttention: a captured step and what comes after it."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HID, NKV, FFN, DIM = 256, 128, 256, 64     # 4 query heads, 2 kv heads


@pytest.fixture(scope="module")
def dgt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import decode_gemv_tensor_gb300 as d
    d.lib()
    return d


def layers(n, seed):
    g = np.random.default_rng(seed)
    shapes = {"q": (HID, HID), "k": (NKV, HID), "v": (NKV, HID), "o": (HID, HID), "gate": (FFN, HID), "up": (FFN, HID),
              "down": (HID, FFN)}
    rand = lambda *s: torch.from_numpy((0.05 * g.normal(size=s)).astype(np.float32)).cuda().bfloat16()
    return ([{p: rand(*s) for p, s in shapes.items()} for _ in range(n)],
            [torch.ones(HID, device="cuda").bfloat16() for _ in range(2 * n + 1)])


def attention(dgt, held):
    """A StepAttention whose sequence holds `held` tokens."""
    c = dgt.KvCache(2, 24, NKV // DIM, DIM, max_seqs=2, max_pages=24)
    g = np.random.default_rng(held)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    start = dgt.kv_reserve(c, i32([1]), i32([held]))
    for l in range(2 if held else 0):
        k, v = (torch.from_numpy(g.normal(size=(held, NKV // DIM, DIM)).astype(np.float32)).cuda().bfloat16()
                for _ in range(2))
        dgt.kv_append(c, l, k, v, i32([1]), start, cu=i32([0, held]))
    return dgt.StepAttention(c, dgt.Rotary(DIM), seq=1)


def inputs(n):
    g = np.random.default_rng(n)
    return [torch.from_numpy(g.normal(size=HID).astype(np.float32)).cuda() for _ in range(n)]


def test_a_captured_step_after_another_was_built(dgt):
    # 1000 tokens: parts that are joined, so that the workspace's counters and parts are used
    w, gam = layers(2, 1)
    x = inputs(6)
    alone = dgt.DecodeStep(w, gam, attention=attention(dgt, 1000))
    want = [alone(v)[0].clone() for v in x]
    att = attention(dgt, 1000)
    step = dgt.DecodeStep(w, gam, attention=att)
    got = [step(x[0])[0].clone()]
    step.capture()
    other = dgt.DecodeStep(w[:1], gam[:3], attention=att)
    # memory of the workspace's size, were it free
    junk = [torch.full((dgt.kv_attention_workspace(att.cache, HID // DIM, 1, 1).numel(),), 255, dtype=torch.uint8,
                       device="cuda") for _ in range(4)]
    got += [step.replay(v)[0].clone() for v in x[1:]]
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert all((j == 255).all() for j in junk)
    other(x[0])
    assert att.status.item() == 0 and att.cache.lens.tolist() == [0, 1007]


def as_r4(dgt, w):
    return [{p: dgt.load_r4(dgt.upload(dgt.pack(t.view(torch.int16).cpu().numpy().view(np.uint16)))) for p, t in l.items()}
            for l in w]


def moe(dgt, w, gam, att):
    """Two experts in every layer, gate, up and down stacked."""
    e = [{p: torch.cat([t, t.flip(0)]) if p in ("gate", "up", "down") else t for p, t in l.items()} for l in w]
    r = [(torch.tensor([1, 0], dtype=torch.int32, device="cuda"), torch.tensor([0.25, 0.75], device="cuda"))]
    return dgt.MoeDecodeStep(e, gam, r, 2, attention=att)


STEPS = {"bf16": lambda dgt, w, gam, att: dgt.DecodeStep(w, gam, attention=att),
         "r4": lambda dgt, w, gam, att: dgt.DecodeStep(as_r4(dgt, w), gam, attention=att), "moe": moe}


@pytest.mark.parametrize("held", [0, 70])
@pytest.mark.parametrize("form", list(STEPS))
def test_a_step_is_captured_without_a_token_of_its_own(dgt, form, held):
    # a prompt of `held` tokens in the cache; the first token that the step appends is the first that is replayed
    w, gam = layers(2, 2)
    x = inputs(4)
    att = attention(dgt, held)
    before = [t.clone() for t in (att.cache.k, att.cache.v, att.cache.table, att.cache.refs)]
    step = STEPS[form](dgt, w, gam, att)
    step.x.copy_(x[0])
    step.capture()
    assert torch.equal(step.x, x[0]) and att.status.item() == 0
    assert att.cache.lens.tolist() == [0, held]
    for a, b in zip((att.cache.k, att.cache.v, att.cache.table, att.cache.refs), before):
        assert torch.equal(a, b)
    got = [step.replay()[0].clone()] + [step.replay(v)[0].clone() for v in x[1:]]
    alone = STEPS[form](dgt, w, gam, attention(dgt, held))
    want = [alone(v)[0].clone() for v in x]
    for a, b in zip(got, want):
        assert torch.equal(a, b)
