"""route against its definition in 64 bits: the same experts, and their weights."""
import pytest

torch = pytest.importorskip("torch")
import decode_gemv_tensor_gb300 as dgt  # noqa: E402

pytestmark = pytest.mark.gpu
INF = float("inf")


def first(x, k):
    return torch.sort(x, dim=-1, descending=True, stable=True)[1][:, :k]


def reference(logits, topk, score="softmax", bias=None, groups=1, group_topk=1, group_best=2, renorm=True, scale=1.0):
    x = logits.double().cpu()
    x = torch.where(x.isnan(), -INF, x)
    m = x.amax(-1, keepdim=True)
    e = torch.where(x == m, (m > -INF).double(), torch.exp(x - m))
    e = torch.where(m == -INF, 0.0, e)
    s = e / e.sum(-1, keepdim=True).clamp(min=1e-300) if score == "softmax" else 1 / (1 + torch.exp(-x))
    c = s if bias is None else s + bias.double().cpu()
    nan = logits.isnan().cpu()
    order = torch.where(nan, -1e300, x if bias is None else c)     # behind every number but -inf
    order = torch.where(nan | (order > -INF), order, -1e200)       # which comes before it
    if groups > 1:
        by = torch.where(nan, -INF, c).view(len(x), groups, -1)
        by = by.topk(min(group_best, by.shape[-1]), dim=-1)[0].sum(-1)
        keep = torch.zeros_like(by, dtype=torch.bool).scatter(1, first(by, group_topk), True)
        order = torch.where(keep.repeat_interleave(x.shape[1] // groups, 1), order, -INF)
    ids = first(order, topk)
    w = s.gather(1, ids)
    if renorm:
        # as quotients by the largest, so that nothing is lost below 64 bits' range either
        lx = x.gather(1, ids)
        if score == "softmax":
            lx = torch.where((lx == INF).any(1, keepdim=True), torch.where(lx == INF, 0.0, -INF), lx)
        log = torch.log_softmax(lx, -1) if score == "softmax" else torch.nn.functional.logsigmoid(lx)
        w = torch.where((lx > -INF).any(1, keepdim=True), torch.softmax(log, -1), 0.0)
        w = torch.where(lx == -INF, 0.0, w)
    return ids.int(), w * scale


def check(logits, topk, **kw):
    """expf is within 2 units in the last place, a softmax sums in at most 37 steps, quotients and products are one
    rounding each: 2^-18 of a weight."""
    ids, p = dgt.route(logits, topk, **kw)
    want, w = reference(logits, topk, **kw)
    assert torch.equal(ids.cpu(), want)
    assert bool(((p.double().cpu() - w).abs() <= w.abs() * 2.0 ** -18 + 1e-37).all())
    return ids, p


def logits(tokens, experts, dtype=torch.float32, seed=0, spread=1.5):
    g = torch.Generator("cuda").manual_seed(seed)
    return (spread * torch.randn(tokens, experts, device="cuda", generator=g)).to(dtype)


def bias_of(experts, seed=1):
    return 0.1 * torch.randn(experts, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))


@pytest.mark.parametrize("experts", [1, 2, 8, 31, 32, 33, 60, 64, 100, 128, 160, 256, 384, 512, 513, 1000, 1024])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_bias", [False, True])
def test_experts(experts, score, dtype, with_bias):
    x = logits(67, experts, dtype, experts)
    for topk in sorted({1, min(experts, 8), min(experts, 32)}):
        for renorm in (False, True):
            check(x, topk, score=score, bias=bias_of(experts) if with_bias else None, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("experts,groups,keep,topk", [(64, 8, 4, 8), (64, 8, 7, 6), (256, 8, 4, 8), (160, 8, 3, 6),
                                                      (384, 4, 2, 10), (60, 4, 2, 8), (32, 32, 5, 5), (96, 3, 1, 32),
                                                      (1024, 32, 9, 8), (16, 2, 2, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("with_bias", [False, True])
def test_groups(experts, groups, keep, topk, score, best, with_bias):
    for dtype in (torch.float32, torch.bfloat16):
        check(logits(130, experts, dtype, experts + groups), topk, score=score, groups=groups, group_topk=keep,
              group_best=best, bias=bias_of(experts) if with_bias else None)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_values_that_differ_by_less_than_fp32_can_tell(score):
    """Choices whose scores and biases add up to nearly the same: the order is that of 64 bits."""
    x = logits(400, 64, seed=5)
    s = torch.softmax(x.double(), -1) if score == "softmax" else torch.sigmoid(x.double())
    # per column one bias can cancel only one row's score: for each row alone
    for r in range(0, 400, 25):
        b = (0.5 - s[r]).float()
        check(x[r:r + 1], 8, score=score, bias=b)
        check(x[r:r + 1], 8, score=score, bias=b, groups=8, group_topk=3)


@pytest.mark.parametrize("experts,groups,keep", [(160, 32, 9), (60, 20, 5), (96, 3, 2), (84, 12, 4), (341, 31, 11),
                                                 (992, 31, 30), (264, 2, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
def test_close_groups(experts, groups, keep, score, best):
    """Groups whose values add up to nearly the same, in numbers of groups that leave lanes over."""
    x = logits(100, experts, seed=experts)
    x[3, ::7] = float("nan")
    x[5, experts // groups:] = -INF
    s = torch.softmax(x.double(), -1) if score == "softmax" else torch.sigmoid(x.double())
    for r in range(6, 100, 13):
        check(x[r:r + 1], min(8, keep), score=score, bias=(0.5 - s[r]).float(), groups=groups, group_topk=keep,
              group_best=best)
    check(x, min(8, keep), score=score, groups=groups, group_topk=keep, group_best=best)


def test_ties_take_the_lower_expert():
    x = torch.zeros(3, 128, device="cuda")
    x[1, 100:] = 1.0
    x[2, ::3] = -0.0
    for kw in (dict(), dict(bias=torch.zeros(128, device="cuda")), dict(groups=8, group_topk=2),
               dict(score="sigmoid", bias=torch.full((128,), 0.25, device="cuda"), groups=4, group_topk=1)):
        check(x, 8, **kw)


def test_masked_infinite_and_not_a_number():
    x = logits(8, 64, seed=9)
    x[0] = -INF                       # nothing left
    x[1, 5:] = -INF                   # fewer than topk left
    x[2, 7] = INF
    x[3, 10], x[3, 20] = INF, INF
    x[4, 3] = float("nan")
    x[5, 1:] = float("nan")           # one number
    x[6] = torch.finfo(torch.float32).min
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            check(x, 8, score=score, renorm=renorm)
            check(x, 8, score=score, renorm=renorm, bias=bias_of(64))
            check(x, 4, score=score, renorm=renorm, bias=bias_of(64), groups=8, group_topk=4)
    b = bias_of(64)
    b[::2] = -INF                     # experts that are switched off
    check(logits(50, 64), 8, bias=b)


def test_not_a_number_beside_negative_logits():
    """A choice without a score takes nothing from the others' weights."""
    x = -logits(40, 64, seed=10).abs() - 0.1
    for r in range(40):
        x[r, torch.randperm(64, generator=torch.Generator().manual_seed(r))[:25 + r].cuda()] = float("nan")
    for renorm in (False, True):
        for kw in (dict(), dict(bias=bias_of(64)), dict(groups=8, group_topk=6)):
            ids, p = check(x, 32, score="sigmoid", renorm=renorm, **kw)
            assert bool((p[:39].sum(1) > 0).all()) and not bool(p[39].any())   # the last holds nothing else


@pytest.mark.parametrize("experts,topk", [(16, 1), (16, 5), (128, 4), (256, 8), (256, 20)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_copies_at_the_cut_hide_no_other(experts, topk, score):
    """The last choice and the next are copies, and a third value is closer to theirs than fp32 can tell."""
    for seed in range(20):
        x = logits(1, experts, seed=seed)
        at = torch.randperm(experts, generator=torch.Generator().manual_seed(seed))[:topk + 2].tolist()
        a, b, c = at[:3]
        x[0, b] = x[0, a]
        s = (torch.softmax(x.double(), -1) if score == "softmax" else torch.sigmoid(x.double()))[0]
        bias = torch.full((experts,), -4.0, device="cuda")
        bias[at[3:]] = 4.0                     # topk - 1 that are chosen in any case
        bias[[a, b]] = 0.25
        bias[c] = (0.25 + s[a] - s[c]).float()
        check(x, topk, score=score, bias=bias)
        if experts == 256 and topk < 9:
            check(x, topk, score=score, bias=bias, groups=4, group_topk=4)


def test_scores_below_the_range_of_fp32_keep_their_quotients():
    x = logits(20, 32, seed=3) - 300.0
    ids, p = check(x, 4, score="sigmoid")
    assert bool((p.sum(1) - 1).abs().max() < 1e-5)
    y = logits(20, 32, seed=4)
    y[:, 0] = 200.0                    # of a group that is closed
    check(y, 4, groups=4, group_topk=3, bias=torch.where(torch.arange(32, device="cuda") < 8, -9.0, 0.0))


@pytest.mark.parametrize("tokens", [0, 1, 3, 4, 5, 1000])
def test_tokens_strides_and_given_outputs(tokens):
    wide = logits(tokens, 150, seed=tokens)
    for at in (0, 3):
        check(wide[:, at:at + 128], 8)
    ids, p = torch.empty(tokens, 8, dtype=torch.int32, device="cuda"), torch.empty(tokens, 8, device="cuda")
    got = dgt.route(wide, 8, ids=ids, p=p)
    assert got[0] is ids and got[1] is p


def test_stream_graph_and_the_experts_products():
    x = logits(6, 16, seed=2)
    want = dgt.route(x, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = dgt.route(x, 2, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ids, p = (torch.empty_like(t) for t in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dgt.route(x, 2, ids=ids, p=p)
    x.copy_(logits(6, 16, seed=11))
    g.replay()
    w = dgt.route(x, 2)
    assert torch.equal(ids, w[0]) and torch.equal(p, w[1])
    W = torch.randn(16 * 32, 64, device="cuda").bfloat16()
    h = torch.randn(6, 64, device="cuda").bfloat16()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, _, out = dgt.moe_gemv_bf16(W, 16, ids, p, h, status=st)
    assert dgt.read_status(st) == 0
    e = torch.einsum("tkno,to->tkn", W.double().view(16, 32, 64)[ids.long()], h.double())
    ref = (e * p.double()[..., None]).sum(1)
    assert float((out.double() - ref).norm() / ref.norm()) < 1e-5


def test_refusals():
    x = logits(4, 64)
    for kw in (dict(score="tanh"), dict(groups=0), dict(group_best=3), dict(bias=torch.zeros(63, device="cuda")),
               dict(bias=torch.zeros(64, device="cuda", dtype=torch.float64)),
               dict(ids=torch.zeros(4, 3, dtype=torch.int32, device="cuda")),
               dict(p=torch.zeros(4, 8, device="cuda").t().contiguous().t())):
        with pytest.raises(ValueError):
            dgt.route(x, 8, **kw)
    with pytest.raises(ValueError):
        dgt.route(x.t(), 2)
    for kw in (dict(topk=33), dict(topk=4, groups=5), dict(topk=9, groups=8, group_topk=1)):
        with pytest.raises(dgt.DgtError):
            dgt.route(x, **kw)
