"""One StepAttention in several steps: what a captured step holds stays as it
is.  The calls are replaced, so that no device is needed."""
import types

import pytest

torch = pytest.importorskip("torch")
import decode_gemv_tensor_gb300 as dgt  # noqa: E402


def test_a_second_step_leaves_the_first_ones_workspace(monkeypatch):
    cache = dgt.KvCache(2, 2, 1, 64, max_seqs=1, max_pages=2, device="cpu")
    calls = []
    for name in ("rotate", "kv_append"):
        monkeypatch.setattr(dgt, name, lambda *a, **kw: None)
    monkeypatch.setattr(dgt, "kv_attention", lambda c, l, q, s, **kw: calls.append((kw["ws"], q.shape, kw["out"].shape)))
    a = dgt.StepAttention(cache, types.SimpleNamespace(axes=1))
    vec = lambda heads: torch.zeros(heads * 64, dtype=torch.bfloat16)

    def step(heads):
        a(0, vec(heads), vec(1), vec(1), vec(heads))
        return calls[-1]
    a.prepare(4 * 64, 1)
    ws, q, out = step(4)
    assert q == out == (1, 4, 64)
    # another depth, then another width, on the same object
    a.prepare(4 * 64, 2)
    assert step(4)[0] is ws
    a.prepare(2 * 64, 1)
    other, q, out = step(2)
    assert q == out == (1, 2, 64) and other is not ws
    got, q, out = step(4)
    assert got is ws and q == out == (1, 4, 64)


@pytest.mark.parametrize("kind", [dgt.DecodeStep, dgt.MoeDecodeStep])
def test_a_steps_input_is_copied_on_its_stream(monkeypatch, kind):
    # an eager step on a stream of its own reads its input there: the copy belongs to the same stream
    import contextlib
    now, seen = ["current"], []

    @contextlib.contextmanager
    def within(stream):
        was = now[0]
        now[0] = was if stream is None else stream
        yield
        now[0] = was
    monkeypatch.setattr(torch.cuda, "stream", within)
    step = kind.__new__(kind)
    step.x = types.SimpleNamespace(copy_=lambda x0: seen.append(now[0]))
    step.out, step.launch = None, lambda stream: seen.append("current" if stream is None else stream)
    step("x0", "side")
    step("x0")
    assert seen == ["side", "side", "current", "current"]
