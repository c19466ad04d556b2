"""Attention with one key that takes almost all of the weight, and a long tail
of keys whose weights are far smaller, against 64 bits.  The key that takes it
has a value of zero, so that the output is the tail's.

Bound of an element: 2^-8 of it (bf16), 2^-10 of the weighted mean of |v| (the
weights' fp16 rounding and the exponentials, as elsewhere), and what fp16 keeps
of a small weight: a weight times its page's value scale is held to 2^-37 of
the largest such product with few rows (fp16's smallest step 2^-24, half of it,
at weights that reach 2^12), to 2^-29 with many (weights of 2^4 at the
reference, which is never above the largest)."""
import numpy as np
import pytest

import kv_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def dgt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import decode_gemv_tensor_gb300 as d
    d.lib()
    return d


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 100])
@pytest.mark.parametrize("binades", [10, 17, 20, 24, 27, 28, 29, 30, 33, 36, 38])
@pytest.mark.parametrize("smaller", [0, 6])
def test_a_long_tail_of_small_weights(dgt, dim, rows, binades, smaller):
    # key 70 scores `binades` ln 2 above the others, which score 0; from token 128 on values are 2^-smaller the size
    n = 4000
    g = np.random.default_rng(binades + smaller)
    c = dgt.KvCache(1, 64, 1, dim, max_seqs=1, max_pages=64)
    c.table[0] = torch.arange(64, dtype=torch.int32, device="cuda")
    c.lens[0] = n
    k, v = np.zeros((n, 1, dim)), g.uniform(0.5, 1.0, size=(n, 1, dim))
    k[70, 0, 0] = 1.0
    v[70] = 0.0
    v[128:] *= 2.0 ** -smaller
    dev = lambda x: torch.from_numpy(x.astype(np.float32)).cuda().bfloat16()
    dgt.kv_append(c, 0, dev(k), dev(v), i32([0]), i32([0]), cu=i32([0, n]))
    kk, vv = (f64(x) for x in dgt.kv_read(c, 0, i32([0]), i32([0]), i32([0, n]), n))
    q = torch.zeros(rows, 1, dim, device="cuda", dtype=torch.bfloat16)
    q[:, 0, 0] = 1
    scale = float(np.float32(binades * np.log(2.0)))
    out = f64(dgt.kv_attention(c, 0, q, i32([0]), cu=None if rows == 1 else i32([0, rows]), scale=scale))
    s = np.repeat(f64(c.v_scale[0, :, 0]), 64)[:n]
    step = 2.0 ** -37 if rows == 1 else 2.0 ** -29
    for i in {0, rows // 2, rows - 1}:
        at = n - rows + i
        ref, _, mag, _ = R.attention(f64(q)[i:i + 1], kk, vv, at, 0, 0, scale)
        w = np.exp(scale * (kk[:at + 1, 0, 0] - 1.0))
        codes = (np.abs(vv[:at + 1, 0]) / s[:at + 1, None]).sum(0)
        small = step * (w * s[:at + 1]).max() * codes / w.sum()
        assert (np.abs(out[i, 0] - ref[0, 0]) <= 2.0 ** -8 * np.abs(ref[0, 0]) + 2.0 ** -10 * mag[0, 0] + small).all(), i
