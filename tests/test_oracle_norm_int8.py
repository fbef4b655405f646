"""Pins of the oracle's norms, 8-bit integers and MXINT8: torch's layer norm and
autograd in fp64, central differences, exact fractions, hand-worked values."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import int8, mx, norm


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("T,D", [(3, 7), (5, 64), (1, 1), (4, 2)])
@pytest.mark.parametrize("affine", [0, 1, 2])
def test_norm_against_autograd_and_differences(rms, T, D, affine):
    rng = np.random.default_rng(T * D + affine)
    x, dy = rng.standard_normal((2, T, D)) * 2 + 0.5
    w = rng.standard_normal(D) if affine else None
    b = rng.standard_normal(D) if affine == 2 else None
    eps = 1e-3
    t = {n: torch.tensor(a, requires_grad=True) for n, a in (("x", x), ("w", w), ("b", b)) if a is not None}
    if rms:
        y = t["x"] / torch.sqrt((t["x"] ** 2).mean(1, keepdim=True) + eps) * t.get("w", 1.0) + t.get("b", 0.0)
    else:
        y = torch.nn.functional.layer_norm(t["x"], (D,), t.get("w"), t.get("b"), eps)
    got, mean, rstd = norm.forward(x, w, b, eps, rms)
    np.testing.assert_allclose(got, y.detach().numpy(), rtol=1e-9, atol=1e-12)
    grads = torch.autograd.grad((y * torch.tensor(dy)).sum(), list(t.values()))
    dx, dw, db = norm.backward(dy, x, w, mean, rstd, rms)
    for n, g in zip(t, grads):
        np.testing.assert_allclose(dict(x=dx, w=dw, b=db)[n], g.numpy(), rtol=1e-7, atol=1e-9)
    # differences, one element of x at a time
    for i in range(min(T * D, 12)):
        step = np.zeros(T * D)
        step[i] = 1e-5
        step = step.reshape(T, D)
        hi, lo = (float((norm.forward(x + s, w, b, eps, rms)[0] * dy).sum()) for s in (step, -step))
        assert abs((hi - lo) / 2e-5 - dx.reshape(-1)[i]) <= 1e-5 * (1 + abs(dx).max())


def test_norm_planted_mistakes_are_seen():
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((2, 4, 16)) + 1
    w = rng.standard_normal(16)
    _, mean, rstd = norm.forward(x, w, None, 1e-5, False)
    good = norm.backward(dy, x, w, mean, rstd, False)
    for bad in (norm.backward(dy, x, w, mean, rstd, True), norm.backward(dy, x, None, mean, rstd, False),
                norm.backward(dy, x, w, mean, rstd ** 2, False)):
        assert max(np.abs(g - h).max() for g, h in zip(good, bad)) > 1e-2


def test_int8_by_hand():
    x = np.array([[127.0, -63.5, 0.49, -0.5, 0.5, 1.5, 2.5, -127.0],
                  [0, 0, 0, 0, 0, 0, 0, -0.0],
                  [np.inf, 1, 2, 3, 4, 5, 6, 7],
                  [np.nan, 1, 2, 3, 4, 5, 6, np.inf]], np.float32)
    q, s = int8.quantize(x)
    assert q[0].tolist() == [127, -64, 0, 0, 0, 2, 2, -127] and s[0] == 1
    assert not q[1:].any() and s[1] == 0 and np.isinf(s[2]) and np.isnan(s[3])
    tiny = np.float32(2.0 ** -149)
    q, s = int8.quantize(np.array([[tiny, 0], [tiny * 100, -tiny * 60]], np.float32))
    assert s[0] == 0 and not q[0].any()                  # amax / 127 rounds to 0: a dead row
    assert s[1] == tiny and q[1].tolist() == [100, -60]  # (100 / 127 of the smallest step rounds to it)


def test_int8_against_fractions():
    """The nearest multiple of the rounded quotient: an fp32 division and one rounding."""
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((20, 16)) * np.exp(rng.uniform(-60, 60, (20, 1)))).astype(np.float32)
    q, s = int8.quantize(x)
    for r in range(20):
        a = max(abs(Fraction(float(v))) for v in x[r])
        assert abs(Fraction(float(s[r])) - a / 127) <= a / 127 / 2 ** 24
        for v, c in zip(x[r], q[r]):
            exact = Fraction(float(v)) / Fraction(float(s[r]))
            assert abs(exact - int(c)) <= Fraction(1, 2) + abs(exact) / 2 ** 24


def test_int8_product_against_integers():
    rng = np.random.default_rng(3)
    aq, bq = rng.integers(-127, 128, (7, 48), dtype=np.int8), rng.integers(-127, 128, (3, 5, 48), dtype=np.int8)
    a_s, b_s = rng.random(7, dtype=np.float32), rng.random((3, 5), dtype=np.float32)
    off = [0, 2, 2, 6]  # an empty expert, a row behind the last
    c = int8.grouped_gemm(aq, a_s, bq, b_s, off)
    assert not c[6].any()
    for r, e in ((0, 0), (1, 0), (2, 2), (5, 2)):
        for n in range(5):
            total = sum(int(u) * int(v) for u, v in zip(aq[r], bq[e, n]))
            assert c[r, n] == np.float32(np.float32(total) * a_s[r]) * b_s[e, n]


def test_mxint8_by_hand():
    x = np.zeros((6, 32), np.float32)
    x[0, :6] = [1.0, 1 / 64, 1 / 128, 3 / 128, -1 / 128, -3 / 128]      # S = 127, step 2^-6: ties to even
    x[1, :3] = [1.99, -1.999, 0.5]                                       # 127.36 and 127.94 clamp
    x[2, :2] = [np.float32(2.0 ** -149), 0]                              # subnormal: S = 0, step 2^-133
    x[3, :2] = [np.inf, 1]
    x[4, :2] = [3.4028235e38, -1.7e38]
    q, s = mx.quantize_int8(x)
    assert s[:, 0].tolist() == [127, 127, 0, 255, 254, 0]
    assert q[0, :6].tolist() == [64, 1, 0, 2, 0, -2]
    assert q[1, :3].tolist() == [127, -127, 32]
    assert not q[2].any() and not q[3].any() and not q[5].any()
    assert q[4, :2].tolist() == [127, -64]
    v = mx.dequantize_int8(q, s)
    assert v[0, 0] == 1 and v[0, 3] == 2 / 64 and v[1, 0] == 127 / 64 and np.isnan(v[3]).all()
    assert v[4, 0] == 127 * 2.0 ** 121


def test_mxint8_is_the_nearest_code():
    rng = np.random.default_rng(4)
    x = (rng.standard_normal((50, 64)) * np.exp(rng.uniform(-80, 80, (50, 1)))).astype(np.float32)
    q, s = mx.quantize_int8(x)
    for r in range(50):
        for b in range(2):
            block = [Fraction(float(v)) for v in x[r, 32 * b:32 * b + 32]]
            a = max(abs(v) for v in block)
            step = Fraction(2) ** (int(s[r, b]) - 133)
            assert step * 64 <= a < step * 128
            for v, c in zip(block, q[r, 32 * b:32 * b + 32]):
                err = abs(v - int(c) * step)
                assert err <= step / 2 or (abs(int(c)) == 127 and err < step)
