"""CPU pins of the router and AdamW oracles: hand-worked values, central
differences, invariants of the 8-bit moments and their random bits; and the
refusals of the new entry points, before any HIP call."""

import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import adamw, router

INF = np.float32(np.inf)


# ---------------------------------------------------------------- router

def test_selection_by_hand():
    l = np.array([[1, 3, 3, -INF, 2], [-INF] * 5, [0.0, -0.0, 0.0, 0.0, -1], [np.nan, 5, -INF, np.nan, 4]], np.float32)
    np.testing.assert_array_equal(router.select(l, None, 3), [[1, 2, 4], [-1, -1, -1], [0, 1, 2], [1, 4, -1]])
    bias = np.array([5, 0, -INF, 0, 0], np.float32)
    np.testing.assert_array_equal(router.select(l, bias, 2), [[0, 1], [-1, -1], [0, 1], [1, 4]])


def test_weights_by_hand():
    l = np.log(np.array([[1, 2, 4, 9]], np.float64)).astype(np.float32)
    ids = np.array([[3, 1, -1]], np.int32)
    np.testing.assert_allclose(router.weights(l, ids, "topk", 2.0), [[18 / 11, 4 / 11, 0]], rtol=1e-6)
    np.testing.assert_allclose(router.weights(l, ids, "all", 1.0), [[9 / 16, 2 / 16, 0]], rtol=1e-6)
    np.testing.assert_allclose(router.lse(l), [np.log(16)], rtol=1e-6)
    np.testing.assert_allclose(router.prob_sum(np.concatenate([l, np.full((1, 4), -INF)])), np.array([1, 2, 4, 9]) / 16,
                               rtol=1e-6)


@pytest.mark.parametrize("score", ["topk", "all"])
def test_router_gradient_against_differences(score):
    rng = np.random.default_rng(0)
    T, E, k = 4, 7, 3
    l = rng.standard_normal((T, E))
    l[2, 4] = -np.inf
    ids = router.select(l, None, k)
    ids[1, 2] = -1
    dw, dl, ds = rng.standard_normal((T, k)), rng.standard_normal(T), rng.standard_normal(E)

    def loss(x):
        return ((router.weights(x, ids, score, 1.5) * dw).sum() + (router.lse(x) * dl).sum() +
                (router.prob_sum(x) * ds).sum())

    got = router.backward(l, ids, score, 1.5, dw, dl, ds)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            if np.isinf(l[t, e]):
                assert got[t, e] == 0
                continue
            a, b = l.copy(), l.copy()
            a[t, e] += h
            b[t, e] -= h
            assert abs((loss(a) - loss(b)) / (2 * h) - got[t, e]) < 1e-8


# ---------------------------------------------------------------- AdamW

def test_adamw_step_by_hand():
    # t = 1 from zero moments: m / (1 - b1) = g, sqrt(v / (1 - b2)) = |g|, so the step is lr * sign(g)
    p, m, v, upd = adamw.step_f64([1.0, -2.0], [0.5, -3.0], [0, 0], [0, 0], 1, 0.1, (0.9, 0.99), 0.0, 0.5)
    np.testing.assert_allclose(upd, [0.1, 0.1])     # magnitudes
    np.testing.assert_allclose(p, [1 * 0.95 - 0.1, -2 * 0.95 + 0.1])
    np.testing.assert_allclose(m, [0.05, -0.3])
    np.testing.assert_allclose(v, [0.0025, 0.09])


def test_codes_by_hand():
    m = np.zeros(300, np.float32)
    v = np.zeros(300, np.float32)
    m[:4] = [448, -1, 2.0 ** -9, 0]
    v[:4] = [8, 1, 8 * 2.0 ** -32 / 1000, 0]
    m[256:259] = [np.nan, -np.inf, 2]
    v[256:259] = [np.inf, np.nan, 3]
    mc, ms, vc, vs = adamw.encode(m, v, np.zeros(300, np.uint32))
    np.testing.assert_array_equal(ms, np.array([448, 2], np.float32) * (np.float32(1) / np.float32(448)))
    np.testing.assert_array_equal(vs, [8, 3])
    np.testing.assert_array_equal(mc[:4], [0x7E, 0x80 | 0x38, 1, 0])
    np.testing.assert_array_equal(vc[:4], [254, 254 - 24, 1, 0])    # a positive v never becomes 0
    # 2 fl(1 / 448) is above 2 / 448, so 2 lies just under 448 scales: without random bits it goes down
    np.testing.assert_array_equal(mc[256:259] & 0x7F, [0x7F, 0x7F, 0x7D])
    np.testing.assert_array_equal(vc[256:259], [255, 255, 254])
    dm, dv = adamw.decode(mc, ms, vc, vs)
    np.testing.assert_array_equal(dm[:4], m[:4])
    np.testing.assert_array_equal(dv[:2], v[:2])
    assert np.isnan(dm[256:258]).all() and np.isnan(dv[256:258]).all()


def test_rounding_is_unbiased_and_within_one_code():
    # 4096 draws of one value between two codes: the mean is off by at most
    # 5 standard errors of a step (step / 2 / 64) plus the 2^-16 resolution
    n = 4096
    for mv, vv in ((300.0, 0.7), (0.01, 2.0 ** -20 * 1.3), (2.0 ** -8 * 1.01, 0.999)):
        m, v = np.full(n, mv, np.float32), np.full(n, vv, np.float32)
        m[::256], v[::256] = 448, 1
        r = adamw.random_bits(7, 11, 3, n)
        dm, dv = adamw.decode(*adamw.encode(m, v, r))
        keep = np.arange(n) % 256 != 0
        for got, want, step in ((dm[keep], mv, max(2.0 ** -9, 2.0 ** (np.floor(np.log2(mv)) - 3))),
                                (dv[keep], vv, 2.0 ** (np.floor(np.log2(vv)) - 3))):
            assert np.abs(got - want).max() <= step
            assert abs(got.mean() - want) <= step * (5 / 2 / np.sqrt(keep.sum()) + 2.0 ** -16)


def test_random_bits_differ_by_seed_step_tensor_and_element():
    base = adamw.random_bits(1, 1, 0, 1 << 16)
    for other in (adamw.random_bits(2, 1, 0, 1 << 16), adamw.random_bits(1, 2, 0, 1 << 16),
                  adamw.random_bits(1, 1, 1, 1 << 16), np.roll(base, 1)):
        # correlation of independent 16-bit halves: sd 1 / 256
        for a, b in ((base >> 16, other >> 16), (base & 0xFFFF, other & 0xFFFF), (base >> 16, other & 0xFFFF)):
            assert abs(np.corrcoef(a, b)[0, 1]) < 5 / 256


# ---------------------------------------------------------------- refusals

FAKE = 0x10000  # an aligned fake device address: never dereferenced


@pytest.fixture(scope="module")
def lib():
    from nvfp4_quantized_moe_token_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built")
    return _lib.load()


def _bad(fn, args, cases):
    for change, rc in cases:
        a = list(args)
        for i, v in change.items():
            a[i] = v
        assert fn(*a) == rc, (change, rc)


def test_router_refusals(lib):
    ws = lib.moe_router_workspace_size(100, 128, 8)
    assert ws == 2 * 128 * 4 and lib.moe_router_workspace_size(-1, 128, 8) == 0   # 64 tokens per workgroup
    assert lib.moe_router_workspace_size(1 << 20, 128, 8) == 256 * 128 * 4
    args = [FAKE, 0, 100, 128, 8, None, 0, 1.0, FAKE, FAKE, FAKE, FAKE, FAKE, ws, None]
    _bad(lib.moe_router, args, [
        ({2: -1}, -1), ({3: 0}, -1), ({4: 0}, -1), ({1: 2}, -1), ({6: 2}, -1), ({0: None}, -1), ({8: None}, -1),
        ({9: None}, -1), ({3: 4097}, -2), ({4: 65, 3: 128}, -2), ({4: 9, 3: 8}, -2), ({2: 1 << 40}, -2),
        ({0: FAKE + 2}, -2), ({5: FAKE + 2}, -2), ({8: FAKE + 2}, -2), ({11: FAKE + 1}, -2), ({12: None}, -5),
        ({13: ws - 1}, -5)])
    args = [FAKE, 1, 100, 128, 8, FAKE, 0, 1.0, FAKE, FAKE, FAKE, FAKE, FAKE, 0, None]
    _bad(lib.moe_router_bwd, args, [
        ({2: -1}, -1), ({1: 2}, -1), ({13: 2}, -1), ({6: -1}, -1), ({0: None}, -1), ({5: None}, -1), ({12: None}, -1),
        ({3: 5000}, -2), ({4: 129}, -2), ({0: FAKE + 1}, -2), ({12: FAKE + 2}, -2), ({8: FAKE + 2}, -2)])


def test_unpermute_bwd_refusals(lib):
    args = [FAKE, 1, FAKE, 1, FAKE, FAKE, FAKE, 4, 10, 8, 64, FAKE, 1, FAKE, FAKE, None]
    _bad(lib.moe_unpermute_bwd, args, [
        ({8: -1}, -1), ({9: 0}, -1), ({7: 0}, -1), ({10: -8}, -1), ({1: 2}, -1), ({3: 2}, -1), ({12: 2}, -1),
        ({0: None}, -1), ({2: None}, -1), ({4: None}, -1), ({6: None}, -1), ({11: None, 13: None, 14: None}, -1),
        ({11: None}, -1), ({10: 60}, -2), ({9: 65}, -2), ({8: 1 << 31}, -2), ({0: FAKE + 8}, -2), ({2: FAKE + 8}, -2),
        ({11: FAKE + 8}, -2), ({13: FAKE + 2}, -2), ({14: FAKE + 2}, -2)])


def test_mxfp4_refusals(lib):
    ws = lib.moe_permute_workspace_size(10, 8, 4)
    args = [FAKE, 10, 8, 4, FAKE, 1, 64, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, ws, None, None]
    _bad(lib.moe_permute_mxfp4, args, [
        ({5: 2}, -1), ({4: None}, -1), ({8: None}, -1), ({6: 48}, -2), ({7: FAKE + 4}, -2), ({3: 5000}, -2),
        ({13: ws - 1}, -5)])
    args = [FAKE, FAKE, FAKE, FAKE, FAKE, 4, 64, 64, 256, FAKE, 0, None]
    _bad(lib.grouped_gemm_mxfp4, args, [
        ({5: 0}, -1), ({6: -1}, -1), ({10: 2}, -1), ({4: None}, -1), ({0: None}, -1), ({3: None}, -1), ({9: None}, -1),
        ({8: 192}, -2), ({7: 48}, -2), ({8: (1 << 22) + 128}, -2), ({0: FAKE + 8}, -2), ({1: FAKE + 2}, -2),
        ({9: FAKE + 8}, -2)])
    args = [FAKE, FAKE, FAKE, FAKE, FAKE, 4, 64, 128, 256, FAKE, FAKE, FAKE, FAKE, FAKE, None]
    _bad(lib.grouped_gemm_mxfp4_silu_gate, args, [
        ({7: -1}, -1), ({13: None}, -1), ({12: None}, -1), ({10: None, 12: None, 13: None}, -1), ({7: 64}, -2),
        ({8: 64}, -2), ({7: 1 << 13, 8: 1 << 18}, -2), ({9: FAKE + 8}, -2), ({12: FAKE + 2}, -2)])


def test_mxfp4_width_limit(lib):
    # a tile's output region is addressed in 32 bits
    _bad(lib.grouped_gemm_mxfp4, [FAKE, FAKE, FAKE, FAKE, FAKE, 4, 64, 64, 256, FAKE, 0, None],
         [({7: (1 << 20) + 32}, -2), ({6: (1 << 31) - 256}, -2)])
    _bad(lib.grouped_gemm_mxfp4_silu_gate,
         [FAKE, FAKE, FAKE, FAKE, FAKE, 4, 64, 128, 256, FAKE, FAKE, FAKE, FAKE, FAKE, None],
         [({7: (1 << 19) + 128, 8: 128}, -2)])


def test_adamw_refusals(lib):
    from nvfp4_quantized_moe_token_amd import _lib

    def one(**kw):
        d = dict(param=FAKE, grad=FAKE, exp_avg=FAKE, exp_avg_sq=FAKE, avg_scale=FAKE, avg_sq_scale=FAKE, n=100)
        d.update(kw)
        return (_lib.AdamWTensor * 1)(_lib.AdamWTensor(**d))

    args = [one(), 1, 0, 0, 8, 1e-3, 0.9, 0.999, 1e-8, 0.1, 1, None, None, None, None, 0, None]
    nan = float("nan")
    _bad(lib.adamw_step, args, [
        ({1: -1}, -1), ({0: None}, -1), ({2: 2}, -1), ({3: 2}, -1), ({4: 16}, -1), ({6: 1.0}, -1), ({7: -0.1}, -1),
        ({8: -1.0}, -1), ({6: nan}, -1), ({10: 0}, -1), ({0: one(n=-1)}, -1), ({0: one(param=None)}, -1),
        ({0: one(grad=None)}, -1), ({0: one(exp_avg=None)}, -1), ({0: one(avg_scale=None)}, -1),
        ({0: one(param_bf16=FAKE), 2: 1}, -1), ({0: one(param=FAKE + 2)}, -2), ({0: one(grad=FAKE + 1), 3: 1}, -2),
        ({0: one(exp_avg=FAKE + 2), 4: 32}, -2), ({11: FAKE + 4}, -2), ({12: FAKE + 2}, -2)])
    ptrs = (ctypes.c_void_p * 1)(FAKE)
    null = (ctypes.c_void_p * 1)(None)
    _bad(lib.adamw_read_state, [one(), 1, ptrs, ptrs, None], [
        ({1: -1}, -1), ({2: None}, -1), ({3: null}, -1), ({0: one(avg_sq_scale=None)}, -1),
        ({2: (ctypes.c_void_p * 1)(FAKE + 2)}, -2)])


def test_structure_matches_the_header():
    from conftest import ROOT
    from nvfp4_quantized_moe_token_amd import _lib
    text = open(os.path.join(ROOT, "include", "nvfp4moe.h")).read()
    body = text[text.index("typedef struct {"):text.index("} nvfp4moe_adamw_tensor;")]
    fields = [ln.split(";")[0].split()[-1].lstrip("*") for ln in body.splitlines()[1:] if ";" in ln]
    assert fields == [n for n, _ in _lib.AdamWTensor._fields_] and ctypes.sizeof(_lib.AdamWTensor) == 64


def test_python_refusals_need_no_gpu():
    from nvfp4_quantized_moe_token_amd import ops, optim
    z = torch.zeros
    i32, u8 = torch.int32, torch.uint8
    for call in (lambda: ops.moe_router(z(4, 8), 2),                                   # not on the GPU
                 lambda: ops.moe_router(z(4, 8, dtype=torch.float16), 2),
                 lambda: ops.moe_router(z(8), 2),
                 lambda: ops.moe_router(z(4, 8), 2, bias=z(7)),
                 lambda: ops.moe_router_bwd(z(4, 8), z(4, 2, dtype=torch.int64), z(4, 2)),
                 lambda: ops.moe_router_bwd(z(4, 8), z(4, 2, dtype=i32), z(4, 3)),
                 lambda: ops.moe_unpermute_bwd(z(4, 8), None, z(8, dtype=i32), z(3, dtype=i32), 2),
                 lambda: ops.moe_unpermute_bwd(z(4, 8), z(7, 8), z(8, dtype=i32), z(3, dtype=i32), 2),
                 lambda: ops.moe_unpermute_bwd(z(4, 8), z(8, 8), z(8, dtype=i32), z(3, dtype=i32), 2),
                 lambda: ops.moe_permute_mxfp4(z(4, 2, dtype=i32), 3, z(5, 32)),
                 lambda: ops.grouped_gemm_mxfp4(z(4, 64, dtype=u8), z(4, 3, dtype=u8), z(2, 32, 64, dtype=u8),
                                                z(2, 32, 4, dtype=u8), z(3, dtype=i32)),
                 lambda: ops.grouped_gemm_mxfp4(z(4, 64, dtype=u8), z(4, 4, dtype=u8), z(2, 32, 64, dtype=u8),
                                                z(2, 32, 4, dtype=u8), z(2, dtype=i32)),
                 lambda: optim.AdamW([]),
                 lambda: optim.AdamW([z(3)]),
                 lambda: optim.AdamW([z(3, dtype=torch.float16)]),
                 lambda: optim.AdamW([z(3)], state_bits=16),
                 lambda: optim.AdamW([z(3)], params_bf16=[z(4, dtype=torch.bfloat16)]),
                 lambda: optim.AdamW([z(3)], params_bf16=[z(3)]),
                 lambda: optim.AdamW([z(3, dtype=torch.bfloat16)], params_bf16=[z(3, dtype=torch.bfloat16)]),
                 lambda: optim.AdamW([z(300)], state_bits=8, state=dict(
                     exp_avg=[z(300, dtype=u8)], exp_avg_sq=[z(300, dtype=u8)], avg_scale=[z(1)], avg_sq_scale=[z(2)]))):
        with pytest.raises(ValueError):
            call()


def test_a_positive_second_moment_never_becomes_zero():
    # quotients from the lowest code's value down to ones that fp32 holds as 0
    v = np.zeros(256, np.float32)
    v[:5] = [2.0 ** 100, 2.0 ** 69, 2.0 ** -48, 2.0 ** -50, 2.0 ** -140]
    for r in (0, 0xFFFFFFFF):
        _, _, vc, vs = adamw.encode(np.zeros(256, np.float32), v, np.full(256, r, np.uint32))
        assert vs[0] == v[0]
        np.testing.assert_array_equal(vc[:6], [254, 6, 1, 1, 1, 0])


def test_router_gradient_of_masked_rows_by_hand():
    """z-loss lse^2 of a row of -inf: its d_lse is -inf, its gradient zero; and
    a masked expert's d_prob_sum reaches nobody."""
    l = np.array([[-INF, -INF, -INF], [0, 0, -INF]], np.float32)
    ids = np.array([[-1], [0]], np.int32)
    dsum = np.array([1, 3, np.inf])
    for dlse in ([-INF, 2], [np.nan, 2]):
        got = router.backward(l, ids, "topk", 1.0, [[np.nan], [5.0]], dlse, dsum)
        np.testing.assert_allclose(got, [[0, 0, 0], [1 + 0.5 * (1 - 2), 1 + 0.5 * (3 - 2), 0]])
