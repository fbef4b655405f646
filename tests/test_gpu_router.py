"""GPU parity of the router and its gradient against the fp64 oracle: ids
exact (ties, masks, NaN, rows with nothing left), weights, lse, probability
sums and gradients within bounds that count fp32 roundings; every layout of
the kernel (experts, choices, alignment); streams; captured replays."""

import numpy as np
import pytest
import torch

from _helpers import gpu, require_gpu, to_gpu, to_np
from oracle import router

pytestmark = gpu

SCORES = {"topk": 0, "all": 1}
U = 2.0 ** -24  # half a unit of fp32


def _logits(rng, T, E, dtype):
    l = to_gpu(rng.standard_normal((T, E)).astype(np.float32) * 2, dtype)
    return l, to_np(l)


def _exp_rel(l, V):
    """Relative error of a softmax entry: the difference l - m and its product
    with log2 e are rounded (2 |l - m| u), the hardware exponential is good to
    1 ulp (2 u), sums of V per lane and 6 exchanges (V + 6) u, then a division
    and a product; numerator and denominator each."""
    f = l[np.isfinite(l)]
    span = float(f.max() - f.min()) if f.size else 0.0
    return (4 * span + 2 * V + 40) * U


CASES = [  # E, k, T: each layout (16 or 64 lanes per token, 4 to 64 logits per lane), whole vectors or not
    (1, 1, 3), (5, 2, 33), (8, 8, 1), (60, 6, 100), (64, 16, 17), (67, 3, 40), (100, 17, 20), (128, 8, 333),
    (130, 8, 35), (200, 16, 9), (255, 4, 21), (256, 8, 65), (260, 64, 7), (512, 8, 5), (515, 9, 6), (1024, 2, 10),
    (1026, 5, 3), (4096, 64, 5)]


@pytest.mark.parametrize("E,k,T", CASES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["topk", "all"])
def test_router_parity(E, k, T, dtype, score):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    rng = np.random.default_rng(E * 131 + k * 7 + T)
    g, l = _logits(rng, T, E, dtype)
    bias = rng.standard_normal(E).astype(np.float32)
    r = ops.moe_router(g, k, bias=to_gpu(bias, torch.float32), score=SCORES[score], scale=2.5, want_lse=True,
                       want_prob_sum=True)
    only = ops.moe_router(g, k, bias=to_gpu(bias, torch.float32), score=SCORES[score], scale=2.5)
    torch.cuda.synchronize()
    ids = router.select(l, bias, k)
    np.testing.assert_array_equal(to_np(r["topk_ids"]), ids)
    rel = _exp_rel(l, 64)
    w = router.weights(l, ids, score, 2.5)
    assert (np.abs(to_np(r["topk_w"]) - w) <= rel * w).all()
    assert torch.equal(only["topk_ids"], r["topk_ids"]) and torch.equal(only["topk_w"], r["topk_w"])
    lse = router.lse(l)
    assert (np.abs(to_np(r["lse"]) - lse) <= rel + 4 * U * np.abs(lse)).all()
    s = router.prob_sum(l)
    # T terms meet in chains of at most T additions
    assert (np.abs(to_np(r["prob_sum"]) - s) <= (rel + (T + 16) * U) * s).all()


def test_ties_masks_and_nan():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    rng = np.random.default_rng(3)
    inf = np.float32(np.inf)
    for E, k in ((128, 8), (130, 8), (40, 20), (300, 12), (2000, 3)):
        l = np.round(rng.standard_normal((64, E)) * 2).astype(np.float32)    # many equal keys
        l[0] = -inf
        l[1, 2:] = -inf                     # fewer left than k
        l[2] = 0.0
        l[2, ::2] = -0.0                    # zeros of both signs tie
        l[3, rng.random(E) < 0.5] = np.nan  # NaN is never chosen
        l[4] = np.nan
        l[5] = -3e38
        bias = np.zeros(E, np.float32)
        bias[1::3] = -inf                   # masked experts, whatever their logit
        l[6, 1::3] = np.nan
        for b in (None, bias):
            r = ops.moe_router(to_gpu(l, torch.float32), k, bias=None if b is None else to_gpu(b, torch.float32),
                               want_lse=True)
            torch.cuda.synchronize()
            ids = router.select(l, b, k)
            np.testing.assert_array_equal(to_np(r["topk_ids"]), ids)
            w = to_np(r["topk_w"])
            assert (w[ids < 0] == 0).all() and np.isfinite(w).all()
            full = (ids >= 0).any(axis=1)
            assert np.abs(w.sum(axis=1) - full).max() <= 64 * U
            assert to_np(r["lse"])[0] == -inf and np.isnan(to_np(r["lse"])[4])


def test_masked_rows_add_nothing_and_have_no_gradient():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    rng = np.random.default_rng(4)
    T, E, k = 50, 128, 8
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[::5] = -np.inf
    l[1::5, 3:] = -np.inf
    g = to_gpu(l, torch.float32)
    for score in ("topk", "all"):
        r = ops.moe_router(g, k, score=SCORES[score], want_lse=True, want_prob_sum=True)
        ids = router.select(l, None, k)
        dw, dl, ds = (rng.standard_normal(n).astype(np.float32) for n in ((T, k), (T,), (E,)))
        d = ops.moe_router_bwd(g, r["topk_ids"], to_gpu(dw, torch.float32), score=SCORES[score], lse=r["lse"],
                               d_lse=to_gpu(dl, torch.float32), d_prob_sum=to_gpu(ds, torch.float32))
        torch.cuda.synchronize()
        s = router.prob_sum(l)
        assert (np.abs(to_np(r["prob_sum"]) - s) <= (_exp_rel(l, 64) + 66 * U) * s).all()
        got = to_np(d)
        assert (got[::5] == 0).all() and (got[np.isneginf(l)] == 0).all()
        want = router.backward(l, ids, score, 1.0, dw, dl, ds)
        assert np.abs(got - want).max() <= _exp_rel(l, 64) * 40


@pytest.mark.parametrize("E,k,T", CASES)
@pytest.mark.parametrize("score", ["topk", "all"])
@pytest.mark.parametrize("dtype,out", [(torch.float32, torch.float32), (torch.bfloat16, torch.float32),
                                       (torch.float32, torch.bfloat16), (torch.bfloat16, torch.bfloat16)])
def test_router_backward_parity(E, k, T, score, dtype, out):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    rng = np.random.default_rng(E * 17 + k + T)
    g, l = _logits(rng, T, E, dtype)
    ids = router.select(l, None, k)
    ids[T // 2, k - 1] = -1
    if T > 1 and k > 1:
        ids[0, 1] = ids[0, 0]              # a repeated id adds up
    dw, dl, ds = (rng.standard_normal(n).astype(np.float32) for n in ((T, k), (T,), (E,)))
    gi, gw, gl, gs = to_gpu(ids, torch.int32), *(to_gpu(x, torch.float32) for x in (dw, dl, ds))
    lse = to_gpu(router.lse(l).astype(np.float32), torch.float32)
    rel = _exp_rel(l, 64)
    for a_dl, a_ds, a_lse in ((None, None, None), (dl, None, None), (None, ds, lse), (dl, ds, lse)):
        d = ops.moe_router_bwd(g, gi, gw, score=SCORES[score], scale=1.5, lse=a_lse, d_lse=None if a_dl is None else gl,
                               d_prob_sum=None if a_ds is None else gs, out_dtype=out)
        torch.cuda.synchronize()
        want = router.backward(l, ids, score, 1.5, dw, a_dl, a_ds)
        # every entry is a sum of products of one probability (or two) with
        # gradients: the terms' magnitudes, each with the softmax's error
        mag = np.zeros((T, E))
        p = np.exp(l - router.lse(l)[:, None])
        q = router.weights(l, ids, score, 1.0)
        u = 1.5 * np.abs(dw)
        t = np.arange(T)[:, None].repeat(k, 1)
        on = ids >= 0
        np.add.at(mag, (t[on], ids[on]), (q * (u + (q * u).sum(1, keepdims=True)))[on])
        mag += p * ((q * u).sum(1, keepdims=True) * (score == "all") + (np.abs(dl)[:, None] if a_dl is not None else 0) +
                    ((np.abs(ds) + (p * np.abs(ds)).sum(1, keepdims=True)) if a_ds is not None else 0))
        tol = 3 * rel * mag + (2.0 ** -8 * np.abs(want) if out == torch.bfloat16 else 0) + 1e-37
        err = np.abs(to_np(d) - want)
        assert (err <= tol).all(), (float((err / tol).max()), score, a_dl is None, a_ds is None)


def test_no_tokens_and_views_off_alignment():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    r = ops.moe_router(torch.zeros((0, 64), device="cuda"), 4, want_lse=True, want_prob_sum=True)
    assert r["topk_ids"].shape == (0, 4) and (to_np(r["prob_sum"]) == 0).all()
    assert ops.moe_router_bwd(torch.zeros((0, 64), device="cuda"), r["topk_ids"], r["topk_w"]).shape == (0, 64)
    for dtype in (torch.float32, torch.bfloat16):
        buf = torch.randn(1 + 50 * 128, device="cuda").to(dtype)
        at1, at0 = buf[1:].view(50, 128), buf[1:].clone().view(50, 128)
        a, b = (ops.moe_router(x, 8, want_lse=True, want_prob_sum=True) for x in (at1, at0))
        assert torch.equal(a["topk_ids"], b["topk_ids"]) and torch.equal(a["topk_w"], b["topk_w"])
        # the lanes hold other experts, so the sums over them meet in another
        # order: each order is off by at most 8 + 6 additions (u of the sum
        # each), the logarithm by 1 ulp of its result (2 u |lse|); the sums over
        # the 50 tokens then carry both errors of exp(l - lse)'s denominator
        rel = 2 * 14 * U
        assert ((a["lse"] - b["lse"]).abs() <= rel + 4 * U * b["lse"].abs()).all()
        assert ((a["prob_sum"] - b["prob_sum"]).abs() <= (rel + 2 * 70 * U) * b["prob_sum"]).all()
        dw = torch.randn(50, 8, device="cuda")
        assert torch.equal(ops.moe_router_bwd(at1, a["topk_ids"], dw), ops.moe_router_bwd(at0, a["topk_ids"], dw))


def test_two_streams_at_once():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    xs = [torch.randn(5000, 128, device="cuda") for _ in range(2)]
    want = [ops.moe_router(x, 8, want_prob_sum=True, want_lse=True) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(ops.moe_router(xs[i], 8, want_prob_sum=True, want_lse=True))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            for n in r:
                assert torch.equal(r[n], want[i][n]), n


def test_captured_router_replays():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    x = torch.randn(700, 128, device="cuda")
    dw, ds = torch.randn(700, 8, device="cuda"), torch.randn(128, device="cuda")

    def step():
        r = ops.moe_router(x, 8, want_prob_sum=True, want_lse=True)
        r["d"] = ops.moe_router_bwd(x, r["topk_ids"], dw, lse=r["lse"], d_prob_sum=ds)
        return r

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for _ in range(3):
        x.copy_(torch.randn_like(x))
        want = step()
        for t in out.values():
            t.fill_(9)
        g.replay()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(out[n], want[n]), n


@pytest.mark.parametrize("E,k", [(60, 4), (128, 8), (130, 3), (300, 12), (600, 2), (2000, 20)])
@pytest.mark.parametrize("score", ["topk", "all"])
def test_gradients_that_are_not_finite_at_masked_places(E, k, score):
    """A z-loss over padded rows hands in -inf or NaN for them, a loss of the
    logarithm of prob_sum an infinity for an expert that is masked everywhere."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    rng = np.random.default_rng(E + k)
    T = 40
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[::4] = -np.inf
    l[:, 3::7] = -np.inf
    g = to_gpu(l, torch.float32)
    r = ops.moe_router(g, k, score=SCORES[score], want_lse=True)
    ids = router.select(l, None, k)
    dw, dl, ds = (rng.standard_normal(n).astype(np.float32) for n in ((T, k), (T,), (E,)))
    dl[::4], dl[4] = -np.inf, np.nan
    ds[3::7] = np.inf
    for lse in (r["lse"], None):
        d = ops.moe_router_bwd(g, r["topk_ids"], to_gpu(dw, torch.float32), score=SCORES[score], lse=lse,
                               d_lse=to_gpu(dl, torch.float32), d_prob_sum=to_gpu(ds, torch.float32))
        torch.cuda.synchronize()
        got, want = to_np(d), router.backward(l, ids, score, 1.0, dw, dl, ds)
        assert (got[::4] == 0).all() and (got[:, 3::7] == 0).all()
        assert np.abs(got - want).max() <= _exp_rel(l, 64) * 40


def test_gradient_of_more_tokens_than_one_dispatch_holds():
    """2^28 + 21 tokens of two experts, 16 per workgroup: over 2^32 work-items.
    Tokens at the start, across both ends of a launch and at the end against
    calls of their own."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    T, E = (1 << 28) + 21, 2
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-256, 256, (T, E), generator=gen, device="cuda", dtype=torch.int16)
    x = x.to(torch.bfloat16).mul_(2.0 ** -6)
    dw = torch.ones((T, 1), device="cuda")
    ids = torch.arange(T, device="cuda", dtype=torch.int32).remainder_(2).view(T, 1)
    d = torch.full((T, E), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.moe_router_bwd(x, ids, dw, score=SCORES["all"], out=d)
    torch.cuda.synchronize()
    per = (1 << 20) * 16
    for lo in (0, per - 50, 5 * per - 3, (1 << 28) - 40, T - 100):
        s = slice(lo, min(lo + 100, T))
        want = ops.moe_router_bwd(x[s].clone(), ids[s].clone(), dw[s].clone(), score=SCORES["all"])
        torch.cuda.synchronize()
        assert torch.equal(d[s], want), lo
    assert not (d == 7.0).any()


@pytest.mark.parametrize("E,k,T", [(128, 8, 16385), (128, 8, 40000), (512, 4, 5000), (300, 20, 9001), (2048, 3, 1100)])
def test_probability_sums_over_several_rounds_of_tokens(E, k, T):
    """More tokens than the workgroups hold at once: each adds up several."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    rng = np.random.default_rng(E + T)
    g, l = _logits(rng, T, E, torch.float32)
    r = ops.moe_router(g, k, want_lse=True, want_prob_sum=True)
    torch.cuda.synchronize()
    ids = router.select(l, None, k)
    np.testing.assert_array_equal(to_np(r["topk_ids"]), ids)
    rel = _exp_rel(l, 64)
    w, lse, s = router.weights(l, ids, "topk", 1.0), router.lse(l), router.prob_sum(l)
    assert (np.abs(to_np(r["topk_w"]) - w) <= rel * w).all()
    assert (np.abs(to_np(r["lse"]) - lse) <= rel + 4 * U * np.abs(lse)).all()
    # a lane's chain of at most 5 tokens, 2 exchanges, 16 waves; 4 rows, 2 exchanges, 16 waves
    assert (np.abs(to_np(r["prob_sum"]) - s) <= (rel + 45 * U) * s).all()
    # probabilities of exactly 1: the sums are counts, whatever the order
    e = rng.integers(0, E, T)
    l = np.full((T, E), -np.inf, np.float32)
    l[np.arange(T), e] = rng.standard_normal(T)
    r = ops.moe_router(to_gpu(l, torch.float32), k, want_prob_sum=True)
    np.testing.assert_array_equal(to_np(r["prob_sum"]), np.bincount(e, minlength=E))
