"""The learner's layer: router, MXFP4 forward, backward down to the router's
weights and AdamW, run together.  Each stage is checked against the entry
points it chains or the oracle, the gradients of the router's losses through
the whole step, then captured replays of whole steps against eager ones."""

import numpy as np
import pytest
import torch

import workloads
from _helpers import assert_gemm_close, gpu, require_gpu, to_gpu, to_np
from oracle import gemm, moe, router

pytestmark = gpu

T, K, E, D, F = 300, 4, 32, 256, 128


def _learner(init, **kw):
    from nvfp4_quantized_moe_token_amd import moe_layer
    g = torch.Generator(device="cuda")
    g.manual_seed(init)
    w = [torch.randn(s, generator=g, device="cuda") * 0.05 for s in ((E, D), (E, 2 * F, D), (E, D, F))]
    return moe_layer.Learner(*w, T, K, lr=1e-3, weight_decay=0.1, **kw)


def _batch(seed):
    d = workloads.moe(T, 1.1, 0.01, 16.0, with_dy=True, seed=seed, E=E, k=K, D=D, F=F, weights=False, name="learner")
    return to_gpu(d["x"], torch.bfloat16), to_gpu(d["dy"], torch.bfloat16)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("bits", [32, 8])
def test_step_stage_by_stage(score, bits):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import moe_layer, ops
    ln = _learner(1, score=score, state_bits=bits, router_bias=torch.randn(E, device="cuda") * 0.1)
    x, dy = _batch(1)
    rng = np.random.default_rng(2)
    dlse, dsum = (to_gpu(rng.standard_normal(n).astype(np.float32) * 1e-3, torch.float32) for n in (T, E))
    out = ln.forward(x).clone()
    dx = ln.backward(dy, d_lse=dlse, d_prob_sum=dsum).clone()
    torch.cuda.synchronize()
    off1 = np.array([0, T])
    xn, wr = to_np(x), to_np(ln.w_r)
    # router: logits, ids, weights
    ref, ab = gemm.grouped_gemm_bf16("NT", xn, wr[None], off1)
    logits = to_np(ln.logits)
    assert_gemm_close(logits, ref, ab, what="logits")
    ids = router.select(logits, to_np(ln.router_bias), K)
    np.testing.assert_array_equal(to_np(ln.topk_ids), ids)
    # experts' forward: the public chain on the same routing
    buf = moe_layer.BuffersMXFP4(T, K, E, D, F, x.device)
    moe_layer.forward_mxfp4(x, ln.topk_ids, ln.topk_w, ln.wq_gu, ln.wq_dn, buf)
    assert torch.equal(buf.out, out)
    # gradient of the routing weights, then of the logits
    y2, dest = to_np(ln.buf.y2).astype(np.float64), to_np(ln.meta["dest"]).reshape(T, K)
    dw = (to_np(dy).astype(np.float64)[:, None, :] * y2[dest]).sum(2)
    dw_abs = np.abs(to_np(dy).astype(np.float64)[:, None, :] * y2[dest]).sum(2)
    assert (np.abs(to_np(ln.d_topk_w) - dw) <= 2.0 ** -19 * dw_abs).all()
    want = router.backward(logits, ids, "all" if score else "topk", 1.0, to_np(ln.d_topk_w), to_np(dlse), to_np(dsum))
    dl = to_np(ln.d_logits)
    assert np.abs(dl - want).max() <= 2.0 ** -8 * np.abs(want).max()
    # weights' gradients and the input's, from the step's own intermediates
    ref, ab = gemm.grouped_gemm_bf16("TN", dl, xn, off1)
    assert_gemm_close(to_np(ln.dw_r), ref, ab, what="router weights")
    off = to_np(ln.meta["offsets"])
    ref, ab = gemm.grouped_gemm_bf16("TN", to_np(ln.buf.dy2), to_np(ln.buf.h), off)
    assert_gemm_close(to_np(ln.buf.dw_dn), ref, ab, what="down weights")
    ref, ab = gemm.grouped_gemm_bf16("TN", to_np(ln.buf.dy1), xn[to_np(ln.meta["src"]) // K], off)
    assert_gemm_close(to_np(ln.buf.dw_gu), ref, ab, what="gate+up weights")
    a, aab = gemm.grouped_gemm_bf16("NN", dl, wr[None], off1)
    b = moe.unpermute(to_np(ln.buf.dx_perm), dest.reshape(-1), K)
    bab = moe.unpermute_absbound(to_np(ln.buf.dx_perm), dest.reshape(-1), K)
    assert (np.abs(to_np(dx) - (a + b)) <= 1e-3 * aab + 2.0 ** -20 * (bab + np.abs(a)) + 1e-30).all()
    # update: the copies follow the masters
    before = [w.clone() for w in ln.master]
    ln.update()
    torch.cuda.synchronize()
    for w, c, w0 in zip(ln.master, ln.copies, before):
        assert torch.equal(c, w.to(torch.bfloat16)) and not torch.equal(w, w0)
    q, s = ops.mx_quantize(ln.w_dn.reshape(E * D, F), ops.MX_E2M1)
    assert torch.equal(ln.wq_dn["q"].view(E * D, F // 2), q) and torch.equal(ln.wq_dn["s"].view(E * D, F // 32), s)


def test_weight_gradient_in_the_nvfp4_path():
    """backward and backward_nvfp4 with d_topk_w: the same dY rows, and the
    combine's weight gradient from the W4A4 forward's Y2."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import moe_layer
    d = workloads.moe(T, 1.1, 0.01, 16.0, with_dy=True, seed=3, E=E, k=K, D=D, F=F, name="learner")
    x, w_gu, w_dn, dy = (to_gpu(d[n], torch.bfloat16) for n in ("x", "w_gu", "w_dn", "dy"))
    ids, tw = to_gpu(d["topk_ids"], torch.int32), to_gpu(d["topk_w"], torch.float32)
    dev = torch.device("cuda")
    buf = moe_layer.Buffers(T, K, E, D, F, dev, backward=True)
    nb = moe_layer.NVFP4BackwardBuffers(T, K, E, D, F, dev)
    wq = [moe_layer.quantize_expert_weights(w) for w in (w_gu, w_dn)]
    wt = [moe_layer.quantize_expert_weights_t(w) for w in (w_gu, w_dn)]
    meta = moe_layer.forward(x, ids, tw, *wq, buf)
    got = []
    for run in (lambda g: moe_layer.backward(dy, tw, w_gu, w_dn, meta, buf, d_topk_w=g),
                lambda g: moe_layer.backward_nvfp4(dy, tw, *wt, meta, buf, nb, d_topk_w=g)):
        g = torch.zeros(T, K, device=dev)
        run(None)
        plain = buf.dy2.clone(), buf.dx.clone(), buf.dw_gu.clone()
        run(g)
        torch.cuda.synchronize()
        for a, b in zip(plain, (buf.dy2, buf.dx, buf.dw_gu)):
            assert torch.equal(a, b)
        got.append(g)
    assert torch.equal(got[0], got[1])
    y2 = to_np(buf.y2).astype(np.float64)[to_np(meta["dest"]).reshape(T, K)]
    terms = to_np(dy).astype(np.float64)[:, None, :] * y2
    assert (np.abs(to_np(got[0]) - terms.sum(2)) <= 2.0 ** -19 * np.abs(terms).sum(2)).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_learner_steps_equal_eager(bits):
    require_gpu()
    a, b = (_learner(7, state_bits=bits, capturable=True, seed=3) for _ in range(2))
    x, dy = _batch(0)

    def step(ln):
        ln.forward(x)
        ln.backward(dy)
        ln.update()

    step(a)
    step(b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(b)
    wq = b.wq_gu, b.wq_dn
    for seed in range(1, 4):
        x2, dy2 = _batch(seed)
        x.copy_(x2)
        dy.copy_(dy2)
        step(a)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.buf.out, b.buf.out), seed
        for u, v in zip(a.master + a.copies + a.grads(), b.master + b.copies + b.grads()):
            assert torch.equal(u, v), seed
    assert b.wq_gu is wq[0]


def test_an_example_trains():
    """The layer runs as a user would: many steps, every gradient finite, the
    weights moving by at most the rate each (loss not judged)."""
    require_gpu()
    ln = _learner(9, state_bits=8)
    for seed in range(6):
        x, dy = _batch(seed)
        before = [w.clone() for w in ln.master]
        ln.forward(x)
        ln.backward(dy)
        ln.update()
        for w, w0, g in zip(ln.master, before, ln.grads()):
            assert torch.isfinite(g).all() and torch.isfinite(w).all()
            # Adam's step is at most (1 - b1) / sqrt(1 - b2) rates (3.2), plus the decay
            assert (w - w0).abs().max() <= 1e-3 * (3.3 + 0.1 * w0.abs().max())


def test_a_step_without_tokens():
    """No tokens, no gradients: the update is the weight decay alone."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import moe_layer
    g = torch.Generator(device="cuda").manual_seed(1)
    w = [torch.randn(s, generator=g, device="cuda") * 0.05 for s in ((E, D), (E, 2 * F, D), (E, D, F))]
    before = [x.clone() for x in w]
    ln = moe_layer.Learner(*w, 0, K, lr=1e-3, weight_decay=0.5)
    for t in ln.grads():
        t.fill_(9)
    x = torch.zeros(0, D, dtype=torch.bfloat16, device="cuda")
    assert ln.forward(x).shape == (0, D)
    assert ln.backward(x).shape == (0, D)
    ln.update()
    torch.cuda.synchronize()
    for t, u, v in zip(ln.grads(), ln.master, before):
        assert (t == 0).all()
        assert (u - v * (1 - 1e-3 * 0.5)).abs().max() <= 2.0 ** -22 * v.abs().max()
