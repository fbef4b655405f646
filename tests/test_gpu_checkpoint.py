"""GPU parity of activations kept in 8 bits: the MXINT8 quantizer bit for bit
against the oracle, the decoder of all MX formats, the gate's backward from kept
codes against fp64, the MXFP4 product's epilogue against the separate steps, the
layer's backward from them, and the learner with every choice of experts,
checkpoint and norm run together as it is used."""

import numpy as np
import pytest
import torch

import workloads
from _helpers import assert_gemm_close, gpu, require_gpu, to_gpu, to_np
from oracle import gemm, moe, mx, norm

pytestmark = gpu

F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8
U = 2.0 ** -24


def _check_quantize(x):
    from nvfp4_quantized_moe_token_amd import ops
    q, s = ops.mx_quantize(x, ops.MX_INT8)
    rq, rs = mx.quantize_int8(to_np(x))
    np.testing.assert_array_equal(to_np(s), rs)
    live = np.repeat(rs != 255, 32, axis=1)
    np.testing.assert_array_equal(np.where(live, to_np(q).view(np.int8), 0), rq)
    v = mx.dequantize_int8(rq, rs)
    f = ops.mx_dequantize(q, s, ops.MX_INT8, out_dtype=F32)
    np.testing.assert_array_equal(to_np(f), v.astype(np.float32))
    b = ops.mx_dequantize(q, s, ops.MX_INT8)
    assert b.dtype == BF16
    np.testing.assert_array_equal(to_np(b), v.astype(np.float32))  # 7 significant bits: exact
    return q, s


@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (130, 1536), (5, 4096), (1000, 96)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_mxint8_bit_exact(rows, K, dtype):
    require_gpu()
    rng = np.random.default_rng(rows * K)
    x = rng.standard_normal((rows, K)) * np.exp(rng.uniform(-30, 30, (rows, 1)))
    _check_quantize(to_gpu(x.astype(np.float32), dtype))


def test_mxint8_where_it_can_go_wrong():
    require_gpu()
    rng = np.random.default_rng(1)
    x = rng.standard_normal((12, 64)).astype(np.float32)
    x[0] = 0
    x[1, :32] *= np.float32(1e-42)
    x[2] = np.float32(2.0 ** -149)
    x[3] = np.float32(3.4028235e38)
    x[4, 3], x[5, 40], x[6, 0] = np.nan, np.inf, -np.inf
    x[7] = (np.arange(64) - 32 + 0.5) / 64     # ties of a block with S = 126 or 127
    x[7, 0] = x[7, 32] = 1
    x[8] = 1.9999999                            # clamps
    x[9, :32] = np.float32(2.0 ** -126)
    x[9, 32:] = np.nextafter(np.float32(2.0 ** -126), np.float32(0))
    for dtype in (F32, BF16):
        _check_quantize(to_gpu(x, dtype))
    v = (np.arange(65536, dtype=np.uint32) << 16).view(np.float32)  # every bf16 value, alone in its block
    x = np.zeros((65536, 32), np.float32)
    x[:, 5] = v
    _check_quantize(to_gpu(x, BF16))


def test_decoder_of_the_floating_formats():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    rng = np.random.default_rng(2)
    for elem, name, cols in ((ops.MX_E4M3, "e4m3", 256), (ops.MX_E2M1, "e2m1", 128)):
        q = rng.integers(0, 256, (64, cols)).astype(np.uint8)
        if name == "e4m3":
            q[0] = np.arange(256)
            q[q & 0x7F == 0x7F] = 0  # (no NaN codes, which the quantizer never gives)
        s = rng.integers(0, 255, (64, 8)).astype(np.uint8)
        s[1, :3] = [0, 254, 1]
        v = mx.dequantize(q, s, name)
        with np.errstate(over="ignore"):
            want = v.astype(np.float32)
        for dtype in (F32, BF16):
            got = ops.mx_dequantize(to_gpu(q, U8), to_gpu(s, U8), elem, out_dtype=dtype)
            ref = torch.from_numpy(want).to(dtype).float().numpy()
            np.testing.assert_array_equal(to_np(got), ref)


def _gate_backward(y1, dh):
    """dG, dU, H and the sizes of what is rounded, in fp64."""
    F = y1.shape[1] // 2
    g, u = y1[:, :F], y1[:, F:]
    sg = 1 / (1 + np.exp(-g))
    return dh * u * sg * (1 + g * (1 - sg)), dh * g * sg, g * sg * u, np.abs(dh * u) * sg * (1 + np.abs(g) * (1 - sg))


def _check_gate_backward(q, s, dh, dy1, h):
    y1 = mx.dequantize_int8(to_np(q).view(np.int8), to_np(s))
    F = y1.shape[1] // 2
    with np.errstate(over="ignore", invalid="ignore"):
        dg, du, hr, size = _gate_backward(y1, to_np(dh).astype(np.float64))
    # fp32: e^-g and its reciprocal are off by two units each, and 1 - sigmoid by as much as sigmoid; ten
    # roundings more at most; then one to bf16.  e^-g's argument is rounded, g (units of g) more.
    g = np.abs(y1[:, :F])
    eps = (16 + g) * 2 * U
    # a sigmoid below 2^-126 (g below -87.3) is 0: 1 + e^-g passes 2^126 there, whose reciprocal the hardware
    # gives as 0 rather than a subnormal.  Off by at most 2^-126 times what it is multiplied with.
    u, d = np.abs(y1[:, F:]), np.abs(to_np(dh).astype(np.float64))
    got = to_np(dy1).astype(np.float64)
    for a, ref, sz, times in ((got[:, :F], dg, size, d * u * (1 + g)), (got[:, F:], du, np.abs(du), d * g),
                              (to_np(h).astype(np.float64), hr, np.abs(hr), g * u)):
        tol = eps * sz + 2.0 ** -126 * times
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol) + 1e-37
        ok = np.abs(a - ref) <= tol
        assert ok[np.isfinite(ref)].all(), float((np.abs(a - ref) / tol)[np.isfinite(ref)].max())


@pytest.mark.parametrize("R,F", [(1, 32), (5, 96), (333, 352), (64, 768), (1333, 128), (2, 9728)])
def test_gate_backward(R, F):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    rng = np.random.default_rng(R + F)
    y1 = to_gpu((rng.standard_normal((R, 2 * F)) * np.exp(rng.uniform(-3, 2, (R, 1)))).astype(np.float32), BF16)
    dh = to_gpu(rng.standard_normal((R, F)).astype(np.float32) * 1e-3, BF16)
    q, s = ops.mx_quantize(y1, ops.MX_INT8)
    flat = torch.full((R * 3 * F + 64,), 5.0, dtype=BF16, device="cuda")
    dy1, h = flat[:2 * R * F].view(R, 2 * F), flat[2 * R * F:3 * R * F].view(R, F)
    ops.silu_gate_bwd_mx(q, s, dh, dy1=dy1, h=h)
    assert (flat[-64:] == 5).all()
    _check_gate_backward(q, s, dh, dy1, h)
    only, none = ops.silu_gate_bwd_mx(q, s, dh, want_h=False)
    assert none is None and torch.equal(only, dy1)
    # the same values kept in bf16 give the same gradient, and H of the forward
    y = ops.mx_dequantize(q, s, ops.MX_INT8)
    assert torch.equal(ops.silu_gate_bwd(y, dh), dy1) and torch.equal(ops.silu_gate_fwd(y)[0], h)


def test_gate_backward_of_extremes():
    """Saturated gates, zeros, and blocks that were not finite: NaN in their features alone."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    R, F = 6, 64
    rng = np.random.default_rng(3)
    y = rng.standard_normal((R, 2 * F)).astype(np.float32)
    y[0] = 0
    y[1, :F] = -90
    y[2, :F] = 90
    y[3, :F] = np.where(np.arange(F) % 2, 200, -200)
    clean = y.copy()
    y[4, 3] = np.nan
    y[5, F + 40] = np.inf
    dh = to_gpu(rng.standard_normal((R, F)).astype(np.float32), BF16)
    q0, s0 = ops.mx_quantize(to_gpu(clean, BF16), ops.MX_INT8)
    q, s = ops.mx_quantize(to_gpu(y, BF16), ops.MX_INT8)
    want, hw = ops.silu_gate_bwd_mx(q0, s0, dh)
    _check_gate_backward(q0, s0, dh, want, hw)
    assert want.isfinite().all() and hw.isfinite().all()
    got, h = ops.silu_gate_bwd_mx(q, s, dh)
    assert torch.equal(got[:4], want[:4]) and torch.equal(h[:4], hw[:4])
    nan = torch.zeros(R, F, dtype=torch.bool, device="cuda")
    nan[4, :32] = nan[5, 32:] = True
    assert torch.equal(h.isnan(), nan) and torch.equal(got[:, :F].isnan(), nan)
    assert got[4, F:F + 32].isnan().all()
    empty, eh = ops.silu_gate_bwd_mx(q[:0], s[:0], dh[:0])
    assert empty.shape == (0, 2 * F) and eh.shape == (0, F)


@pytest.mark.parametrize("counts,F,K", [([0, 1, 300, 0, 37], 128, 256), ([600, 0, 520, 1], 256, 128), ([5, 0, 1, 40] * 8, 128, 640),
                                        ([90, 100, 120], 384, 128), ([64, 33, 50], 256, 384)])
@pytest.mark.parametrize("form", ["q", "h", "all"])
def test_mxfp4_epilogue_keeps_y1(counts, F, K, form):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M, E, end = int(off[-1]) + 2, len(counts), int(off[-1])
    g = torch.Generator(device="cuda").manual_seed(M + F)
    a = ops.mx_quantize(torch.randn(M, K, generator=g, device="cuda"), ops.MX_E2M1)
    b = ops.mx_quantize(torch.randn(E * 2 * F, K, generator=g, device="cuda") * 0.1, ops.MX_E2M1)
    b = (b[0].view(E, 2 * F, K // 2), b[1].view(E, 2 * F, K // 32))
    offs = to_gpu(off, torch.int32)
    want = ops.grouped_gemm_mxfp4_silu_gate(*a, *b, offs, want_q=True)
    wq, ws = ops.mx_quantize(want["y1"], ops.MX_INT8)
    u8 = dict(dtype=U8, device="cuda")
    q_y1, s_y1 = torch.full((M, 2 * F), 77, **u8), torch.full((M, 2 * F // 32), 77, **u8)
    am, am0 = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    ops.grouped_gemm_mxfp4_silu_gate(*a, *b, offs, amax_out=am0)
    r = ops.grouped_gemm_mxfp4_silu_gate(*a, *b, offs, want_y1=form == "all", want_h=form != "q", want_q=form != "h",
                                         q_y1=q_y1, s_y1=s_y1, amax_out=am)
    assert torch.equal(r["q_y1"][:end], wq[:end]) and torch.equal(r["s_y1"][:end], ws[:end])
    assert (q_y1[end:] == 77).all() and (s_y1[end:] == 77).all()
    assert torch.equal(am, am0)
    for n in dict(q=("q_h", "s_h"), h=("h",), all=("y1", "h", "q_h", "s_h"))[form]:
        assert torch.equal(r[n][:end], want[n][:end]), n


# ------------------------------------------------------------------ the layer

T, K, E, D, F = 300, 4, 32, 256, 128


def _batch(seed):
    d = workloads.moe(T, 1.1, 0.01, 16.0, with_dy=True, seed=seed, E=E, k=K, D=D, F=F, weights=False, name="learner")
    return to_gpu(d["x"], BF16), to_gpu(d["dy"], BF16)


def _learner(init, norm=None, **kw):
    from nvfp4_quantized_moe_token_amd import moe_layer
    g = torch.Generator(device="cuda").manual_seed(init)
    w = [torch.randn(s, generator=g, device="cuda") * 0.05 for s in ((E, D), (E, 2 * F, D), (E, D, F))]
    if norm is not None:
        w_n = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
        kw.update(norm_kind=norm, norm=(w_n, None if norm else 0.1 * torch.randn(D, generator=g, device="cuda")))
    return moe_layer.Learner(*w, T, K, lr=1e-3, weight_decay=0.1, **kw)


@pytest.mark.parametrize("experts", ["mxfp4", "int8"])
@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("kind", [None, 0, 1])
def test_learner_step_stage_by_stage(experts, checkpoint, kind):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import moe_layer, ops
    ln = _learner(1, norm=kind, experts=experts, checkpoint=checkpoint)
    x, dy = _batch(1)
    out = ln.forward(x).clone()
    b = ln.buf
    # the norm
    if kind is None:
        xn = x
        assert ln.x is x
    else:
        w = ln.norm[0], ln.norm[1] if len(ln.norm) > 1 else None
        f = ops.layer_norm(x, *w, eps=1e-6, kind=kind)
        xn = f["y"]
        assert torch.equal(ln.x, xn)
    # the experts' forward: the public chain on the same routing, nothing kept
    buffers, forward, quantize = dict(mxfp4=(moe_layer.BuffersMXFP4, moe_layer.forward_mxfp4, moe_layer.quantize_expert_weights_mx),
                                      int8=(moe_layer.BuffersInt8, moe_layer.forward_int8,
                                            moe_layer.quantize_expert_weights_int8))[experts]
    alone = buffers(T, K, E, D, F, x.device)
    forward(xn, ln.topk_ids, ln.topk_w, quantize(ln.w_gu), quantize(ln.w_dn), alone)
    assert torch.equal(alone.out, out)
    kept = buffers(T, K, E, D, F, x.device, backward=True)
    forward(xn, ln.topk_ids, ln.topk_w, ln.wq_gu, ln.wq_dn, kept, keep=True)
    if checkpoint:
        assert b.y1 is None
        q, s = ops.mx_quantize(kept.y1, ops.MX_INT8)
        assert torch.equal(b.q_y1, q) and torch.equal(b.s_y1, s)
        y1 = ops.mx_dequantize(q, s, ops.MX_INT8)
    else:
        assert b.q_y1 is None and torch.equal(b.y1, kept.y1) and torch.equal(b.h, kept.h)
        y1 = kept.y1
    # the backward pass, from Y1 as it was kept
    dx = ln.backward(dy).clone()
    torch.cuda.synchronize()
    assert torch.equal(b.dy1, ops.silu_gate_bwd(y1, b.dh)) and torch.equal(b.h, ops.silu_gate_fwd(y1)[0])
    off = to_np(ln.meta["offsets"])
    ref, ab = gemm.grouped_gemm_bf16("TN", to_np(b.dy2), to_np(b.h), off)
    assert_gemm_close(to_np(b.dw_dn), ref, ab, what="down weights")
    ref, ab = gemm.grouped_gemm_bf16("TN", to_np(b.dy1), to_np(xn)[to_np(ln.meta["src"]) // K], off)
    assert_gemm_close(to_np(b.dw_gu), ref, ab, what="gate+up weights")
    if kind is not None:
        want = ops.layer_norm_bwd(b.dx, x, ln.norm[0], f["mean"], f["rstd"], kind=kind, dx_dtype=F32, want_db=len(ln.norm) > 1)
        assert torch.equal(dx, want["dx"]) and torch.equal(ln.grads()[3], want["dw"])
        if len(ln.norm) > 1:
            assert torch.equal(ln.grads()[4], want["db"])
        assert len(ln.grads()) == 3 + len(ln.norm)
    else:
        assert torch.equal(dx, b.dx) and len(ln.grads()) == 3
    # the update: every weight moves, and the quantized copies follow
    before = [t.clone() for t in ln.master + (ln.norm or [])]
    ln.update()
    for t, t0 in zip(ln.master + (ln.norm or []), before):
        assert not torch.equal(t, t0)
    for n, w in (("wq_gu", ln.w_gu), ("wq_dn", ln.w_dn)):
        again = quantize(w)
        assert torch.equal(getattr(ln, n)["q"], again["q"]) and torch.equal(getattr(ln, n)["s"], again["s"])


def test_the_norms_weights_do_not_decay():
    require_gpu()
    ln = _learner(2, norm=0)
    x, dy = _batch(2)
    ln.forward(x)
    ln.backward(dy)
    for t in ln.grads():
        t.zero_()
    before = [t.clone() for t in ln.norm], [t.clone() for t in ln.master]
    ln.update()
    assert all(torch.equal(a, b) for a, b in zip(before[0], ln.norm))
    assert all(not torch.equal(a, b) for a, b in zip(before[1], ln.master))
    ln.update(skip=torch.ones(1, dtype=torch.int32, device="cuda"))
    assert all(torch.equal(a, b) for a, b in zip(before[0], ln.norm))


@pytest.mark.parametrize("experts", ["mxfp4", "int8"])
def test_the_weight_gradients_may_run_on_a_stream_of_their_own(experts):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import moe_layer
    ln = _learner(3, experts=experts, checkpoint=True)
    x, dy = _batch(3)
    ln.forward(x)
    ln.backward(dy)
    want = [t.clone() for t in (ln.buf.dw_dn, ln.buf.dw_gu)]
    for t in (ln.buf.dw_dn, ln.buf.dw_gu, ln.buf.h, ln.buf.dy1):
        t.fill_(3)
    moe_layer.backward(dy, ln.topk_w, ln.w_gu, ln.w_dn, ln.meta, ln.buf, wgrad_stream=torch.cuda.Stream(), x=x)
    torch.cuda.synchronize()
    assert torch.equal(ln.buf.dw_dn, want[0]) and torch.equal(ln.buf.dw_gu, want[1])


@pytest.mark.parametrize("experts", ["mxfp4", "int8"])
def test_captured_steps_equal_eager(experts):
    require_gpu()
    a, b = (_learner(7, norm=0, experts=experts, checkpoint=True, capturable=True) for _ in range(2))
    x, dy = _batch(0)

    def step(ln):
        out = ln.forward(x)
        return out, ln.backward(dy), ln.update()

    step(a)
    step(b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, dx, _ = step(b)
    for seed in range(1, 4):
        x2, dy2 = _batch(seed)
        x.copy_(x2)
        dy.copy_(dy2)
        want = step(a)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(want[0], out) and torch.equal(want[1], dx), seed
        for u, v in zip(a.master + a.copies + a.norm + a.grads(), b.master + b.copies + b.norm + b.grads()):
            assert torch.equal(u, v), seed


def test_the_gradient_is_the_functions():
    """Differences of the plain layer in fp64 (dense over a token's experts, no quantization) against the
    step's gradients: the direction and size agree as far as 8-bit products allow."""
    require_gpu()
    ln = _learner(11, norm=0, experts="int8", checkpoint=True)
    x, dy = _batch(5)
    ln.forward(x)
    dx = ln.backward(dy).double()
    ids, dest = ln.topk_ids.long(), None
    leaf = [t.detach().double().requires_grad_(True) for t in (x, *ln.master, *ln.norm)]
    X, wr, gu, dn, nw, nb = leaf
    m = X.mean(1, keepdim=True)
    h = (X - m) / torch.sqrt(((X - m) ** 2).mean(1, keepdim=True) + 1e-6) * nw + nb
    tw = torch.softmax(torch.gather(h @ wr.t(), 1, ids), 1)
    out = torch.zeros_like(X)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if len(t):
            y = h[t] @ gu[e].t()
            out = out.index_add(0, t, (torch.nn.functional.silu(y[:, :F]) * y[:, F:]) @ dn[e].t() * tw[t, j, None])
    grads = torch.autograd.grad((out * dy.double()).sum(), leaf)
    # relative errors of one 8-bit operand are about 1 % of its size, and a chain has four of them; a wrong
    # term shows as tens of per cent
    for got, want in zip([dx] + ln.grads(), grads):
        err = (got.double() - want).norm() / want.norm()
        assert err < 0.06, float(err)


def test_an_example_trains():
    require_gpu()
    ln = _learner(9, norm=1, experts="int8", checkpoint=True, state_bits=8)
    for seed in range(5):
        x, dy = _batch(seed)
        ln.forward(x)
        ln.backward(dy)
        ln.update()
        for t in ln.master + ln.norm + ln.grads():
            assert torch.isfinite(t).all()


def test_a_step_without_tokens():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import moe_layer
    w = [torch.randn(s, device="cuda") * 0.05 for s in ((E, D), (E, 2 * F, D), (E, D, F))]
    ln = moe_layer.Learner(*w, 0, K, experts="int8", checkpoint=True, norm=(torch.ones(D, device="cuda"), None), lr=1e-3)
    x = torch.zeros(0, D, dtype=BF16, device="cuda")
    assert ln.forward(x).shape == (0, D) and ln.backward(x).shape == (0, D)
    ln.update()
    assert all((t == 0).all() for t in ln.grads()) and (ln.norm[0] == 1).all()
