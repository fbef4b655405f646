"""GPU parity of the AdamW step: fp32 moments and parameters against fp64
within counted roundings, 8-bit moments bit for bit against the oracle's fp32
steps and codes, over odd sizes, unaligned views, more tensors than one launch
takes, every dtype; skips, gradient scales, device step and rate; captured
replays; the learner's layer step that uses it."""

import numpy as np
import pytest
import torch

from _helpers import gpu, require_gpu, to_np
from oracle import adamw

pytestmark = gpu

U = 2.0 ** -24
HYPER = dict(lr=3e-4, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)
F32, BF16 = torch.float32, torch.bfloat16


def _np32(t):
    return t.detach().float().cpu().numpy().reshape(-1)


def _tensors(sizes, dtype, gen, scale, gap=0):
    """Views of one buffer, `gap` elements between them (odd gaps: unaligned)."""
    total = sum(sizes) + gap * (len(sizes) + 1)
    buf = (torch.randn(total, generator=gen, device="cuda") * scale).to(dtype)
    out, at = [], gap
    for n in sizes:
        out.append(buf[at:at + n])
        at += n + gap
    return buf, out


def _check_params(got, p, upd, bf16):
    """p (1 - lr wd) - rate * (m / (sqrt(v) * r + eps)): the first product, its
    factor (2 roundings) and the difference, relative to |p| and the update;
    and in the update the moments' constants, products and sum (3, relative to
    the magnitudes of the terms that m adds, `upd`, since they may cancel; 5,
    halved under the root), root, r, product, sum, quotient, product and the
    rate's 2: 14 with room to spare."""
    tol = 5 * U * (np.abs(p) + upd) + 14 * U * upd + 1e-37
    if bf16:
        tol = tol + 2.0 ** -7 * np.abs(p)  # rounded up or down, not to nearest: a whole step
    err = np.abs(got.astype(np.float64) - p)
    assert (err <= tol).all(), float((err / tol).max())


SIZES = [1, 3, 255, 256, 257, 1024, 4095, 4096, 4097, 100003]


@pytest.mark.parametrize("gap", [0, 1, 64])
@pytest.mark.parametrize("grad", [F32, BF16])
@pytest.mark.parametrize("param", [F32, BF16])
@pytest.mark.parametrize("bits", [32, 8])
def test_three_steps(bits, param, grad, gap):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import optim
    gen = torch.Generator(device="cuda")
    gen.manual_seed(bits + gap)
    pbuf, params = _tensors(SIZES, param, gen, 0.02, gap)
    copies = None
    if param == F32:
        cbuf, copies = _tensors(SIZES, BF16, gen, 0.0, gap)
        copies[2] = None
    opt = optim.AdamW(params, params_bf16=copies, state_bits=bits, seed=77, **HYPER)
    pad0 = pbuf.clone()
    for step in range(1, 4):
        _, grads = _tensors(SIZES, grad, gen, 1e-3, gap)
        gs = None if step == 1 else torch.full((1,), 0.37, device="cuda")
        old = [(_np32(p), *(_np32(x) for x in (m, v)))
               for p, m, v in zip(params, *[[t.clone() for t in s] for s in opt.state_values()])]
        opt.step(grads, grad_scale=gs)
        torch.cuda.synchronize()
        new = opt.state_values()
        for i, n in enumerate(SIZES):
            p, m, v = old[i]
            g = _np32(grads[i])
            g32 = g * np.float32(1 if gs is None else 0.37)
            want_p, want_m, want_v, upd = adamw.step_f64(p, g32, m, v, step, HYPER["lr"], HYPER["betas"], HYPER["eps"],
                                                         HYPER["weight_decay"])
            m32, v32 = adamw.moments_f32(g, m, v, HYPER["betas"], 1.0 if gs is None else 0.37)
            if bits == 32:
                np.testing.assert_array_equal(_np32(new[0][i]), m32)
                np.testing.assert_array_equal(_np32(new[1][i]), v32)
                assert (np.abs(m32 - want_m) <= 3 * U * (np.abs(0.9 * m) + np.abs(0.1 * g32))).all()
            else:
                r = adamw.random_bits(77, step, i, n)
                mc, ms, vc, vs = adamw.encode(m32, v32, r)
                np.testing.assert_array_equal(to_np(opt.state["exp_avg"][i]), mc)
                np.testing.assert_array_equal(to_np(opt.state["exp_avg_sq"][i]), vc)
                np.testing.assert_array_equal(to_np(opt.state["avg_scale"][i]), ms)
                np.testing.assert_array_equal(to_np(opt.state["avg_sq_scale"][i]), vs)
                dm, dv = adamw.decode(mc, ms, vc, vs)
                np.testing.assert_array_equal(_np32(new[0][i]), dm)
                np.testing.assert_array_equal(_np32(new[1][i]), dv)
            _check_params(_np32(params[i]), want_p, upd, param == BF16)
            if param == F32 and copies[i] is not None:
                assert torch.equal(copies[i], params[i].to(BF16))
    # nothing between the tensors was written
    at = 0
    for n in SIZES:
        assert torch.equal(pbuf[at:at + gap], pad0[at:at + gap])
        at += gap + n


def test_bf16_parameters_move_by_less_than_a_step_on_average():
    """Updates of 2^-11 of a parameter, a sixteenth of its bf16 step: to
    nearest nothing would move.  The mean of n stochastic roundings is off by
    at most 5 standard errors, step / 2 / sqrt(n) each."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import optim
    n = 1 << 16
    p = torch.ones(n, dtype=BF16, device="cuda")
    opt = optim.AdamW([p], lr=2.0 ** -11, betas=(0.9, 0.999), eps=0.0, weight_decay=0.0)
    opt.step([torch.ones(n, device="cuda")])
    step = 2.0 ** -8                       # below 1
    assert set(p.float().unique().tolist()) == {1.0, 1.0 - step}
    assert abs(p.double().mean().item() - (1 - 2.0 ** -11)) <= 5 * step / 2 / n ** 0.5 + 2.0 ** -20


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_and_empty_ones(bits):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import optim
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    sizes = [(i * 97) % 700 if i % 5 else 0 for i in range(131)]      # three launches, empty tensors among them
    one = optim.AdamW(_tensors(sizes, F32, gen, 0.02, 64)[1], state_bits=bits, seed=5, **HYPER)
    two = optim.AdamW([p.clone() for p in one.params], state_bits=bits, seed=5, **HYPER)
    grads = _tensors(sizes, F32, gen, 1e-3, 64)[1]
    before = [p.clone() for p in one.params]
    one.step(grads)
    two.step([g.clone() for g in grads])
    torch.cuda.synchronize()
    m, v = one.state_values()
    for i, n in enumerate(sizes):
        assert torch.equal(one.params[i], two.params[i])
        want, _, _, upd = adamw.step_f64(_np32(before[i]), _np32(grads[i]), 0, 0, 1, HYPER["lr"], HYPER["betas"],
                                         HYPER["eps"], HYPER["weight_decay"])
        _check_params(_np32(one.params[i]), want, upd, False)
        if bits == 8 and n:                                          # the tensor's place in the list counts
            m32, v32 = adamw.moments_f32(_np32(grads[i]), np.zeros(n), np.zeros(n), HYPER["betas"])
            mc, _, vc, _ = adamw.encode(m32, v32, adamw.random_bits(5, 1, i, n))
            np.testing.assert_array_equal(to_np(one.state["exp_avg"][i]), mc)
            np.testing.assert_array_equal(to_np(one.state["exp_avg_sq"][i]), vc)


@pytest.mark.parametrize("bits", [32, 8])
def test_skip_and_device_step_and_rate(bits):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import optim
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    p0, g = (torch.randn(5000, generator=gen, device="cuda") for _ in range(2))
    a = optim.AdamW([p0.clone()], state_bits=bits, **HYPER)
    b = optim.AdamW([p0.clone()], state_bits=bits, capturable=True, **HYPER)
    skip = torch.zeros(1, dtype=torch.int32, device="cuda")
    for flag in (0, 1, 0):
        skip.fill_(flag)
        was = a.params[0].clone(), [t.clone() for t in a.state_values()[0]]
        a.step([g], skip=skip)
        b.step([g], skip=skip)
        torch.cuda.synchronize()
        assert torch.equal(a.params[0], b.params[0])
        assert all(torch.equal(x, y) for s in a.state for x, y in zip(a.state[s], b.state[s]))
        if flag:
            assert torch.equal(a.params[0], was[0]) and torch.equal(a.state_values()[0][0], was[1][0])
        else:
            assert not torch.equal(a.params[0], was[0])
    assert a.steps == 3 and b.step_dev.item() == 3
    b.lr_dev.zero_()
    was = b.params[0].clone()
    b.step([g])
    torch.cuda.synchronize()
    assert torch.equal(b.params[0], was)   # rate 0: neither update nor decay


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_count_on(bits):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import optim
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    sizes = [1000, 257, 30000]
    ps = [torch.randn(n, generator=gen, device="cuda") for n in sizes]
    grads = [torch.randn(n, generator=gen, device="cuda") for n in sizes]
    eager = optim.AdamW([p.clone() for p in ps], state_bits=bits, seed=9, **HYPER)
    cap = optim.AdamW([p.clone() for p in ps], state_bits=bits, seed=9, capturable=True, **HYPER)
    eager.step(grads)
    cap.step(grads)                        # (a first step outside the graph)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap.step(grads)
    for _ in range(3):
        for x in grads:
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        eager.step(grads)
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(eager.params, cap.params):
            assert torch.equal(x, y)
        for s in eager.state:
            for x, y in zip(eager.state[s], cap.state[s]):
                assert torch.equal(x, y)


def test_not_finite_gradients_stay_where_they_are():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import optim
    n = 1024
    g = torch.ones(n, device="cuda")
    g[5], g[300], g[301] = float("nan"), float("inf"), -float("inf")
    bad = ~torch.isfinite(g)
    for bits in (32, 8):
        opt = optim.AdamW([torch.ones(n, device="cuda")], state_bits=bits, seed=1, **HYPER)
        opt.step([g])
        m, v = opt.state_values()
        torch.cuda.synchronize()
        assert torch.isfinite(opt.params[0][~bad]).all() and torch.isnan(opt.params[0][bad]).all()
        assert torch.isfinite(m[0][~bad]).all() and torch.isfinite(v[0][~bad]).all()
        assert not torch.isfinite(m[0][bad]).any() and not torch.isfinite(v[0][bad]).any()


def test_refusals():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import optim
    p = torch.zeros(100, device="cuda")
    opt = optim.AdamW([p])
    for bad in ([], [p, p], [p[:99]], [p.half()], [p.cpu()], [torch.zeros(100, 2, device="cuda")[:, 0]]):
        with pytest.raises(ValueError):
            opt.step(bad)
    for kw in (dict(grad_scale=torch.ones(2, device="cuda")), dict(skip=torch.zeros(1, device="cuda"))):
        with pytest.raises(ValueError):
            opt.step([p], **kw)
    with pytest.raises(ValueError):
        optim.AdamW([torch.zeros(100, 2, device="cuda").t()])
    assert opt.steps == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_a_refused_step_changes_nothing(bits):
    """Gradients on the host, missing, strided or of the wrong number are
    refused; the step count and the weights stay, and the next step counts on."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import optim
    shapes = [(0,), (), (300,)]
    params = [torch.ones(s, device="cuda") for s in shapes]
    good = [torch.ones(s, device="cuda") for s in shapes]
    opt = optim.AdamW(params, state_bits=bits, lr=0.1, weight_decay=0.0)
    bad = [[good[0], torch.ones(()), good[2]], good[:2], [good[0], None, good[2]],
           [good[0], good[1], torch.ones(600, device="cuda")[::2]], [good[0], good[1].bfloat16(), good[2]]]
    for grads in bad:
        with pytest.raises(ValueError):
            opt.step(grads)
    torch.cuda.synchronize()
    assert opt.steps == 0 and all((p == 1).all() for p in params)
    opt.step(good)
    torch.cuda.synchronize()
    # m / sqrt(v) of a first step is 1: the weights move by the rate, to a few roundings
    assert opt.steps == 1 and all((p - 0.9).abs().max() < 1e-6 for p in params if p.numel())


@pytest.mark.parametrize("bits", [32, 8])
def test_weights_moved_away_and_back(bits):
    """Parameters, copies and moments whose storage was replaced between steps:
    the next step works on the new one, and the old one stays as it was."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import optim
    gen = torch.Generator(device="cuda")
    gen.manual_seed(8)
    sizes = [300, 4097]
    ps, gs = ([torch.randn(n, generator=gen, device="cuda") for n in sizes] for _ in range(2))
    a, b = (optim.AdamW([p.clone() for p in ps], params_bf16=[p.to(BF16) for p in ps], state_bits=bits, seed=2, **HYPER)
            for _ in range(2))
    a.step(gs)
    b.step(gs)
    held = [*a.params, *a.params_bf16, *(t for ts in a.state.values() for t in ts)]
    old = [t.data for t in held]
    was = [t.clone() for t in old]
    for t in held:
        t.data = t.data.clone()
    a.step(gs)
    b.step(gs)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(old, was))
    for x, y in zip(held, [*b.params, *b.params_bf16, *(t for ts in b.state.values() for t in ts)]):
        assert torch.equal(x, y)
    a.params[0].data = a.params[0].data.cpu()
    with pytest.raises(ValueError):
        a.step(gs)
    assert a.steps == 2


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("capturable", [False, True])
def test_skipped_steps_leave_no_trace(bits, capturable):
    """Steps with and without the skip flag set, eager and replayed: the same
    bits as an optimizer that was never asked for the skipped ones."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import optim
    gen = torch.Generator(device="cuda")
    gen.manual_seed(12)
    p0 = torch.randn(3000, generator=gen, device="cuda")
    gs = [torch.randn(3000, generator=gen, device="cuda") for _ in range(6)]
    a, b = (optim.AdamW([p0.clone()], state_bits=bits, seed=4, capturable=c, **HYPER) for c in (capturable, False))
    skip = torch.zeros(1, dtype=torch.int32, device="cuda")

    def same():
        torch.cuda.synchronize()
        assert torch.equal(a.params[0], b.params[0]) and a.updates() == b.steps
        for s in a.state:
            assert torch.equal(a.state[s][0], b.state[s][0])

    for g, flag in zip(gs, (1, 1, 0, 1, None, 0)):
        skip.fill_(flag or 0)
        a.step([g], skip=None if flag is None else skip)
        if not flag:
            b.step([g])
        same()
    if not capturable:
        return
    x = gs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step([x], skip=skip)
    a.steps -= 1                            # (captured, not run)
    for g, flag in zip(gs, (0, 1, 0, 1, 1, 0)):
        skip.fill_(flag)
        x.copy_(g)
        graph.replay()
        if not flag:
            b.step([g])
        same()


def test_a_positive_second_moment_never_becomes_zero():
    """Gradients whose squares lie so far apart that fp32 has no quotient."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import optim
    g = torch.zeros(512, device="cuda")
    g[:5] = torch.tensor([2.0 ** 50, 2.0 ** 30, 2.0 ** -24, 2.0 ** -30, -2.0 ** -60])
    opt = optim.AdamW([torch.ones(512, device="cuda")], state_bits=8, seed=6, **HYPER)
    opt.step([g])
    torch.cuda.synchronize()
    m32, v32 = adamw.moments_f32(_np32(g), np.zeros(512, np.float32), np.zeros(512, np.float32), HYPER["betas"])
    _, _, vc, vs = adamw.encode(m32, v32, adamw.random_bits(6, 1, 0, 512))
    got = to_np(opt.state["exp_avg_sq"][0])
    np.testing.assert_array_equal(got, vc)
    np.testing.assert_array_equal(to_np(opt.state["avg_sq_scale"][0]), vs)
    assert (got[:5] > 0).all() and (got[5:] == 0).all()
