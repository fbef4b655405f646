"""GPU parity of the combine's gradient: dY rows bit for bit against
moe_scatter, routing-weight gradients against fp64 dot products (odd sizes,
one token to thousands, dropped assignments, more than 8 and 16 choices), each
output alone, and captured replays."""

import numpy as np
import pytest
import torch

from _helpers import gpu, require_gpu, to_gpu, to_np

pytestmark = gpu

U = 2.0 ** -24


def _case(rng, T, k, E, D, dt_out, dt_y, drop=0):
    from nvfp4_quantized_moe_token_amd import ops
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    if drop:
        ids.reshape(-1)[rng.choice(T * k, min(drop, T * k), replace=False)] = -1
    p = ops.moe_permute(to_gpu(ids, torch.int32), E)
    dout = to_gpu(rng.standard_normal((T, D)).astype(np.float32), dt_out)
    y = to_gpu(rng.standard_normal((T * k, D)).astype(np.float32), dt_y)
    w = to_gpu(rng.random((T, k)).astype(np.float32), torch.float32)
    return p, dout, y, w


def _dw_check(got, dout, y, dest, T, k, D):
    d, yy = to_np(dout).astype(np.float64), to_np(y).astype(np.float64)
    dest = dest.reshape(T, k)
    rows = np.where(dest >= 0, dest, 0)
    want, mag = np.zeros((T, k)), np.zeros((T, k))
    for j in range(k):
        want[:, j] = (d * yy[rows[:, j]]).sum(1)
        mag[:, j] = np.abs(d * yy[rows[:, j]]).sum(1)
    want[dest < 0] = 0
    # a lane's chain of fused products (8 per 512 elements, or per 2048), then
    # 6 exchanges and up to 3 additions across waves
    assert (np.abs(got - want) <= (D / 64 + 20) * U * mag + 1e-37).all()
    assert (got[dest < 0] == 0).all()


F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("T,k,E,D,drop", [
    (1, 1, 1, 8, 0), (1, 8, 16, 2048, 1), (5, 3, 4, 16, 2), (33, 8, 16, 520, 5), (333, 4, 40, 2560, 5),
    (60, 9, 12, 264, 3), (41, 17, 30, 136, 7), (20, 64, 64, 72, 9), (2100, 2, 8, 512, 4), (2500, 8, 128, 200, 0),
    (7, 8, 16, 4104, 56), (3000, 1, 3, 1024, 1)])
@pytest.mark.parametrize("dt", [(BF16, BF16, BF16), (F32, F32, F32), (BF16, F32, BF16), (F32, BF16, F32),
                                (BF16, BF16, F32), (F32, BF16, BF16)])
def test_unpermute_bwd_parity(T, k, E, D, drop, dt):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    rng = np.random.default_rng(T * 31 + k * 7 + D)
    p, dout, y, w = _case(rng, T, k, E, D, dt[0], dt[1], drop)
    amax, amax_ref = (torch.full((1,), 9.0, device="cuda") for _ in range(2))
    dy, dw = ops.moe_unpermute_bwd(dout, y, p["dest"], p["offsets"], k, topk_w=w, dy_dtype=dt[2], amax_out=amax)
    ref = ops.moe_scatter(dout, p["dest"], p["offsets"], k, topk_w=w, out_dtype=dt[2], amax_out=amax_ref)
    torch.cuda.synchronize()
    assert torch.equal(dy, ref) and torch.equal(amax, amax_ref)
    _dw_check(to_np(dw), dout, y, to_np(p["dest"]), T, k, D)
    # without the amax, and each output alone: the same bits
    dy2, dw2 = ops.moe_unpermute_bwd(dout, y, p["dest"], p["offsets"], k, topk_w=w, dy_dtype=dt[2])
    dy3, none = ops.moe_unpermute_bwd(dout, None, p["dest"], p["offsets"], k, topk_w=w, dy_dtype=dt[2], want_dw=False)
    none2, dw3 = ops.moe_unpermute_bwd(dout, y, p["dest"], p["offsets"], k, topk_w=w, want_dy=False)
    torch.cuda.synchronize()
    assert none is None and none2 is None
    assert torch.equal(dy2, dy) and torch.equal(dy3, dy) and torch.equal(dw2, dw) and torch.equal(dw3, dw)


def test_without_weights_and_all_dropped():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    rng = np.random.default_rng(1)
    T, k, E, D = 50, 4, 8, 256
    p, dout, y, _ = _case(rng, T, k, E, D, BF16, BF16, drop=T * k)
    y.fill_(float("nan"))                       # nothing of it belongs to a token
    dout[3] = float("inf")
    dy, dw = ops.moe_unpermute_bwd(dout, y, p["dest"], p["offsets"], k)
    torch.cuda.synchronize()
    assert (dw == 0).all() and (dy == 0).all()
    p, dout, y, _ = _case(rng, T, k, E, D, BF16, BF16)
    dy, dw = ops.moe_unpermute_bwd(dout, y, p["dest"], p["offsets"], k)
    torch.cuda.synchronize()
    assert torch.equal(dy, ops.moe_gather(dout, p["src"], k))
    _dw_check(to_np(dw), dout, y, to_np(p["dest"]), T, k, D)


def test_no_tokens_and_no_width():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    e = torch.empty
    i32 = dict(dtype=torch.int32, device="cuda")
    dy, dw = ops.moe_unpermute_bwd(e(0, 64, device="cuda"), e(0, 64, device="cuda"), e(0, **i32),
                                   torch.zeros(5, **i32), 8)
    assert dy.shape == (0, 64) and dw.shape == (0, 8)
    dw = torch.full((3, 2), 7.0, device="cuda")
    ops.moe_unpermute_bwd(e(3, 0, device="cuda"), e(6, 0, device="cuda"), torch.arange(6, **i32),
                          torch.tensor([0, 6], **i32), 2, d_topk_w=dw)
    torch.cuda.synchronize()
    assert (dw == 0).all()


def test_weight_gradient_against_differences():
    """d/dw of sum(out * dout) with the framework's own forward, in fp32: the
    combine is linear in w, so a difference over a step of 1 has no error but
    the roundings of two sums of D products."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    rng = np.random.default_rng(2)
    T, k, E, D = 6, 3, 4, 128
    p, dout, y, w = _case(rng, T, k, E, D, F32, F32)
    _, dw = ops.moe_unpermute_bwd(dout, y, p["dest"], p["offsets"], k, topk_w=w, want_dy=False)
    for t in range(T):
        for j in range(k):
            w2 = w.clone()
            w2[t, j] += 1
            a, b = (ops.moe_unpermute(y, p["dest"], T, k, topk_w=x, out_dtype=F32).double() for x in (w2, w))
            got = ((a - b) * dout.double()).sum().item()
            mag = (4 * y.abs().max() * dout.abs().max()).item() * D
            assert abs(got - dw[t, j].item()) <= (2 * k + D / 64 + 20) * U * mag


def test_captured_replays():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    rng = np.random.default_rng(5)
    T, k, E, D = 300, 8, 32, 256
    p, dout, y, w = _case(rng, T, k, E, D, BF16, BF16, drop=3)
    amax = torch.zeros(1, device="cuda")

    def step():
        return ops.moe_unpermute_bwd(dout, y, p["dest"], p["offsets"], k, topk_w=w, amax_out=amax)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for _ in range(3):
        dout.copy_(torch.randn_like(dout))
        want, a = step(), amax.clone()
        for t in (*out, amax):
            t.fill_(5)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]) and torch.equal(amax, a)


@pytest.mark.parametrize("T,k,E,D,drop", [(2500, 8, 16, 2048, 5), (9000, 2, 8, 64, 3), (2050, 10, 24, 1544, 4)])
def test_workgroups_with_several_tokens(T, k, E, D, drop):
    """With the maximum wanted 2048 workgroups walk the tokens, four waves of
    one token (D > 1536) sharing their sums through LDS again and again."""
    test_unpermute_bwd_parity(T, k, E, D, drop, (BF16, BF16, BF16))
