"""GPU parity of layer norm and RMS norm with their gradients against the fp64
oracle: every kernel by the row's length, lengths that vectors do not divide,
unaligned pointers, dtypes, absent weights, rows where it can go wrong, and the
same bits on every run, on a second stream and in replayed graphs."""

import numpy as np
import pytest
import torch

from _helpers import gpu, require_gpu, to_gpu, to_np
from oracle import norm

pytestmark = gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: U, BF16: 2.0 ** -8}


def _chain(D):
    """Additions behind one another in a row's sum: a thread's elements (at most 64), 6 steps across the
    wave, then up to 16 waves."""
    return 64 + 6 + 16


def _data(seed, T, D, dtype, mean=0.5):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, D)) * np.exp(rng.uniform(-1, 1, D)) + mean
    return to_gpu(x.astype(np.float32), dtype), rng


def _weights(rng, D, n, dtype):
    w = to_gpu((1 + 0.2 * rng.standard_normal(D)).astype(np.float32), dtype) if n > 0 else None
    b = to_gpu(rng.standard_normal(D).astype(np.float32), dtype) if n > 1 else None
    return w, b


def _f64(t):
    return None if t is None else to_np(t).astype(np.float64)


def _check_forward(x, w, b, eps, kind, r, out_dtype):
    xn, D = _f64(x), x.shape[1]
    y, mean, rstd = norm.forward(xn, _f64(w), _f64(b), eps, kind == 1)
    n = _chain(D)
    # the mean: n roundings of sums no larger than mean |x|, and 1 / D's
    dm = np.zeros(len(xn)) if kind == 1 else (n + 3) * U * np.abs(xn).mean(1)
    v = np.abs(xn - mean[:, None])
    # r: half the relative error of the mean square (the differences are off by dm and one rounding), and
    # the roundings of 1 / D, the product, the sum with eps, the root and the quotient
    ms = (v * v).mean(1)
    er = 0.5 * ((n + 4) * U + (2 * v.mean(1) * dm + dm * dm) / (ms + eps)) + 6 * U
    assert (np.abs(_f64(r["rstd"]) - rstd) <= 1.01 * er * rstd).all()
    if kind == 0:
        assert (np.abs(_f64(r["mean"]) - mean) <= dm + U * np.abs(mean)).all()
    else:
        assert r["mean"] is None
    wa = np.ones(D) if w is None else np.abs(_f64(w))
    core = v * rstd[:, None] * wa
    tol = 1.01 * (core * (er[:, None] + 4 * U) + dm[:, None] * rstd[:, None] * wa) + U * np.abs(y)
    tol = tol + HALF[out_dtype] * (np.abs(y) + tol) + 1e-38
    got = _f64(r["y"])
    assert (np.abs(got - y) <= tol).all(), float((np.abs(got - y) / tol).max())


LENGTHS = [1, 2, 7, 8, 31, 64, 65, 128, 129, 500, 512, 513, 520, 1000, 1024, 1025, 1536, 2040, 2047, 2048, 2049, 2056,
           2557, 4096, 4097, 6000, 8192, 8200, 12345, 16383, 16384]


@pytest.mark.parametrize("D", LENGTHS)
def test_forward_by_length(D):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    for i, (dtype, out, wd, kind, n) in enumerate([(BF16, BF16, F32, 0, 2), (F32, F32, F32, 1, 1), (BF16, F32, BF16, 1, 2),
                                                   (F32, BF16, BF16, 0, 1), (F32, F32, F32, 0, 0)]):
        x, rng = _data(D + i, 7, D, dtype)
        w, b = _weights(rng, D, n, wd)
        r = ops.layer_norm(x, w, b, eps=1e-5, kind=kind, out_dtype=out)
        assert r["y"].dtype == out
        _check_forward(x, w, b, 1e-5, kind, r, out)


@pytest.mark.parametrize("D", [500, 512, 1024, 2047, 2048, 4096, 8192, 16383, 16384])
@pytest.mark.parametrize("power", [10, 16, 20])
def test_forward_of_a_large_mean(D, power):
    """The rounding of the mean's sum leaves no trace: elements of mean 2^power and deviation 1 (fp32 holds them
    to 2^(power - 23)).  The differences d from the first mean are off by nothing (it is off by less than 2^(power -
    15), so an element and it lie within a factor of 2 of each other) or by half a step of d; their sums by a chain
    of roundings; and the mean of d, which the second sum takes out, is off by that of the second sum alone."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    rng = np.random.default_rng(D + power)
    x = to_gpu((2.0 ** power + rng.standard_normal((33, D))).astype(np.float32), F32)
    x[3] = 2.0 ** power + 0.125 if power < 20 else 2.0 ** power + 1  # a row without deviation
    x[4] = -x[4]
    w, b = _weights(rng, D, 2, F32)
    xn = _f64(x)
    y, mean, rstd = norm.forward(xn, _f64(w), _f64(b), 1e-5, False)
    r = ops.layer_norm(x, w, b, eps=1e-5)
    n = _chain(D)
    # the first mean's error, and what its correction leaves
    dm = (n + 3) * U * np.abs(xn).mean(1)
    v = np.abs(xn - mean[:, None])
    dc = (n + 3) * U * (v.mean(1) + dm)
    # the mean square of d, (n + 4) roundings of something as large as it, less the square of d's mean
    ms, big = (v * v).mean(1), ((v + dm[:, None]) ** 2).mean(1)
    er = 0.5 * ((n + 8) * U * big + 2 * dm * dc + dc * dc) / (ms + 1e-5) + 6 * U
    live = np.arange(33) != 3
    assert er[live].max() < 0.002
    assert (np.abs(_f64(r["rstd"]) - rstd) <= 1.01 * er * rstd)[live].all()
    assert (np.abs(_f64(r["mean"]) - mean) <= dc + U * np.abs(mean))[live].all()
    wa = np.abs(_f64(w))
    tol = 1.01 * ((v + dm[:, None]) * rstd[:, None] * wa * (er[:, None] + 5 * U) + dc[:, None] * rstd[:, None] * wa)
    tol = tol + U * 2 * (np.abs(y) + tol) + 1e-38
    assert (np.abs(_f64(r["y"]) - y) <= tol)[live].all()
    # without deviation: the variance is at most what the sums' roundings make of dm^2
    assert np.isfinite(_f64(r["y"])[3]).all() and (np.abs(_f64(r["mean"])[3] - xn[3, 0]) <= dc[3] + U * xn[3, 0])
    assert (np.abs(_f64(r["y"])[3] - _f64(b)) <= 1.01 * dc[3] / np.sqrt(1e-5) * wa + U * 2 * np.abs(_f64(b)) + 1e-6).all()


def _check_backward(dy, x, w, mean, rstd, kind, r, blocks, groups):
    T, D = x.shape
    want = norm.backward(_f64(dy), _f64(x), _f64(w), _f64(mean), _f64(rstd), kind == 1)
    dyn, rn = np.abs(_f64(dy)), _f64(rstd)[:, None]
    xn = _f64(x) - (0 if kind == 1 else _f64(mean)[:, None])
    h = np.abs(xn) * rn
    eh = 2.01 * U * h   # the difference and the product, each rounded once (x, mean and r are given)
    wa = np.ones(D) if w is None else np.abs(_f64(w))
    g = dyn * wa
    n = _chain(D) + 4
    if r["dx"] is not None:
        egh = (g * h).mean(1, keepdims=True) * ((n + 4) * U)
        eg = 0 if kind == 1 else g.mean(1, keepdims=True) * ((n + 2) * U)
        gh = np.abs((_f64(dy) * (1 if w is None else _f64(w)) * xn * rn).mean(1, keepdims=True))
        gm = 0 if kind == 1 else np.abs((_f64(dy) * (1 if w is None else _f64(w))).mean(1, keepdims=True))
        tol = rn * (5 * U * (g + gm + h * (gh + egh)) + eg + h * egh + eh * (gh + egh)) * 1.01
        tol = tol + HALF[r["dx"].dtype] * (np.abs(want[0]) + tol) + 1e-37
        assert (np.abs(_f64(r["dx"]) - want[0]) <= tol).all(), float((np.abs(_f64(r["dx"]) - want[0]) / tol).max())
    if T <= 384:
        # one launch: a thread's rows of a column (every 16th), then five steps across lanes at most
        chain = -(-T // 16) + 5 + 1
    else:
        # a thread's rows, the groups of its workgroup, then at most 256 workgroups' sums: eight by a thread,
        # and five steps across 32 lanes
        chain = -(-T // (blocks * groups)) + groups + 8 + 5 + 1
    for got, ref, terms, e in ((r["dw"], want[1], dyn * h, (dyn * eh).sum(0)), (r["db"], want[2], dyn, 0)):
        if got is not None:
            assert got.dtype == F32
            tol = 1.01 * ((chain + 1) * U * terms.sum(0) + e) + 1e-37
            assert (np.abs(_f64(got) - ref) <= tol).all(), float((np.abs(_f64(got) - ref) / tol).max())


def _grid(T, D, vec):
    """Workgroups, and the rows that one takes at a time."""
    if vec:
        groups = 8 if D <= 1024 else 4 if D <= 2048 else 2 if D <= 4096 else 1
    else:
        groups = 8 if D <= 512 else 2 if D <= 4096 else 1
    return min(-(-T // groups), 256), groups


@pytest.mark.parametrize("D", LENGTHS)
def test_backward_by_length(D):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    for i, (xd, dd, od, wd, kind, n) in enumerate([(BF16, F32, F32, F32, 0, 2), (F32, F32, F32, F32, 1, 1),
                                                   (BF16, BF16, BF16, BF16, 0, 1), (F32, BF16, BF16, F32, 1, 2)]):
        T = (9, 5, 1, 13)[i]
        x, rng = _data(D + 100 + i, T, D, xd)
        dy = to_gpu(rng.standard_normal((T, D)).astype(np.float32), dd)
        w, b = _weights(rng, D, n, wd)
        f = ops.layer_norm(x, w, b, kind=kind)
        r = ops.layer_norm_bwd(dy, x, w, f["mean"], f["rstd"], kind=kind, dx_dtype=od, want_db=b is not None)
        assert r["dx"].dtype == od and (r["db"] is None) == (b is None)
        _check_backward(dy, x, w, f["mean"], f["rstd"], kind, r, *_grid(T, D, D % 8 == 0))


@pytest.mark.parametrize("D", [520, 1001, 2048, 12000])
@pytest.mark.parametrize("xd,dd,od,wd,kind", [(F32, F32, F32, F32, 1), (F32, BF16, BF16, BF16, 0), (BF16, BF16, F32, F32, 1),
                                              (BF16, F32, BF16, BF16, 1)])
def test_backward_in_two_launches_by_type(xd, dd, od, wd, kind, D):
    """Rows of either type, more than go in one launch, with and without means."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    T = 611
    x, rng = _data(D + kind, T, D, xd)
    dy = to_gpu(rng.standard_normal((T, D)).astype(np.float32), dd)
    w, b = _weights(rng, D, 2, wd)
    f = ops.layer_norm(x, w, b, kind=kind, want_stats=True)
    mean = f["mean"] if kind == 0 else None
    r = ops.layer_norm_bwd(dy, x, w, mean, f["rstd"], kind=kind, dx_dtype=od, want_db=True)
    assert r["dx"].dtype == od
    _check_backward(dy, x, w, mean, f["rstd"], kind, r, *_grid(T, D, D % 8 == 0))
    sums = ops.layer_norm_bwd(dy, x, w, mean, f["rstd"], kind=kind, want_dx=False, want_db=True)
    assert sums["dx"] is None and torch.equal(sums["dw"], r["dw"]) and torch.equal(sums["db"], r["db"])


@pytest.mark.parametrize("T,D", [(1, 2048), (3, 256), (1023, 256), (1024, 2048), (1025, 512), (5000, 64), (333, 2557),
                                 (257, 4096), (700, 5000), (300, 9001), (384, 1000), (385, 1000), (600, 2557), (400, 16384),
                                 (390, 9001), (2100, 8192), (3000, 2048), (513, 33), (2500, 1536)])
def test_backward_by_rows(T, D):
    """Few rows in one launch and more in two: fewer than workgroups take, as many, and groups that go round."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    x, rng = _data(T + D, T, D, BF16)
    dy = to_gpu(rng.standard_normal((T, D)).astype(np.float32) * 1e-3, F32)
    w, b = _weights(rng, D, 2, F32)
    f = ops.layer_norm(x, w, b)
    _check_forward(x, w, b, 1e-5, 0, f, BF16)
    r = ops.layer_norm_bwd(dy, x, w, f["mean"], f["rstd"], want_db=True)
    _check_backward(dy, x, w, f["mean"], f["rstd"], 0, r, *_grid(T, D, D % 8 == 0))
    again = ops.layer_norm_bwd(dy, x, w, f["mean"], f["rstd"], want_db=True)
    for n in ("dx", "dw", "db"):
        assert torch.equal(r[n], again[n])


def test_pointers_that_are_not_16_byte_aligned():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    T, D = 6, 1024
    for dtype in (BF16, F32):
        x0, rng = _data(3, T, D, dtype)
        dy0 = to_gpu(rng.standard_normal((T, D)).astype(np.float32), F32)
        w0, b0 = _weights(rng, D, 2, F32)

        def off(t):  # the same values one element further
            s = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view(t.shape)
            s.copy_(t)
            return s

        for which in range(5):
            x, dy, w, b = (off(t) if i == which else t for i, t in enumerate((x0, dy0, w0, b0)))
            out = off(x0) if which == 4 else None
            f = ops.layer_norm(x, w, b, y=out)
            _check_forward(x, w, b, 1e-5, 0, f, dtype)
            r = ops.layer_norm_bwd(dy, x, w, f["mean"], f["rstd"], want_db=True, dx=off(x0) if which == 4 else None)
            _check_backward(dy, x, w, f["mean"], f["rstd"], 0, r, *_grid(T, D, which == 3))


def test_rows_where_it_can_go_wrong():
    """A mean far above the deviations, constant and zero rows, huge and tiny values; rows with NaN or an
    infinity are NaN and touch no other row."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    T, D = 8, 768
    x, rng = _data(5, T, D, F32)
    x[0] += 3000
    x[1] = 2.5
    x[2] = 0
    x[3] *= 1e15
    x[4] *= 1e-15
    w, b = _weights(rng, D, 2, F32)
    for kind in (0, 1):
        r = ops.layer_norm(x, w, b, eps=1e-6, kind=kind)
        _check_forward(x, w, b, 1e-6, kind, r, F32)
    assert torch.equal(ops.layer_norm(x, w, b)["y"][2], b)  # a zero row gives the bias
    bad = x.clone()
    bad[5, 7] = float("nan")
    bad[6, 700] = float("inf")
    good, got = ops.layer_norm(x, w, b)["y"], ops.layer_norm(bad, w, b)["y"]
    rows = torch.tensor([0, 1, 2, 3, 4, 7], device="cuda")
    assert torch.equal(good[rows], got[rows]) and got[5].isnan().all() and got[6].isnan().all()
    # a constant row without eps: 0 / 0 in neither direction is hidden
    one = ops.layer_norm(x[2:3].contiguous(), eps=0.0)
    assert one["rstd"].isinf().all() and one["y"].isnan().all()


def test_parts_of_the_gradient_and_no_rows():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    for T in (50, 500):
        x, rng = _data(6, T, 300, BF16)
        dy = to_gpu(rng.standard_normal((T, 300)).astype(np.float32), F32)
        w, b = _weights(rng, 300, 2, F32)
        f = ops.layer_norm(x, w, b)
        args = (dy, x, w, f["mean"], f["rstd"])
        whole = ops.layer_norm_bwd(*args, want_db=True)
        for kw, names in ((dict(want_dw=False), ["dx"]), (dict(want_dx=False), ["dw"]),
                          (dict(want_dx=False, want_dw=False, want_db=True), ["db"])):
            part = ops.layer_norm_bwd(*args, **kw)
            assert [n for n in ("dx", "dw", "db") if part[n] is not None] == names
            for n in names:
                assert torch.equal(part[n], whole[n])
    r = ops.layer_norm(x, w, b, want_stats=False)
    assert r["mean"] is None and r["rstd"] is None and torch.equal(r["y"], f["y"])
    e = x[:0]
    f = ops.layer_norm(e, w, b)
    assert f["y"].shape == (0, 300)
    dw = torch.full((300,), 7.0, device="cuda")
    r = ops.layer_norm_bwd(dy[:0], e, w, f["mean"], f["rstd"], dw=dw, want_db=True)
    assert (dw == 0).all() and (r["db"] == 0).all() and r["dx"].shape == (0, 300)


def test_outputs_stay_inside_their_tensors():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    for T, D in ((5, 777), (9, 2048), (2, 5000), (400, 777), (401, 2048)):
        x, rng = _data(T, T, D, BF16)
        dy = to_gpu(rng.standard_normal((T, D)).astype(np.float32), BF16)
        w, b = _weights(rng, D, 2, F32)
        flat = [torch.full((n + 64,), 3.0, dtype=dt, device="cuda") for n, dt in
                ((T * D, BF16), (T, F32), (T, F32), (T * D, BF16), (D, F32), (D, F32))]
        y, mean, rstd, dx, dw, db = (t[:n].view(s) for t, n, s in zip(flat, (T * D, T, T, T * D, D, D),
                                                                      ((T, D), (T,), (T,), (T, D), (D,), (D,))))
        ops.layer_norm(x, w, b, y=y, mean=mean, rstd=rstd)
        ops.layer_norm_bwd(dy, x, w, mean, rstd, dx=dx, dw=dw, db=db)
        for t in flat:
            assert (t[-64:] == 3).all()


@pytest.mark.parametrize("T", [300, 900])
def test_streams_and_graphs(T):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    D = 2048
    x, rng = _data(8, T, D, BF16)
    dy = to_gpu(rng.standard_normal((T, D)).astype(np.float32), F32)
    w, b = _weights(rng, D, 2, F32)

    def step():
        f = ops.layer_norm(x, w, b)
        r = ops.layer_norm_bwd(dy, x, w, f["mean"], f["rstd"], want_db=True)
        return [f["y"], f["mean"], f["rstd"], r["dx"], r["dw"], r["db"]]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    graphs = []
    for _ in range(2):  # two graphs, each with workspaces of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step()
        graphs.append((g, outs))
    for seed in range(3):
        nx, r2 = _data(20 + seed, T, D, BF16)
        x.copy_(nx)
        want = step()
        for g, outs in graphs:
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(want, outs)), seed
