"""GPU parity of the MXFP4 path: the quantization fused into the permutation
(bit for bit against mx_quantize and the oracle), the grouped MXFP4 x MXFP4
GEMM against the fp64 oracle (every tile configuration; empty, one-row and
ragged experts, odd tiles of N and K, more experts than the kernel keeps
offsets for), the SiLU-gate epilogue and its quantized H bit for bit against
the separate steps, and the layer's forward."""

import numpy as np
import pytest
import torch

import workloads
from _helpers import gpu, require_gpu, to_gpu, to_np
from oracle import gemm, moe, mx
from oracle.layer import bf16_round

pytestmark = gpu

E2M1 = 1
U = 2.0 ** -24
BF16 = torch.bfloat16


def _operands(rng, M, N, K, E, spread=1.0):
    a = (rng.standard_normal((M, K)) * np.exp(rng.uniform(-spread, spread, (M, 1)))).astype(np.float32)
    b = (rng.standard_normal((E * N, K)) * 0.05).astype(np.float32)
    aq, as_ = mx.quantize(a, "e2m1")
    bq, bs = mx.quantize(b, "e2m1")
    return aq, as_, bq.reshape(E, N, K // 2), bs.reshape(E, N, K // 32)


def _gpu(*arrays):
    return [to_gpu(a, torch.uint8) for a in arrays]


def _off(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def _check(got, ref, ab, K, bf16):
    # one MFMA adds 64 exact products to the accumulator: a rounding (or
    # truncation) of its size for each, K / 64 of them, and the alignment of
    # the 64 products among themselves
    tol = 2 * (K / 64 + 64) * U * ab + 1e-37
    if bf16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    err = np.abs(np.asarray(got, np.float64) - ref)
    assert (err <= tol).all(), "%d of %d out of bounds, worst %.3g of it" % (
        (err > tol).sum(), err.size, float((err / tol).max()))


COUNTS = [
    ([0, 1, 300, 0, 37, 256, 511], 96, 256),      # 192-row tiles: empty, one-row, tails; N not a tile multiple
    ([0, 1, 600, 0, 37, 512, 511], 96, 256),      # 256-row tiles: the same
    ([300, 0, 400], 288, 128),                    # and a single half stage
    ([700], 512, 384),                            # one expert (dense), K % 256 == 128
    ([300, 0, 129], 288, 128),                    # a single half stage
    ([64, 65, 0, 1, 33, 90], 256, 640),           # 64-row tiles
    ([100, 192, 0, 193, 31, 160], 544, 384),
    ([3] * 40 + [257, 0], 1056, 512),             # small tiles: many small experts and one large
    ([1], 32, 2048),                              # one row
    ([0, 2, 0, 0, 5, 32, 31, 1], 544, 768),
]


@pytest.mark.parametrize("counts,N,K", COUNTS)
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_gemm_parity(counts, N, K, out_dtype):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    rng = np.random.default_rng(sum(counts) + N + K)
    off = _off(counts)
    R = int(off[-1])
    M = R + 5                                     # rows behind the last expert stay as they are
    ops_np = _operands(rng, M, N, K, len(counts))
    c = torch.full((M, N), 7.0, dtype=out_dtype, device="cuda")
    ops.grouped_gemm_mxfp4(*_gpu(*ops_np), to_gpu(off, torch.int32), out=c)
    torch.cuda.synchronize()
    ref, ab = gemm.grouped_gemm_w4a8(*ops_np, off, a_elem="e2m1")
    got = to_np(c)
    _check(got[:R], ref[:R], ab[:R], K, out_dtype == torch.bfloat16)
    assert (got[R:] == 7.0).all()


def test_gemm_many_experts_and_extreme_scales():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    rng = np.random.default_rng(8)
    E, N, K = 1100, 32, 128                       # offsets stay in global memory
    counts = rng.integers(0, 4, E)
    off = _off(counts)
    M = int(off[-1])
    aq, as_, bq, bs = _operands(rng, M, N, K, E)
    as_[::7] = 1                                  # 2^-126
    bs[3::5] = 200                                # 2^73
    ref, ab = gemm.grouped_gemm_w4a8(aq, as_, bq, bs, off, a_elem="e2m1")
    got = to_np(ops.grouped_gemm_mxfp4(*_gpu(aq, as_, bq, bs), to_gpu(off, torch.int32)))
    # products below fp32's normal range may be flushed
    fine = ab > 2.0 ** -100
    _check(np.where(fine, got, 0), np.where(fine, ref, 0), ab, K, False)


def test_gemm_empty_and_zero_width():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    u8 = dict(dtype=torch.uint8, device="cuda")
    off0 = torch.zeros(4, dtype=torch.int32, device="cuda")
    z = torch.zeros
    assert ops.grouped_gemm_mxfp4(z(0, 64, **u8), z(0, 4, **u8), z(3, 32, 64, **u8), z(3, 32, 4, **u8),
                                  off0).shape == (0, 32)
    c = torch.full((5, 32), 3.0, device="cuda")   # rows, but no expert has any
    ops.grouped_gemm_mxfp4(z(5, 64, **u8), z(5, 4, **u8), z(3, 32, 64, **u8), z(3, 32, 4, **u8), off0, out=c)
    torch.cuda.synchronize()
    assert (c == 3.0).all()
    off = torch.tensor([0, 5, 5, 5], dtype=torch.int32, device="cuda")
    ops.grouped_gemm_mxfp4(z(5, 0, **u8), z(5, 0, **u8), z(3, 32, 0, **u8), z(3, 32, 0, **u8), off, out=c)
    torch.cuda.synchronize()
    assert (c == 0).all()


@pytest.mark.parametrize("counts,F,K", [([0, 5, 260, 1, 513, 64], 256, 384), ([700, 33], 384, 512),
                                        ([1, 0, 2, 30, 7], 128, 256), ([70, 0, 95, 60], 128, 640),
                                        ([150, 193, 40], 256, 384), ([0, 5, 560, 1, 813, 64], 256, 384),
                                        ([4], 768, 2048)])
def test_silu_epilogue_equals_the_separate_steps(counts, F, K):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    rng = np.random.default_rng(sum(counts) + F + K)
    E, off = len(counts), _off(counts)
    R = int(off[-1])
    M = R + 3
    g = _gpu(*_operands(rng, M, 2 * F, K, E, spread=2.0))
    offs = to_gpu(off, torch.int32)
    y1 = ops.grouped_gemm_mxfp4(*g, offs, out_dtype=torch.bfloat16)
    h, amax = ops.silu_gate_fwd(y1[:R].contiguous())
    rq, rs = ops.mx_quantize(h, E2M1)
    got_amax = torch.full((1,), 1e9, device="cuda")
    r = ops.grouped_gemm_mxfp4_silu_gate(*g, offs, amax_out=got_amax, want_q=True)
    plain = ops.grouped_gemm_mxfp4_silu_gate(*g, offs)
    only = ops.grouped_gemm_mxfp4_silu_gate(*g, offs, want_y1=False, want_h=False, want_q=True)
    torch.cuda.synchronize()
    assert only["y1"] is None and only["h"] is None and plain["q_h"] is None
    for x in (r, plain):
        assert torch.equal(x["y1"][:R].view(torch.int16), y1[:R].view(torch.int16))
        assert torch.equal(x["h"][:R].view(torch.int16), h.view(torch.int16))
    for x in (r, only):
        assert torch.equal(x["q_h"][:R], rq) and torch.equal(x["s_h"][:R], rs)
    assert torch.equal(got_amax, amax)


def test_silu_epilogue_leaves_rows_behind():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    rng = np.random.default_rng(1)
    for counts in ([40, 3], [300, 130]):
        off = _off(counts)
        R = int(off[-1])
        M, F, K = R + 9, 128, 128
        g = _gpu(*_operands(rng, M, 2 * F, K, 2))
        y1 = torch.full((M, 2 * F), 7.0, dtype=torch.bfloat16, device="cuda")
        h = torch.full((M, F), 7.0, dtype=torch.bfloat16, device="cuda")
        q_h, s_h = (torch.full((M, n), 77, dtype=torch.uint8, device="cuda") for n in (F // 2, F // 32))
        ops.grouped_gemm_mxfp4_silu_gate(*g, to_gpu(off, torch.int32), y1=y1, h=h, q_h=q_h, s_h=s_h)
        torch.cuda.synchronize()
        assert (y1[R:] == 7).all() and (h[R:] == 7).all() and (q_h[R:] == 77).all() and (s_h[R:] == 77).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,E,D", [(500, 8, 24, 512), (333, 3, 40, 320), (1, 1, 1, 32), (7, 64, 64, 96),
                                     (2000, 2, 300, 128)])
def test_permute_mxfp4_equals_quantize_then_gather(dtype, T, k, E, D):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    rng = np.random.default_rng(T + k + D)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    bad = 0
    if T > 100:
        ids[7, 1], ids[99, 0], bad = E + 3, -1, 2
    x_np = (rng.standard_normal((T, D)) * np.exp(rng.uniform(-6, 6, (T, 1)))).astype(np.float32)
    x_np[T // 2, :32] = 0.0
    got = ops.moe_permute_mxfp4(to_gpu(ids, torch.int32), E, to_gpu(x_np, dtype))
    pm = ops.moe_permute(to_gpu(ids, torch.int32), E)
    torch.cuda.synchronize()
    for name in ("offsets", "dest", "src"):
        assert torch.equal(got[name], pm[name]), name
    n = int(to_np(got["offsets"])[-1])
    assert n == T * k - bad
    assert (to_np(got["q"])[n:] == 0).all() and (to_np(got["scales"])[n:] == 0).all()
    xv = x_np if dtype == torch.float32 else bf16_round(x_np)
    rq, rs = mx.quantize(xv[to_np(got["src"])[:n] // k], "e2m1")
    np.testing.assert_array_equal(to_np(got["q"])[:n], rq)
    np.testing.assert_array_equal(to_np(got["scales"])[:n], rs)


@pytest.mark.parametrize("T,k,E,D,F,drop", [(1, 2, 8, 128, 128, 0), (37, 4, 16, 256, 128, 3), (900, 8, 16, 384, 256, 5)])
def test_forward_stage_by_stage(T, k, E, D, F, drop):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import moe_layer
    d = workloads.moe(T, 1.1, 0.01, 16.0, seed=T, E=E, k=k, D=D, F=F, name="mxfp4")
    ids = d["topk_ids"].copy()
    ids.reshape(-1)[:drop] = -1
    wq = [moe_layer.quantize_expert_weights_mx(to_gpu(d[n], torch.bfloat16)) for n in ("w_gu", "w_dn")]
    buf = moe_layer.BuffersMXFP4(T, k, E, D, F, torch.device("cuda"), backward=True)
    x, gi, tw = to_gpu(d["x"], torch.bfloat16), to_gpu(ids, torch.int32), to_gpu(d["topk_w"], torch.float32)
    meta = moe_layer.forward_mxfp4(x, gi, tw, *wq, buf)
    out0 = buf.out.clone()
    meta = moe_layer.forward_mxfp4(x, gi, tw, *wq, buf, keep=True)
    torch.cuda.synchronize()
    assert torch.equal(buf.out, out0)
    off, dest, src = (to_np(meta[n]) for n in ("offsets", "dest", "src"))
    n = int(off[-1])
    assert n == T * k - drop and (dest[:drop] == -1).all()
    aq, as_ = mx.quantize(d["x"][src[:n] // k], "e2m1")
    np.testing.assert_array_equal(to_np(buf.a1_q)[:n], aq)
    np.testing.assert_array_equal(to_np(buf.a1_s)[:n], as_)
    ref, ab = gemm.grouped_gemm_w4a8(aq, as_, to_np(wq[0]["q"]), to_np(wq[0]["s"]), off, a_elem="e2m1")
    y1 = to_np(buf.y1)[:n]
    _check(y1, ref, ab, D, True)
    h = to_np(buf.h)[:n]
    hr = moe.silu_gate_fwd(y1)
    assert (np.abs(h - hr) <= 2.0 ** -8 * np.abs(hr) + 2.0 ** -20 * np.abs(hr) + 1e-37).all()
    hq, hs = mx.quantize(h, "e2m1")
    np.testing.assert_array_equal(to_np(buf.a2_q)[:n], hq)
    np.testing.assert_array_equal(to_np(buf.a2_s)[:n], hs)
    ref, ab = gemm.grouped_gemm_w4a8(hq, hs, to_np(wq[1]["q"]), to_np(wq[1]["s"]), off, a_elem="e2m1")
    y2 = to_np(buf.y2)
    _check(y2[:n], ref, ab, F, True)
    w = np.where(dest.reshape(T, k) >= 0, d["topk_w"], 0)    # dropped assignments add nothing
    y2[n:] = 0
    dest = np.maximum(dest, 0)
    want = moe.unpermute(y2, dest, k, w)
    bound = moe.unpermute_absbound(y2, dest, k, w)
    assert (np.abs(to_np(buf.out) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -16 * bound + 1e-30).all()


def test_forward_without_tokens():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import moe_layer
    k, E, D, F = 2, 8, 256, 128
    dev = torch.device("cuda")
    gu = moe_layer.quantize_expert_weights_mx(torch.ones(E, 2 * F, D, dtype=torch.bfloat16, device=dev))
    dn = moe_layer.quantize_expert_weights_mx(torch.ones(E, D, F, dtype=torch.bfloat16, device=dev))
    buf = moe_layer.BuffersMXFP4(0, k, E, D, F, dev)
    moe_layer.forward_mxfp4(torch.zeros(0, D, dtype=torch.bfloat16, device=dev),
                            torch.zeros(0, k, dtype=torch.int32, device=dev), torch.zeros(0, k, device=dev), gu, dn, buf)
    torch.cuda.synchronize()
    assert buf.out.shape == (0, D)


def test_full_size_sampled():
    """The 8192-token gate+up product (65536 rows, 128 experts, 2F = 1536, K =
    2048), rows of four experts against the oracle."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import moe_layer, ops
    d = workloads.moe_8k_update()
    E, k = d["E"], d["k"]
    wq = moe_layer.quantize_expert_weights_mx(to_gpu(d["w_gu"], torch.bfloat16))
    p = ops.moe_permute_mxfp4(to_gpu(d["topk_ids"], torch.int32), E, to_gpu(d["x"], torch.bfloat16))
    y1 = ops.grouped_gemm_mxfp4(p["q"], p["scales"], wq["q"], wq["s"], p["offsets"])
    torch.cuda.synchronize()
    off, _, src = moe.permute_metadata(d["topk_ids"], E)
    rng = np.random.default_rng(5)
    rows = np.unique(np.concatenate([[off[e], off[e + 1] - 1] + rng.integers(off[e], off[e + 1], 6).tolist()
                                     for e in (0, 40, 77, E - 1)]).astype(np.int64))
    aq, as_ = mx.quantize(d["x"][src[rows] // k], "e2m1")
    ref, ab = gemm.grouped_gemm_w4a8(aq, as_, to_np(wq["q"]), to_np(wq["s"]), off, rows=rows, a_elem="e2m1")
    _check(to_np(y1[torch.from_numpy(rows).cuda()]), ref, ab, d["D"], False)


@pytest.mark.parametrize("E,N", [(260, 16384), (600, 8192)])
def test_more_tiles_than_a_workgroup_looks_up_at_once(E, N):
    """16640 and 19200 tiles of 32 x 256, over 64 per workgroup of a 256-CU
    grid, with the offsets in LDS and in global memory; sampled experts."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    g = torch.Generator(device="cuda").manual_seed(E)
    K = 128
    counts = torch.randint(1, 4, (E,), generator=g, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = counts.cumsum(0)
    M = int(off[-1])

    def u8(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.uint8)

    aq, as_, bq, bs = u8(0, 256, M, K // 2), u8(120, 135, M, K // 32), u8(0, 256, E, N, K // 2), u8(120, 135, E, N, K // 32)
    got = to_np(ops.grouped_gemm_mxfp4(aq, as_, bq, bs, off))
    offs = to_np(off)
    for e in [0, 1, E // 3, E // 2, E - 2, E - 1]:
        lo, hi = int(offs[e]), int(offs[e + 1])
        a = mx.dequantize(to_np(aq[lo:hi]), to_np(as_[lo:hi]), "e2m1").astype(np.float64)
        b = mx.dequantize(to_np(bq[e]), to_np(bs[e]), "e2m1").astype(np.float64)
        _check(got[lo:hi], a @ b.T, np.abs(a) @ np.abs(b).T, K, False)


def test_two_streams_and_captured_replays():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import moe_layer
    T, k, E, D, F = 400, 8, 16, 256, 256
    dev = torch.device("cuda")
    runs = []
    for seed in (1, 2):
        d = workloads.moe(T, 1.1, seed=seed, E=E, k=k, D=D, F=F, name="mxfp4")
        wq = [moe_layer.quantize_expert_weights_mx(to_gpu(d[n], torch.bfloat16)) for n in ("w_gu", "w_dn")]
        args = (to_gpu(d["x"], torch.bfloat16), to_gpu(d["topk_ids"], torch.int32), to_gpu(d["topk_w"], torch.float32), *wq)
        buf = moe_layer.BuffersMXFP4(T, k, E, D, F, dev)
        moe_layer.forward_mxfp4(*args, buf)
        torch.cuda.synchronize()
        runs.append((args, buf, buf.out.clone(), torch.cuda.Stream()))
    for _, buf, _, _ in runs:
        buf.out.zero_()
    torch.cuda.synchronize()
    for _ in range(4):
        for args, buf, _, st in runs:
            with torch.cuda.stream(st):
                moe_layer.forward_mxfp4(*args, buf)
    torch.cuda.synchronize()
    for _, buf, want, _ in runs:
        assert torch.equal(buf.out, want)
    args, buf, want, _ = runs[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe_layer.forward_mxfp4(*args, buf)
    for _ in range(3):
        args[0].copy_(torch.randn_like(args[0]))
        moe_layer.forward_mxfp4(*args, buf)
        want = buf.out.clone()
        for t in (buf.out, buf.y2, buf.a1_q, buf.a2_q, buf.a2_s):
            t.fill_(1)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf.out, want)


@pytest.mark.parametrize("K", [256, 384, 640])                # one, two and three stages per tile
@pytest.mark.parametrize("mean", [16, 48, 128, 300])          # each row block of the tile rule
def test_workgroups_with_several_tiles(mean, K):
    """768 to 2500 tiles on 256 CUs: the loads of a next tile run under an
    epilogue and the waits behind it allow for its stores, whichever outputs it
    has.  Every row of every form against products of one expert at a time
    (a tile per workgroup at most) and the separate steps, bit for bit."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    E, F = 96, 1024
    N = 2 * F
    g = torch.Generator(device="cuda").manual_seed(mean * 1000 + K)
    counts = torch.randint(0, 2 * mean, (E,), generator=g, device="cuda")
    counts[3], counts[40] = 0, 1
    offs = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offs[1:] = counts.cumsum(0)
    ends = offs.tolist()
    R = ends[-1]
    M = R + 7
    assert (24 < R / E) == (mean > 16) and (72 < R / E) == (mean > 48) and (176 < R / E) == (mean > 128)

    def u8(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.uint8)

    aq, as_, bq, bs = u8(0, 256, M, K // 2), u8(120, 128, M, K // 32), u8(0, 256, E, N, K // 2), u8(120, 128, E, N, K // 32)
    want = torch.full((M, N), 7.0, device="cuda")
    for e in range(E):
        lo, hi = ends[e], ends[e + 1]
        if hi > lo:
            one = torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")
            want[lo:hi] = ops.grouped_gemm_mxfp4(aq[lo:hi].clone(), as_[lo:hi].clone(), bq[e:e + 1], bs[e:e + 1], one)
    y1 = torch.full((M, N), 7.0, dtype=BF16, device="cuda")
    y1[:R] = want[:R].to(BF16)
    h = torch.full((M, F), 7.0, dtype=BF16, device="cuda")
    h[:R] = ops.silu_gate_fwd(y1[:R].contiguous())[0]
    q, s = (torch.full((M, n), 77, dtype=torch.uint8, device="cuda") for n in (F // 2, F // 32))
    q[:R], s[:R] = ops.mx_quantize(h[:R].contiguous(), E2M1)
    for _ in range(2):
        for dt, ref in ((torch.float32, want), (BF16, y1)):
            c = torch.full((M, N), 7.0, dtype=dt, device="cuda")
            ops.grouped_gemm_mxfp4(aq, as_, bq, bs, offs, out=c)
            assert torch.equal(c, ref), dt
        for keep_y1, keep_h, quant in ((1, 1, 0), (0, 1, 0), (0, 0, 1), (1, 1, 1), (1, 0, 1)):
            out = dict(y1=torch.full_like(y1, 7.0) if keep_y1 else None, h=torch.full_like(h, 7.0) if keep_h else None,
                       q_h=torch.full_like(q, 77) if quant else None, s_h=torch.full_like(s, 77) if quant else None)
            ops.grouped_gemm_mxfp4_silu_gate(aq, as_, bq, bs, offs, want_y1=bool(keep_y1), want_h=bool(keep_h), **out)
            for name, ref in (("y1", y1), ("h", h), ("q_h", q), ("s_h", s)):
                assert out[name] is None or torch.equal(out[name], ref), (name, keep_y1, keep_h, quant)
