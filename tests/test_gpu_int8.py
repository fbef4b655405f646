"""GPU parity of the 8-bit integer path, bit for bit: the row quantizer against
the oracle, its fusion into the permutation, the grouped products against exact
integer sums (every tile configuration; empty, one-row and ragged experts, tails
of N and K, more experts than the kernel keeps offsets for, the largest sums),
the SiLU-gate epilogue with Y1 kept in 8 bits against the separate steps, and the
layer's forward."""

import numpy as np
import pytest
import torch

import workloads
from _helpers import gpu, require_gpu, to_gpu, to_np
from oracle import int8, moe
from oracle.layer import bf16_round

pytestmark = gpu

F32, BF16 = torch.float32, torch.bfloat16


def _bits(t):
    return t.view(torch.int32) if t.dtype == F32 else t


def _same(a, b):
    """Equal bits (NaNs of any kind are one)."""
    if a.dtype in (F32, BF16):
        nan = a.isnan()
        return torch.equal(nan, b.isnan()) and torch.equal(a[~nan].view(torch.int16 if a.dtype == BF16 else torch.int32),
                                                           b[~nan].view(torch.int16 if a.dtype == BF16 else torch.int32))
    return torch.equal(a, b)


def _check_quantize(x):
    from nvfp4_quantized_moe_token_amd import ops
    q, s = ops.int8_quantize(x)
    rq, rs = int8.quantize(to_np(x))
    np.testing.assert_array_equal(q.cpu().numpy(), rq)
    np.testing.assert_array_equal(to_np(s), rs)  # (NaN equals NaN)


@pytest.mark.parametrize("rows,K", [(1, 16), (3, 32), (5, 48), (130, 768), (7, 1024), (9, 1040), (33, 2048), (4, 2064),
                                    (6, 4096), (5, 4112), (3, 9728), (2, 20000), (1, 131072)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize_bit_exact(rows, K, dtype):
    require_gpu()
    rng = np.random.default_rng(rows * K)
    x = rng.standard_normal((rows, K)) * np.exp(rng.uniform(-20, 20, (rows, 1)))
    _check_quantize(to_gpu(x.astype(np.float32), dtype))


def test_quantize_where_it_can_go_wrong():
    require_gpu()
    rng = np.random.default_rng(0)
    x = rng.standard_normal((16, 64)).astype(np.float32)
    x[0] = 0
    x[1] = -0.0
    x[2, 5] = np.inf
    x[3, 5], x[3, 6] = np.nan, np.inf
    x[4, 63] = -np.inf
    x[5] *= np.float32(1e-44)     # subnormal: scales of a few steps
    x[6] *= np.float32(1e-38)
    x[7] *= np.float32(1e38)
    x[8] = np.float32(2.0 ** -149)
    x[9] = np.float32(3.4028235e38)
    x[10] = np.linspace(-127.5, 127.5, 64)  # s near 1: quotients near the borders
    x[10, 0] = 127
    x[11] = np.arange(64) - 31.5
    x[11, 0] = 127                           # s == 1: ties to even
    for dtype in (F32, BF16):
        _check_quantize(to_gpu(x, dtype))
    # many rows whose quotients lie next to a border
    s = rng.uniform(0.5, 2, (400, 1)).astype(np.float32)
    x = ((rng.integers(-126, 126, (400, 256)) + 0.5) * s).astype(np.float32)
    x = np.nextafter(x, x + rng.integers(-1, 2, x.shape).astype(np.float32) * 1e9).astype(np.float32)
    x[:, 0] = 127 * s[:, 0]
    _check_quantize(to_gpu(x, F32))


def test_every_bf16_value():
    require_gpu()
    v = np.arange(65536, dtype=np.uint32)
    x = (v << 16).astype(np.uint32).view(np.float32)
    x = x[np.isfinite(x)]
    x = np.concatenate([x, np.zeros(-len(x) % 16, np.float32)]).reshape(-1, 16)
    _check_quantize(to_gpu(x, BF16))


@pytest.mark.parametrize("T,k,E,D,bad", [(1, 1, 1, 16, 0), (300, 4, 32, 256, 0), (333, 3, 40, 2064, 5), (77, 8, 128, 2048, 3),
                                         (5, 2, 4, 4112, 1), (64, 2, 600, 32, 2)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_permute_quantize(T, k, E, D, bad, dtype):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    rng = np.random.default_rng(T * D)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    if bad:
        ids.reshape(-1)[rng.choice(T * k, bad, replace=False)] = [E, -1, E + 7, -5, 1 << 30][:bad]
    x = to_gpu((rng.standard_normal((T, D)) * 2).astype(np.float32), dtype)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = ops.moe_permute_int8(to_gpu(ids, torch.int32), E, x, status=st)
    ref = ops.moe_permute(to_gpu(ids, torch.int32), E)
    for n in ("offsets", "dest", "src"):
        assert torch.equal(r[n], ref[n]), n
    assert int(st) == (1 if bad else 0)
    q, s = ops.int8_quantize(x)
    src = r["src"].long()
    live = src >= 0
    tok = src.clamp(min=0) // k
    assert torch.equal(r["q"], torch.where(live[:, None], q[tok], torch.zeros_like(q[tok])))
    assert torch.equal(r["scales"], torch.where(live, s[tok], torch.zeros_like(s[tok])))


def test_permute_without_tokens():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    r = ops.moe_permute_int8(torch.zeros(0, 4, dtype=torch.int32, device="cuda"), 9,
                             torch.zeros(0, 64, dtype=BF16, device="cuda"))
    assert (r["offsets"] == 0).all() and r["q"].shape == (0, 64) and r["scales"].shape == (0,)


@pytest.mark.parametrize("bad", [0, 3])
def test_permute_of_rows_without_elements(bad):
    """A row has its scale, 0, however wide it is: the products without a reduction are then zeros."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    T, k, E, N = 37, 2, 5, 64
    rng = np.random.default_rng(bad)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids.reshape(-1)[:bad] = E
    scales = torch.full((T * k,), float("nan"), device="cuda")
    x = torch.zeros(T, 0, dtype=BF16, device="cuda")
    r = ops.moe_permute_int8(to_gpu(ids, torch.int32), E, x, scales=scales)
    assert r["scales"] is scales and (scales == 0).all()
    assert (ops.int8_quantize(x)[1] == 0).all()
    ref = ops.moe_permute(to_gpu(ids, torch.int32), E)
    for n in ("offsets", "dest", "src"):
        assert torch.equal(r[n], ref[n]), n
    out = torch.full((T * k, N), 7.0, device="cuda")
    ops.grouped_gemm_int8(r["q"], scales, torch.zeros(E, N, 0, dtype=torch.int8, device="cuda"),
                          torch.ones(E, N, device="cuda"), r["offsets"], out=out)
    end = T * k - bad
    assert (out[:end] == 0).all() and (out[end:] == 7).all()


def _operands(seed, M, N, K, E, full=False):
    """Codes and scales on the GPU; full: codes of the greatest magnitude."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int32).to(torch.int8)  # noqa: E731
    aq, bq = rnd(M, K), rnd(E, N, K)
    if full:
        aq, bq = torch.where(aq < 0, -128, 127).to(torch.int8), torch.where(bq < 0, -128, 127).to(torch.int8)
        aq[::3], bq[:, ::3] = 127, 127
    a_s = torch.rand(M, generator=g, device="cuda") * 0.1 + 1e-3
    b_s = torch.rand(E, N, generator=g, device="cuda") * 1e-2 + 1e-4
    return aq, a_s, bq, b_s


def _reference(aq, a_s, bq, b_s, off, out_dtype, before):
    """The definition in torch: fp64 products (whole numbers, exact), fp32 roundings; other rows as before."""
    c = before.clone()
    for e in range(bq.shape[0]):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            n = aq[lo:hi].double() @ bq[e].double().t()
            c[lo:hi] = (n.float() * a_s[lo:hi, None] * b_s[e]).to(out_dtype)
    return c


def _off(counts):
    return [0] + np.cumsum(counts).tolist()


COUNTS = [
    ([0, 1, 300, 0, 37, 256, 511], 96, 256),
    ([0, 1, 600, 0, 37, 512, 511], 96, 144),
    ([300, 0, 400], 288, 16),
    ([700], 512, 400),
    ([300, 0, 129], 288, 128),
    ([64, 65, 0, 1, 33, 90], 256, 656),
    ([100, 192, 0, 193, 31, 160], 544, 208),
    ([3] * 40 + [257, 0], 1056, 512),
    ([1] * 7, 32, 1040),
    ([24] * 5, 320, 2048),
    ([2, 0, 1] * 200, 64, 96),                # 600 experts: more than are kept in LDS
    ([40] * 520, 32, 48),
]


@pytest.mark.parametrize("counts,N,K", COUNTS)
@pytest.mark.parametrize("out_dtype", [F32, BF16])
def test_product_bit_exact(counts, N, K, out_dtype):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    off = _off(counts)
    M = off[-1] + 3  # rows behind the last expert: left as they were
    a = _operands(M + N + K, M, N, K, len(counts))
    out = torch.full((M, N), 7.0, dtype=out_dtype, device="cuda")
    want = _reference(*a, off, out_dtype, out)
    got = ops.grouped_gemm_int8(*a, to_gpu(np.array(off), torch.int32), out=out)
    assert got is out and _same(got, want)


@pytest.mark.parametrize("M,N,K", [(40, 32, 131072), (300, 64, 20000), (1, 32, 4096)])
def test_largest_sums(M, N, K):
    """Codes of 127 and -128 throughout: sums up to 128 * 128 * 131072 = 2^31 less 127's share."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    a = _operands(M, M, N, K, 1, full=True)
    off = [0, M]
    want = _reference(*a, off, F32, torch.zeros(M, N, device="cuda"))
    got = ops.grouped_gemm_int8(*a, to_gpu(np.array(off), torch.int32))
    assert _same(got, want)


@pytest.mark.parametrize("M,E", [(1, 1), (40, 1), (100, 3), (300, 3), (400, 3), (600, 3), (900, 3), (1200, 3)])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
def test_the_sum_that_int32_does_not_hold(M, E, out_dtype):
    """A row and a channel of -128 throughout with the longest K: 128 * 128 * 131072 = 2^31; with its neighbours."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    N, K = 64, 131072
    aq = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    bq = torch.full((E, N, K), -128, dtype=torch.int8, device="cuda")
    bq[:, 1::4] = 127        # the lowest sum
    bq[:, 2::4, 77] = -127   # 128 less than 2^31
    aq[1::3, 131071] = 0
    a_s, b_s = torch.rand(M, device="cuda") + 0.5, torch.rand(E, N, device="cuda") + 0.5
    off = [0] + [M * (e + 1) // E for e in range(E)]
    got = ops.grouped_gemm_int8(aq, a_s, bq, b_s, to_gpu(np.array(off), torch.int32), out_dtype=out_dtype)
    assert (got[0, 0::4] > 0).all()
    # whole numbers by hand: the products in fp64 would read 8-byte copies of the codes
    n = torch.full((M, N), 1 << 31, dtype=torch.int64, device="cuda")
    n[:, 1::4] = -127 * 128 * K
    n[:, 2::4] -= 128
    n[1::3] -= torch.where(torch.arange(N, device="cuda") % 4 == 1, -127 * 128, 128 * 128)
    e = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.tensor(off, device="cuda").diff())
    assert _same(got, (n.float() * a_s[:, None] * b_s[e]).to(out_dtype))


@pytest.mark.parametrize("M", [3, 300])
def test_the_sum_that_int32_does_not_hold_in_the_gate(M):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    F, K = 128, 131072
    aq = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    bq = torch.full((1, 2 * F, K), -128, dtype=torch.int8, device="cuda")
    bq[:, 1::2] = 127
    a = aq, torch.full((M,), 2.0 ** -31, device="cuda"), bq, torch.rand(1, 2 * F, device="cuda") + 0.5
    off = to_gpu(np.array([0, M]), torch.int32)
    y1 = ops.grouped_gemm_int8(*a, off, out_dtype=BF16)
    assert (y1[:, 0::2] > 0).all() and (y1[:, 1::2] < 0).all()
    r = ops.grouped_gemm_int8_silu_gate(*a, off, want_ckpt=True)
    assert torch.equal(r["y1"], y1) and torch.equal(r["h"], ops.silu_gate_fwd(y1)[0])
    q, s = ops.mx_quantize(y1, ops.MX_INT8)
    assert torch.equal(r["q_y1"], q) and torch.equal(r["s_y1"], s)


def test_scales_that_are_not_finite_and_no_reduction():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    M, N, K = 200, 96, 160
    aq, a_s, bq, b_s = _operands(5, M, N, K, 2)
    x = torch.randn(M, K, device="cuda")
    x[7, 3], x[150, 100] = float("nan"), float("inf")
    aq, a_s = ops.int8_quantize(x)
    b_s[1, 5] = float("nan")
    a_s[20] = 0
    off = [0, 90, 200]
    want = _reference(aq, a_s, bq, b_s, off, F32, torch.zeros(M, N, device="cuda"))
    got = ops.grouped_gemm_int8(aq, a_s, bq, b_s, to_gpu(np.array(off), torch.int32))
    assert _same(got, want)
    assert got[7].isnan().all() and got[150].isnan().all() and got[90:, 5].isnan().all()
    rest = torch.ones(M, N, dtype=torch.bool, device="cuda")
    rest[7] = rest[150] = False
    rest[90:, 5] = False
    assert got[rest].isfinite().all() and (got[20] == 0).all()
    # K == 0: zeros
    none = ops.grouped_gemm_int8(aq[:, :0].contiguous(), a_s.abs().nan_to_num(1, 1), bq[:, :, :0].contiguous(),
                                 b_s.nan_to_num(1), to_gpu(np.array(off), torch.int32))
    assert (none == 0).all()


def test_scales_at_any_word():
    """a_s and b_s aligned to 4 bytes only."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    for M, N in ((333, 96), (20, 288), (70, 544)):
        off = to_gpu(np.array([0, M // 3, M]), torch.int32)
        aq, a_s, bq, b_s = _operands(M, M, N, 64, 2)
        want = ops.grouped_gemm_int8(aq, a_s, bq, b_s, off)
        for shift in (1, 2, 3):
            pa, pb = torch.empty(M + 4, device="cuda"), torch.empty(2 * N + 4, device="cuda")
            a2, b2 = pa[shift:shift + M], pb[shift:shift + 2 * N].view(2, N)
            a2.copy_(a_s)
            b2.copy_(b_s)
            assert torch.equal(ops.grouped_gemm_int8(aq, a2, bq, b2, off), want)


def test_offsets_that_do_not_fit():
    """Offsets past M_total are taken back to it, as everywhere in the library."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    aq, a_s, bq, b_s = _operands(9, 50, 64, 64, 3)
    out = torch.full((50, 64), 5.0, device="cuda")
    want = _reference(aq, a_s, bq, b_s, [0, 20, 50, 50], F32, out)
    got = ops.grouped_gemm_int8(aq, a_s, bq, b_s, to_gpu(np.array([-4, 20, 70, 90]), torch.int32), out=out)
    assert _same(got, want)


GATE = [([0, 1, 300, 0, 37], 128, 256), ([600, 0, 520, 1], 256, 144), ([5, 0, 1, 40] * 8, 128, 528), ([90, 100, 120], 384, 64),
        ([1], 128, 16), ([64, 33, 50], 256, 400)]


@pytest.mark.parametrize("counts,F,K", GATE)
@pytest.mark.parametrize("form", ["y1", "ckpt", "both", "h"])
def test_silu_gate_epilogue(counts, F, K, form):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    off = _off(counts)
    M = off[-1] + 2
    a = _operands(M + F + K, M, 2 * F, K, len(counts))
    offs = to_gpu(np.array(off), torch.int32)
    y1 = ops.grouped_gemm_int8(*a, offs, out=torch.zeros(M, 2 * F, dtype=BF16, device="cuda"))
    h, amax = ops.silu_gate_fwd(y1)
    q, s = ops.mx_quantize(y1, ops.MX_INT8)
    am = torch.full((1,), 9.0, device="cuda")
    u8 = dict(dtype=torch.uint8, device="cuda")
    q0, s0 = torch.full((M, 2 * F), 77, **u8), torch.full((M, 2 * F // 32), 77, **u8)
    kw = dict(q_y1=q0, s_y1=s0) if form in ("ckpt", "both") else {}
    r = ops.grouped_gemm_int8_silu_gate(*a, offs, want_y1=form in ("y1", "both"), amax_out=am, **kw)
    end = off[-1]
    assert torch.equal(r["h"][:end], h[:end])
    assert torch.equal(am, amax)
    if form in ("y1", "both"):
        assert torch.equal(r["y1"][:end], y1[:end])
    else:
        assert r["y1"] is None
    if kw:
        assert torch.equal(r["q_y1"][:end], q[:end]) and torch.equal(r["s_y1"][:end], s[:end])
        assert (r["q_y1"][end:] == 77).all() and (r["s_y1"][end:] == 77).all()
    else:
        assert r["q_y1"] is None and r["s_y1"] is None


@pytest.mark.parametrize("T,k,E,D,F,zipf", [(300, 4, 32, 256, 128, 1.1), (37, 3, 8, 400, 256, 0.0), (37, 3, 8, 416, 256, 0.0),
                                            (1, 2, 4, 128, 128, 0.0), (700, 2, 5, 2048, 384, 1.6)])
def test_layer_forward(T, k, E, D, F, zipf):
    """Stage by stage against the oracle, each fed with the stage before as stored."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import moe_layer, ops
    d = workloads.moe(T, zipf, 0.01, 16.0, seed=4, E=E, k=k, D=D, F=F, name="int8")
    x, w_gu, w_dn = (to_gpu(d[n], BF16) for n in ("x", "w_gu", "w_dn"))
    ids, tw = to_gpu(d["topk_ids"], torch.int32), to_gpu(d["topk_w"], F32)
    gu, dn = moe_layer.quantize_expert_weights_int8(w_gu), moe_layer.quantize_expert_weights_int8(w_dn)
    buf = moe_layer.BuffersInt8(T, k, E, D, F, x.device, backward=True)
    if D % 32:  # a product's output rows are 32 columns wide or a multiple
        with pytest.raises(ops.NVFP4MoEError, match="shape"):
            moe_layer.forward_int8(x, ids, tw, gu, dn, buf, keep=True)
        return
    meta = moe_layer.forward_int8(x, ids, tw, gu, dn, buf, keep=True)
    off, dest, src = moe.permute_metadata(d["topk_ids"], E)
    np.testing.assert_array_equal(to_np(meta["offsets"]), off)
    np.testing.assert_array_equal(to_np(meta["dest"]), dest)
    rq, rs = int8.quantize(d["x"])
    np.testing.assert_array_equal(buf.a1_q.cpu().numpy(), rq[src // k])
    np.testing.assert_array_equal(to_np(buf.a1_s), rs[src // k])
    wq, ws = int8.quantize(d["w_gu"].reshape(-1, D))
    np.testing.assert_array_equal(gu["q"].cpu().numpy().reshape(-1, D), wq)
    y1 = int8.grouped_gemm(rq[src // k], rs[src // k], wq.reshape(E, 2 * F, D), ws.reshape(E, 2 * F), off)
    np.testing.assert_array_equal(to_np(buf.y1), bf16_round(y1))
    h = moe.silu_gate_fwd(to_np(buf.y1))
    assert (np.abs(to_np(buf.h) - h) <= 2.0 ** -8 * np.abs(h) * 1.001 + 2.0 ** -21 * np.abs(h) + 1e-37).all()
    hq, hs = int8.quantize(to_np(buf.h))
    np.testing.assert_array_equal(buf.a2_q.cpu().numpy(), hq)
    wq, ws = int8.quantize(d["w_dn"].reshape(-1, F))
    y2 = int8.grouped_gemm(hq, hs, wq.reshape(E, D, F), ws.reshape(E, D), off)
    np.testing.assert_array_equal(to_np(buf.y2), bf16_round(y2))
    out = moe.unpermute(to_np(buf.y2), dest, k, d["topk_w"])
    ab = moe.unpermute_absbound(to_np(buf.y2), dest, k, d["topk_w"])
    assert (np.abs(to_np(buf.out) - out) <= 2.0 ** -8 * np.abs(out) + 2.0 ** -20 * ab).all()


def test_a_tokens_result_does_not_depend_on_its_batch():
    """Scales are per token: the same row in another batch gives the same bits."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import moe_layer
    E, D, F, k = 16, 256, 128, 2
    d = workloads.moe(900, 0.0, 0.01, 16.0, seed=5, E=E, k=k, D=D, F=F, name="int8")
    gu, dn = (moe_layer.quantize_expert_weights_int8(to_gpu(d[n], BF16)) for n in ("w_gu", "w_dn"))
    outs = []
    for T in (20, 300, 900):
        x, ids, tw = (to_gpu(d[n][:T], dt) for n, dt in (("x", BF16), ("topk_ids", torch.int32), ("topk_w", F32)))
        buf = moe_layer.BuffersInt8(T, k, E, D, F, x.device)
        moe_layer.forward_int8(x, ids, tw, gu, dn, buf)
        outs.append(buf.out[:20].clone())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_two_streams_and_graphs():
    require_gpu()
    from nvfp4_quantized_moe_token_amd import moe_layer
    E, D, F, k, T = 32, 256, 128, 4, 500
    d = [workloads.moe(T, 1.1, 0.01, 16.0, seed=s, E=E, k=k, D=D, F=F, name="int8") for s in range(4)]
    gu, dn = (moe_layer.quantize_expert_weights_int8(to_gpu(d[0][n], BF16)) for n in ("w_gu", "w_dn"))
    ins = [[to_gpu(c[n], dt) for n, dt in (("x", BF16), ("topk_ids", torch.int32), ("topk_w", F32))] for c in d]
    want, bufs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for i in ins:
        buf = moe_layer.BuffersInt8(T, k, E, D, F, i[0].device)
        moe_layer.forward_int8(*i, gu, dn, buf)
        want.append(buf.out.clone())
    torch.cuda.synchronize()
    for st, i in zip(streams, ins):  # two at once
        with torch.cuda.stream(st):
            bufs.append(moe_layer.BuffersInt8(T, k, E, D, F, i[0].device))
            moe_layer.forward_int8(*i, gu, dn, bufs[-1])
    torch.cuda.synchronize()
    assert torch.equal(bufs[0].out, want[0]) and torch.equal(bufs[1].out, want[1])
    x, ids, tw = (t.clone() for t in ins[0])
    buf = bufs[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe_layer.forward_int8(x, ids, tw, gu, dn, buf)
    for n in (1, 2, 3, 0):
        for a, b in zip((x, ids, tw), ins[n]):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf.out, want[n]), n
