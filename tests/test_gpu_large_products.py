"""Grouped products of codes whose output is too large for the caches and leaves
non-temporally: the same bits as from calls on parts of the rows, whose output
is small, with rows behind the last sequence left as they were; and every tile,
with weights loaded once or kept in the caches, against another one."""

import pytest
import torch

from _helpers import gpu, require_gpu

pytestmark = gpu

K, E = 256, 3
LARGE = 336 << 20  # bytes from which the output leaves as a stream


def _codes(rows, bits, g):
    if bits == 8:
        return (torch.randint(-127, 128, (rows, K), dtype=torch.int8, device="cuda", generator=g),
                torch.rand(rows, device="cuda", generator=g) * 1e-3 + 1e-4)
    return (torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device="cuda", generator=g),
            torch.randint(118, 124, (rows, K // 32), dtype=torch.uint8, device="cuda", generator=g))


def _operands(bits, M, N):
    g = torch.Generator(device="cuda")
    g.manual_seed(bits + N)
    a = _codes(M, bits, g)
    b = [t.view(E, N, *t.shape[1:]) for t in _codes(E * N, bits, g)]
    off = torch.tensor([0, M // 3 + 77, M // 2 + 5, M - 100], dtype=torch.int32, device="cuda")
    return a, b, off


def _parts(a, off, M):
    """The rows of either half of M, with the offsets as they fall there."""
    for lo, hi in ((0, M // 2), (M // 2, M)):
        yield lo, hi, [t[lo:hi] for t in a], (off.clamp(lo, hi) - lo)


@pytest.mark.parametrize("bits,dtype,N", [(8, torch.bfloat16, 2048), (4, torch.bfloat16, 1952), (8, torch.float32, 992),
                                          (4, torch.float32, 1024)])
def test_product(bits, dtype, N):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    gemm = ops.grouped_gemm_int8 if bits == 8 else ops.grouped_gemm_mxfp4
    size = torch.empty((), dtype=dtype).element_size()
    M = LARGE // (N * size) + 4001
    a, b, off = _operands(bits, M, N)
    out = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
    gemm(*a, *b, off, out=out)
    assert bool((out[M - 100:] == 7.0).all())
    for lo, hi, part, at in _parts(a, off, M):
        want = torch.full((hi - lo, N), 7.0, dtype=dtype, device="cuda")
        assert want.numel() * size < LARGE
        gemm(*part, *b, at, out=want)
        assert torch.equal(out[lo:hi], want)


@pytest.mark.parametrize("bits", [8, 4])
def test_gate(bits):
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    gate = ops.grouped_gemm_int8_silu_gate if bits == 8 else ops.grouped_gemm_mxfp4_silu_gate
    F = 768
    M = LARGE // (4 * F) + 3001
    a, b, off = _operands(bits, M, 2 * F)
    more = {} if bits == 8 else dict(want_q=True)
    whole = gate(*a, *b, off, **more)
    for lo, hi, part, at in _parts(a, off, M):
        want, end = gate(*part, *b, at, **more), int(at[-1])
        assert want["y1"].numel() * 2 < LARGE
        for n in ("y1", "h") + (("q_h", "s_h") if more else ()):
            assert torch.equal(whole[n][lo:lo + end], want[n][:end]), n


@pytest.mark.parametrize("rows", [10, 30, 100, 130, 150, 200, 250, 300, 400])
@pytest.mark.parametrize("bits", [8, 4])
def test_same_bits_by_rows_per_expert(bits, rows):
    """Every tile, with weights loaded once or kept: the sums go the same way, so empty experts, which lower the
    mean and so choose another tile, change nothing."""
    require_gpu()
    from nvfp4_quantized_moe_token_amd import ops
    gemm = ops.grouped_gemm_int8 if bits == 8 else ops.grouped_gemm_mxfp4
    gate = ops.grouped_gemm_int8_silu_gate if bits == 8 else ops.grouped_gemm_mxfp4_silu_gate
    N, M = 256 + 256 * (bits == 4), E * rows
    a, b, _ = _operands(bits, M, N)
    off = torch.tensor([0, rows + 7, rows + 7, M], dtype=torch.int32, device="cuda")
    more, at = [torch.cat([t, t.flip(0), t, t, t]) for t in b], torch.cat([off, off[-1:].expand(4 * E)])
    out = gemm(*a, *b, off)
    assert torch.equal(out, gemm(*a, *more, at))
    if bits == 8:  # sums below 2^24 are exact in fp32
        e = torch.repeat_interleave(torch.arange(E, device="cuda"), (off[1:] - off[:-1]).long())
        for i in range(E):
            p = (a[0][e == i].double().cpu() @ b[0][i].double().cpu().T).float().cuda()
            assert torch.equal(out[e == i], p * a[1][e == i][:, None] * b[1][i])
    x, y = gate(*a, *b, off), gate(*a, *more, at)
    assert torch.equal(x["y1"], y["y1"]) and torch.equal(x["h"], y["h"])
