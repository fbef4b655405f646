"""Grouped products of codes (MXFP4, 8-bit integers) on every tile that the mean
rows per expert choose, each against a reference of its own: the products against
exact sums, the SiLU-gate epilogue in every form against the separate steps, with
ragged, empty and one-row experts, reductions of a part of a stage, one stage and
several, and workgroups that go round over several tiles.  The cases are held to
the kernels' own rules, so that a rule that moves empties none of them."""

import os
import re

import pytest
import torch

from _helpers import gpu, require_gpu
from conftest import ROOT

CSRC = os.path.join(ROOT, "nvfp4_quantized_moe_token_amd", "csrc")
F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8
MEANS = [10, 30, 50, 90, 130, 200, 250, 300, 420]  # rows per expert


def _counts(mean, times=1):
    return [2 * mean + 7, 0, mean - 8, 1, 2 * mean] * times


def _rows(counts):
    return sum(counts) + 2  # two rows behind the last expert


def _borders(source):
    """Rows per expert at which the rule of a source file passes to another tile."""
    once = re.search(r"constexpr int64_t kOnceRows = (\d+);", open(os.path.join(CSRC, "gemm_codes.hpp")).read()).group(1)
    text = open(os.path.join(CSRC, source)).read().replace("kOnceRows *", once + " *")
    rule = text[text.index("int launch_epi("):]
    rule = rule[:rule.index("\n}")]
    tiles = re.findall(r"launch_tiles<\w+, (\d+),", rule)
    found = sorted({int(n) for n in re.findall(r"M (?:<=|>) (\d+) \* (?:\(int64_t\)p\.)?(?:p\.)?E", rule)})
    assert len(found) >= len(tiles) - 1  # every return but the last has its border
    return found


@pytest.mark.parametrize("source", ["gemm_int8.hip", "gemm_mxfp4.hip"])
def test_the_cases_reach_every_tile(source):
    borders = _borders(source)
    for times in (1, 3):
        reached = {sum(_rows(_counts(m, times)) > b * len(_counts(m, times)) for b in borders) for m in MEANS}
        assert reached == set(range(len(borders) + 1)), (source, borders, reached)


def _codes(bits, rows, K, g):
    """(codes, scales) whose sums are exact: integers, or E2M1 with scales of 1 and 1/2 (products are multiples of
    1/16, sums below 36 K)."""
    if bits == 8:
        return (torch.randint(-128, 128, (rows, K), dtype=torch.int32, device="cuda", generator=g).to(torch.int8),
                torch.rand(rows, device="cuda", generator=g) * 1e-2 + 1e-4)
    return (torch.randint(0, 256, (rows, K // 2), dtype=U8, device="cuda", generator=g),
            torch.randint(126, 128, (rows, K // 32), dtype=U8, device="cuda", generator=g))


def _operands(bits, counts, N, K):
    g = torch.Generator(device="cuda").manual_seed(bits + N + K + counts[0])
    E, M = len(counts), _rows(counts)
    a, b = _codes(bits, M, K, g), _codes(bits, E * N, K, g)
    off = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
    return (*a, b[0].view(E, N, -1), b[1].view(E, N, -1) if bits == 4 else b[1].view(E, N), off)


def _values(q, s):
    e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=q.device)
    e2m1 = torch.cat([e2m1, -e2m1])
    v = torch.stack([e2m1[(q & 15).long()], e2m1[(q >> 4).long()]], -1).flatten(-2)
    return v * torch.exp2(s.float() - 127).repeat_interleave(32, -1)


def _exact(bits, a_q, a_s, b_q, b_s, off, dtype, fill):
    """The product from its definition; rows behind the last expert hold `fill`."""
    out = torch.full((a_q.shape[0], b_q.shape[1]), fill, dtype=dtype, device="cuda")
    ends = off.tolist()
    for e in range(len(ends) - 1):
        lo, hi = ends[e], ends[e + 1]
        if hi == lo:
            continue
        if bits == 8:
            c = (a_q[lo:hi].double() @ b_q[e].double().t()).float() * a_s[lo:hi, None] * b_s[e]
        else:
            c = (_values(a_q[lo:hi], a_s[lo:hi]).double() @ _values(b_q[e], b_s[e]).double().t()).float()
        out[lo:hi] = c.to(dtype)
    return out


def _gemm(bits):
    from nvfp4_quantized_moe_token_amd import ops
    return ops.grouped_gemm_int8 if bits == 8 else ops.grouped_gemm_mxfp4


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("mean", MEANS)
@pytest.mark.parametrize("bits", [8, 4])
def test_products(bits, mean, dtype):
    require_gpu()
    for N, K in ((288, 128), (544, 384)) + (((96, 112), (256, 400)) if bits == 8 else ((96, 256), (256, 640))):
        a = _operands(bits, _counts(mean), N, K)
        want = _exact(bits, *a, dtype, 7.0)
        out = torch.full_like(want, 7.0)
        assert torch.equal(_gemm(bits)(*a, out=out), want), (N, K)


def _gate(bits, a, F, form, end):
    """The gate's epilogue in a form; every output has to be the separate steps', rows behind the end as before."""
    from nvfp4_quantized_moe_token_amd import ops
    M = a[0].shape[0]
    y1 = _exact(bits, *a, BF16, 0.0)
    h, amax = ops.silu_gate_fwd(y1)
    want = dict(y1=y1, h=h)
    want["q_y1"], want["s_y1"] = ops.mx_quantize(y1, ops.MX_INT8)
    want["q_h"], want["s_h"] = ops.mx_quantize(h, ops.MX_E2M1)
    new = lambda n, dt, v=77: torch.full((M, n), v, dtype=dt, device="cuda")  # noqa: E731
    kw = dict(h=new(F, BF16)) if bits == 8 or "h" in form else dict(want_h=False)
    if "y" in form:
        kw["y1"] = new(2 * F, BF16)
    else:
        kw["want_y1"] = False
    if "c" in form:
        kw["q_y1"], kw["s_y1"] = new(2 * F, U8), new(2 * F // 32, U8)
    if bits == 4 and "q" in form:
        kw["q_h"], kw["s_h"] = new(F // 2, U8), new(F // 32, U8)
    am = torch.full((1,), 9.0, device="cuda")
    gate = ops.grouped_gemm_int8_silu_gate if bits == 8 else ops.grouped_gemm_mxfp4_silu_gate
    r = gate(*a, amax_out=am, **kw)
    assert torch.equal(am, amax)
    for n, t in kw.items():
        if torch.is_tensor(t):
            assert r[n] is t and torch.equal(t[:end], want[n][:end]), n
            assert (t[end:] == 77).all(), n


# y: Y1 in bf16, h: H, c: Y1 in 8 bits, q: H in MXFP4 (of MXFP4 products)
FORMS = [(8, f) for f in ("h", "yh", "hc", "yhc")] + [(4, f) for f in ("h", "yh", "hc", "yhc", "q", "yhq", "qc", "yhqc")]


@gpu
@pytest.mark.parametrize("bits,form", FORMS)
@pytest.mark.parametrize("mean", MEANS)
def test_gate_epilogues(bits, mean, form):
    require_gpu()
    counts = _counts(mean)
    for F, K in ((128, 128), (384, 112 if bits == 8 else 384)):
        _gate(bits, _operands(bits, counts, 2 * F, K), F, form, sum(counts))


@gpu
@pytest.mark.parametrize("bits,form", [(8, "hc"), (8, "yhc"), (4, "hc"), (4, "yhqc")])
@pytest.mark.parametrize("mean", MEANS)
def test_gate_epilogues_of_many_tiles(bits, mean, form):
    """More tiles than a card has workgroups for twice over: each goes round, its loads running ahead across tiles."""
    require_gpu()
    counts, F, K = _counts(mean, 3), 8192, 128
    # (row blocks of 256 at most: at least one per expert that has rows, 64 column tiles each)
    assert sum(c > 0 for c in counts) * (2 * F // 256) >= 2 * 256
    _gate(bits, _operands(bits, counts, 2 * F, K), F, form, sum(counts))


@gpu
@pytest.mark.parametrize("bits", [8, 4])
def test_gate_that_leaves_as_a_stream(bits):
    """Y1 of more than the bytes from which it is stored non-temporally."""
    require_gpu()
    stream = eval(re.search(r"kStreamBytes = (\d+)LL << 20;", open(os.path.join(CSRC, "gemm_codes.hpp")).read()).group(1)) << 20
    F, K = 768, 128
    M = stream // (4 * F) + 1000
    counts = [M // 2 - 77, 3, 0, M // 2 + 70]
    _gate(bits, _operands(bits, counts, 2 * F, K), F, "yh" if bits == 8 else "yhq", sum(counts))
