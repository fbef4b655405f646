"""Calls of the norms, the 8-bit integer path and the 8-bit checkpoints that are
refused, without a GPU: by the library before any HIP call, by the Python layer
before anything is launched."""

import contextlib
import os

import pytest
import torch

from nvfp4_quantized_moe_token_amd import _lib, moe_layer, ops

FAKE = 0x10000
F32, BF16, I8, U8, I32 = torch.float32, torch.bfloat16, torch.int8, torch.uint8, torch.int32


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built (run __graft_entry__.build())")
    return _lib.load()


def _refused(f, ok, cases):
    for at, value, rc in cases:
        args = list(ok)
        for i, v in zip(at, value) if isinstance(at, tuple) else ((at, value),):
            args[i] = v
        assert f(*args) == rc, (f.__name__, at, value)


def test_layer_norm(lib):
    #        x    xd T  D   w     b    wd eps  kind y   yd mean  rstd  stream
    ok = [FAKE, 1, 4, 64, FAKE, FAKE, 0, 1e-5, 0, FAKE, 1, FAKE, FAKE, None]
    _refused(lib.layer_norm, ok, [
        (0, None, -1), (1, 2, -1), (2, -1, -1), (3, -1, -1), (6, 2, -1), (7, -1.0, -1), (7, float("nan"), -1),
        (8, 2, -1), (8, 1, -1), (9, None, -1), (10, 2, -1),   # (8 = 1: a mean is not given with RMS)
        (3, 0, -2), (3, 16385, -2), (0, FAKE + 1, -2), (9, FAKE + 1, -2), (4, FAKE + 2, -2), (11, FAKE + 2, -2),
        (12, FAKE + 1, -2)])
    size = lib.layer_norm_bwd_workspace_size
    assert size(385, 64) == 2 * 256 * 64 * 4 and size(100000, 2048) == 2 * 256 * 2048 * 4
    assert size(0, 64) == size(384, 64) == size(4000, 0) == size(4000, 16385) == 0  # (few rows need none)
    #      dy   dd  x   xd T    D   w   wd mean  rstd kind dx  od  dw    db    ws   bytes     stream
    ok = [FAKE, 0, FAKE, 1, 400, 64, FAKE, 0, FAKE, FAKE, 0, FAKE, 0, FAKE, FAKE, FAKE, 1 << 20, None]
    _refused(lib.layer_norm_bwd, ok, [
        (0, None, -1), (1, 2, -1), (2, None, -1), (3, 2, -1), (4, -1, -1), (7, 2, -1), (8, None, -1), (9, None, -1),
        (10, 2, -1), (12, 2, -1), ((11, 13, 14), (None, None, None), -1),
        (5, 0, -2), (5, 16385, -2), (0, FAKE + 2, -2), (11, FAKE + 2, -2), (13, FAKE + 2, -2), (15, FAKE + 8, -2),
        (15, None, -5), (16, size(400, 64) - 1, -5)])


def test_int8_entry_points(lib):
    _refused(lib.int8_quantize, [FAKE, 1, 4, 64, FAKE, FAKE, None], [
        (0, None, -1), (1, 2, -1), (2, -1, -1), (3, -1, -1), (4, None, -1), (5, None, -1),
        (3, 40, -2), (0, FAKE + 8, -2), (4, FAKE + 8, -2), (5, FAKE + 2, -2)])
    ok = [FAKE, FAKE, FAKE, FAKE, FAKE, 4, 64, 64, 64, FAKE, 0, None]
    _refused(lib.grouped_gemm_int8, ok, [
        (0, None, -1), (1, None, -1), (2, None, -1), (3, None, -1), (4, None, -1), (5, 0, -1), (6, -1, -1), (7, -1, -1),
        (8, -1, -1), (9, None, -1), (10, 2, -1),
        (8, 40, -2), (8, (1 << 17) + 16, -2), (7, 48, -2), (7, (1 << 20) + 32, -2), (6, 0x7FFFFF00, -2),
        (0, FAKE + 8, -2), (1, FAKE + 2, -2), (2, FAKE + 8, -2), (3, FAKE + 1, -2), (4, FAKE + 2, -2), (9, FAKE + 8, -2)])
    #                                          E  M   F    K    y1   h     amax  q     s
    ok = [FAKE, FAKE, FAKE, FAKE, FAKE, 4, 64, 128, 64, FAKE, FAKE, FAKE, FAKE, FAKE, None]
    _refused(lib.grouped_gemm_int8_silu_gate, ok, [
        (10, None, -1), (12, None, -1), (13, None, -1), (7, -128, -1), (4, None, -1), (1, None, -1),
        (7, 64, -2), (8, 24, -2), (12, FAKE + 4, -2), (11, FAKE + 2, -2), ((7, 8), (1 << 13, 1 << 17), -2)])
    T, k, E = 100, 8, 128
    ws = lib.moe_permute_workspace_size(T, k, E)
    ok = [FAKE, T, k, E, FAKE, 1, 64, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, ws, None, None]
    _refused(lib.moe_permute_int8, ok, [
        (2, 0, -1), (5, 2, -1), (4, None, -1), (7, None, -1), (8, None, -1), (9, None, -1),
        (3, 5000, -2), (2, 65, -2), (6, 24, -2), (4, FAKE + 8, -2), (7, FAKE + 8, -2), (8, FAKE + 2, -2),
        (13, ws - 1, -5), (12, None, -5)])


def test_rows_without_elements_have_scales(lib):
    T, k, E = 100, 8, 128
    ws = lib.moe_permute_workspace_size(T, k, E)
    ok = [FAKE, T, k, E, None, 1, 0, None, FAKE, FAKE, FAKE, FAKE, FAKE, ws, None, None]
    _refused(lib.moe_permute_int8, ok, [(8, None, -1), (8, FAKE + 2, -2)])


def test_checkpoint_entry_points(lib):
    q = lib.mx_quantize
    assert q(FAKE, 1, 4, 64, _lib.MX_INT8, FAKE + 8, FAKE, None) == -2
    assert q(FAKE, 1, 4, 48, _lib.MX_INT8, FAKE, FAKE, None) == -2
    ok = [FAKE, FAKE, 4, 64, _lib.MX_INT8, FAKE, 1, None]
    _refused(lib.mx_dequantize, ok, [
        (0, None, -1), (1, None, -1), (2, -1, -1), (3, -32, -1), (4, 3, -1), (4, -1, -1), (5, None, -1), (6, 2, -1),
        (3, 48, -2), (0, FAKE + 8, -2), (5, FAKE + 8, -2), ((4, 0), (_lib.MX_E2M1, FAKE + 4), -2)])
    _refused(lib.silu_gate_bwd_mx, [FAKE, FAKE, FAKE, 4, 64, FAKE, FAKE, None], [
        (0, None, -1), (1, None, -1), (2, None, -1), (3, -1, -1), (4, -1, -1), (5, None, -1),
        (4, 48, -2), (0, FAKE + 8, -2), (2, FAKE + 8, -2), (5, FAKE + 8, -2), (6, FAKE + 8, -2)])
    #                                          E  M   F    K    y1    h     amax  qh    sh    qy    sy
    ok = [FAKE, FAKE, FAKE, FAKE, FAKE, 4, 64, 128, 128, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None]
    _refused(lib.grouped_gemm_mxfp4_silu_gate_ckpt, ok, [
        (14, None, -1), (15, None, -1), (12, None, -1), ((10, 12, 13), (None, None, None), -1), (7, -128, -1),
        (7, 64, -2), (8, 64, -2), (14, FAKE + 4, -2)])


@pytest.fixture
def launched(monkeypatch):
    """Calls of the library that got past the checks (none is made)."""
    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or 0

    monkeypatch.setattr(ops._lib, "load", lambda *a: Library())
    monkeypatch.setattr(ops, "_stream", lambda: None)
    monkeypatch.setattr(ops, "_on_device", lambda *ts: contextlib.nullcontext())
    monkeypatch.setattr(ops, "_dev", lambda *ts: None)
    return calls


def z(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


def f(*shape):
    return z(*shape, dtype=F32)


STATS = f(4), f(4)
OFF = torch.tensor([0, 3, 6], dtype=I32)
GEMM = dict(a_q=z(6, 64, dtype=I8), a_s=f(6), b_q=z(2, 256, 64, dtype=I8), b_s=f(2, 256), offsets=OFF)


@pytest.mark.parametrize("call", [
    lambda: ops.layer_norm(z(4, 8, dtype=torch.float16)),
    lambda: ops.layer_norm(z(8)),
    lambda: ops.layer_norm(z(4, 8), f(7)),
    lambda: ops.layer_norm(z(4, 8), f(8), z(8)),                    # two dtypes of weights
    lambda: ops.layer_norm(z(4, 8), f(8), y=z(4, 9)),
    lambda: ops.layer_norm(z(4, 8), f(8), out_dtype=torch.float16),
    lambda: ops.layer_norm(z(4, 8), f(8), mean=f(5)),
    lambda: ops.layer_norm(z(4, 8), f(8), rstd=z(4)),
    lambda: ops.layer_norm_bwd(f(4, 9), z(4, 8), f(8), *STATS),
    lambda: ops.layer_norm_bwd(f(4, 8), z(4, 8), f(8), None, STATS[1]),
    lambda: ops.layer_norm_bwd(f(4, 8), z(4, 8), f(8), STATS[0], None),
    lambda: ops.layer_norm_bwd(f(4, 8), z(4, 8), f(8), *STATS, dw=z(8)),
    lambda: ops.layer_norm_bwd(f(4, 8), z(4, 8), f(8), *STATS, dx_dtype=torch.float16),
    lambda: ops.int8_quantize(z(4, 32, dtype=torch.float16)),
    lambda: ops.int8_quantize(z(4, 32), q=z(4, 32, dtype=U8)),
    lambda: ops.int8_quantize(z(4, 32), scales=f(5)),
    lambda: ops.moe_permute_int8(z(4, 2, dtype=torch.int64), 8, z(4, 32)),
    lambda: ops.moe_permute_int8(z(4, 2, dtype=I32), 8, z(5, 32)),
    lambda: ops.moe_permute_int8(z(4, 2, dtype=I32), 8, z(4, 32), status=z(1, dtype=U8)),
    lambda: ops.grouped_gemm_int8(**{**GEMM, "a_q": z(6, 64, dtype=U8)}),
    lambda: ops.grouped_gemm_int8(**{**GEMM, "a_s": f(5)}),
    lambda: ops.grouped_gemm_int8(**{**GEMM, "b_s": f(2, 255)}),
    lambda: ops.grouped_gemm_int8(**{**GEMM, "b_q": z(2, 256, 80, dtype=I8)}),
    lambda: ops.grouped_gemm_int8(**{**GEMM, "offsets": OFF[:2]}),
    lambda: ops.grouped_gemm_int8(**GEMM, out=z(6, 255)),
    lambda: ops.grouped_gemm_int8(**GEMM, out_dtype=torch.float16),
    lambda: ops.grouped_gemm_int8_silu_gate(**GEMM, h=z(6, 256)),
    lambda: ops.grouped_gemm_int8_silu_gate(**GEMM, q_y1=z(6, 256, dtype=I8)),
    lambda: ops.grouped_gemm_int8_silu_gate(**GEMM, s_y1=z(6, 9, dtype=U8)),
    lambda: ops.mx_quantize(z(4, 64), ops.MX_INT8, q=z(4, 32, dtype=U8)),          # a buffer of 4-bit codes
    lambda: ops.mx_quantize(z(4, 64), ops.MX_INT8, scales=z(4, 1, dtype=U8)),
    lambda: ops.mx_dequantize(z(4, 64, dtype=I8), z(4, 2, dtype=U8), ops.MX_INT8),
    lambda: ops.mx_dequantize(z(4, 64, dtype=U8), z(4, 3, dtype=U8), ops.MX_INT8),
    lambda: ops.mx_dequantize(z(4, 64, dtype=U8), z(4, 2, dtype=U8), ops.MX_E2M1),
    lambda: ops.mx_dequantize(z(4, 64, dtype=U8), z(4, 2, dtype=U8), ops.MX_INT8, out_dtype=torch.float16),
    lambda: ops.silu_gate_bwd_mx(z(4, 128, dtype=U8), z(4, 4, dtype=U8), f(4, 64)),
    lambda: ops.silu_gate_bwd_mx(z(4, 64, dtype=U8), z(4, 4, dtype=U8), z(4, 64)),
    lambda: ops.silu_gate_bwd_mx(z(4, 128, dtype=U8), z(4, 4, dtype=U8), z(4, 64), dy1=z(4, 64)),
    lambda: moe_layer.Learner(f(32, 128), f(32, 256, 128), f(32, 128, 128), 4, 2, experts="fp8"),
])
def test_refused_in_python(launched, call):
    with pytest.raises(ValueError):
        call()
    assert launched == []


@pytest.mark.parametrize("elem", [ops.MX_E4M3, ops.MX_E2M1, ops.MX_INT8])
def test_mx_quantizer_refuses_other_dtypes(launched, elem):
    for x in (z(4, 64, dtype=torch.float16), z(4, 64, dtype=U8), z(2, 4, 64)):
        with pytest.raises(ValueError):
            ops.mx_quantize(x, elem)
    assert launched == []


@pytest.mark.parametrize("call", [
    lambda: ops.mx_quantize(z(4, 64), ops.MX_E4M3),
    lambda: ops.mx_quantize(z(4, 64), ops.MX_E2M1),
    lambda: ops.mx_quantize(z(4, 64), ops.MX_INT8),
    lambda: ops.mx_dequantize(z(4, 64, dtype=U8), z(4, 2, dtype=U8), ops.MX_INT8),
    lambda: ops.int8_quantize(z(4, 32)),
    lambda: ops.moe_permute_int8(z(4, 2, dtype=I32), 8, z(4, 32), workspace=z(64, dtype=U8)),
    lambda: ops.grouped_gemm_int8(**GEMM),
    lambda: ops.grouped_gemm_int8_silu_gate(**GEMM),
    lambda: ops.silu_gate_bwd_mx(z(4, 128, dtype=U8), z(4, 4, dtype=U8), z(4, 64)),
    lambda: ops.layer_norm(z(4, 8), f(8)),
    lambda: ops.layer_norm_bwd(f(4, 8), z(4, 8), None, *STATS),
])
def test_launched_with_the_tensors_gpu_current(launched, monkeypatch, call):
    """The stream is taken, and the library called, while the inputs' GPU is the current one."""
    inside, stream = [], []

    @contextlib.contextmanager
    def on_device(first, *ts):
        inside.append(first)
        yield
        inside.pop()

    monkeypatch.setattr(ops, "_on_device", on_device)
    monkeypatch.setattr(ops, "_stream", lambda: stream.append(len(inside)))
    call()
    assert len(launched) == 1 and stream == [1] and inside == []


def test_cpu_tensors_are_refused():
    for call in (lambda: ops.layer_norm(z(4, 8)), lambda: ops.int8_quantize(z(4, 32)),
                 lambda: ops.silu_gate_bwd_mx(z(4, 128, dtype=U8), z(4, 4, dtype=U8), z(4, 64))):
        with pytest.raises(ValueError):
            call()


def test_the_learners_norm_is_checked(launched):
    w = f(32, 128), f(32, 256, 128), f(32, 128, 128)
    for bad in ((f(64), None), (z(128), None), (f(128), f(129))):
        with pytest.raises(ValueError, match="norm"):
            moe_layer.Learner(*w, 4, 2, norm=bad)


def test_checkpoint_buffers_hold_a_third():
    """Of the bytes of Y1 and H, which a layer keeps between its passes without them."""
    for cls in (moe_layer.BuffersMXFP4, moe_layer.BuffersInt8):
        a, b = (cls(64, 2, 4, 128, 128, torch.device("cpu"), backward=True, checkpoint=c) for c in (False, True))
        bytes_ = lambda *ts: sum(t.numel() * t.element_size() for t in ts)  # noqa: E731
        assert a.q_y1 is None and b.y1 is None
        assert bytes_(b.q_y1, b.s_y1) / bytes_(a.y1, a.h) == pytest.approx(33 / 96)


def test_what_the_checkpoint_takes_from_the_buffers():
    """All of the buffers: Y1's bytes less those of its codes and scales, and nothing else (H keeps its place)."""
    T, k, E, D, F = 64, 2, 4, 128, 128
    for cls in (moe_layer.BuffersMXFP4, moe_layer.BuffersInt8):
        a, b = (cls(T, k, E, D, F, torch.device("cpu"), backward=True, checkpoint=c) for c in (False, True))
        size = lambda o: sum(t.numel() * t.element_size() for t in vars(o).values() if torch.is_tensor(t))  # noqa: E731
        y1, h = T * k * 2 * F * 2, T * k * F * 2
        assert size(a) - size(b) == y1 - y1 // 2 * 33 // 32
        assert (b.q_y1.numel() + b.s_y1.numel() + b.h.numel() * 2) / (y1 + h) == pytest.approx(65 / 96)
