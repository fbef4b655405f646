"""Calls that the learner's layer and its BF16 products refuse, without a GPU:
each raises before anything is launched."""

import contextlib

import pytest
import torch

from nvfp4_quantized_moe_token_amd import moe_layer, ops, optim

BF16 = torch.bfloat16


@pytest.fixture
def launched(monkeypatch):
    """Calls of the library that got past the checks (none is made)."""
    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or 0

    monkeypatch.setattr(ops._lib, "load", lambda *a: Library())
    monkeypatch.setattr(ops, "_stream", lambda: None)
    monkeypatch.setattr(ops, "_dev", lambda *ts: None)
    return calls


def z(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


OFF = torch.tensor([0, 3, 6], dtype=torch.int32)


@pytest.mark.parametrize("layout,a,b", [
    (ops.NT, z(6, 64, dtype=torch.float32), z(2, 32, 64)),      # fp32 bytes are not bf16 values
    (ops.NT, z(6, 64), z(2, 32, 64, dtype=torch.float32)),
    (ops.NT, z(6, 64, dtype=torch.float16), z(2, 32, 64)),
    (ops.NT, z(6, 96), z(2, 32, 64)),                           # reads past b
    (ops.NN, z(6, 64), z(2, 32, 64)),
    (ops.NT, z(6, 64), z(1, 32, 64)),                           # fewer experts than the offsets have
    (ops.NN, z(6, 64), z(1, 64, 32)),
    (ops.TN, z(6, 64), z(5, 32)),
    (ops.TN, z(6, 64), z(6, 32, dtype=torch.float32))])
def test_bf16_products_take_bf16_operands_that_fit(launched, layout, a, b):
    with pytest.raises(ValueError):
        ops.grouped_gemm_bf16(layout, a, b, OFF)
    assert launched == []


def test_bf16_gather_product_takes_bf16(launched):
    src = torch.zeros(6, dtype=torch.int32)
    for a, b in ((z(6, 64, dtype=torch.float32), z(3, 32)), (z(6, 64), z(3, 32, dtype=torch.float32))):
        with pytest.raises(ValueError):
            ops.grouped_gemm_bf16_tn_gather(a, b, src, 2, OFF)
    assert launched == []


def _learner(T=4, E=32, D=128):
    """What forward looks at, without the buffers on a GPU."""
    ln = object.__new__(moe_layer.Learner)
    ln.logits, ln.w_r, ln.k = z(T, E, dtype=torch.float32), z(E, D), 2
    ln.one_group = torch.tensor([0, T], dtype=torch.int32)
    return ln


@pytest.mark.parametrize("x", [z(4, 128, dtype=torch.float32), z(4, 128, dtype=torch.float16), z(5, 128), z(3, 128),
                               z(4, 256), z(4, 64), z(4, 2, 64)])
def test_learner_refuses_other_inputs(launched, x):
    with pytest.raises(ValueError):
        _learner().forward(x)
    assert launched == []


T, E, D, F, K = 4, 32, 128, 128, 2


@pytest.fixture
def inside(launched, monkeypatch):
    """`launched`, on tensors in host memory; inside["names"] are the calls made
    while the tensors' GPU was the current one."""
    depth, seen = [0], dict(names=[])

    @contextlib.contextmanager
    def on_device(*ts):
        depth[0] += 1
        yield
        depth[0] -= 1

    class Library:
        def __getattr__(self, name):
            return lambda *a: (launched.append(name), seen["names"].append(name) if depth[0] else None) and 0

    monkeypatch.setattr(ops._lib, "load", lambda *a: Library())
    for m in (ops, optim):
        monkeypatch.setattr(m, "_on_device", on_device)
    monkeypatch.setattr(optim, "_stream", lambda: None)
    monkeypatch.setattr(optim, "_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: None)
    return seen


def _f32(*shape):
    return z(*shape, dtype=torch.float32)


def test_every_launch_of_the_learner_is_on_the_weights_gpu(inside, launched):
    """Also when another GPU is the current one."""
    ln = moe_layer.Learner(_f32(E, D), _f32(E, 2 * F, D), _f32(E, D, F), T, K)
    ln.forward(z(T, D))
    ln.backward(z(T, D))
    ln.update()
    queries = {"moe_permute_workspace_size", "moe_router_workspace_size"}
    assert [n for n in launched if n not in queries] == [n for n in inside["names"] if n not in queries]
    assert len(launched) > 15


def test_mxfp4_forward_is_on_the_inputs_gpu(inside, launched):
    buf = moe_layer.BuffersMXFP4(T, K, E, D, F, torch.device("cpu"))
    u8 = dict(dtype=torch.uint8)
    gu, dn = (dict(q=z(E, n, k // 2, **u8), s=z(E, n, k // 32, **u8)) for n, k in ((2 * F, D), (D, F)))
    ids = z(T, K, dtype=torch.int32)
    launched.clear()
    moe_layer.forward_mxfp4(z(T, D), ids, _f32(T, K), gu, dn, buf)
    assert launched == inside["names"][-len(launched):] and "moe_unpermute" in launched


def test_mxfp4_forward_takes_fp32_weights_of_its_tokens(launched):
    """Others would be read as fp32, past their end."""
    buf = moe_layer.BuffersMXFP4(T, K, E, D, F, torch.device("cpu"))
    u8 = dict(dtype=torch.uint8)
    gu, dn = (dict(q=z(E, n, k // 2, **u8), s=z(E, n, k // 32, **u8)) for n, k in ((2 * F, D), (D, F)))
    launched.clear()
    for tw in (z(T, K), z(T, K + 1, dtype=torch.float32), z(T * K, dtype=torch.float32)):
        with pytest.raises(ValueError, match="topk_w"):
            moe_layer.forward_mxfp4(z(T, D), z(T, K, dtype=torch.int32), tw, gu, dn, buf)
    assert launched == []


def test_the_learner_needs_its_steps_in_order(inside, launched):
    """An update before any backward would take whatever its buffers hold."""
    ln = moe_layer.Learner(_f32(E, D), _f32(E, 2 * F, D), _f32(E, D, F), T, K)
    launched.clear()
    with pytest.raises(RuntimeError):
        ln.update()
    with pytest.raises(RuntimeError):
        ln.backward(z(T, D))
    assert launched == [] and ln.opt.steps == 0
    ln.forward(z(T, D))
    with pytest.raises(RuntimeError):
        ln.update()
    ln.backward(z(T, D))
    ln.update()
    assert ln.opt.steps == 1


def test_the_copies_of_parameters_are_outside_the_autograd_graph(inside):
    """A live graph of the leaves would meet a backward pass that the caller
    captures over the same parameters."""
    w = [torch.nn.Parameter(_f32(*s)) for s in ((E, D), (E, 2 * F, D), (E, D, F))]
    ln = moe_layer.Learner(*w, T, K)
    for t in (*ln.copies, ln.forward(z(T, D)), ln.backward(z(T, D)), *ln.grads()):
        assert not t.requires_grad and t.grad_fn is None


def test_mxfp4_permutation_takes_an_int32_status(launched):
    """The library writes four bytes there."""
    for status in (z(1, dtype=torch.uint8), z(1, dtype=torch.int64), z(0, dtype=torch.int32)):
        with pytest.raises(ValueError, match="status"):
            ops.moe_permute_mxfp4(z(T, K, dtype=torch.int32), E, z(T, D), status=status)
    assert launched == []
