"""Calls that the learner's layer and its BF16 products refuse, without a GPU:
each raises before anything is launched."""

import pytest
import torch

from nvfp4_quantized_moe_token_amd import moe_layer, ops

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
