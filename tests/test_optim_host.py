"""The optimizer's host side, without a GPU: the library's call is recorded
instead of made, on tensors in host memory."""

import contextlib
import copy
import ctypes
import io

import pytest
import torch

from nvfp4_quantized_moe_token_amd import _lib, optim

FIELDS = [n for n, _ in _lib.AdamWTensor._fields_]


class Library:
    """Records the calls; answers with `rc`."""

    def __init__(self):
        self.rc, self.calls = _lib.OK, []

    def _record(self, name, args):
        self.calls.append((name, [{f: getattr(d, f) for f in FIELDS} for d in args[0]], args))
        return self.rc

    def adamw_step(self, *args):
        return self._record("step", args)

    def adamw_read_state(self, *args):
        return self._record("read", args)

    def nvfp4moe_status_string(self, rc):
        return b"refused"


@pytest.fixture
def library(monkeypatch):
    lib = Library()

    def on_device(*ts):
        if any(t is not None and not t.is_contiguous() for t in ts):
            raise ValueError("contiguous tensors")
        return contextlib.nullcontext()

    monkeypatch.setattr(_lib, "load", lambda *a: lib)
    monkeypatch.setattr(optim, "_on_device", on_device)
    monkeypatch.setattr(optim, "_stream", lambda: None)
    monkeypatch.setattr(optim, "_capturing", lambda: False, raising=False)
    return lib


def _held(opt, i):
    """Name in the library's record -> tensor, of parameter i."""
    return dict({k: t[i] for k, t in opt.state.items()}, param=opt.params[i], param_bf16=opt.params_bf16[i])


def _check_record(record, opt):
    for i, d in enumerate(record):
        assert d["n"] == opt.params[i].numel()
        for name, t in _held(opt, i).items():
            assert d[name] == (None if t is None else t.data_ptr()), (i, name)


@pytest.mark.parametrize("bits", [32, 8])
def test_replaced_storage_is_noticed(library, bits):
    """`.data =` on a parameter, a copy or a moment: the next call takes the
    new address (the old storage may be anyone's by then)."""
    params = [torch.zeros(n) for n in (5, 600, 1)]
    copies = [torch.zeros(5, dtype=torch.bfloat16), None, torch.zeros(1, dtype=torch.bfloat16)]
    opt = optim.AdamW(params, params_bf16=copies, state_bits=bits)
    grads = [torch.zeros(p.shape) for p in params]
    opt.step(grads)
    _check_record(library.calls[-1][1], opt)
    assert [d["grad"] for d in library.calls[-1][1]] == [g.data_ptr() for g in grads]
    for name in _held(opt, 0):
        for i in (2, 0):
            t = _held(opt, i)[name]
            t.data = t.data.clone()
            opt.step(grads)
            _check_record(library.calls[-1][1], opt)
    if bits == 8:
        opt.state["avg_scale"][1].data = torch.zeros(3)
        opt.state_values()
        assert library.calls[-1][0] == "read"
        _check_record(library.calls[-1][1], opt)


def test_replaced_storage_is_checked(library):
    def fresh():
        return optim.AdamW([torch.zeros(64), torch.zeros(8)])

    def shrink(o):                             # where it was, but less of it
        o.params[0].data = o.params[0].data[:60]

    def other_type(o):                         # and as another type
        o.params[0].data = o.params[0].data.view(torch.int32)

    for change in (shrink, other_type, lambda o: setattr(o.params[0], "data", torch.zeros(65)),
                   lambda o: setattr(o.params[1], "data", torch.zeros(8, dtype=torch.bfloat16)),
                   lambda o: setattr(o.params[0], "data", torch.zeros(64, 2)[:, 0]),
                   lambda o: setattr(o.state["exp_avg"][0], "data", torch.zeros(32)),
                   lambda o: setattr(o.state["exp_avg_sq"][1], "data", torch.zeros(8, dtype=torch.float16))):
        opt = fresh()
        change(opt)
        before = len(library.calls)
        for _ in range(2):                     # refused again, not forgotten
            with pytest.raises(ValueError):
                opt.step([torch.zeros(p.shape) for p in opt.params])
        assert len(library.calls) == before and opt.steps == 0


def test_tensors_cannot_be_assigned(library):
    """The library works on the tensors the optimizer was made with; an
    assignment that it would not see is refused."""
    opt = optim.AdamW([torch.zeros(4)], state_bits=8)
    for name in ("params", "params_bf16", "state"):
        with pytest.raises(AttributeError):
            setattr(opt, name, [torch.zeros(4)])
    for seq in (opt.params, opt.params_bf16, *opt.state.values()):
        with pytest.raises(TypeError):
            seq[0] = torch.zeros(4)


@pytest.mark.parametrize("kw", [dict(betas=(0.9, 1.0)), dict(betas=(-0.1, 0.9)), dict(betas=(0.9,)),
                                dict(betas=(float("nan"), 0.9)), dict(eps=-1e-8), dict(eps=float("nan")),
                                dict(step=-1)])
def test_hyperparameters_are_checked_at_once(library, kw):
    with pytest.raises(ValueError):
        optim.AdamW([torch.zeros(4)], **kw)


@pytest.mark.parametrize("capturable", [False, True])
def test_a_step_that_the_library_refuses_does_not_count(library, capturable):
    opt = optim.AdamW([torch.zeros(4)], step=5, capturable=capturable)
    grads = [torch.zeros(4)]
    opt.step(grads)
    library.rc = _lib.EINVAL
    for _ in range(3):
        with pytest.raises(RuntimeError):
            opt.step(grads)
    assert opt.steps == 6 and (not capturable or opt.step_dev.item() == 6)
    library.rc = _lib.OK
    opt.step(grads)
    assert opt.steps == 7 and (not capturable or opt.step_dev.item() == 7)
    assert library.calls[-1][2][10] == 7


@pytest.mark.parametrize("capturable", [False, True])
def test_bias_corrections_go_by_the_updates_made(library, monkeypatch, capturable):
    """A skipped step leaves the moments, so t, the number of updates in them,
    stays too; the steps taken count on."""
    numbers = []

    def record(*args):
        numbers.append(args[10] if args[11] is None else ctypes.c_int64.from_address(args[11]).value)
        return _lib.OK

    monkeypatch.setattr(Library, "adamw_step", lambda self, *args: record(*args))
    opt = optim.AdamW([torch.zeros(4)], step=10, capturable=capturable)
    grads, updates = [torch.zeros(4)], 10
    for flag in (None, 0, 1, None, 5, -1, 0, None):
        opt.step(grads, skip=None if flag is None else torch.tensor([flag], dtype=torch.int32))
        if not flag:
            updates += 1
            assert numbers[-1] == updates
        assert opt.updates() == updates
    assert opt.steps == 18 and (not capturable or opt.step_dev.item() == 18)


def test_a_captured_step_counts_or_is_refused(library, monkeypatch):
    """Replays of a step whose number was taken on the host would all have the
    same bias corrections and the same random bits."""
    opts = [optim.AdamW([torch.zeros(4)], capturable=c) for c in (False, True)]
    monkeypatch.setattr(optim, "_capturing", lambda: True, raising=False)
    with pytest.raises(RuntimeError):
        opts[0].step([torch.zeros(4)])
    assert library.calls == [] and opts[0].steps == 0
    opts[1].step([torch.zeros(4)])
    assert library.calls[-1][2][11] is not None


def test_overlapping_tensors_are_refused(library):
    """Two workgroups would update the same elements at the same time."""
    p, q = torch.zeros(1000), torch.zeros(1000)
    zeros = [torch.zeros(1000), torch.zeros(1000)]
    for bad in (lambda: optim.AdamW([p, q, p]),
                lambda: optim.AdamW([p[:600], p[599:]]),
                lambda: optim.AdamW([p, q], state=dict(exp_avg=zeros, exp_avg_sq=[zeros[1], torch.zeros(1000)])),
                lambda: optim.AdamW([p, q], state=dict(exp_avg=[zeros[0], p], exp_avg_sq=[zeros[1], torch.zeros(1000)]))):
        with pytest.raises(ValueError):
            bad()
    opt = optim.AdamW([p[:600], p[600:], p[:0], q])     # neighbours, and an empty view of one
    opt.step([torch.zeros(t.shape) for t in opt.params])
    opt = optim.AdamW([p, torch.zeros(700)])
    opt.params[1].data = p.data[300:]
    with pytest.raises(ValueError):
        opt.step([torch.zeros(t.shape) for t in opt.params])
    assert len(library.calls) == 1


@pytest.mark.parametrize("bits", [32, 8])
def test_moments_are_read_into_tensors_that_fit(library, bits):
    """Lists too short, or tensors that the moments would be spread over."""
    opt = optim.AdamW([torch.zeros(4), torch.zeros(3)], state_bits=bits)
    z = torch.zeros
    for out in (([z(4)], [z(4)]), ([z(4), z(3)],), ([z(4), z(5, 3)], [z(4), z(3)]), ([z(4), z(3)], [z(4), None]),
                ([z(4), z(3)], [z(4), z(3, dtype=torch.bfloat16)])):
        with pytest.raises(ValueError):
            opt.state_values(out=out)
    assert library.calls == []
    out = [z(2, 2), z(3)], [z(4), z(3, 1)]
    assert opt.state_values(out=out) is out


def test_the_state_can_be_saved_and_gone_on_with(library):
    opt = optim.AdamW([torch.zeros(300), torch.zeros(4)], state_bits=8)
    opt.state["exp_avg"][0].fill_(3)
    file = io.BytesIO()
    torch.save(opt.state, file)
    file.seek(0)
    for state in (torch.load(file, weights_only=True), copy.deepcopy(opt.state), copy.copy(opt.state), dict(opt.state)):
        assert type(state) is dict and list(state) == ["exp_avg", "exp_avg_sq", "avg_scale", "avg_sq_scale"]
        again = optim.AdamW([torch.zeros(300), torch.zeros(4)], state_bits=8, state=state, step=opt.steps)
        for k in state:
            assert all(torch.equal(a, b) for a, b in zip(again.state[k], opt.state[k]))


def test_moments_put_in_place_of_the_old_ones(library):
    params = [torch.zeros(300), torch.zeros(4)]
    opt = optim.AdamW(params, state_bits=8)
    grads = [torch.zeros(p.shape) for p in params]
    opt.state["exp_avg"] = [torch.zeros(n, dtype=torch.uint8) for n in (300, 4)]
    opt.step(grads)
    _check_record(library.calls[-1][1], opt)
    opt.state.update(avg_scale=[torch.zeros(2), torch.zeros(1)])
    opt.state_values()
    _check_record(library.calls[-1][1], opt)
    before = len(library.calls)
    for k, ts in (("exp_avg", [torch.zeros(300), torch.zeros(4)]), ("avg_scale", [torch.zeros(2)]),
                  ("exp_avg_sq", [torch.zeros(299, dtype=torch.uint8), torch.zeros(4, dtype=torch.uint8)])):
        good = opt.state[k]
        opt.state[k] = ts
        for _ in range(2):
            with pytest.raises(ValueError):
                opt.step(grads)
        opt.state[k] = good
    opt.step(grads)
    assert len(library.calls) == before + 1 and opt.steps == 2
