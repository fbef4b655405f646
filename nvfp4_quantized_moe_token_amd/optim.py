"""AdamW for the learner's weights on the library's adamw_step: one launch for
56 or 72 tensors, moments in fp32 or in 8 bits.

The class owns the moments and the list of pointers that the C entry point
takes; every step of the arithmetic runs in the HIP kernel.
"""

import ctypes

import torch

from . import _lib
from .ops import _DT, _FLOATS, _check, _on_device, _ptr, _stream

BLOCK = _lib.ADAMW_BLOCK
_WORDS = ctypes.sizeof(_lib.AdamWTensor) // 8  # 8-byte fields of the C record

# Methods called over whole lists: half the time of a loop of bound calls.
_PTR, _NUMEL, _DEVICE, _CONTIGUOUS = (torch.Tensor.data_ptr, torch.Tensor.numel, torch.Tensor.get_device,
                                      torch.Tensor.is_contiguous)
_capturing = torch.cuda.is_current_stream_capturing
# torch's comparison of many tensors' addresses with known ones (183 in 5 us).
_same_addresses = getattr(torch._C, "_tensors_data_ptrs_at_indices_equal",
                          lambda ts, ptrs, at: list(map(_PTR, ts)) == ptrs)


class AdamW:
    """AdamW (decoupled weight decay) over a list of contiguous parameters of
    one dtype (fp32, or bf16 rounded stochastically) on one GPU.

    params_bf16: for each fp32 parameter a bf16 tensor that every step
    overwrites with its rounded value (or None, for all or for one).
    state_bits: 32, or 8 (codes with one fp32 scale per 256 elements, rounded
    stochastically).  seed: of that rounding, whose bits depend on it, the
    update's number, the tensor's place in the list and the element: several
    optimizers of one model (groups with other hyperparameters) take different
    seeds.  step: updates already made.
    state: moments to go on with, a dict of lists: exp_avg, exp_avg_sq, and
    for 8 bits avg_scale, avg_sq_scale (kept, not copied); zeros otherwise.
    capturable: the step count and the learning rate live on the device
    (``step_dev`` int64 [1], ``lr_dev`` fp32 [1]), so a captured step counts
    on at every replay; without it a step is refused while a graph is captured.

    ``params``, ``params_bf16`` and the tuples of ``state`` hold the tensors and
    cannot be assigned to.  A tensor whose storage was replaced (``p.data =
    ...``) and a list put in ``state`` in a tuple's place are noticed at the
    next call, checked like new ones, and used from there on; a captured graph
    keeps the addresses that it was captured with.
    """

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, params_bf16=None,
                 state_bits=32, seed=0, step=0, state=None, capturable=False):
        self._params = tuple(params)
        if not self.params:
            raise ValueError("AdamW needs at least one parameter")
        if state_bits not in (8, 32):
            raise ValueError("state_bits: 8 or 32, got %r" % (state_bits,))
        if not (all(0.0 <= b < 1.0 for b in betas) and len(betas) == 2 and eps >= 0.0 and step >= 0):
            raise ValueError("AdamW: two betas in [0, 1), eps and step not negative; got %r, %r, %r" % (betas, eps, step))
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        self.state_bits, self.seed, self.steps = state_bits, seed & 0xFFFFFFFF, step
        n = len(self.params)
        self._params_bf16 = (None,) * n if params_bf16 is None else tuple(params_bf16)
        self._state = {}
        self._validate()
        if state is None:
            state = self._new_state()
        self._names = ("exp_avg", "exp_avg_sq") + (("avg_scale", "avg_sq_scale") if state_bits == 8 else ())
        self._state = {k: state[k] for k in self._names}
        self._list = (_lib.AdamWTensor * n)()
        self._words = (ctypes.c_void_p * (_WORDS * n)).from_buffer(self._list)  # its fields, _WORDS per tensor
        self._take()
        dev = self.params[0].device
        self.step_dev = torch.full((1,), step, dtype=torch.int64, device=dev) if capturable else None
        self.lr_dev = torch.full((1,), lr, dtype=torch.float32, device=dev) if capturable else None
        # 1 less the steps skipped: added to the steps taken it is the number
        # of the next update.  Only the GPU knows it once a flag was given.
        self._next = torch.ones((1,), dtype=torch.int64, device=dev)
        self._skips = capturable  # (a captured step goes on after an eager one was skipped)

    # The tensors are fixed for good (their storage is not): another set is
    # another optimizer.
    @property
    def params(self):
        return self._params

    @property
    def params_bf16(self):
        return self._params_bf16

    @property
    def state(self):
        return self._state

    def _validate(self):
        """Refuses tensors of the wrong dtype, size, device or layout."""
        dt = self.params[0].dtype
        if dt not in (torch.float32, torch.bfloat16) or any(p.dtype != dt for p in self.params):
            raise ValueError("AdamW takes parameters of one dtype, fp32 or bf16")
        self._same_sizes("params_bf16", self.params_bf16, torch.bfloat16)
        if dt != torch.float32 and any(c is not None for c in self.params_bf16):
            raise ValueError("params_bf16 goes with fp32 parameters")
        moments = torch.uint8 if self.state_bits == 8 else torch.float32
        for k, ts in self._state.items():
            scales = k.endswith("_scale")
            self._same_sizes(k, ts, torch.float32 if scales else moments, required=True, blocks=scales)
        held = [t for t in (*self.params, *self.params_bf16, *(t for ts in self._state.values() for t in ts))
                if t is not None]
        _on_device(*held)
        # A tensor given twice (shared weights) would be updated by two
        # workgroups at once.
        ends = sorted((t.data_ptr(), t.data_ptr() + t.nbytes) for t in held if t.numel())
        if any(a[1] > b[0] for a, b in zip(ends, ends[1:])):
            raise ValueError("AdamW: two of the tensors overlap in memory (shared parameters go in once)")

    def _take(self):
        """Checks the tensors and lists their addresses for the library."""
        self._dtype = None
        for k in self._names:
            self._state[k] = tuple(self._state[k])
        self._validate()
        self._numel = list(map(_NUMEL, self.params))
        lists = dict(self._state, param=self.params, param_bf16=self.params_bf16)
        for i, d in enumerate(self._list):
            d.n = self._numel[i]
            for k, ts in lists.items():
                setattr(d, k, _ptr(ts[i]))
        self._moments = [self._state[k] for k in self._names]
        self._held = [t for ts in (self.params, self.params_bf16, *self._moments) for t in ts if t is not None]
        self._ptrs, self._all = list(map(_PTR, self._held)), list(range(len(self._held)))
        self._dtype = self.params[0].dtype

    def _refresh(self):
        """A tensor's storage may be another since the last call (``p.data =``,
        weights moved away and back): then the new one is checked and taken."""
        if (self.params[0].dtype is not self._dtype
                or any(self._state[k] is not ts for k, ts in zip(self._names, self._moments))
                or not _same_addresses(self._held, self._ptrs, self._all)):
            self._take()

    def _same_sizes(self, name, ts, dtype, required=False, blocks=False):
        if len(ts) != len(self.params):
            raise ValueError("%s: %d tensors for %d parameters" % (name, len(ts), len(self.params)))
        for p, t in zip(self.params, ts):
            if t is None and not required:
                continue
            if t is None or t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
                raise ValueError("%s: %s tensors expected" % (name, dtype))
            if t.numel() != (-(-p.numel() // BLOCK) if blocks else p.numel()):
                raise ValueError("%s: %d elements for a parameter of %d" % (name, t.numel(), p.numel()))

    def _new_state(self):
        def z(dtype, blocks=False):
            return [torch.zeros((-(-p.numel() // BLOCK),) if blocks else p.shape, dtype=dtype, device=p.device)
                    for p in self.params]

        if self.state_bits == 32:
            return dict(exp_avg=z(torch.float32), exp_avg_sq=z(torch.float32))
        return dict(exp_avg=z(torch.uint8), exp_avg_sq=z(torch.uint8), avg_scale=z(torch.float32, True),
                    avg_sq_scale=z(torch.float32, True))

    def step(self, grads, grad_scale=None, skip=None):
        """One step with one gradient per parameter (fp32 or bf16, all the
        same).  grad_scale (fp32 [1], device): a factor on every gradient.
        skip (int32 [1], device): nothing changes when it is not 0.  The step
        counts in ``steps`` and ``step_dev``, but the bias corrections (and
        the rounding's bits) go by the updates made: see ``updates``."""
        grads = list(grads)
        self._refresh()
        try:
            dts = {g.dtype for g in grads}
            gdt = dts.pop() if len(dts) == 1 else None
            ok = (gdt in _FLOATS and list(map(_NUMEL, grads)) == self._numel and all(map(_CONTIGUOUS, grads))
                  and set(map(_DEVICE, grads)) == {self.params[0].get_device()})
        except (AttributeError, TypeError):  # not a tensor
            ok = False
        if not ok:  # say which
            self._take()
            self._same_sizes("grads", grads, _FLOATS, required=True)
            if any(g.dtype != grads[0].dtype for g in grads):
                raise ValueError("grads: one dtype for all")
            _on_device(self.params[0], *grads)
        self._words[1::_WORDS] = list(map(_PTR, grads))
        for name, t, dt in (("grad_scale", grad_scale, torch.float32), ("skip", skip, torch.int32)):
            if t is not None and (t.dtype != dt or t.numel() != 1):
                raise ValueError("%s: one %s on the GPU" % (name, dt))
        with _on_device(self.params[0], grad_scale, skip):
            if self.step_dev is None and _capturing():
                raise RuntimeError("AdamW: a step that is captured needs capturable=True (replays would all be step %d)"
                                   % (self.steps + 1))
            self._skips = self._skips or skip is not None
            t_dev = self._next + (self.steps if self.step_dev is None else self.step_dev) if self._skips else None
            rc = _lib.load().adamw_step(self._list, len(grads), _DT[self.params[0].dtype], _DT[gdt],
                                        self.state_bits, self.lr, self.betas[0], self.betas[1], self.eps,
                                        self.weight_decay, self.steps + 1, _ptr(t_dev), _ptr(self.lr_dev),
                                        _ptr(grad_scale), _ptr(skip), self.seed, _stream())
            _check("adamw_step", rc)
            self.steps += 1  # (a step that was refused does not count)
            if self.step_dev is not None:
                self.step_dev.add_(1)
            if skip is not None:
                self._next.add_(skip.view(1).ne(0), alpha=-1)

    def updates(self):
        """The steps that were not skipped (those of ``step=`` included): what
        ``step=`` of an optimizer that goes on with these moments takes.
        Waits for the GPU."""
        return (self.steps if self.step_dev is None else self.step_dev.item()) + self._next.item() - 1

    def state_values(self, out=None):
        """The moments as fp32 tensors, two lists (exp_avg, exp_avg_sq):
        written to ``out`` (two lists of fp32 tensors) when given.  With fp32
        moments and no ``out`` these are the moments themselves."""
        self._refresh()
        if out is None:
            if self.state_bits == 32:
                return list(self.state["exp_avg"]), list(self.state["exp_avg_sq"])
            out = tuple([torch.empty(p.shape, dtype=torch.float32, device=p.device) for p in self.params]
                        for _ in range(2))
        if len(out) != 2:
            raise ValueError("out: two lists, got %d" % len(out))
        for t in out:
            self._same_sizes("out", t, torch.float32, required=True)
        if self.state_bits == 32:
            for d, s in zip((*out[0], *out[1]), (*self.state["exp_avg"], *self.state["exp_avg_sq"])):
                d.copy_(s.view(d.shape))
            return out
        with _on_device(self.params[0], *out[0], *out[1]):
            ptrs = [(ctypes.c_void_p * len(t))(*[x.data_ptr() for x in t]) for t in out]
            rc = _lib.load().adamw_read_state(self._list, len(self.params), ptrs[0], ptrs[1], _stream())
        _check("adamw_read_state", rc)
        return out
