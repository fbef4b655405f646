"""Thin Python binding of the nvfp4moe C ABI.

Same names as the C entry points.  torch supplies device memory (outputs are
allocated here with torch.empty) and the current HIP stream; every step of
the computation runs in the library's HIP kernels.  Argument marshalling
only: no arithmetic happens in Python.
"""

import contextlib

import torch

from . import _lib

F32, BF16, U8 = _lib.F32, _lib.BF16, _lib.U8
NT, NN, TN = _lib.NT, _lib.NN, _lib.TN

_DT = {torch.float32: F32, torch.bfloat16: BF16, torch.uint8: U8}
_TORCH = {F32: torch.float32, BF16: torch.bfloat16, U8: torch.uint8}


class NVFP4MoEError(RuntimeError):
    def __init__(self, fn, rc):
        super().__init__("%s failed: %s (%d)" % (fn, _lib.status_string(rc), rc))
        self.rc = rc


def _check(fn, rc):
    if rc != _lib.OK:
        raise NVFP4MoEError(fn, rc)


def _ptr(t):
    return None if t is None else t.data_ptr()


# torch's handle of the current stream, without the Stream object that
# torch.cuda.current_stream() builds (which takes longer than the rest of a
# small operator's call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream():
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(_device())


def _dev(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("nvfp4moe ops take GPU tensors")
            if not t.is_contiguous():
                raise ValueError("nvfp4moe ops take contiguous tensors")


def _need(t, name, dtype, *shape):
    """Checks one argument: dtype (or one of several) and shape (None: any extent)."""
    if t is None:
        return
    dt, sh = t.dtype, t.shape
    if dt is not dtype and (isinstance(dtype, torch.dtype) or dt not in dtype):
        raise ValueError("%s: dtype %s is not supported" % (name, dt))
    if sh != shape:
        ok = len(sh) == len(shape)
        for n, m in zip(shape, sh):
            if n is not None and n != m:
                ok = False
        if not ok:
            raise ValueError("%s: shape %s, expected %s" % (name, tuple(sh), tuple(shape)))


_SAME_DEVICE = contextlib.nullcontext()


def _on_device(first, *ts):
    """Checks that the tensors are contiguous and share one GPU, and returns a
    context in which that GPU is the current one (its current stream is then
    the one the library is given)."""
    dev = first.get_device()
    ok = dev >= 0 and first.is_contiguous()
    for t in ts:
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            ok = False
    if not ok:
        _dev(first, *ts)
        raise ValueError("nvfp4moe ops take tensors of one GPU, got %s"
                         % sorted({str(t.device) for t in (first, *ts) if t is not None}))
    return _SAME_DEVICE if dev == _device() else torch.cuda.device(dev)


_FLOATS = (torch.float32, torch.bfloat16)


def _dt_code(t, name="out"):
    if t.dtype not in _FLOATS:
        raise ValueError("%s: dtype %s is not supported" % (name, t.dtype))
    return _DT[t.dtype]


def nvfp4_quantize(x, groups=1, amax_in=None, amax_out=None, q=None, scales=None, gscale=None):
    """NVFP4-quantize a [rows, K] fp32/bf16 tensor.  Returns (q, scales,
    gscale, amax) where amax is amax_in when given, else the computed one."""
    _dev(x, amax_in, amax_out, q, scales, gscale)
    rows, K = x.shape
    dev = x.device
    q = torch.empty((rows, K // 2), dtype=torch.uint8, device=dev) if q is None else q
    scales = torch.empty((rows, K // 16), dtype=torch.uint8, device=dev) if scales is None else scales
    gscale = torch.empty((groups,), dtype=torch.float32, device=dev) if gscale is None else gscale
    if amax_in is None and amax_out is None:
        amax_out = torch.empty((groups,), dtype=torch.float32, device=dev)
    lib = _lib.load()
    rc = lib.nvfp4_quantize(_ptr(x), _DT[x.dtype], rows, K, groups, _ptr(amax_in), _ptr(amax_out),
                            _ptr(q), _ptr(scales), _ptr(gscale), None, _stream())
    _check("nvfp4_quantize", rc)
    return q, scales, gscale, (amax_in if amax_in is not None else amax_out)



def nvfp4_quantize_onepass(x, groups=1, amax_out=None, q=None, scales=None, gscale=None, workspace=None):
    """nvfp4_quantize with the amax of each group computed, x read once
    (same outputs).  Returns (q, scales, gscale, amax)."""
    _dev(x, amax_out, q, scales, gscale, workspace)
    rows, K = x.shape
    dev = x.device
    q = torch.empty((rows, K // 2), dtype=torch.uint8, device=dev) if q is None else q
    scales = torch.empty((rows, K // 16), dtype=torch.uint8, device=dev) if scales is None else scales
    gscale = torch.empty((groups,), dtype=torch.float32, device=dev) if gscale is None else gscale
    amax_out = torch.empty((groups,), dtype=torch.float32, device=dev) if amax_out is None else amax_out
    lib = _lib.load()
    ws_bytes = lib.nvfp4_quantize_onepass_workspace_size(rows, K, groups)
    if workspace is None:
        workspace = torch.empty((max(ws_bytes, 1),), dtype=torch.uint8, device=dev)
    rc = lib.nvfp4_quantize_onepass(_ptr(x), _DT[x.dtype], rows, K, groups, _ptr(amax_out), _ptr(q), _ptr(scales),
                                    _ptr(gscale), _ptr(workspace), workspace.numel(), _stream())
    _check("nvfp4_quantize_onepass", rc)
    return q, scales, gscale, amax_out


ROUTER_TOPK_SOFTMAX, ROUTER_SOFTMAX = _lib.ROUTER_TOPK_SOFTMAX, _lib.ROUTER_SOFTMAX


def moe_router(logits, k, bias=None, score=ROUTER_TOPK_SOFTMAX, scale=1.0, want_lse=False, want_prob_sum=False,
               topk_ids=None, topk_w=None, lse=None, prob_sum=None, workspace=None):
    """Top-k experts of logits [T, E] (fp32 or bf16; plus the fp32 selection
    bias [E]) and their softmax weights.  Returns a dict with topk_ids [T, k]
    int32, topk_w [T, k] fp32, lse [T] and prob_sum [E] (None unless wanted
    or given)."""
    _need(logits, "logits", _FLOATS, None, None)
    T, E = logits.shape
    _need(bias, "bias", torch.float32, E)
    _need(topk_ids, "topk_ids", torch.int32, T, k)
    _need(topk_w, "topk_w", torch.float32, T, k)
    _need(lse, "lse", torch.float32, T)
    _need(prob_sum, "prob_sum", torch.float32, E)
    with _on_device(logits, bias, topk_ids, topk_w, lse, prob_sum, workspace):
        new, f32 = logits.new_empty, torch.float32
        topk_ids = new((T, k), dtype=torch.int32) if topk_ids is None else topk_ids
        topk_w = new((T, k), dtype=f32) if topk_w is None else topk_w
        if lse is None and want_lse:
            lse = new((T,), dtype=f32)
        if prob_sum is None and want_prob_sum:
            prob_sum = new((E,), dtype=f32)
        lib = _lib.load()
        ws_bytes = 0
        if prob_sum is not None:
            if workspace is None:
                workspace = new((lib.moe_router_workspace_size(T, E, k),), dtype=torch.uint8)
            ws_bytes = workspace.numel() * workspace.element_size()
        rc = lib.moe_router(_ptr(logits), _DT[logits.dtype], T, E, k, _ptr(bias), score, scale, _ptr(topk_ids),
                            _ptr(topk_w), _ptr(lse), _ptr(prob_sum), _ptr(workspace), ws_bytes, _stream())
    _check("moe_router", rc)
    return dict(topk_ids=topk_ids, topk_w=topk_w, lse=lse, prob_sum=prob_sum)


def moe_router_bwd(logits, topk_ids, d_topk_w, score=ROUTER_TOPK_SOFTMAX, scale=1.0, lse=None, d_lse=None,
                   d_prob_sum=None, out=None, out_dtype=None):
    """Gradient of moe_router's topk_w, lse and prob_sum with respect to the
    logits (d_topk_w, d_lse, d_prob_sum: None for zeros).  Returns d_logits
    [T, E] of out_dtype (default: the logits' dtype), written to out when given
    (which must not overlap the logits)."""
    _need(logits, "logits", _FLOATS, None, None)
    T, E = logits.shape
    _need(topk_ids, "topk_ids", torch.int32, T, None)
    k = topk_ids.shape[1]
    _need(d_topk_w, "d_topk_w", torch.float32, T, k)
    _need(lse, "lse", torch.float32, T)
    _need(d_lse, "d_lse", torch.float32, T)
    _need(d_prob_sum, "d_prob_sum", torch.float32, E)
    _need(out, "out", _FLOATS, T, E)
    with _on_device(logits, topk_ids, d_topk_w, lse, d_lse, d_prob_sum, out):
        if out is None:
            out = logits.new_empty((T, E), dtype=out_dtype)
        rc = _lib.load().moe_router_bwd(_ptr(logits), _DT[logits.dtype], T, E, k, _ptr(topk_ids), score, scale,
                                        _ptr(d_topk_w), _ptr(lse), _ptr(d_lse), _ptr(d_prob_sum), _ptr(out),
                                        _DT[out.dtype], _stream())
    _check("moe_router_bwd", rc)
    return out


def moe_permute_workspace_size(T, k, E):
    return _lib.load().moe_permute_workspace_size(T, k, E)


def moe_permute(topk_ids, num_experts, x=None, x_perm=None, amax_out=None, want_amax=False, status=None,
                workspace=None):
    """Routing metadata (offsets, dest, src) and the optional gather of x
    rows into the contiguous per-expert layout.  Returns a dict."""
    _dev(topk_ids, x, x_perm, amax_out, status)
    T, k = topk_ids.shape
    dev = topk_ids.device
    R = T * k
    offsets = torch.empty((num_experts + 1,), dtype=torch.int32, device=dev)
    dest = torch.empty((R,), dtype=torch.int32, device=dev)
    src = torch.empty((R,), dtype=torch.int32, device=dev)
    lib = _lib.load()
    ws_bytes = lib.moe_permute_workspace_size(T, k, num_experts)
    if workspace is None:
        workspace = torch.empty((max(ws_bytes, 1),), dtype=torch.uint8, device=dev)
    row_elems = 0
    x_dtype = BF16
    if x is not None:
        row_elems = x.shape[1] if x.dim() == 2 else x[0].numel()
        x_dtype = _DT[x.dtype]
        if x_perm is None:
            x_perm = torch.empty((R,) + tuple(x.shape[1:]), dtype=x.dtype, device=dev)
        if want_amax and amax_out is None:
            amax_out = torch.empty((1,), dtype=torch.float32, device=dev)
    rc = lib.moe_permute(_ptr(topk_ids), T, k, num_experts, _ptr(x), x_dtype, row_elems, _ptr(x_perm),
                         _ptr(offsets), _ptr(dest), _ptr(src), _ptr(amax_out), _ptr(workspace),
                         workspace.numel(), _ptr(status), _stream())
    _check("moe_permute", rc)
    return dict(offsets=offsets, dest=dest, src=src, x_perm=x_perm, amax=amax_out)



def moe_permute_mx(topk_ids, num_experts, x, q=None, scales=None, status=None, workspace=None):
    """moe_permute fused with the MXFP8 (E4M3) quantization of the permuted
    rows: codes [T*k, D] and E8M0 scales [T*k, D/32].  Returns a dict with
    offsets, dest, src, q and scales."""
    _dev(topk_ids, x, q, scales, status, workspace)
    T, k = topk_ids.shape
    D = x.shape[1]
    dev = x.device
    R = T * k
    lib = _lib.load()
    offsets = torch.empty((num_experts + 1,), dtype=torch.int32, device=dev)
    dest = torch.empty((R,), dtype=torch.int32, device=dev)
    src = torch.empty((R,), dtype=torch.int32, device=dev)
    q = torch.empty((R, D), dtype=torch.uint8, device=dev) if q is None else q
    scales = torch.empty((R, D // 32), dtype=torch.uint8, device=dev) if scales is None else scales
    ws_bytes = lib.moe_permute_workspace_size(T, k, num_experts)
    if workspace is None:
        workspace = torch.empty((max(ws_bytes, 1),), dtype=torch.uint8, device=dev)
    rc = lib.moe_permute_mx(_ptr(topk_ids), T, k, num_experts, _ptr(x), _DT[x.dtype], D, _ptr(q), _ptr(scales),
                            _ptr(offsets), _ptr(dest), _ptr(src), _ptr(workspace), workspace.numel(), _ptr(status),
                            _stream())
    _check("moe_permute_mx", rc)
    return dict(offsets=offsets, dest=dest, src=src, q=q, scales=scales)


def moe_permute_mxfp4(topk_ids, num_experts, x, q=None, scales=None, status=None, workspace=None):
    """moe_permute fused with the MXFP4 (E2M1) quantization of the permuted
    rows: codes [T*k, D/2] and E8M0 scales [T*k, D/32].  Returns a dict with
    offsets, dest, src, q and scales."""
    _need(topk_ids, "topk_ids", torch.int32, None, None)
    T, k = topk_ids.shape
    _need(x, "x", _FLOATS, T, None)
    D, R = x.shape[1], T * k
    _need(q, "q", torch.uint8, R, D // 2)
    _need(scales, "scales", torch.uint8, R, D // 32)
    if status is not None and (status.dtype != torch.int32 or status.numel() < 1):
        raise ValueError("status: one int32 on the GPU")
    with _on_device(topk_ids, x, q, scales, status, workspace):
        dev, i32, u8 = x.device, torch.int32, torch.uint8
        lib = _lib.load()
        offsets = torch.empty((num_experts + 1,), dtype=i32, device=dev)
        dest = torch.empty((R,), dtype=i32, device=dev)
        src = torch.empty((R,), dtype=i32, device=dev)
        q = torch.empty((R, D // 2), dtype=u8, device=dev) if q is None else q
        scales = torch.empty((R, D // 32), dtype=u8, device=dev) if scales is None else scales
        if workspace is None:
            workspace = torch.empty((max(lib.moe_permute_workspace_size(T, k, num_experts), 1),), dtype=u8, device=dev)
        rc = lib.moe_permute_mxfp4(_ptr(topk_ids), T, k, num_experts, _ptr(x), _DT[x.dtype], D, _ptr(q),
                                   _ptr(scales), _ptr(offsets), _ptr(dest), _ptr(src), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _ptr(status), _stream())
    _check("moe_permute_mxfp4", rc)
    return dict(offsets=offsets, dest=dest, src=src, q=q, scales=scales)


def moe_permute_int8(topk_ids, num_experts, x, q=None, scales=None, status=None, workspace=None):
    """moe_permute fused with the 8-bit integer quantization of the permuted
    rows: codes [T*k, D] int8 and scales [T*k] fp32.  Returns a dict with
    offsets, dest, src, q and scales."""
    _need(topk_ids, "topk_ids", torch.int32, None, None)
    T, k = topk_ids.shape
    _need(x, "x", _FLOATS, T, None)
    D, R = x.shape[1], T * k
    _need(q, "q", torch.int8, R, D)
    _need(scales, "scales", torch.float32, R)
    if status is not None and (status.dtype != torch.int32 or status.numel() < 1):
        raise ValueError("status: one int32 on the GPU")
    with _on_device(topk_ids, x, q, scales, status, workspace):
        new, i32 = x.new_empty, torch.int32
        lib = _lib.load()
        offsets, dest, src = new((num_experts + 1,), dtype=i32), new((R,), dtype=i32), new((R,), dtype=i32)
        q = new((R, D), dtype=torch.int8) if q is None else q
        scales = new((R,), dtype=torch.float32) if scales is None else scales
        if workspace is None:
            workspace = new((max(lib.moe_permute_workspace_size(T, k, num_experts), 1),), dtype=torch.uint8)
        rc = lib.moe_permute_int8(_ptr(topk_ids), T, k, num_experts, _ptr(x), _DT[x.dtype], D, _ptr(q), _ptr(scales),
                                  _ptr(offsets), _ptr(dest), _ptr(src), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _ptr(status), _stream())
    _check("moe_permute_int8", rc)
    return dict(offsets=offsets, dest=dest, src=src, q=q, scales=scales)


def moe_permute_nvfp4(topk_ids, num_experts, x, x_perm=None, want_x_perm=True, amax_in=None, amax_out=None,
                      q=None, scales=None, gscale=None, status=None, workspace=None):
    """moe_permute fused with the NVFP4 quantization of the gathered rows.
    Returns a dict with offsets, dest, src, x_perm (or None), q, scales,
    gscale and amax."""
    _dev(topk_ids, x, x_perm, amax_in, amax_out, q, scales, gscale, status)
    T, k = topk_ids.shape
    D = x.shape[1]
    dev = x.device
    R = T * k
    lib = _lib.load()
    offsets = torch.empty((num_experts + 1,), dtype=torch.int32, device=dev)
    dest = torch.empty((R,), dtype=torch.int32, device=dev)
    src = torch.empty((R,), dtype=torch.int32, device=dev)
    if x_perm is None and want_x_perm:
        x_perm = torch.empty((R, D), dtype=x.dtype, device=dev)
    q = torch.empty((R, D // 2), dtype=torch.uint8, device=dev) if q is None else q
    scales = torch.empty((R, D // 16), dtype=torch.uint8, device=dev) if scales is None else scales
    gscale = torch.empty((1,), dtype=torch.float32, device=dev) if gscale is None else gscale
    if amax_in is None and amax_out is None:
        amax_out = torch.empty((1,), dtype=torch.float32, device=dev)
    ws_bytes = lib.moe_permute_workspace_size(T, k, num_experts)
    if workspace is None:
        workspace = torch.empty((max(ws_bytes, 1),), dtype=torch.uint8, device=dev)
    if x.dtype != torch.bfloat16:
        raise ValueError("moe_permute_nvfp4 takes bf16 activations")
    rc = lib.moe_permute_nvfp4(_ptr(topk_ids), T, k, num_experts, _ptr(x), D, _ptr(x_perm), _ptr(amax_in),
                               _ptr(amax_out), _ptr(q), _ptr(scales), _ptr(gscale), _ptr(offsets), _ptr(dest),
                               _ptr(src), _ptr(workspace), workspace.numel(), _ptr(status), _stream())
    _check("moe_permute_nvfp4", rc)
    return dict(offsets=offsets, dest=dest, src=src, x_perm=x_perm, q=q, scales=scales, gscale=gscale,
                amax=amax_in if amax_in is not None else amax_out)


def moe_permute_nvfp4_noalloc(topk_ids, num_experts, x, x_perm=None, want_x_perm=True, amax_in=None,
                              amax_out=None, q=None, scales=None, gscale=None, status=None):
    """moe_permute_nvfp4 without a workspace: the library's own per-GPU
    scratch array holds the histograms (for callers that cannot allocate;
    every output buffer passed in is written, nothing else is allocated by
    the library).  Calls on one GPU must not overlap in time."""
    _dev(topk_ids, x, x_perm, amax_in, amax_out, q, scales, gscale, status)
    T, k = topk_ids.shape
    D = x.shape[1]
    dev = x.device
    R = T * k
    offsets = torch.empty((num_experts + 1,), dtype=torch.int32, device=dev)
    dest = torch.empty((R,), dtype=torch.int32, device=dev)
    src = torch.empty((R,), dtype=torch.int32, device=dev)
    if x_perm is None and want_x_perm:
        x_perm = torch.empty((R, D), dtype=x.dtype, device=dev)
    q = torch.empty((R, D // 2), dtype=torch.uint8, device=dev) if q is None else q
    scales = torch.empty((R, D // 16), dtype=torch.uint8, device=dev) if scales is None else scales
    gscale = torch.empty((1,), dtype=torch.float32, device=dev) if gscale is None else gscale
    if amax_in is None and amax_out is None:
        amax_out = torch.empty((1,), dtype=torch.float32, device=dev)
    if x.dtype != torch.bfloat16:
        raise ValueError("moe_permute_nvfp4_noalloc takes bf16 activations")
    rc = _lib.load().moe_permute_nvfp4_noalloc(_ptr(topk_ids), T, k, num_experts, _ptr(x), D, _ptr(x_perm),
                                               _ptr(amax_in), _ptr(amax_out), _ptr(q), _ptr(scales), _ptr(gscale),
                                               _ptr(offsets), _ptr(dest), _ptr(src), _ptr(status), _stream())
    _check("moe_permute_nvfp4_noalloc", rc)
    return dict(offsets=offsets, dest=dest, src=src, x_perm=x_perm, q=q, scales=scales, gscale=gscale,
                amax=amax_in if amax_in is not None else amax_out)


def moe_gather(x, src, k, topk_w=None, out=None, out_dtype=None):
    """out[p] = w[src[p]] * x[src[p] // k] (a verbatim row copy when no weights)."""
    _dev(x, src, topk_w, out)
    R = src.numel()
    row_elems = x.shape[1] if x.dim() == 2 else x[0].numel()
    odt = x.dtype if out_dtype is None else out_dtype
    out = torch.empty((R,) + tuple(x.shape[1:]), dtype=odt, device=x.device) if out is None else out
    rc = _lib.load().moe_gather(_ptr(x), _DT[x.dtype], row_elems, _ptr(src), _ptr(topk_w), k, R, _ptr(out),
                                _DT[out.dtype], _stream())
    _check("moe_gather", rc)
    return out


def moe_scatter(x, dest, offsets, k, topk_w=None, out=None, out_dtype=None, amax_out=None):
    """out[dest[t*k+j]] = w[t*k+j] * x[t]: the weighted gather written from the
    token side (each row of x read once); rows past offsets[E] are zeros.
    amax_out (fp32 [1], optional) receives max |out|."""
    _dev(x, dest, offsets, topk_w, out, amax_out)
    T = x.shape[0]
    R = T * k
    E = offsets.numel() - 1
    row_elems = x.shape[1] if x.dim() == 2 else x[0].numel()
    odt = x.dtype if out_dtype is None else out_dtype
    out = torch.empty((R,) + tuple(x.shape[1:]), dtype=odt, device=x.device) if out is None else out
    rc = _lib.load().moe_scatter(_ptr(x), _DT[x.dtype], row_elems, _ptr(dest), _ptr(topk_w), _ptr(offsets), E, T,
                                 k, _ptr(out), _DT[out.dtype], _ptr(amax_out), _stream())
    _check("moe_scatter", rc)
    return out


def moe_unpermute(y_perm, dest, T, k, topk_w=None, out=None, out_dtype=torch.bfloat16):
    """out[t] = sum_j w[t, j] * y_perm[dest[t*k + j]]."""
    _dev(y_perm, dest, topk_w, out)
    D = y_perm.shape[1]
    out = torch.empty((T, D), dtype=out_dtype, device=y_perm.device) if out is None else out
    rc = _lib.load().moe_unpermute(_ptr(y_perm), _DT[y_perm.dtype], _ptr(dest), _ptr(topk_w), T, k, D, _ptr(out),
                                   _DT[out.dtype], _stream())
    _check("moe_unpermute", rc)
    return out


def moe_unpermute_bwd(dout, y_perm, dest, offsets, k, topk_w=None, dy_perm=None, want_dy=True, dy_dtype=None,
                      d_topk_w=None, want_dw=True, amax_out=None):
    """Gradient of moe_unpermute in one pass: dy_perm[dest[t*k+j]] = w[t, j] *
    dout[t] (rows past offsets[E] are zeros) and d_topk_w[t, j] =
    <dout[t], y_perm[dest[t*k+j]]> (fp32).  y_perm may be None without the
    weight gradient.  amax_out (fp32 [1], optional) receives max |dy_perm|.
    dy_perm must not overlap dout or y_perm.  Returns (dy_perm or None,
    d_topk_w or None)."""
    _need(dout, "dout", _FLOATS, None, None)
    T, D = dout.shape
    R = T * k
    want_dw = want_dw or d_topk_w is not None
    want_dy = want_dy or dy_perm is not None
    if want_dw and y_perm is None:
        raise ValueError("the weight gradient needs y_perm")
    _need(y_perm, "y_perm", _FLOATS, R, D)
    _need(dest, "dest", torch.int32, R)
    _need(offsets, "offsets", torch.int32, None)
    _need(topk_w, "topk_w", torch.float32, T, k)
    _need(dy_perm, "dy_perm", _FLOATS, R, D)
    _need(d_topk_w, "d_topk_w", torch.float32, T, k)
    _need(amax_out, "amax_out", torch.float32, 1)
    with _on_device(dout, y_perm, dest, offsets, topk_w, dy_perm, d_topk_w, amax_out):
        if dy_perm is None and want_dy:
            dy_perm = dout.new_empty((R, D), dtype=dy_dtype)
        if d_topk_w is None and want_dw:
            d_topk_w = dout.new_empty((T, k), dtype=torch.float32)
        rc = _lib.load().moe_unpermute_bwd(
            _ptr(dout), _DT[dout.dtype], _ptr(y_perm), _DT[y_perm.dtype] if y_perm is not None else BF16, _ptr(dest),
            _ptr(topk_w), _ptr(offsets), offsets.numel() - 1, T, k, D, _ptr(dy_perm),
            _DT[dy_perm.dtype] if dy_perm is not None else BF16, _ptr(d_topk_w), _ptr(amax_out), _stream())
    _check("moe_unpermute_bwd", rc)
    return dy_perm, d_topk_w


def grouped_gemm_w4a4(a_q, a_s, a_g, b_q, b_s, b_g, offsets, out=None, out_dtype=torch.float32):
    """C[r] = a_g * b_g[e] * deq(A)[r] . deq(B_e)^T for rows r of expert e."""
    _dev(a_q, a_s, a_g, b_q, b_s, b_g, offsets, out)
    M = a_q.shape[0]
    K = a_q.shape[1] * 2
    E, N = b_q.shape[0], b_q.shape[1]
    out = torch.empty((M, N), dtype=out_dtype, device=a_q.device) if out is None else out
    rc = _lib.load().grouped_gemm_w4a4(_ptr(a_q), _ptr(a_s), _ptr(a_g), _ptr(b_q), _ptr(b_s), _ptr(b_g),
                                       _ptr(offsets), E, M, N, K, _ptr(out), _DT[out.dtype], _lib.EPI_NONE,
                                       None, None, 0, _stream())
    _check("grouped_gemm_w4a4", rc)
    return out


def grouped_gemm_w4a4_scaled_mfma(a_q, a_s, a_g, b_q, b_s, b_g, offsets, out=None, out_dtype=torch.float32):
    """grouped_gemm_w4a4 by scale factoring onto the fp4 scaled MFMA (the
    alternative design, for measurement)."""
    _dev(a_q, a_s, a_g, b_q, b_s, b_g, offsets, out)
    M = a_q.shape[0]
    K = a_q.shape[1] * 2
    E, N = b_q.shape[0], b_q.shape[1]
    out = torch.empty((M, N), dtype=out_dtype, device=a_q.device) if out is None else out
    rc = _lib.load().grouped_gemm_w4a4_scaled_mfma(_ptr(a_q), _ptr(a_s), _ptr(a_g), _ptr(b_q), _ptr(b_s), _ptr(b_g),
                                                   _ptr(offsets), E, M, N, K, _ptr(out), _DT[out.dtype], _stream())
    _check("grouped_gemm_w4a4_scaled_mfma", rc)
    return out


def grouped_gemm_w4a4_silu_gate(a_q, a_s, a_g, b_q, b_s, b_g, offsets, y1=None, want_y1=True, h=None,
                                amax_out=None, want_amax=True):
    """Gate+up W4A4 GEMM with the SiLU gate (and amax of H) in its epilogue.
    B_e = [gate; up] rows.  Returns (y1 or None, h, amax or None)."""
    _dev(a_q, a_s, a_g, b_q, b_s, b_g, offsets, y1, h, amax_out)
    M = a_q.shape[0]
    K = a_q.shape[1] * 2
    E, N = b_q.shape[0], b_q.shape[1]
    F = N // 2
    dev = a_q.device
    if y1 is None and want_y1:
        y1 = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    h = torch.empty((M, F), dtype=torch.bfloat16, device=dev) if h is None else h
    if amax_out is None and want_amax:
        amax_out = torch.empty(1, dtype=torch.float32, device=dev)
    rc = _lib.load().grouped_gemm_w4a4_silu_gate(_ptr(a_q), _ptr(a_s), _ptr(a_g), _ptr(b_q), _ptr(b_s), _ptr(b_g),
                                                 _ptr(offsets), E, M, F, K, _ptr(y1), _ptr(h), _ptr(amax_out),
                                                 _stream())
    _check("grouped_gemm_w4a4_silu_gate", rc)
    return y1, h, amax_out


def grouped_gemm_w4a4_silu_gate_nvfp4(a_q, a_s, a_g, b_q, b_s, b_g, offsets, amax_h_in, y1=None, h=None,
                                      amax_out=None, want_amax=True, q_h=None, s_h=None, g_h=None):
    """Gate+up W4A4 GEMM with the SiLU gate and the NVFP4 requantization of
    H (with the handed-in amax_h_in) in its epilogue.  Returns (q_h, s_h,
    g_h, amax or None); y1 and h are stored only when given."""
    _dev(a_q, a_s, a_g, b_q, b_s, b_g, offsets, amax_h_in, y1, h, amax_out, q_h, s_h, g_h)
    M = a_q.shape[0]
    K = a_q.shape[1] * 2
    E, N = b_q.shape[0], b_q.shape[1]
    F = N // 2
    dev = a_q.device
    q_h = torch.empty((M, F // 2), dtype=torch.uint8, device=dev) if q_h is None else q_h
    s_h = torch.empty((M, F // 16), dtype=torch.uint8, device=dev) if s_h is None else s_h
    g_h = torch.empty((1,), dtype=torch.float32, device=dev) if g_h is None else g_h
    if amax_out is None and want_amax:
        amax_out = torch.empty(1, dtype=torch.float32, device=dev)
    rc = _lib.load().grouped_gemm_w4a4_silu_gate_nvfp4(
        _ptr(a_q), _ptr(a_s), _ptr(a_g), _ptr(b_q), _ptr(b_s), _ptr(b_g), _ptr(offsets), E, M, F, K, _ptr(y1),
        _ptr(h), _ptr(amax_out), _ptr(amax_h_in), _ptr(q_h), _ptr(s_h), _ptr(g_h), _stream())
    _check("grouped_gemm_w4a4_silu_gate_nvfp4", rc)
    return q_h, s_h, g_h, amax_out


def padded_extent(M_total, E):
    """Row length of the column-wise layout: 64 * (M_total // 64 + E)."""
    return 64 * (M_total // 64 + E)


def nvfp4_quantize_colwise(x, offsets, amax_in, Kp=None, q_t=None, s_t=None, gscale=None):
    """Column-wise NVFP4 of a row-grouped [M_total, N] bf16 tensor, stored
    transposed ([N, Kp/2] codes, [N, Kp/16] scales; expert e's segment at
    column 64 * (offsets[e] // 64 + e)).  Returns (q_t, s_t, gscale)."""
    _dev(x, offsets, amax_in, q_t, s_t, gscale)
    M, N = x.shape
    E = offsets.numel() - 1
    Kp = padded_extent(M, E) if Kp is None else Kp
    dev = x.device
    q_t = torch.empty((N, Kp // 2), dtype=torch.uint8, device=dev) if q_t is None else q_t
    s_t = torch.empty((N, Kp // 16), dtype=torch.uint8, device=dev) if s_t is None else s_t
    gscale = torch.empty((1,), dtype=torch.float32, device=dev) if gscale is None else gscale
    rc = _lib.load().nvfp4_quantize_colwise(_ptr(x), _DT[x.dtype], M, N, _ptr(offsets), E, _ptr(amax_in), _ptr(q_t),
                                            _ptr(s_t), _ptr(gscale), Kp, _stream())
    _check("nvfp4_quantize_colwise", rc)
    return q_t, s_t, gscale


def nvfp4_quantize_transposed(x, amax_in=None, amax_out=None, q_t=None, s_t=None, gscale=None):
    """NVFP4 of each matrix of x [G, L, N] along its rows' index: codes of
    the transposed matrices, q_t [G, N, L/2], s_t [G, N, L/16], gscale [G].
    Returns (q_t, s_t, gscale, amax)."""
    _dev(x, amax_in, amax_out, q_t, s_t, gscale)
    G, L, N = x.shape
    dev = x.device
    q_t = torch.empty((G, N, L // 2), dtype=torch.uint8, device=dev) if q_t is None else q_t
    s_t = torch.empty((G, N, L // 16), dtype=torch.uint8, device=dev) if s_t is None else s_t
    gscale = torch.empty((G,), dtype=torch.float32, device=dev) if gscale is None else gscale
    if amax_in is None and amax_out is None:
        amax_out = torch.empty((G,), dtype=torch.float32, device=dev)
    rc = _lib.load().nvfp4_quantize_transposed(_ptr(x), _DT[x.dtype], G, L, N, _ptr(amax_in), _ptr(amax_out),
                                               _ptr(q_t), _ptr(s_t), _ptr(gscale), _stream())
    _check("nvfp4_quantize_transposed", rc)
    return q_t, s_t, gscale, amax_in if amax_in is not None else amax_out


def grouped_gemm_w4a4_wgrad(a, b, offsets, M_total, out=None, out_dtype=torch.float32):
    """NVFP4 weight gradient: C_e = deq(A_e)^T . deq(B_e) over expert e's
    rows, a and b the (q_t, s_t, gscale) of nvfp4_quantize_colwise.
    Returns C [E, N1, N2]."""
    (aq, as_, ag), (bq, bs, bg) = a, b
    _dev(aq, as_, ag, bq, bs, bg, offsets, out)
    E = offsets.numel() - 1
    N1, Kp = aq.shape[0], aq.shape[1] * 2
    N2 = bq.shape[0]
    out = torch.empty((E, N1, N2), dtype=out_dtype, device=aq.device) if out is None else out
    rc = _lib.load().grouped_gemm_w4a4_wgrad(_ptr(aq), _ptr(as_), _ptr(ag), _ptr(bq), _ptr(bs), _ptr(bg),
                                             _ptr(offsets), E, M_total, Kp, N1, N2, _ptr(out), _DT[out.dtype],
                                             _stream())
    _check("grouped_gemm_w4a4_wgrad", rc)
    return out


MX_E4M3, MX_E2M1, MX_INT8 = _lib.MX_E4M3, _lib.MX_E2M1, _lib.MX_INT8


def mx_quantize(x, elem=MX_E4M3, q=None, scales=None):
    """MX-quantize a [rows, K] fp32/bf16 tensor (E8M0 scale per 32 along K):
    elem MX_E4M3 (MXFP8, one byte per element), MX_E2M1 (MXFP4, packed
    pairs) or MX_INT8 (MXINT8, one two's complement byte per element: the
    form of activations kept for the backward pass).  Returns (q, scales)."""
    _need(x, "x", _FLOATS, None, None)
    rows, K = x.shape
    qcols = K // 2 if elem == MX_E2M1 else K
    if elem == MX_INT8:
        _need(q, "q", torch.uint8, rows, K)
        _need(scales, "scales", torch.uint8, rows, K // 32)
    with _on_device(x, q, scales):
        q = x.new_empty((rows, qcols), dtype=torch.uint8) if q is None else q
        scales = x.new_empty((rows, K // 32), dtype=torch.uint8) if scales is None else scales
        rc = _lib.load().mx_quantize(_ptr(x), _DT[x.dtype], rows, K, elem, _ptr(q), _ptr(scales), _stream())
    _check("mx_quantize", rc)
    return q, scales


def mx_dequantize(q, scales, elem=MX_E4M3, out=None, out_dtype=torch.bfloat16):
    """The values [rows, K] of mx_quantize's codes (fp32 or bf16; a scale byte
    of 255 gives NaN)."""
    _need(q, "q", torch.uint8, None, None)
    rows, K = q.shape[0], q.shape[1] * (2 if elem == MX_E2M1 else 1)
    _need(scales, "scales", torch.uint8, rows, K // 32)
    _need(out, "out", _FLOATS, rows, K)
    with _on_device(q, scales, out):
        out = q.new_empty((rows, K), dtype=out_dtype) if out is None else out
        rc = _lib.load().mx_dequantize(_ptr(q), _ptr(scales), rows, K, elem, _ptr(out), _dt_code(out), _stream())
    _check("mx_dequantize", rc)
    return out


def grouped_gemm_w4a8(a_q, a_s, b_q, b_s, offsets, out=None, out_dtype=torch.float32):
    """C[r] = deq(A)[r] . deq(B_e)^T for rows r of expert e; A MXFP8 [M, K],
    B MXFP4 [E, N, K/2], E8M0 scales per 32."""
    _dev(a_q, a_s, b_q, b_s, offsets, out)
    M, K = a_q.shape
    E, N = b_q.shape[0], b_q.shape[1]
    out = torch.empty((M, N), dtype=out_dtype, device=a_q.device) if out is None else out
    rc = _lib.load().grouped_gemm_w4a8(_ptr(a_q), _ptr(a_s), _ptr(b_q), _ptr(b_s), _ptr(offsets), E, M, N, K,
                                       _ptr(out), _DT[out.dtype], _stream())
    _check("grouped_gemm_w4a8", rc)
    return out


def grouped_gemm_w4a8_silu_gate(a_q, a_s, b_q, b_s, offsets, y1=None, want_y1=True, h=None, amax_out=None,
                                want_amax=True):
    """Gate+up W4A8 GEMM with the SiLU gate (and amax of H) in its epilogue.
    Returns (y1 or None, h, amax or None)."""
    _dev(a_q, a_s, b_q, b_s, offsets, y1, h, amax_out)
    M, K = a_q.shape
    E, N = b_q.shape[0], b_q.shape[1]
    F = N // 2
    dev = a_q.device
    if y1 is None and want_y1:
        y1 = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    h = torch.empty((M, F), dtype=torch.bfloat16, device=dev) if h is None else h
    if amax_out is None and want_amax:
        amax_out = torch.empty(1, dtype=torch.float32, device=dev)
    rc = _lib.load().grouped_gemm_w4a8_silu_gate(_ptr(a_q), _ptr(a_s), _ptr(b_q), _ptr(b_s), _ptr(offsets), E, M,
                                                 F, K, _ptr(y1), _ptr(h), _ptr(amax_out), _stream())
    _check("grouped_gemm_w4a8_silu_gate", rc)
    return y1, h, amax_out


def grouped_gemm_w4a8_silu_gate_mx(a_q, a_s, b_q, b_s, offsets, q_h=None, s_h=None, y1=None, h=None,
                                   amax_out=None):
    """Gate+up W4A8 GEMM with the SiLU gate and the MXFP8 quantization of H
    in its epilogue.  y1, h (bf16) and amax_out are written only when given.
    Returns (q_h, s_h)."""
    _dev(a_q, a_s, b_q, b_s, offsets, q_h, s_h, y1, h, amax_out)
    M, K = a_q.shape
    E, N = b_q.shape[0], b_q.shape[1]
    F = N // 2
    dev = a_q.device
    q_h = torch.empty((M, F), dtype=torch.uint8, device=dev) if q_h is None else q_h
    s_h = torch.empty((M, F // 32), dtype=torch.uint8, device=dev) if s_h is None else s_h
    rc = _lib.load().grouped_gemm_w4a8_silu_gate_mx(_ptr(a_q), _ptr(a_s), _ptr(b_q), _ptr(b_s), _ptr(offsets), E,
                                                    M, F, K, _ptr(y1), _ptr(h), _ptr(amax_out), _ptr(q_h), _ptr(s_h),
                                                    _stream())
    _check("grouped_gemm_w4a8_silu_gate_mx", rc)
    return q_h, s_h


def _mxfp4_operands(a_q, a_s, b_q, b_s, offsets):
    _need(a_q, "a_q", torch.uint8, None, None)
    M, K = a_q.shape[0], a_q.shape[1] * 2
    _need(a_s, "a_s", torch.uint8, M, K // 32)
    _need(b_q, "b_q", torch.uint8, None, None, K // 2)
    E, N = b_q.shape[0], b_q.shape[1]
    _need(b_s, "b_s", torch.uint8, E, N, K // 32)
    _need(offsets, "offsets", torch.int32, E + 1)
    return M, K, E, N


def grouped_gemm_mxfp4(a_q, a_s, b_q, b_s, offsets, out=None, out_dtype=torch.float32):
    """C[r] = deq(A)[r] . deq(B_e)^T for rows r of expert e; A MXFP4
    [M, K/2], B MXFP4 [E, N, K/2], E8M0 scales per 32."""
    M, K, E, N = _mxfp4_operands(a_q, a_s, b_q, b_s, offsets)
    _need(out, "out", _FLOATS, M, N)
    with _on_device(a_q, a_s, b_q, b_s, offsets, out):
        out = a_q.new_empty((M, N), dtype=out_dtype) if out is None else out
        rc = _lib.load().grouped_gemm_mxfp4(_ptr(a_q), _ptr(a_s), _ptr(b_q), _ptr(b_s), _ptr(offsets), E, M, N, K,
                                            _ptr(out), _DT[out.dtype], _stream())
    _check("grouped_gemm_mxfp4", rc)
    return out


def grouped_gemm_mxfp4_silu_gate(a_q, a_s, b_q, b_s, offsets, y1=None, want_y1=True, h=None, want_h=True,
                                 amax_out=None, q_h=None, s_h=None, want_q=False, q_y1=None, s_y1=None,
                                 want_ckpt=False):
    """Gate+up MXFP4 GEMM (B_e = [gate; up] rows) with the SiLU gate and,
    when wanted, the MXFP4 quantization of H and the MXINT8 form of Y1 (which
    silu_gate_bwd_mx takes) in its epilogue.  Returns a dict with y1 [M, 2F]
    and h [M, F] (bf16), q_h [M, F/2], s_h [M, F/32], q_y1 [M, 2F] and s_y1
    [M, 2F/32] (None unless wanted or given).  amax_out (fp32 [1], optional)
    receives max |H|."""
    M, K, E, N = _mxfp4_operands(a_q, a_s, b_q, b_s, offsets)
    if N % 2:
        raise ValueError("b_q: gate and up rows, an even number")
    F = N // 2
    bf, u8 = torch.bfloat16, torch.uint8
    _need(y1, "y1", bf, M, N)
    _need(h, "h", bf, M, F)
    _need(amax_out, "amax_out", torch.float32, 1)
    _need(q_h, "q_h", u8, M, F // 2)
    _need(s_h, "s_h", u8, M, F // 32)
    _need(q_y1, "q_y1", u8, M, N)
    _need(s_y1, "s_y1", u8, M, N // 32)
    want_q = want_q or q_h is not None or s_h is not None
    want_ckpt = want_ckpt or q_y1 is not None or s_y1 is not None
    with _on_device(a_q, a_s, b_q, b_s, offsets, y1, h, amax_out, q_h, s_h, q_y1, s_y1):
        new = a_q.new_empty
        y1 = new((M, N), dtype=bf) if y1 is None and want_y1 else y1
        h = new((M, F), dtype=bf) if h is None and want_h else h
        if want_q:
            q_h = new((M, F // 2), dtype=u8) if q_h is None else q_h
            s_h = new((M, F // 32), dtype=u8) if s_h is None else s_h
        fn, args = "grouped_gemm_mxfp4_silu_gate", (_ptr(q_h), _ptr(s_h))
        if want_ckpt:
            q_y1 = new((M, N), dtype=u8) if q_y1 is None else q_y1
            s_y1 = new((M, N // 32), dtype=u8) if s_y1 is None else s_y1
            fn, args = fn + "_ckpt", args + (_ptr(q_y1), _ptr(s_y1))
        rc = getattr(_lib.load(), fn)(_ptr(a_q), _ptr(a_s), _ptr(b_q), _ptr(b_s), _ptr(offsets), E, M, F, K, _ptr(y1),
                                      _ptr(h), _ptr(amax_out), *args, _stream())
    _check(fn, rc)
    return dict(y1=y1, h=h, q_h=q_h, s_h=s_h, q_y1=q_y1, s_y1=s_y1)


def int8_quantize(x, q=None, scales=None):
    """8-bit integers of the rows of x [rows, K] (fp32 or bf16) with one fp32
    scale per row (amax / 127): a token's, or a weight's output channel's.
    Returns (q [rows, K] int8, scales [rows])."""
    _need(x, "x", _FLOATS, None, None)
    rows, K = x.shape
    _need(q, "q", torch.int8, rows, K)
    _need(scales, "scales", torch.float32, rows)
    with _on_device(x, q, scales):
        q = x.new_empty((rows, K), dtype=torch.int8) if q is None else q
        scales = x.new_empty((rows,), dtype=torch.float32) if scales is None else scales
        rc = _lib.load().int8_quantize(_ptr(x), _DT[x.dtype], rows, K, _ptr(q), _ptr(scales), _stream())
    _check("int8_quantize", rc)
    return q, scales


def _int8_operands(a_q, a_s, b_q, b_s, offsets):
    _need(a_q, "a_q", torch.int8, None, None)
    M, K = a_q.shape
    _need(a_s, "a_s", torch.float32, M)
    _need(b_q, "b_q", torch.int8, None, None, K)
    E, N = b_q.shape[0], b_q.shape[1]
    _need(b_s, "b_s", torch.float32, E, N)
    _need(offsets, "offsets", torch.int32, E + 1)
    return M, K, E, N


def grouped_gemm_int8(a_q, a_s, b_q, b_s, offsets, out=None, out_dtype=torch.float32):
    """C[r] = (a_q[r] . b_q[e]^T) * a_s[r] * b_s[e] for rows r of expert e:
    8-bit integers a_q [M, K], b_q [E, N, K] (exact sums), one fp32 scale per
    token a_s [M] and per channel b_s [E, N]."""
    M, K, E, N = _int8_operands(a_q, a_s, b_q, b_s, offsets)
    _need(out, "out", _FLOATS, M, N)
    with _on_device(a_q, a_s, b_q, b_s, offsets, out):
        out = a_q.new_empty((M, N), dtype=out_dtype) if out is None else out
        rc = _lib.load().grouped_gemm_int8(_ptr(a_q), _ptr(a_s), _ptr(b_q), _ptr(b_s), _ptr(offsets), E, M, N, K,
                                           _ptr(out), _dt_code(out), _stream())
    _check("grouped_gemm_int8", rc)
    return out


def grouped_gemm_int8_silu_gate(a_q, a_s, b_q, b_s, offsets, y1=None, want_y1=True, h=None, amax_out=None, q_y1=None,
                                s_y1=None, want_ckpt=False):
    """Gate+up GEMM of 8-bit integers (B_e = [gate; up] rows) with the SiLU
    gate and, when wanted, the MXINT8 form of Y1 (which silu_gate_bwd_mx takes)
    in its epilogue.  Returns a dict with y1 [M, 2F] and h [M, F] (bf16), q_y1
    [M, 2F] and s_y1 [M, 2F/32] (y1 None unless wanted or given, q_y1 and s_y1
    likewise).  amax_out (fp32 [1], optional) receives max |H|."""
    M, K, E, N = _int8_operands(a_q, a_s, b_q, b_s, offsets)
    if N % 2:
        raise ValueError("b_q: gate and up rows, an even number")
    F, bf, u8 = N // 2, torch.bfloat16, torch.uint8
    _need(y1, "y1", bf, M, N)
    _need(h, "h", bf, M, F)
    _need(amax_out, "amax_out", torch.float32, 1)
    _need(q_y1, "q_y1", u8, M, N)
    _need(s_y1, "s_y1", u8, M, N // 32)
    want_ckpt = want_ckpt or q_y1 is not None or s_y1 is not None
    with _on_device(a_q, a_s, b_q, b_s, offsets, y1, h, amax_out, q_y1, s_y1):
        new = a_q.new_empty
        y1 = new((M, N), dtype=bf) if y1 is None and want_y1 else y1
        h = new((M, F), dtype=bf) if h is None else h
        if want_ckpt:
            q_y1 = new((M, N), dtype=u8) if q_y1 is None else q_y1
            s_y1 = new((M, N // 32), dtype=u8) if s_y1 is None else s_y1
        rc = _lib.load().grouped_gemm_int8_silu_gate(_ptr(a_q), _ptr(a_s), _ptr(b_q), _ptr(b_s), _ptr(offsets), E, M,
                                                     F, K, _ptr(y1), _ptr(h), _ptr(amax_out), _ptr(q_y1), _ptr(s_y1),
                                                     _stream())
    _check("grouped_gemm_int8_silu_gate", rc)
    return dict(y1=y1, h=h, q_y1=q_y1, s_y1=s_y1)


def grouped_gemm_bf16(layout, a, b, offsets, num_experts=None, out=None, out_dtype=torch.float32, accumulate=False):
    """Grouped BF16 GEMM; layout NT / NN / TN as in the C header."""
    _need(a, "a", torch.bfloat16, None, None)
    M, K = a.shape
    E = offsets.numel() - 1 if num_experts is None else num_experts
    if layout == NT:
        _need(b, "b", torch.bfloat16, None, None, K)
        N = b.shape[1]
        shape = (M, N)
    elif layout == NN:
        _need(b, "b", torch.bfloat16, None, K, None)
        N = b.shape[2]
        shape = (M, N)
    elif layout == TN:
        _need(b, "b", torch.bfloat16, M, None)
        N = b.shape[1]
        shape = (E, K, N)
    else:
        raise ValueError("layout must be NT, NN or TN")
    if layout != TN and b.shape[0] < E:
        raise ValueError("b: %d experts, the offsets are of %d" % (b.shape[0], E))
    _dev(a, b, offsets, out)
    out = torch.empty(shape, dtype=out_dtype, device=a.device) if out is None else out
    rc = _lib.load().grouped_gemm_bf16(layout, _ptr(a), _ptr(b), _ptr(offsets), E, M, N, K, _ptr(out),
                                       _DT[out.dtype], int(bool(accumulate)), None, 0, _stream())
    _check("grouped_gemm_bf16", rc)
    return out


def grouped_gemm_bf16_tn_gather(a, b, src, k, offsets, num_experts=None, out=None, out_dtype=torch.float32,
                                accumulate=False):
    """TN weight gradient with B rows gathered: C_e = sum_{r in e} a[r]^T b[src[r] // k]."""
    _need(a, "a", torch.bfloat16, None, None)
    _need(b, "b", torch.bfloat16, None, None)
    _dev(a, b, src, offsets, out)
    M, K = a.shape
    N = b.shape[1]
    E = offsets.numel() - 1 if num_experts is None else num_experts
    out = torch.empty((E, K, N), dtype=out_dtype, device=a.device) if out is None else out
    rc = _lib.load().grouped_gemm_bf16_tn_gather(_ptr(a), _ptr(b), _ptr(src), int(k), b.shape[0], _ptr(offsets), E,
                                                 M, N, K, _ptr(out), _DT[out.dtype], int(bool(accumulate)),
                                                 _stream())
    _check("grouped_gemm_bf16_tn_gather", rc)
    return out


def silu_gate_fwd(y1, h=None, amax_out=None, want_amax=True):
    """H = silu(G) * U for y1 = [G | U]; returns (h, amax)."""
    _dev(y1, h, amax_out)
    R, F2 = y1.shape
    F = F2 // 2
    h = torch.empty((R, F), dtype=torch.bfloat16, device=y1.device) if h is None else h
    if want_amax and amax_out is None:
        amax_out = torch.empty((1,), dtype=torch.float32, device=y1.device)
    rc = _lib.load().silu_gate_fwd(_ptr(y1), R, F, _ptr(h), _ptr(amax_out), _stream())
    _check("silu_gate_fwd", rc)
    return h, amax_out


def silu_gate_bwd(y1, dh, dy1=None, amax_out=None):
    """dY1 = [dG | dU] from Y1 and dH; amax_out (fp32 [1], optional)
    receives max |dY1|."""
    _dev(y1, dh, dy1, amax_out)
    R, F2 = y1.shape
    dy1 = torch.empty((R, F2), dtype=torch.bfloat16, device=y1.device) if dy1 is None else dy1
    rc = _lib.load().silu_gate_bwd(_ptr(y1), _ptr(dh), R, F2 // 2, _ptr(dy1), _ptr(amax_out), _stream())
    _check("silu_gate_bwd", rc)
    return dy1


def silu_gate_bwd_mx(q_y1, s_y1, dh, dy1=None, h=None, want_h=True):
    """dY1 = [dG | dU] and H from Y1 kept in 8 bits (q_y1 [R, 2F], s_y1
    [R, 2F/32]: the products' want_ckpt, or mx_quantize with MX_INT8) and dH
    [R, F] bf16.  Returns (dy1, h or None); neither may overlap an input."""
    _need(dh, "dh", torch.bfloat16, None, None)
    R, F = dh.shape
    _need(q_y1, "q_y1", torch.uint8, R, 2 * F)
    _need(s_y1, "s_y1", torch.uint8, R, 2 * F // 32)
    _need(dy1, "dy1", torch.bfloat16, R, 2 * F)
    _need(h, "h", torch.bfloat16, R, F)
    with _on_device(dh, q_y1, s_y1, dy1, h):
        dy1 = dh.new_empty(R, 2 * F) if dy1 is None else dy1
        h = torch.empty_like(dh) if h is None and want_h else h
        rc = _lib.load().silu_gate_bwd_mx(_ptr(q_y1), _ptr(s_y1), _ptr(dh), R, F, _ptr(dy1), _ptr(h), _stream())
    _check("silu_gate_bwd_mx", rc)
    return dy1, h


NORM_LAYER, NORM_RMS = _lib.NORM_LAYER, _lib.NORM_RMS


def _norm_weights(w, b, D):
    """The weights' dtype code (that of both)."""
    _need(w, "w", _FLOATS, D)
    _need(b, "b", _FLOATS, D)
    if w is not None and b is not None and w.dtype != b.dtype:
        raise ValueError("w and b: one dtype, got %s and %s" % (w.dtype, b.dtype))
    t = b if w is None else w
    return F32 if t is None else _DT[t.dtype]


def layer_norm(x, w=None, b=None, eps=1e-5, kind=NORM_LAYER, y=None, out_dtype=None, want_stats=True, mean=None,
               rstd=None):
    """Layer norm of the rows of x [T, D] (fp32 or bf16): (x - mean) * rstd * w
    + b, or with kind NORM_RMS without the mean.  w, b [D]: fp32 or bf16, None
    for ones and zeros.  Returns a dict with y [T, D] (of out_dtype, default
    x's, which must not overlap x) and mean, rstd [T] fp32, which layer_norm_bwd
    takes (None unless wanted or given; mean always with NORM_RMS)."""
    _need(x, "x", _FLOATS, None, None)
    T, D = x.shape
    wdt = _norm_weights(w, b, D)
    _need(y, "y", _FLOATS, T, D)
    _need(mean, "mean", torch.float32, T)
    _need(rstd, "rstd", torch.float32, T)
    with _on_device(x, w, b, y, mean, rstd):
        y = torch.empty_like(x, dtype=out_dtype) if y is None else y
        if want_stats:
            if mean is None and kind == NORM_LAYER:
                mean = x.new_empty(T, dtype=torch.float32)
            rstd = x.new_empty(T, dtype=torch.float32) if rstd is None else rstd
        rc = _lib.load().layer_norm(_ptr(x), _DT[x.dtype], T, D, _ptr(w), _ptr(b), wdt, eps, kind, _ptr(y), _dt_code(y),
                                    _ptr(mean), _ptr(rstd), _stream())
    _check("layer_norm", rc)
    return dict(y=y, mean=mean, rstd=rstd)


def layer_norm_bwd(dy, x, w, mean, rstd, kind=NORM_LAYER, dx=None, want_dx=True, dx_dtype=None, dw=None, want_dw=None,
                   db=None, want_db=False, workspace=None):
    """Gradient of layer_norm: dx [T, D] (of dx_dtype, default x's) and, summed
    over the rows, dw and db [D] (fp32; dw is wanted when w is given, unless
    want_dw says otherwise).  dy, x [T, D] fp32 or bf16; w as in layer_norm, or
    None; mean (None with NORM_RMS) and rstd as layer_norm gave them.  Outputs
    must not overlap inputs.  Returns a dict with dx, dw and db (None unless
    wanted or given)."""
    _need(x, "x", _FLOATS, None, None)
    T, D = x.shape
    _need(dy, "dy", _FLOATS, T, D)
    wdt = _norm_weights(w, None, D)
    _need(mean, "mean", torch.float32, T)
    _need(rstd, "rstd", torch.float32, T)
    if rstd is None or (mean is None and kind == NORM_LAYER):
        raise ValueError("layer_norm_bwd needs the forward's rstd, and its mean unless kind is NORM_RMS")
    f32 = torch.float32
    _need(dx, "dx", _FLOATS, T, D)
    _need(dw, "dw", f32, D)
    _need(db, "db", f32, D)
    with _on_device(x, dy, w, mean, rstd, dx, dw, db, workspace):
        dx = torch.empty_like(x, dtype=dx_dtype) if dx is None and want_dx else dx
        odt = F32 if dx is None else _dt_code(dx, "dx")
        if dw is None and (w is not None if want_dw is None else want_dw):
            dw = x.new_empty(D, dtype=f32)
        db = x.new_empty(D, dtype=f32) if db is None and want_db else db
        lib = _lib.load()
        ws_bytes = 0
        if dw is not None or db is not None:
            if workspace is not None:
                ws_bytes = workspace.numel() * workspace.element_size()
            else:
                ws_bytes = lib.layer_norm_bwd_workspace_size(T, D)
                workspace = x.new_empty((ws_bytes,), dtype=torch.uint8) if ws_bytes else None
        rc = lib.layer_norm_bwd(_ptr(dy), _DT[dy.dtype], _ptr(x), _DT[x.dtype], T, D, _ptr(w), wdt, _ptr(mean),
                                _ptr(rstd), kind, _ptr(dx), odt, _ptr(dw),
                                _ptr(db), _ptr(workspace), ws_bytes, _stream())
    _check("layer_norm_bwd", rc)
    return dict(dx=dx, dw=dw, db=db)
