"""One MoE layer on the NVFP4 token-wise path, chained from the C-ABI entry
points (every step runs in the library's HIP kernels; this module only
orders the calls and owns the buffers).

Forward ("miniTE報告、NVFP4強化学習の安定性を検証", fourth paragraph:
contiguous layout, device-side metadata, amax reuse, grouped GEMM, fusion):
  moe_permute_nvfp4 (amax of X once, metadata, gather fused with the NVFP4
  quantization of the gathered rows; the bf16 permuted rows are kept for the
  backward's gate+up weight gradient unless it gathers them from X)  ->  grouped_gemm_w4a4_silu_gate (gate+up with the SiLU gate and
  the amax of H in its epilogue; Y1 is stored only for the backward)  ->
  nvfp4_quantize(H, amax_in=amax_H)  ->  grouped_gemm_w4a4 (down)  ->
  moe_unpermute (routing-weighted combine).  When F is not a multiple of 128
  the gate+up GEMM and silu_gate_fwd run as two launches.
Backward in BF16 (same page, first paragraph), no amax reduction at all:
  moe_scatter(dY, weighted)  ->  NN dgrad of the down projection  ->
  silu_gate_bwd  ->  TN wgrad of the down projection  ->  NN dgrad of gate+up
  ->  moe_unpermute (unweighted sum back to tokens)  ->  TN wgrad of gate+up,
  on the kept permuted rows, or with its activation rows gathered from X
  through the routing's src (grouped_gemm_bf16_tn_gather: no 268 MB copy at
  8192 tokens, measured ~0.1 ms slower than the copy's TN plus its write).
W4A8 forward (same page, third paragraph: the W4A8 variant with MXFP8
activations; MXFP4 expert weights): MX scales are per 32-element block with
no tensor amax, so X is quantized once per token and the packed rows are
permuted afterwards (quantize(permute(X)) == permute(quantize(X)) row by
row):
  mx_quantize(X, E4M3)  ->  moe_permute (metadata + gather of the code rows)
  + moe_gather (scale rows)  ->  grouped_gemm_w4a8_silu_gate  ->
  mx_quantize(H, E4M3)  ->  grouped_gemm_w4a8 (down)  ->  moe_unpermute.
MXFP4 forward (both operands in the 4-bit format that gfx950 multiplies as
stored):
  moe_permute_mxfp4  ->  grouped_gemm_mxfp4_silu_gate (H quantized in its
  epilogue)  ->  grouped_gemm_mxfp4 (down)  ->  moe_unpermute.
``Learner`` is the layer as a learner trains it: router, MXFP4 forward, BF16
backward down to the router's weights, AdamW.
"""

import torch

from . import ops, optim


def quantize_expert_weights(w):
    """NVFP4 weights of stacked experts [E, N, K] (one global scale per
    expert), each expert read once.  Runs once per optimizer step, outside
    the per-batch path."""
    E, N, K = w.shape
    q, s, g, amax = ops.nvfp4_quantize_onepass(w.reshape(E * N, K), groups=E)
    return dict(q=q.view(E, N, K // 2), s=s.view(E, N, K // 16), g=g, amax=amax)


class Buffers:
    """Device buffers of one layer step, allocated once and reused."""

    def __init__(self, T, k, E, D, F, device, backward=False):
        R = T * k
        bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
        e = lambda *s, dt=bf: torch.empty(s, dtype=dt, device=device)  # noqa: E731
        self.T, self.k, self.E, self.D, self.F = T, k, E, D, F
        self.ws = e(max(ops.moe_permute_workspace_size(T, k, E), 1), dt=u8)
        self.x_perm = e(R, D)
        self.amax = e(2, dt=f32)            # [amax_X, amax_H]
        self.a1_q, self.a1_s, self.a1_g = e(R, D // 2, dt=u8), e(R, D // 16, dt=u8), e(1, dt=f32)
        self.y1 = e(R, 2 * F)
        self.h = e(R, F)
        self.a2_q, self.a2_s, self.a2_g = e(R, F // 2, dt=u8), e(R, F // 16, dt=u8), e(1, dt=f32)
        self.y2 = e(R, D)
        self.out = e(T, D)
        if backward:
            self.dy2 = e(R, D)
            self.dh = e(R, F)
            self.dy1 = e(R, 2 * F)
            self.dx_perm = e(R, D)
            self.dx = e(T, D)
            self.dw_dn = e(E, D, F, dt=f32)
            self.dw_gu = e(E, 2 * F, D, dt=f32)


def forward(x, topk_ids, topk_w, wq_gu, wq_dn, buf, keep_y1=True, keep_x_perm=True, fuse_silu=True,
            amax_h_in=None, amax_x_in=None):
    """W4A4 MoE forward; returns the routing metadata dict.  Y1 (buf.y1) is
    written when keep_y1 and the bf16 permuted rows (buf.x_perm) when
    keep_x_perm (the BF16 backward needs Y1, and X_perm unless it gathers
    from X).

    With ``amax_h_in`` (a [1] fp32 device tensor: a delayed amax of H, e.g.
    the previous step's buf.amax[1]) H is requantized inside the gate+up
    GEMM's epilogue with that amax; bf16 H is then stored only when keep_y1
    (the backward needs it), and buf.amax[1] still receives this step's
    max |H|.  With ``amax_x_in`` ([1] fp32 device) X is quantized with that
    amax instead of its own (buf.amax[0] is then not written)."""
    E = buf.E
    meta = ops.moe_permute_nvfp4(topk_ids, E, x, x_perm=buf.x_perm if keep_x_perm else None,
                                 want_x_perm=keep_x_perm, amax_in=amax_x_in,
                                 amax_out=None if amax_x_in is not None else buf.amax[0:1], q=buf.a1_q,
                                 scales=buf.a1_s, gscale=buf.a1_g, workspace=buf.ws)
    wgu = (wq_gu["q"], wq_gu["s"], wq_gu["g"])
    if amax_h_in is not None and buf.F % 128 == 0:
        ops.grouped_gemm_w4a4_silu_gate_nvfp4(buf.a1_q, buf.a1_s, buf.a1_g, *wgu, meta["offsets"], amax_h_in,
                                              y1=buf.y1 if keep_y1 else None, h=buf.h if keep_y1 else None,
                                              amax_out=buf.amax[1:2], q_h=buf.a2_q, s_h=buf.a2_s, g_h=buf.a2_g)
        ops.grouped_gemm_w4a4(buf.a2_q, buf.a2_s, buf.a2_g, wq_dn["q"], wq_dn["s"], wq_dn["g"], meta["offsets"],
                              out=buf.y2)
        ops.moe_unpermute(buf.y2, meta["dest"], buf.T, buf.k, topk_w=topk_w, out=buf.out)
        return meta
    if fuse_silu and buf.F % 128 == 0:
        ops.grouped_gemm_w4a4_silu_gate(buf.a1_q, buf.a1_s, buf.a1_g, *wgu, meta["offsets"],
                                        y1=buf.y1 if keep_y1 else None, want_y1=keep_y1, h=buf.h,
                                        amax_out=buf.amax[1:2])
    else:
        ops.grouped_gemm_w4a4(buf.a1_q, buf.a1_s, buf.a1_g, *wgu, meta["offsets"], out=buf.y1)
        ops.silu_gate_fwd(buf.y1, h=buf.h, amax_out=buf.amax[1:2])
    ops.nvfp4_quantize(buf.h, amax_in=buf.amax[1:2], q=buf.a2_q, scales=buf.a2_s, gscale=buf.a2_g)
    ops.grouped_gemm_w4a4(buf.a2_q, buf.a2_s, buf.a2_g, wq_dn["q"], wq_dn["s"], wq_dn["g"], meta["offsets"],
                          out=buf.y2)
    ops.moe_unpermute(buf.y2, meta["dest"], buf.T, buf.k, topk_w=topk_w, out=buf.out)
    return meta


def backward(dy, topk_w, w_gu, w_dn, meta, buf, wgrad_stream=None, x=None, d_topk_w=None):
    """BF16 backward of ``forward`` (weight gradients in fp32).  Each
    elementwise consumer runs right after its producer, before a weight-
    gradient GEMM streams its fp32 output through the caches.  With ``x``
    (the forward's [T, D] tokens) the gate+up weight gradient gathers its
    activation rows from x; without it, from buf.x_perm (forward with
    keep_x_perm=True).

    With ``wgrad_stream`` (a torch stream) the two weight-gradient GEMMs run
    there, each after the op whose output it reads, overlapping the rest of
    the backward; the current stream waits for them before returning, so the
    caller's next step cannot overwrite their inputs early.

    With ``d_topk_w`` (fp32 [T, k]) the gradient of the routing weights is
    written there, in the pass that scatters dY (moe_unpermute_bwd; buf.y2
    must still hold the forward's)."""
    main = torch.cuda.current_stream()
    off = meta["offsets"]

    def tn(a, b, out, gather):
        if gather:
            ops.grouped_gemm_bf16_tn_gather(a, b, meta["src"], buf.k, off, out=out)
        else:
            ops.grouped_gemm_bf16(ops.TN, a, b, off, out=out)

    def wgrad(a, b, out, gather=False):
        if wgrad_stream is None:
            tn(a, b, out, gather)
            return
        ready = torch.cuda.Event()
        ready.record(main)
        wgrad_stream.wait_event(ready)
        with torch.cuda.stream(wgrad_stream):
            tn(a, b, out, gather)

    if d_topk_w is not None:
        ops.moe_unpermute_bwd(dy, buf.y2, meta["dest"], off, buf.k, topk_w=topk_w, dy_perm=buf.dy2, d_topk_w=d_topk_w)
    else:
        ops.moe_scatter(dy, meta["dest"], meta["offsets"], buf.k, topk_w=topk_w, out=buf.dy2)
    if wgrad_stream is not None:
        wgrad(buf.dy2, buf.h, buf.dw_dn)
    ops.grouped_gemm_bf16(ops.NN, buf.dy2, w_dn, off, out=buf.dh)
    ops.silu_gate_bwd(buf.y1, buf.dh, dy1=buf.dy1)
    if wgrad_stream is None:
        wgrad(buf.dy2, buf.h, buf.dw_dn)
    ops.grouped_gemm_bf16(ops.NN, buf.dy1, w_gu, off, out=buf.dx_perm)
    ops.moe_unpermute(buf.dx_perm, meta["dest"], buf.T, buf.k, topk_w=None, out=buf.dx)
    if x is not None:
        wgrad(buf.dy1, x, buf.dw_gu, gather=True)
    else:
        wgrad(buf.dy1, buf.x_perm, buf.dw_gu)
    if wgrad_stream is not None:
        done = torch.cuda.Event()
        done.record(wgrad_stream)
        main.wait_event(done)


def quantize_expert_weights_mx(w, out=None):
    """MXFP4 weights of stacked experts [E, N, K] (E8M0 scale per 32 along
    K; no per-expert scale), into ``out`` (an earlier result) when given.
    Once per optimizer step."""
    E, N, K = w.shape
    into = {} if out is None else dict(q=out["q"].view(E * N, K // 2), scales=out["s"].view(E * N, K // 32))
    q, sc = ops.mx_quantize(w.reshape(E * N, K), ops.MX_E2M1, **into)
    return dict(q=q.view(E, N, K // 2), s=sc.view(E, N, K // 32))


class BuffersW4A8:
    """Device buffers of one W4A8 forward step, allocated once and reused."""

    def __init__(self, T, k, E, D, F, device):
        R = T * k
        bf, u8 = torch.bfloat16, torch.uint8
        e = lambda *s, dt=bf: torch.empty(s, dtype=dt, device=device)  # noqa: E731
        self.T, self.k, self.E, self.D, self.F = T, k, E, D, F
        self.ws = e(max(ops.moe_permute_workspace_size(T, k, E), 1), dt=u8)
        self.a1_q, self.a1_s = e(R, D, dt=u8), e(R, D // 32, dt=u8)
        self.h = e(R, F)
        self.a2_q, self.a2_s = e(R, F, dt=u8), e(R, F // 32, dt=u8)
        self.y2 = e(R, D)
        self.out = e(T, D)


def forward_w4a8(x, topk_ids, topk_w, wq_gu, wq_dn, buf, keep_h=False):
    """W4A8 MoE forward (MXFP8 activations, MXFP4 weights); returns the
    routing metadata dict.  X is quantized inside the permutation and H
    inside the gate+up epilogue; H is kept in bf16 (buf.h) only with
    ``keep_h`` (a forward-only path)."""
    E = buf.E
    meta = ops.moe_permute_mx(topk_ids, E, x, q=buf.a1_q, scales=buf.a1_s, workspace=buf.ws)
    ops.grouped_gemm_w4a8_silu_gate_mx(buf.a1_q, buf.a1_s, wq_gu["q"], wq_gu["s"], meta["offsets"], q_h=buf.a2_q,
                                       s_h=buf.a2_s, h=buf.h if keep_h else None)
    ops.grouped_gemm_w4a8(buf.a2_q, buf.a2_s, wq_dn["q"], wq_dn["s"], meta["offsets"], out=buf.y2)
    ops.moe_unpermute(buf.y2, meta["dest"], buf.T, buf.k, topk_w=topk_w, out=buf.out)
    return meta


def quantize_expert_weights_t(w, amax=None):
    """NVFP4 of each expert weight transposed (W_e^T [K, N] of W [E, N, K]),
    blocks along the weight's output dimension: the B operand of the NVFP4
    backward's data gradients.  ``amax`` (the forward weights' per-expert
    amax, the same values) is reused when given.  Once per optimizer step."""
    q, sc, g, a = ops.nvfp4_quantize_transposed(w, amax_in=amax)
    return dict(q=q, s=sc, g=g, amax=a)


class NVFP4BackwardBuffers:
    """Buffers of the NVFP4 backward variant (besides Buffers(backward=True))."""

    def __init__(self, T, k, E, D, F, device):
        R = T * k
        Kp = ops.padded_extent(R, E)
        u8, f32 = torch.uint8, torch.float32
        e = lambda *s, dt=u8: torch.empty(s, dtype=dt, device=device)  # noqa: E731
        self.Kp = Kp
        self.amax = e(2, dt=f32)                      # [amax_dY2, amax_dY1]
        self.a_dy2 = (e(R, D // 2), e(R, D // 16), e(1, dt=f32))
        self.a_dy1 = (e(R, F), e(R, 2 * F // 16), e(1, dt=f32))
        self.c_dy2 = (e(D, Kp // 2), e(D, Kp // 16), e(1, dt=f32))
        self.c_h = (e(F, Kp // 2), e(F, Kp // 16), e(1, dt=f32))
        self.c_dy1 = (e(2 * F, Kp // 2), e(2 * F, Kp // 16), e(1, dt=f32))
        self.c_x = (e(D, Kp // 2), e(D, Kp // 16), e(1, dt=f32))


def backward_nvfp4(dy, topk_w, wt_gu, wt_dn, meta, buf, nb, amax_x=None, d_topk_w=None):
    """The NVFP4 backward variant of ``backward``: the same dataflow with the
    four grouped GEMMs in W4A4.  Each gradient's amax comes out of the kernel
    that writes the gradient (the weighted scatter for dY2, the SiLU backward
    for dY1) and is reused by its row-wise and column-wise quantizations; H
    and X_perm reuse the forward's amaxes (buf.amax, or ``amax_x`` when the
    forward was given a fixed one).  wt_gu / wt_dn: quantize_expert_weights_t
    of the bf16 weights.  Weight gradients fp32, activation gradients bf16.
    ``d_topk_w``: as in ``backward``."""
    off = meta["offsets"]
    R = buf.T * buf.k
    amax_x = buf.amax[0:1] if amax_x is None else amax_x
    if d_topk_w is not None:
        ops.moe_unpermute_bwd(dy, buf.y2, meta["dest"], off, buf.k, topk_w=topk_w, dy_perm=buf.dy2, d_topk_w=d_topk_w,
                              amax_out=nb.amax[0:1])
    else:
        ops.moe_scatter(dy, meta["dest"], off, buf.k, topk_w=topk_w, out=buf.dy2, amax_out=nb.amax[0:1])
    q, sc, g = nb.a_dy2
    ops.nvfp4_quantize(buf.dy2, amax_in=nb.amax[0:1], q=q, scales=sc, gscale=g)
    ops.grouped_gemm_w4a4(q, sc, g, wt_dn["q"], wt_dn["s"], wt_dn["g"], off, out=buf.dh)
    ops.silu_gate_bwd(buf.y1, buf.dh, dy1=buf.dy1, amax_out=nb.amax[1:2])
    ops.nvfp4_quantize_colwise(buf.dy2, off, nb.amax[0:1], Kp=nb.Kp, q_t=nb.c_dy2[0], s_t=nb.c_dy2[1],
                               gscale=nb.c_dy2[2])
    ops.nvfp4_quantize_colwise(buf.h, off, buf.amax[1:2], Kp=nb.Kp, q_t=nb.c_h[0], s_t=nb.c_h[1], gscale=nb.c_h[2])
    ops.grouped_gemm_w4a4_wgrad(nb.c_dy2, nb.c_h, off, R, out=buf.dw_dn)
    q, sc, g = nb.a_dy1
    ops.nvfp4_quantize(buf.dy1, amax_in=nb.amax[1:2], q=q, scales=sc, gscale=g)
    ops.grouped_gemm_w4a4(q, sc, g, wt_gu["q"], wt_gu["s"], wt_gu["g"], off, out=buf.dx_perm)
    ops.moe_unpermute(buf.dx_perm, meta["dest"], buf.T, buf.k, topk_w=None, out=buf.dx)
    ops.nvfp4_quantize_colwise(buf.dy1, off, nb.amax[1:2], Kp=nb.Kp, q_t=nb.c_dy1[0], s_t=nb.c_dy1[1],
                               gscale=nb.c_dy1[2])
    ops.nvfp4_quantize_colwise(buf.x_perm, off, amax_x, Kp=nb.Kp, q_t=nb.c_x[0], s_t=nb.c_x[1], gscale=nb.c_x[2])
    ops.grouped_gemm_w4a4_wgrad(nb.c_dy1, nb.c_x, off, R, out=buf.dw_gu)


class BuffersMXFP4:
    """Device buffers of one MXFP4 forward step, allocated once and reused;
    with ``backward`` also those of ``backward`` (dx in ``dx_dtype``)."""

    def __init__(self, T, k, E, D, F, device, backward=False, dx_dtype=torch.bfloat16):
        R = T * k
        bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
        e = lambda *s, dt=bf: torch.empty(s, dtype=dt, device=device)  # noqa: E731
        self.T, self.k, self.E, self.D, self.F = T, k, E, D, F
        self.ws = e(max(ops.moe_permute_workspace_size(T, k, E), 1), dt=u8)
        self.a1_q, self.a1_s = e(R, D // 2, dt=u8), e(R, D // 32, dt=u8)
        self.a2_q, self.a2_s = e(R, F // 2, dt=u8), e(R, F // 32, dt=u8)
        self.y2 = e(R, D)
        self.out = e(T, D)
        if backward:
            self.y1, self.h = e(R, 2 * F), e(R, F)
            self.dy2, self.dh, self.dy1, self.dx_perm = e(R, D), e(R, F), e(R, 2 * F), e(R, D)
            self.dx = e(T, D, dt=dx_dtype)
            self.dw_dn, self.dw_gu = e(E, D, F, dt=f32), e(E, 2 * F, D, dt=f32)


def forward_mxfp4(x, topk_ids, topk_w, wq_gu, wq_dn, buf, keep=False):
    """MXFP4 MoE forward (weights from quantize_expert_weights_mx); returns
    the routing metadata dict.  X is quantized inside the permutation and H
    inside the gate+up epilogue.  ``keep``: bf16 Y1 and H are stored too
    (buf.y1, buf.h), for ``backward``, which then gathers its activation rows
    from x."""
    ops._need(topk_w, "topk_w", torch.float32, buf.T, buf.k)
    with ops._on_device(x, topk_ids, topk_w, buf.out):
        meta = ops.moe_permute_mxfp4(topk_ids, buf.E, x, q=buf.a1_q, scales=buf.a1_s, workspace=buf.ws)
        ops.grouped_gemm_mxfp4_silu_gate(buf.a1_q, buf.a1_s, wq_gu["q"], wq_gu["s"], meta["offsets"],
                                         y1=buf.y1 if keep else None, want_y1=keep, h=buf.h if keep else None,
                                         want_h=keep, q_h=buf.a2_q, s_h=buf.a2_s)
        ops.grouped_gemm_mxfp4(buf.a2_q, buf.a2_s, wq_dn["q"], wq_dn["s"], meta["offsets"], out=buf.y2)
        ops.moe_unpermute(buf.y2, meta["dest"], buf.T, buf.k, topk_w=topk_w, out=buf.out)
    return meta


class Learner:
    """One MoE layer trained in MXFP4: fp32 master weights with bf16 and
    MXFP4 copies, ``forward``, ``backward`` (to the input, the experts' and
    the router's weights) and ``update`` (one AdamW step, copies renewed).

    w_r [E, D], w_gu [E, 2F, D], w_dn [E, D, F]: fp32 master weights on the
    GPU, updated in place.  The gradient of the logits is rounded to bf16 for
    the BF16 products that take it to x and w_r, as all other gradients that
    enter a product are (half a step, 2^-8 relative).  T: tokens per step.  E, D % 32 == 0 (the router's
    GEMM), D, F % 128 == 0.  ``adamw``: keyword arguments of optim.AdamW."""

    def __init__(self, w_r, w_gu, w_dn, T, k, router_bias=None, score=ops.ROUTER_TOPK_SOFTMAX, **adamw):
        E, D = w_r.shape
        F = w_dn.shape[2]
        dev = w_r.device
        self.k, self.score, self.router_bias = k, score, router_bias
        self.master = [w_r, w_gu, w_dn]
        # (detached: a copy of a leaf would keep the leaf's node of the autograd graph)
        self.w_r, self.w_gu, self.w_dn = self.copies = [w.detach().to(torch.bfloat16) for w in self.master]
        self.buf = BuffersMXFP4(T, k, E, D, F, dev, backward=True, dx_dtype=torch.float32)
        e = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device=dev)  # noqa: E731
        self.logits, self.d_logits = e(T, E), e(T, E, dt=torch.bfloat16)
        self.topk_ids, self.topk_w, self.d_topk_w = e(T, k, dt=torch.int32), e(T, k), e(T, k)
        self.lse, self.prob_sum = e(T), e(E)
        self.router_ws = e(max(ops._lib.load().moe_router_workspace_size(T, E, k), 1), dt=torch.uint8)
        self.dw_r = e(1, E, D)
        self.one_group = torch.tensor([0, T], dtype=torch.int32, device=dev)
        self.x = self.meta = None        # of the last forward
        self.has_grads = False           # the gradients' buffers hold some
        self.opt = optim.AdamW(self.master, params_bf16=self.copies, **adamw)
        with ops._on_device(self.w_r):
            self.wq_gu, self.wq_dn = quantize_expert_weights_mx(self.w_gu), quantize_expert_weights_mx(self.w_dn)

    def forward(self, x):
        """The layer's output [T, D] (bf16, the layer's own buffer) for x [T, D]
        bf16; the router's lse and prob_sum stay in ``lse`` and ``prob_sum`` for
        its losses.  x is kept, not copied: ``backward`` reads it again."""
        ops._need(x, "x", torch.bfloat16, self.logits.shape[0], self.w_r.shape[1])
        with ops._on_device(x, self.w_r):
            self.x = x
            ops.grouped_gemm_bf16(ops.NT, x, self.w_r.unsqueeze(0), self.one_group, out=self.logits)
            ops.moe_router(self.logits, self.k, bias=self.router_bias, score=self.score, topk_ids=self.topk_ids,
                           topk_w=self.topk_w, lse=self.lse, prob_sum=self.prob_sum, workspace=self.router_ws)
            self.meta = forward_mxfp4(x, self.topk_ids, self.topk_w, self.wq_gu, self.wq_dn, self.buf, keep=True)
        return self.buf.out

    def backward(self, dy, d_lse=None, d_prob_sum=None):
        """Gradient of the input (fp32 [T, D]) for dy [T, D] bf16 and the
        gradients of the router's losses; the weights' gradients stay in
        ``grads()``."""
        if self.meta is None:
            raise RuntimeError("Learner.backward before a forward")
        b = self.buf
        with ops._on_device(dy, self.w_r):
            backward(dy, self.topk_w, self.w_gu, self.w_dn, self.meta, b, x=self.x, d_topk_w=self.d_topk_w)
            ops.moe_router_bwd(self.logits, self.topk_ids, self.d_topk_w, score=self.score, lse=self.lse, d_lse=d_lse,
                               d_prob_sum=d_prob_sum, out=self.d_logits)
            ops.grouped_gemm_bf16(ops.TN, self.d_logits, self.x, self.one_group, out=self.dw_r)
            ops.grouped_gemm_bf16(ops.NN, self.d_logits, self.w_r.unsqueeze(0), self.one_group, out=b.dx,
                                  accumulate=True)
        self.has_grads = True
        return b.dx

    def grads(self):
        return [self.dw_r[0], self.buf.dw_gu, self.buf.dw_dn]

    def update(self, grad_scale=None, skip=None):
        """One optimizer step with the last backward's gradients; the bf16 and
        MXFP4 weights follow."""
        if not self.has_grads:
            raise RuntimeError("Learner.update before a backward: there are no gradients")
        with ops._on_device(self.w_r):
            self.opt.step(self.grads(), grad_scale=grad_scale, skip=skip)
            quantize_expert_weights_mx(self.w_gu, out=self.wq_gu)
            quantize_expert_weights_mx(self.w_dn, out=self.wq_dn)
