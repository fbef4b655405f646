"""More operators of an MoE learner's step, as cases to measure.

Three families: the layer norm in front of the layer (and its RMS form) with its gradients, the experts'
products in 8-bit integers with a scale per token and per channel (W8A8), and activations kept for the backward
pass in 8 bits (MXINT8: an 8-bit integer per element, a power-of-two scale per 32).  Each case is plain data;
`prepare` makes its inputs from a seed, `run` makes one pass (through elementary torch operations, or through
this package where `own` is set), `exact` computes the same outputs in 64 bits from the definitions.
"""

import math

import torch

own = False

BLOCK = 32   # elements per scale of an MXINT8 checkpoint
EPS = 1e-6   # of the norms


# ------------------------------------------------------------------ cases

def listed():
    moe = dict(E=128, k=8, D=2048, F=768)  # the layer of the 30B-A3B workloads
    return [
        # a serving step of a few sequences: the norm's latency
        dict(name="norm decode", op="norm", T=16, D=2048, kind="rms", bias=False, dtype="bf16"),
        # a learner's forward at 16k tokens
        dict(name="norm 16k", op="norm", T=16384, D=2048, kind="layer", bias=True, dtype="bf16"),
        # the norm's gradient in the 8k update step: bf16 activations, the fp32 gradient that the layer gives
        dict(name="norm backward 8k", op="norm_bwd", T=8192, D=2048, kind="layer", bias=True, dtype="bf16", grad="f32"),
        # a ragged batch in fp32 with rows of an odd length
        dict(name="norm backward 333", op="norm_bwd", T=333, D=2557, kind="rms", bias=False, dtype="f32", grad="f32"),
        # a decode step's gate+up product: 128 rows over 128 experts, weights read once
        dict(name="int8 product decode", op="i8_gemm", T=16, E=128, k=8, N=1536, K=2048, zipf=0.0, out="bf16"),
        # the down projection of a heavily skewed 16k batch (empty experts, one very large)
        dict(name="int8 product 16k skewed", op="i8_gemm", T=16384, E=128, k=8, N=2048, K=768, zipf=1.6, out="bf16"),
        # gate+up with the SiLU gate at 8k tokens, Y1 and H kept
        dict(name="int8 gate+up 8k", op="i8_gate", T=8192, E=128, k=8, F=768, K=2048, zipf=0.0),
        # the layer's forward in W8A8 at 8k tokens: permute-quantize, gate+up, requantize, down, combine
        dict(name="int8 forward 8k", op="i8_forward", T=8192, zipf=0.0, **moe),
        # the hidden states between two layers of a 16k batch, kept in 8 bits and read back
        dict(name="checkpoint save 16k", op="ckpt_save", R=16384, W=2048, dtype="bf16"),
        # gate+up at 8k tokens with Y1 kept in 8 bits alone, then the gate's gradient from them
        dict(name="checkpoint gate+up 8k", op="ckpt_gate", T=8192, E=128, k=8, F=768, K=2048, zipf=0.0),
        # the gate's gradient in the 8k update step, from Y1 kept in 8 bits
        dict(name="checkpoint backward 8k", op="ckpt_bwd", R=65536, F=768),
        # the same for a ragged batch of a narrow layer
        dict(name="checkpoint backward 1333", op="ckpt_bwd", R=1333, F=352),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))

    op = rng.choice(["norm", "norm_bwd", "i8_gemm", "i8_gate", "i8_forward", "ckpt_save", "ckpt_gate", "ckpt_bwd"])
    if op in ("norm", "norm_bwd"):
        D = log(32, 8192)
        if rng.random() < 0.5:
            D = D // 8 * 8
        c = dict(op=op, T=log(1, (16384 if op == "norm" else 8192) * min(1.0, 2048 / D)), D=D, kind=rng.choice(["layer", "rms"]),
                 bias=rng.random() < 0.5, dtype=rng.choice(["bf16", "f32"]))
        return dict(c, grad=rng.choice(["bf16", "f32"])) if op == "norm_bwd" else c
    if op == "ckpt_save":
        W = 32 * log(1, 64)
        return dict(op=op, R=log(1, 16384), W=W, dtype=rng.choice(["bf16", "f32"]))
    if op == "ckpt_bwd":
        return dict(op=op, R=log(1, 65536), F=32 * log(1, 24))
    T, E, zipf = log(1, 16384 if op == "i8_gemm" else 8192), log(4, 128), rng.choice([0.0, 1.1, 1.6])
    c = dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), zipf=zipf)
    if op == "i8_gemm":
        return dict(c, N=32 * log(2, 64), K=16 * log(4, 96), out=rng.choice(["bf16", "f32"]))
    if op == "i8_forward":
        return dict(c, D=128 * rng.randint(1, 16), F=128 * rng.randint(1, 6))
    return dict(c, F=128 * rng.randint(1, 6), K=16 * log(4, 128))


def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        T, D, b = case["T"], case["D"], 4 if case["dtype"] == "f32" else 2
        stats = T * (4 if case["kind"] == "rms" else 8)
        vec = D * 4 * (2 if case["bias"] else 1)
        if op == "norm":
            return dict(bytes=2 * T * D * b + stats + vec, flops=8 * T * D)
        g = 4 if case["grad"] == "f32" else 2
        return dict(bytes=T * D * (2 * b + g) + stats + D * 4 + vec, flops=16 * T * D)
    if op == "ckpt_save":
        n, b = case["R"] * case["W"], 4 if case["dtype"] == "f32" else 2
        return dict(bytes=n * (2 * b + 2 * 33 / 32), flops=4 * n)  # codes and scales written, then read
    if op == "ckpt_bwd":
        n = case["R"] * case["F"]
        return dict(bytes=n * (2 * 33 / 32 + 2 + 4 + 2), flops=20 * n)
    M, E = case["T"] * case["k"], case["E"]
    used = min(E, M)  # experts that can have rows at all
    if op == "i8_gemm":
        N, K = case["N"], case["K"]
        return dict(bytes=(M + used * N) * K + 4 * (M + used * N) + M * N * (2 if case["out"] == "bf16" else 4),
                    flops=2 * M * N * K)
    if op == "i8_forward":
        D, F = case["D"], case["F"]
        return dict(bytes=case["T"] * D * 4 + used * (3 * F * D + 4 * (2 * F + D)), flops=6 * M * D * F)
    F, K = case["F"], case["K"]
    bytes = (M + used * 2 * F) * K + 4 * (M + used * 2 * F)
    if op == "i8_gate":
        return dict(bytes=bytes + M * 3 * F * 2, flops=4 * M * F * K)
    # H written; the codes written and read, the gradient read, dY1 and H written
    return dict(bytes=bytes + M * F * (2 + 4 * 33 / 32 + 2 + 4 + 2), flops=4 * M * F * K)


# ------------------------------------------------------------------ inputs

def _dt(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _routing(g, T, E, k, zipf):
    """Distinct expert ids per token from biased logits, weights of the chosen, and the sorted layout."""
    logits = torch.randn(T, E, generator=g, device="cuda")
    rank = torch.randperm(E, generator=g, device="cuda") + 1
    ids = torch.sort(logits - zipf * torch.log(rank.float()), dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.softmax(torch.gather(logits, 1, ids), dim=1).contiguous()
    ids = ids.to(torch.int32).contiguous()
    flat = ids.view(-1).long()
    offsets = torch.cat([flat.new_zeros(1), torch.bincount(flat, minlength=E).cumsum(0)]).to(torch.int32)
    order = torch.sort(flat, stable=True).indices
    dest = torch.empty(T * k, dtype=torch.int32, device="cuda")
    dest[order] = torch.arange(T * k, dtype=torch.int32, device="cuda")
    ends = offsets.tolist()
    segments = [(e, ends[e], ends[e + 1]) for e in range(E) if ends[e + 1] > ends[e]]
    return ids, w, offsets, dest, order, segments


def _outliers(g, x, part=0.005, factor=16.0):
    return torch.where(torch.rand(x.shape, generator=g, device="cuda") < part, x * factor, x)


def _i8(x):
    """Codes and scales of the rows of x: s = amax / 127, the code the nearest whole number to x / s."""
    x = x.float()
    s = x.abs().amax(-1, keepdim=True) / 127
    q = torch.where(s > 0, torch.round(x / s), torch.zeros_like(x)).clamp(-127, 127)
    return q.to(torch.int8), s.squeeze(-1)


def _pow2(x, e):
    """x * 2^e exactly (e in [-254, 254], whole): by two powers made from their bits, each a normal number."""
    half = e.to(torch.int32) >> 1
    rest = e.to(torch.int32) - half
    return x * ((half + 127) << 23).view(torch.float32) * ((rest + 127) << 23).view(torch.float32)


def _mxint8(x):
    """MXINT8 codes (whole numbers in 32 bits) and unbiased exponents, in blocks along the last axis of x."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    a = b.abs().amax(-1, keepdim=True)
    e = torch.where(a > 0, torch.frexp(a).exponent - 1, torch.full_like(a, -127, dtype=torch.int32)).clamp(-127, 127)
    return torch.round(_pow2(b, 6 - e)).clamp(-127, 127), e


def _weights(g, *shape):
    return _i8((torch.randn(*shape, generator=g, device="cuda") * 0.02).to(torch.bfloat16))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("norm", "norm_bwd"):
        T, D = case["T"], case["D"]
        # a residual stream: columns of unlike size and mean, a few outliers
        scale = torch.exp(torch.randn(D, generator=g, device="cuda") * 0.5)
        x = (torch.randn(T, D, generator=g, device="cuda") + torch.randn(D, generator=g, device="cuda") * 0.3) * scale
        s["x"] = _outliers(g, x).to(_dt(case["dtype"]))
        s["w"] = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
        s["b"] = 0.1 * torch.randn(D, generator=g, device="cuda") if case["bias"] else None
        if op == "norm_bwd":
            s["dy"] = (torch.randn(T, D, generator=g, device="cuda") * 1e-3).to(_dt(case["grad"]))
            x = s["x"].double()
            mean = x.mean(1) if case["kind"] == "layer" else torch.zeros_like(x[:, 0])
            s["rstd"] = (((x - mean[:, None]) ** 2).mean(1) + EPS).rsqrt().float()
            s["mean"] = mean.float() if case["kind"] == "layer" else None
        return s
    if op == "ckpt_save":
        x = torch.randn(case["R"], case["W"], generator=g, device="cuda")
        s["x"] = _outliers(g, x).to(_dt(case["dtype"]))
        return s
    if op == "ckpt_bwd":
        R, F = case["R"], case["F"]
        q, e = _mxint8((torch.randn(R, 2 * F, generator=g, device="cuda") * 0.9).to(torch.bfloat16))
        s["q"] = q.flatten(-2).to(torch.int8).view(torch.uint8)
        s["s"] = (e.squeeze(-1) + 127).to(torch.uint8)
        s["dh"] = (torch.randn(R, F, generator=g, device="cuda") * 1e-3).to(torch.bfloat16)
        return s
    T, E, k = case["T"], case["E"], case["k"]
    s["ids"], s["w"], s["offsets"], s["dest"], order, s["segments"] = _routing(g, T, E, k, case["zipf"])
    if op == "i8_forward":
        D, F = case["D"], case["F"]
        s["x"] = _outliers(g, torch.randn(T, D, generator=g, device="cuda")).to(torch.bfloat16)
        s["gu"], s["dn"] = _weights(g, E, 2 * F, D), _weights(g, E, D, F)
        if own:  # the buffers of one layer, which a program allocates once
            from nvfp4_quantized_moe_token_amd import moe_layer
            s["buf"] = moe_layer.BuffersInt8(T, k, E, D, F, torch.device("cuda"))
        return s
    s["a"] = _i8(torch.randn(T, case["K"], generator=g, device="cuda").to(torch.bfloat16))
    s["a"] = tuple(a[order // k].contiguous() for a in s["a"])
    s["b"] = _weights(g, E, case["N"] if op == "i8_gemm" else 2 * case["F"], case["K"])
    if op == "ckpt_gate":
        s["dh"] = (torch.randn(T * k, case["F"], generator=g, device="cuda") * 1e-3).to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _OWN[s["case"]["op"]](s) if own else _PLAIN[s["case"]["op"]](s)


# ---- plain forms

def _norm(s):
    x = s["x"].float()
    out = {}
    if s["case"]["kind"] == "layer":
        mean = x.mean(1, keepdim=True)
        out["mean"] = mean.squeeze(1)
        x = x - mean
    r = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    out["rstd"] = r.squeeze(1)
    y = x * r * s["w"]
    if s["b"] is not None:
        y = y + s["b"]
    out["y"] = y.to(s["x"].dtype)
    return out


def _norm_bwd(s):
    x, dy, r = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    layer = s["case"]["kind"] == "layer"
    h = (x - s["mean"][:, None] if layer else x) * r
    g = dy * s["w"]
    dx = g - h * (g * h).mean(1, keepdim=True)
    if layer:
        dx = dx - g.mean(1, keepdim=True)
    out = dict(dx=(dx * r).to(s["x"].dtype), dw=(dy * h).sum(0))
    if s["case"]["bias"]:
        out["db"] = dy.sum(0)
    return out


# The experts' products go expert by expert (a loop over the experts that have rows): their row counts differ.
# A code's products and their sums are whole numbers, exact in 32 bits up to 2^24, which these stay below.

def _i8_products(a, b, segments, out):
    for e, lo, hi in segments:
        out[lo:hi] = (a[0][lo:hi].float() @ b[0][e].float().t()) * a[1][lo:hi, None] * b[1][e]
    return out


def _new(s, n, dtype):
    return torch.empty(s["dest"].numel(), n, dtype=dtype, device="cuda")


def _i8_gemm(s):
    return _i8_products(s["a"], s["b"], s["segments"], _new(s, s["case"]["N"], _dt(s["case"]["out"])))


def _silu_gate(y1):
    g, u = y1.float().chunk(2, -1)
    return (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16)


def _i8_gate(s):
    y1 = _i8_products(s["a"], s["b"], s["segments"], _new(s, 2 * s["case"]["F"], torch.bfloat16))
    return dict(y1=y1, h=_silu_gate(y1))


def _i8_forward(s):
    c = s["case"]
    order = torch.sort(s["ids"].view(-1), stable=True).indices
    a = [t[order // c["k"]] for t in _i8(s["x"])]
    y1 = _i8_products(a, s["gu"], s["segments"], _new(s, 2 * c["F"], torch.bfloat16))
    y2 = _i8_products(_i8(_silu_gate(y1)), s["dn"], s["segments"], _new(s, c["D"], torch.bfloat16))
    dest = torch.empty_like(order)
    dest[order] = torch.arange(order.numel(), device="cuda")
    return (y2[dest].float().view(c["T"], c["k"], c["D"]) * s["w"][:, :, None]).sum(1).to(torch.bfloat16)


def _ckpt_save(s):
    q, e = _mxint8(s["x"])
    q, e = q.to(torch.int8), (e + 127).to(torch.uint8)  # what is kept
    return _pow2(q.float(), e.to(torch.int32) - 133).flatten(-2).to(s["x"].dtype)


def _gate_grad(q, e, dh):
    """dY1 and H from the codes and exponents of Y1."""
    g, u = _pow2(q.float(), e - 6).flatten(-2).chunk(2, -1)
    dh = dh.float()
    sg = 1 / (1 + torch.exp(-g))
    dy1 = torch.cat([dh * u * (sg * (1 + g * (1 - sg))), dh * g * sg], -1)
    return dict(dy1=dy1.to(torch.bfloat16), h_again=(g * sg * u).to(torch.bfloat16))


def _ckpt_gate(s):
    y1 = _i8_products(s["a"], s["b"], s["segments"], _new(s, 2 * s["case"]["F"], torch.bfloat16))
    h = _silu_gate(y1)
    q, e = _mxint8(y1)
    q = q.to(torch.int8)  # what is kept
    del y1
    return dict(_gate_grad(q, e, s["dh"]), h=h)


def _ckpt_bwd(s):
    q = s["q"].view(torch.int8).unflatten(-1, (-1, BLOCK))
    return _gate_grad(q, s["s"].to(torch.int32)[..., None] - 127, s["dh"])


_PLAIN = dict(norm=_norm, norm_bwd=_norm_bwd, i8_gemm=_i8_gemm, i8_gate=_i8_gate, i8_forward=_i8_forward,
              ckpt_save=_ckpt_save, ckpt_gate=_ckpt_gate, ckpt_bwd=_ckpt_bwd)


# ---- through the package

def _kind(ops, c):
    return ops.NORM_LAYER if c["kind"] == "layer" else ops.NORM_RMS


def _own_norm(s):
    from nvfp4_quantized_moe_token_amd import ops
    r = ops.layer_norm(s["x"], s["w"], s["b"], eps=EPS, kind=_kind(ops, s["case"]))
    return {n: t for n, t in r.items() if t is not None}


def _own_norm_bwd(s):
    from nvfp4_quantized_moe_token_amd import ops
    r = ops.layer_norm_bwd(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], kind=_kind(ops, s["case"]),
                           want_db=s["case"]["bias"], dx_dtype=s["x"].dtype)
    return {n: t for n, t in r.items() if t is not None}


def _own_i8_gemm(s):
    from nvfp4_quantized_moe_token_amd import ops
    return ops.grouped_gemm_int8(*s["a"], *s["b"], s["offsets"], out_dtype=_dt(s["case"]["out"]))


def _own_i8_gate(s):
    from nvfp4_quantized_moe_token_amd import ops
    r = ops.grouped_gemm_int8_silu_gate(*s["a"], *s["b"], s["offsets"])
    return dict(y1=r["y1"], h=r["h"])


def _own_i8_forward(s):
    from nvfp4_quantized_moe_token_amd import moe_layer
    gu, dn = (dict(q=q, s=sc) for q, sc in (s["gu"], s["dn"]))
    moe_layer.forward_int8(s["x"], s["ids"], s["w"], gu, dn, s["buf"])
    return s["buf"].out


def _own_ckpt_save(s):
    from nvfp4_quantized_moe_token_amd import ops
    q, sc = ops.mx_quantize(s["x"], ops.MX_INT8)
    return ops.mx_dequantize(q, sc, ops.MX_INT8, out_dtype=s["x"].dtype)


def _own_ckpt_gate(s):
    from nvfp4_quantized_moe_token_amd import ops
    r = ops.grouped_gemm_int8_silu_gate(*s["a"], *s["b"], s["offsets"], want_y1=False, want_ckpt=True)
    dy1, h = ops.silu_gate_bwd_mx(r["q_y1"], r["s_y1"], s["dh"])
    return dict(dy1=dy1, h_again=h, h=r["h"])


def _own_ckpt_bwd(s):
    from nvfp4_quantized_moe_token_amd import ops
    dy1, h = ops.silu_gate_bwd_mx(s["q"], s["s"], s["dh"])
    return dict(dy1=dy1, h_again=h)


_OWN = dict(norm=_own_norm, norm_bwd=_own_norm_bwd, i8_gemm=_own_i8_gemm, i8_gate=_own_i8_gate,
            i8_forward=_own_i8_forward, ckpt_save=_own_ckpt_save, ckpt_gate=_own_ckpt_gate, ckpt_bwd=_own_ckpt_bwd)


# ------------------------------------------------------------------ the same in 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s, case)


def _x_norm(s, c):
    x = s["x"].double()
    mean = x.sum(1) / c["D"]
    if c["kind"] == "rms":
        mean = torch.zeros_like(mean)
    var = ((x - mean[:, None]) ** 2).sum(1) / c["D"]
    r = 1 / torch.sqrt(var + EPS)
    y = (x - mean[:, None]) * r[:, None] * s["w"].double()
    if c["bias"]:
        y = y + s["b"].double()
    return dict(mean=mean, rstd=r, y=y) if c["kind"] == "layer" else dict(rstd=r, y=y)


def _x_norm_bwd(s, c):
    x, dy, w, r = s["x"].double(), s["dy"].double(), s["w"].double(), s["rstd"].double()[:, None]
    if c["kind"] == "layer":
        x = x - s["mean"].double()[:, None]
    # dL/dx = r w dy - (r^3 x) (w dy . x) / D, less its mean where the mean was taken out
    dx = r * w * dy - r ** 3 * x * ((w * dy * x).sum(1, keepdim=True) / c["D"])
    if c["kind"] == "layer":
        dx = dx - r * ((w * dy).sum(1, keepdim=True) / c["D"])
    out = dict(dx=dx, dw=(dy * x * r).sum(0))
    if c["bias"]:
        out["db"] = dy.sum(0)
    return out


def _x_products(a, b, segments, n):
    out = torch.zeros(a.shape[0], n, dtype=torch.float64, device="cuda")
    for e, lo, hi in segments:
        out[lo:hi] = a[lo:hi] @ (b[0][e].double() * b[1][e].double()[:, None]).t()
    return out


def _x_values(a):
    return a[0].double() * a[1].double()[:, None]


def _x_i8_gemm(s, c):
    return _x_products(_x_values(s["a"]), s["b"], s["segments"], c["N"])


def _x_gate(y1):
    F = y1.shape[1] // 2
    return y1[:, :F] * torch.sigmoid(y1[:, :F]) * y1[:, F:]


def _x_i8_gate(s, c):
    y1 = _x_products(_x_values(s["a"]), s["b"], s["segments"], 2 * c["F"])
    return dict(y1=y1, h=_x_gate(y1.to(torch.bfloat16).double()))  # H is defined on the bf16 values of Y1


def _x_quant(x):
    """Values of the rows of x after 8-bit integers with a scale per row."""
    s = x.abs().amax(1, keepdim=True) / 127
    q = torch.where(s > 0, torch.round(x / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(x))
    return q * s


def _x_i8_forward(s, c):
    dest = s["dest"].long()
    src = torch.empty_like(dest)
    src[dest] = torch.arange(dest.numel(), device="cuda")
    a = _x_quant(s["x"].double())[src // c["k"]]
    y1 = _x_products(a, s["gu"], s["segments"], 2 * c["F"]).to(torch.bfloat16).double()
    h = _x_quant(_x_gate(y1).to(torch.bfloat16).double())  # H and Y2 are stored in bf16
    del a, y1
    y2 = _x_products(h, s["dn"], s["segments"], c["D"]).to(torch.bfloat16)
    out = torch.zeros(c["T"], c["D"], dtype=torch.float64, device="cuda")
    for j in range(c["k"]):
        out += s["w"][:, j, None].double() * y2[dest.view(c["T"], c["k"])[:, j]].double()
    return out


def _x_power(e):
    """2^e in 64 bits, exactly: the exponent field itself."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _x_mxint8(x):
    """Values of x (in 64 bits) after MXINT8: the nearest multiple of 2^(e-6) up to 127 of them, e of the block's maximum."""
    b = x.unflatten(-1, (-1, BLOCK))
    a = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a))))
    e = torch.where(_x_power(e) > a, e - 1, e)              # log2 may round up to the next power
    e = torch.where(_x_power(e + 1) <= a, e + 1, e)
    step = _x_power(torch.where(a > 0, e.clamp(-127, 127), torch.full_like(e, -127.0)) - 6)
    return (torch.round(b / step).clamp(-127, 127) * step).flatten(-2)


def _x_gate_grad(y1, dh):
    F = y1.shape[1] // 2
    g, u, dh = y1[:, :F], y1[:, F:], dh.double()
    sg = torch.sigmoid(g)
    return dict(dy1=torch.cat([dh * u * (sg + g * sg * (1 - sg)), dh * g * sg], 1), h_again=g * sg * u)


def _x_ckpt_gate(s, c):
    y1 = _x_products(_x_values(s["a"]), s["b"], s["segments"], 2 * c["F"]).to(torch.bfloat16).double()
    return dict(_x_gate_grad(_x_mxint8(y1), s["dh"]), h=_x_gate(y1))


def _x_ckpt_bwd(s, c):
    step = _x_power(s["s"].long() - 133)
    y1 = s["q"].view(torch.int8).double().unflatten(-1, (-1, BLOCK)) * step[..., None]
    return _x_gate_grad(y1.flatten(-2), s["dh"])


_EXACT = dict(norm=_x_norm, norm_bwd=_x_norm_bwd, i8_gemm=_x_i8_gemm, i8_gate=_x_i8_gate, i8_forward=_x_i8_forward,
              ckpt_save=lambda s, c: _x_mxint8(s["x"].double()), ckpt_gate=_x_ckpt_gate, ckpt_bwd=_x_ckpt_bwd)
