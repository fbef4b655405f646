"""The operators of an MoE learner step around the quantized expert path, as cases to measure.

Four operators: the router (top-k of biased logits, softmax weights, and its gradient), the gradient of the
weighted combine, the experts' MXFP4 products (activations quantized on the way), and the AdamW step with
states in 32 or in 8 bits.  Each case is plain data; `prepare` makes its inputs from a seed, `run` makes one
pass (through elementary torch operations, or through this package where `own` is set), `exact` computes the
same outputs in 64 bits from the definitions.
"""

import math
import random

import torch

own = False

BLOCK = 32          # elements per MX scale
STATE_BLOCK = 256   # elements per scale of an 8-bit optimizer state
M32 = 0xFFFFFFFF


# ------------------------------------------------------------------ cases

def listed():
    moe = dict(E=128, k=8, D=2048, F=768)  # the layer of the 30B-A3B workloads
    return [
        # a serving step of a few sequences: the router's latency
        dict(name="router decode", op="router", T=16, E=128, k=8, dtype="f32", bias=True, score="topk", aux=False),
        # a learner's forward at 16k tokens, with the sums that the auxiliary losses need
        dict(name="router 16k", op="router", T=16384, E=128, k=8, dtype="f32", bias=True, score="topk", aux=True),
        # the router's gradient in the 8k update step, auxiliary losses included
        dict(name="router backward 8k", op="router_bwd", T=8192, E=128, k=8, dtype="f32", score="topk", aux=True),
        # the combine's gradient in the 8k update step
        dict(name="combine backward 8k", op="combine_bwd", T=8192, dtype="bf16", bad=0, **{n: moe[n] for n in "EkD"}),
        # a ragged tail batch in fp32 with a few dropped assignments
        dict(name="combine backward 333", op="combine_bwd", T=333, E=40, k=4, D=2560, dtype="f32", bad=5),
        # a decode step's gate+up product: 128 rows over 128 experts, weights read once
        dict(name="mx product decode", op="mx_gemm", T=16, E=128, k=8, N=1536, K=2048, zipf=0.0, out="bf16"),
        # the down projection of a heavily skewed 16k batch (empty experts, one very large)
        dict(name="mx product 16k skewed", op="mx_gemm", T=16384, E=128, k=8, N=2048, K=768, zipf=1.6, out="bf16"),
        # gate+up with the SiLU gate at 8k tokens, Y1 and H kept for a backward pass
        dict(name="mx gate+up 8k", op="mx_gate", T=8192, E=128, k=8, F=768, K=2048, zipf=0.0),
        # the layer's forward in MXFP4 at 8k tokens: permute-quantize, gate+up, requantize, down, combine
        dict(name="mx forward 8k", op="mx_forward", T=8192, zipf=0.0, **moe),
        # both projections of the layer, fp32 master weights and states, bf16 copies written
        dict(name="adamw layer 32 bit", op="adamw", split="experts", bits=32, grad="f32", param="f32", copy=True, tensors=2,
             elems=128 * 3 * 768 * 2048),
        # the same with 8-bit states, read back as values
        dict(name="adamw layer 8 bit", op="adamw", split="experts", bits=8, grad="f32", param="f32", copy=True, tensors=2,
             elems=128 * 3 * 768 * 2048),
        # the many small tensors of a model: norms, biases, routers, of odd sizes
        dict(name="adamw 61 small", op="adamw", split="spread", bits=32, grad="bf16", param="f32", copy=False, tensors=61,
             elems=1_500_007),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["router", "router_bwd", "combine_bwd", "mx_gemm", "mx_gate", "mx_forward", "adamw", "adamw"])
    if op in ("router", "router_bwd"):
        E = log(4, 512)
        c = dict(op=op, T=log(1, 16384), E=E, k=rng.randint(1, min(8, E)), dtype=rng.choice(["f32", "bf16"]),
                 score=rng.choice(["topk", "all"]), aux=rng.random() < 0.5)
        return dict(c, bias=rng.random() < 0.5) if op == "router" else c
    if op == "combine_bwd":
        return dict(op=op, T=log(1, 8192), E=log(4, 256), k=rng.randint(1, 8), D=8 * log(8, 320),
                    dtype=rng.choice(["f32", "bf16"]) if rng.random() < 0.5 else "bf16", bad=rng.choice([0, 0, 1, 3]))
    if op in ("mx_gemm", "mx_gate", "mx_forward"):
        T, E, zipf = log(1, 16384 if op == "mx_gemm" else 8192), log(4, 128), rng.choice([0.0, 1.1, 1.6])
        k = rng.randint(1, min(8, E))
        if op == "mx_gemm":
            return dict(op=op, T=T, E=E, k=k, N=32 * log(2, 64), K=128 * rng.randint(1, 12), zipf=zipf,
                        out=rng.choice(["bf16", "f32"]))
        if op == "mx_gate":
            return dict(op=op, T=T, E=E, k=k, F=128 * rng.randint(1, 8), K=128 * rng.randint(1, 16), zipf=zipf)
        return dict(op=op, T=T, E=E, k=k, D=128 * rng.randint(1, 16), F=128 * rng.randint(1, 8), zipf=zipf)
    n = log(1, 64)
    return dict(op=op, split="spread", bits=rng.choice([32, 8]), grad=rng.choice(["f32", "bf16"]),
                param=rng.choice(["f32", "f32", "bf16"]), copy=False, tensors=n, elems=max(n * 8, log(1000, 200_000_000)))


def sizes(case):
    """Elements of each tensor of an adamw case."""
    if case["split"] == "experts":
        return [case["elems"] // 3 * 2, case["elems"] // 3]
    r = random.Random(case["tensors"] * 7919 + case["elems"])
    w = [math.exp(r.uniform(0, 6)) for _ in range(case["tensors"])]
    return [max(1, int(case["elems"] * x / sum(w))) for x in w]


def work(case):
    op = case["op"]
    if op in ("router", "router_bwd"):
        T, E, k, b = case["T"], case["E"], case["k"], 4 if case["dtype"] == "f32" else 2
        if op == "router":
            return dict(bytes=T * E * b + T * k * 8 + (E * 4 if case["bias"] else 0) + (T * 4 + E * 4 if case["aux"] else 0),
                        flops=4 * T * E)
        return dict(bytes=T * E * (b + 4) + T * k * 8 + (T * 8 + E * 4 if case["aux"] else 0), flops=8 * T * E)
    if op == "combine_bwd":
        T, k, D, b = case["T"], case["k"], case["D"], 4 if case["dtype"] == "f32" else 2
        return dict(bytes=T * D * b + 2 * T * k * D * b + T * k * 12, flops=3 * T * k * D)
    if op.startswith("mx"):
        M, E = case["T"] * case["k"], case["E"]
        used = min(E, M)  # experts that can have rows at all
        per = 17 / 32     # bytes per element: half a byte and a scale per 32
        if op == "mx_gemm":
            N, K = case["N"], case["K"]
            return dict(bytes=(M + used * N) * K * per + M * N * (2 if case["out"] == "bf16" else 4), flops=2 * M * N * K)
        if op == "mx_gate":
            F, K = case["F"], case["K"]
            return dict(bytes=(M + used * 2 * F) * K * per + M * 3 * F * 2, flops=4 * M * F * K)
        D, F = case["D"], case["F"]
        return dict(bytes=case["T"] * D * 4 + used * 3 * F * D * per, flops=6 * M * D * F)
    n = sum(sizes(case))
    g, p = 4 if case["grad"] == "f32" else 2, 8 if case["param"] == "f32" else 4
    s = 16 if case["bits"] == 32 else 4 + 16 / STATE_BLOCK + 8
    return dict(bytes=n * (p + g + s + (2 if case["copy"] else 0)), flops=20 * n)


# ------------------------------------------------------------------ inputs

def _dt(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _routing(g, T, E, k, zipf, bad=0):
    """Distinct expert ids per token from biased logits, weights of the chosen, and the sorted layout."""
    logits = torch.randn(T, E, generator=g, device="cuda")
    rank = torch.randperm(E, generator=g, device="cuda") + 1
    ids = torch.sort(logits - zipf * torch.log(rank.float()), dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.softmax(torch.gather(logits, 1, ids), dim=1).contiguous()
    ids = ids.to(torch.int32).contiguous()
    if bad:
        at = torch.randperm(T * k, generator=g, device="cuda")[:bad]
        ids.view(-1)[at] = -1
    flat = ids.view(-1).long()
    valid = flat >= 0
    counts = torch.bincount(flat[valid], minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    order = torch.sort(torch.where(valid, flat, torch.full_like(flat, E)), stable=True).indices
    dest = torch.empty(T * k, dtype=torch.int32, device="cuda")
    dest[order] = torch.arange(T * k, dtype=torch.int32, device="cuda")
    dest[~valid] = -1
    ends = offsets.tolist()
    segments = [(e, ends[e], ends[e + 1]) for e in range(E) if ends[e + 1] > ends[e]]
    return ids, w, offsets, dest, order, segments


def _e2m1_values(device="cuda"):
    return torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6], device=device)


def _scaled(x, e):
    """x * 2^e exactly (e in [-254, 254], whole): by two powers made from their bits, each a normal number."""
    half = e.to(torch.int32) >> 1
    rest = e.to(torch.int32) - half
    return x * ((half + 127) << 23).view(torch.float32) * ((rest + 127) << 23).view(torch.float32)


def _mx_blocks(x):
    """MX elements (as values before their scale) and unbiased scale exponents of the last axis of x, in 32 bits."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    a = b.abs().amax(-1, keepdim=True)
    e = torch.where(a > 0, torch.frexp(a).exponent - 3, torch.full_like(a, -127, dtype=torch.int32)).clamp(-127, 127)
    r = _scaled(b, -e)
    mag = r.abs()
    q = torch.where(mag < 2, torch.round(mag * 2) / 2, torch.where(mag < 4, torch.round(mag), torch.round(mag / 2) * 2))
    return torch.copysign(q.clamp(max=6), r), e


def _mx_pack(x):
    """Packed E2M1 codes [..., K/2] and E8M0 bytes [..., K/32] of x."""
    v, e = _mx_blocks(x)
    mag = torch.bucketize(v.abs(), torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.], device=x.device))
    code = (mag + 8 * torch.signbit(v)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e.squeeze(-1) + 127).to(torch.uint8)


def _weights(g, *shape):
    return _mx_pack((torch.randn(*shape, generator=g, device="cuda") * 0.02).to(torch.bfloat16))


def _state_scale_codes(m, v, n):
    """8-bit states of a tensor in mid-training: codes and block scales of the values m and v."""
    half = torch.full((n,), 0x80008000, dtype=torch.int64, device="cuda")
    return _store8(m, v, half)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("router", "router_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = (torch.randn(T, E, generator=g, device="cuda") * 1.5).to(_dt(case["dtype"]))
        s["bias"] = torch.randn(E, generator=g, device="cuda") * 0.1 if case.get("bias") else None
        if op == "router_bwd":
            s["ids"] = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True).indices[:, :k].int().contiguous()
            s["dw"] = torch.randn(T, k, generator=g, device="cuda") * 1e-2
            s["lse"] = torch.logsumexp(s["logits"].float(), 1)
            s["dlse"] = torch.randn(T, generator=g, device="cuda") * 1e-3 if case["aux"] else None
            s["dsum"] = torch.randn(E, generator=g, device="cuda") * 1e-3 if case["aux"] else None
        return s
    if op == "combine_bwd":
        T, E, k, D, dt = case["T"], case["E"], case["k"], case["D"], _dt(case["dtype"])
        s["ids"], s["w"], s["offsets"], s["dest"], _, _ = _routing(g, T, E, k, 0.0, min(case["bad"], T * k))
        s["dout"] = (torch.randn(T, D, generator=g, device="cuda") * 1e-3).to(dt)
        s["y"] = torch.randn(T * k, D, generator=g, device="cuda").to(dt)
        return s
    if op.startswith("mx"):
        T, E, k = case["T"], case["E"], case["k"]
        s["ids"], s["w"], s["offsets"], s["dest"], order, s["segments"] = _routing(g, T, E, k, case["zipf"])
        if op == "mx_forward":
            D, F = case["D"], case["F"]
            x = torch.randn(T, D, generator=g, device="cuda")
            s["x"] = torch.where(torch.rand(T, D, generator=g, device="cuda") < 0.005, x * 16, x).to(torch.bfloat16)
            s["gu"], s["dn"] = _weights(g, E, 2 * F, D), _weights(g, E, D, F)
            if own:  # the buffers of one layer, which a program allocates once
                from nvfp4_quantized_moe_token_amd import moe_layer
                s["buf"] = moe_layer.BuffersMXFP4(T, k, E, D, F, torch.device("cuda"))
            return s
        s["a"] = _mx_pack(torch.randn(T, case["K"], generator=g, device="cuda").to(torch.bfloat16))
        s["a"] = tuple(a[order // k].contiguous() for a in s["a"])
        s["b"] = _weights(g, E, case["N"] if op == "mx_gemm" else 2 * case["F"], case["K"])
        return s
    # adamw: views of flat buffers, every tensor at a multiple of 64 elements, as trainers keep them
    n = sizes(case)
    starts = [0]
    for x in n:
        starts.append(starts[-1] + (x + 63) // 64 * 64)
    total = starts[-1]

    def views(t):
        return [t[a:a + x] for a, x in zip(starts, n)]

    s["views"] = views

    flat = (torch.randn(total, generator=g, device="cuda") * 0.02).to(_dt(case["param"]))
    grad = (torch.randn(total, generator=g, device="cuda") * 1e-3).to(_dt(case["grad"]))
    m = torch.randn(total, generator=g, device="cuda") * 3e-4
    v = torch.rand(total, generator=g, device="cuda") * 2e-6 + 1e-8
    s.update(step=99, seed=12345, p=views(flat), g=views(grad),
             hyper=dict(lr=3e-4, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1))
    s["flat"] = dict(p=flat, m=m, v=v)
    s["copy"] = None
    if case["copy"]:
        s["flat"]["copy"] = flat.to(torch.bfloat16)
        s["copy"] = views(s["flat"]["copy"])
    if case["bits"] == 32:
        s["m"], s["v"] = views(m), views(v)
        state = dict(exp_avg=s["m"], exp_avg_sq=s["v"])
    else:
        packed = [_state_scale_codes(a, b, x) for a, b, x in zip(views(m), views(v), n)]
        s["m"], s["ms"], s["v"], s["vs"] = (list(t) for t in zip(*packed))
        s["values"] = views(m), views(v)  # where the states are read back to
        state = dict(exp_avg=s["m"], avg_scale=s["ms"], exp_avg_sq=s["v"], avg_sq_scale=s["vs"])
    if own:  # the optimizer, which a program makes once
        from nvfp4_quantized_moe_token_amd import optim
        s["opt"] = optim.AdamW(s["p"], params_bf16=s["copy"], state_bits=case["bits"], step=s["step"], seed=s["seed"],
                               state=state, **s["hyper"])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _OWN[s["case"]["op"]](s) if own else _PLAIN[s["case"]["op"]](s)


# ---- plain forms

def _router(s):
    c = s["case"]
    l = s["logits"].float()
    key = l + s["bias"] if s["bias"] is not None else l
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    chosen = torch.gather(l, 1, ids)
    top = l.amax(1, keepdim=True)
    ex = torch.exp(l - top)
    total = ex.sum(1, keepdim=True)
    if c["score"] == "topk":
        w = torch.exp(chosen - chosen.amax(1, keepdim=True))
        w = w / w.sum(1, keepdim=True)
    else:
        w = torch.exp(chosen - top) / total
    out = dict(ids=ids.to(torch.int32), w=w)
    if c["aux"]:
        out["lse"] = (top + torch.log(total)).squeeze(1)
        out["prob_sum"] = (ex / total).sum(0)
    return out


def _router_bwd(s):
    c = s["case"]
    l, ids, dw = s["logits"].float(), s["ids"].long(), s["dw"]
    p = torch.exp(l - s["lse"][:, None])
    chosen = torch.gather(l, 1, ids)
    if c["score"] == "topk":
        q = torch.exp(chosen - chosen.amax(1, keepdim=True))
        q = q / q.sum(1, keepdim=True)
        d = torch.zeros_like(l).scatter_add(1, ids, q * (dw - (q * dw).sum(1, keepdim=True)))
    else:
        q = torch.gather(p, 1, ids)
        d = torch.zeros_like(l).scatter_add(1, ids, q * dw) - p * (q * dw).sum(1, keepdim=True)
    if c["aux"]:
        d = d + p * (s["dlse"][:, None] + s["dsum"] - (p * s["dsum"]).sum(1, keepdim=True))
    return d


def _combine_bwd(s):
    c = s["case"]
    T, k, D = c["T"], c["k"], c["D"]
    dest = s["dest"].long()
    ok = (dest >= 0)[:, None]
    rows = dest.clamp(min=0)
    up = s["dout"].float()[:, None, :].expand(T, k, D)
    y = torch.where(ok, s["y"][rows].float(), torch.zeros((), device="cuda")).view(T, k, D)
    dw = (up * y).sum(2)
    dy = torch.zeros(T * k + 1, D, dtype=s["y"].dtype, device="cuda")  # dropped assignments go to the row behind the last
    dy[torch.where(ok[:, 0], dest, T * k)] = (up * s["w"][:, :, None]).to(dy.dtype).view(T * k, D)
    return dict(dy=dy[:T * k], dw=dw)


def _dequant(q, scale):
    code = torch.stack((q & 15, q >> 4), -1).flatten(-2).long()
    v = _e2m1_values()[code].unflatten(-1, (-1, BLOCK))
    return _scaled(v, scale.int()[..., None] - 127).flatten(-2)


def _silu_gate(y1):
    g, u = y1.float().chunk(2, -1)
    return (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16)


# The experts' products go expert by expert (a loop over the experts that have rows): their row counts differ.

def _mx_gemm(s):
    a = _dequant(*s["a"])
    c = torch.empty(a.shape[0], s["case"]["N"], dtype=_dt(s["case"]["out"]), device="cuda")
    for e, lo, hi in s["segments"]:
        c[lo:hi] = a[lo:hi] @ _dequant(s["b"][0][e], s["b"][1][e]).t()
    return c


def _mx_gate(s):
    a = _dequant(*s["a"])
    y1 = torch.empty(a.shape[0], 2 * s["case"]["F"], dtype=torch.bfloat16, device="cuda")
    for e, lo, hi in s["segments"]:
        y1[lo:hi] = a[lo:hi] @ _dequant(s["b"][0][e], s["b"][1][e]).t()
    return dict(y1=y1, h=_silu_gate(y1))


def _mx_values(x):
    v, e = _mx_blocks(x)
    return _scaled(v, e).flatten(-2)


def _mx_forward(s):
    c = s["case"]
    order = torch.sort(s["ids"].view(-1), stable=True).indices
    a = _mx_values(s["x"])[order // c["k"]]
    y2 = torch.empty(a.shape[0], c["D"], dtype=torch.bfloat16, device="cuda")
    for e, lo, hi in s["segments"]:
        y1 = (a[lo:hi] @ _dequant(s["gu"][0][e], s["gu"][1][e]).t()).to(torch.bfloat16)
        y2[lo:hi] = _mx_values(_silu_gate(y1)) @ _dequant(s["dn"][0][e], s["dn"][1][e]).t()
    dest = torch.empty_like(order)
    dest[order] = torch.arange(order.numel(), device="cuda")
    return (y2[dest].float().view(c["T"], c["k"], c["D"]) * s["w"][:, :, None]).sum(1).to(torch.bfloat16)


def _mix(x):
    """A 32-bit mixer (multiply and xor-shift), on int64 tensors that hold 32 bits; also on plain ints."""
    x = x ^ (x >> 16)
    x = (x * 0x9E3779B9) & M32
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & M32
    return x ^ (x >> 16)


def _random_bits(seed, step, tensor, n):
    key = _mix((_mix((_mix(seed & M32) + step) & M32) + tensor) & M32)
    i = torch.arange(n, dtype=torch.int64, device="cuda")
    return _mix(((i * 0x9E3779B1) & M32) ^ key ^ (((i >> 32) * 0x6A09E667) & M32))


def _in_blocks(x):
    pad = -x.numel() % STATE_BLOCK
    return (torch.cat([x, x.new_zeros(pad)]) if pad else x).view(-1, STATE_BLOCK)


def _store8(m, v, r):
    """Codes and block scales of first and second moments m and v, rounded with the random bits r."""
    n = m.numel()
    ms = _in_blocks(m).abs().amax(1) / 448
    vs = _in_blocks(v).amax(1)
    sm, sv = (t.repeat_interleave(STATE_BLOCK)[:n] for t in (ms, vs))
    y = torch.where(sm > 0, m.abs() / sm, torch.zeros_like(m)).clamp(max=448)
    hi = (r >> 16).to(torch.int32)
    low = torch.floor(y * 512 + hi.float() / 65536).to(torch.int32)
    code = torch.where(y < 2 ** -6, low, ((y.view(torch.int32) + (hi << 4)) >> 20) - (120 << 3))
    mc = (code | torch.where(torch.signbit(m), 128, 0)).to(torch.uint8)
    y = torch.where(sv > 0, v / sv, torch.zeros_like(v))
    code = ((y.view(torch.int32) + ((r & 0xFFFF) << 4).to(torch.int32)) >> 20) - 762
    vc = torch.where(y > 0, code.clamp(1, 254), 0).to(torch.uint8)
    return mc, ms, vc, vs


def _load8(mc, ms, vc, vs):
    n = mc.numel()
    sm, sv = (t.repeat_interleave(STATE_BLOCK)[:n] for t in (ms, vs))
    v = ((vc.to(torch.int32) + 762) << 20).view(torch.float32)
    return mc.view(torch.float8_e4m3fn).float() * sm, torch.where(vc > 0, v, torch.zeros_like(v)) * sv


def _adamw(s):
    h, eight = s["hyper"], s["case"]["bits"] == 8
    b1, b2 = h["betas"]
    s["step"] += 1
    g = [x.float() for x in s["g"]]
    p = [x.float() for x in s["p"]]
    m, v = s["m"], s["v"]
    if eight:
        m, v = (list(t) for t in zip(*[_load8(*x) for x in zip(s["m"], s["ms"], s["v"], s["vs"])]))
    m = torch._foreach_add(torch._foreach_mul(m, b1), torch._foreach_mul(g, 1 - b1))
    v = torch._foreach_add(torch._foreach_mul(v, b2), torch._foreach_mul(torch._foreach_mul(g, g), 1 - b2))
    del g
    den = torch._foreach_sqrt(v)
    torch._foreach_mul_(den, 1 / math.sqrt(1 - b2 ** s["step"]))
    torch._foreach_add_(den, h["eps"])
    den = torch._foreach_div(m, den)
    torch._foreach_mul_(den, -h["lr"] / (1 - b1 ** s["step"]))
    p = torch._foreach_add(torch._foreach_mul(p, 1 - h["lr"] * h["weight_decay"]), den)
    del den
    bits = [_random_bits(s["seed"], s["step"], i, x.numel()) if eight or s["case"]["param"] == "bf16" else None
            for i, x in enumerate(p)]
    if s["case"]["param"] == "bf16":
        p = [((x.view(torch.int32) + (_mix((r + 0x6A09E667) & M32) >> 16).to(torch.int32)) & -65536).view(torch.float32)
             for x, r in zip(p, bits)]
    torch._foreach_copy_(s["p"], p)
    if s["copy"]:
        torch._foreach_copy_(s["copy"], p)
    if eight:
        new = [_store8(a, b, r) for a, b, r in zip(m, v, bits)]
        for name, t in zip(("m", "ms", "v", "vs"), zip(*new)):
            torch._foreach_copy_(s[name], list(t))
        m, v = (list(t) for t in zip(*[_load8(*x) for x in new]))
        torch._foreach_copy_(s["values"][0], m)
        torch._foreach_copy_(s["values"][1], v)
    else:
        torch._foreach_copy_(s["m"], m)
        torch._foreach_copy_(s["v"], v)
    return s["flat"]


_PLAIN = dict(router=_router, router_bwd=_router_bwd, combine_bwd=_combine_bwd, mx_gemm=_mx_gemm, mx_gate=_mx_gate,
              mx_forward=_mx_forward, adamw=_adamw)


# ---- through the package

def _own_router(s):
    from nvfp4_quantized_moe_token_amd import ops
    c = s["case"]
    r = ops.moe_router(s["logits"], c["k"], bias=s["bias"], score=_score(ops, c), want_lse=c["aux"], want_prob_sum=c["aux"])
    out = dict(ids=r["topk_ids"], w=r["topk_w"])
    if c["aux"]:
        out.update(lse=r["lse"], prob_sum=r["prob_sum"])
    return out


def _score(ops, c):
    return ops.ROUTER_TOPK_SOFTMAX if c["score"] == "topk" else ops.ROUTER_SOFTMAX


def _own_router_bwd(s):
    from nvfp4_quantized_moe_token_amd import ops
    return ops.moe_router_bwd(s["logits"], s["ids"], s["dw"], score=_score(ops, s["case"]), lse=s["lse"], d_lse=s["dlse"],
                              d_prob_sum=s["dsum"], out_dtype=torch.float32)


def _own_combine_bwd(s):
    from nvfp4_quantized_moe_token_amd import ops
    dy, dw = ops.moe_unpermute_bwd(s["dout"], s["y"], s["dest"], s["offsets"], s["case"]["k"], topk_w=s["w"])
    return dict(dy=dy, dw=dw)


def _own_mx_gemm(s):
    from nvfp4_quantized_moe_token_amd import ops
    return ops.grouped_gemm_mxfp4(*s["a"], *s["b"], s["offsets"], out_dtype=_dt(s["case"]["out"]))


def _own_mx_gate(s):
    from nvfp4_quantized_moe_token_amd import ops
    r = ops.grouped_gemm_mxfp4_silu_gate(*s["a"], *s["b"], s["offsets"])
    return dict(y1=r["y1"], h=r["h"])


def _own_mx_forward(s):
    from nvfp4_quantized_moe_token_amd import moe_layer
    gu, dn = (dict(q=q, s=sc) for q, sc in (s["gu"], s["dn"]))
    moe_layer.forward_mxfp4(s["x"], s["ids"], s["w"], gu, dn, s["buf"])
    return s["buf"].out


def _own_adamw(s):
    s["opt"].step(s["g"])
    if s["case"]["bits"] == 8:
        s["opt"].state_values(out=s["values"])
    return s["flat"]


_OWN = dict(router=_own_router, router_bwd=_own_router_bwd, combine_bwd=_own_combine_bwd, mx_gemm=_own_mx_gemm,
            mx_gate=_own_mx_gate, mx_forward=_own_mx_forward, adamw=_own_adamw)


# ------------------------------------------------------------------ the same in 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s, case)


def _x_pick(key, k):
    """The k best columns of each row, best first, ties to the lower column, one at a time."""
    key, got = key.clone(), []
    for _ in range(k):
        best = key.max(1, keepdim=True).values
        col = torch.arange(key.shape[1], device=key.device).expand_as(key)
        i = torch.where(key == best, col, key.shape[1]).min(1, keepdim=True).values
        got.append(i)
        key.scatter_(1, i, -math.inf)
    return torch.cat(got, 1)


def _x_router(s, c):
    l = s["logits"].double()
    key = s["logits"].float() + (s["bias"] if s["bias"] is not None else 0)
    ids = _x_pick(key, c["k"])
    logp = torch.log_softmax(l, 1)
    w = torch.gather(logp, 1, ids)
    w = torch.softmax(w, 1) if c["score"] == "topk" else w.exp()
    out = dict(ids=None, w=w)
    if c["aux"]:
        out.update(lse=torch.logsumexp(l, 1), prob_sum=logp.exp().sum(0))
    return out


def _x_router_bwd(s, c):
    l = s["logits"].double().requires_grad_(True)
    logp = torch.log_softmax(l, 1)
    w = torch.gather(logp, 1, s["ids"].long())
    w = torch.softmax(w, 1) if c["score"] == "topk" else w.exp()
    loss = (w * s["dw"].double()).sum()
    if c["aux"]:
        loss = loss + (torch.logsumexp(l, 1) * s["dlse"].double()).sum() + (logp.exp().sum(0) * s["dsum"].double()).sum()
    return torch.autograd.grad(loss, l)[0]


def _x_combine_bwd(s, c):
    T, k = c["T"], c["k"]
    dest, w = s["dest"].long().view(T, k), s["w"].double()
    up, y = s["dout"].double(), s["y"].double()
    dy, dw = torch.zeros_like(y), torch.zeros_like(w)
    for j in range(k):
        t = torch.nonzero(dest[:, j] >= 0).squeeze(1)
        d = dest[t, j]
        dy[d] = up[t] * w[t, j, None]
        dw[t, j] = (up[t] * y[d]).sum(1)
    return dict(dy=dy, dw=dw)


def _x_pow2(e):
    """2^e in 64 bits, exactly: the exponent field itself."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _x_deq(q, scale):
    lo, hi = (q & 15).long(), (q >> 4).long()
    code = torch.empty(*q.shape[:-1], q.shape[-1] * 2, dtype=torch.long, device=q.device)
    code[..., 0::2], code[..., 1::2] = lo, hi
    v = _e2m1_values().double()[code]
    return v * _x_pow2(scale.long() - 127).repeat_interleave(BLOCK, -1)


def _x_products(a, b, segments, n):
    out = torch.zeros(a.shape[0], n, dtype=torch.float64, device="cuda")
    for e, lo, hi in segments:
        out[lo:hi] = a[lo:hi] @ _x_deq(b[0][e], b[1][e]).t()
    return out


def _x_mx_gemm(s, c):
    return _x_products(_x_deq(*s["a"]), s["b"], s["segments"], c["N"])


def _x_gate(y1):
    # H is defined on the bf16 values of Y1
    y = y1.to(torch.bfloat16).double()
    F = y.shape[1] // 2
    return y[:, :F] * torch.sigmoid(y[:, :F]) * y[:, F:]


def _x_mx_gate(s, c):
    y1 = _x_products(_x_deq(*s["a"]), s["b"], s["segments"], 2 * c["F"])
    return dict(y1=y1, h=_x_gate(y1))


def _x_quant(x):
    """Values of x (bf16 values in 64 bits) after MXFP4: the nearest element, ties to the even code."""
    b = x.unflatten(-1, (-1, BLOCK))
    a = b.abs().amax(-1, keepdim=True)
    e = torch.where(a > 0, torch.floor(torch.log2(a)) - 2, torch.full_like(a, -127.0)).clamp(-1000, 1000)
    e = torch.where(_x_pow2(e + 2) > a, e - 1, e)           # log2 may round up to the next power
    e = torch.where(_x_pow2(e + 3) <= a, e + 1, e).clamp(-127, 127)
    e = torch.where(a > 0, e, torch.full_like(e, -127.0))
    r = (b.abs() / _x_pow2(e)).clamp(max=6.0)
    grid = _e2m1_values().double()[:8]
    mid = (grid[1:] + grid[:-1]) / 2
    at = torch.bucketize(r, mid)                                    # a tie stays with the lower code
    tie = (r == mid[at.clamp(max=6)]) & (at % 2 == 1)               # the lower code is odd: take the even one above
    return (grid[at + tie] * _x_pow2(e) * torch.sign(b)).flatten(-2)


def _x_mx_forward(s, c):
    dest = s["dest"].long()
    src = torch.empty_like(dest)
    src[dest] = torch.arange(dest.numel(), device="cuda")
    a = _x_quant(s["x"].double())[src // c["k"]]
    y1 = _x_products(a, s["gu"], s["segments"], 2 * c["F"])
    h = _x_quant(_x_gate(y1).to(torch.bfloat16).double())           # H and Y2 are stored in bf16
    del a, y1
    y2 = _x_products(h, s["dn"], s["segments"], c["D"]).to(torch.bfloat16)
    out = torch.zeros(c["T"], c["D"], dtype=torch.float64, device="cuda")
    for j in range(c["k"]):
        out += s["w"][:, j, None].double() * y2[dest.view(c["T"], c["k"])[:, j]].double()
    return out


def _x_adamw(s, c):
    h, t = s["hyper"], s["step"] + 1
    b1, b2 = h["betas"]
    out = {name: x.double() for name, x in s["flat"].items()}
    at = {name: s["views"](x) for name, x in out.items()}
    for i, g in enumerate(s["g"]):
        g = g.double()
        if c["bits"] == 8:
            n = g.numel()
            sm, sv = (x[i].double().repeat_interleave(STATE_BLOCK)[:n] for x in (s["ms"], s["vs"]))
            a = s["m"][i].view(torch.float8_e4m3fn).double() * sm
            code = s["v"][i].double()
            # 254 stands for 1, eight codes per octave, linear within one; 0 for zero
            e, f = torch.floor((code + 762) / 8) - 127, (code + 762) % 8
            b = torch.where(code > 0, _x_pow2(e) * (1 + f / 8), torch.zeros_like(code)) * sv
        else:
            a, b = s["m"][i].double(), s["v"][i].double()
        a, b = b1 * a + (1 - b1) * g, b2 * b + (1 - b2) * g * g
        step = (a / (1 - b1 ** t)) / ((b / (1 - b2 ** t)).sqrt() + h["eps"])
        w = s["p"][i].double()
        w = w - h["lr"] * (step + h["weight_decay"] * w)
        at["p"][i].copy_(w)
        at["m"][i].copy_(a)
        at["v"][i].copy_(b)
        if c["copy"]:
            at["copy"][i].copy_(w)
    if c["bits"] == 8:  # rounded with random bits: these have no value of their own in 64 bits
        out.update(m=None, v=None)
    return out


_EXACT = dict(router=_x_router, router_bwd=_x_router_bwd, combine_bwd=_x_combine_bwd, mx_gemm=_x_mx_gemm,
              mx_gate=_x_mx_gate, mx_forward=_x_mx_forward, adamw=_x_adamw)
