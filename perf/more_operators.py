"""Measured cases of the MXFP4 experts and of the orthogonalised update.

Operators (the formulas are those of include/moe.h):

  quantise       E2M1 codes with one power-of-two scale for each block of 32
                 values of a row, and the values that those stand for
  experts        both expert layers over the expert segments: codes and block
                 scales in, bf16 rows out, the hidden rows as codes in between
  down           second expert layer alone
  layer          the whole MoE layer with such experts, from bf16 tokens to bf16 y
  orthogonalise  momentum and Newton-Schulz products of a batch of gradients

Where ``own`` is true, ``run`` calls the library; else it computes the plain
form with elementary torch operations.
"""
import math

import torch

own = False

BLOCK = 32
STEPS = 5
BETA = 0.95
COEF = (3.4445, -4.7750, 2.0315)


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a decoding batch's tokens before the experts: latency of two small calls
        dict(name="quantise tokens, decode", kind="quantise", rows=8, K=4096, src="bf16"),
        # fp32 master weights of an expert after an optimiser step, for the next forward
        dict(name="quantise weights", kind="quantise", rows=28672, K=4096, src="f32"),
        # one token of one sequence: two experts' weights are streamed
        dict(name="experts, one token", kind="experts", T=1, d=4096, E=8, k=2, F=14336, act="swiglu", skew=0.0),
        # a prompt batch with uneven experts
        dict(name="experts, prompt", kind="experts", T=4096, d=4096, E=8, k=2, F=14336, act="swiglu", skew=1.2),
        # many small experts with few, ragged rows each
        dict(name="experts, many", kind="experts", T=16383, d=1024, E=512, k=2, F=512, act="relu", skew=0.0),
        # a decoding batch
        dict(name="down, decode", kind="down", T=33, d=4096, E=8, k=2, F=14336, act="swiglu", skew=0.0),
        # mid-sized segments of a prompt batch
        dict(name="down, prompt", kind="down", T=4096, d=4608, E=16, k=2, F=12288, act="swiglu", skew=0.0),
        # the layer on a small serving batch of short experts
        dict(name="layer, serving", kind="layer", T=61, d=512, E=64, k=2, F=1024, act="relu", normalize=False, cf=0.0),
        # the layer on a prompt batch: normalised gate, capacity limit
        dict(name="layer, prompt", kind="layer", T=4096, d=4608, E=16, k=2, F=12288, act="swiglu", normalize=True, cf=1.25),
        # the gate's weights: a short wide matrix
        dict(name="orthogonalise, gate", kind="orthogonalise", count=1, rows=8, cols=4096, src="f32", momentum="nesterov"),
        # the first layers of many small experts, gradients kept in bf16, the momentum elsewhere
        dict(name="orthogonalise, many", kind="orthogonalise", count=64, rows=1024, cols=512, src="bf16", momentum="none"),
        # the second layers of two large experts
        dict(name="orthogonalise, large", kind="orthogonalise", count=2, rows=4096, cols=14336, src="f32", momentum="nesterov"),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["quantise", "experts", "experts", "down", "layer", "orthogonalise", "orthogonalise"])
    if kind == "quantise":
        K = BLOCK * _log_int(rng, 1, 448)
        rows = _log_int(rng, 1, max(2, min(65536, 110_000_000 // K)))
        return dict(kind=kind, rows=rows, K=K, src=rng.choice(["bf16", "f32"]))
    if kind == "orthogonalise":
        rows, cols = _log_int(rng, 1, 6000), _log_int(rng, 1, 6000)
        m, n = min(rows, cols), max(rows, cols)
        most = max(1, min(64, int(1.0e12 / (4.0 * m * m * n + 2.0 * m * m * m)), 60_000_000 // (m * n)))
        return dict(kind=kind, count=_log_int(rng, 1, most), rows=rows, cols=cols, src=rng.choice(["bf16", "f32"]),
                    momentum=rng.choice(["none", "plain", "nesterov"]))
    d = 128 * _log_int(rng, 2, 36)
    F = 128 * _log_int(rng, 2, 96)
    E = _log_int(rng, 2, 128)
    E = max(2, min(E, 400_000_000 // (d * F)))
    k = rng.randint(1, min(E, 4))
    T = max(1, _log_int(rng, 1, 8192) // k)
    act = rng.choice(["relu", "swiglu"])
    if kind == "layer":
        return dict(kind=kind, T=T, d=d, E=E, k=k, F=F, act=act, normalize=rng.random() < 0.5, cf=rng.choice([0.0, 1.0, 1.25]))
    return dict(kind=kind, T=T, d=d, E=E, k=k, F=F, act=act, skew=rng.choice([0.0, 1.2]) if E <= 16 else 0.0)


# ------------------------------------------------------------------ the inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _scale_exponent(amax):
    """The smallest e with amax <= 6 * 2^e, at least -127; 0 for amax 0."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.75, x - 3, x - 2)
    return torch.where(amax > 0, e, torch.zeros_like(e)).clamp(min=-127)


def _code(v):
    """E2M1 code of each v, |v| <= 6: the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even code, and the sign bit."""
    a = v.abs()
    c = (a > 0.25).to(torch.uint8)
    for low, even in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        c += (a >= low) if even else (a > low)
    return c | (torch.signbit(v).to(torch.uint8) << 3)


def _value(c):
    """fp32 value of each E2M1 code."""
    m = (c & 7).float()
    a = torch.where(m < 4, 0.5 * m, torch.where(m < 6, m - 2, 2 * m - 8))
    return torch.where(c >= 8, -a, a)


def _quantise(x):
    """Packed codes [..., K / 2] (the even value in the low half) and scale bytes [..., K / 32] of x [..., K] (fp32)."""
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    e = _scale_exponent(b.abs().amax(dim=-1))
    c = _code(torch.ldexp(b, -e[..., None])).reshape(*x.shape[:-1], -1, 2)
    return c[..., 0] | (c[..., 1] << 4), (e + 127).to(torch.uint8)


def _widen(codes, scales):
    """fp32 values [..., K] of packed codes and scale bytes."""
    v = _value(torch.stack([codes & 15, codes >> 4], dim=-1))
    v = v.reshape(*scales.shape, BLOCK) * torch.ldexp(torch.ones(scales.shape, device=scales.device), scales.to(torch.int32) - 127)[..., None]
    return v.reshape(*codes.shape[:-1], -1)


def _weights(g, E, rows, cols):
    """Codes [E][rows][cols/2] and scales [E][rows][cols/32] of weights N(0, 0.02^2)."""
    codes = torch.empty(E, rows, cols // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, rows, cols // BLOCK, dtype=torch.uint8, device="cuda")
    part = max(1, 64_000_000 // (rows * cols))  # experts at a time
    for e in range(0, E, part):
        n = min(part, E - e)
        codes[e : e + n], scales[e : e + n] = _quantise(torch.randn(n, rows, cols, device="cuda", generator=g) * 0.02)
    return codes, scales


def _rows_of_codes(g, rows, K):
    """Codes and scales of activations with rows of uneven size."""
    x = torch.randn(rows, K, device="cuda", generator=g)
    return _quantise(x * torch.exp(torch.randn(rows, 1, device="cuda", generator=g)))


def _routing(g, c):
    """Expert segments of T tokens with k experts each: src_token [T*k], offsets [E+1]."""
    T, E, k = c["T"], c["E"], c["k"]
    z = torch.randn(T, E, device="cuda", generator=g)
    z = z - c["skew"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    idx = torch.topk(z, k, dim=1).indices.reshape(-1)
    order = torch.sort(idx, stable=True).indices
    counts = torch.bincount(idx, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    return (order // k).to(torch.int32), offsets, int(counts.max())


def _gradients(g, count, rows, cols, tokens):
    """Weight gradients: sums over tokens of uneven size of (output gradient) x (input)."""
    a = torch.randn(count, rows, tokens, device="cuda", generator=g) * torch.exp(torch.randn(count, 1, tokens, device="cuda", generator=g))
    b = torch.relu(torch.randn(count, tokens, cols, device="cuda", generator=g))
    return torch.bmm(a, b) * (1e-4 / math.sqrt(tokens))


def prepare(case, seed):
    c, g = dict(case), _generator(seed)
    if c["kind"] == "quantise":
        src = torch.randn(c["rows"], c["K"], device="cuda", generator=g) * 0.02
        src = src * torch.exp(torch.randn(c["rows"], 1, device="cuda", generator=g))
        return dict(case=c, src=src.to(torch.bfloat16) if c["src"] == "bf16" else src, kept={})
    if c["kind"] == "orthogonalise":
        n, rows, cols = c["count"], c["rows"], c["cols"]
        # the momentum holds many steps' tokens; without one the gradient is a large batch's
        many, few = 2 * min(rows, cols) + 64, min(rows, cols) // 2 + 16
        held = c["momentum"] != "none"
        grad = _gradients(g, n, rows, cols, few if held else many)
        mom = _gradients(g, n, rows, cols, many) * 8.0 if held else None
        return dict(case=c, grad=grad.to(torch.bfloat16) if c["src"] == "bf16" else grad, mom=mom, kept={})
    d, F, E = c["d"], c["F"], c["E"]
    n1 = 2 * F if c["act"] == "swiglu" else F
    w2, s2 = _weights(g, E, d, F)
    if c["kind"] == "down":
        src, offsets, longest = _routing(g, c)
        a, sa = _rows_of_codes(g, c["T"] * c["k"], F)
        return dict(case=c, a=a, sa=sa, offsets=offsets, longest=longest, w2=w2, s2=s2, kept={})
    w1, s1 = _weights(g, E, n1, d)
    if c["kind"] == "experts":
        src, offsets, longest = _routing(g, c)
        a, sa = _rows_of_codes(g, c["T"], d)
        return dict(case=c, a=a, sa=sa, src=src, offsets=offsets, longest=longest, w1=w1, s1=s1, w2=w2, s2=s2, kept={})
    x = torch.randn(c["T"], d, device="cuda", generator=g).to(torch.bfloat16)
    gate = (torch.randn(E, d, device="cuda", generator=g) / math.sqrt(d)).to(torch.bfloat16)
    bias = torch.randn(E, device="cuda", generator=g) * 0.1
    return dict(case=c, x=x, gate=gate, bias=bias, w1=w1, s1=s1, w2=w2, s2=s2, kept={})


# ------------------------------------------------------------------ the plain forms
def _plain_grouped(a, w, offsets, longest):
    """Row r of expert e's segment times w[e]^T: the segments padded to the longest, one batched product."""
    E, P = w.shape[0], a.shape[0]
    first = offsets[:-1].long()
    count = offsets[1:].long() - first
    at = torch.arange(longest, device=a.device)
    row = first[:, None] + at[None, :]
    held = at[None, :] < count[:, None]
    padded = a[row.clamp(max=P - 1)] * held[:, :, None]
    out = torch.bmm(w, padded.transpose(1, 2).contiguous())  # [E][n][longest]
    rows = torch.arange(P, device=a.device)
    e = torch.searchsorted(offsets[1:].long(), rows, right=True).clamp(max=E - 1)
    return out.transpose(1, 2)[e, (rows - first[e]).clamp(0, max(longest - 1, 0))]


def _plain_activation(u, act):
    if act == "relu":
        return torch.clamp(u, min=0)
    g, v = u.chunk(2, dim=1)
    return g / (1 + torch.exp(-g)) * v


def _plain_experts(a, st, offsets, longest):
    """Expert outputs (fp32) of fp32 rows a that are values of codes."""
    u = _plain_grouped(a, _widen(st["w1"], st["s1"]), offsets, longest)
    h = _widen(*_quantise(_plain_activation(u, st["case"]["act"])))
    del u
    return _plain_grouped(h, _widen(st["w2"], st["s2"]), offsets, longest)


def _plain_layer(st):
    c = st["case"]
    T, E, k = c["T"], c["E"], c["k"]
    x = st["x"].float()
    # the gate's logits decide which experts a token takes: 64 bits, rounded once
    z = (st["x"].double() @ st["gate"].double().t() + st["bias"].double()).float()
    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
    t = z.double()
    if c["normalize"]:
        t = t - t.mean(dim=1, keepdim=True)
        t = t / t.square().mean(dim=1, keepdim=True).sqrt()
    t = torch.exp(t - t.amax(dim=1, keepdim=True))
    p = (t / t.sum(dim=1, keepdim=True)).float()
    weight = p.gather(1, order)
    chosen = torch.zeros(T, E, dtype=torch.int64, device=x.device).scatter_(1, order, 1)
    rank = (chosen.cumsum(0) - chosen).gather(1, order)
    limit = math.ceil(c["cf"] * T * k / E) if c["cf"] > 0 else T
    kept = rank < limit
    count = chosen.sum(0).clamp(max=limit)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=x.device)
    offsets[1:] = torch.cumsum(count, 0)
    # a dropped choice takes the row behind the last one
    slot = torch.where(kept, offsets[order].long() + rank, T * k)
    token = torch.zeros(T * k + 1, dtype=torch.int64, device=x.device)
    token[slot.reshape(-1)] = torch.arange(T, device=x.device).repeat_interleave(k)
    a = _widen(*_quantise(x))
    y = _plain_experts(a[token[: T * k]], st, offsets, min(T, limit))
    y = y[slot.clamp(max=T * k - 1)] * (weight * kept)[:, :, None]
    return dict(y=y.sum(dim=1).to(torch.bfloat16), topk_idx=order.to(torch.int32), topk_w=weight)


def _plain_orthogonalise(st):
    c = st["case"]
    u = st["grad"].float()
    if st["mom"] is not None:
        st["mom"].mul_(BETA).add_(u)
        u = u + BETA * st["mom"] if c["momentum"] == "nesterov" else st["mom"]
    norm = u.double().square().sum(dim=(1, 2), keepdim=True).sqrt()
    x = u * torch.where(norm > 0, 1 / norm, torch.zeros_like(norm)).float()
    tall = c["rows"] > c["cols"]
    if tall:
        x = x.transpose(1, 2).contiguous()
    a, b, q = COEF
    for _ in range(STEPS):
        s = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * s + q * torch.bmm(s, s), x)
    out = (x.transpose(1, 2) if tall else x).to(torch.bfloat16).contiguous()
    return dict(out=out, momentum=st["mom"]) if st["mom"] is not None else dict(out=out)


def _plain(st):
    c = st["case"]
    if c["kind"] == "quantise":
        codes, scales = _quantise(st["src"].float())
        return dict(values=_widen(codes, scales).to(torch.bfloat16), scales=scales.view(torch.float8_e8m0fnu))
    if c["kind"] == "orthogonalise":
        return _plain_orthogonalise(st)
    if c["kind"] == "layer":
        return _plain_layer(st)
    a = _widen(st["a"], st["sa"])
    if c["kind"] == "down":
        return dict(y=_plain_grouped(a, _widen(st["w2"], st["s2"]), st["offsets"], st["longest"]).to(torch.bfloat16))
    return dict(y=_plain_experts(a[st["src"].long()], st, st["offsets"], st["longest"]).to(torch.bfloat16))


# ------------------------------------------------------------------ the library's calls
def _own(st):
    import mixture_experts_layer_logit_amd as moe

    c, kept = st["case"], st["kept"]
    new = not kept

    def keep(name, *shape, dtype):
        if new:
            kept[name] = torch.empty(*shape, dtype=dtype, device="cuda")
        return kept[name]

    if c["kind"] == "quantise":
        rows, K = c["rows"], c["K"]
        codes = keep("codes", rows, K // 2, dtype=torch.uint8)
        scales = keep("scales", rows, K // BLOCK, dtype=torch.uint8)
        values = keep("values", rows, K, dtype=torch.bfloat16)
        moe.moe_quantize_mxfp4(st["src"], codes, scales)
        moe.moe_dequantize_mxfp4(codes, scales, values)
        return dict(values=values, scales=scales.view(torch.float8_e8m0fnu))
    if c["kind"] == "orthogonalise":
        n, rows, cols = c["count"], c["rows"], c["cols"]
        if new:
            kept["ws"] = torch.empty(moe.moe_orthogonalize_workspace_size(n, rows, cols), dtype=torch.uint8, device="cuda")
        out = keep("out", n, rows, cols, dtype=torch.bfloat16)
        moe.moe_orthogonalize(st["grad"], out, momentum=st["mom"], beta=BETA, nesterov=c["momentum"] == "nesterov", steps=STEPS,
                              ws=kept["ws"])
        return dict(out=out, momentum=st["mom"]) if st["mom"] is not None else dict(out=out)
    T, d, E, k, F = c["T"], c["d"], c["E"], c["k"], c["F"]
    if new:
        kept["p"] = moe.problem(T, d, E, k, F, act=c["act"], normalize=c.get("normalize", False), cf=c.get("cf", 0.0))
        kept["ws"] = torch.empty(moe.moe_mxfp4_workspace_size(kept["p"]), dtype=torch.uint8, device="cuda")
    p, ws = kept["p"], kept["ws"]
    if c["kind"] == "layer":
        y = keep("y", T, d, dtype=torch.bfloat16)
        idx = keep("idx", T, k, dtype=torch.int32)
        weight = keep("weight", T, k, dtype=torch.float32)
        moe.moe_forward_mxfp4(p, st["x"], st["gate"], st["bias"], st["w1"], st["s1"], st["w2"], st["s2"], y,
                              info=dict(topk_idx=idx, topk_w=weight), ws=ws)
        return dict(y=y, topk_idx=idx, topk_w=weight)
    y = keep("y", T * k, d, dtype=torch.bfloat16)
    if c["kind"] == "down":
        moe.moe_expert_down_mxfp4(p, st["a"], st["sa"], st["offsets"], st["w2"], st["s2"], y, ws=ws)
        return dict(y=y)
    hq = keep("hq", T * k, F // 2, dtype=torch.uint8)
    hs = keep("hs", T * k, F // BLOCK, dtype=torch.uint8)
    moe.moe_expert_up_mxfp4(p, st["a"], st["sa"], st["src"], st["offsets"], st["w1"], st["s1"], hq, hs, ws=ws)
    moe.moe_expert_down_mxfp4(p, hq, hs, st["offsets"], st["w2"], st["s2"], y, ws=ws)
    return dict(y=y)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the least work
def work(case):
    c = case
    if c["kind"] == "quantise":
        n, b = c["rows"] * c["K"], 2 if c["src"] == "bf16" else 4
        return dict(bytes=n * (b + 2) + 2 * (n // 2 + n // BLOCK), flops=3 * n)
    if c["kind"] == "orthogonalise":
        m, n = min(c["rows"], c["cols"]), max(c["rows"], c["cols"])
        b = (2 if c["src"] == "bf16" else 4) + 2 + (0 if c["momentum"] == "none" else 8)
        # x x^T and its square are symmetric: half of each
        return dict(bytes=c["count"] * m * n * b, flops=c["count"] * STEPS * (3 * m * m * n + m * m * m))
    T, d, E, k, F = c["T"], c["d"], c["E"], c["k"], c["F"]
    n1 = 2 * F if c["act"] == "swiglu" else F
    rows = T * k
    if c["kind"] == "layer" and c["cf"] > 0:
        rows = min(rows, E * math.ceil(c["cf"] * rows / E))
    busy = min(E, rows)  # experts that hold rows
    packed = 0.5 + 1.0 / BLOCK  # bytes of a value with its share of a scale
    up, down = 2 * rows * d * n1, 2 * rows * F * d
    if c["kind"] == "down":
        return dict(bytes=busy * d * F * packed + rows * (F * packed + 2 * d), flops=down)
    weights = busy * (n1 * d + d * F) * packed
    if c["kind"] == "experts":
        return dict(bytes=weights + T * d * packed + rows * 2 * d, flops=up + down)
    return dict(bytes=weights + 4 * T * d, flops=up + down + 2 * T * E * d)


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_rounded(v):
    """The values that the codes and scales of v [..., K] (64 bits) stand for, and the scales."""
    b = v.reshape(*v.shape[:-1], -1, BLOCK)
    top = b.abs().amax(dim=-1, keepdim=True)
    e = torch.where(top > 0, torch.ceil(torch.log2(top.clamp(min=1e-300) / 6)), torch.zeros_like(top)).clamp(min=-127)
    e = e + (top > 6 * torch.exp2(e)).double() - ((top > 0) & (top <= 6 * torch.exp2(e - 1)) & (e > -127)).double()
    s = torch.exp2(e)
    w = b / s
    # spacing of the codes around w: half of its power of two, 0.5 below 1
    step = torch.exp2(torch.floor(torch.log2(w.abs().clamp(min=1.0))) - 1)
    return (torch.round(w / step) * step * s).reshape(v.shape), s[..., 0]


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_values(codes, scales):
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float64, device=codes.device)
    v = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device=codes.device)
    v[..., 0::2] = table[(codes % 16).long()]
    v[..., 1::2] = table[(codes // 16).long()]
    return v * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, dim=-1)


def _exact_expert(a, w1, s1, w2, s2, act, F):
    u = a @ _exact_values(w1, s1).t()
    h = u.clamp(min=0) if act == "relu" else u[:, :F] * torch.sigmoid(u[:, :F]) * u[:, F:]
    return _exact_rounded(h)[0] @ _exact_values(w2, s2).t()


def _exact_orthogonal(u):
    """The Newton-Schulz iterate of one matrix, as a sum over its columns or rows, whichever are fewer."""
    norm = torch.linalg.matrix_norm(u)
    x = u / norm if norm > 0 else u
    wide = u.shape[0] <= u.shape[1]
    a, b, q = COEF
    eye = torch.eye(min(u.shape), dtype=torch.float64, device=u.device)
    for _ in range(STEPS):
        s = x @ x.t() if wide else x.t() @ x
        p = a * eye + s @ (b * eye + q * s)
        x = p @ x if wide else x @ p
    return x


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    if c["kind"] == "quantise":
        part = 4096  # rows at a time
        got = [_exact_rounded(st["src"][r : r + part].double()) for r in range(0, c["rows"], part)]
        return dict(values=torch.cat([v for v, _ in got]), scales=torch.cat([s for _, s in got]))
    if c["kind"] == "orthogonalise":
        out = torch.empty(c["count"], c["rows"], c["cols"], dtype=torch.float64, device="cuda")
        mom = None if st["mom"] is None else torch.empty_like(out)
        for i in range(c["count"]):
            u = st["grad"][i].double()
            if mom is not None:
                mom[i] = BETA * st["mom"][i].double() + u
                u = u + BETA * mom[i] if c["momentum"] == "nesterov" else mom[i]
            out[i] = _exact_orthogonal(u)
        return dict(out=out) if mom is None else dict(out=out, momentum=mom)
    T, d, E, k, F = c["T"], c["d"], c["E"], c["k"], c["F"]
    if c["kind"] == "layer":
        z = (st["x"].double() @ st["gate"].double().t() + st["bias"].double()).float().double()
        idx = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
        if c["normalize"]:
            z = (z - z.mean(dim=1, keepdim=True)) / z.std(dim=1, keepdim=True, unbiased=False)
        weight = torch.softmax(z, dim=1).gather(1, idx)
        a = _exact_rounded(st["x"].double())[0]
        limit = math.ceil(c["cf"] * T * k / E) if c["cf"] > 0 else T
        y = torch.zeros(T, d, dtype=torch.float64, device="cuda")
        for e in range(E):
            token, j = torch.nonzero(idx == e, as_tuple=True)
            token, j = token[:limit], j[:limit]
            if token.numel():
                y[token] += weight[token, j][:, None] * _exact_expert(a[token], st["w1"][e], st["s1"][e], st["w2"][e], st["s2"][e], c["act"], F)
        return dict(y=y, topk_idx=None, topk_w=weight)
    o = st["offsets"].tolist()
    a = _exact_values(st["a"], st["sa"])
    y = torch.empty(T * k, d, dtype=torch.float64, device="cuda")
    for e in range(E):
        lo, hi = o[e], o[e + 1]
        if lo == hi:
            continue
        if c["kind"] == "down":
            y[lo:hi] = a[lo:hi] @ _exact_values(st["w2"][e], st["s2"][e]).t()
        else:
            y[lo:hi] = _exact_expert(a[st["src"][lo:hi].long()], st["w1"][e], st["s1"][e], st["w2"][e], st["s2"][e], c["act"], F)
    return dict(y=y)
