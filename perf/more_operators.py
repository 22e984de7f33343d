"""Workloads of the mixture-of-experts operators on INT8 ConvRot weights: the router, products of grouped
rows with their group's weight, the whole gated expert layer, and their gradients through frozen weights.

A case names an operator and its sizes.  Dimensions: m tokens, e experts (or groups), top experts per token,
k input channels, f hidden channels of an expert, n output channels and s rows of the grouped products.  Every operator
runs either through the library (``own``) or as plain torch operations that state the definition:

  moe_route       experts = the top scores' indices (ties to the lowest), weights = their scores
  linear_grouped  y = bf16((qx . wq^T) sx sw) with the weight of the row's group
  moe_ffn_gated   h = bf16(act(gate) * up) per slot,  y = bf16(sum over a token's slots of weight * linear(h) + residual)
  *_backward      input gradients with the token quantizer as the identity, and the slots' weights' gradients

In products of 32-bit floats the plain forms gather each used expert's rows in a padded batch.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("relu", "silu", "gelu", "gelu_tanh")


def listed():
    return [
        # the router of one decoded token: latency
        dict(name="route_token", op="route", m=1, e=64, top=8, score="softmax", normalize=True, scale=1.0, bias=False,
             x="f32"),
        # a long prompt's router with sigmoid scores and a load-balancing bias on the choice
        dict(name="route_prompt", op="route", m=8192, e=256, top=8, score="sigmoid", normalize=True, scale=2.5, bias=True,
             x="f32"),
        # its gradient in training, weights not normalised, logits of a bf16 linear
        dict(name="route_bwd", op="route_backward", m=8192, e=128, top=6, score="softmax", normalize=False, scale=1.0,
             bias=False, x="bf16"),
        # a few rows that arrived for each of a card's experts
        dict(name="grouped_decode", op="grouped", s=48, e=32, k=5120, n=2048, x="bf16"),
        # projections with a weight per kind of token, an odd width, fp32 rows
        dict(name="grouped_ragged", op="grouped", s=2500, e=6, k=2688, n=1001, x="f32"),
        # a prompt's rows sorted by expert
        dict(name="grouped_prompt", op="grouped", s=8192, e=16, k=5376, n=5376, x="bf16"),
        # the gradient of such rows through their weights
        dict(name="grouped_bwd", op="grouped_backward", s=4097, e=8, k=2688, n=5376, add=True),
        # one decoded token through an expert layer: weight streaming and latency
        dict(name="moe_token", op="moe", m=1, e=64, top=8, k=2048, f=1024, act="silu", residual=True, save=False,
             drop=False, x="bf16"),
        # 12 tokens (a text encoder's conditioning pass, or a decode batch) through many small experts
        dict(name="moe_decode", op="moe", m=12, e=128, top=8, k=5120, f=1280, act="silu", residual=True, save=False,
             drop=False, x="bf16"),
        # training forward of a short, odd batch through few experts: what the backward pass reads is kept
        dict(name="moe_ragged_save", op="moe", m=301, e=16, top=3, k=2688, f=1344, act="gelu_tanh", residual=False,
             save=True, drop=False, x="f32"),
        # a prompt through an expert layer
        dict(name="moe_prompt", op="moe", m=4096, e=64, top=6, k=2048, f=1408, act="silu", residual=True, save=False,
             drop=False, x="bf16"),
        # a prompt's gradient through an expert layer
        dict(name="moe_bwd_prompt", op="moe_backward", m=2048, e=32, top=4, k=2048, f=1408, act="silu", add=True,
             drop=False),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


MAX_WEIGHTS = 2_600_000_000         # codes of a case's weights


def draw(rng):
    most = max(work(c)["flops"] for c in listed())
    while True:
        op = rng.choice(["route", "route_backward", "grouped", "grouped_backward", "moe", "moe", "moe_backward"])
        case = dict(op=op)
        if op.startswith("route"):
            e = _log_int(rng, 4, 512)
            score, normalize = rng.choice(["softmax", "sigmoid"]), rng.random() < 0.6
            # (the one weight of a normalised choice is constant: it has no gradient)
            least = 2 if op == "route_backward" and normalize else 1
            case.update(m=_log_int(rng, 1, 16384), e=e, top=min(e, rng.randint(least, 12)), score=score, normalize=normalize,
                        scale=rng.choice([1.0, 2.5]), bias=rng.random() < 0.4, x=rng.choice(["f32", "bf16"]))
            return case
        if op.startswith("grouped"):
            case.update(s=_log_int(rng, 1, 16384), e=_log_int(rng, 2, 64), k=64 * _log_int(rng, 4, 84),
                        n=_log_int(rng, 200, 8192))
            weights = case["e"] * case["n"] * case["k"]
        else:
            e = _log_int(rng, 4, 128)
            case.update(m=_log_int(rng, 1, 4096), e=e, top=min(e, rng.randint(1, 8)), k=64 * _log_int(rng, 8, 84),
                        f=64 * _log_int(rng, 4, 64), act=rng.choice(ACTS), drop=rng.random() < 0.25)
            weights = 3 * e * case["f"] * case["k"]
        if op == "moe":
            case.update(residual=rng.random() < 0.5, save=not case["drop"] and rng.random() < 0.3)
        if op in ("grouped", "moe"):
            case["x"] = rng.choice(["bf16", "bf16", "f32"])
        if op.endswith("backward"):
            case["add"] = rng.random() < 0.5
        if weights <= MAX_WEIGHTS and work(case)["flops"] <= most:
            return case


def work(case):
    """Bytes read and written once, and operations, of one pass.  A weight counts where a row is expected to use it."""
    op, e = case["op"], case["e"]
    if op.startswith("route"):
        m, top, es = case["m"], case["top"], 4 if case["x"] == "f32" else 2
        back = op == "route_backward"
        return {"bytes": m * e * es * (1 + back) + 8 * m * top + 4 * e * case["bias"] * (not back), "flops": 4 * m * e}
    if op.startswith("grouped"):
        s, k, n = case["s"], case["k"], case["n"]
        weights = min(e, s) * n * (k + 4)
        if op == "grouped":
            rows = s * k * (4 if case["x"] == "f32" else 2) + 2 * s * n
        else:
            rows = 2 * s * n + 2 * s * k * (1 + case["add"])
        return {"bytes": weights + rows, "flops": 2 * s * n * k}
    m, top, k, f = case["m"], case["top"], case["k"], case["f"]
    slots = m * top * (0.5 if case["drop"] else 1.0)
    used = e * (1.0 - (1.0 - slots / (m * e)) ** m)
    weights = used * (3 * f * k + 4 * (2 * f + k))
    if op == "moe":
        rows = m * k * (4 if case["x"] == "f32" else 2) + 2 * m * k * (1 + case["residual"]) + 8 * m * top
        rows += (4 * slots * f + 2 * slots * k) * case["save"]
    else:
        rows = 2 * m * k * (2 + case["add"]) + 2 * slots * k + 4 * slots * f + 12 * m * top
    return {"bytes": weights + rows, "flops": 6 * slots * f * k}


# ---------------------------------------------------------------------------------------------
# inputs


def _rotation(k):
    """Rotation group of a width: the largest power of two up to 256 that divides it."""
    return math.gcd(k, 256)


def _weights(gen, e, n, k):
    """Row-wise INT8 codes [e, n, k] and fp32 scales [e, n] of N(0, 0.02) rows (a rotated Gaussian row is one too)."""
    codes = torch.empty(e, n, k, dtype=torch.int8, device="cuda")
    scales = torch.empty(e, n, device="cuda")
    for i in range(e):
        w = torch.randn(n, k, generator=gen, device="cuda") * 0.02
        scales[i] = w.abs().amax(1) / 127.0
        codes[i] = torch.round(w / scales[i][:, None]).to(torch.int8)
    return codes, scales


def _tokens(gen, m, k, dtype):
    """Heavy-tailed activations (Student t with 4 degrees of freedom), 1% outlier channels x30, behind the norm that
    stands before such a layer: every token has unit rms."""
    x = torch.randn(m, k, generator=gen, device="cuda")
    v = torch.zeros(m, k, device="cuda")
    for _ in range(4):
        v += torch.randn(m, k, generator=gen, device="cuda").square_()
    x /= torch.sqrt(v * 0.25)
    channels = torch.randperm(k, generator=gen, device="cuda")[: max(1, k // 100)]
    x[:, channels] *= 30.0
    return (x / x.square().mean(1, keepdim=True).sqrt()).to(dtype)


def _normal(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def _gradient(gen, m, n):
    """A loss gradient: Gaussian per channel, its size log-normal over the tokens."""
    size = torch.exp(torch.randn(m, 1, generator=gen, device="cuda")) * 1e-3
    return (torch.randn(m, n, generator=gen, device="cuda") * size).to(torch.bfloat16)


def _logits(gen, m, e, dtype=torch.float32):
    """Router outputs: some experts are liked by most tokens."""
    liked = torch.randn(e, generator=gen, device="cuda") * 0.7
    return (torch.randn(m, e, generator=gen, device="cuda") * 1.5 + liked).to(dtype)


def _hadamard(g):
    i = torch.arange(g, device="cuda")
    both = i[:, None] & i[None, :]
    ones = sum((both >> b) & 1 for b in range(8))
    return (1 - 2 * (ones & 1)).float() / math.sqrt(g)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, e = case["op"], case["e"]
    s = dict(case)
    if op.startswith("route"):
        s["logits"] = _logits(gen, case["m"], e, DTYPES[case["x"]])
        s["balance"] = _normal(gen, e, std=0.05, dtype=torch.float32) if case["bias"] else None
        if op == "route_backward":
            s["experts"], _ = _choose(s["logits"], s["balance"], case)
            s["grad"] = _normal(gen, case["m"], case["top"], std=1e-2, dtype=torch.float32)
        return s
    k = case["k"]
    s["group"], s["hadamard"] = _rotation(k), _hadamard(_rotation(k))
    if op.startswith("grouped"):
        rows, n = case["s"], case["n"]
        share = torch.exp(torch.randn(e, generator=gen, device="cuda") * 0.7)
        if e > 2:
            share[e // 2] = 0.0                                   # a group without rows
        of = torch.multinomial(share, rows, replacement=True, generator=gen)
        counts = torch.bincount(of, minlength=e)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["w"] = _weights(gen, e, n, k)
        if op == "grouped":
            s["x"] = _tokens(gen, rows, k, DTYPES[case["x"]])
        else:
            s["dy"] = _gradient(gen, rows, n)
            s["dx_add"] = _gradient(gen, rows, k) if case["add"] else None
        return s
    m, top, f = case["m"], case["top"], case["f"]
    s["group_h"], s["hadamard_h"] = _rotation(f), _hadamard(_rotation(f))
    s["gate"], s["up"], s["down"] = _weights(gen, e, f, k), _weights(gen, e, f, k), _weights(gen, e, k, f)
    logits = _logits(gen, m, e)
    value, chosen = torch.topk(logits, top, 1)
    s["weights"], s["experts"] = torch.softmax(value, 1), chosen.to(torch.int32)
    if case["drop"]:
        # half of the slots belong to another card's experts
        s["experts"][torch.rand(m, top, generator=gen, device="cuda") < 0.5] = -1
    if op == "moe":
        s["x"] = _tokens(gen, m, k, DTYPES[case["x"]])
        s["residual"] = _normal(gen, m, k, std=4.0) if case["residual"] else None
    else:
        s["dy"] = _gradient(gen, m, k)
        s["pre"] = _normal(gen, 2, m, top, f, std=1.5)
        s["d"] = _normal(gen, m, top, k, std=0.5)
        s["dx_add"] = s["dy"] if case["add"] else None
    return s


# ---------------------------------------------------------------------------------------------
# one pass


def run(s):
    return {"route": _route, "route_backward": _route_backward, "grouped": _grouped, "grouped_backward": _grouped_backward,
            "moe": _moe, "moe_backward": _moe_backward}[s["op"]](s)


def _route(s):
    if own:
        from int4_quantized_linear_amd import convrot
        return convrot.moe_route(s["logits"], s["top"], bias=s["balance"], score=s["score"], normalize=s["normalize"],
                                 scale=s["scale"])
    return _choose(s["logits"], s["balance"], s)


def _route_backward(s):
    if own:
        from int4_quantized_linear_amd import convrot
        return convrot.moe_route_backward(s["grad"], s["logits"], s["experts"], score=s["score"], normalize=s["normalize"],
                                          scale=s["scale"])
    logits, chosen, grad = s["logits"].double(), s["experts"].long(), s["grad"].double() * s["scale"]
    score = torch.exp(logits - logits.amax(1, keepdim=True)) if s["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-logits))
    if s["score"] == "softmax":
        score = score / score.sum(1, keepdim=True)
    value = score.gather(1, chosen)
    inner = grad
    if s["normalize"]:
        value = value / value.sum(1, keepdim=True)
        inner = grad - (grad * value).sum(1, keepdim=True)
    if s["score"] == "sigmoid":
        inner = inner * (1.0 - score.gather(1, chosen))
    back = torch.zeros_like(logits).scatter_add(1, chosen, value * inner)
    if s["score"] == "softmax" and not s["normalize"]:
        back = back - score * (grad * value).sum(1, keepdim=True)
    return back.to(s["logits"].dtype)


def _grouped(s):
    if own:
        from int4_quantized_linear_amd import convrot
        return convrot.linear_grouped(s["x"], *s["w"], s["offsets"], group=s["group"])
    rows, counts = _rows_of(s["offsets"], s["s"])
    q, sx = _quantize(s["x"], s["hadamard"])
    return (_products(q, rows, counts, s["w"][0], True) * sx * s["w"][1][rows]).to(torch.bfloat16)


def _grouped_backward(s):
    if own:
        from int4_quantized_linear_amd import convrot
        return convrot.linear_grouped_backward(s["dy"], *s["w"], s["offsets"], group=s["group"], dx_add=s["dx_add"])
    rows, counts = _rows_of(s["offsets"], s["s"])
    dx = _rotate(_products(s["dy"].float() * s["w"][1][rows], rows, counts, s["w"][0], False), s["hadamard"])
    if s["dx_add"] is not None:
        dx = dx + s["dx_add"].float()
    return dx.to(torch.bfloat16)


def _moe(s):
    if own:
        from int4_quantized_linear_amd import convrot
        return convrot.moe_ffn_gated(s["x"], s["experts"], s["weights"], *s["gate"], *s["up"], *s["down"], act=s["act"],
                                     residual=s["residual"], group=s["group"], group_h=s["group_h"], save=s["save"])
    m, top, k, f = s["m"], s["top"], s["k"], s["f"]
    slots, of, counts = _slots_of(s["experts"], s["e"])
    q, sx = _quantize(s["x"], s["hadamard"])
    q, sx = q[slots // top], sx[slots // top]
    g = _products(q, of, counts, s["gate"][0], True) * sx * s["gate"][1][of]
    u = _products(q, of, counts, s["up"][0], True) * sx * s["up"][1][of]
    h, sh = _quantize((_act(g, s["act"]) * u).to(torch.bfloat16), s["hadamard_h"])
    d = _products(h, of, counts, s["down"][0], True) * sh * s["down"][1][of]
    every = d.new_zeros(m * top, k)
    every[slots] = d
    y = (every.view(m, top, k) * s["weights"][:, :, None]).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    y = y.to(torch.bfloat16)
    if not s["save"]:
        return y
    pre = g.new_zeros(2, m * top, f)
    pre[0, slots], pre[1, slots] = g, u
    return y, pre.view(2, m, top, f).to(torch.bfloat16), every.view(m, top, k).to(torch.bfloat16)


def _moe_backward(s):
    if own:
        from int4_quantized_linear_amd import convrot
        return convrot.moe_ffn_gated_backward(s["dy"], s["pre"], s["d"], s["experts"], s["weights"], *s["gate"], *s["up"],
                                              *s["down"], act=s["act"], group=s["group"], group_h=s["group_h"],
                                              dx_add=s["dx_add"])
    m, top, k, f = s["m"], s["top"], s["k"], s["f"]
    slots, of, counts = _slots_of(s["experts"], s["e"])
    dy = s["dy"].float()
    chosen = (s["experts"] >= 0).float()
    dweights = (dy[:, None, :] * s["d"].float()).sum(2) * chosen
    dd = dy[slots // top] * s["weights"].view(-1, 1)[slots]
    dh = _rotate(_products(dd * s["down"][1][of], of, counts, s["down"][0], False), s["hadamard_h"])
    dh = dh.to(torch.bfloat16).float()
    pre = s["pre"].view(2, m * top, f)
    g, u = pre[0, slots].float(), pre[1, slots].float()
    dg, du = dh * u * _act_derivative(g, s["act"]), dh * _act(g, s["act"])
    part = _products(dg * s["gate"][1][of], of, counts, s["gate"][0], False)
    part = part + _products(du * s["up"][1][of], of, counts, s["up"][0], False)
    every = part.new_zeros(m * top, k)
    every[slots] = part
    dx = _rotate(every.view(m, top, k).sum(1), s["hadamard"])
    if s["dx_add"] is not None:
        dx = dx + s["dx_add"].float()
    return dx.to(torch.bfloat16), dweights


# the definition in 32 bits


def _choose(logits, balance, case):
    """experts and weights of each token; the keys of the choice in 64 bits, where neighbours may be close."""
    x = logits.double()
    if case["score"] == "softmax":
        score = torch.exp(x - x.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    key = x if balance is None else score + balance.double()
    chosen = torch.sort(key, dim=1, descending=True, stable=True)[1][:, : case["top"]]
    value = score.gather(1, chosen)
    if case["normalize"]:
        value = value / value.sum(1, keepdim=True)
    return chosen.to(torch.int32), (value * case["scale"]).float()


def _rows_of(offsets, rows):
    """Group of each row, and the groups' sizes."""
    counts = (offsets[1:] - offsets[:-1]).long()
    return torch.repeat_interleave(torch.arange(counts.numel(), device="cuda"), counts, output_size=rows), counts


def _slots_of(experts, e):
    """Slots that have an expert, sorted by it; their experts; the experts' sizes."""
    flat = experts.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    order = order[(flat < 0).sum():]
    of = flat[order]
    return order, of, torch.bincount(of, minlength=e)


def _products(a, of, counts, codes, transposed):
    """a[r] . codes[of[r]]^T (transposed), or a[r] . codes[of[r]]; rows sorted by ``of``.  One batched product over the
    used groups, padded to the largest."""
    used = torch.nonzero(counts)[:, 0]
    out = codes.shape[1] if transposed else codes.shape[2]
    if used.numel() == 0:
        return a.new_zeros(0, out)
    size = int(counts.max())
    batch = torch.cumsum((counts > 0).long(), 0)[of] - 1
    place = torch.arange(of.numel(), device="cuda") - (torch.cumsum(counts, 0) - counts)[of]
    padded = a.new_zeros(used.numel(), size, a.shape[1])
    padded[batch, place] = a
    w = codes[used].float()
    return torch.bmm(padded, w.transpose(1, 2) if transposed else w)[batch, place]


def _rotate(x, hadamard):
    g = hadamard.shape[0]
    return (x.float().reshape(-1, g) @ hadamard).reshape(x.shape)


def _quantize(x, hadamard):
    """INT8 codes (as floats) and scales of the rotated rows, in 64 bits: some quotients lie next to a code's border."""
    g = hadamard.shape[0]
    signs = torch.sign(hadamard).double()                         # (the rotation is orthonormal: signs / sqrt(g))
    v = (x.double().reshape(-1, g) @ signs).reshape(x.shape) / math.sqrt(g)
    sx = v.abs().amax(1, keepdim=True) / 127.0
    return torch.round(torch.where(sx > 0, v / sx, torch.zeros_like(v))).float(), sx.float()


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(z * -math.sqrt(0.5))
    return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))


def _act_derivative(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        return 0.5 * torch.special.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits, expert by expert


def _act64(z, act):
    """(act(z), act'(z)) from the sigmoid and the normal distribution."""
    if act == "relu":
        return torch.relu(z), (z > 0).double()
    if act == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        t, dt = z, torch.ones_like(z)
    else:  # gelu_tanh: (1 + tanh(v)) / 2 = sigmoid(2 v)
        a = 2 * math.sqrt(2 / math.pi)
        t, dt = a * z + a * 0.044715 * z ** 3, a + 3 * a * 0.044715 * z ** 2
    p = torch.sigmoid(t)
    return z * p, p + z * p * torch.sigmoid(-t) * dt


def _transform64(v, g):
    """Orthonormal Walsh-Hadamard transform of each g consecutive channels, by halves."""
    rows, k = v.shape
    half = 1
    while half < g:
        v = v.reshape(rows, k // (2 * half), 2, half)
        v = torch.stack([v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]], 2).reshape(rows, k)
        half *= 2
    return v / math.sqrt(g)


def _linear64(x, codes, scale, g):
    v = _transform64(x.double(), g)
    sx = v.abs().amax(1, keepdim=True) / 127
    q = torch.round(v / torch.where(sx == 0, torch.ones_like(sx), sx))
    return torch.mm(q, codes.double().t()) * sx * scale.double()


def _back64(dz, codes, scale):
    return torch.mm(dz * scale.double(), codes.double())


def _route64(s):
    x = s["logits"].double()
    logs = torch.log_softmax(x, 1) if s["score"] == "softmax" else torch.nn.functional.logsigmoid(x)
    if s["op"] == "route":
        key = logs.exp() + s["balance"].double() if s["balance"] is not None else x
        chosen = torch.argsort(key, dim=1, descending=True, stable=True)[:, : s["top"]]
        value = logs.gather(1, chosen)
        value = torch.softmax(value, 1) if s["normalize"] else value.exp()
        return None, value * s["scale"]                          # whole numbers are compared with the plain form's
    chosen, grad = s["experts"].long(), s["grad"].double() * s["scale"]
    with torch.enable_grad():
        x = x.requires_grad_(True)
        logs = torch.log_softmax(x, 1) if s["score"] == "softmax" else torch.nn.functional.logsigmoid(x)
        value = logs.gather(1, chosen)
        value = torch.softmax(value, 1) if s["normalize"] else value.exp()
        (value * grad).sum().backward()
    return x.grad.detach()


def exact(case, seed):
    s = prepare(case, seed)
    op, g = s["op"], s.get("group")
    if op.startswith("route"):
        return _route64(s)
    if op.startswith("grouped"):
        ends = s["offsets"].tolist()
        parts = []
        for i in range(s["e"]):
            lo, hi = ends[i], ends[i + 1]
            codes, scale = s["w"][0][i], s["w"][1][i]
            if op == "grouped":
                parts.append(_linear64(s["x"][lo:hi], codes, scale, g))
            else:
                dx = _transform64(_back64(s["dy"][lo:hi].double(), codes, scale), g)
                parts.append(dx if s["dx_add"] is None else dx + s["dx_add"][lo:hi].double())
        return torch.cat(parts)
    m, top, k, f, gh = s["m"], s["top"], s["k"], s["f"], s["group_h"]
    f64 = dict(dtype=torch.float64, device="cuda")
    total = torch.zeros(m, k, **f64)
    pre, d = torch.zeros(2, m, top, f, **f64), torch.zeros(m, top, k, **f64)
    dw = torch.zeros(m, top, **f64)
    for i in range(s["e"]):
        token, slot = torch.nonzero(s["experts"] == i, as_tuple=True)
        if token.numel() == 0:
            continue
        gate, up, down = ((s[w][0][i], s[w][1][i]) for w in ("gate", "up", "down"))
        share = s["weights"][token, slot].double()[:, None]
        if op == "moe":
            a, b = _linear64(s["x"][token], *gate, g), _linear64(s["x"][token], *up, g)
            hidden = (_act64(a, s["act"])[0] * b).to(torch.bfloat16)      # the layer's hidden type
            out = _linear64(hidden, *down, gh)
            total.index_add_(0, token, out * share)
            if s["save"]:
                pre[0, token, slot], pre[1, token, slot], d[token, slot] = a, b, out
        else:
            dy = s["dy"][token].double()
            dw[token, slot] = (dy * s["d"][token, slot].double()).sum(1)
            dh = _transform64(_back64(dy * share, *down), gh)
            a, b = s["pre"][0, token, slot].double(), s["pre"][1, token, slot].double()
            value, slope = _act64(a, s["act"])
            total.index_add_(0, token, _back64(dh * b * slope, *gate) + _back64(dh * value, *up))
    if op == "moe":
        y = total if s["residual"] is None else total + s["residual"].double()
        return (y, pre, d) if s["save"] else y
    dx = _transform64(total, g)
    return (dx if s["dx_add"] is None else dx + s["dx_add"].double()), dw
