"""Workloads of the fused ConvRot operators: linears with activation and residual, gated feed-forward
blocks, and their input gradients through frozen INT8 weights.

A case names an operator and its sizes.  Dimensions: m tokens, k input channels, n output channels
(linears), f hidden channels (feed-forward blocks).  Every operator runs either through the library
(``own``) or as plain torch operations in 32 bits that state the definition:

  z = (qx . wq^T) sx sw + bias,  qx, sx the INT8 codes and scales of the rotated tokens
  linear_act            y = act(z) + residual
  ffn_gated             h = bf16(act(gate) * up),  y = linear(h) + residual
  linear_act_backward   dz = dy act'(pre),  dx = ((dz sw) wq) R,  dbias = sum of dz over tokens
  ffn_gated_backward    the same through down, the product and gate|up;  dx + dy for the residual path
"""
import math

import torch

own = False

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a handful of tokens through a small fp32 linear: nothing but latency
        dict(name="act_tiny", op="linear_act", m=4, k=512, n=256, act="relu", bias=True, residual=False, x="f32"),
        # down projection of a decoder layer for 12 tokens, residual stream added: weight streaming
        dict(name="act_decode_residual", op="linear_act", m=12, k=25600, n=5120, act="none", bias=False, residual=True,
             x="bf16"),
        # a ragged batch through a width that 256 does not divide, odd output width
        dict(name="act_ragged", op="linear_act", m=333, k=2688, n=1001, act="silu", bias=True, residual=True, x="bf16"),
        # first linear of an ungated MLP over a prompt
        dict(name="act_prefill_gelu", op="linear_act", m=4096, k=5376, n=16128, act="gelu_tanh", bias=True,
             residual=False, x="bf16"),
        # one token through a decoder layer's feed-forward block
        dict(name="ffn_token", op="ffn_gated", m=1, k=5120, f=25600, act="silu", bias=False, residual=True, save=False,
             x="bf16"),
        # the conditioning pass of a text encoder: 12 tokens
        dict(name="ffn_decode", op="ffn_gated", m=12, k=5120, f=25600, act="silu", bias=False, residual=True,
             save=False, x="bf16"),
        # training forward of a narrower block: the pre-activations are kept for the backward pass
        dict(name="ffn_ragged_save", op="ffn_gated", m=300, k=2688, f=5376, act="gelu_tanh", bias=True, residual=False,
             save=True, x="bf16"),
        # a prompt through a decoder layer's feed-forward block
        dict(name="ffn_prompt", op="ffn_gated", m=2048, k=5120, f=25600, act="silu", bias=False, residual=True,
             save=False, x="bf16"),
        # gradient of a few tokens (prompt tuning) through one projection
        dict(name="act_bwd_decode", op="linear_act_backward", m=12, k=5120, n=8192, act="none", bias=False,
             add=True),
        # gradient through the first linear of an ungated MLP, with the bias gradient
        dict(name="act_bwd_prefill", op="linear_act_backward", m=4096, k=5376, n=16128, act="gelu_tanh", bias=True,
             add=False),
        # an odd-sized batch through the narrower block
        dict(name="ffn_bwd_ragged", op="ffn_gated_backward", m=301, k=2688, f=5376, act="gelu", add=False),
        # a prompt's gradient through a decoder layer's block, the residual path added
        dict(name="ffn_bwd_prompt", op="ffn_gated_backward", m=2048, k=5120, f=25600, act="silu", add=True),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    most = max(work(c)["flops"] for c in listed())
    while True:
        op = rng.choice(["linear_act", "ffn_gated", "linear_act_backward", "ffn_gated_backward"])
        case = dict(op=op, m=_log_int(rng, 1, 4096), k=64 * _log_int(rng, 4, 400 if op == "linear_act" else 84))
        if op.startswith("ffn"):
            case["f"] = 64 * _log_int(rng, 4, 400)
        else:
            case["n"] = _log_int(rng, 200, 16384)
        if op.endswith("backward"):
            case["add"] = rng.random() < 0.5
        else:
            case["residual"] = rng.random() < 0.5
            case["x"] = rng.choice(["bf16", "bf16", "f32"])
        if op != "ffn_gated_backward":
            case["bias"] = rng.random() < 0.5
        if op == "ffn_gated":
            case["save"] = rng.random() < 0.3
        case["act"] = rng.choice(ACTS if op.startswith("linear") else ACTS[1:])
        if work(case)["flops"] <= most:
            return case


def work(case):
    """Bytes read and written once, and operations, of one pass."""
    m, k, op = case["m"], case["k"], case["op"]
    if op.startswith("linear"):
        n = case["n"]
        flops, weights = 2 * m * n * k, n * k + 4 * n + 4 * n * case["bias"]
        if op == "linear_act":
            rows = m * k * (4 if case["x"] == "f32" else 2) + 2 * m * n * (1 + case["residual"])
        else:
            rows = 2 * m * n * (1 + (case["act"] != "none")) + 2 * m * k * (1 + case["add"])
    else:
        f = case["f"]
        flops, weights = 6 * m * f * k, 3 * f * k + 4 * (2 * f + k)
        if op == "ffn_gated":
            rows = m * k * (4 if case["x"] == "f32" else 2) + 2 * m * k * (1 + case["residual"])
            rows += 4 * m * f * case["save"] + 4 * (2 * f + k) * case["bias"]
        else:
            rows = 2 * m * k * 2 + 4 * m * f
    return {"bytes": rows + weights, "flops": flops}


# ---------------------------------------------------------------------------------------------
# inputs


def _group(k):
    """Rotation group of a width: the largest power of two up to 256 that divides it."""
    return math.gcd(k, 256)


def _weight(gen, n, k):
    """Row-wise INT8 codes and fp32 scales of N(0, 0.02) rows (a rotated Gaussian row is one too)."""
    w = torch.randn(n, k, generator=gen, device="cuda") * 0.02
    scale = w.abs().amax(1) / 127.0
    return torch.round(w / scale[:, None]).to(torch.int8), scale


def _tokens(gen, m, k, dtype):
    """Heavy-tailed activations (Student t with 4 degrees of freedom), 1% outlier channels x30."""
    x = torch.randn(m, k, generator=gen, device="cuda")
    v = torch.zeros(m, k, device="cuda")
    for _ in range(4):
        v += torch.randn(m, k, generator=gen, device="cuda").square_()
    x /= torch.sqrt(v * 0.25)
    channels = torch.randperm(k, generator=gen, device="cuda")[: max(1, k // 100)]
    x[:, channels] *= 30.0
    return x.to(dtype)


def _normal(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def _gradient(gen, m, n):
    """A loss gradient: Gaussian per channel, its size log-normal over the tokens."""
    size = torch.exp(torch.randn(m, 1, generator=gen, device="cuda")) * 1e-3
    return (torch.randn(m, n, generator=gen, device="cuda") * size).to(torch.bfloat16)


def _hadamard(g):
    i = torch.arange(g, device="cuda")
    both = i[:, None] & i[None, :]
    ones = sum((both >> b) & 1 for b in range(8))
    return (1 - 2 * (ones & 1)).float() / math.sqrt(g)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    m, k, op = case["m"], case["k"], case["op"]
    s = {"op": op, "act": case["act"], "group": _group(k), "hadamard": _hadamard(_group(k))}
    if op.startswith("linear"):
        n = case["n"]
        s["w"] = _weight(gen, n, k)
        if op == "linear_act":
            s["x"] = _tokens(gen, m, k, DTYPES[case["x"]])
            s["bias"] = _normal(gen, n, dtype=torch.float32) if case["bias"] else None
            s["residual"] = _normal(gen, m, n, std=4.0) if case["residual"] else None
        else:
            s["dy"] = _gradient(gen, m, n)
            s["pre"] = _normal(gen, m, n, std=1.5) if case["act"] != "none" else None
            s["bias_grad"] = case["bias"]
            s["add"] = _gradient(gen, m, k) if case["add"] else None
        return s
    f = case["f"]
    s["group_h"], s["hadamard_h"] = _group(f), _hadamard(_group(f))
    s["gate"], s["up"], s["down"] = _weight(gen, f, k), _weight(gen, f, k), _weight(gen, k, f)
    if op == "ffn_gated":
        s["x"] = _tokens(gen, m, k, DTYPES[case["x"]])
        s["residual"] = _normal(gen, m, k, std=4.0) if case["residual"] else None
        for name, width in (("bias_gate", f), ("bias_up", f), ("bias_down", k)):
            s[name] = _normal(gen, width, dtype=torch.float32) if case["bias"] else None
        s["save"] = case["save"]
    else:
        s["dy"] = _gradient(gen, m, k)
        s["pre"] = _normal(gen, 2, m, f, std=1.5)
        s["add"] = s["dy"] if case["add"] else None
    return s


# ---------------------------------------------------------------------------------------------
# one pass


def run(s):
    return {"linear_act": _linear_act, "ffn_gated": _ffn_gated, "linear_act_backward": _linear_act_backward,
            "ffn_gated_backward": _ffn_gated_backward}[s["op"]](s)


def _linear_act(s):
    if own:
        from int4_quantized_linear_amd import convrot
        return convrot.linear_act(s["x"], *s["w"], bias=s["bias"], act=s["act"], residual=s["residual"],
                                  group=s["group"])
    y = _act(_linear(s["x"], s["w"], s["bias"], s["hadamard"]), s["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(torch.bfloat16)


def _ffn_gated(s):
    if own:
        from int4_quantized_linear_amd import convrot
        return convrot.ffn_gated(s["x"], *s["gate"], *s["up"], *s["down"], bias_gate=s["bias_gate"],
                                 bias_up=s["bias_up"], bias_down=s["bias_down"], act=s["act"],
                                 residual=s["residual"], group=s["group"], group_h=s["group_h"], save_pre=s["save"])
    g = _linear(s["x"], s["gate"], s["bias_gate"], s["hadamard"])
    u = _linear(s["x"], s["up"], s["bias_up"], s["hadamard"])
    h = (_act(g, s["act"]) * u).to(torch.bfloat16)
    y = _linear(h, s["down"], s["bias_down"], s["hadamard_h"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    y = y.to(torch.bfloat16)
    return (y, torch.stack([g, u]).to(torch.bfloat16)) if s["save"] else y


def _linear_act_backward(s):
    if own:
        from int4_quantized_linear_amd import convrot
        return convrot.linear_act_backward(s["dy"], *s["w"], pre=s["pre"], act=s["act"], group=s["group"],
                                           bias_grad=s["bias_grad"], dx_add=s["add"])
    dz = s["dy"].float()
    if s["act"] != "none":
        dz = dz * _act_derivative(s["pre"].float(), s["act"])
    dx = _rotate((dz * s["w"][1]) @ s["w"][0].float(), s["hadamard"])
    if s["add"] is not None:
        dx = dx + s["add"].float()
    return dx.to(torch.bfloat16), (dz.sum(0) if s["bias_grad"] else None)


def _ffn_gated_backward(s):
    if own:
        from int4_quantized_linear_amd import convrot
        return convrot.ffn_gated_backward(s["dy"], s["pre"], *s["gate"], *s["up"], *s["down"], act=s["act"],
                                          group=s["group"], group_h=s["group_h"], dx_add=s["add"])
    dh = _rotate((s["dy"].float() * s["down"][1]) @ s["down"][0].float(), s["hadamard_h"])
    dh = dh.to(torch.bfloat16).float()
    g, u = s["pre"][0].float(), s["pre"][1].float()
    dg, du = dh * u * _act_derivative(g, s["act"]), dh * _act(g, s["act"])
    dx = (dg * s["gate"][1]) @ s["gate"][0].float() + (du * s["up"][1]) @ s["up"][0].float()
    dx = _rotate(dx, s["hadamard"])
    if s["add"] is not None:
        dx = dx + s["add"].float()
    return dx.to(torch.bfloat16)


# the definition in 32 bits


def _rotate(x, hadamard):
    g = hadamard.shape[0]
    return (x.float().reshape(-1, g) @ hadamard).reshape(x.shape)


def _linear(x, weight, bias, hadamard):
    """Rotated tokens to INT8 codes with one scale each, the product of the codes, both scales, the bias."""
    wq, sw = weight
    v = _rotate(x, hadamard)
    sx = v.abs().amax(1, keepdim=True) / 127.0
    q = torch.round(torch.where(sx > 0, v / sx, torch.zeros_like(v)))
    z = (q @ wq.float().t()) * (sx * sw)
    return z if bias is None else z + bias


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(z * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_derivative(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        return 0.5 * torch.special.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits


class _Activations64:
    """Activation and derivative in 64 bits, from the sigmoid and the normal distribution."""

    @staticmethod
    def of(z, act):
        """(act(z), act'(z))"""
        if act == "none":
            return z, torch.ones_like(z)
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
        v = v.reshape(rows, -1, 2, half)
        v = torch.stack([v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]], 2).reshape(rows, k)
        half *= 2
    return v / math.sqrt(g)


def _product64(x, weight, bias, g):
    v = _transform64(x.double(), g)
    sx = v.abs().max(1, keepdim=True).values / 127
    codes = torch.round(v / torch.where(sx == 0, torch.ones_like(sx), sx))
    z = torch.mm(codes, weight[0].double().t()) * sx * weight[1].double()
    return z + bias.double() if bias is not None else z


def _gradient64(dz, weight):
    return torch.mm(dz * weight[1].double(), weight[0].double())


def exact(case, seed):
    s = prepare(case, seed)
    act, g = s["act"], s["group"]
    if s["op"] == "linear_act":
        y, _ = _Activations64.of(_product64(s["x"], s["w"], s["bias"], g), act)
        return y if s["residual"] is None else y + s["residual"].double()
    if s["op"] == "linear_act_backward":
        dz = s["dy"].double()
        if s["pre"] is not None:
            dz = dz * _Activations64.of(s["pre"].double(), act)[1]
        dx = _transform64(_gradient64(dz, s["w"]), g)
        if s["add"] is not None:
            dx = dx + s["add"].double()
        return dx, (dz.sum(0) if s["bias_grad"] else None)
    if s["op"] == "ffn_gated":
        gate = _product64(s["x"], s["gate"], s["bias_gate"], g)
        up = _product64(s["x"], s["up"], s["bias_up"], g)
        hidden = (_Activations64.of(gate, act)[0] * up).to(torch.bfloat16)   # the block's hidden type
        y = _product64(hidden, s["down"], s["bias_down"], s["group_h"])
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return (y, torch.stack([gate, up])) if s["save"] else y
    dh = _transform64(_gradient64(s["dy"].double(), s["down"]), s["group_h"])
    gate, up = s["pre"].double()
    value, slope = _Activations64.of(gate, act)
    dx = _transform64(_gradient64(dh * up * slope, s["gate"]) + _gradient64(dh * value, s["up"]), g)
    return dx if s["add"] is None else dx + s["add"].double()
