"""Plain 64-bit reference of the fused linears' epilogues and of the input gradients, and the error
bounds the tests hold the kernels to.

Bounds.  u = 2^-24 is half a step of fp32, and bf16 rounding is off by at most 2^-8 of the value
(torch.finfo(torch.bfloat16).eps / 2).
  z: (float)acc, sx * sw, their product with the bias in one fma: |dz| <= 3 u |acc sx sw| + u |z|.
  act: every activation is 1.2-Lipschitz (the steepest, gelu, has slope 1.13).  Its own evaluation
    rounds an exponent argument of size at most 2 z^2 + 2 |z| (z^2 / 2 in erfc, 2 |z| (0.8 +
    0.036 z^2) in the tanh form, |z| in silu) a few times and then takes exp, rcp (1 ulp each) or erfc
    (below 16 ulp): relative error at most (16 + 4 (z^2 + |z|)) 2 u, of |act(z)|.  The tanh form's
    argument grows as z^3, but where it exceeds 2 z^2 + 2 |z| (z > 54) the result is z or 0.
    Values the hardware exponential flushes are below 2^-120: an absolute 1e-30.
"""
import numpy as np
from scipy import special

U = 2.0 ** -24
BF16 = 2.0 ** -8
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def act(z, name):
    z = np.asarray(z, dtype=np.float64)
    if name == "none":
        return z
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "silu":
        return z * special.expit(z)
    if name == "gelu":
        return z * special.ndtr(z)
    if name == "gelu_tanh":
        return z * special.expit(2.0 * np.sqrt(2.0 / np.pi) * (z + 0.044715 * z ** 3))
    raise ValueError(name)


def act_slope(z, name):
    z = np.asarray(z, dtype=np.float64)
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        p = special.expit(z)
        return p + z * p * special.expit(-z)
    if name == "gelu":
        return special.ndtr(z) + z * np.exp(-0.5 * z * z) / np.sqrt(2.0 * np.pi)
    if name == "gelu_tanh":
        c = 2.0 * np.sqrt(2.0 / np.pi)
        t = c * (z + 0.044715 * z ** 3)
        p = special.expit(t)
        return p + z * p * special.expit(-t) * c * (1.0 + 3 * 0.044715 * z * z)
    raise ValueError(name)


def linear_z(qx, sx, qw, sw, bias):
    """z and its fp32 error bound from the operands' own codes and scales."""
    acc = qx.astype(np.float64) @ qw.astype(np.float64).T
    p = acc * sx.astype(np.float64)[:, None] * sw.astype(np.float64)[None, :]
    z = p + (0.0 if bias is None else bias.astype(np.float64)[None, :])
    return z, 3 * U * np.abs(p) + U * np.abs(z)


def act_bound(z, dz, name):
    """act(z) and the bound of its fp32 evaluation at a z that is off by up to dz."""
    a = act(z, name)
    own = 0.0 if name in ("none", "relu") else (16 + 4 * (z * z + np.abs(z))) * 2 * U * np.abs(a) + 1e-30
    return a, 1.2 * dz + own


def rounded(v, dv):
    """Bound of bf16(v') against v for |v' - v| <= dv."""
    return dv + BF16 * (np.abs(v) + dv) + 1e-38


def check(got, ref, bound, what):
    err = np.abs(got.astype(np.float64) - ref)
    worst = float((err / bound).max(initial=0.0))
    assert np.isfinite(got).all() and worst <= 1.0, "%s: error is %.3g times its bound" % (what, worst)
    return worst


def hadamard(g):
    i = np.arange(g)
    ones = np.array([[bin(a & b).count("1") for b in i] for a in i])
    return (1.0 - 2.0 * (ones & 1)) / np.sqrt(g)


def rotate(v, g):
    h = hadamard(g)
    return (v.reshape(-1, g) @ h).reshape(v.shape)


def rotate_abs(v, g):
    """Bound of |rotate(w)| for |w| <= v: each channel sums its whole group's magnitudes / sqrt(g)."""
    s = v.reshape(-1, g).sum(1, keepdims=True) / np.sqrt(g)
    return np.broadcast_to(s, (s.shape[0], g)).reshape(v.shape)
