"""Plain 64-bit forms of the mixture-of-experts operators and the error bounds the tests hold the kernels to (u = 2^-24,
bf16 rounding at most 2^-8 of the value, as in fused_reference.py).

Router.  Shares and gradients are formed in 64 bits and rounded once, except the softmax's sum over all experts (fp32
exponentials of fp32 differences): each term is off by at most (|l - max| + 3) u, relative, and e^-x (x + 3) <= 3, so the sum
by at most 3 u of its largest term per expert that counts; 8 u of the result holds all of it for up to 1024 experts whose
logits spread (the sum of e^-x (x + 3) over the sum of e^-x is at most 3 + the mean of x, below 6 for any of the tests' rows).
"""
import numpy as np
import torch
from scipy import special

from tests import fused_reference as R

ROUTE_TOL = 10 * R.U


def scores(logits, score):
    x = np.asarray(logits, dtype=np.float64)
    if score == "sigmoid":
        return special.expit(x)
    top = np.max(x, axis=1, keepdims=True)
    e = np.exp(x - np.where(np.isfinite(top), top, 0.0))
    total = e.sum(1, keepdims=True)
    return e / np.where(total == 0, 1.0, total)


def log_scores(logits, score):
    """log s up to a constant per row, finite wherever the logit is."""
    x = np.asarray(logits, dtype=np.float64)
    return special.log_expit(x) if score == "sigmoid" else x


def route(logits, top, bias=None, score="softmax", normalize=True, scale=1.0):
    x = np.asarray(logits, dtype=np.float64)
    s = scores(x, score)
    key = x if bias is None else s + np.asarray(bias, dtype=np.float64)
    key = np.where(np.isneginf(x), -np.inf, key)
    experts = np.argsort(-key, axis=1, kind="stable")[:, :top]
    gone = np.isneginf(np.take_along_axis(key, experts, 1))
    if normalize:
        v = np.where(gone, -np.inf, np.take_along_axis(log_scores(x, score), experts, 1))
        most = v.max(1, keepdims=True)
        w = np.where(gone, 0.0, np.exp(v - np.where(np.isfinite(most), most, 0.0)))
        total = w.sum(1, keepdims=True)
        w = w / np.where(total == 0, 1.0, total)
    else:
        w = np.where(gone, 0.0, np.take_along_axis(s, experts, 1))
    return np.where(gone, -1, experts), w * scale


def route_backward(dw, logits, experts, score="softmax", normalize=True, scale=1.0):
    """By automatic differentiation of the weights' formula; slots without an expert add nothing."""
    x = torch.from_numpy(np.asarray(logits, dtype=np.float64)).clone()
    masked = torch.isneginf(x)
    x = torch.where(masked, torch.full_like(x, -1e4), x).requires_grad_()
    e = torch.from_numpy(np.asarray(experts)).long()
    ok = (e >= 0) & (e < x.shape[1])
    at = torch.where(ok, e, torch.zeros_like(e))
    ok = ok & ~masked.gather(1, at)
    if normalize:
        logs = torch.nn.functional.logsigmoid(x) if score == "sigmoid" else x
        v = torch.where(ok, logs.gather(1, at), torch.full_like(x[:, :1], -torch.inf))
        most = v.detach().max(1, keepdim=True).values
        w = torch.where(ok, torch.exp(v - torch.where(torch.isfinite(most), most, torch.zeros_like(most))), torch.zeros_like(v))
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        s = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, 1)
        w = torch.where(ok, s.gather(1, at), torch.zeros_like(s[:, :1]))
    (w * torch.from_numpy(np.asarray(dw, dtype=np.float64)) * scale).sum().backward()
    return torch.where(masked, torch.zeros_like(x), x.grad).numpy()


def slots_of(experts, e):
    """(token, slot) of the slots of expert e, in slot order."""
    return np.nonzero(np.asarray(experts) == e)


def moe_backward(dy, pre, d, experts, weights, gate, up, down, act, g, gh):
    """Formula gradients in 64 bits: (dx without dx_add, dweights); gate, up, down = (codes, scales) per expert."""
    M, K = dy.shape
    dx, dw = np.zeros((M, K)), np.zeros(experts.shape)
    for e in range(gate[0].shape[0]):
        t, j = slots_of(experts, e)
        if not len(t):
            continue
        dw[t, j] = (dy[t] * d[t, j]).sum(1)
        dh = R.rotate((dy[t] * weights[t, j][:, None] * down[1][e]) @ down[0][e], gh)
        z, u = pre[0][t, j], pre[1][t, j]
        part = (dh * u * R.act_slope(z, act) * gate[1][e]) @ gate[0][e] + (dh * R.act(z, act) * up[1][e]) @ up[0][e]
        np.add.at(dx, t, R.rotate(part, g))
    return dx, dw
