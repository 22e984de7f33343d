"""The router's gradient where one or two logits lead all others: the terms of a token's gradient then cancel to about the
share of the rest, and every entry has to keep its digits.

The reference sums differences, dl_i = s_i sum_k s_k (G_i - G_k) with G the gradients a logit's slots received (and the same
over the chosen shares where they are normalised), in 80 bits, so that nothing in it cancels.
Bound: the kernel forms an entry in 64 bits, off by at most E^2 2^-53 of the row's largest entry (sums of up to E terms, each
at most the entry of its own logit or the sum itself), below 2^-33 of it, and rounds it once: u |entry| in fp32, u = 2^-24, and 2^-8
|entry| more to bf16.  2 u of the row's largest entry are allowed besides, and 1e-37 where fp32 ends."""
import numpy as np
import pytest
import torch

from tests import fused_reference as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
KINDS = [(s, n) for s in ("softmax", "sigmoid") for n in (True, False)]
LEADS = [0.0, 2.0, 8.0, 12.0, 16.0, 18.0, 20.0, 30.0, 45.0, 60.0, 80.0]


@pytest.fixture(scope="module")
def cr():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from int4_quantized_linear_amd import convrot
    convrot.load()
    return convrot


def _np(t):
    return t.detach().double().cpu().numpy()


def reference(dw, logits, experts, score, normalize, scale):
    out = np.zeros(logits.shape)
    for m in range(logits.shape[0]):
        l, g = logits[m].astype(np.longdouble), dw[m].astype(np.longdouble) * np.longdouble(scale)
        at, row = experts[m], np.zeros(logits.shape[1], dtype=np.longdouble)
        if normalize:
            v = l[at] if score == "softmax" else -np.logaddexp(np.longdouble(0), -l[at])
            q = np.exp(v - v.max())
            q = q / q.sum()
            part = q * ((g[:, None] - g[None, :]) * q[None, :]).sum(1)
        elif score == "sigmoid":
            part = g / (1 + np.exp(-l[at]))
        if score == "softmax" and not normalize:
            s = np.exp(l - l.max())
            s = s / s.sum()
            big = np.zeros_like(s)
            np.add.at(big, at, g)
            row = s * ((big[:, None] - big[None, :]) * s[None, :]).sum(1)
        else:
            if score == "sigmoid":
                part = part / (1 + np.exp(l[at]))
            np.add.at(row, at, part)
        out[m] = row
    return out


def _check(cr, x, dw, experts, score, normalize):
    for dtype in (torch.float32, torch.bfloat16):
        y = x.to(dtype)
        ref = reference(_np(dw), _np(y), experts.cpu().numpy(), score, normalize, 2.5)
        got = _np(cr.moe_route_backward(dw, y, experts, score=score, normalize=normalize, scale=2.5))
        step = R.U if dtype is torch.float32 else R.BF16
        bound = step * np.abs(ref) + 2 * R.U * np.abs(ref).max(1, keepdims=True) + 1e-37
        R.check(got, ref, bound, "dlogits")


@pytest.mark.parametrize("score,normalize", KINDS)
@pytest.mark.parametrize("E,top", [(2, 1), (9, 2), (64, 1), (64, 5), (65, 2), (200, 6), (1024, 32)])
def test_leading_logits(cr, E, top, score, normalize):
    """One and two leading logits, the second a little behind or equal; the leaders' incoming gradients far apart, near and
    equal."""
    gen = torch.Generator().manual_seed(E + top)
    rows, grads = [], []
    for lead in LEADS:
        for second in (None, 0.0, 0.375):
            l = torch.randn(E, generator=gen)
            first = int(torch.randint(E, (1,), generator=gen))
            most = l.max()
            l[first] = most + lead
            if second is not None:
                l[(first + 1) % E] = most + lead - second
            for kind in range(3):
                g = torch.randn(top, generator=gen)
                if kind == 1:
                    g = 1.0 + g * 2.0 ** -20
                if kind == 2:
                    g[:] = g[0]
                rows.append(l)
                grads.append(g)
    x, dw = torch.stack(rows).to(DEV), torch.stack(grads).to(DEV)
    # logits of bf16, so that both types have the same experts
    x = x.bfloat16().float()
    experts, _ = cr.moe_route(x, top, score=score, normalize=normalize)
    _check(cr, x, dw, experts, score, normalize)


@pytest.mark.parametrize("score,normalize", KINDS)
def test_leading_logit_without_a_slot(cr, score, normalize):
    """Experts chosen by a bias: the leading logit has no slot, and the chosen ones share next to nothing."""
    x = torch.randn(12, 70, generator=torch.Generator().manual_seed(2)).to(DEV).bfloat16().float()
    x[:, 3] = torch.linspace(2, 40, 12, device=DEV).bfloat16().float()
    b = torch.zeros(70, device=DEV)
    b[3], b[40:44] = -torch.inf, 10.0
    experts, _ = cr.moe_route(x, 4, bias=b, score=score, normalize=normalize)
    assert ((experts >= 40) & (experts < 44)).all()
    dw = torch.randn(12, 4, generator=torch.Generator().manual_seed(3)).to(DEV)
    _check(cr, x, dw, experts, score, normalize)


@pytest.mark.parametrize("score,normalize", KINDS)
def test_slots_of_one_expert_that_cancel(cr, score, normalize):
    """An expert in two slots whose gradients nearly cancel gets the sum of both, not of their roundings."""
    x = torch.randn(6, 20, generator=torch.Generator().manual_seed(2)).to(DEV).bfloat16().float()
    experts = torch.tensor([[3, 3], [0, 0], [19, 19], [5, 5], [3, 3], [7, 7]], dtype=torch.int32, device=DEV)
    dw = torch.randn(6, 2, generator=torch.Generator().manual_seed(3)).to(DEV)
    dw[:, 1] = -dw[:, 0] * (1 + 2.0 ** -16)
    if normalize:                                                # (a third expert, or every share is constant)
        experts = torch.cat([experts, (experts[:, :1] + 1) % 20], 1).contiguous()
        dw = torch.cat([dw, dw[:, :1] * 2.0 ** -18], 1).contiguous()
    _check(cr, x, dw, experts, score, normalize)
