"""The router and its gradient against their definition in 64 bits: every score, normalisation, type and width class, ties,
masked experts, rows with nothing to choose from, lowest and highest values, NaN, biases that decide beyond fp32."""
import numpy as np
import pytest
import torch

from tests import fused_reference as R
from tests import moe_reference as MR
from tests import parity as P

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
KINDS = [(s, n) for s in ("softmax", "sigmoid") for n in (True, False)]


@pytest.fixture(scope="module")
def cr():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from int4_quantized_linear_amd import convrot
    convrot.load()
    return convrot


def _logits(M, E, seed, dtype=torch.float32, std=2.0):
    return (torch.randn(M, E, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).to(DEV)


def _np(t):
    return t.detach().double().cpu().numpy()


def _check(cr, logits, top, bias=None, score="softmax", normalize=True, scale=1.0):
    experts, weights = cr.moe_route(logits, top, bias=bias, score=score, normalize=normalize, scale=scale)
    e, w = MR.route(_np(logits), top, None if bias is None else _np(bias), score, normalize, scale)
    assert experts.dtype == torch.int32 and weights.dtype == torch.float32
    assert np.array_equal(experts.cpu().numpy(), e)
    assert np.all(np.abs(_np(weights) - w) <= MR.ROUTE_TOL * np.abs(w) + 1e-37)
    return experts, weights


# one and several logits per lane, whole and ragged; top up to all experts and to the largest
SIZES = [(1, 1, 1), (1, 64, 8), (3, 2, 2), (5, 7, 7), (33, 63, 1), (70, 65, 6), (9, 128, 32), (257, 200, 8), (12, 256, 8),
         (6, 257, 5), (4, 512, 12), (3, 513, 3), (5, 1024, 32)]


@pytest.mark.parametrize("score,normalize", KINDS)
@pytest.mark.parametrize("M,E,top", SIZES)
def test_route(cr, M, E, top, score, normalize):
    P.say("moe_route M=%d E=%d top=%d %s %s" % (M, E, top, score, normalize))
    for dtype in (torch.float32, torch.bfloat16):               # bf16 logits tie
        x = _logits(M, E, M + E, dtype)
        _check(cr, x, top, score=score, normalize=normalize, scale=2.5)
        b = torch.randn(E, generator=torch.Generator().manual_seed(E)).mul_(0.1).to(DEV)
        _check(cr, x, top, bias=b, score=score, normalize=normalize)


@pytest.mark.parametrize("score,normalize", KINDS)
def test_route_ties_and_zeros(cr, score, normalize):
    x = torch.zeros(4, 100, device=DEV)
    x[1, ::2] = -0.0                                             # equal to 0: the lowest index still wins
    x[2, 50:] = 1.0
    x[3, 99] = 1.0
    e, _ = _check(cr, x, 5, score=score, normalize=normalize)
    assert e[0].tolist() == [0, 1, 2, 3, 4] and e[1].tolist() == [0, 1, 2, 3, 4]
    assert e[2].tolist() == [50, 51, 52, 53, 54] and e[3].tolist() == [99, 0, 1, 2, 3]
    _check(cr, x, 5, bias=torch.zeros(100, device=DEV), score=score, normalize=normalize)


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("score,normalize", KINDS)
def test_route_masks(cr, score, normalize, biased):
    """Experts masked by -inf, down to fewer than top and to none."""
    x = _logits(6, 70, 1)
    x[0, 1:] = -torch.inf
    x[1, :] = -torch.inf
    x[2, 4:] = -torch.inf
    x[3, ::2] = -torch.inf
    b = torch.linspace(-1, 1, 70, device=DEV) if biased else None
    e, w = _check(cr, x, 6, bias=b, score=score, normalize=normalize)
    assert e[1].tolist() == [-1] * 6 and w[1].tolist() == [0.0] * 6
    assert e[0].tolist() == [0] + [-1] * 5 and (e[2] >= 0).sum() == 4
    if biased:
        b[5] = -torch.inf                                        # a bias masks too
        x[4, :] = -torch.inf
        x[4, 5] = 3.0
        e, w = cr.moe_route(x, 6, bias=b, score=score, normalize=normalize)
        assert not (e == 5).any() and e[4].tolist() == [-1] * 6 and w[4].tolist() == [0.0] * 6


@pytest.mark.parametrize("score,normalize", KINDS)
def test_route_extremes(cr, score, normalize):
    """The type's lowest and largest values, where every score is 0 or 1 in fp32."""
    low = torch.finfo(torch.float32).min
    x = torch.full((5, 9), low, device=DEV)
    x[1, 3] = 5.0
    x[2] = -200.0 - torch.arange(9, device=DEV)
    x[3] = 3e38
    x[4] = 100.0 + torch.arange(9, device=DEV)
    e, w = _check(cr, x, 3, score=score, normalize=normalize)
    assert w.isfinite().all()
    if normalize:
        assert torch.allclose(w.sum(1), torch.ones(5, device=DEV))
    x = torch.full((1, 9), torch.finfo(torch.bfloat16).min, dtype=torch.bfloat16, device=DEV)
    _check(cr, x, 3, score=score, normalize=normalize)


@pytest.mark.parametrize("score,normalize", KINDS)
def test_route_nan(cr, score, normalize):
    """A NaN reaches its own row's weights, and no other; the experts stay distinct and in range."""
    x = _logits(5, 80, 2)
    x[1, 7] = torch.nan
    x[3] = torch.nan
    e, w = cr.moe_route(x, 8, score=score, normalize=normalize)
    assert w[1].isnan().all() and w[3].isnan().all() and w[[0, 2, 4]].isfinite().all()
    assert len(set(e[1].tolist())) == 8 and 7 not in e[1].tolist() and e[3].tolist() == [-1] * 8
    want = cr.moe_route(x[[0, 2, 4]].contiguous(), 8, score=score, normalize=normalize)
    assert torch.equal(e[[0, 2, 4]], want[0]) and torch.equal(w[[0, 2, 4]], want[1])
    if score == "sigmoid" or not normalize:
        x = _logits(1, 80, 2)
        x[0, 9] = torch.inf
        e, w = cr.moe_route(x, 2, score=score, normalize=normalize)
        assert e[0, 0] == 9 and (w.isfinite().all() if score == "sigmoid" else w.isnan().all())


def test_route_keys_beyond_fp32(cr):
    """Scores and biases whose sums differ by less than a step of fp32: the larger one is chosen."""
    E = 64
    x = torch.zeros(1, E, device=DEV)
    b = torch.zeros(E, device=DEV)
    b[10], b[3] = 2.0 ** -30, 2.0 ** -31                         # 1/2 + 2^-30 and 1/2 + 2^-31 are 1/2 in fp32
    e, _ = cr.moe_route(x, 3, bias=b, score="sigmoid")
    assert e[0].tolist() == [10, 3, 0]


@pytest.mark.parametrize("score,normalize", KINDS)
@pytest.mark.parametrize("M,E,top", SIZES)
def test_route_backward(cr, M, E, top, score, normalize):
    P.say("moe_route_backward M=%d E=%d top=%d %s %s" % (M, E, top, score, normalize))
    x = _logits(M, E, M + E)
    if E > 40:
        x[0, 5:30] = -torch.inf
    x[M // 2, 1:] = -torch.inf                                   # one expert left
    experts, _ = cr.moe_route(x, top, score=score, normalize=normalize)
    dw = torch.randn(M, top, generator=torch.Generator().manual_seed(3)).to(DEV)
    got = cr.moe_route_backward(dw, x, experts, score=score, normalize=normalize, scale=2.5)
    ref = MR.route_backward(_np(dw), _np(x), experts.cpu().numpy(), score, normalize, 2.5)
    # fp32 shares (ROUTE_TOL) of terms that may cancel: relative to the row's largest gradient term
    size = 2.5 * np.abs(_np(dw)).max(1, keepdims=True) + 1e-30
    assert np.all(np.abs(_np(got) - ref) <= MR.ROUTE_TOL * size + R.U * np.abs(ref))
    assert torch.isfinite(got).all()
    # bf16 logits: the gradient is rounded to their type; in place of the logits' own buffer
    y = x.bfloat16()
    ref = MR.route_backward(_np(dw), _np(y), experts.cpu().numpy(), score, normalize, 2.5)
    place = y.clone()
    got = cr.moe_route_backward(dw, place, experts, score=score, normalize=normalize, scale=2.5, out=place)
    assert got is place and np.all(np.abs(_np(got) - ref) <= MR.ROUTE_TOL * size + R.BF16 * np.abs(ref) + 1e-38)


@pytest.mark.parametrize("score,normalize", KINDS)
def test_route_backward_of_chosen_experts(cr, score, normalize):
    """Experts that the caller put there: twice the same, and values outside the range."""
    x = _logits(4, 20, 7)
    experts = torch.tensor([[3, 3, 5], [-1, 2, 20], [-1, -7, 1 << 30], [0, 19, 0]], dtype=torch.int32, device=DEV)
    dw = torch.randn(4, 3, generator=torch.Generator().manual_seed(1)).to(DEV)
    got = cr.moe_route_backward(dw, x, experts, score=score, normalize=normalize)
    ref = MR.route_backward(_np(dw), _np(x), experts.cpu().numpy(), score, normalize)
    assert np.abs(_np(got) - ref).max() <= 2 * MR.ROUTE_TOL * np.abs(_np(dw)).max()
    assert (got[2] == 0).all()


@pytest.mark.parametrize("score,normalize", KINDS)
def test_route_backward_against_differences(cr, score, normalize):
    """Central differences of the forward weights, with the choice fixed."""
    M, E, top, step = 6, 40, 4, 2.0 ** -7
    x = _logits(M, E, 11, std=1.0)
    experts, _ = cr.moe_route(x, top, score=score, normalize=normalize)
    dw = torch.randn(M, top, generator=torch.Generator().manual_seed(5)).to(DEV)
    v = torch.randn(M, E, generator=torch.Generator().manual_seed(6)).to(DEV)

    def loss(z):
        e, w = cr.moe_route(z, top, score=score, normalize=normalize)
        order = torch.argsort(e, 1)                              # the same set in another order
        back = torch.argsort(torch.argsort(experts, 1), 1)
        assert torch.equal(torch.gather(e, 1, order).gather(1, back), experts)
        return (torch.gather(w, 1, order).gather(1, back).double() * dw.double()).sum(1)

    # experts stay chosen: lift them above the others by more than the steps can move (shares of the rest tend to 0)
    x = x.scatter_add(1, experts.long(), torch.full((M, top), 3.0, device=DEV))
    got = (cr.moe_route_backward(dw, x, experts, score=score, normalize=normalize).double() * v.double()).sum(1)
    diff = (loss(x + step * v) - loss(x - step * v)) / (2 * step)
    # third derivatives of softmax and sigmoid are below 1: step^2 / 6 |v|_1^3 sum|dw|; rounding 2 u / step
    bound = (step ** 2 / 6 * v.abs().max().item() ** 3 * 8 + 4 * R.U / step) * dw.abs().sum(1).double()
    assert (got - diff).abs().le(bound).all()


def test_route_empty_and_views(cr):
    e, w = cr.moe_route(torch.empty(0, 8, device=DEV), 2)
    assert e.shape == (0, 2) and w.shape == (0, 2)
    flat = _logits(1, 65, 3).flatten()
    view = flat[1:].view(1, 64)                                  # 4-byte aligned only
    assert torch.equal(cr.moe_route(view, 4)[0], cr.moe_route(view.clone(), 4)[0])
    with pytest.raises(ValueError, match="contiguous"):
        cr.moe_route(_logits(8, 16, 1).t(), 2)


def test_route_long(cr):
    """More tokens than one launch row of workgroups, against torch."""
    x = _logits(50001, 96, 5)
    e, w = cr.moe_route(x, 4)
    v, i = torch.topk(x, 4, 1)
    assert torch.equal(e.long(), i)
    assert (w - torch.softmax(v, 1)).abs().max() < 1e-6
