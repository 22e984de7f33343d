"""Infinite and NaN logits and biases in the router: the rows they touch show it, and no others change.

An infinite logit under a softmax has no share that is a number, so its row's weights are NaN, in every slot and with every
normalisation, with a bias as without one; the row's experts are the largest logits' that no bias masks.  Under a
sigmoid it is a share of 1.  A NaN in the bias concerns every row: their weights are NaN and its expert is in none."""
import numpy as np
import pytest
import torch

from tests import moe_reference as MR

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
KINDS = [(s, n) for s in ("softmax", "sigmoid") for n in (True, False)]


@pytest.fixture(scope="module")
def cr():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from int4_quantized_linear_amd import convrot
    convrot.load()
    return convrot


def _np(t):
    return t.detach().double().cpu().numpy()


def _rows(E, seed, dtype):
    """Rows 1, 3, 5 and 6 with infinite logits: one, two, one that is alone, all."""
    x = torch.randn(8, E, generator=torch.Generator().manual_seed(seed)) * 2.0
    x[1, 7] = torch.inf
    x[3, 5], x[3, 8] = torch.inf, torch.inf
    x[5] = -torch.inf
    x[5, 2] = torch.inf
    x[6] = torch.inf
    return x.to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("score,normalize", KINDS)
@pytest.mark.parametrize("E,top", [(9, 1), (9, 9), (80, 8), (200, 3), (1024, 32)])
def test_infinite_logits(cr, E, top, score, normalize, biased, dtype):
    x = _rows(E, E + top, dtype)
    # (the bias would lift expert 0 over any share)
    b = torch.linspace(3, -3, E, device=DEV) if biased else None
    e, w = cr.moe_route(x, top, bias=b, score=score, normalize=normalize, scale=2.5)
    clean, infinite = [0, 2, 4, 7], [1, 3, 5, 6]
    want = cr.moe_route(x[clean].contiguous(), top, bias=b, score=score, normalize=normalize, scale=2.5)
    assert torch.equal(e[clean], want[0]) and torch.equal(w[clean], want[1])
    if score == "sigmoid":
        we, ww = MR.route(_np(x), top, None if b is None else _np(b), score, normalize, 2.5)
        assert np.array_equal(e.cpu().numpy(), we)
        assert np.all(np.abs(_np(w) - ww) <= MR.ROUTE_TOL * np.abs(ww) + 1e-37)
        return
    assert w[infinite].isnan().all(), "weights of rows with an infinite logit"
    order = MR.route(np.where(np.isposinf(_np(x)), 1e30, _np(x)), top, None, "sigmoid", False)[0]
    assert np.array_equal(e[infinite].cpu().numpy(), order[infinite]), "experts of rows with an infinite logit"


@pytest.mark.parametrize("normalize", [True, False])
def test_infinite_logits_of_masked_experts(cr, normalize):
    """A bias of -inf keeps its expert out, also where its logit is infinite and where nothing else is left."""
    x = _rows(40, 1, torch.float32)
    b = torch.zeros(40, device=DEV)
    b[2], b[7] = -torch.inf, -torch.inf
    e, w = cr.moe_route(x, 6, bias=b, score="softmax", normalize=normalize)
    assert not ((e == 2) | (e == 7)).any()
    assert w[[1, 3, 5, 6]].isnan().all() and w[[0, 2, 4, 7]].isfinite().all()
    assert e[5].tolist() == [-1] * 6 and e[6].tolist() == [0, 1, 3, 4, 5, 6] and e[3].tolist()[:2] == [5, 8]
    assert len(set(e[1].tolist())) == 6 and (e[1] >= 0).all()


@pytest.mark.parametrize("score,normalize", KINDS)
def test_nan_in_the_bias(cr, score, normalize):
    x = torch.randn(5, 70, generator=torch.Generator().manual_seed(4)).to(DEV)
    b = torch.linspace(-1, 1, 70, device=DEV)
    b[66] = torch.nan
    e, w = cr.moe_route(x, 6, bias=b, score=score, normalize=normalize)
    assert w.isnan().all() and not (e == 66).any()
    assert (e >= 0).all() and all(len(set(row)) == 6 for row in e.tolist())
