"""Backward calls whose contraction over two weights runs in 256-token tiles: whole and in slices, with the last step of
each weight whole and ragged (which kernel and slices a size takes is pinned in test_fused_plans_host.py).

Bounds as in test_gpu_fused_backward.py: an operand's rounding (2^-8 of a term at most) reaches dx with the same
relative mean square, the output's own adds another: 0.82 * 2^-8 in the 2-norm, held to 2^-8.  In the block dh's
own error passes through the second product next to that one's: twice."""
import pytest
import torch

from tests import fused_reference as R
from tests import parity as P
from tests.test_gpu_fused_precision import DEV, _gen, _product, _rotate, _weight, cr  # noqa: F401

pytestmark = pytest.mark.gpu


def _randn(*shape, seed, std=1.0):
    return (torch.randn(*shape, generator=_gen(seed), device=DEV) * std).bfloat16()


def _silu(z):
    """silu and its derivative in 64 bits."""
    z = z.double()
    p = torch.sigmoid(z)
    return z * p, p + z * p * torch.sigmoid(-z)


def _norm_check(got, ref, tol, what):
    rel = ((got.double() - ref).norm() / ref.norm()).item()
    P.say("%s: relative error %.2e (bound %.2e)" % (what, rel, tol))
    assert rel <= tol, what


def _gated(dh, pre, gate, up, g):
    """dx before dx_add, dg and du of the gated linear, in 64 bits."""
    value, slope = _silu(pre[0])
    dg, du = dh.double() * pre[1].double() * slope, dh.double() * value
    return _rotate(_product(dg * gate[1].double(), gate[0]) + _product(du * up[1].double(), up[0]), g), dg, du


# whole tiles, ragged ends; sliced, one slice beginning with the second weight; sliced, the second weight inside a slice
GATED = [(4096, 1001, 4096, 256), (1728, 65, 4864, 64), (1100, 16100, 1280, 256), (2048, 9001, 5120, 32)]


@pytest.mark.parametrize("M,N,K,g", GATED)
def test_gated_backward_256_token_tiles(cr, M, N, K, g):  # noqa: F811
    P.say("linear_gated_backward M=%d N=%d K=%d g=%d" % (M, N, K, g))
    gate, up = _weight(cr, N, K, g, 1), _weight(cr, N, K, g, 2)
    dh, pre, add = _randn(M, N, seed=1), _randn(2, M, N, seed=2, std=2.0), _randn(M, K, seed=3, std=0.1)
    dx, dbg, dbu = cr.linear_gated_backward(dh, pre, *gate, *up, group=g, bias_grad=True, dx_add=add)
    inner, dg, du = _gated(dh, pre, gate, up, g)
    _norm_check(dx, inner + add.double(), R.BF16, "dx")
    # M fp32 additions; an activation's or slope's own error is (24 + 6 (z^2 + |z|)) 2 u of its size, 115 u in the mean
    # for z of N(0, 2), against a mean |slope| of 0.6: 500 u of the sum of |terms|, and both doubled
    for got, terms in ((dbg, dg), (dbu, du)):
        assert ((got.double() - terms.sum(0)).abs() <= 2 * (M + 500) * R.U * terms.abs().sum(0)).all()
    assert torch.equal(cr.linear_gated_backward(dh, pre, *gate, *up, group=g, dx_add=add), dx)


# both steps whole; both sliced; the first partly whole, partly sliced
BLOCKS = [(4096, 4096, 2944), (1500, 4096, 3008), (2048, 5120, 9024)]


@pytest.mark.parametrize("M,K,F", BLOCKS)
def test_block_backward_256_token_tiles(cr, M, K, F):  # noqa: F811
    P.say("ffn_gated_backward M=%d K=%d F=%d" % (M, K, F))
    g, gh = cr.dynamic_group(K), cr.dynamic_group(F)
    gate, up, down = _weight(cr, F, K, g, 1), _weight(cr, F, K, g, 2), _weight(cr, K, F, gh, 3)
    dy, pre = _randn(M, K, seed=5), _randn(2, M, F, seed=6, std=1.5)
    dx, dbg, dbu, dbd = cr.ffn_gated_backward(dy, pre, *gate, *up, *down, group=g, group_h=gh, bias_grad=True)
    assert torch.equal(cr.ffn_gated_backward(dy, pre, *gate, *up, *down, group=g, group_h=gh), dx)
    dh, dbd2 = cr.linear_act_backward(dy, *down, group=gh, bias_grad=True)
    dx2, dbg2, dbu2 = cr.linear_gated_backward(dh, pre, *gate, *up, group=g, bias_grad=True)
    for a, b in ((dx, dx2), (dbg, dbg2), (dbu, dbu2), (dbd, dbd2)):
        assert torch.equal(a, b)
    dh64 = _rotate(_product(dy.double() * down[1].double(), down[0]), gh)
    _norm_check(dh, dh64, R.BF16, "dh")
    _norm_check(dx, _gated(dh64, pre, gate, up, g)[0], 2 * R.BF16, "dx")
