"""dx in the place of dy or of pre, which a backward call has read before it writes dx: the same bits as in a buffer of its
own, for few tokens and many, with and without bias gradients, with dx_add the same buffer too."""
import pytest
import torch

from tests import parity as P
from tests.test_gpu_fused_precision import DEV, _gen, _weight, cr  # noqa: F401

pytestmark = pytest.mark.gpu


def _randn(*shape, seed):
    return torch.randn(*shape, generator=_gen(seed), device=DEV).bfloat16()


def _same(got, want):
    got, want = [[t for t in r if t is not None] if isinstance(r, tuple) else [r] for r in (got, want)]
    return len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("M", [1, 16, 17, 300, 2048])
def test_linear(cr, M, bias):  # noqa: F811
    N = K = 1024
    P.say("in place, linear M=%d" % M)
    w = _weight(cr, N, K, 256, 1)
    dy, pre = _randn(M, N, seed=1), _randn(M, N, seed=2)
    run = lambda d, p, **kw: cr.linear_act_backward(d, *w, pre=p, act="gelu", bias_grad=bias, **kw)
    want, added = run(dy, pre), run(dy, pre, dx_add=dy)
    for place in ("dy", "pre"):
        d, p = dy.clone(), pre.clone()
        assert _same(run(d, p, out=d if place == "dy" else p), want), place
    d = dy.clone()
    assert _same(run(d, pre, dx_add=d, out=d), added)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("M", [1, 16, 17, 300, 2048])
def test_gated_and_block(cr, M, bias):  # noqa: F811
    K, F = 1024, 1024
    P.say("in place, gated and block M=%d" % M)
    gate, up, down = (_weight(cr, 1024, 1024, 256, s) for s in (1, 2, 3))
    dy, pre = _randn(M, K, seed=1), _randn(2, M, F, seed=2)
    for call, weights in ((cr.linear_gated_backward, (*gate, *up)), (cr.ffn_gated_backward, (*gate, *up, *down))):
        run = lambda d, p, **kw: call(d, p, *weights, bias_grad=bias, **kw)
        want, added = run(dy, pre), run(dy, pre, dx_add=dy)
        for place in ("dy", "gate", "up"):
            d, p = dy.clone(), pre.clone()
            assert _same(run(d, p, out={"dy": d, "gate": p[0], "up": p[1]}[place]), want), (call.__name__, place)
        d = dy.clone()
        assert _same(run(d, pre, dx_add=d, out=d), added), call.__name__
