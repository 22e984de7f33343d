"""What the expert layer's sums over a token's slots keep: fp32 from the down product, and from each slot's gradient, to the one
rounding to bf16, whatever the sizes of neighbouring channels, for every number of slots.

Bounds (u = 2^-24).  y: as in test_gpu_moe.py, 3 u |acc sx sw| for each slot's result, (top + 2) u of the sum of magnitudes, one
bf16 rounding, with nothing else between.  A token's bits are those that it gets in a call of its own.
dx: with one slot per token and a weight of 1, the layer's gradient is its expert's dense block's: the same operands, the sums of
2 F products in fp32 in an order of their own, each within (2 F + 16) u of the sum of magnitudes.  Both are taken with the dense result
subtracted (dx_add), so that what is left shows what lies below its bf16 rounding: equal to twice the sums' error, u of
the value for each subtraction, and the two roundings of the rest."""
import numpy as np
import pytest
import torch

from tests import fused_reference as R
from tests import parity as P
from tests.test_gpu_moe import DEV, _experts, _expert_by_expert, _layer, _np, _randn, cr  # noqa: F401  (cr is a fixture)

pytestmark = pytest.mark.gpu

# M, top, E, F, K, group_h, group: products in 64-, 128- and 256-row tiles (the last three among them)
SIZES = [(33, 2, 5, 128, 192, 64, 64), (301, 3, 16, 448, 640, 64, 128), (700, 1, 3, 256, 320, 256, 64), (901, 3, 3, 1088, 1344, 64, 64),
         (1500, 3, 5, 2112, 1024, 64, 256), (2100, 2, 4, 1344, 2688, 64, 128)]


def _uneven(down, seed):
    """One of 64 neighbouring output channels 4096 times as large as the others, another one 64 times."""
    q, s = down
    s = s.clone()
    gen = torch.Generator().manual_seed(seed)
    for first in range(0, s.shape[1], 64):
        a, b = torch.randperm(64, generator=gen)[:2].tolist()
        s[:, first + a] *= 4096.0
        s[:, first + b] *= 64.0
    return q, s


@pytest.mark.parametrize("M,top,E,F,K,gh,g", SIZES)
def test_uneven_output_channels(cr, M, top, E, F, K, gh, g):
    P.say("moe precision M=%d top=%d E=%d F=%d K=%d" % (M, top, E, F, K))
    gate, up, down = _layer(cr, E, F, K, gh, g)
    down = _uneven(down, M)
    experts, w = _experts(M, top, E, M + top, "dropped" if M == 301 else "mixed")
    x, res = _randn(M, K, seed=M), _randn(M, K, seed=M + 1, std=0.01)
    call = dict(group=g, group_h=gh)
    y = cr.moe_ffn_gated(x, experts, w, *gate, *up, *down, residual=res, **call)
    _, _, d64, dd = _expert_by_expert(cr, x, experts, gate, up, down, "silu", g, gh)
    wn = _np(w)[:, :, None]
    ref = (d64 * wn).sum(1) + _np(res)
    size = (np.abs(d64) * wn).sum(1) + np.abs(_np(res))
    R.check(_np(y), ref, R.rounded(ref, (dd * wn).sum(1) + (top + 2) * R.U * size), "y")
    # below the rounding: the same with bf16(y) taken off
    less = cr.moe_ffn_gated(x, experts, w, *gate, *up, *down, residual=-y, **call)
    ref = (d64 * wn).sum(1) - _np(y)
    size = (np.abs(d64) * wn).sum(1) + np.abs(_np(y))
    R.check(_np(less), ref, R.rounded(ref, (dd * wn).sum(1) + (top + 2) * R.U * size), "y - bf16(y)")


@pytest.mark.parametrize("M,top,E,F,K,gh,g", SIZES)
def test_a_token_alone_gets_the_same_bits(cr, M, top, E, F, K, gh, g):
    """Calls of at most 64 slots have kernels of their own."""
    gate, up, down = _layer(cr, E, F, K, gh, g)
    experts, w = _experts(M, top, E, M + top, "dropped")
    x, res, call = _randn(M, K, seed=M), _randn(M, K, seed=M + 1), dict(group=g, group_h=gh)
    for r in (res, None):
        y = cr.moe_ffn_gated(x, experts, w, *gate, *up, *down, residual=r, **call)
        for first in (0, M // 2, M - 20):
            at = slice(first, first + 20)
            own = lambda t: None if t is None else t[at].clone()
            alone = cr.moe_ffn_gated(own(x), own(experts), own(w), *gate, *up, *down, residual=own(r), **call)
            assert torch.equal(alone, y[at]), first


# M, E, F, K: gradient tiles of 64 and of 256 rows
BACKWARD = [(90, 4, 64, 128), (300, 3, 192, 320), (9000, 2, 1344, 128)]


@pytest.mark.parametrize("size", [1.0, 2.0 ** -112])
@pytest.mark.parametrize("M,E,F,K", BACKWARD)
def test_uneven_gradient_channels(cr, M, E, F, K, size):
    """Rotation groups of one channel, so that a gate or up column of small codes is a channel of small gradients, also next to the
    end of the range.  The first contraction is over whole numbers and exact, so that both calls round the same dh."""
    gen = torch.Generator(device=DEV).manual_seed(F)
    stack = lambda n, k: torch.randint(-127, 128, (E, n, k), generator=gen, device=DEV, dtype=torch.int8)
    even = lambda n, scale: torch.full((E, n), scale, device=DEV)
    gate, up, down = (stack(F, K), even(F, 0.25)), (stack(F, K), even(F, 0.25)), (stack(K, F), even(K, 2.0 ** -12))
    for q in (gate[0], up[0]):
        q[:, :, torch.arange(K, device=DEV) % 64 != 5] = torch.randint(-1, 2, (E, F, K - K // 64), generator=gen, device=DEV, dtype=torch.int8)
    experts = torch.randint(0, E, (M, 1), generator=torch.Generator().manual_seed(1), dtype=torch.int32).to(DEV)
    ones = torch.ones(M, 1, device=DEV)
    dy = (torch.randint(-4, 5, (M, K), generator=gen, device=DEV) * size).bfloat16()
    pre = _randn(2, M, 1, F, seed=2)
    layer = lambda add: cr.moe_ffn_gated_backward(dy, pre, None, experts, ones, *gate, *up, *down, group=1, group_h=1, dx_add=add)[0]
    dense, rest, bound = torch.zeros_like(dy), torch.zeros_like(dy), np.zeros((M, K))
    for e in range(E):
        m = torch.nonzero(experts[:, 0] == e)[:, 0]
        p = [v for w in (gate, up, down) for v in (w[0][e], w[1][e])]
        block = lambda add: cr.ffn_gated_backward(dy[m].contiguous(), pre[:, m, 0].contiguous(), *p, group=1, group_h=1, dx_add=add)
        dense[m] = block(None)
        rest[m] = block(-dense[m])
        dh = (_np(dy[m]) * _np(down[1][e])) @ _np(down[0][e])
        z, u = _np(pre[0, m, 0]), _np(pre[1, m, 0])
        a, b = dh * u * R.act_slope(z, "silu") * _np(gate[1][e]), dh * R.act(z, "silu") * _np(up[1][e])
        # (1 + 2^-6: the operands' own roundings)
        total = np.abs(a) @ np.abs(_np(gate[0][e])) + np.abs(b) @ np.abs(_np(up[0][e]))
        bound[m.cpu().numpy()] = 2 * (2 * F + 16) * R.U * (1 + 2.0 ** -6) * total
    got, dense64, rest64 = _np(layer(-dense)), _np(dense), _np(rest)
    bound += 2 * R.U * np.abs(dense64) + R.BF16 * (np.abs(rest64) + np.abs(got)) + 2.0 ** -126
    R.check(got, rest64, bound, "what dx has below its rounding")
