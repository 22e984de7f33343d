"""More rows, slots and tokens than one dimension of a launch holds workgroups of 256 threads (2^24): gradients and router, against the
same calls on parts and formulas in 64 bits."""
import numpy as np
import pytest
import torch

from tests import fused_reference as R
from tests import moe_reference as MR
from tests import parity as P
from tests.test_gpu_moe import DEV, _layer, _np, _weights, cr  # noqa: F401  (cr is a fixture)

pytestmark = pytest.mark.gpu


def _big(*shape, seed, std=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.empty(*shape, dtype=torch.bfloat16, device=DEV).normal_(0.0, std, generator=gen)


def _around(n):
    """Parts of n rows at both ends and around 2^22 and 2^24."""
    return [(0, 100), ((1 << 22) - 50, (1 << 22) + 50), ((1 << 24) - 50, min((1 << 24) + 50, n)), (n - 60, n)]


def test_grouped_gradient_of_many_rows(cr):
    rows, N, K = (1 << 24) + 300, 64, 64
    P.say("linear_grouped_backward rows=%d" % rows)
    wq, ws = _weights(cr, 3, N, K, 64, 1)
    ends = [5, 700, (1 << 24) - 7, rows - 3]                      # the first 5 and last 3 rows of no group
    offsets = torch.tensor(ends, dtype=torch.int32, device=DEV)
    dy = _big(rows, N, seed=1)
    out = torch.full((rows, K), float("nan"), dtype=torch.bfloat16, device=DEV)
    cr.linear_grouped_backward(dy, wq, ws, offsets, group=64, out=out)
    assert out[:5].isnan().all() and out[-3:].isnan().all() and out[5:-3].isfinite().all()
    group = torch.searchsorted(offsets, torch.arange(rows, device=DEV, dtype=torch.int32), right=True) - 1
    for lo, hi in _around(rows):
        for e in range(3):
            m = lo + torch.nonzero(group[lo:hi] == e)[:, 0]
            if not len(m):
                continue
            a, q = _np((dy[m].float() * ws[e]).bfloat16()), _np(wq[e])
            ref = R.rotate(a @ q, 64)
            R.check(_np(out[m]), ref, R.rounded(ref, (N + 16) * R.U * R.rotate_abs(np.abs(a) @ np.abs(q), 64)), "dx")


def test_layer_gradient_of_many_slots(cr):
    M, top, E, F, K = (1 << 21) + 9, 8, 8, 64, 64
    P.say("moe_ffn_gated_backward M=%d top=%d" % (M, top))
    gate, up, down = _layer(cr, E, F, K, 64, 64)
    gen = torch.Generator(device=DEV).manual_seed(1)
    experts = torch.randint(-1, E, (M, top), generator=gen, device=DEV, dtype=torch.int32)
    w = torch.rand(M, top, generator=gen, device=DEV)
    dy, pre, d = _big(M, K, seed=2), _big(2, M, top, F, seed=3, std=1.5), _big(M, top, K, seed=4)
    dx, dw = cr.moe_ffn_gated_backward(dy, pre, d, experts, w, *gate, *up, *down, group=64, group_h=64)
    assert dx.isfinite().all() and dw.isfinite().all() and (dw[experts < 0] == 0).all()
    for lo, hi in [(0, 40), ((1 << 19) - 20, (1 << 19) + 20), ((1 << 21) - 20, (1 << 21) + 9)]:
        at = slice(lo, hi)
        own = lambda t: t[at].clone()
        _, part = cr.moe_ffn_gated_backward(own(dy), pre[:, at].clone(), own(d), own(experts), own(w), *gate, *up, *down, group=64,
                                            group_h=64)
        assert torch.equal(dw[at], part)
        ref, _ = MR.moe_backward(_np(dy[at]), _np(pre[:, at]), _np(d[at]), experts[at].cpu().numpy(), _np(w[at]),
                                 *[(_np(p[0]), _np(p[1])) for p in (gate, up, down)], "silu", 64, 64)
        assert np.linalg.norm(_np(dx[at]) - ref) <= 2 * R.BF16 * np.linalg.norm(ref)


def test_router_of_the_most_tokens(cr):
    M, E = (1 << 26) - 1, 2
    P.say("moe_route M=%d" % M)
    x = _big(M, E, seed=1)
    experts, w = cr.moe_route(x, 1, normalize=False)
    want = (x[:, 1] > x[:, 0]).to(torch.int32)
    assert torch.equal(experts[:, 0], want)
    far = (x[:, 0].float() - x[:, 1].float()).abs()
    share = 1.0 / (1.0 + torch.exp(-far))
    # the test's own difference, exponential and quotient in fp32 (a share moves by u / 4 of the difference, at most 12): 8 u
    assert (w[:, 0] - share).abs().max() <= MR.ROUTE_TOL + 8 * R.U
    del experts, w, share
    dw = torch.ones(M, 1, device=DEV)
    dx = cr.moe_route_backward(dw, x, want[:, None].contiguous(), normalize=False)
    for lo, hi in _around(M) + [((1 << 25) - 50, (1 << 25) + 50)]:
        ref = MR.route_backward(np.ones((hi - lo, 1)), x[lo:hi].double().cpu().numpy(), want[lo:hi, None].cpu().numpy(), "softmax", False)
        got = dx[lo:hi].double().cpu().numpy()
        assert np.all(np.abs(got - ref) <= R.BF16 * np.abs(ref) + MR.ROUTE_TOL)
    assert dx.isfinite().all() and (dx.float().abs().amax(1) > 0).float().mean() > 0.99
