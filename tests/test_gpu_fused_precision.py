"""Input gradients of one sign over long contractions, and near both ends of their range, against 64-bit
products of the same bf16 operand.

The output's own rounding would hide an error of the sums, so each call is made twice: dx1, then the same with
dx_add = -dx1.  The second returns v - dx1, at most 2^-8 |v|, rounded to bf16, so dx1 + dx2 is the sum v before its
rounding to within 2^-16 |v|.

Bounds.  The operand bf16(dz sw) is reproduced exactly (fp32 products, one rounding) and a product with a code is exact.
A sum of T terms in fp32 rounds at most T times, each time by at most u = 2^-24 of a partial sum.  The codes
of a rotated weight row have either sign, so partial sums grow as a random walk: the t-th is sqrt(t / T) of the last in the
mean square, the roundings are independent and uniform (1 / sqrt 3 of their largest), and the relative error is
u sqrt(T / 6) in the 2-norm, held to u sqrt(T); norm, rotation (8 steps) and slices add fewer than 16 roundings.  One
channel is held to 8 times the token's root mean square of that: 8 deviations of fewer than 2^24 channels."""
import pytest
import torch

from tests import fused_reference as R
from tests import parity as P

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def cr():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from int4_quantized_linear_amd import convrot
    convrot.load()
    return convrot


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _weight(cr, N, K, g, seed):
    return cr.prepare_weight((torch.randn(N, K, generator=_gen(seed), device=DEV) * 0.05).bfloat16(), g, 8)


def _one_signed(kind, M, N, seed):
    """[M, N] of one sign: all the same, or 1 +- 1/2 scattered; every third token negative."""
    t = torch.ones(M, N, device=DEV)
    if kind == "scattered":
        t += 0.5 * (2 * torch.rand(M, N, generator=_gen(seed), device=DEV) - 1)
    t[::3] *= -1
    return t


def _rotate(v, g):
    h = torch.from_numpy(R.hadamard(g)).to(DEV)
    return (v.reshape(-1, g) @ h).reshape(v.shape)


def _product(a, q):
    """a q in 64 bits, a few thousand rows of q at a time."""
    out = 0
    for n in range(0, q.shape[0], 8192):
        out = out + a[:, n:n + 8192].double() @ q[n:n + 8192].double()
    return out


def _unrounded(call):
    first = call(None)
    return first.double() + call(-first).double()


def _check(v, ref, terms, what):
    assert v.isfinite().all(), "%s: not finite" % what
    sums = R.U * (terms ** 0.5 + 16)
    err = (v - ref).abs()
    rel = (err.norm() / ref.norm()).item()
    rms = ref.pow(2).mean(1, keepdim=True).sqrt()
    worst = (err / (8 * sums * rms + 2.0 ** -16 * ref.abs())).max().item()
    P.say("%s: relative error %.2e (bound %.2e), worst channel %.2f of its bound" % (what, rel, sums + 2.0 ** -16, worst))
    assert rel <= sums + 2.0 ** -16 and worst <= 1.0, what


# 64-token tiles, sliced (the first two) and whole; 256-token tiles, sliced; the longest contractions, 64-token tiles
LINEAR = [(12, 16128, 5376, 256), (300, 16128, 640, 128), (4096, 2048, 2048, 256), (1024, 5120, 5120, 256),
          (4096, 16128, 2048, 256), (5, 524288, 128, 64), (600, 1048575, 64, 64)]


@pytest.mark.parametrize("kind", ["constant", "scattered"])
@pytest.mark.parametrize("M,N,K,g", LINEAR)
def test_one_signed_gradient(cr, M, N, K, g, kind):
    what = "linear_act_backward %s M=%d N=%d K=%d" % (kind, M, N, K)
    P.say(what)
    wq, ws = _weight(cr, N, K, g, N + K)
    dy = (_one_signed(kind, M, N, 7) * 1e-3).bfloat16()
    a = (dy.float() * ws).bfloat16()
    v = _unrounded(lambda add: cr.linear_act_backward(dy, wq, ws, group=g, dx_add=add)[0])
    _check(v, _rotate(_product(a, wq), g), N, what)


# 64-token tiles: sliced, whole; 256-token tiles: whole with whole, then ragged last steps of both weights, sliced in
# the middle of the second weight, sliced with ragged last steps
GATED = [(12, 25600, 1024, 256), (2752, 1000, 1536, 256), (4096, 1024, 4096, 256), (4096, 1001, 4096, 256), (1728, 65, 4864, 64),
         (2048, 25600, 5120, 256), (2048, 9001, 5120, 128)]


@pytest.mark.parametrize("kind", ["constant", "scattered"])
@pytest.mark.parametrize("M,N,K,g", GATED)
def test_one_signed_gated_gradient(cr, M, N, K, g, kind):
    """dg = dh u and du = dh g (no activation) of one sign through both weights."""
    what = "linear_gated_backward %s M=%d N=%d K=%d" % (kind, M, N, K)
    P.say(what)
    (q1, s1), (q2, s2) = _weight(cr, N, K, g, 1), _weight(cr, N, K, g, 2)
    dh = (_one_signed(kind, M, N, 7) * 1e-3).bfloat16()
    pre = torch.stack([_one_signed(kind, M, N, 8), _one_signed(kind, M, N, 9)]).abs().bfloat16()
    a1 = (dh.float() * pre[1].float() * s1).bfloat16()
    a2 = (dh.float() * pre[0].float() * s2).bfloat16()
    v = _unrounded(lambda add: cr.linear_gated_backward(dh, pre, q1, s1, q2, s2, act="none", group=g, dx_add=add))
    _check(v, _rotate(_product(a1, q1) + _product(a2, q2), g), 2 * N, what)


@pytest.mark.parametrize("scale", [1e-33, 1e-25, 1e12, 1e17, 1e25, 1e34])
@pytest.mark.parametrize("M,N,K,g", [(70, 264, 256, 256), (1728, 65, 4864, 256)])
def test_range_of_the_gradient(cr, M, N, K, g, scale):
    """Terms dz sw of one sign from the smallest bf16 holds in full to sums near fp32's largest (at most 127 * 264 times a
    term of 1e34 * 2e-3, and 16 of those through the rotation: 1e37), in 64- and 256-token tiles."""
    P.say("range M=%d N=%d K=%d scale %g" % (M, N, K, scale))
    wq, ws = _weight(cr, N, K, g, 3)
    dy = (_one_signed("scattered", M, N, 7) * scale).bfloat16()
    dy[1::4] = 0
    a = (dy.float() * ws).bfloat16()
    dx, _ = cr.linear_act_backward(dy, wq, ws, group=g)
    ref = _rotate(_product(a, wq), g)
    assert dx.isfinite().all() and not dx[1::4].any()
    bound = R.U * (N + 16) * _rotate_abs(_product(a.abs(), wq.abs()), g) + R.BF16 * ref.abs()
    assert ((dx.double() - ref).abs() <= bound * (1 + R.BF16) + 1e-38).all()


def _rotate_abs(v, g):
    return (v.reshape(-1, g).sum(1, keepdim=True) / g ** 0.5).expand(-1, g).reshape(v.shape)
