"""Input and bias gradients of the fused linears against their formulas in 64 bits, against central
differences of the forward calls, and in the ways a training loop calls them.

Bounds.  With act none the matrix core's operand a = bf16(dz sw) is reproduced exactly (one fp32
product, one rounding), so dx is off by fp32 sums alone: at most (N + 16) u of the sum of the absolute
terms, then the bf16 rounding.  The terms are a (q + 128), of which 128 sum(a) is taken back, itself a sum of
N terms: |a| (|q| + 256) bounds both.  With an activation a's rounding (2^-8 of a term at most, uniform:
2^-8 / sqrt 3 in the mean square) is independent over the terms, so it reaches dx with the same
relative mean square, and the output's own rounding adds another: 0.82 * 2^-8 of |dx| together,
held to 2^-8 in the 2-norm.  The slopes' fp32 errors are below 2^-18 for the inputs used here and vanish in that."""
import numpy as np
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


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _weight(cr, N, K, g, seed):
    gen = torch.Generator().manual_seed(seed)
    return cr.prepare_weight((torch.randn(N, K, generator=gen) * 0.05).bfloat16().to(DEV), g, 8)


def _randn(*shape, seed, std=1.0, dtype=torch.bfloat16):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * std).to(dtype).to(DEV)


def _norm_check(got, ref, what, tol=R.BF16):
    rel = np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-30)
    assert np.isfinite(got).all() and rel <= tol, "%s: relative error %.3g" % (what, rel)


def _slope_bound(z, act):
    """Absolute fp32 error of act'(z): the relative bound of fused_reference on each of its two terms,
    the second with three more factors."""
    if act in ("none", "relu"):
        return np.zeros_like(z)
    step = 1e-3
    size = np.abs(R.act(z, act)) / np.maximum(np.abs(z), 1e-30) + np.abs(z) * np.abs(
        R.act_slope(z + step, act) - R.act_slope(z - step, act)) / step + np.abs(R.act_slope(z, act)) + 1e-30
    return (24 + 6 * (z * z + np.abs(z))) * 2 * R.U * size


# one token, below and past a tile; N below a step, ragged, long; K and its group: one group per
# tile, several, none (g = 1), a last tile that is half empty
SHAPES = [(1, 1, 64, 64), (1, 4096, 256, 256), (3, 65, 320, 64), (16, 520, 512, 2), (33, 1001, 2688, 128),
          (130, 264, 192, 1), (255, 63, 64, 16), (257, 136, 640, 32), (300, 2000, 1024, 256), (600, 72, 1280, 8),
          (64, 192, 384, 4),
          # 256-token tiles: whole, a sliced last round, all sliced (the sizes above run 64-token tiles, whole and sliced)
          (1728, 65, 4864, 256), (1729, 64, 4864, 32), (3328, 384, 5120, 128), (2752, 3008, 1536, 256)]


@pytest.mark.parametrize("M,N,K,g", SHAPES)
def test_linear_backward_exact_operand(cr, M, N, K, g):
    P.say("linear_act_backward M=%d N=%d K=%d g=%d" % (M, N, K, g))
    wq, ws = _weight(cr, N, K, g, N + K)
    dy, add = _randn(M, N, seed=M, std=1e-3), _randn(M, K, seed=M + 1, std=1e-3)
    dy[M // 2] = 0
    dx, none = cr.linear_act_backward(dy, wq, ws, group=g)
    assert none is None
    a = (dy.float() * ws).bfloat16()
    q = _np(wq)
    ref = R.rotate(_np(a) @ q, g)
    terms = R.rotate_abs(np.abs(_np(a)) @ (np.abs(q) + 256), g)
    bound = (N + 16) * R.U * terms
    R.check(_np(dx), ref, R.rounded(ref, bound), "dx")
    dx2, db = cr.linear_act_backward(dy, wq, ws, group=g, dx_add=add, bias_grad=True)
    ref2 = ref + _np(add)
    R.check(_np(dx2), ref2, R.rounded(ref2, bound + R.U * np.abs(ref2)), "dx + add")
    sums = np.abs(_np(dy)).sum(0)
    R.check(db.double().cpu().numpy(), _np(dy).sum(0), (M + 8) * R.U * sums + 1e-38, "db")
    # in place, twice the same bits, and in place of dy's own buffer where the shapes allow it
    place = add.clone()
    got, _ = cr.linear_act_backward(dy, wq, ws, group=g, dx_add=place, out=place)
    assert got is place and torch.equal(place, dx2)
    assert torch.equal(cr.linear_act_backward(dy, wq, ws, group=g)[0], dx)


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("M,N,K,g", [(1, 520, 256, 256), (40, 1001, 640, 128), (300, 776, 320, 64)])
def test_linear_backward_with_activation(cr, M, N, K, g, act):
    P.say("linear_act_backward %s M=%d N=%d K=%d" % (act, M, N, K))
    wq, ws = _weight(cr, N, K, g, 3)
    dy, pre = _randn(M, N, seed=1), _randn(M, N, seed=2, std=3.0)
    dx, db = cr.linear_act_backward(dy, wq, ws, pre=pre, act=act, group=g, bias_grad=True)
    z = _np(pre)
    dz = _np(dy) * R.act_slope(z, act)
    _norm_check(_np(dx), R.rotate((dz * _np(ws)) @ _np(wq), g), "dx")
    err = (np.abs(_np(dy)) * _slope_bound(z, act)).sum(0) + (M + 8) * R.U * np.abs(dz).sum(0) + 1e-30
    R.check(db.double().cpu().numpy(), dz.sum(0), err, "db")


def test_slopes_far_out(cr):
    """Pre-activations up to 1e30 on both sides: slopes 0 and 1, no NaN from inf * 0."""
    N, K = 264, 256
    wq, ws = _weight(cr, N, K, 256, 3)
    z = torch.logspace(-30, 30, N // 2)
    pre = torch.cat([z, -z]).bfloat16().repeat(2, 1).to(DEV)
    dy = torch.ones(2, N, dtype=torch.bfloat16, device=DEV)
    for act in R.ACTS[1:]:
        _, db = cr.linear_act_backward(dy, wq, ws, pre=pre, act=act, bias_grad=True)
        ref = 2 * R.act_slope(_np(pre[0]), act)
        assert np.abs(db.double().cpu().numpy() - ref).max() < 1e-4, act


def test_slopes_at_infinity(cr):
    """Pre-activations of -inf and +inf (a lowest fp32 number in bf16): slopes 0 and 1; a masked gate passes nothing
    on to up."""
    N, K = 264, 256
    wq, ws = _weight(cr, N, K, 256, 3)
    pre = _randn(2, N, seed=1)
    pre[:, 0], pre[:, 9] = -torch.inf, torch.inf
    dy = torch.ones(2, N, dtype=torch.bfloat16, device=DEV)
    for act in R.ACTS[1:]:
        dx, db = cr.linear_act_backward(dy, wq, ws, pre=pre, act=act, bias_grad=True)
        assert db[0] == 0 and db[9] == 2 and db.isfinite().all() and dx.isfinite().all(), act
        both = torch.stack([pre, _randn(2, N, seed=2)])
        both[0, :, 9] = 0
        dx, dg, du = cr.linear_gated_backward(dy, both, wq, ws, wq, ws, act=act, bias_grad=True)
        assert dg[0] == 0 and du[0] == 0 and dx.isfinite().all(), act


GATED = [(1, 64, 64, 64), (5, 33, 320, 64), (40, 1001, 640, 128), (257, 136, 192, 64), (300, 776, 1024, 256)]


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("M,N,K,g", GATED)
def test_linear_gated_backward(cr, M, N, K, g, act):
    P.say("linear_gated_backward %s M=%d N=%d K=%d" % (act, M, N, K))
    gate, up = _weight(cr, N, K, g, 1), _weight(cr, N, K, g, 2)
    dh, pre, add = _randn(M, N, seed=1), _randn(2, M, N, seed=2, std=2.0), _randn(M, K, seed=3, std=0.1)
    dx, dbg, dbu = cr.linear_gated_backward(dh, pre, *gate, *up, act=act, group=g, bias_grad=True, dx_add=add)
    gz, u, d = _np(pre[0]), _np(pre[1]), _np(dh)
    dg, du = d * u * R.act_slope(gz, act), d * R.act(gz, act)
    ref = R.rotate((dg * _np(gate[1])) @ _np(gate[0]) + (du * _np(up[1])) @ _np(up[0]), g) + _np(add)
    _norm_check(_np(dx), ref, "dx")
    eg = (np.abs(d * u) * (_slope_bound(gz, act) + 2 * R.U)).sum(0) + (M + 8) * R.U * np.abs(dg).sum(0) + 1e-30
    eu = (np.abs(d) * R.act_bound(gz, 0.0, act)[1]).sum(0) + (M + 8) * R.U * np.abs(du).sum(0) + 1e-30
    R.check(dbg.double().cpu().numpy(), dg.sum(0), eg, "gate bias")
    R.check(dbu.double().cpu().numpy(), du.sum(0), eu, "up bias")
    assert torch.equal(cr.linear_gated_backward(dh, pre, *gate, *up, act=act, group=g, dx_add=add), dx)


@pytest.mark.parametrize("M,K,F", [(1, 64, 64), (12, 512, 1344), (100, 2688, 1024), (260, 320, 640), (1, 5120, 2560),
                                   (1728, 64, 4864), (3328, 384, 5120), (2752, 3008, 1536)])
def test_training_step(cr, M, K, F):
    """Forward with saved pre-activations, then the backward pass: one call is the two calls, and the
    chain is the formula's."""
    P.say("training step M=%d K=%d F=%d" % (M, K, F))
    g, gh = cr.dynamic_group(K), cr.dynamic_group(F)
    gate, up, down = _weight(cr, F, K, g, 1), _weight(cr, F, K, g, 2), _weight(cr, K, F, gh, 3)
    x, dy = _randn(M, K, seed=4), _randn(M, K, seed=5)
    y, pre = cr.ffn_gated(x, *gate, *up, *down, residual=x, group=g, group_h=gh, save_pre=True)
    dx, dbg, dbu, dbd = cr.ffn_gated_backward(dy, pre, *gate, *up, *down, group=g, group_h=gh, dx_add=dy, bias_grad=True)
    dh, dbd2 = cr.linear_act_backward(dy, *down, group=gh, bias_grad=True)
    dx2, dbg2, dbu2 = cr.linear_gated_backward(dh, pre, *gate, *up, group=g, dx_add=dy, bias_grad=True)
    for a, b in ((dx, dx2), (dbg, dbg2), (dbu, dbu2), (dbd, dbd2)):
        assert torch.equal(a, b)
    assert torch.equal(cr.ffn_gated_backward(dy, pre, *gate, *up, *down, group=g, group_h=gh, dx_add=dy), dx)
    d = R.rotate((_np(dy) * _np(down[1])) @ _np(down[0]), gh)
    _norm_check(_np(dh), d, "dh")
    gz, u = _np(pre[0]), _np(pre[1])
    dg, du = d * u * R.act_slope(gz, "silu"), d * R.act(gz, "silu")
    inner = R.rotate((dg * _np(gate[1])) @ _np(gate[0]) + (du * _np(up[1])) @ _np(up[0]), g)
    # dh's own error (0.82 of 2^-8) passes through the second product next to that one's
    _norm_check(_np(dx) - _np(dy), inner, "dx", 2 * R.BF16 * (1 + np.linalg.norm(_np(dy)) / np.linalg.norm(inner)))


@pytest.mark.parametrize("op", ["linear", "gated"])
def test_against_differences_of_the_forward(cr, op):
    """<c, f(x + e v) - f(x - e v)> / 2 e = <dx, v> with v along dx.  The forward's token quantization
    moves each x by at most half a step (0.02 here, independent, mean 0) against 2 e |v| = 0.1 sqrt(K)
    per token: 0.5%.  Curvature: the z move by about 0.1, error about 0.1^2 / 2: 0.5%.  y's rounding averages
    out.  Held to 2%."""
    M, N, K, e = 64, 512, 1024, 0.05
    a, b = _weight(cr, N, K, 256, 1), _weight(cr, N, K, 256, 2)
    x, c = _randn(M, K, seed=1, dtype=torch.float32), _randn(M, N, seed=2)
    if op == "linear":
        f = lambda t: cr.linear_act(t, *a, act="gelu")
        _, pre = cr.linear_act(x, *a, act="gelu", save_pre=True)
        dx, _ = cr.linear_act_backward(c, *a, pre=pre, act="gelu")
    else:
        f = lambda t: cr.linear_gated(t, *a, *b, act="silu")
        _, pre = cr.linear_gated(x, *a, *b, act="silu", save_pre=True)
        dx = cr.linear_gated_backward(c, pre, *a, *b, act="silu")
    v = dx.float() / dx.float().pow(2).mean(1, keepdim=True).sqrt()
    slope = ((f(x + e * v).double() - f(x - e * v).double()) * c.double()).sum() / (2 * e)
    want = (dx.double() * v.double()).sum()
    assert abs(slope.item() / want.item() - 1) < 0.02, (slope.item(), want.item())


def test_reference_slopes_against_differences():
    z = np.linspace(-6, 6, 241) + 0.013
    for act in R.ACTS:
        diff = (R.act(z + 1e-5, act) - R.act(z - 1e-5, act)) / 2e-5
        assert np.abs(diff - R.act_slope(z, act)).max() < 1e-8, act


def test_empty_batch_and_no_channels(cr):
    gate, up, down = _weight(cr, 128, 64, 64, 1), _weight(cr, 128, 64, 64, 2), _weight(cr, 64, 128, 128, 3)
    dy = torch.empty((0, 128), dtype=torch.bfloat16, device=DEV)
    dx, db = cr.linear_act_backward(dy, *gate, group=64, bias_grad=True)
    assert dx.shape == (0, 64) and torch.equal(db, torch.zeros(128, device=DEV))
    out = cr.ffn_gated_backward(dx, torch.empty((2, 0, 128), dtype=torch.bfloat16, device=DEV), *gate, *up, *down,
                                group=64, group_h=128, bias_grad=True)
    assert out[0].shape == (0, 64) and all(not t.any() for t in out[1:])
    with pytest.raises(cr.ConvRotError, match="SHAPE"):
        none = (torch.empty((0, 64), dtype=torch.int8, device=DEV), torch.empty(0, device=DEV))
        cr.linear_act_backward(torch.empty((3, 0), dtype=torch.bfloat16, device=DEV), *none, group=64)


def test_offsets_past_32_bits(cr):
    """dy and the operand hold more than 2^31 elements; the last tokens are checked against the same tokens alone
    (another tile choice: equal up to the order of fp32 sums)."""
    M, N, K = 2100, 1048568, 64
    wq = torch.randint(-127, 128, (N, K), dtype=torch.int8, device=DEV)
    ws = torch.rand(N, device=DEV) * 1e-3
    dy = torch.randn(M, N, device=DEV, dtype=torch.bfloat16)
    dx, db = cr.linear_act_backward(dy, wq, ws, group=64, bias_grad=True)
    few, _ = cr.linear_act_backward(dy[-5:].clone(), wq, ws, group=64)
    _norm_check(_np(dx[-5:]), _np(few), "last tokens", 2 * R.BF16)
    cols = dy[:, -8:].double().sum(0)
    bound = (M + 8) * R.U * dy[:, -8:].double().abs().sum(0)
    assert ((db[-8:].double() - cols).abs() <= bound).all()


def test_extreme_gradients(cr):
    """Gradients near both ends of the range the operand is carried in, and rows of zeros between them."""
    M, N, K = 70, 200, 256
    wq, ws = _weight(cr, N, K, 256, 1)
    for scale in (1e-15, 1e-8, 1e8, 1e15):
        dy = (_randn(M, N, seed=3, dtype=torch.float32) * scale).bfloat16()
        dy[::3] = 0
        dx, _ = cr.linear_act_backward(dy, wq, ws)
        ref = R.rotate(_np((dy.float() * ws).bfloat16()) @ _np(wq), 256)
        _norm_check(_np(dx), ref, "dx at %g" % scale)
        assert not dx[::3].any()


def test_streams_and_graph(cr):
    """Two backward calls at once on two streams, and one captured: replays follow their inputs."""
    M, K, F = 70, 512, 1024
    gate, up, down = _weight(cr, F, K, 256, 1), _weight(cr, F, K, 256, 2), _weight(cr, K, F, 256, 3)
    dy, pre = _randn(M, K, seed=1), _randn(2, M, F, seed=2)
    run = lambda d: cr.ffn_gated_backward(d, pre, *gate, *up, *down, dx_add=d, bias_grad=True)
    dy2 = _randn(M, K, seed=9)
    refs = run(dy), run(dy2)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s, d in zip(streams, (dy, dy2)):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(run(d))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(got, refs):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured = run(dy)
    for i in range(4):
        dy.copy_(_randn(M, K, seed=20 + i))
        graph.replay()
        eager = run(dy)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(captured, eager)), "replay %d" % i


def test_binding_refusals(cr):
    wq, ws = _weight(cr, 128, 64, 64, 1)
    dy = _randn(4, 128, seed=1)
    with pytest.raises(cr.ConvRotError, match="NULL"):
        cr.linear_act_backward(dy, wq, ws, act="silu", group=64)              # no pre
    with pytest.raises(ValueError, match="dy has shape"):
        cr.linear_act_backward(_randn(4, 64, seed=1), wq, ws, group=64)
    with pytest.raises(TypeError, match="dy"):
        cr.linear_act_backward(dy.float(), wq, ws, group=64)
    with pytest.raises(ValueError, match="pre has shape"):
        cr.linear_gated_backward(dy, dy, wq, ws, wq, ws, group=64)
    with pytest.raises(cr.ConvRotError, match="OVERLAP"):
        buf = _randn(5, 64, seed=1)
        cr.linear_act_backward(dy, wq, ws, group=64, dx_add=buf[:4], out=buf[1:])
