"""The fused forward linears against their definition in 64 bits: activation, residual, saved
pre-activations, gate|up product, feed-forward block.

The references start from the kernels' own INT8 codes and scales (held to the oracle by
test_gpu_parity.py), so what is left is the epilogue's fp32 arithmetic and one bf16 rounding; the
bounds are derived in fused_reference.py."""
import itertools

import numpy as np
import pytest
import torch

from int4_quantized_linear_amd import workloads
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
    return t.detach().float().cpu().numpy() if t.dtype == torch.bfloat16 else t.detach().cpu().numpy()


def _weight(cr, N, K, g, seed):
    gen = torch.Generator().manual_seed(seed)
    w = (torch.randn(N, K, generator=gen) * 0.05).bfloat16().to(DEV)
    return cr.prepare_weight(w, g, 8)


def _tokens(M, K, seed, dtype=torch.bfloat16):
    gen = torch.Generator().manual_seed(1000 + seed)
    return torch.randn(M, K, generator=gen).to(dtype).to(DEV)


def _randn(*shape, seed, std=1.0, dtype=torch.bfloat16):
    gen = torch.Generator().manual_seed(2000 + seed)
    return (torch.randn(*shape, generator=gen) * std).to(dtype).to(DEV)


# M: the GEMV's ends, its border to the GEMM, one and several row tiles; N: below a fragment, ragged
# (element stores), a multiple of 8, past a column tile; K and its group
SHAPES = [(1, 1, 64, 64), (2, 7, 320, 64), (12, 520, 512, 256), (15, 4100, 256, 256), (16, 264, 1024, 256),
          (16, 16400, 256, 256), (17, 264, 1024, 256), (17, 33, 320, 64), (130, 1001, 2688, 128),
          (257, 520, 192, 64), (300, 1000, 4096, 256), (513, 264, 640, 128)]


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("M,N,K,g", SHAPES)
def test_linear_act(cr, M, N, K, g, act):
    P.say("linear_act M=%d N=%d K=%d g=%d %s" % (M, N, K, g, act))
    x, (wq, ws) = _tokens(M, K, M + N), _weight(cr, N, K, g, N + K)
    x[M // 2] = 0                                             # a token with scale 0: z is the bias
    b, r = _randn(N, seed=N, dtype=torch.float32), _randn(M, N, seed=M, std=3.0)
    xq, xs = cr.quantize_act(x, g, 8)
    for bias, res, save in itertools.product((None, b), (None, r), (False, True)):
        got = cr.linear_act(x, wq, ws, bias, act=act, residual=res, group=g, save_pre=save)
        y, pre = got if save else (got, None)
        torch.cuda.synchronize()
        z, dz = R.linear_z(_np(xq), _np(xs), _np(wq), _np(ws), None if bias is None else _np(bias))
        a, da = R.act_bound(z, dz, act)
        ref = a + (0.0 if res is None else _np(res).astype(np.float64))
        R.check(_np(y), ref, R.rounded(ref, da + R.U * np.abs(ref)), "y")
        if save:
            R.check(_np(pre), z, R.rounded(z, dz), "pre")
            again = cr.linear_act(None, wq, ws, bias, act=act, residual=res, group=g, xq=xq, x_scale=xs)
            assert torch.equal(again, y), "pre-quantized tokens, or not saving, change the result"
        if res is not None:
            place = res.clone()
            assert cr.linear_act(x, wq, ws, bias, act=act, residual=place, group=g, out=place) is place
            assert torch.equal(place, y), "adding in place differs"


@pytest.mark.parametrize("M,N,K,g", SHAPES)
def test_linear_act_none_is_linear(cr, M, N, K, g):
    x, (wq, ws) = _tokens(M, K, 7, torch.float32), _weight(cr, N, K, g, 8)
    b = _randn(N, seed=3, dtype=torch.float32)
    assert torch.equal(cr.linear_act(x, wq, ws, b, group=g), cr.linear(x, wq, ws, b, group=g))


GATED = [(1, 1, 64, 64), (3, 9, 320, 64), (12, 520, 512, 256), (16, 8200, 256, 256), (17, 264, 1024, 256),
         (40, 33, 320, 64), (130, 1001, 2688, 128), (257, 136, 192, 64), (300, 504, 4096, 256), (513, 392, 640, 128)]


def _gated_reference(xq, xs, gate, up, bg, bu, act):
    n = lambda t: None if t is None else _np(t)
    g, dg = R.linear_z(_np(xq), _np(xs), _np(gate[0]), _np(gate[1]), n(bg))
    u, du = R.linear_z(_np(xq), _np(xs), _np(up[0]), _np(up[1]), n(bu))
    a, da = R.act_bound(g, dg, act)
    h = a * u
    return g, dg, u, du, h, da * np.abs(u) + (np.abs(a) + da) * du + R.U * np.abs(h)


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("M,N,K,g", GATED)
def test_linear_gated(cr, M, N, K, g, act):
    P.say("linear_gated M=%d N=%d K=%d g=%d %s" % (M, N, K, g, act))
    x = _tokens(M, K, M + N)
    gate, up = _weight(cr, N, K, g, N + K), _weight(cr, N, K, g, N + K + 1)
    bg, bu = _randn(N, seed=1, dtype=torch.float32), _randn(N, seed=2, dtype=torch.float32)
    xq, xs = cr.quantize_act(x, g, 8)
    for b1, b2 in ((None, None), (bg, bu), (bg, None), (None, bu)):
        h, pre = cr.linear_gated(x, *gate, *up, b1, b2, act=act, group=g, save_pre=True)
        torch.cuda.synchronize()
        gr, dg, ur, du, hr, dh = _gated_reference(xq, xs, gate, up, b1, b2, act)
        R.check(_np(h), hr, R.rounded(hr, dh), "h")
        R.check(_np(pre[0]), gr, R.rounded(gr, dg), "gate")
        R.check(_np(pre[1]), ur, R.rounded(ur, du), "up")
        alone = cr.linear_gated(None, *gate, *up, b1, b2, act=act, group=g, xq=xq, x_scale=xs)
        assert torch.equal(alone, h), "pre-quantized tokens, or not saving, change the result"


# Every choice of tiles and slices of K gives the same bits: with a workspace the call slices where that
# is faster, without one it runs whole.  The sizes cover 64- and 128-token tiles, sliced and whole, 256 x 256
# tiles with and without a sliced tail, and ragged N on each.  A token's outputs do not depend on the
# others, so a few tokens alone (other tiles) have to give the same bits too.
@pytest.mark.parametrize("M,N,K", [(64, 4096, 5120), (300, 504, 4096), (17, 264, 1024), (2048, 512, 5120), (100, 41, 8192),
                                   (130, 3000, 4096), (640, 2049, 2112), (1500, 2056, 1024), (1400, 8200, 576),
                                   (3328, 3736, 512), (3328, 3737, 512), (1792, 3488, 512), (2304, 7208, 2048),
                                   (1536, 5472, 1536)])
def test_tiles_and_slices_are_bit_identical(cr, M, N, K):
    P.say("tiles and slices M=%d N=%d K=%d" % (M, N, K))
    g = cr.dynamic_group(K)
    x, gate, up = _tokens(M, K, 5), _weight(cr, N, K, g, 1), _weight(cr, N, K, g, 2)
    xq, xs = cr.quantize_act(x, g, 8)
    r = _randn(M, N, seed=6)
    st = torch.cuda.current_stream().cuda_stream
    y = cr.linear_act(x, gate[0], gate[1], act="gelu", residual=r, group=g)
    h, pre = cr.linear_gated(x, *gate, *up, act="silu", group=g, save_pre=True)
    y2, h2, pre2 = torch.empty_like(y), torch.empty_like(h), torch.empty_like(pre)
    ptr = cr._ptr
    cr._call("convrot_linear_act", None, 0, ptr(xq), ptr(xs), M, N, K, g, ptr(gate[0]), ptr(gate[1]), None, 3, ptr(r),
             None, ptr(y2), None, 0, st)
    cr._call("convrot_linear_gated", None, 0, ptr(xq), ptr(xs), M, N, K, g, ptr(gate[0]), ptr(gate[1]), None,
             ptr(up[0]), ptr(up[1]), None, 2, ptr(pre2), ptr(h2), None, 0, st)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(h, h2) and torch.equal(pre, pre2)
    for a, b in ((0, min(M, 77)), (max(0, M - 5), M)):
        q = dict(group=g, xq=xq[a:b].clone(), x_scale=xs[a:b].clone())
        assert torch.equal(cr.linear_act(None, *gate, act="gelu", residual=r[a:b].clone(), **q), y[a:b])
        assert torch.equal(cr.linear_gated(None, *gate, *up, act="silu", **q), h[a:b])


@pytest.mark.parametrize("M,K,F,dtype", [(1, 64, 64, torch.bfloat16), (1, 5120, 2560, torch.bfloat16),
                                         (12, 512, 1344, torch.float32), (16, 320, 192, torch.bfloat16),
                                         (17, 320, 192, torch.float32), (100, 2688, 5376, torch.bfloat16),
                                         (300, 1024, 2048, torch.bfloat16)])
def test_ffn_gated(cr, M, K, F, dtype):
    P.say("ffn_gated M=%d K=%d F=%d %s" % (M, K, F, dtype))
    g, gh = cr.dynamic_group(K), cr.dynamic_group(F)
    x = _tokens(M, K, M, dtype)
    gate, up, down = _weight(cr, F, K, g, 1), _weight(cr, F, K, g, 2), _weight(cr, K, F, gh, 3)
    bd, r = _randn(K, seed=4, dtype=torch.float32), _randn(M, K, seed=5)
    y, pre = cr.ffn_gated(x, *gate, *up, *down, bias_down=bd, residual=r, group=g, group_h=gh, save_pre=True)
    # one call is the two calls
    h, pre2 = cr.linear_gated(x, *gate, *up, group=g, save_pre=True)
    y2 = cr.linear_act(h, *down, bd, residual=r, group=gh)
    assert torch.equal(y, y2) and torch.equal(pre, pre2)
    place = r.clone()
    cr.ffn_gated(x, *gate, *up, *down, bias_down=bd, residual=place, group=g, group_h=gh, out=place)
    assert torch.equal(place, y)
    # and the definition, from the codes of x and h
    (xq, xs), (hq, hs) = cr.quantize_act(x, g, 8), cr.quantize_act(h, gh, 8)
    _, _, _, _, hr, dh = _gated_reference(xq, xs, gate, up, None, None, "silu")
    R.check(_np(h), hr, R.rounded(hr, dh), "h")
    z, dz = R.linear_z(_np(hq), _np(hs), _np(down[0]), _np(down[1]), _np(bd))
    ref = z + _np(r)
    R.check(_np(y), ref, R.rounded(ref, dz + R.U * np.abs(ref)), "y")


def test_large_and_extreme_values(cr):
    """Pre-activations far out on both sides: no overflow of an exponential or of z^3 may reach y."""
    M, N, K = 18, 264, 256
    x = torch.zeros(M, K, device=DEV)
    wq, ws = _weight(cr, N, K, 256, 3)
    b = torch.logspace(-30, 30, N // 2, device=DEV)
    b = torch.cat([b, -b])
    for act in R.ACTS:
        for m in (M, 4):
            y = cr.linear_act(x[:m].contiguous(), wq, ws, b, act=act)
            a, da = R.act_bound(_np(b).astype(np.float64), 0.0, act)
            ref, bound = np.broadcast_to(a, (m, N)), np.broadcast_to(R.rounded(a, da), (m, N))
            R.check(_np(y), ref, bound, act)


def test_infinite_and_nan_preactivations(cr):
    """A bias of -inf, of fp32's lowest number or of +inf gives the activation's limit there, and a NaN stays one; the
    other channels are not touched."""
    N, K = 264, 256
    (wq, ws), (up, us) = _weight(cr, N, K, 256, 3), _weight(cr, N, K, 256, 4)
    b = torch.zeros(N, device=DEV)
    b[0], b[9], b[18], b[27] = -torch.inf, torch.finfo(torch.float32).min, torch.inf, torch.nan
    rest = [n for n in range(N) if n not in (0, 9, 18, 27)]
    for m in (4, 40):
        x = _tokens(m, K, m)
        for act in R.ACTS[1:]:
            y, pre = cr.linear_act(x, wq, ws, b, act=act, save_pre=True)
            plain = cr.linear_act(x, wq, ws, act=act)
            assert (y[:, 0] == 0).all() and (y[:, 9] == 0).all() and (y[:, 18] == torch.inf).all(), act
            assert y[:, 27].isnan().all() and pre[:, 27].isnan().all(), act
            assert torch.equal(y[:, rest], plain[:, rest]), act
            h = cr.linear_gated(x, wq, ws, up, us, b, act=act)
            assert (h[:, 0] == 0).all() and (h[:, 9] == 0).all() and h[:, 27].isnan().all(), act
            assert torch.equal(h[:, rest], cr.linear_gated(x, wq, ws, up, us, act=act)[:, rest]), act


def test_offsets_past_32_bits(cr):
    """More than 2^31 outputs, through the GEMM and through the decode kernel: the last columns and tokens against
    the same ones alone."""
    K = 64
    for M, N in ((300, 8000008), (16, 140000008)):
        wq = torch.randint(-127, 128, (N, K), dtype=torch.int8, device=DEV)
        ws = torch.rand(N, device=DEV) * 1e-3
        xq, xs = cr.quantize_act(_tokens(M, K, 1), 64, 8)
        y = cr.linear_act(None, wq, ws, act="silu", group=64, xq=xq, x_scale=xs)
        tail = cr.linear_act(None, wq[-264:].clone(), ws[-264:].clone(), act="silu", group=64, xq=xq, x_scale=xs)
        assert torch.equal(y[:, -264:], tail)
        h = cr.linear_gated(None, wq, ws, wq, ws, act="relu", group=64, xq=xq, x_scale=xs)
        tail = cr.linear_gated(None, wq[-264:].clone(), ws[-264:].clone(), wq[-264:].clone(), ws[-264:].clone(), act="relu",
                               group=64, xq=xq, x_scale=xs)
        assert torch.equal(h[:, -264:], tail)
        del y, h


def test_empty_batches(cr):
    gate, up, down = _weight(cr, 128, 64, 64, 1), _weight(cr, 128, 64, 64, 2), _weight(cr, 64, 128, 128, 3)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    assert cr.linear_act(x, *gate, group=64, act="silu").shape == (0, 128)
    assert cr.linear_gated(x, *gate, *up, group=64).shape == (0, 128)
    y, pre = cr.ffn_gated(x, *gate, *up, *down, group=64, group_h=128, save_pre=True)
    assert y.shape == (0, 64) and pre.shape == (2, 0, 128)
    none = (torch.empty((0, 64), dtype=torch.int8, device=DEV), torch.empty(0, device=DEV))
    assert cr.linear_act(_tokens(3, 64, 1), *none, group=64).shape == (3, 0)


def test_other_stream_and_graph(cr):
    """The block on a side stream, and captured: every replay gives the eager result on its inputs."""
    M, K, F = 40, 512, 1024
    gate, up, down = _weight(cr, F, K, 256, 1), _weight(cr, F, K, 256, 2), _weight(cr, K, F, 256, 3)
    x, r = _tokens(M, K, 1), _randn(M, K, seed=2)
    ref = cr.ffn_gated(x, *gate, *up, *down, residual=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = cr.ffn_gated(x, *gate, *up, *down, residual=r)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, ref)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured = cr.ffn_gated(x, *gate, *up, *down, residual=r)
    for i in range(4):
        x.copy_(_tokens(M, K, 10 + i))
        graph.replay()
        eager = cr.ffn_gated(x, *gate, *up, *down, residual=r)
        torch.cuda.synchronize()
        assert torch.equal(captured, eager), "replay %d" % i


def test_binding_refusals(cr):
    (wq, ws), x = _weight(cr, 128, 64, 64, 1), _tokens(4, 64, 1)
    with pytest.raises(ValueError, match="act"):
        cr.linear_act(x, wq, ws, group=64, act="tanh")
    with pytest.raises(ValueError, match="residual has shape"):
        cr.linear_act(x, wq, ws, group=64, residual=_randn(4, 64, seed=1))
    with pytest.raises(TypeError, match="residual"):
        cr.linear_act(x, wq, ws, group=64, residual=torch.zeros(4, 128, device=DEV))
    with pytest.raises(ValueError, match="contiguous"):
        cr.linear_act(x, wq, ws, group=64, residual=_randn(128, 4, seed=1).t())
    with pytest.raises(ValueError, match="is on cpu"):
        cr.linear_act(x.cpu(), wq, ws, group=64)
    with pytest.raises(ValueError, match="wq_up has shape"):
        cr.linear_gated(x, wq, ws, wq[:64].contiguous(), ws[:64].contiguous(), group=64)
    with pytest.raises(ValueError, match="wq_down has shape"):
        cr.ffn_gated(x, wq, ws, wq, ws, wq, ws, group=64)
    with pytest.raises(cr.ConvRotError, match="OVERLAP"):
        buf = torch.zeros(5, 128, dtype=torch.bfloat16, device=DEV)
        cr.linear_act(x, wq, ws, group=64, residual=buf[:4], out=buf[1:])
