"""Products of grouped rows and the gated expert layer: bit for bit against the library's own linears run expert by expert
(the products are exact integer sums with the same epilogue), the weighted sum against 64 bits, gradients against their
formulas in 64 bits and against differences, and the whole chain as a training step runs it.

Bounds.  y: each d is within 3 u |acc sx sw| of its 64-bit value (linear_z); on its way to the sum it may be held in 16 bits with a
scale of max / 32767 per 64 channels, off by half a step, 2^-16 of that maximum; the sum of top terms and the residual in fp32
adds (top + 2) u of the sum of their magnitudes, then one bf16 rounding.
Grouped gradients: the operand bf16(dy sw) is reproduced exactly, so dx is off by fp32 sums alone: (N + 16) u of the sum of
absolute terms, then the bf16 rounding.
Layer gradients, 2-norm: four bf16 roundings (both operands, dh, dx), each uniform within 2^-8 of a value at most and
independent: 2^-8 / sqrt 3 each in the mean square, 2^-8 sqrt(4 / 3) together; held to 2 * 2^-8, since few terms spread
around the mean.  dweights: K products in fp32, (K + 8) u of the sum of their magnitudes."""
import numpy as np
import pytest
import torch

from tests import fused_reference as R
from tests import moe_reference as MR
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


def _weights(cr, E, N, K, g, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    w = (torch.randn(E * N, K, generator=gen, device=DEV) * 0.05).bfloat16()
    q, s = cr.prepare_weight(w, g, 8)
    return q.view(E, N, K), s.view(E, N)


def _randn(*shape, seed, std=1.0, dtype=torch.bfloat16):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * std).to(dtype).to(DEV)


def _offsets(counts, first=0):
    return torch.tensor([first] + list(first + np.cumsum(counts)), dtype=torch.int32, device=DEV)


# counts of the groups; N, K, group
GROUPED = [([1], 1, 64, 64), ([0, 0, 3, 0], 7, 320, 64), ([1] * 40, 264, 512, 256), ([16, 17, 0, 63, 64, 65], 33, 192, 64),
           ([130, 1, 0, 127, 128, 129], 520, 640, 128), ([600, 3, 300], 1001, 1024, 256), ([5, 0, 2] * 100, 96, 128, 128),
           ([1, 0] * 512, 40, 64, 2), ([300] * 9, 200, 2688, 128)]


# sizes that take tiles of 128 rows, and of 256 with a last round that is more and less than half full, whole and odd N, one
# K-tile and many, whole and half
LARGE_GROUPED = [([700, 1, 900, 130], 1408, 1088, 64), ([1041, 0, 257, 700, 5, 1500], 2688, 1088, 64), ([3000, 100, 5900], 2001, 64, 64),
                 ([1041, 0, 257, 700, 5, 1500], 2001, 1344, 64), ([3000, 100, 5900], 2688, 128, 128), ([513, 512, 511, 1], 5376, 192, 64)]


@pytest.mark.parametrize("counts,N,K,g", GROUPED + LARGE_GROUPED)
def test_linear_grouped(cr, counts, N, K, g):
    P.say("linear_grouped %d groups N=%d K=%d" % (len(counts), N, K))
    wq, ws = _weights(cr, len(counts), N, K, g, N + K)
    first, after = 3, 5                                          # rows of no group before and behind
    rows = first + sum(counts) + after
    offsets = _offsets(counts, first)
    for dtype in (torch.bfloat16, torch.float32):
        x = _randn(rows, K, seed=rows, dtype=dtype)
        x[rows // 2] = 0
        out = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device=DEV)
        assert cr.linear_grouped(x, wq, ws, offsets, group=g, out=out) is out
        at = first
        for e, n in enumerate(counts):
            if n:
                assert torch.equal(out[at:at + n], cr.linear(x[at:at + n].clone(), wq[e], ws[e], group=g)), (e, n)
            at += n
        assert (out[:first] == 7).all() and (out[at:] == 7).all(), "rows of no group were written"
        xq, xs = cr.quantize_act(x, g, 8)
        again = cr.linear_grouped(None, wq, ws, offsets, group=g, xq=xq, x_scale=xs)
        assert torch.equal(again[first:at], out[first:at])


def test_linear_grouped_all_rows_of_no_group(cr):
    wq, ws = _weights(cr, 3, 64, 64, 64, 1)
    x, out = _randn(9, 64, seed=1), torch.full((9, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    for offsets in ([0, 0, 0, 0], [9, 9, 9, 9], [4, 4, 4, 4]):
        o = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        cr.linear_grouped(x, wq, ws, o, group=64, out=out)
        cr.linear_grouped_backward(_randn(9, 64, seed=2), wq, ws, o, group=64, out=out)
        assert (out == 3).all()
    assert cr.linear_grouped(x[:0], wq, ws, o, group=64).shape == (0, 64)
    assert cr.linear_grouped_backward(x[:0], wq, ws, o, group=64).shape == (0, 64)


def test_linear_grouped_offsets_are_held_to_the_rows(cr):
    """Offsets outside the rows count as the nearer end; one below an earlier one as that one."""
    wq, ws = _weights(cr, 3, 64, 64, 64, 1)
    x, dy = _randn(20, 64, seed=1), _randn(20, 64, seed=2)
    want = torch.tensor([0, 5, 5, 20], dtype=torch.int32, device=DEV)
    for offsets in ([-5, 5, 5, 1 << 30], [-(1 << 31), 5, 5, (1 << 31) - 1], [0, 5, 5, 21]):
        o = torch.tensor(offsets, dtype=torch.int64).to(torch.int32).to(DEV)
        assert torch.equal(cr.linear_grouped(x, wq, ws, o, group=64), cr.linear_grouped(x, wq, ws, want, group=64))
        assert torch.equal(cr.linear_grouped_backward(dy, wq, ws, o, group=64),
                           cr.linear_grouped_backward(dy, wq, ws, want, group=64))
    o = torch.tensor([8, 3, 3, 20], dtype=torch.int32, device=DEV)    # groups 0 and 1 are empty, rows 0 .. 7 belong to none
    for call, v in ((cr.linear_grouped, x), (cr.linear_grouped_backward, dy)):
        out = torch.full((20, 64), 3.0, dtype=torch.bfloat16, device=DEV)
        call(v, wq, ws, o, group=64, out=out)
        want = call(v, wq, ws, torch.tensor([8, 8, 8, 20], dtype=torch.int32, device=DEV), group=64)
        assert (out[:8] == 3).all() and torch.equal(out[8:], want[8:])


@pytest.mark.parametrize("counts,N,K,g", GROUPED + [([257, 0, 700, 256], 72, 1280, 256), ([1024, 511], 321, 512, 32),
                                                    ([300, 1], 264, 192, 1), ([3000, 100, 5900], 65, 1344, 64), ([4097], 1001, 2688, 128)])
def test_linear_grouped_backward(cr, counts, N, K, g):
    P.say("linear_grouped_backward %d groups N=%d K=%d" % (len(counts), N, K))
    wq, ws = _weights(cr, len(counts), N, K, g, N + K)
    first, after = 2, 4
    rows = first + sum(counts) + after
    offsets = _offsets(counts, first)
    dy, add = _randn(rows, N, seed=rows, std=1e-3), _randn(rows, K, seed=rows + 1, std=1e-3)
    dy[rows // 2] = 0
    out = torch.full((rows, K), 7.0, dtype=torch.bfloat16, device=DEV)
    cr.linear_grouped_backward(dy, wq, ws, offsets, group=g, out=out)
    place = add.clone()
    assert cr.linear_grouped_backward(dy, wq, ws, offsets, group=g, dx_add=place, out=place) is place
    at = first
    for e, n in enumerate(counts):
        if n:
            a, q = _np((dy[at:at + n].float() * ws[e]).bfloat16()), _np(wq[e])
            ref = R.rotate(a @ q, g)
            bound = (N + 16) * R.U * R.rotate_abs(np.abs(a) @ np.abs(q), g)
            R.check(_np(out[at:at + n]), ref, R.rounded(ref, bound), "dx of group %d" % e)
            ref2 = ref + _np(add[at:at + n])
            R.check(_np(place[at:at + n]), ref2, R.rounded(ref2, bound + R.U * np.abs(ref2)), "dx + add of group %d" % e)
        at += n
    assert (out[:first] == 7).all() and (out[at:] == 7).all(), "rows of no group were written"
    assert torch.equal(place[:first], add[:first]) and torch.equal(place[at:], add[at:])
    again = torch.full_like(out, 7.0)
    cr.linear_grouped_backward(dy, wq, ws, offsets, group=g, out=again)
    assert torch.equal(again, out)


def _experts(M, top, E, seed, kind="mixed"):
    gen = torch.Generator().manual_seed(seed)
    e = torch.stack([torch.randperm(E, generator=gen)[:top] for _ in range(M)]).to(torch.int32)
    if kind == "one":                                            # every token takes the same experts
        e[:] = e[0]
    if kind == "twice" and top > 1:
        e[:, 1] = e[:, 0]
    if kind == "dropped":
        e[torch.rand(M, top, generator=gen) < 0.4] = -1
        e[M // 2] = torch.tensor([-1, E, -7, 1 << 30] * top, dtype=torch.int32)[:top]
    if kind == "none":
        e[:] = -1
    w = torch.rand(M, top, generator=gen) + 0.05
    return e.to(DEV), w.to(DEV)


# M, top, E, F, K, group_h, group, experts
LAYERS = [(1, 1, 1, 64, 64, 64, 64, "mixed"), (1, 8, 64, 256, 512, 256, 256, "mixed"), (1, 1, 4, 128, 320, 128, 64, "none"),
          (2, 3, 5, 192, 64, 64, 64, "twice"), (5, 4, 6, 320, 256, 64, 256, "dropped"), (7, 32, 40, 64, 192, 64, 64, "mixed"),
          (16, 2, 1024, 64, 64, 64, 64, "mixed"), (17, 2, 3, 1344, 576, 64, 64, "mixed"), (40, 8, 8, 512, 1024, 256, 256, "twice"),
          (64, 2, 9, 704, 512, 64, 256, "one"), (130, 4, 7, 192, 2688, 64, 128, "dropped"), (301, 3, 16, 448, 640, 64, 128, "mixed"),
          (700, 1, 3, 256, 320, 256, 64, "mixed"), (333, 6, 12, 384, 256, 128, 256, "one"), (1200, 2, 4, 128, 192, 128, 64, "dropped")]


# the same for layers: tiles of 128 and 256 rows in the first, the second or both products
LARGE_LAYERS = [(901, 3, 3, 1088, 1344, 64, 64, "mixed"), (2100, 2, 4, 1344, 4096, 64, 256, "dropped"), (4000, 2, 3, 1344, 64, 64, 64, "twice"),
                (1500, 3, 5, 2112, 1024, 64, 256, "mixed"), (2100, 2, 4, 1344, 2688, 64, 128, "one")]


def _layer(cr, E, F, K, gh, g, seed=1):
    return _weights(cr, E, F, K, g, seed), _weights(cr, E, F, K, g, seed + 1), _weights(cr, E, K, F, gh, seed + 2)


def _expert_by_expert(cr, x, experts, gate, up, down, act, g, gh):
    """(pre, d as bf16, d in 64 bits, its bound) of every slot, through the library's dense linears."""
    M, top = experts.shape
    E, F, K = gate[0].shape
    pre = torch.zeros(2, M, top, F, dtype=torch.bfloat16, device=DEV)
    d = torch.zeros(M, top, K, dtype=torch.bfloat16, device=DEV)
    d64, bound = np.zeros((M, top, K)), np.zeros((M, top, K))
    for e in range(E):
        t, j = torch.nonzero(experts == e, as_tuple=True)
        if not len(t):
            continue
        h, p = cr.linear_gated(x[t].contiguous(), gate[0][e], gate[1][e], up[0][e], up[1][e], act=act, group=g, save_pre=True)
        pre[:, t, j] = p
        d[t, j] = cr.linear(h, down[0][e], down[1][e], group=gh)
        hq, hs = cr.quantize_act(h, gh, 8)
        at = (t.cpu().numpy(), j.cpu().numpy())
        d64[at], bound[at] = R.linear_z(_np(hq), _np(hs), _np(down[0][e]), _np(down[1][e]), None)
    return pre, d, d64, bound


@pytest.mark.parametrize("M,top,E,F,K,gh,g,kind", LAYERS + LARGE_LAYERS)
def test_moe_ffn_gated(cr, M, top, E, F, K, gh, g, kind):
    P.say("moe_ffn_gated M=%d top=%d E=%d F=%d K=%d %s" % (M, top, E, F, K, kind))
    gate, up, down = _layer(cr, E, F, K, gh, g)
    experts, w = _experts(M, top, E, M + top, kind)
    acts = R.ACTS if M in (5, 130) else ("silu",)
    for act in acts:
        for dtype in (torch.bfloat16, torch.float32):
            x, res = _randn(M, K, seed=M, dtype=dtype), _randn(M, K, seed=M + 1, std=0.5)
            x[M // 2] = 0
            call = dict(act=act, group=g, group_h=gh)
            y, pre, d = cr.moe_ffn_gated(x, experts, w, *gate, *up, *down, residual=res, save=True, **call)
            want_pre, want_d, d64, dd = _expert_by_expert(cr, x, experts, gate, up, down, act, g, gh)
            ok = ((experts >= 0) & (experts < E))
            assert torch.equal(pre[:, ok], want_pre[:, ok]), "pre"
            assert torch.equal(d[ok], want_d[ok]), "d"
            wn = _np(w)[:, :, None]
            ref = (d64 * wn).sum(1) + _np(res)
            size = (np.abs(d64) * wn).sum(1) + np.abs(_np(res))
            held = np.repeat(np.abs(d64).reshape(M, top, K // 64, 64).max(3), 64, 2) * (2.0 ** -16 * (1 + 8 * R.U))
            bound = ((dd + held) * wn).sum(1) + (top + 2) * R.U * size
            R.check(_np(y), ref, R.rounded(ref, bound), "y")
            assert torch.equal(cr.moe_ffn_gated(x, experts, w, *gate, *up, *down, residual=res, **call), y), "not saving"
            place = res.clone()
            assert cr.moe_ffn_gated(x, experts, w, *gate, *up, *down, residual=place, out=place, **call) is place
            assert torch.equal(place, y), "adding in place"
            alone = cr.moe_ffn_gated(x, experts, w, *gate, *up, *down, **call)
            ref = (d64 * wn).sum(1)
            R.check(_np(alone), ref, R.rounded(ref, bound), "y without residual")
            if not ok[M // 2].any():
                assert torch.equal(y[M // 2], res[M // 2])


FEW = [(1, 8, 64), (2, 8, 16), (3, 4, 4), (2, 32, 40), (8, 8, 64), (16, 4, 24), (13, 1, 3), (64, 1, 5), (32, 2, 2), (21, 3, 700), (65, 1, 4)]


@pytest.mark.parametrize("kind", ["mixed", "twice", "one", "dropped", "none"])
@pytest.mark.parametrize("M,top,E", FEW)
def test_moe_ffn_gated_few_slots(cr, M, top, E, kind):
    """At most 64 slots take kernels of their own, here against the dense linears.  The rotation groups go through all sizes,
    the widths through whole and part 256-channel pieces and more pieces than wavefronts."""
    experts, w = _experts(M, top, E, M + top, kind)
    for i, (F, K, gh, g) in enumerate([(64, 64, 1, 2), (128, 320, 4, 8), (192, 1088, 16, 32), (320, 2688, 64, 128), (2304, 512, 256, 256)]):
        if E > 100 and i != M % 5:
            continue
        P.say("moe few M=%d top=%d E=%d F=%d K=%d %s" % (M, top, E, F, K, kind))
        gate, up, down = _layer(cr, E, F, K, gh, g)
        for dtype in (torch.bfloat16, torch.float32):
            x, res = _randn(M, K, seed=M + i, dtype=dtype), _randn(M, K, seed=M + 1, std=0.5)
            x[M // 2] *= 1e-37 if dtype is torch.float32 else 1.0
            x[M // 3] = 0
            call = dict(act=R.ACTS[i % 5], group=g, group_h=gh)
            ok, wn = (experts >= 0) & (experts < E), _np(w)[:, :, None]
            want_pre, want_d, d64, dd = _expert_by_expert(cr, x, experts, gate, up, down, call["act"], g, gh)
            held = np.repeat(np.abs(d64).reshape(M, top, K // 64, 64).max(3), 64, 2) * (2.0 ** -16 * (1 + 8 * R.U))
            if M * top <= 64:
                held = 0.0                                       # nothing between the product and the sum
            for r in (res, None):
                y, pre, d = cr.moe_ffn_gated(x, experts, w, *gate, *up, *down, residual=r, save=True, **call)
                assert torch.equal(pre[:, ok], want_pre[:, ok]) and torch.equal(d[ok], want_d[ok])
                add = 0.0 if r is None else _np(r)
                ref = (d64 * wn).sum(1) + add
                bound = ((dd + held) * wn).sum(1) + (top + 2) * R.U * ((np.abs(d64) * wn).sum(1) + np.abs(add))
                R.check(_np(y), ref, R.rounded(ref, bound), "y")
                assert torch.equal(cr.moe_ffn_gated(x, experts, w, *gate, *up, *down, residual=r, **call), y), "not saving"
        place = x.bfloat16()                                     # y in the place of x
        want = cr.moe_ffn_gated(place, experts, w, *gate, *up, *down, residual=res, save=True, **call)[0]
        assert cr.moe_ffn_gated(place, experts, w, *gate, *up, *down, residual=res, out=place, **call) is place
        assert torch.equal(place, want)


def test_moe_ffn_gated_keeps_rows_without_an_expert(cr):
    """pre and d of slots without an expert are left as they were."""
    M, top, E, F, K = 20, 3, 4, 64, 128
    gate, up, down = _layer(cr, E, F, K, 64, 128)
    experts, w = _experts(M, top, E, 3, "dropped")
    x = _randn(M, K, seed=1)
    pre = torch.full((2, M, top, F), 5.0, dtype=torch.bfloat16, device=DEV)
    d = torch.full((M, top, K), 5.0, dtype=torch.bfloat16, device=DEV)
    y = torch.empty(M, K, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(cr.workspace_bytes_moe_ffn(M, top, E, F, K), dtype=torch.uint8, device=DEV)
    p = lambda t: t.data_ptr()
    cr._call("convrot_moe_ffn_gated", p(x), 1, p(experts), p(w), M, top, E, F, K, 128, 64, p(gate[0]), p(gate[1]), p(up[0]),
             p(up[1]), p(down[0]), p(down[1]), cr.ACTS["silu"], None, p(pre), p(d), p(y), p(ws), ws.numel(),
             torch.cuda.current_stream().cuda_stream)
    none = (experts < 0) | (experts >= E)
    assert none.any() and (pre[:, none] == 5).all() and (d[none] == 5).all()
    assert not (pre[:, ~none] == 5).all(-1).any()


def test_moe_ffn_gated_extremes(cr):
    """Weights of 0, negative and very large router weights; a token whose hidden channels are all zero; infinite
    router weights reach their own tokens only."""
    M, top, E, F, K = 9, 2, 4, 64, 64
    gate, up, down = _layer(cr, E, F, K, 64, 64)
    experts, w = _experts(M, top, E, 3)
    w[0], w[1], w[2], w[3, 0] = 0.0, -1.0, 1e30, torch.inf
    x = _randn(M, K, seed=1)
    x[4] = 0
    y = cr.moe_ffn_gated(x, experts, w, *gate, *up, *down, group=64, group_h=64)
    _, _, d64, _ = _expert_by_expert(cr, x, experts, gate, up, down, "silu", 64, 64)
    ref = (d64 * _np(w)[:, :, None]).sum(1)
    assert (y[0] == 0).all() and (y[4] == 0).all() and not torch.isfinite(y[3]).all()
    for m in (1, 2, 5, 6, 7, 8):
        assert np.linalg.norm(_np(y[m]) - ref[m]) <= R.BF16 * np.linalg.norm(ref[m]), m


# (the last two: tiles of 256 rows for both contractions, and for the first alone)
BACKWARD = [c for c in LAYERS if c[0] != 16] + [(900, 2, 3, 512, 256, 256, 256, "mixed"), (1100, 1, 4, 320, 448, 64, 64, "one"),
                                                (4000, 2, 3, 1344, 1344, 64, 64, "dropped"), (9000, 1, 2, 1344, 128, 64, 128, "mixed")]


@pytest.mark.parametrize("M,top,E,F,K,gh,g,kind", BACKWARD)
def test_moe_ffn_gated_backward(cr, M, top, E, F, K, gh, g, kind):
    P.say("moe_ffn_gated_backward M=%d top=%d E=%d F=%d K=%d %s" % (M, top, E, F, K, kind))
    gate, up, down = _layer(cr, E, F, K, gh, g)
    experts, w = _experts(M, top, E, M + top, kind)
    acts = R.ACTS if M in (5, 130) else ("silu",)
    nq = lambda p: (_np(p[0]), _np(p[1]))
    for act in acts:
        dy, pre, d = _randn(M, K, seed=1), _randn(2, M, top, F, seed=2, std=1.5), _randn(M, top, K, seed=3)
        add = _randn(M, K, seed=4, std=2.0)
        call = dict(act=act, group=g, group_h=gh)
        dx, dw = cr.moe_ffn_gated_backward(dy, pre, d, experts, w, *gate, *up, *down, **call)
        e = experts.cpu().numpy()
        ref, rw = MR.moe_backward(_np(dy), _np(pre), _np(d), e, _np(w), nq(gate), nq(up), nq(down), act, g, gh)
        size = np.abs(_np(dy)[:, None, :] * _np(d)).sum(2)
        assert np.all(np.abs(dw.double().cpu().numpy() - rw) <= (K + 8) * R.U * size)
        assert (dw[(experts < 0) | (experts >= E)] == 0).all()
        if np.linalg.norm(ref) == 0:
            assert (dx == 0).all()
        else:
            rel = np.linalg.norm(_np(dx) - ref) / np.linalg.norm(ref)
            assert torch.isfinite(dx).all() and rel <= 2 * R.BF16, rel
        both, dw2 = cr.moe_ffn_gated_backward(dy, pre, d, experts, w, *gate, *up, *down, dx_add=add, **call)
        assert torch.equal(dw2, dw)
        rel = np.linalg.norm(_np(both) - ref - _np(add)) / np.linalg.norm(ref + _np(add))
        assert rel <= 2 * R.BF16, rel
        place = add.clone()
        got, none = cr.moe_ffn_gated_backward(dy, pre, None, experts, w, *gate, *up, *down, dx_add=place, out=place, **call)
        assert none is None and got is place and torch.equal(place, both), "in place, without dweights"


def test_moe_gradients_against_differences(cr):
    """Central differences of the forward call along a direction, for dx; the sum is linear in the weights, so
    dweights against whole steps.  The forward's INT8 codes change by steps of their own: with a relative step of 1/8 the
    difference of 2 x 256 tokens averages them out to below 3%."""
    M, top, E, F, K = 256, 3, 6, 512, 512
    gate, up, down = _layer(cr, E, F, K, 256, 256)
    experts, w = _experts(M, top, E, 5)
    x, dy = _randn(M, K, seed=1, dtype=torch.float32), _randn(M, K, seed=2)
    y, pre, d = cr.moe_ffn_gated(x, experts, w, *gate, *up, *down, save=True)
    dx, dw = cr.moe_ffn_gated_backward(dy, pre, d, experts, w, *gate, *up, *down)
    v = dx.float() / dx.float().norm() * x.norm()                 # along the gradient: the signal adds up
    step = 0.125
    loss = lambda z: (cr.moe_ffn_gated(z, experts, w, *gate, *up, *down).double() * dy.double()).sum()
    diff = ((loss(x + step * v) - loss(x - step * v)) / (2 * step)).item()
    want = (dx.double() * v.double()).sum().item()
    assert abs(diff - want) <= 0.03 * abs(want), (diff, want)
    for j in range(top):
        more = w.clone()
        more[:, j] += 1.0
        part = ((cr.moe_ffn_gated(x, experts, more, *gate, *up, *down).double() - y.double()) * dy.double()).sum(1)
        # two bf16 roundings of y against dy, and d's own
        y2 = y.double() + d[:, j].double()
        bound = R.BF16 * ((y.double().abs() + y2.abs() + d[:, j].double().abs()) * dy.double().abs()).sum(1)
        assert (part - dw[:, j].double()).abs().le(bound).all()


class _MoE(torch.autograd.Function):
    """The layer in a training loop: weights frozen, gradients of the tokens and of the router's weights."""

    @staticmethod
    def forward(ctx, cr, x, experts, weights, gate, up, down, group, group_h):
        y, pre, d = cr.moe_ffn_gated(x, experts, weights, *gate, *up, *down, residual=x, group=group, group_h=group_h, save=True)
        ctx.cr, ctx.packed, ctx.groups = cr, (gate, up, down), (group, group_h)
        ctx.save_for_backward(pre, d, experts, weights)
        return y

    @staticmethod
    def backward(ctx, dy):
        pre, d, experts, weights = ctx.saved_tensors
        gate, up, down = ctx.packed
        dy = dy.contiguous()
        dx, dw = ctx.cr.moe_ffn_gated_backward(dy, pre, d, experts, weights, *gate, *up, *down, group=ctx.groups[0],
                                               group_h=ctx.groups[1], dx_add=dy)
        return None, dx, None, dw, None, None, None, None, None


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, cr, logits, top):
        experts, weights = cr.moe_route(logits, top)
        ctx.cr = cr
        ctx.save_for_backward(logits, experts)
        ctx.mark_non_differentiable(experts)
        return experts, weights

    @staticmethod
    def backward(ctx, _, dw):
        logits, experts = ctx.saved_tensors
        return None, ctx.cr.moe_route_backward(dw.contiguous(), logits, experts), None


def test_router_layer_and_gradients_together(cr):
    """Router, layer and both gradients as a training step chains them, against autograd of the same step in 64 bits on the
    weights' values.  The step's own INT8 tokens are off by 1/254 of a row's largest channel, about 1% of a value, and
    hidden channels again: held to 3% in the 2-norm."""
    M, E, top, F, K, g = 96, 8, 2, 256, 256, 256
    gate, up, down = _layer(cr, E, F, K, 256, 256)
    x0, wr0, t = _randn(M, K, seed=1), _randn(E, K, seed=2, std=0.1, dtype=torch.float32), _randn(M, K, seed=3)
    x = x0.clone().requires_grad_()
    wr = wr0.clone().requires_grad_()
    experts, weights = _Route.apply(cr, x.float() @ wr.t(), top)
    y = _MoE.apply(cr, x, experts, weights, gate, up, down, g, 256)
    (y.float() * t.float()).sum().backward()

    a = x0.double().cpu().requires_grad_()
    r = wr0.double().cpu().requires_grad_()
    logits = a @ r.t()
    v, i = torch.topk(logits, top, 1)
    assert torch.equal(i.to(torch.int32), experts.cpu())
    share = torch.softmax(v, 1)
    real = lambda p: torch.from_numpy(R.rotate(_np(p[0]) * _np(p[1])[..., None], 256))
    wg, wu, wd = real(gate), real(up), real(down)
    out = a.clone()
    for j in range(top):
        for e in range(E):
            m = (i[:, j] == e).nonzero()[:, 0]
            h = torch.nn.functional.silu(a[m] @ wg[e].t()) * (a[m] @ wu[e].t())
            out = out.index_add(0, m, (h @ wd[e].t()) * share[m, j:j + 1])
    (out * t.double().cpu()).sum().backward()
    far = lambda got, ref: (np.linalg.norm(_np(got) - ref.detach().numpy()) / np.linalg.norm(ref.detach().numpy()))
    assert far(y, out) <= 0.03 and far(x.grad, a.grad) <= 0.03 and far(wr.grad, r.grad) <= 0.03


@pytest.mark.parametrize("M,top,E,kind", [(11003, 3, 37, "dropped"), (32769, 1, 1024, "mixed"), (16500, 4, 5, "twice"), (40001, 1, 2, "none")])
def test_many_slots_as_in_parts(cr, M, top, E, kind):
    """Slots beyond what one pass of the sort keeps: the same bits as the tokens taken a third at a time."""
    F, K = 64, 128
    gate, up, down = _layer(cr, E, F, K, 64, 128)
    experts, w = _experts(M, top, E, M, kind)
    x, dy, call = _randn(M, K, seed=1), _randn(M, K, seed=2), dict(group=128, group_h=64)
    y, pre, d = cr.moe_ffn_gated(x, experts, w, *gate, *up, *down, save=True, **call)
    dx, dw = cr.moe_ffn_gated_backward(dy, pre, d, experts, w, *gate, *up, *down, **call)
    ok = (experts >= 0) & (experts < E)
    for at in (slice(0, M // 3), slice(M // 3, 2 * M // 3), slice(2 * M // 3, M)):
        own = lambda t: t[at].clone()
        wy, wp, wd = cr.moe_ffn_gated(own(x), own(experts), own(w), *gate, *up, *down, save=True, **call)
        o = ok[at]
        assert torch.equal(y[at], wy) and torch.equal(pre[:, at][:, o], wp[:, o]) and torch.equal(d[at][o], wd[o])
        wx, ww = cr.moe_ffn_gated_backward(own(dy), pre[:, at].clone(), own(d), own(experts), own(w), *gate, *up, *down, **call)
        assert torch.equal(dx[at], wx) and torch.equal(dw[at], ww)


def test_large_rows(cr):
    """Row offsets past 32 bits: 2^31 elements of y, of dy's operand and of the saved arrays."""
    E, N, K, rows = 2, 4096, 64, 600_000                           # 2.46e9 outputs
    wq, ws = _weights(cr, E, N, K, 64, 1)
    x = _randn(rows, K, seed=1)
    offsets = _offsets([300_001, 299_999])
    y = cr.linear_grouped(x, wq, ws, offsets, group=64)
    for lo, hi, e in ((0, 300, 0), (299_900, 300_001, 0), (300_001, 300_200, 1), (599_800, 600_000, 1)):
        assert torch.equal(y[lo:hi], cr.linear(x[lo:hi].clone(), wq[e], ws[e], group=64)), lo
    dx = cr.linear_grouped_backward(y, wq, ws, offsets, group=64)
    for lo, hi, e in ((0, 200, 0), (300_001, 300_200, 1), (599_800, 600_000, 1)):
        a, q = _np((y[lo:hi].float() * ws[e]).bfloat16()), _np(wq[e])
        ref = R.rotate(a @ q, 64)
        bound = (N + 16) * R.U * R.rotate_abs(np.abs(a) @ np.abs(q), 64)
        R.check(_np(dx[lo:hi]), ref, R.rounded(ref, bound), "dx")
    del y, dx
    M, top, F, K = 80_000, 8, 64, 4096                            # 2.6e9 elements of d and of its 16-bit copies
    gate, up, down = _layer(cr, 8, F, K, 64, 256)
    experts = torch.arange(8, dtype=torch.int32, device=DEV).repeat(M, 1)
    w = torch.rand(M, top, device=DEV)
    x = _randn(M, K, seed=2)
    y, pre, d = cr.moe_ffn_gated(x, experts, w, *gate, *up, *down, group=256, group_h=64, save=True)
    at = slice(M - 40, M)
    want = cr.moe_ffn_gated(x[at].clone(), experts[at].clone(), w[at].clone(), *gate, *up, *down, group=256, group_h=64, save=True)
    assert torch.equal(y[at], want[0]) and torch.equal(pre[:, at], want[1]) and torch.equal(d[at], want[2])
    dx, dw = cr.moe_ffn_gated_backward(x, pre, d, experts, w, *gate, *up, *down, group=256, group_h=64)
    assert torch.equal(dw[at], cr.moe_ffn_gated_backward(x[at].clone(), want[1], want[2], experts[at].clone(), w[at].clone(),
                                                         *gate, *up, *down, group=256, group_h=64)[1])
    rx, _ = MR.moe_backward(_np(x[at]), _np(pre[:, at]), _np(d[at]), experts[at].cpu().numpy(), _np(w[at]),
                            *[(_np(p[0]), _np(p[1])) for p in (gate, up, down)], "silu", 256, 64)
    assert np.linalg.norm(_np(dx[at]) - rx) <= 2 * R.BF16 * np.linalg.norm(rx)
