"""The router, the grouped linears and the expert layer through the C calls, in memory the caller provides: a workspace of
exactly the reported size and outputs of exactly their own size, each between guard bytes that have to survive; a workspace
whose contents on entry are NaN patterns; graphs that share a workspace, replayed on other routings than the captured one;
calls on two streams at once; outputs in the place of inputs; pointers aligned to their elements only where that is allowed.
Results are compared with the binding's, bit for bit."""
import pytest
import torch

from tests import parity as P
from tests.test_gpu_fused_bounds import DEV, Guarded, _p, _randn, cr  # noqa: F401  (cr is a fixture)

pytestmark = pytest.mark.gpu


def _stacked(cr, E, N, K, g, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    q, s = cr.prepare_weight((torch.randn(E * N, K, generator=gen, device=DEV) * 0.05).bfloat16(), g, 8)
    return q.view(E, N, K), s.view(E, N)


def _routing(M, top, E, seed):
    """Experts (some slots without one, some twice in a row) and weights."""
    gen = torch.Generator().manual_seed(seed)
    e = torch.randint(-1, E, (M, top), generator=gen, dtype=torch.int32)
    return e.to(DEV), (torch.rand(M, top, generator=gen) + 0.05).to(DEV)


def _sorted_offsets(rows, E, seed):
    gen = torch.Generator().manual_seed(seed)
    o = torch.randint(0, rows + 1, (E + 1,), generator=gen).sort().values
    return o.to(torch.int32).to(DEV)


class Call:
    """One entry point on fixed inputs: run() enqueues it into guarded memory, want() is the binding's result in memory that
    holds the same bytes before."""

    def __init__(self, cr, op, M, E, top, N, K, g, seed=0, dtype=torch.bfloat16):
        stream = lambda: torch.cuda.current_stream().cuda_stream
        code = cr.CONVROT_DTYPE_BF16 if dtype is torch.bfloat16 else cr.CONVROT_DTYPE_F32
        ones = lambda *shape: torch.full(shape, -1, dtype=torch.int16, device=DEV).view(torch.bfloat16)
        gh = cr.dynamic_group(N) if N % 64 == 0 else 1
        self.ws = Guarded(0)
        if op.startswith("route"):
            score, scale = cr.SCORES["sigmoid" if seed % 2 else "softmax"], 1.5
            name = "sigmoid" if seed % 2 else "softmax"
            logits = _randn(M, E, seed=seed, dtype=dtype)
            bias = _randn(E, seed=seed + 1, dtype=torch.float32) if seed % 3 else None
            self.routing = [logits]
            if op == "route":
                e, w = Guarded(M * top * 4), Guarded(M * top * 4)
                self.outs = [e, w]
                self.run = lambda: cr._call("convrot_moe_route", _p(logits), code, M, E, top, score, 1, scale, _p(bias), e.ptr, w.ptr,
                                            stream())
                self.want = lambda: cr.moe_route(logits, top, bias=bias, score=name, scale=scale)
            else:
                experts = cr.moe_route(logits, top)[0]
                dw = _randn(M, top, seed=seed + 2, dtype=torch.float32)
                out = Guarded(logits.numel() * logits.element_size())
                self.outs = [out]
                self.run = lambda: cr._call("convrot_moe_route_backward", _p(dw), _p(logits), code, M, E, top, score, 0, scale,
                                            _p(experts), out.ptr, stream())
                self.want = lambda: (cr.moe_route_backward(dw, logits, experts, score=name, normalize=False, scale=scale),)
        elif op.startswith("linear_grouped"):
            a = _stacked(cr, E, N, K, g, 1 + seed)
            offsets = _sorted_offsets(M, E, seed)
            self.routing = [offsets]
            if op == "linear_grouped":
                x, y = _randn(M, K, seed=seed, dtype=dtype), Guarded(M * N * 2)
                self.outs, self.ws = [y], Guarded(cr.workspace_bytes_grouped(M, E, N, K))
                self.run = lambda: cr._call("convrot_linear_grouped", _p(x), code, None, None, M, N, K, g, _p(offsets), E, _p(a[0]),
                                            _p(a[1]), y.ptr, self.ws.ptr, self.ws.n, stream())
                self.want = lambda: (cr.linear_grouped(x, *a, offsets, group=g, out=ones(M, N)),)
            else:
                dy, add, dx = _randn(M, N, seed=seed), _randn(M, K, seed=seed + 1), Guarded(M * K * 2)
                self.outs, self.ws = [dx], Guarded(cr.workspace_bytes_grouped_backward(M, E, N, K))
                self.run = lambda: cr._call("convrot_linear_grouped_backward", _p(dy), M, N, K, g, _p(offsets), E, _p(a[0]), _p(a[1]),
                                            _p(add), dx.ptr, self.ws.ptr, self.ws.n, stream())
                self.want = lambda: (cr.linear_grouped_backward(dy, *a, offsets, group=g, dx_add=add, out=ones(M, K)),)
        else:
            F = N
            a, b, d = _stacked(cr, E, F, K, g, 1 + seed), _stacked(cr, E, F, K, g, 2 + seed), _stacked(cr, E, K, F, gh, 3 + seed)
            experts, w = _routing(M, top, E, seed)
            self.routing = [experts, w]
            weights = (_p(a[0]), _p(a[1]), _p(b[0]), _p(b[1]), _p(d[0]), _p(d[1]))
            call = dict(group=g, group_h=gh)
            if op == "moe":
                x, r = _randn(M, K, seed=seed, dtype=dtype), _randn(M, K, seed=seed + 1)
                y, pre, dd = Guarded(M * K * 2), Guarded(2 * M * top * F * 2), Guarded(M * top * K * 2)
                self.outs, self.ws = [y, pre, dd], Guarded(cr.workspace_bytes_moe_ffn(M, top, E, F, K))
                self.run = lambda: cr._call("convrot_moe_ffn_gated", _p(x), code, _p(experts), _p(w), M, top, E, F, K, g, gh, *weights,
                                            cr.ACTS["silu"], _p(r), pre.ptr, dd.ptr, y.ptr, self.ws.ptr, self.ws.n, stream())

                def want():                                      # rows of slots without an expert are left as they were
                    y, p, s = cr.moe_ffn_gated(x, experts, w, *a, *b, *d, residual=r, save=True, **call)
                    none = (experts < 0) | (experts >= E)
                    p[:, none], s[none] = ones(1), ones(1)
                    return y, p, s
                self.want = want
            else:
                dy, pre, s = _randn(M, K, seed=seed), _randn(2, M, top, F, seed=seed + 1), _randn(M, top, K, seed=seed + 2)
                dx, dw = Guarded(M * K * 2), Guarded(M * top * 4)
                self.outs, self.ws = [dx, dw], Guarded(cr.workspace_bytes_moe_ffn_backward(M, top, E, F, K))
                self.run = lambda: cr._call("convrot_moe_ffn_gated_backward", _p(dy), _p(pre), _p(s), _p(experts), _p(w), M, top, E, F,
                                            K, g, gh, *weights, cr.ACTS["silu"], _p(dy), dx.ptr, dw.ptr, self.ws.ptr, self.ws.n, stream())
                self.want = lambda: cr.moe_ffn_gated_backward(dy, pre, s, experts, w, *a, *b, *d, dx_add=dy, **call)

    def same(self, want):
        return all(torch.equal(o.bytes(), w.contiguous().view(torch.uint8).flatten()) for o, w in zip(self.outs, want))

    def intact(self):
        return self.ws.intact() and all(o.intact() for o in self.outs)

    def clear(self):
        for o in self.outs:
            o.bytes().fill_(0xff)


OPS = ("route", "route_backward", "linear_grouped", "linear_grouped_backward", "moe", "moe_backward")
# M (rows), E, top, N (hidden), K, group: up to 64 slots and more, 64-, 128- and 256-row tiles, more groups than rows
SIZES = [(1, 1, 1, 64, 64, 64), (3, 64, 8, 64, 320, 64), (32, 5, 2, 192, 512, 256), (33, 1024, 2, 64, 64, 1), (70, 7, 3, 1024, 192, 64),
         (301, 16, 3, 448, 640, 128), (700, 3, 2, 1344, 576, 64), (2100, 4, 2, 1280, 2688, 128)]


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("M,E,top,N,K,g", SIZES)
def test_stays_in_its_memory(cr, op, M, E, top, N, K, g):
    P.say("%s M=%d E=%d top=%d N=%d K=%d" % (op, M, E, top, N, K))
    for dtype in (torch.bfloat16, torch.float32):
        if op.startswith("linear") and dtype is torch.float32:
            N = N - 23                                           # an odd width
        c = Call(cr, op, M, E, top, N, K, g, seed=M, dtype=dtype)
        c.run()
        torch.cuda.synchronize()
        assert c.ws.intact(), "workspace guards"
        assert all(o.intact() for o in c.outs), "output guards"
        assert c.same(c.want())


def _new_routing(c, op, rep):
    """Other values in the tensors that decide the routing, in place."""
    for t in c.routing:
        if t.dtype is torch.int32 and op.startswith("linear"):
            t.copy_(t // 2 if rep == 0 else t + 1)
        else:
            t.copy_(t.roll(1, 0))


@pytest.mark.parametrize("op", OPS)
def test_two_graphs_share_a_workspace(cr, op):
    """Calls of three sizes captured into graphs with one workspace, replayed in turn on other routings than the captured
    ones, with eager calls between."""
    calls = [Call(cr, op, 300, 16, 3, 448, 640, 128, 10), Call(cr, op, 12, 40, 4, 192, 320, 64, 21), Call(cr, op, 1500, 4, 2, 1344, 512, 256, 30)]
    shared = max((c.ws for c in calls), key=lambda w: w.n)
    for c in calls:
        c.ws.buf, c.ws.at, c.ws.n = shared.buf, shared.at, shared.n
        c.want()
    graphs = []
    torch.cuda.synchronize()
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for rep in range(3):
        wants = []
        for c in calls:
            _new_routing(c, op, rep)
            wants.append(c.want())
            c.clear()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for c, w in zip(calls, wants):
            assert c.same(w), "replay %d" % rep
            assert c.same(c.want()) and c.intact()


@pytest.mark.parametrize("op", OPS)
def test_two_streams_at_once(cr, op):
    """The same call on other inputs on another stream at the same time, each with its own workspace."""
    for M in (4, 130, 900):
        P.say("%s M=%d" % (op, M))
        pair = [Call(cr, op, M, 12, 2, 512, 1024, 256, 30), Call(cr, op, M, 12, 2, 512, 1024, 256, 41)]
        wants = [c.want() for c in pair]
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            for s, c in zip(streams, pair):
                with torch.cuda.stream(s):
                    c.run()
        torch.cuda.synchronize()
        assert all(c.same(w) and c.intact() for c, w in zip(pair, wants)), M


@pytest.mark.parametrize("M,E,top", [(9, 64, 8), (600, 12, 2)])
def test_outputs_in_the_place_of_inputs(cr, M, E, top):
    """dx in the place of dy or of dx_add, dlogits in that of the logits, y in that of x or the residual."""
    F, K = 192, 320
    gate, up, down = _stacked(cr, E, F, K, 64, 1), _stacked(cr, E, F, K, 64, 2), _stacked(cr, E, K, F, 64, 3)
    experts, w = _routing(M, top, E, 1)
    x, r = _randn(M, K, seed=1), _randn(M, K, seed=2)
    call = dict(group=64, group_h=64)
    want, pre, d = cr.moe_ffn_gated(x, experts, w, *gate, *up, *down, residual=r, save=True, **call)
    for out in (x.clone(), r.clone()):
        first, second = (out, r) if torch.equal(out, x) else (x, out)
        assert torch.equal(cr.moe_ffn_gated(first, experts, w, *gate, *up, *down, residual=second, out=out, **call), want)
    both = x.clone()                                             # y, x and the residual the same array
    want = cr.moe_ffn_gated(x, experts, w, *gate, *up, *down, residual=x, **call)
    assert torch.equal(cr.moe_ffn_gated(both, experts, w, *gate, *up, *down, residual=both, out=both, **call), want)
    dy, add = _randn(M, K, seed=3), _randn(M, K, seed=4)
    wdx, wdw = cr.moe_ffn_gated_backward(dy, pre, d, experts, w, *gate, *up, *down, dx_add=add, **call)
    for out in (dy.clone(), add.clone()):
        first, second = (out, add) if torch.equal(out, dy) else (dy, out)
        dx, dw = cr.moe_ffn_gated_backward(first, pre, d, experts, w, *gate, *up, *down, dx_add=second, out=out, **call)
        assert torch.equal(dx, wdx) and torch.equal(dw, wdw)
    wdx, wdw = cr.moe_ffn_gated_backward(dy, pre, d, experts, w, *gate, *up, *down, dx_add=dy, **call)
    place = dy.clone()
    dx, dw = cr.moe_ffn_gated_backward(place, pre, d, experts, w, *gate, *up, *down, dx_add=place, out=place, **call)
    assert torch.equal(dx, wdx) and torch.equal(dw, wdw)
    logits, dw = _randn(M, E, seed=5, dtype=torch.float32), _randn(M, top, seed=6, dtype=torch.float32)
    chosen = cr.moe_route(logits, top)[0]
    for normalize in (True, False):
        want = cr.moe_route_backward(dw, logits, chosen, normalize=normalize)
        place = logits.clone()
        assert torch.equal(cr.moe_route_backward(dw, place, chosen, normalize=normalize, out=place), want)


def test_smallest_alignment(cr):
    """The router's arrays, offsets, experts, weights and scales at odd multiples of their elements."""
    def odd(t):
        room = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        room[1:] = t.flatten()
        return room[1:].view(t.shape)
    for M, E, top in ((3, 9, 4), (130, 9, 2)):
        F, K = 64, 320
        gate, up, down = _stacked(cr, E, F, K, 64, 1), _stacked(cr, E, F, K, 64, 2), _stacked(cr, E, K, F, 64, 3)
        scales = lambda *ws: [v for q, s in ws for v in (q, odd(s))]
        for dtype in (torch.float32, torch.bfloat16):
            logits, bias = _randn(M, E, seed=1, dtype=dtype), _randn(E, seed=2, dtype=torch.float32)
            experts, w = cr.moe_route(logits, top, bias=bias)
            got = cr.moe_route(odd(logits), top, bias=odd(bias))
            assert torch.equal(got[0], experts) and torch.equal(got[1], w)
            dw = _randn(M, top, seed=3, dtype=torch.float32)
            assert torch.equal(cr.moe_route_backward(odd(dw), odd(logits), odd(experts), out=odd(logits)),
                               cr.moe_route_backward(dw, logits, experts))
        x, dy = _randn(M, K, seed=4), _randn(M, K, seed=5)
        call = dict(group=64, group_h=64)
        want = cr.moe_ffn_gated(x, experts, w, *gate, *up, *down, save=True, **call)
        got = cr.moe_ffn_gated(x, odd(experts), odd(w), *scales(gate, up, down), save=True, **call)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        back = cr.moe_ffn_gated_backward(dy, want[1], want[2], experts, w, *gate, *up, *down, **call)
        got = cr.moe_ffn_gated_backward(dy, want[1], want[2], odd(experts), odd(w), *scales(gate, up, down), **call)
        assert all(torch.equal(a, b) for a, b in zip(got, back))
        offsets = _sorted_offsets(M, E, 1)
        offsets[0], offsets[-1] = 0, M
        assert torch.equal(cr.linear_grouped(x, gate[0], odd(gate[1]), odd(offsets), group=64), cr.linear_grouped(x, *gate, offsets, group=64))
        dh = _randn(M, F, seed=6)
        assert torch.equal(cr.linear_grouped_backward(dh, gate[0], odd(gate[1]), odd(offsets), group=64),
                           cr.linear_grouped_backward(dh, *gate, offsets, group=64))


@pytest.mark.parametrize("M", [5, 90, 700])
def test_rows_without_an_expert_are_not_read(cr, M):
    """pre and d of slots without an expert may hold anything, NaN included."""
    E, top, F, K = 3, 2, 192, 320
    gate, up, down = _stacked(cr, E, F, K, 64, 1), _stacked(cr, E, F, K, 64, 2), _stacked(cr, E, K, F, 64, 3)
    experts, w = _routing(M, top, E, 2)
    experts[0, 1], experts[M // 2] = -1, E
    none = (experts < 0) | (experts >= E)
    pre, d, dy = _randn(2, M, top, F, seed=1), _randn(M, top, K, seed=2), _randn(M, K, seed=3)
    want = cr.moe_ffn_gated_backward(dy, pre, d, experts, w, *gate, *up, *down, group=64, group_h=64)
    pre[:, none], d[none], w[none] = float("nan"), float("inf"), float("nan")
    got = cr.moe_ffn_gated_backward(dy, pre, d, experts, w, *gate, *up, *down, group=64, group_h=64)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and (got[1][none] == 0).all()
    x = _randn(M, K, seed=4)
    y = cr.moe_ffn_gated(x, experts, w, *gate, *up, *down, group=64, group_h=64)
    assert torch.equal(y, cr.moe_ffn_gated(x, experts, torch.where(none, 0.5, w), *gate, *up, *down, group=64, group_h=64))


@pytest.mark.parametrize("M,top", [(5, 2), (90, 2), (700, 2)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_bad_values_stay_in_their_tokens(cr, M, top, value):
    """An infinity or NaN in a token, in its gradient or in its weights changes that token's results alone, and shows there."""
    E, F, K = 3, 192, 320
    gate, up, down = _stacked(cr, E, F, K, 64, 1), _stacked(cr, E, F, K, 64, 2), _stacked(cr, E, K, F, 64, 3)
    experts, w = _routing(M, top, E, 2)
    bad = M // 2
    experts[bad] = torch.tensor([0, 2], dtype=torch.int32)
    others = torch.arange(M, device=DEV) != bad
    x, r, call = _randn(M, K, seed=1), _randn(M, K, seed=2), dict(group=64, group_h=64)
    y, pre, d = cr.moe_ffn_gated(x, experts, w, *gate, *up, *down, residual=r, save=True, **call)
    for which in ("x", "weight", "residual", "d"):
        x2, w2, r2, p = x.clone(), w.clone(), r.clone(), [gate, up, down]
        if which == "x":                                         # (what the quantizer makes of it is the linears' matter)
            x2[bad, 3] = value
        elif which == "weight":
            w2[bad, 1] = value
        elif which == "residual":
            r2[bad, 7] = value
        else:                                                    # an expert's scale: all of its tokens, and no others
            s = down[1].clone()
            s[2, 5] = value
            p[2] = (down[0], s)
        got = cr.moe_ffn_gated(x2, experts, w2, *p[0], *p[1], *p[2], residual=r2, **call)
        hit = ~others if which != "d" else (experts == 2).any(1)
        assert torch.equal(got[~hit], y[~hit]), which
        assert which == "x" or not got[hit].isfinite().all(1).any(), which
    dy, add = _randn(M, K, seed=3), _randn(M, K, seed=4)
    dx, dw = cr.moe_ffn_gated_backward(dy, pre, d, experts, w, *gate, *up, *down, dx_add=add, **call)
    for which in ("dy", "pre", "d", "weight"):
        dy2, pre2, d2, w2 = dy.clone(), pre.clone(), d.clone(), w.clone()
        if which == "dy":
            dy2[bad, 3] = value
        elif which == "pre":
            pre2[1, bad, 1, 9] = value
        elif which == "d":
            d2[bad, 0, 9] = value
        else:
            w2[bad, 0] = value
        gx, gw = cr.moe_ffn_gated_backward(dy2, pre2, d2, experts, w2, *gate, *up, *down, dx_add=add, **call)
        assert torch.equal(gx[others], dx[others]) and torch.equal(gw[others], dw[others]), which
        if which == "d":
            assert torch.equal(gx, dx) and not gw[bad].isfinite().all()
        else:
            assert not gx[bad].isfinite().all(), which
