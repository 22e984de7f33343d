"""The fused linears and their gradients through the C calls, in memory the caller provides: a workspace of exactly
the reported size and outputs of exactly their own size, each between guard bytes that have to survive; a
workspace whose contents on entry are NaN patterns; one workspace shared by two captured graphs; calls
on two streams at once.  Results are compared with the binding's, bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
GUARD = 4096


@pytest.fixture(scope="module")
def cr():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from int4_quantized_linear_amd import convrot
    convrot.load()
    return convrot


def _weight(cr, N, K, g, seed):
    gen = torch.Generator().manual_seed(seed)
    return cr.prepare_weight((torch.randn(N, K, generator=gen) * 0.05).bfloat16().to(DEV), g, 8)


def _randn(*shape, seed, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


class Guarded:
    """nbytes of device memory between guards; 0xff everywhere (a NaN in bf16 and fp32)."""

    def __init__(self, nbytes):
        self.n = nbytes
        self.buf = torch.full((GUARD + nbytes + GUARD + 256,), 0xff, dtype=torch.uint8, device=DEV)
        self.at = GUARD + -(self.buf.data_ptr() + GUARD) % 256

    @property
    def ptr(self):
        return self.buf.data_ptr() + self.at

    def bytes(self):
        return self.buf[self.at:self.at + self.n]

    def intact(self):
        return bool((self.buf[:self.at] == 0xff).all() and (self.buf[self.at + self.n:] == 0xff).all())


def _p(t):
    return None if t is None else t.data_ptr()


class Call:
    """One entry point on fixed inputs: run(stream) enqueues it into guarded memory, want() is the binding's result."""

    def __init__(self, cr, op, M, N, K, g, seed=0):
        self.cr, self.op = cr, op
        stream = lambda: torch.cuda.current_stream().cuda_stream
        forward = not op.endswith("backward")
        sizes = dict(linear_act=lambda: cr.workspace_bytes_act(M, N, K), linear_gated=lambda: cr.workspace_bytes_gated(M, N, K),
                     ffn_gated=lambda: cr.workspace_bytes_ffn(M, N, K),
                     linear_act_backward=lambda: cr.workspace_bytes_backward(M, N, K),
                     linear_gated_backward=lambda: cr.workspace_bytes_gated_backward(M, N, K),
                     ffn_gated_backward=lambda: cr.workspace_bytes_ffn_backward(M, N, K))
        self.ws = ws = Guarded(sizes[op]())
        a, b = _weight(cr, N, K, g, 1 + seed), _weight(cr, N, K, g, 2 + seed)
        act, code = ("silu", cr.ACTS["silu"])
        new = lambda n: Guarded(n)
        if op.startswith("ffn"):
            gh = cr.dynamic_group(N)
            d = _weight(cr, K, N, gh, 3 + seed)
        if op == "linear_act":
            x, r = _randn(M, K, seed=seed), _randn(M, N, seed=seed + 1)
            y, pre = new(M * N * 2), new(M * N * 2)
            self.outs = [y, pre]
            self.run = lambda: cr._call("convrot_linear_act", _p(x), cr.CONVROT_DTYPE_BF16, None, None, M, N, K, g, _p(a[0]),
                                        _p(a[1]), None, code, _p(r), pre.ptr, y.ptr, ws.ptr, ws.n, stream())
            self.want = lambda: cr.linear_act(x, *a, act=act, residual=r, group=g, save_pre=True)
        elif op == "linear_gated":
            x = _randn(M, K, seed=seed, dtype=torch.float32)
            h, pre = new(M * N * 2), new(M * N * 4)
            self.outs = [h, pre]
            self.run = lambda: cr._call("convrot_linear_gated", _p(x), cr.CONVROT_DTYPE_F32, None, None, M, N, K, g, _p(a[0]),
                                        _p(a[1]), None, _p(b[0]), _p(b[1]), None, code, pre.ptr, h.ptr, ws.ptr, ws.n, stream())
            self.want = lambda: cr.linear_gated(x, *a, *b, act=act, group=g, save_pre=True)
        elif op == "ffn_gated":
            x, r = _randn(M, K, seed=seed), _randn(M, K, seed=seed + 1)
            y, pre = new(M * K * 2), new(M * N * 4)
            self.outs = [y, pre]
            self.run = lambda: cr._call("convrot_ffn_gated", _p(x), cr.CONVROT_DTYPE_BF16, M, N, K, g, gh, _p(a[0]), _p(a[1]), None,
                                        _p(b[0]), _p(b[1]), None, _p(d[0]), _p(d[1]), None, code, _p(r), pre.ptr, y.ptr, ws.ptr,
                                        ws.n, stream())
            self.want = lambda: cr.ffn_gated(x, *a, *b, *d, act=act, residual=r, group=g, group_h=gh, save_pre=True)
        elif op == "linear_act_backward":
            dy, pre, add = _randn(M, N, seed=seed), _randn(M, N, seed=seed + 1), _randn(M, K, seed=seed + 2)
            dx, db = new(M * K * 2), new(N * 4)
            self.outs = [dx, db]
            self.run = lambda: cr._call("convrot_linear_act_backward", _p(dy), _p(pre), M, N, K, g, _p(a[0]), _p(a[1]), code, _p(add),
                                        dx.ptr, db.ptr, ws.ptr, ws.n, stream())
            self.want = lambda: cr.linear_act_backward(dy, *a, pre=pre, act=act, group=g, bias_grad=True, dx_add=add)
        elif op == "linear_gated_backward":
            dh, pre = _randn(M, N, seed=seed), _randn(2, M, N, seed=seed + 1)
            dx, dg, du = new(M * K * 2), new(N * 4), new(N * 4)
            self.outs = [dx, dg, du]
            self.run = lambda: cr._call("convrot_linear_gated_backward", _p(dh), _p(pre), M, N, K, g, _p(a[0]), _p(a[1]), _p(b[0]),
                                        _p(b[1]), code, None, dx.ptr, dg.ptr, du.ptr, ws.ptr, ws.n, stream())
            self.want = lambda: cr.linear_gated_backward(dh, pre, *a, *b, act=act, group=g, bias_grad=True)
        else:
            dy, pre = _randn(M, K, seed=seed), _randn(2, M, N, seed=seed + 1)
            dx = new(M * K * 2)
            self.outs = [dx]
            self.run = lambda: cr._call("convrot_ffn_gated_backward", _p(dy), _p(pre), M, N, K, g, gh, _p(a[0]), _p(a[1]), _p(b[0]),
                                        _p(b[1]), _p(d[0]), _p(d[1]), code, _p(dy), dx.ptr, None, None, None, ws.ptr, ws.n, stream())
            self.want = lambda: (cr.ffn_gated_backward(dy, pre, *a, *b, *d, act=act, group=g, group_h=gh, dx_add=dy),)

    def same(self, want):
        return all(torch.equal(o.bytes(), w.contiguous().view(torch.uint8).flatten()) for o, w in zip(self.outs, want))


OPS = ("linear_act", "linear_gated", "ffn_gated", "linear_act_backward", "linear_gated_backward", "ffn_gated_backward")
# M, N (hidden), K, group; N of the blocks is a multiple of 64
SIZES = [(1, 64, 64, 64), (7, 33, 320, 64), (16, 192, 512, 256), (17, 1001, 320, 64), (70, 1024, 512, 256),
         (300, 1344, 2688, 128), (301, 391, 1024, 256), (1100, 576, 1536, 256)]


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("M,N,K,g", SIZES)
def test_stays_in_its_memory(cr, op, M, N, K, g):
    if op.startswith("ffn"):
        N = (N + 63) // 64 * 64
    c = Call(cr, op, M, N, K, g)
    c.run()
    torch.cuda.synchronize()
    assert c.ws.intact(), "workspace guards"
    assert all(o.intact() for o in c.outs), "output guards"
    assert c.same(c.want())


@pytest.mark.parametrize("op", OPS)
def test_two_graphs_share_a_workspace(cr, op):
    """Two sizes captured into two graphs with one workspace, replayed in turn with eager calls between."""
    calls = [Call(cr, op, 300, 1344, 2688, 128, 10), Call(cr, op, 40, 512, 1024, 256, 20)]
    shared = max((c.ws for c in calls), key=lambda w: w.n)
    for c in calls:
        c.ws.buf, c.ws.at, c.ws.n = shared.buf, shared.at, shared.n
    wants = [c.want() for c in calls]
    graphs = []
    torch.cuda.synchronize()
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for rep in range(3):
        for g, c, w in zip(graphs, calls, wants):
            for o in c.outs:
                o.bytes().fill_(0xff)
            g.replay()
            torch.cuda.synchronize()
            assert c.same(w), "replay %d" % rep
            assert c.same(c.want())


def test_two_streams_at_once(cr):
    """Every entry point on one stream while the same runs on other inputs on another."""
    for op in OPS:
        for M in (5, 130, 600):
            pair = [Call(cr, op, M, 1024, 1024, 256, 30), Call(cr, op, M, 1024, 1024, 256, 40)]
            wants = [c.want() for c in pair]
            streams = [torch.cuda.Stream(), torch.cuda.Stream()]
            for s in streams:
                s.wait_stream(torch.cuda.current_stream())
            for _ in range(3):
                for s, c in zip(streams, pair):
                    with torch.cuda.stream(s):
                        c.run()
            torch.cuda.synchronize()
            assert all(c.same(w) for c, w in zip(pair, wants)), (op, M)


@pytest.mark.parametrize("M", [0, 1, 16, 17, 600])
def test_one_of_two_bias_gradients(cr, M):
    """Either bias gradient of the gated linear alone, and neither, as with both."""
    N, K, g = 1001, 320, 64
    a, b = _weight(cr, N, K, g, 1), _weight(cr, N, K, g, 2)
    dh, pre = _randn(M, N, seed=1), _randn(2, M, N, seed=2)
    want = cr.linear_gated_backward(dh, pre, *a, *b, group=g, bias_grad=True)
    ws = Guarded(max(cr.workspace_bytes_gated_backward(M, N, K), 256))
    for first, second in ((True, False), (False, True), (False, False)):
        dx, dg, du = Guarded(M * K * 2), Guarded(N * 4), Guarded(N * 4)
        cr._call("convrot_linear_gated_backward", _p(dh), _p(pre), M, N, K, g, _p(a[0]), _p(a[1]), _p(b[0]), _p(b[1]),
                 cr.ACTS["silu"], None, dx.ptr, dg.ptr if first else None, du.ptr if second else None, ws.ptr, ws.n,
                 torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        for got, ref, asked in ((dx, want[0], True), (dg, want[1], first), (du, want[2], second)):
            assert got.intact()
            if asked:
                assert torch.equal(got.bytes(), ref.contiguous().view(torch.uint8).flatten())
            else:
                assert (got.bytes() == 0xff).all()
