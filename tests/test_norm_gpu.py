"""The norm on its own, forward and backward, against the formulas in 64 bits: both kinds,
each type, one row to many, one column to rows longer than a block's registers, widths that
allow no wide access; the gradient against differences as well; non-finite rows, refusals,
repeats, streams and graphs.

Tolerances.  u = 2^-24.  A sum over a row of K runs over at most `steps` additions one after
the other (a thread's own elements, then trees), so a mean is off by at most
(steps + 2) u times the mean of the magnitudes; the other operations round once each.  The
bounds below add these up to first order and double them for the higher ones."""
import pytest
import torch

from gpu_util import check_guard, guarded_empty
from ternary_weight_bit_absmean_b200 import binding as B

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = "cuda"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
RMS, LAYER = B.BL_NORM_RMS, B.BL_NORM_LAYER


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from ternary_weight_bit_absmean_b200 import build_lib
    build_lib.build()
    B.lib()


def inputs(M, K, seed, xt=BF16, dt=F32, mean=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x = n(M, K) * torch.where(torch.rand(K, generator=g, device=DEV) < 0.01, 20.0, 1.0) + mean
    dy = n(M, K) * 1e-3 * torch.exp(n(M, 1))
    return x.to(xt), (1 + 0.1 * n(K)), 0.1 * n(K), dy.to(dt)


def steps(K):
    return max(32, K // 1024 + 1) + 12


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


class Exact:
    """Forward and backward in 64 bits, with the first-order error bounds of each."""

    def __init__(self, x, w, kind, eps):
        self.x, K = x.double(), x.shape[1]
        self.w = w.double() if w is not None else torch.ones(K, dtype=torch.float64, device=x.device)
        self.kind, self.K = kind, K
        mean_abs = self.x.abs().mean(1, keepdim=True)
        mu = self.x.mean(1, keepdim=True) if kind == LAYER else torch.zeros_like(mean_abs)
        v = (self.x - mu).square().mean(1, keepdim=True)
        self.r = 1 / torch.sqrt(v + eps)
        self.n = (self.x - mu) * self.r
        s = steps(K)
        dmu = (s + 2) * U * mean_abs if kind == LAYER else 0.0 * mean_abs
        self.rho = (s / 2 + 8) * U                       # r and the roundings of n, relative
        self.dn = self.r * dmu + self.n.abs() * self.rho  # absolute

    def forward(self, b):
        y = self.n * self.w
        tol = self.dn * self.w.abs() + 2 * U * y.abs()
        if b is not None:
            y = y + b.double()
            tol = tol + U * y.abs()
        return y, 2 * tol

    def backward(self, dy):
        dy = dy.double()
        s = steps(self.K)
        g = dy * self.w
        c1 = (g * self.n).mean(1, keepdim=True)
        c2 = g.mean(1, keepdim=True) if self.kind == LAYER else torch.zeros_like(c1)
        dx = self.r * (g - c2 - self.n * c1)
        gm = g.abs().mean(1, keepdim=True)
        dc2 = (s + 3) * U * gm
        dc1 = (s + 4) * U * (g * self.n).abs().mean(1, keepdim=True) + (g.abs() * self.dn).mean(1, keepdim=True) \
            + c1.abs() * self.rho
        mag = g.abs() + c2.abs() + (self.n * c1).abs()
        tol = self.r * ((self.rho + 4 * U) * mag + dc2 + self.n.abs() * dc1 + c1.abs() * self.dn)
        # rows of a block in order, its groups, the blocks' partial sums in strips and a tree
        deep = (dy.shape[0] // 148 + 64) * U
        dw = (dy * self.n).sum(0)
        tw = (dy.abs() * self.dn).sum(0) + deep * (dy * self.n).abs().sum(0)
        db = dy.sum(0)
        tb = deep * dy.abs().sum(0)
        return (dx, 2 * tol), (dw, 2 * tw), (db, 2 * tb)


def close(got, want, tol, what):
    tol = tol + half_step(got.dtype) * want.abs() + 1e-37
    err = (got.double() - want).abs()
    assert (err <= tol).all(), "%s: %g of the tolerance at worst" % (what, (err / tol).max().item())


SHAPES = [(1, 1), (3, 5), (1, 8), (2, 31), (7, 256), (33, 1000), (5, 1537), (64, 1536), (16, 3200), (301, 4096),
          (9, 8192), (17, 8640), (3, 9999), (5, 16384), (2, 28672), (3, 32768), (2, 32769), (2, 40000), (3, 77696), (9, 9705), (10, 9712), (9, 9713), (30, 4097), (25, 4104),
          (2, 77697), (3, 80003), (2, 77689)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("kind", [RMS, LAYER])
def test_forward(M, K, kind):
    for xt, yt in [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)]:
        x, w, b, _ = inputs(M, K, seed=M + K, xt=xt, mean=3.0 if K > 100 else 0.0)
        e = Exact(x, w, kind, 1e-5)
        out = guarded_empty((M, K), yt)
        B.bitlinear_norm_forward(x, w, b, kind, 1e-5, out)
        close(out, *e.forward(b), "y %s %s" % (xt, yt))
        check_guard(out)
        close(B.norm_forward(x, w, kind=kind, out_dtype=yt), *e.forward(None), "y without a bias")
        plain = Exact(x, None, kind, 1e-3)
        close(B.norm_forward(x, None, kind=kind, norm_eps=1e-3, out_dtype=yt), *plain.forward(None), "y without w")


@pytest.mark.parametrize("M,K", SHAPES + [(2049, 200), (700, 1537), (2500, 96), (640, 8640), (400, 9000)])
@pytest.mark.parametrize("kind", [RMS, LAYER])
def test_backward(M, K, kind):
    for xt, dt, ot in [(BF16, F32, F32), (F32, F32, F32), (BF16, BF16, BF16), (F32, BF16, F32)]:
        x, w, _, dy = inputs(M, K, seed=M + K + 1, xt=xt, dt=dt, mean=3.0 if K > 100 else 0.0)
        (dx, tx), (dw, tw), (db, tb) = Exact(x, w, kind, 1e-5).backward(dy)
        gx, gw, gb = guarded_empty((M, K), ot), guarded_empty((K,), F32), guarded_empty((K,), F32)
        n = B.bitlinear_norm_backward_workspace_size(M, K)
        ws = guarded_empty((n,), torch.uint8, fill=0xFF) if n else None  # NaN in it must not show
        if n:
            ws.fill_(0xFF)
        B.bitlinear_norm_backward(dy, x, w, kind, 1e-5, gx, gw, gb, ws)
        close(gx, dx, tx, "dx %s %s" % (xt, dt))
        close(gw, dw, tw, "dw")
        close(gb, db, tb, "db")
        for t in [gx, gw, gb] + ([ws] if n else []):
            check_guard(t)
        # each output left out in turn changes nothing in the others
        hx, hw, hb = B.norm_backward(dy, x, w, kind, dx_dtype=ot)
        assert hb is None and torch.equal(hx, gx) and torch.equal(hw, gw)
        hx, hw, hb = B.norm_backward(dy, x, None, kind, bias=True, dx_dtype=ot)
        assert hw is None and torch.equal(hb, gb)
        (px, ptx), _, _ = Exact(x, None, kind, 1e-5).backward(dy)
        close(hx, px, ptx, "dx without w")


# One shape for every way in which rows are laid over blocks: one to three chunks a thread, one row
# of a block or several, whole chunks or not, a block or a cluster to a row.
@pytest.mark.parametrize("M,K", [(1200, 256), (1210, 129), (700, 1536), (310, 2051), (400, 3201), (400, 4096), (310, 4607),
                                 (300, 4864), (200, 5121), (170, 7680), (330, 7999), (310, 8192), (300, 8447),
                                 (170, 9001), (160, 16384), (90, 16389)])
@pytest.mark.parametrize("kind", [RMS, LAYER])
def test_backward_in_every_layout(M, K, kind):
    test_backward(M, K, kind)


@pytest.mark.parametrize("kind", [RMS, LAYER])
def test_backward_against_differences(kind):
    """Central differences of L = sum dy y(x, w, b) in 64 bits, every input element."""
    M, K, h = 3, 40, 1e-5
    x, w, b, dy = inputs(M, K, seed=9, xt=F32)
    dx, dw, db = B.norm_backward(dy, x, w, kind, bias=True)

    def loss(x, w, b):
        mu = x.mean(1, keepdim=True) if kind == LAYER else 0.0
        n = (x - mu) / torch.sqrt((x - mu).square().mean(1, keepdim=True) + 1e-5)
        return (dy.double() * (n * w + b)).sum()

    args = [x.double(), w.double(), b.double()]
    for i, got in enumerate([dx, dw, db]):
        want = torch.zeros_like(args[i])
        for j in range(want.numel()):
            e = torch.zeros_like(args[i]).view(-1)
            e[j] = h
            e = e.view_as(args[i])
            up = loss(*[a + e if k == i else a for k, a in enumerate(args)])
            dn = loss(*[a - e if k == i else a for k, a in enumerate(args)])
            want.view(-1)[j] = (up - dn) / (2 * h)
        # h^2 times a third derivative and 1e-16 / h: both below 1e-8 of the largest; the
        # kernel's own error is 64 u of the largest at most
        assert (got.double() - want).abs().max() <= (64 * U + 1e-8) * want.abs().max()


@pytest.mark.parametrize("K", [256, 1537, 8640, 40000, 80000])
def test_non_finite_values_spread_as_the_formulas_say(K):
    x, w, _, dy = inputs(6, K, seed=2, xt=F32)
    x[1, K // 2], x[3, 0] = float("nan"), float("inf")
    dy[4, K - 1] = float("nan")
    y = B.norm_forward(x, w, kind=LAYER)
    assert torch.isnan(y[1]).all() and torch.isnan(y[3]).all()
    assert torch.isfinite(y[[0, 2, 4, 5]]).all()
    dx, dw, db = B.norm_backward(dy, x, w, LAYER, bias=True)
    assert torch.isnan(dx[[1, 3, 4]]).all() and torch.isfinite(dx[[0, 2, 5]]).all()
    assert torch.isnan(dw).all()                       # rows 1 and 3 reach every column
    assert torch.isnan(db[K - 1]) and torch.isfinite(db[:K - 1]).all()


def test_constant_and_zero_rows():
    x = torch.zeros(4, 512, device=DEV)
    x[1], x[2] = 7.0, -1e30
    y = B.norm_forward(x, kind=LAYER)
    assert torch.equal(y[0], torch.zeros_like(y[0])) and torch.equal(y[1], torch.zeros_like(y[1]))
    z = B.norm_forward(x[:2].contiguous(), kind=RMS)
    assert torch.equal(z[0], torch.zeros_like(z[0]))
    assert (z[1].double() - 1.0).abs().max() <= 1e-5 / 49 + 32 * U  # 7 / sqrt(49 + 1e-5)


def test_results_repeat_and_do_not_depend_on_the_stream():
    x, w, b, dy = inputs(777, 1536, seed=3)
    want = B.norm_backward(dy, x, w, LAYER, bias=True)
    y = B.norm_forward(x, w, b, kind=LAYER)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [(B.norm_backward(dy, x, w, LAYER, bias=True, stream=s), B.norm_forward(x, w, b, kind=LAYER, stream=s))
           for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    for g, gy in got:
        assert all(torch.equal(p, q) for p, q in zip(g, want)) and torch.equal(gy, y)


def test_captured_and_replayed_on_new_inputs():
    x, w, b, dy = inputs(130, 3200, seed=4)
    B.norm_backward(dy, x, w, RMS)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = B.norm_forward(x, w, b)
        dx, dw, db = B.norm_backward(dy, x, w, bias=True)
    x2, _, _, dy2 = inputs(130, 3200, seed=5)
    x.copy_(x2)
    dy.copy_(dy2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, B.norm_forward(x2, w, b))
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), B.norm_backward(dy2, x2, w, bias=True)))


@pytest.mark.parametrize("M,K", [(40, 100), (700, 515), (100, 9000), (60, 20000)])
def test_one_call_does_not_read_what_another_left(M, K):
    """Back to back on the same workspace and outputs: each call's sums are its own."""
    a, w, _, da = inputs(M, K, seed=21)
    b, _, _, db = inputs(M, K, seed=22)
    n = max(1, B.bitlinear_norm_backward_workspace_size(M, K))
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    out = [torch.empty(M, K, device=DEV), torch.empty(K, device=DEV), torch.empty(K, device=DEV)]
    for x, dy in ((a, da), (b, db), (a, da)):
        B.bitlinear_norm_backward(dy, x, w, LAYER, 1e-5, *out, ws)
        assert all(torch.equal(p, q) for p, q in zip(out, B.norm_backward(dy, x, w, LAYER, bias=True)))


def test_two_graphs_with_workspaces_of_their_own():
    x, w, _, dy = inputs(500, 1536, seed=23)
    x2, _, _, dy2 = inputs(500, 1536, seed=24)
    want, want2 = B.norm_backward(dy, x, w, bias=True), B.norm_backward(dy2, x2, w, bias=True)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for a, d in ((x, dy), (x2, dy2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(B.norm_backward(d, a, w, bias=True))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(outs[0], want))
    assert all(torch.equal(p, q) for p, q in zip(outs[1], want2))


def test_offsets_past_32_bits():
    M, K = 70001, 32768                                 # 2.3e9 elements
    x = torch.empty(M, K, dtype=BF16, device=DEV)
    x[:-3] = 0.5
    tail, w, b, dyt = inputs(3, K, seed=6, dt=BF16)
    x[-3:] = tail
    y = B.norm_forward(x, w, b)
    assert torch.equal(y[-3:], B.norm_forward(tail, w, b))
    dy = torch.zeros(M, K, dtype=BF16, device=DEV)
    dy[-3:] = dyt
    dx = B.norm_backward(dy, x, w, RMS)[0]
    assert torch.equal(dx[-3:], B.norm_backward(dyt, tail, w, RMS)[0])
    assert not dx[:16].any()


def test_refusals():
    x = torch.zeros(4, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    with pytest.raises(TypeError):
        B.norm_forward(x.half())
    with pytest.raises(TypeError):
        B.norm_forward(x, w.double())
    with pytest.raises(TypeError):
        B.norm_forward(x, w.cpu())
    with pytest.raises(ValueError):
        B.norm_forward(x.t())
    with pytest.raises(ValueError):
        B.norm_forward(x, w[:32])
    with pytest.raises(ValueError):
        B.norm_backward(x[:2], x)
    with pytest.raises(ValueError):
        B.norm_forward(x[0])
    with pytest.raises(B.BitLinearError):
        B.norm_forward(torch.zeros(0, 64, device=DEV))
    with pytest.raises(B.BitLinearError):
        B.norm_forward(x, norm_eps=-1.0)
    x = torch.zeros(64, 64, device=DEV)                # several blocks: needs its workspace
    with pytest.raises(B.BitLinearError):
        B.bitlinear_norm_backward(x, x, w, RMS, 1e-5, torch.empty_like(x), torch.empty_like(w), None, None)


def test_gradient_of_a_ternary_layer_reaches_x():
    """Quant(LN(x)) -> ternary product -> straight-through backward -> the norm's backward."""
    from ternary_weight_bit_absmean_b200 import synth
    M, N, K = 96, 512, 256
    X = synth.activations(M, K, seed=1).to(DEV)
    W = synth.weight(N, K, seed=1).to(DEV)
    w = 1 + 0.1 * torch.randn(K, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    gamma, packed = B.quantize_weights(W)
    xq, s = B.norm_quantize_act(X, w, B.BL_NORM_LAYER)
    dY = torch.randn(M, N, device=DEV, generator=torch.Generator(device=DEV).manual_seed(2))
    dXn, dW = B.ste_backward(dY, packed, xq, s, gamma)
    dX, dw, db = B.norm_backward(dXn, X, w, B.BL_NORM_LAYER, bias=True)
    (ex, tx), (ew, tw), (eb, tb) = Exact(X, w, LAYER, 1e-5).backward(dXn)
    close(dX, ex, tx, "dX")
    close(dw, ew, tw, "dw")
    close(db, eb, tb, "db")
    # the quantiser's input is what norm_forward returns, up to the quantiser's half step
    y = B.norm_forward(X, w, kind=B.BL_NORM_LAYER, out_dtype=F32)
    back = xq.double() / s.double()[:, None]
    assert ((y.double() - back).abs() <= (0.5 + 1e-4) / s.double()[:, None]).all()
