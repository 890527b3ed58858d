"""The e4m3 quantisers and the 8-bit block-scaled products against the definitions in 64 bits.

Codes and scales are compared for equality: the quotients and the product of the definition
are single IEEE fp32 operations, which 64-bit arithmetic followed by a rounding to fp32
reproduces (53 bits are more than twice 24), and the rounding to e4m3 is to nearest even.

Products.  u = 2^-24.  Products of codes are exact; a group's 128 of them are added in fp32
by the tensor cores, in an order and with a rounding of their own (at most 2 u of the
magnitudes per addition: 256 u), the two scales and their product round three times, and the
G groups, and up to 8 partial sums, are added in fp32: (256 + 4 + G + 8) u of
sum |x w| in all, and half a step of the output type."""
import pytest
import torch

from gpu_util import check_guard, guarded_empty
from ternary_weight_bit_absmean_b200 import binding as B

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = "cuda"
U = 2.0 ** -24
F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from ternary_weight_bit_absmean_b200 import build_lib
    build_lib.build()
    B.lib()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def acts(M, K, seed, dtype=F32):
    g = gen(seed)
    x = torch.randn(M, K, generator=g, device=DEV) * torch.exp(torch.randn(M, 1, generator=g, device=DEV))
    return (x * torch.where(torch.rand(K, generator=g, device=DEV) < 0.01, 20.0, 1.0)).to(dtype)


def up16(n):
    return -(-n // 16) * 16


def blocks(n):
    return -(-n // 128)


# ------------------------------------------------------------ the definition in 64 bits --

def to_e4m3(v):
    """The nearest e4m3 value of v in 64 bits, ties to even, NaN kept."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def f32(v):
    return v.float().double()


def definition(x, rows, cols, eps):
    """(codes as 64-bit values, scales [row blocks, column blocks]) for blocks of rows x cols."""
    R, C = x.shape
    x = x.double()
    p = torch.nn.functional.pad(x.abs(), (0, blocks(C) * cols - C if cols > 1 else 0,
                                          0, blocks(R) * rows - R if rows > 1 else 0))
    a = p.view(p.shape[0] // rows, rows, p.shape[1] // cols, cols).amax((1, 3))  # keeps NaN
    m = torch.where(a < float(torch.tensor(eps, dtype=F32)), float(torch.tensor(eps, dtype=F32)), a)
    d, ratio = f32(m / 448.0), f32(448.0 / m)
    full = ratio.repeat_interleave(rows, 0)[:R].repeat_interleave(cols, 1)[:, :C]
    return to_e4m3(f32(x * full)), d


def same(a, b):
    return torch.equal(torch.nan_to_num(a.double(), nan=1234.0, posinf=2345.0), torch.nan_to_num(b.double(), nan=1234.0, posinf=2345.0)) \
        and torch.equal(torch.isnan(a.float()), torch.isnan(b.float()))


def check_codes(got, want, n):
    """Codes of n elements a row, and zero bytes behind them."""
    assert got.shape == (want.shape[0], up16(n))
    assert same(got[:, :n].float(), want)
    assert not got.view(torch.uint8)[:, n:].any()


def check_act(x, eps=1e-5):
    M, K = x.shape
    xq, sx = guarded_empty((M, up16(K)), E4M3), guarded_empty((blocks(K), M), F32)
    xt, st = guarded_empty((K, up16(M)), E4M3), guarded_empty((blocks(M), K), F32)
    q, d = definition(x, 1, 128, eps)
    B.bitlinear_fp8_quantize_act(x, eps, xq, sx)
    check_codes(xq, q, K)
    assert same(sx, d.t())
    B.bitlinear_fp8_quantize_act(x, eps, None, None, xt, st)
    qt, dt = definition(x.t(), 1, 128, eps)
    check_codes(xt, qt, M)
    assert same(st, dt.t())
    both = B.fp8_quantize_act(x, eps, transposed=True)
    for got, want in zip(both, (xq, sx, xt, st)):
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    for t in (xq, sx, xt, st):
        check_guard(t)


def check_weights(w, eps=1e-5):
    N, K = w.shape
    q, d = definition(w, 128, 128, eps)
    wq, wt, sw = guarded_empty((N, up16(K)), E4M3), guarded_empty((K, up16(N)), E4M3), guarded_empty((blocks(N), blocks(K)), F32)
    B.bitlinear_fp8_quantize_weights(w, eps, wq, sw, wt)
    check_codes(wq, q, K)
    check_codes(wt, q.t(), N)
    assert same(sw, d)
    for t in (wq, wt, sw):
        check_guard(t)
    a, s = B.fp8_quantize_weights(w, eps)
    assert torch.equal(a.view(torch.uint8), wq.view(torch.uint8)) and same(s, sw)
    sw2, wt2 = torch.empty_like(sw), torch.empty_like(wt)
    B.bitlinear_fp8_quantize_weights(w, eps, None, sw2, wt2)
    assert torch.equal(wt2.view(torch.uint8), wt.view(torch.uint8)) and same(sw2, sw)


SIZES = [(1, 1), (1, 128), (2, 5), (3, 127), (16, 129), (17, 130), (127, 256), (128, 128), (129, 132), (130, 1543),
         (1, 8192), (16, 3200), (300, 520), (33, 28672), (1000, 257)]


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantisers(M, K, dtype):
    check_act(acts(M, K, seed=M + K, dtype=dtype))
    check_weights(0.02 * acts(M, K, seed=M * K, dtype=dtype).contiguous())


def test_quantiser_edges():
    x = acts(140, 300, seed=1)
    x[0], x[1, :128], x[2] = 0.0, 0.0, 1e-20            # below eps: the scale is eps / 448
    x[3, 5], x[4, 200], x[5, 299] = float("nan"), float("inf"), float("-inf")
    x[6], x[7] = 3.0e38, -0.0
    check_act(x)
    check_act(x, eps=1e-30)
    check_weights(x)
    # every tie between neighbouring codes, and the codes themselves
    grid = torch.arange(0, 0x7F, dtype=torch.uint8, device=DEV).view(E4M3).float()
    ties = torch.cat([grid, (grid[1:] + grid[:-1]) / 2])
    x = torch.zeros(2, 256, device=DEV)
    x[0, :ties.numel()], x[1, :ties.numel()] = ties, -ties
    x[:, 127::128] = 448.0                               # ratio 1 in every group
    check_act(x)


# --------------------------------------------------------------------------- products --

def rows_of(q, s, n):
    return q[:, :n].double() * s.double().t().repeat_interleave(128, 1)[:, :n]


def blocks_of(q, s, n):
    return q[:, :n].double() * s.double().repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :n]


def close(got, a, b, what):
    want = a @ b.t()
    tol = (256 + 12 + blocks(a.shape[1])) * U * (a.abs() @ b.abs().t()) + torch.finfo(got.dtype).eps / 2 * want.abs()
    err = (got.double() - want).abs()
    assert (err <= tol).all(), "%s: %g of the tolerance at worst" % (what, (err / tol).max().item())


def problem(M, N, K, seed):
    x, w = acts(M, K, seed), 0.02 * acts(N, K, seed + 1)
    dy = 1e-3 * acts(M, N, seed + 2)
    return x, w, dy


def check_products(M, N, K, seed=0):
    x, w, dy = problem(M, N, K, seed)
    xq, sx, xt, sxt = B.fp8_quantize_act(x, transposed=True)
    dq, sd, dt, sdt = B.fp8_quantize_act(dy, 1e-12, transposed=True)
    wq, sw, wt = B.fp8_quantize_weights(w, transposed=True)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for t in (F32, BF16):
        y, dx, dw = guarded_empty((M, N), t), guarded_empty((M, K), t), guarded_empty((N, K), t)
        raw(B.lib().bitlinear_fp8_forward, xq, sx, wq, sw, M, N, K, y, err)
        raw(B.lib().bitlinear_fp8_backward_input, dq, sd, wt, sw, M, N, K, dx, err)
        raw(B.lib().bitlinear_fp8_backward_weight, dt, sdt, xt, sxt, M, N, K, dw, err)
        close(y, rows_of(xq, sx, K), blocks_of(wq, sw, K), "y")
        close(dx, rows_of(dq, sd, N), blocks_of(wt, sw.t(), N), "dX")
        close(dw, rows_of(dt, sdt, M), rows_of(xt, sxt, M), "dW")
        for o in (y, dx, dw):
            check_guard(o)
        # the binding takes the padded row length for the contraction's: same results
        assert torch.equal(B.fp8_forward(xq, sx, wq, sw, t), y)
        assert torch.equal(B.fp8_backward_input(dq, sd, wt, sw, t), dx)
        assert torch.equal(B.fp8_backward_weight(dt, sdt, xt, sxt, t), dw)
    assert err.item() == 0


def raw(f, q, sq, p, sp, M, N, K, out, err):
    """A product through the C entry point with the true (unpadded) sizes."""
    st = f(q.data_ptr(), sq.data_ptr(), p.data_ptr(), sp.data_ptr(), M, N, K, out.data_ptr(),
           B.BL_OUT_BF16 if out.dtype == BF16 else B.BL_OUT_F32, err.data_ptr(),
           torch.cuda.current_stream().cuda_stream)
    assert st == B.BL_OK


@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 16, 128), (2, 3, 5), (1, 129, 127), (1, 1024, 8192), (3, 28672, 520), (16, 3200, 3200),
    (17, 200, 1543), (32, 512, 256), (33, 130, 257), (64, 1536, 4096), (77, 4099, 1543), (128, 128, 128),
    (129, 257, 385), (200, 100, 8640), (257, 1000, 300), (300, 2000, 640), (1000, 520, 2000), (1537, 777, 1031),
    (2048, 3200, 1536)])
def test_products(M, N, K):
    check_products(M, N, K, seed=M)


# One shape for every form the products choose between: token tiles of 16 to 128 with and without a
# split of the contraction, tiles of 256 x 128 and 256 x 256, one round of tiles and several.
@pytest.mark.parametrize("M,N,K", [
    (5, 28700, 1000), (16, 1024, 8192), (30, 129, 2048), (60, 3000, 1100), (100, 1024, 4099), (130, 8192, 300),
    (512, 4096, 1536), (1000, 9000, 256), (2304, 5000, 400), (257, 19000, 129)])
def test_every_form_of_the_products(M, N, K):
    check_products(M, N, K, seed=N)


def test_tall_and_flat_weight_gradients():
    """dW = dY^T x with few outputs and many tokens, and the reverse."""
    for M, N, K in [(20000, 130, 70), (3, 2100, 1800), (129, 4000, 260)]:
        x, _, dy = problem(M, N, K, 3)
        _, _, xt, sxt = B.fp8_quantize_act(x, transposed=True)
        _, _, dt, sdt = B.fp8_quantize_act(dy, 1e-12, transposed=True)
        close(B.fp8_backward_weight(dt, sdt, xt, sxt), rows_of(dt, sdt, M), rows_of(xt, sxt, M), (M, N, K))


def test_group_sums_keep_fp32_digits():
    """Large products that cancel within a group next to small ones: what the accumulation
    keeps of the small ones is bounded by the fp32 rounding of the large ones' magnitude."""
    M, N, K = 128, 256, 256
    a = torch.full((M, K), 448.0, device=DEV)
    a[:, 1::2] = -448.0
    a[:, 6::32] = 2.0 ** -6
    b = torch.full((N, K), 448.0, device=DEV)
    b[:, 6::32] = 2.0 ** -6
    a[:, 7::32] = 0.0
    q, s = a.to(E4M3), torch.ones(2, M, device=DEV)
    y = B.fp8_forward(q, s, b.to(E4M3), torch.ones(2, 2, device=DEV))
    close(y, a.double(), b.double(), "cancelling sums")


def test_gradients_against_differences():
    """The products are linear in the values that the codes stand for, so the differences of
    L = sum dY (x w^T) in those values are the gradients themselves."""
    M, N, K = 9, 20, 33
    x, w, dy = problem(M, N, K, 5)
    xq, sx, xt, sxt = B.fp8_quantize_act(x, transposed=True)
    dq, sd, dt, sdt = B.fp8_quantize_act(dy, 1e-12, transposed=True)
    wq, sw, wt = B.fp8_quantize_weights(w, transposed=True)
    gx = B.fp8_backward_input(dq, sd, wt, sw)[:, :K]
    gw = B.fp8_backward_weight(dt, sdt, xt, sxt)
    W, D, X, DW = blocks_of(wq, sw, K), rows_of(dq, sd, N), rows_of(xt, sxt, M).t(), rows_of(dt, sdt, M).t()
    loss = lambda x, w, d: (d * (x @ w.t())).sum()  # noqa: E731
    x0 = rows_of(xq, sx, K)
    for i, j in [(0, 0), (4, 17), (8, 32)]:
        e = torch.zeros_like(x0)
        e[i, j] = 0.5
        want = loss(x0 + e, W, D) - loss(x0 - e, W, D)
        assert abs(gx[i, j].item() - want.item()) <= 300 * U * (D[i].abs() @ W[:, j].abs()).item() + 1e-12
    for i, j in [(0, 0), (7, 17), (19, 32)]:
        e = torch.zeros_like(W)
        e[i, j] = 0.5
        want = loss(X, W + e, DW) - loss(X, W - e, DW)
        assert abs(gw[i, j].item() - want.item()) <= 300 * U * (DW[:, i].abs() @ X[:, j].abs()).item() + 1e-12


@pytest.mark.parametrize("M", [3, 70, 700])
def test_non_finite_values_reach_their_row(M):
    N, K = 300, 640
    x, w, _ = problem(M, N, K, 6)
    x[1, 200], x[2, 639] = float("nan"), float("inf")
    xq, sx = B.fp8_quantize_act(x)
    wq, sw = B.fp8_quantize_weights(w)
    y = B.fp8_forward(xq, sx, wq, sw)
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()
    rest = [i for i in range(M) if i not in (1, 2)]
    assert torch.isfinite(y[rest]).all()
    w[131, 5] = float("nan")                           # its 128 x 128 block: columns 128 .. 255
    wq, sw = B.fp8_quantize_weights(w)
    y = B.fp8_forward(xq, sx, wq, sw)
    assert torch.isnan(y[0, 128:256]).all() and torch.isfinite(y[0, :128]).all() and torch.isfinite(y[0, 256:]).all()


@pytest.mark.parametrize("M", [1, 48, 600])
def test_results_repeat_on_several_streams_at_once(M):
    N, K = 1030, 3200
    x, w, dy = problem(M, N, K, 7)
    ops = B.fp8_quantize_act(x) + B.fp8_quantize_weights(w)
    want = B.fp8_forward(*ops)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [B.fp8_forward(*ops, stream=s) for _ in range(4) for s in streams]
    codes = [B.fp8_quantize_act(x, transposed=True, stream=s) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    assert all(torch.equal(c[0].view(torch.uint8), ops[0].view(torch.uint8)) and torch.equal(c[1], ops[1]) for c in codes)


@pytest.mark.parametrize("M", [1, 600])
def test_captured_and_replayed_on_new_inputs(M):
    N, K = 640, 1543
    x, w, dy = problem(M, N, K, 8)

    def step():
        xq, sx, xt, sxt = B.fp8_quantize_act(x, transposed=True)
        wq, sw, wt = B.fp8_quantize_weights(w, transposed=True)
        dq, sd, dt, sdt = B.fp8_quantize_act(dy, 1e-12, transposed=True)
        return (B.fp8_forward(xq, sx, wq, sw), B.fp8_backward_input(dq, sd, wt, sw),
                B.fp8_backward_weight(dt, sdt, xt, sxt))

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for t, v in zip((x, w, dy), problem(M, N, K, 9)):
        t.copy_(v)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_offsets_past_32_bits():
    M, N, K = 65600, 65568, 16                          # 4.3e9 outputs
    x, w = acts(256, K, 10), acts(N, K, 11)
    xq, sx = B.fp8_quantize_act(x)
    wq, sw = B.fp8_quantize_weights(w)
    tail = B.fp8_forward(xq, sx, wq, sw, BF16)
    X = torch.zeros(M, K, device=DEV)
    X[-256:] = x
    Xq, sX = B.fp8_quantize_act(X)
    y = B.fp8_forward(Xq, sX, wq, sw, BF16)
    assert torch.equal(y[-256:], tail) and not y[:256].any()
    del y
    rows = 300000                                       # 2.4e9 codes, both orientations
    big = torch.zeros(rows, 8192, dtype=BF16, device=DEV)
    big[-40:] = acts(40, 8192, 12, BF16)
    q, s, qt, st = B.fp8_quantize_act(big, transposed=True)
    a, sa = B.fp8_quantize_act(big[-40:].contiguous())
    assert torch.equal(q[-40:].view(torch.uint8), a.view(torch.uint8)) and torch.equal(s[:, -40:], sa)
    # 300000 = 2343 * 128 + 96: the last group of every column is its last 96 rows
    want, d = definition(big[-96:, -8:].t(), 1, 128, 1e-5)
    assert same(qt[-8:, -96:].float(), want) and same(st[-1:, -8:].t(), d)


def test_refusals():
    x = torch.ones(32, 64, device=DEV)
    xq, sx = B.fp8_quantize_act(x)
    wq, sw, wt = B.fp8_quantize_weights(x, transposed=True)
    with pytest.raises(TypeError):
        B.fp8_quantize_act(x.half())
    with pytest.raises(ValueError):
        B.fp8_quantize_act(x.t())
    with pytest.raises(ValueError):
        B.fp8_quantize_act(x[0])
    with pytest.raises(B.BitLinearError):
        B.fp8_quantize_act(x, eps=0.0)
    with pytest.raises(B.BitLinearError):
        B.fp8_quantize_act(torch.empty(0, 64, device=DEV))
    with pytest.raises(TypeError):
        B.fp8_forward(xq.view(torch.uint8), sx, wq, sw)
    with pytest.raises(ValueError):
        B.fp8_forward(xq, sx.t().contiguous(), wq, sw)
    with pytest.raises(ValueError):
        B.fp8_forward(xq, sx, wt, sw)                   # rows of 32 codes against rows of 64
    with pytest.raises(ValueError):
        B.fp8_forward(xq, sx, wq[:, :32], sw)
    with pytest.raises(TypeError):
        B.fp8_forward(xq, sx, wq, sw, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        B.fp8_forward(xq, sx.cpu(), wq, sw)
    with pytest.raises(TypeError):
        B.bitlinear_fp8_forward(xq, sx, wq, sw, torch.empty(32, 32, device=DEV, dtype=torch.int32))


def test_head_with_its_norm_forward_and_backward():
    """norm -> codes -> product, and the gradient back through the product and the norm."""
    M, N, K = 200, 1000, 520
    g = gen(13)
    X = acts(M, K, 13, BF16)
    w = 1 + 0.1 * torch.randn(K, generator=g, device=DEV)
    W = 0.02 * torch.randn(N, K, generator=g, device=DEV)
    dY = 1e-3 * torch.randn(M, N, generator=g, device=DEV)
    n = B.norm_forward(X, w, out_dtype=F32)
    xq, sx, xt, sxt = B.fp8_quantize_act(n, transposed=True)
    wq, sw, wt = B.fp8_quantize_weights(W, transposed=True)
    y = B.fp8_forward(xq, sx, wq, sw)
    dq, sd, dt, sdt = B.fp8_quantize_act(dY, 1e-12, transposed=True)
    dn = B.fp8_backward_input(dq, sd, wt, sw)
    dW = B.fp8_backward_weight(dt, sdt, xt, sxt)
    dX, dw, _ = B.norm_backward(dn, X, w)

    # the same in 64 bits without any 8-bit rounding: each code is within 2^-4 relative of its
    # value (plus half the smallest step, 2^-10 of a scale), so each product is within 2^-3 and
    # a little of the magnitudes' product
    x = X.double()
    r = 1 / torch.sqrt(x.square().mean(1, keepdim=True) + 1e-5)
    ln = x * r * w.double()
    close_to = lambda got, a, b, f: bool(((got.double() - a @ b).abs() <= f * (a.abs() @ b.abs()) + 1e-9).all())  # noqa: E731
    assert close_to(y, ln, W.double().t(), 0.13)
    assert close_to(dW, dY.double().t(), ln, 0.13)
    assert close_to(dn, dY.double(), W.double(), 0.13)
    gn = dY.double() @ W.double() * w.double()
    want = r * (gn - x * r * (gn * x * r).mean(1, keepdim=True))
    rel = (dX.double() - want).norm() / want.norm()
    assert rel <= 2 * 2.0 ** -4, rel                     # two roundings of at most half a step
    rel = (dw.double() - ((dY.double() @ W.double()) * x * r).sum(0)).norm() / ((dY.double() @ W.double()) * x * r).sum(0).norm()
    assert rel <= 2 * 2.0 ** -4, rel
