"""The layer norm of rows whose mean is large against their spread, forward and backward, and of
constant rows, against the formulas in 64 bits.

Tolerances.  u = 2^-24, and a sum over a row of K runs over at most `steps` additions one after
the other.  The kernels sum differences from ref, a mean of eight elements of the row (or one of
them), so |ref - mean| <= R = max |x - mean|.  A difference is right to u of itself, so the mean
comes out as mu + lo to
  e = (steps + 4) u (mean|x - mean| + R),   |lo| <= L = u |mean|,
and c = x - mu with |c| <= C = |x - mean| + L + e to u C.  The variance mean c^2 - lo^2 is then off by
  e_v = (steps + 5) u mean C^2 + 2 (L + e) e + 3 u L^2,
r by e_v / 2 (v + eps) of itself and two roundings, n = (c - lo) r by r (u C + e + 2 u L) besides.
Through the gradient these go as the formulas say.  All bounds are first order and doubled for the
higher ones."""
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
LAYER = B.BL_NORM_LAYER
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from ternary_weight_bit_absmean_b200 import build_lib
    build_lib.build()
    B.lib()


def steps(K):
    return max(32, K // 1024 + 1) + 12


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


class Exact:
    def __init__(self, x, w):
        x, self.w = x.double(), w.double()
        self.s = s = steps(x.shape[1])
        mean = x.mean(1, keepdim=True)
        c = x - mean
        v = c.square().mean(1, keepdim=True)
        self.r = 1 / torch.sqrt(v + EPS)
        self.n = c * self.r
        L = U * mean.abs()
        self.e = (s + 4) * U * (c.abs().mean(1, keepdim=True) + c.abs().amax(1, keepdim=True))
        self.lo = L + self.e
        self.C = c.abs() + self.lo
        e_v = (s + 5) * U * self.C.square().mean(1, keepdim=True) + 2 * self.lo * self.e + 3 * U * L ** 2
        self.rho = e_v / (2 * (v + EPS)) + 4 * U
        self.dn = self.r * (U * self.C + self.e + 2 * U * L) + self.n.abs() * self.rho

    def forward(self, b):
        y = self.n * self.w
        tol = self.dn * self.w.abs() + 2 * U * y.abs()
        return y + b.double(), 2 * (tol + U * (y + b.double()).abs())

    def backward(self, dy):
        dy, s = dy.double(), self.s
        g = dy * self.w
        gm = g.abs().mean(1, keepdim=True)
        c1, c2 = (g * self.n).mean(1, keepdim=True), g.mean(1, keepdim=True)
        dx = self.r * (g - c2 - self.n * c1)
        dc2 = (s + 3) * U * gm
        dc1 = self.r * ((s + 6) * U * (g.abs() * self.C).mean(1, keepdim=True) + self.e * c2.abs()
                        + self.lo * (s + 6) * U * gm) + c1.abs() * self.rho
        mag = g.abs() + c2.abs() + (self.n * c1).abs()
        tx = self.r * ((self.rho + 4 * U) * mag + dc2 + self.n.abs() * dc1 + c1.abs() * self.dn)
        deep = (dy.shape[0] // 148 + 64) * U  # rows in order, groups, parts in strips and a tree
        tw = (dy.abs() * self.dn).sum(0) + deep * (dy * self.n).abs().sum(0)
        return (dx, 2 * tx), ((dy * self.n).sum(0), 2 * tw), (dy.sum(0), 2 * deep * dy.abs().sum(0))


def close(got, want, tol, what):
    tol = tol + torch.finfo(got.dtype).eps / 2 * want.abs() + 1e-37
    err = (got.double() - want).abs()
    assert (err <= tol).all(), "%s: %g of the tolerance at worst" % (what, (err / tol).max().item())


def check(x, seed, what):
    M, K = x.shape
    w, b = 1 + 0.1 * torch.randn(K, generator=gen(seed), device=DEV), 0.1 * torch.randn(K, generator=gen(seed + 1), device=DEV)
    e = Exact(x, w)
    y = guarded_empty((M, K), F32)
    B.bitlinear_norm_forward(x, w, b, LAYER, EPS, y)
    close(y, *e.forward(b), "y " + what)
    check_guard(y)
    dy = torch.randn(M, K, generator=gen(seed + 2), device=DEV) + 0.5  # its own mean: lo enters c1
    (dx, tx), (dw, tw), (db, tb) = e.backward(dy)
    gx, gw, gb = B.norm_backward(dy, x, w, LAYER, EPS, bias=True, dx_dtype=F32)
    close(gx, dx, tx, "dx " + what)
    close(gw, dw, tw, "dw " + what)
    close(gb, db, tb, "db " + what)
    hx, hw, hb = B.norm_backward(dy, x, w, LAYER, EPS, dx_dtype=F32)
    assert hb is None and torch.equal(hx, gx) and torch.equal(hw, gw)


# widths of every layout: groups of a warp, one to three chunks, whole chunks or not, clusters,
# rows that a block reads again
WIDTHS = [(700, 200), (5, 1000), (64, 1536), (33, 1537), (300, 3200), (160, 4097), (9, 5120), (160, 8192), (9, 8999),
          (5, 12816), (3, 16389), (3, 40000), (2, 80003)]


@pytest.mark.parametrize("M,K", WIDTHS)
@pytest.mark.parametrize("mean,spread", [(1000.0, 0.01), (-1e4, 0.1), (3e5, 1.0)])
def test_mean_far_above_the_spread(M, K, mean, spread):
    x = mean + spread * torch.randn(M, K, generator=gen(K), device=DEV, dtype=torch.float64)
    check(x.float(), K, "%g +- %g" % (mean, spread))


@pytest.mark.parametrize("M,K", WIDTHS + [(900, 1544), (900, 3208), (600, 8184)])
def test_bf16_rows_nearly_constant(M, K):
    """1000, and 1008 (two steps of the type further) in some places."""
    x = 1000.0 + 8.0 * (torch.rand(M, K, generator=gen(K), device=DEV) < 1e-2).float()
    check(x.to(BF16), K, "bf16")


@pytest.mark.parametrize("K", [96, 1000, 1537, 3200, 8191, 9713, 16384, 40000, 80003])
def test_constant_rows(K):
    values = torch.tensor([7.0, 1000.0, 1e4 / 3, -0.1, 1e18, -1e30], device=DEV)
    x = values[:, None].expand(-1, K).contiguous()
    assert not B.norm_forward(x, kind=LAYER).any()  # c and lo are zero
    check(x[:4].contiguous(), K, "constant")
    dx, dw, db = B.norm_backward(torch.ones_like(x), x, kind=LAYER, bias=True)
    assert torch.isfinite(dx).all() and dw is None and torch.equal(db, torch.full_like(db, len(values)))


def test_one_value_beside_constants():
    """(K - 1) of one value and a neighbouring one: n is sqrt(K - 1) there."""
    K = 4000
    x = torch.full((2, K), 1000.0, device=DEV)
    x[0, 7], x[1, K - 1] = 1000.0625, 999.0
    check(x, 3, "one value")
    y = B.norm_forward(x, kind=LAYER)
    assert abs(y[1, K - 1].item() + (K - 1) ** 0.5) < 0.05 * K ** 0.5  # eps 1e-5 against a variance of 2.5e-4
