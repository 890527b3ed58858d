"""What the 8-bit products' sums keep: small products beside large ones that cancel.

u = 2^-24.  Per group of 128, +448^2 and -448^2 stand next to 126 products of 4 = 2 * 2.  Sums that
keep fp32 digits are off by at most (256 + 4) u of the magnitudes per group and (G + 8) u for the
adding of G groups (the bound of the products' other tests), about 6.5 a group, where the small
products add up to 504.  A sum of 14 bits at that magnitude counts in steps of 32, in which a product of 4
is lost, and its total with it."""
import pytest
import torch

from ternary_weight_bit_absmean_b200 import binding as B

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from ternary_weight_bit_absmean_b200 import build_lib
    build_lib.build()
    B.lib()


def operands(M, N, K, plus, minus):
    a, b = torch.full((M, K), 2.0, device=DEV), torch.full((N, K), 2.0, device=DEV)
    a[:, plus::128], a[:, minus::128] = 448.0, -448.0
    b[:, plus::128] = b[:, minus::128] = 448.0
    return a, b


def check(got, a, b):
    groups = a.shape[1] // 128
    want = a.double() @ b.double().t()
    tol = (256 + 12 + groups) * U * (a.double().abs() @ b.double().abs().t())
    assert want.min() > 50 * tol.max()  # a result without the small products fails
    err = (got.double() - want).abs()
    assert (err <= tol).all(), "%g of the tolerance" % (err / tol).max().item()


# the two large products in one MMA of 32 or in different ones, before and behind the small ones
@pytest.mark.parametrize("plus,minus", [(0, 1), (0, 127), (127, 0), (31, 32), (64, 65), (126, 127)])
# 16 to 128 tokens a tile, with a cluster to a tile and without, and pairs of SMs
@pytest.mark.parametrize("M,N,K", [(1, 256, 128), (16, 1024, 8192), (30, 256, 512), (60, 1024, 4096), (100, 18000, 512),
                                   (512, 4096, 1536), (4096, 8192, 640)])
def test_small_products_beside_large_ones(M, N, K, plus, minus):
    a, b = operands(M, N, K, plus, minus)
    G = K // 128
    one = lambda *s: torch.ones(*s, device=DEV)  # noqa: E731
    aq, bq = a.to(torch.float8_e4m3fn), b.to(torch.float8_e4m3fn)
    check(B.fp8_forward(aq, one(G, M), bq, one(-(-N // 128), G)), a, b)
    check(B.fp8_backward_input(aq, one(G, M), bq, one(G, -(-N // 128))), a, b)
    check(B.fp8_backward_weight(aq, one(G, M), bq, one(G, N)), a, b)
