"""Codes whose padding to a multiple of 16 is not zeros: with the true length of the contraction the
products do not read it, through the package as through the C entry points."""
import pytest
import torch

from ternary_weight_bit_absmean_b200 import binding as B

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from ternary_weight_bit_absmean_b200 import build_lib
    build_lib.build()
    B.lib()


def spoil(q, n):
    """Bytes of a NaN and of 1.0 in turn behind the first n codes of every row."""
    b = q.view(torch.uint8)
    b[:, n:] = 0x38
    b[:, n::2] = 0x7F
    return q


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (3, 37, 129), (17, 130, 1543), (77, 200, 257), (300, 1001, 520), (1030, 777, 1031)])
def test_true_length_of_the_contraction(M, N, K):
    g = torch.Generator(device=DEV).manual_seed(M)
    x, w, dy = (torch.randn(*s, generator=g, device=DEV) for s in ((M, K), (N, K), (M, N)))
    xq, sx, xt, sxt = B.fp8_quantize_act(x, transposed=True)
    dq, sd, dt, sdt = B.fp8_quantize_act(dy, transposed=True)
    wq, sw, wt = B.fp8_quantize_weights(w, transposed=True)
    y, dx, dw = B.fp8_forward(xq, sx, wq, sw), B.fp8_backward_input(dq, sd, wt, sw), B.fp8_backward_weight(dt, sdt, xt, sxt)
    for q, n in ((xq, K), (wq, K), (dq, N), (wt, N), (dt, M), (xt, M)):
        spoil(q, n)
    assert torch.equal(B.fp8_forward(xq, sx, wq, sw, K=K), y)
    assert torch.equal(B.fp8_backward_input(dq, sd, wt, sw, N=N), dx)
    assert torch.equal(B.fp8_backward_weight(dt, sdt, xt, sxt, M=M), dw)
    out = torch.empty_like(y)
    B.bitlinear_fp8_forward(xq, sx, wq, sw, out, K=K)
    assert torch.equal(out, y)


def test_lengths_that_rows_do_not_hold():
    x = torch.ones(20, 40, device=DEV)                  # rows of 48 codes
    xq, sx = B.fp8_quantize_act(x)
    wq, sw = B.fp8_quantize_weights(x)
    for bad in (0, -1, 32, 49, 64):
        with pytest.raises(ValueError):
            B.fp8_forward(xq, sx, wq, sw, K=bad)
    assert torch.equal(B.fp8_forward(xq, sx, wq, sw, K=48), B.fp8_forward(xq, sx, wq, sw, K=33 + 7))
