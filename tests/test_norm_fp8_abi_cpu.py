"""Refusals of the norm and e4m3 entry points, made on the host before any launch, and the
Python binding's argument checks (no GPU needed)."""
import pytest
import torch

pytestmark = pytest.mark.cpu

BL_OK, INVALID, SHAPE, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4
F32, BF16, I32 = 0, 1, 2
RMS, LAYER = 0, 1
FAKE = 1 << 20          # 16-byte aligned, never dereferenced: every case fails validation first
ODD = FAKE + 4
BIG = (1 << 30) + 1


@pytest.fixture(scope="module")
def L():
    from ternary_weight_bit_absmean_b200 import binding, build_lib
    build_lib.build()
    return binding.lib()


def replaced(args, i, v):
    return [*args[:i], v, *args[i + 1:]]


def test_norm_forward_refusals(L):
    f = L.bitlinear_norm_forward
    #       X     type  w     b     M  K   kind eps   Y     type stream
    good = [FAKE, BF16, FAKE, FAKE, 8, 64, RMS, 1e-5, FAKE, BF16, None]
    for i, v, want in [(0, None, INVALID), (1, I32, INVALID), (1, 7, INVALID), (4, 0, INVALID), (5, -1, INVALID),
                       (4, BIG, SHAPE), (5, BIG, SHAPE), (6, 2, INVALID), (7, -1.0, INVALID),
                       (7, float("nan"), INVALID), (7, float("inf"), INVALID), (8, None, INVALID), (9, I32, INVALID),
                       (0, ODD, MISALIGNED), (2, ODD, MISALIGNED), (3, ODD, MISALIGNED), (8, ODD, MISALIGNED)]:
        assert f(*replaced(good, i, v)) == want, (i, v)
    assert f(*replaced(replaced(good, 4, 1 << 21), 5, 1 << 20)) == SHAPE  # M K > 2^40


def test_norm_backward_refusals(L):
    f = L.bitlinear_norm_backward
    need = L.bitlinear_norm_backward_workspace_size(64, 512)
    assert need > 0
    #       dY    type X     type  w     M   K    kind   eps   dX    type dw    db    ws    bytes err   stream
    good = [FAKE, F32, FAKE, BF16, FAKE, 64, 512, LAYER, 1e-5, FAKE, F32, FAKE, FAKE, FAKE, need, None, None]
    for i, v, want in [(0, None, INVALID), (1, I32, INVALID), (2, None, INVALID), (3, I32, INVALID), (5, 0, INVALID),
                       (6, 0, INVALID), (5, BIG, SHAPE), (6, BIG, SHAPE), (7, 5, INVALID), (8, -1.0, INVALID),
                       (9, None, INVALID), (10, I32, INVALID), (0, ODD, MISALIGNED), (2, ODD, MISALIGNED),
                       (4, ODD, MISALIGNED), (9, ODD, MISALIGNED), (11, ODD, MISALIGNED), (12, ODD, MISALIGNED),
                       (13, ODD, MISALIGNED), (13, None, WORKSPACE), (14, need - 1, WORKSPACE)]:
        assert f(*replaced(good, i, v)) == want, (i, v)


def test_norm_backward_workspace_size(L):
    f = L.bitlinear_norm_backward_workspace_size
    assert f(0, 64) == 0 and f(64, 0) == 0 and f(BIG, 4) == 0
    assert f(1, 512) == 0                      # one row: its sums are the result
    sizes = [f(m, 4096) for m in (1, 8, 64, 512, 4096, 1 << 20)]
    assert sizes == sorted(sizes)
    assert f(1 << 20, 4096) == f(4096, 4096)   # bounded by the blocks that fill a GPU


def test_fp8_row_bytes(L):
    assert [L.bitlinear_fp8_row_bytes(k) for k in (-1, 0, 1, 15, 16, 17, 8640)] == [0, 0, 16, 16, 16, 32, 8640]


def test_fp8_quantize_refusals(L):
    f = L.bitlinear_fp8_quantize_act
    #       X     type  M  K   eps   xq    s     xqt   st    stream
    good = [FAKE, BF16, 8, 64, 1e-5, FAKE, FAKE, FAKE, FAKE, None]
    for i, v, want in [(0, None, INVALID), (1, I32, INVALID), (2, 0, INVALID), (3, 0, INVALID), (2, BIG, SHAPE),
                       (3, BIG, SHAPE), (4, 0.0, INVALID), (4, 1e-31, INVALID), (4, float("inf"), INVALID),
                       (4, float("nan"), INVALID), (5, None, INVALID), (6, None, INVALID), (7, None, INVALID),
                       (8, None, INVALID), (0, ODD, MISALIGNED), (5, ODD, MISALIGNED), (6, ODD, MISALIGNED),
                       (7, ODD, MISALIGNED), (8, ODD, MISALIGNED)]:
        assert f(*replaced(good, i, v)) == want, (i, v)
    assert f(FAKE, BF16, 8, 64, 1e-5, None, None, None, None, None) == INVALID
    f = L.bitlinear_fp8_quantize_weights
    #       W     type N  K   eps   wq    s     wqt   stream
    good = [FAKE, F32, 8, 64, 1e-5, FAKE, FAKE, FAKE, None]
    for i, v, want in [(0, None, INVALID), (1, I32, INVALID), (2, 0, INVALID), (3, 0, INVALID), (2, BIG, SHAPE),
                       (4, -1.0, INVALID), (6, None, INVALID), (0, ODD, MISALIGNED), (5, ODD, MISALIGNED),
                       (6, ODD, MISALIGNED), (7, ODD, MISALIGNED)]:
        assert f(*replaced(good, i, v)) == want, (i, v)
    assert f(FAKE, F32, 8, 64, 1e-5, None, FAKE, None, None) == INVALID


@pytest.mark.parametrize("name", ["bitlinear_fp8_forward", "bitlinear_fp8_backward_input",
                                  "bitlinear_fp8_backward_weight"])
def test_fp8_product_refusals(L, name):
    f = getattr(L, name)
    good = [FAKE, FAKE, FAKE, FAKE, 8, 64, 128, FAKE, BF16, None, None]
    for i in (0, 1, 2, 3, 7):
        assert f(*replaced(good, i, None)) == INVALID
        assert f(*replaced(good, i, ODD)) == MISALIGNED
    for i in (4, 5, 6):
        assert f(*replaced(good, i, 0)) == INVALID
        assert f(*replaced(good, i, BIG)) == SHAPE
    assert f(*replaced(good, 8, I32)) == INVALID
    assert f(*replaced(replaced(good, 4, 1 << 21), 5, 1 << 20)) == SHAPE


def test_binding_refuses_cpu_tensors():
    from ternary_weight_bit_absmean_b200 import binding as B
    x = torch.zeros(4, 16)
    for call in [lambda: B.norm_forward(x), lambda: B.norm_backward(x, x), lambda: B.fp8_quantize_act(x),
                 lambda: B.fp8_quantize_weights(x),
                 lambda: B.fp8_forward(x.to(torch.float8_e4m3fn), x, x.to(torch.float8_e4m3fn), x)]:
        with pytest.raises(TypeError):
            call()


def test_package_exports_the_operators():
    import ternary_weight_bit_absmean_b200 as bl
    for name in ["norm_forward", "norm_backward", "fp8_quantize_act", "fp8_quantize_weights", "fp8_forward",
                 "fp8_backward_input", "fp8_backward_weight", "BL_NORM_RMS", "BL_NORM_LAYER"]:
        assert hasattr(bl, name)
