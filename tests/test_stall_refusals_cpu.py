"""Refusals of the stall tests of the bounded waits, made on the host before any launch."""
import pytest

pytestmark = pytest.mark.cpu

INVALID, MISALIGNED = 1, 3
FAKE = 1 << 20          # 16-byte aligned, never dereferenced: every case fails validation first


@pytest.fixture(scope="module")
def L():
    from ternary_weight_bit_absmean_b200 import binding, build_lib
    build_lib.build()
    return binding.lib()


def replaced(args, i, v):
    return [*args[:i], v, *args[i + 1:]]


def test_fp8_stall_test_refusals(L):
    f = L.bitlinear_fp8_stall_test
    #       xq    sx    wq    sw    M  N   K    out   type err   limit    stall stream
    good = [FAKE, FAKE, FAKE, FAKE, 4, 64, 128, FAKE, 0, None, 1_000_000, 1, None]
    for i, v, want in [(10, 0, INVALID), (10, 2_000_000_001, INVALID), (11, -1, INVALID), (0, None, INVALID),
                       (4, 0, INVALID), (8, 2, INVALID), (7, FAKE + 4, MISALIGNED)]:
        assert f(*replaced(good, i, v)) == want, (i, v)


def test_norm_backward_stall_test_refusals(L):
    f = L.bitlinear_norm_backward_stall_test
    #       dY    type X     type w     M  K    kind eps   dX    type dw    db    ws    bytes    err   limit      stall stream
    good = [FAKE, 0, FAKE, 0, FAKE, 8, 64, 1, 1e-5, FAKE, 0, FAKE, FAKE, FAKE, 1 << 20, None, 1_000_000, 1, None]
    for i, v, want in [(16, 0, INVALID), (16, 2_000_000_001, INVALID), (17, -1, INVALID), (0, None, INVALID),
                       (5, 0, INVALID), (7, 2, INVALID), (9, FAKE + 4, MISALIGNED)]:
        assert f(*replaced(good, i, v)) == want, (i, v)
