"""The bounded waits of the 8-bit products: each block's load producer stops after a few loads and
every wait is limited to 1 ms.  The waits for the next load run out, the kernel ends with what is in
flight waited for, reports BL_ERRBIT_TIMEOUT and returns; the next call on the stream gives the bits
that it gave before."""
import pytest
import torch

from gpu_util import check_guard, guarded_empty
from ternary_weight_bit_absmean_b200 import binding as B

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = "cuda"
LIMIT = 1_000_000  # 1 ms


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from ternary_weight_bit_absmean_b200 import build_lib
    build_lib.build()
    B.lib()


def problem(M, N, K):
    g = torch.Generator(device=DEV).manual_seed(M + N + K)
    x, w = torch.randn(M, K, generator=g, device=DEV), 0.02 * torch.randn(N, K, generator=g, device=DEV)
    return B.fp8_quantize_act(x) + B.fp8_quantize_weights(w)


# one shape for every form: 16, 32, 64 and 128 tokens a tile, one block or a cluster to a tile, pairs
# of SMs with tiles of 128 and of 256 columns and with several tiles of a pair one after the other
FORMS = [(3, 28672, 4096), (16, 1024, 8192), (30, 1024, 4096), (60, 1024, 8192), (128, 1024, 8192), (100, 18000, 1024),
         (512, 4096, 1536), (2304, 5000, 1024), (4096, 8192, 640)]


@pytest.mark.parametrize("stall", [0, 1, 3])
@pytest.mark.parametrize("M,N,K", FORMS)
def test_waits_run_out_then_the_next_call_is_right(M, N, K, stall):
    ops = problem(M, N, K)
    want = B.fp8_forward(*ops)
    out = guarded_empty((M, N), torch.float32)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.bitlinear_fp8_stall_test(*ops, out, err, LIMIT, stall)
    torch.cuda.synchronize()
    check_guard(out)
    assert err.item() == B.BL_ERRBIT_TIMEOUT
    for _ in range(2):
        err.zero_()
        assert torch.equal(B.fp8_forward(*ops, err_word=err), want)
        assert err.item() == 0


@pytest.mark.parametrize("M,N,K", [(3, 28672, 4096), (60, 1024, 8192), (512, 4096, 1536)])
def test_a_stall_no_block_reaches_changes_nothing(M, N, K):
    ops = problem(M, N, K)
    out = torch.empty(M, N, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.bitlinear_fp8_stall_test(*ops, out, err, 2_000_000_000, 1 << 20)
    assert torch.equal(out, B.fp8_forward(*ops)) and err.item() == 0


def test_without_an_error_word():
    ops = problem(300, 1024, 1024)
    want = B.fp8_forward(*ops)
    B.bitlinear_fp8_stall_test(*ops, torch.empty_like(want), None, LIMIT, 1)
    assert torch.equal(B.fp8_forward(*ops), want)
