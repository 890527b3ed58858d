"""The bounded waits of the norm's backward: the warp that loads a block's rows stops after a few loads
and every wait is limited to 1 ms.  The waits for the next load, and the cluster's for a block's row
sums, run out; the kernel comes to its end, reports BL_ERRBIT_TIMEOUT and returns; the next call on the
stream gives the bits that it gave before."""
import pytest
import torch

from gpu_util import check_guard, guarded_empty
from ternary_weight_bit_absmean_b200 import binding as B

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = "cuda"
LIMIT = 1_000_000  # 1 ms
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from ternary_weight_bit_absmean_b200 import build_lib
    build_lib.build()
    B.lib()


def problem(M, K, xt):
    g = torch.Generator(device=DEV).manual_seed(M + K)
    x, dy = torch.randn(M, K, generator=g, device=DEV), torch.randn(M, K, generator=g, device=DEV)
    return x.to(xt), 1 + 0.1 * torch.randn(K, generator=g, device=DEV), dy


# several rows of a block at a time and one, whole chunks and not, clusters of two, four and eight
LAYOUTS = [(20000, 129), (6000, 1536), (3000, 3200), (1000, 4097), (1000, 8192), (1000, 9001), (400, 16384), (200, 20001),
           (200, 70000)]


@pytest.mark.parametrize("stall", [0, 1, 3])
@pytest.mark.parametrize("kind", [B.BL_NORM_RMS, B.BL_NORM_LAYER])
@pytest.mark.parametrize("M,K", LAYOUTS)
def test_waits_run_out_then_the_next_call_is_right(M, K, kind, stall):
    for xt in (F32, BF16):
        x, w, dy = problem(M, K, xt)
        want = B.norm_backward(dy, x, w, kind, bias=True)
        out = [guarded_empty((M, K), F32), guarded_empty((K,), F32), guarded_empty((K,), F32)]
        ws = guarded_empty((max(16, B.bitlinear_norm_backward_workspace_size(M, K)),), torch.uint8)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        B.bitlinear_norm_backward_stall_test(dy, x, w, kind, 1e-5, *out, ws, err, LIMIT, stall)
        torch.cuda.synchronize()
        for t in out + [ws]:
            check_guard(t)
        assert err.item() == B.BL_ERRBIT_TIMEOUT
        err.zero_()
        got = B.norm_backward(dy, x, w, kind, bias=True, err_word=err)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and err.item() == 0


@pytest.mark.parametrize("M,K", [(700, 1536), (300, 8192), (40, 16384), (3, 80000)])
def test_a_stall_no_block_reaches_changes_nothing(M, K):
    x, w, dy = problem(M, K, F32)
    out = [torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)]
    ws = torch.empty(max(16, B.bitlinear_norm_backward_workspace_size(M, K)), dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.bitlinear_norm_backward_stall_test(dy, x, w, B.BL_NORM_LAYER, 1e-5, *out, ws, err, 2_000_000_000, 1 << 20)
    assert all(torch.equal(a, b) for a, b in zip(out, B.norm_backward(dy, x, w, B.BL_NORM_LAYER, bias=True)))
    assert err.item() == 0
