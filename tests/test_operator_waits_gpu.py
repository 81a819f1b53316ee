"""The products' bounded waits: a call whose waits run out reports it, and leaves nothing behind
that the next call meets (loads on their way to shared memory, tensor memory that is not freed)."""
import pytest
import torch

import unpermute_ep_dispatch_gb300 as epd
from test_operators_gpu import check_ok, forward_case
from unpermute_ep_dispatch_gb300 import _binding

pytestmark = pytest.mark.gpu

# many tiles a pair of blocks; few, whose reduction is shared by pairs; one tile
SHAPES = {"many": ([300, 0, 700] * 8, 512, 1536), "shared": ([40, 7], 4096, 512), "one": ([16], 512, 128)}


def product(shape, act, fp8):
    counts, K, N = SHAPES[shape]
    x, w, cnt, kw, real, y, _, tol, _ = forward_case(counts, K, N, act, 5, fp8=fp8)
    out = torch.empty(x.shape[0], N, dtype=torch.bfloat16, device="cuda")

    def stalled(**how):
        status = epd.new_status()
        _binding.epd_test_expert_matmul_stalled(x, w, cnt, kw["expert_start_loc"], status, out, act, kw.get("x_scale"),
                                                kw.get("w_scale"), **how)
        torch.cuda.synchronize()
        return int(status.item())

    def check():
        status = epd.new_status()
        epd.ep_expert_matmul(x, w, cnt, status, y=out, **kw)
        check_ok(status)
        assert ((out[real].double() - y[real]).abs() <= tol[real]).all()
    return stalled, check


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("fp8", [False, True])
def test_matrix_instructions_that_never_come(shape, act, fp8):
    stalled, check = product(shape, act, fp8)
    check()
    for tile in (0, 1) if shape == "many" else (0,):
        assert stalled(stalled_tile=tile) == epd.EPD_ERR_TIMEOUT
        check()
    # none left out, and time enough
    assert stalled(stalled_tile=-1, wait_ns=2_000_000_000) == epd.EPD_OK
    check()
