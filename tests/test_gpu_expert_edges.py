"""The experts' E4M3 products at the ends of their range: no rows at all."""
import numpy as np
import pytest
import torch

from combine_ep_get_02_amd import ep, experts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("sizes,over", [([0, 0, 0], 0), ([0, 5, 0], ep.EP_DEV_RECV_OVERFLOW), ([-4, -1, 0], 0),
                                        ([0] * 299 + [1], ep.EP_DEV_RECV_OVERFLOW),
                                        ([2147483647] * 3, ep.EP_DEV_RECV_OVERFLOW)], ids=lambda v: str(v)[-20:])
def test_segments_that_pass_a_buffer_of_no_rows(sizes, over, swiglu):
    E, n, k = len(sizes), 256, 384
    rows = torch.from_numpy(np.array(sizes, np.int32)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, xs = torch.empty(0, k, dtype=torch.uint8, device="cuda"), torch.empty(0, k // 128, device="cuda")
    w = torch.zeros(E, n * (2 if swiglu else 1), k, dtype=torch.uint8, device="cuda")
    ws = torch.ones(E, w.shape[1] // 128, k // 128, device="cuda")
    for given in ((x, xs), (None, None)):
        status.zero_()
        if swiglu:
            out, outs = torch.empty(0, n, dtype=torch.uint8, device="cuda"), torch.empty(0, n // 128, device="cuda")
            experts.ep_expert_gemm_swiglu_fp8(E, n, k, *given, w, ws, rows, 0, out, outs, status)
        else:
            experts.ep_expert_gemm_fp8(E, n, k, *given, w, ws, rows, 0, torch.empty(0, n, dtype=torch.bfloat16, device="cuda"), status)
        assert int(status.item()) == over


def test_no_rows_and_nothing_to_flag():
    """Without sizes, or without a status to set, a call of no rows does nothing."""
    k, n = 128, 8
    w, ws = torch.zeros(1, n, k, dtype=torch.uint8, device="cuda"), torch.ones(1, 1, 1, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    experts.ep_expert_gemm_fp8(1, n, k, None, None, w, ws, None, 0, None, status)
    experts.ep_expert_gemm_fp8(1, n, k, None, None, w, ws, torch.ones(1, dtype=torch.int32, device="cuda"), 0, None)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
