"""GPU parity at the edges of expert routing and combining."""
import numpy as np
import pytest
import torch

import micro_scaled_fp4_amd as fp4
from gpu_util import DEV, announce
from test_gpu_moe import gpu, host

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("H", [16, 2056, 7])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_dropped_slots_have_no_weight_gradient(H, dtype):
    """0 for a slot without a row, whatever dy holds."""
    announce(f"combine backward of dropped slots H={H} {dtype}")
    T, k = 6, 3
    slot_rows = np.full((T, k), -1, np.int32)
    slot_rows[:, 1] = np.arange(T)
    row_slots = np.full(T * k, -1, np.int32)
    row_slots[:T] = np.arange(T) * k + 1
    slot_rows[5, 2] = T * k            # past the rows
    dy = torch.ones(T, H, device=DEV).to(dtype)
    for t, v in enumerate((float("inf"), float("-inf"), float("nan"), 3e38, 1.0, float("inf"))):
        dy[t, t % H] = v
    rows = torch.ones(T * k, H, device=DEV).to(dtype)
    w = gpu(np.full((T, k), 0.5, np.float32))
    dr, dw = fp4.moe_combine_backward(dy, rows, w, gpu(slot_rows), gpu(row_slots))
    dw = host(dw)
    assert (dw[:, 0] == 0).all() and (dw[:, 2] == 0).all()
    assert np.isposinf(dw[0, 1]) and np.isneginf(dw[1, 1]) and np.isnan(dw[2, 1]) and dw[4, 1] == H
    assert not dr[T:].float().ne(0).any()
