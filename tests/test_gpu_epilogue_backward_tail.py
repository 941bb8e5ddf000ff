"""GPU: the epilogue's backward pass writes zeros to the rows past the last group
(slots that were dropped), whatever the memory held, and the groups' rows as without
them: dz bit for bit the call's on the groups' rows alone, whose bias sums may be
split otherwise (n float32 terms in either order: 2 n 2^-24 of their magnitudes)."""
import numpy as np
import pytest
import torch

import micro_scaled_fp4_amd as fp4
import moe_reference as ref
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def backward_into(dz, dD, z, off, act, gated, bias_grad=True):
    """fp4_epilogue_backward into a given dz; returns dbias or None."""
    lib = fp4.load_library()
    M, N, E = z.shape[0], z.shape[1], off.numel() - 1
    need = lib.fp4_epilogue_backward_workspace_bytes(E, M, N)
    db = torch.empty(E, N, device=DEV) if bias_grad else None
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    code = {F32: fp4.FP4_F32, BF: fp4.FP4_BF16}
    st = lib.fp4_epilogue_backward(dD.data_ptr(), code[dD.dtype], z.data_ptr(), code[z.dtype], E, off.data_ptr(), M, N,
                                   act, int(gated), dz.data_ptr(), code[dz.dtype], None if db is None else db.data_ptr(),
                                   ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    return db


@pytest.mark.parametrize("N", [80, 1040, 82, 514])     # whole 16-byte pieces, and not
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("sizes,tail", [([0, 3, 200, 0, 1, 90, 0], 4), ([5], 300), ([0, 0], 7), ([64, 64], 0)])
@pytest.mark.parametrize("gated,bias_grad", [(True, True), (False, False)])
def test_rows_past_the_last_group_are_zeros(N, dtype, sizes, tail, gated, bias_grad):
    announce(f"epilogue backward tail N={N} {dtype} {sizes} + {tail} gated={gated}")
    off = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device=DEV)
    live, M = sum(sizes), sum(sizes) + tail
    g = torch.Generator(device=DEV)
    g.manual_seed(N + M)
    z = torch.randn(M, N, generator=g, device=DEV).to(dtype)
    dD = torch.randn(M, N // 2 if gated else N, generator=g, device=DEV).to(dtype)
    z[live:], dD[live:] = float("nan"), float("nan")       # rows of no slot are not read
    for out in (F32, BF):
        dz = torch.full((M, N), float("nan"), dtype=out, device=DEV)
        db = backward_into(dz, dD, z, off, ref.SILU, gated, bias_grad)
        assert not dz[live:].float().ne(0).any()
        if live:
            alone = torch.empty(live, N, dtype=out, device=DEV)
            want = backward_into(alone, dD[:live].contiguous(), z[:live].contiguous(), off, ref.SILU, gated, bias_grad)
            assert torch.equal(dz[:live], alone)
            if bias_grad and out == F32:
                at = 0
                for e, n in enumerate(sizes):
                    tol = 2 * n * 2.0 ** -24 * alone[at:at + n].double().abs().sum(0) + 1e-30
                    assert ((db[e].double() - want[e].double()).abs() <= tol).all()
                    at += n
        elif bias_grad:
            assert not db.ne(0).any()
