"""GPU parity: GEMMs whose K is one 256-value stage, with more tiles than compute
units.  A workgroup then loads its next tile's first two stages of which only the
first exists; the second must add exact zeros, not the next rows' values."""
import numpy as np
import pytest
import torch

import micro_scaled_fp4_amd as fp4
import workloads
from oracle import fp4_oracle as o
from gpu_util import announce, to_gpu_u8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_one_stage_and_several_tiles_per_workgroup(fmt):
    M, N, K = 2100, 8496, 256
    announce(f"gemm {fmt} {M}x{N}x{K}")
    qa, qw = workloads.random_codes((M, K // 2), 1), workloads.random_codes((N, K // 2), 2)
    if fmt == "nv":
        sa, sw = workloads.random_bytes((M, K // 16), 0x20, 0x50, 3), workloads.random_bytes((N, K // 16), 0x20, 0x50, 4)
        A, W = o.nv_operand_f64(qa, sa, 1.0, K), o.nv_operand_f64(qw, sw, 0.5, K)
        ga, gw = torch.ones(1, device="cuda:0"), torch.full((1,), 0.5, device="cuda:0")
        f = fp4.FP4_NVFP4
    else:
        sa, sw = workloads.random_bytes((M, K // 32), 120, 134, 3), workloads.random_bytes((N, K // 32), 120, 134, 4)
        A, W = o.mx_operand_f64(qa, sa, K), o.mx_operand_f64(qw, sw, K)
        ga = gw = None
        f = fp4.FP4_MXFP4
    D = fp4.fp4_scaled_gemm(f, to_gpu_u8(qa), to_gpu_u8(sa), ga, to_gpu_u8(qw), to_gpu_u8(sw), gw, K,
                            out_dtype=torch.float32).cpu().numpy()
    ref, mag = A @ W.T, np.abs(A) @ np.abs(W).T
    assert (np.abs(D - ref) <= 1e-5 * mag).all()
