"""GPU parity of every kernel that a fused FP4 product can take (product_sizes), against
the 64-bit plain form with the tolerances of test_gpu_fused_gemm."""
import numpy as np
import pytest
import torch

import micro_scaled_fp4_amd as fp4
import moe_reference as ref
import test_gpu_fused_gemm as fused
from gpu_util import announce, to_gpu_u8
from product_sizes import DENSE, GROUPED, SHORT

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def ident(case):
    return "-".join(str(len(x)) + "groups" if isinstance(x, list) else str(x) for x in case)


@pytest.mark.parametrize("case", DENSE, ids=ident)
def test_dense(case):
    rows, fmt, M, N, K = case
    announce(f"product kernel of {rows} rows {fmt} {M}x{N}x{K}")
    fused.run_dense(fmt, M, N, K, ref.SILU, True, BF, F32, BF, F32, M + N)
    if M * N < 4000000:
        fused.run_dense(fmt, M, N, K, ref.GELU, False, F32, BF, F32, BF, K, -0.25)
        fused.run_dense(fmt, M, N, K, ref.NONE, False, None, None, BF, None, N)


@pytest.mark.parametrize("case", GROUPED, ids=ident)
def test_grouped(case):
    rows, fmt, sizes, tail, N, K = case
    announce(f"grouped product kernel of {rows} rows {fmt} {sizes}+{tail} {N}x{K}")
    E, M = len(sizes), sum(sizes) + tail
    f = fp4.FP4_NVFP4 if fmt == "nv" else fp4.FP4_MXFP4
    qa, sa, ga = fused.operand(fmt, M, K, 1)
    qw, sw, gw = fused.operand(fmt, N, K, 2, E)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    rng = np.random.default_rng(N)
    t = lambda g: None if g is None else torch.from_numpy(g).to(fused.DEV)  # noqa: E731
    A = fused.values(fmt, qa, sa, None if ga is None else ga[0], K)
    for act, gated, bias_t, res_t, out, pre in ((ref.SILU, True, F32, BF, BF, F32), (ref.GELU, False, BF, None, F32, None)):
        bias = fused.gpu(rng.normal(0, 1, (E, N)), bias_t)
        res = None if res_t is None else fused.gpu(rng.normal(0, 1, (M, N // 2 if gated else N)), res_t)
        got = fp4.fp4_grouped_gemm_fused(f, to_gpu_u8(qa), to_gpu_u8(sa), t(ga), to_gpu_u8(qw).view(E, N, -1),
                                         to_gpu_u8(sw).view(E, N, -1), t(gw), t(off), K, 0.5, activation=act, gated=gated,
                                         bias=bias, residual=res, preact_dtype=pre, out_dtype=out)
        D, z = got if pre is not None else (got, None)
        for e in range(E):
            if sizes[e] == 0:
                continue
            r, w = slice(off[e], off[e + 1]), slice(e * N, (e + 1) * N)
            W = fused.values(fmt, qw[w], sw[w], None if gw is None else gw[e], K)
            b = fused.host(bias[e])
            z_ref = 0.5 * (A[r] @ W.T) + b
            z_err = 0.5e-5 * (np.abs(A[r]) @ np.abs(W).T)
            fused.check(fused.host(D[r]), z_ref, z_err, b, act, gated, None if res is None else fused.host(res[r]), out)
            if z is not None:
                assert (np.abs(fused.host(z[r]) - z_ref) <= z_err + fused.E23 * (np.abs(z_ref) + np.abs(b))).all()
        assert not D[off[-1]:].ne(0).any() and (z is None or not z[off[-1]:].ne(0).any())


@pytest.mark.parametrize("case", SHORT, ids=ident)
def test_several_tiles_per_workgroup_repeat(case):
    """The 256 x 256 tiles' persistent loop with one to three stages a tile: the same
    bits on every run and those of the plain product, with other inputs' tiles in shared
    memory in between."""
    _, fmt, M, N, K = case
    announce(f"persistent tiles {fmt} {M}x{N}x{K}")
    f = fp4.FP4_NVFP4 if fmt == "nv" else fp4.FP4_MXFP4
    t = lambda g: None if g is None else torch.from_numpy(g).to(fused.DEV)  # noqa: E731
    args = []
    for seed in (1, 2):
        qa, sa, ga = fused.operand(fmt, M, K, seed)
        qw, sw, gw = fused.operand(fmt, N, K, seed + 10)
        args.append((f, to_gpu_u8(qa), to_gpu_u8(sa), t(ga), to_gpu_u8(qw), to_gpu_u8(sw), t(gw), K))
    want = [fp4.fp4_scaled_gemm(*a, out_dtype=F32) for a in args]
    for i in range(8):
        assert torch.equal(fp4.fp4_scaled_gemm_fused(*args[i & 1], out_dtype=F32), want[i & 1])
