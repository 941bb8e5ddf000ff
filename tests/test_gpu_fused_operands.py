"""GPU: the fused products' binding refuses operands whose sizes or types do not fit
each other before anything is launched, and takes the forms that fit."""
import pytest
import torch

import micro_scaled_fp4_amd as fp4
from gpu_util import DEV

pytestmark = pytest.mark.gpu

M, N, K, E = 5, 32, 64, 3


def operands(fmt, groups=0):
    nsc = K // (16 if fmt == fp4.FP4_NVFP4 else 32)
    b = lambda *s: torch.full(s, 0x38, dtype=torch.uint8, device=DEV)  # noqa: E731
    lead = (groups,) if groups else ()
    g = torch.ones(1, device=DEV) if fmt == fp4.FP4_NVFP4 else None
    a = {"A": b(M, K // 2), "a_scales": b(M, nsc), "g_a": g, "W": b(*lead, N, K // 2), "w_scales": b(*lead, N, nsc),
         "g_b": g if not groups or g is None else torch.ones(groups, device=DEV), "K": K}
    if groups:
        a["offsets"] = torch.tensor([0, 2, 2, M], dtype=torch.int32, device=DEV)
    return a


def bad_ones(a):
    """(operand, value) that must be refused."""
    sa, sw = a["a_scales"], a["w_scales"]
    yield "a_scales", sa[:, :-1]
    yield "a_scales", sa[:-1]
    yield "a_scales", sa.T.contiguous()
    yield "a_scales", torch.cat([sa, sa])
    yield "a_scales", sa.float()
    yield "w_scales", sw[..., :-1]
    yield "w_scales", sw[..., :-1, :]
    yield "w_scales", sw.transpose(-1, -2).contiguous()
    yield "w_scales", sw.to(torch.int32)
    yield "w_scales", sw.cpu()
    yield "A", a["A"].to(torch.int16)
    yield "A", a["A"][:, :-1]
    yield "W", a["W"].float()
    yield "W", a["W"][..., :-1]
    if a["g_a"] is not None:
        yield "g_a", a["g_a"].double()
        yield "g_a", torch.ones(2, device=DEV)
        yield "g_a", a["g_a"].cpu()
        yield "g_b", a["g_b"].to(torch.bfloat16)
        yield "g_b", torch.ones(E + 1, device=DEV)


@pytest.mark.parametrize("fmt", [fp4.FP4_NVFP4, fp4.FP4_MXFP4])
@pytest.mark.parametrize("groups", [0, E])
def test_operands_that_do_not_fit_are_refused(fmt, groups):
    call = fp4.fp4_grouped_gemm_fused if groups else fp4.fp4_scaled_gemm_fused
    a = operands(fmt, groups)
    want = call(fmt, **a)
    for name, value in bad_ones(a):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            call(fmt, **{**a, name: value})
    # one byte per scale is what counts, and W's scales may be one row per row of W
    kind = torch.float8_e4m3fn if fmt == fp4.FP4_NVFP4 else torch.uint8
    again = call(fmt, **{**a, "a_scales": a["a_scales"].view(kind),
                         "w_scales": a["w_scales"].view(kind).reshape(-1, a["w_scales"].shape[-1])})
    assert torch.equal(again, want)


def test_workspaces_elsewhere_are_refused():
    z = torch.ones(3, 32, device=DEV)
    for ws in (torch.empty(1 << 16, dtype=torch.uint8), torch.empty(1 << 17, dtype=torch.uint8, device=DEV)[::2]):
        with pytest.raises(ValueError):
            fp4.fp4_epilogue_backward(z, z, 0, workspace=ws)
        with pytest.raises(ValueError):
            fp4.moe_dispatch(fp4.FP4_MXFP4, z, torch.zeros(3, 1, dtype=torch.int32, device=DEV), 2, workspace=ws)
    with pytest.raises(fp4.FP4Error):
        fp4.fp4_epilogue_backward(z, z, 0, workspace=torch.empty(4, dtype=torch.uint8, device=DEV))
