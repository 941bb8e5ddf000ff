"""The expert layer of examples/moe_layer.py, all operators together, against the
same computation in plain torch on the dequantized operands.

The layer's own roundings are the plain form's (bf16 hidden rows and expert
outputs, FP4 hidden rows); where the two sums round a hidden value to different
sides of an FP4 rounding point, one step of one of `inner` values differs, so the
outputs agree to a few 1e-3 of their norm and not bit for bit."""
import os
import sys

import pytest
import torch

import micro_scaled_fp4_amd as fp4
from gpu_util import announce

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [fp4.FP4_NVFP4, fp4.FP4_MXFP4])
@pytest.mark.parametrize("tokens", [1, 7, 300, 2000])
def test_layer_matches_plain_torch(fmt, tokens):
    announce(f"moe layer fmt={fmt} tokens={tokens}")
    layer = moe_layer.MoELayer(512, 256, 32, 4, fmt, groups=4, top_groups=2, seed=tokens)
    g = torch.Generator(device="cuda:0")
    g.manual_seed(tokens)
    x = torch.randn(tokens, 512, generator=g, device="cuda:0").to(torch.bfloat16)
    keep = {}
    y = layer.forward(x, keep)
    want = layer.plain_forward(x)
    out = want - x.float()
    # y is rounded to bf16 with the residual: 2^-8 of |y|, and the FP4 steps above
    tol = 2.0 ** -8 * want.norm() + 0.02 * out.norm()
    assert float((y.float() - want).norm()) <= float(tol)
    assert torch.equal(layer.forward(x), y)
    grads = layer.backward(torch.ones_like(x), keep, torch.ones(tokens * 4, 256, device="cuda:0").to(torch.bfloat16))
    assert all(bool(torch.isfinite(t.float()).all()) for t in grads.values())
    assert grads["logits"].shape == (tokens, 32) and grads["bias"].shape == (32, 512)
