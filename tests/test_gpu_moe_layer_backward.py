"""The backward steps of the layer in examples/moe_layer.py against autograd in 64 bits
of the same steps on the values that the forward kept.  A bf16 gradient is rounded
once, 2^-8 relative; a weight's gradient sums H float32 products, H 2^-24 of their
magnitudes, and reaches the logits through factors of at most 1."""
import os
import sys

import pytest
import torch

import micro_scaled_fp4_amd as fp4
from gpu_util import announce

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer  # noqa: E402

pytestmark = pytest.mark.gpu

E24, BF16 = 2.0 ** -24, 2.0 ** -8


def f64(t, grad=False):
    return t.detach().double().cpu().requires_grad_(grad)


@pytest.mark.parametrize("fmt", [fp4.FP4_NVFP4, fp4.FP4_MXFP4])
@pytest.mark.parametrize("tokens", [1, 37, 300])
def test_gradients_match_autograd(fmt, tokens):
    announce(f"moe layer backward fmt={fmt} tokens={tokens}")
    H, inner, experts, k = 512, 256, 32, 4
    layer = moe_layer.MoELayer(H, inner, experts, k, fmt, groups=4, top_groups=2, seed=tokens)
    g = torch.Generator(device="cuda:0")
    g.manual_seed(tokens)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda:0").to(torch.bfloat16)  # noqa: E731
    keep = {}
    layer.forward(rand(tokens, H), keep)
    dy, d_hidden = rand(tokens, H), rand(tokens * k, inner)
    got = {n: t.double().cpu() for n, t in layer.backward(dy, keep, d_hidden).items()}

    # y = x + sum of weight * row: rows, and the logits through the weights (ids fixed)
    logits, rows = f64(keep["logits"], True), f64(keep["rows"], True)
    ids, slot_rows = keep["ids"].long().cpu(), keep["slot_rows"].long().cpu()
    score = torch.sigmoid(logits).gather(1, ids)
    weights = score / score.sum(1, keepdim=True)
    y = (weights[..., None] * rows[slot_rows]).sum(1)
    d_logits, d_rows = torch.autograd.grad((y * f64(dy)).sum(), (logits, rows))
    # (the weight itself is float32, 4e-6 relative)
    assert ((got["rows"] - d_rows).abs() <= (BF16 + 4e-6) * d_rows.abs()).all()
    parts = f64(dy)[:, None] * rows.detach()[slot_rows]
    most = parts.sum(2).abs().amax()
    tol = 2 * (H + 2) * E24 * parts.abs().sum(2).amax() + 2e-5 * most
    assert ((got["logits"] - d_logits).abs() <= BF16 * d_logits.abs() + tol).all()

    # hidden = silu(z even) * z odd; the biases' gradients are dz's sums per expert
    z = f64(keep["z"], True)
    hidden = torch.nn.functional.silu(z[:, 0::2]) * z[:, 1::2]
    dz, = torch.autograd.grad((hidden * f64(d_hidden)).sum(), z)
    other = z.detach().abs()
    factor = f64(d_hidden).abs().repeat_interleave(2, 1) * (1 + other) * (1 + other.view(-1, inner, 2).flip(2).reshape(other.shape))
    own = 1e-5 * (1 + other) * factor                    # the activation's and the derivative's own error
    assert ((got["z"] - dz).abs() <= BF16 * dz.abs() + own).all()
    off = keep["offsets"].tolist()
    for e in range(experts):
        r = slice(off[e], off[e + 1])
        n = off[e + 1] - off[e]
        tol = own[r].sum(0) + n * E24 * dz[r].abs().sum(0) + 1e-30
        assert ((got["bias"][e] - dz[r].sum(0)).abs() <= tol).all()
