"""GPU: activations and derivatives over the whole finite range of float32, where
powers of the argument leave it."""
import numpy as np
import pytest
import torch

import micro_scaled_fp4_amd as fp4
import moe_reference as ref
from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name,act", sorted(ref.ACTS.items()))
def test_derivatives_of_large_arguments(name, act):
    """Far from 0 the derivative is 0 on the left (1 without an activation), 1 on the right."""
    mags = np.array([40.0, 1e3, 1e10, 3e12, 1e13, 6e18, 2e19, 6e19, 1e20, 1e30, 3e38], np.float32)
    z = torch.from_numpy(np.concatenate([mags, -mags])[None]).to(DEV)
    dz, db = fp4.fp4_epilogue_backward(torch.ones_like(z), z, act, out_dtype=torch.float32)
    want = np.concatenate([np.ones(mags.size), np.full(mags.size, 1.0 if act == ref.NONE else 0.0)])
    np.testing.assert_allclose(dz.cpu().numpy()[0], want, rtol=0, atol=1e-6)
    # gated: the gate's value (x or 0) and its derivative, each times the other operand
    g = torch.stack([z, torch.full_like(z, 0.5)], dim=2).flatten(1)
    dz, _ = fp4.fp4_epilogue_backward(torch.ones_like(z), g, act, gated=True, out_dtype=torch.float32)
    dz = dz.cpu().numpy()[0]
    np.testing.assert_allclose(dz[0::2], 0.5 * want, rtol=0, atol=1e-6)
    np.testing.assert_allclose(dz[1::2], np.concatenate([mags, -mags if act == ref.NONE else 0 * mags]), rtol=1e-6, atol=1e-6)
