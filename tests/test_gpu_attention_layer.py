"""The attention layer of examples/attention_layer.py: projections, cache and attention together, for prompts
and for decoding steps out of a captured graph."""
import os
import sys

import pytest

from gpu_util import announce

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import attention_layer  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("tokens,steps", [(200, 6), (1, 3), (1000, 4)])
def test_layer_runs_and_attends(fmt, tokens, steps):
    """2^-8 of each bf16 output value for its rounding, and 2^-11 of the weighted values' sizes for the fp16
    weights: a weighted mean's size is below a few of its own, so 2^-8 + 4 * 2^-11 of the norm holds both."""
    announce(f"attention layer {fmt} {tokens} tokens {steps} steps")
    off = attention_layer.main(["--format", fmt, "--tokens", str(tokens), "--steps", str(steps), "--check"])
    assert len(off) == steps and max(off) <= 2.0 ** -8 + 4 * 2.0 ** -11
