"""GPU: attention where the factor of the scores, the scores or the queries are near the ends of float32."""
import numpy as np
import pytest
import torch

import kv_reference as ref
import micro_scaled_fp4_amd as fp4
from gpu_util import DEV, announce
from test_gpu_kv_attention import check, queries
from test_gpu_kv_cache import gpu_cache, tables

pytestmark = pytest.mark.gpu

TOKENS, PROMPTS, LONG = [(200, 1), (77, 1)], [(90, 90), (150, 70)], [(5000, 1), (3, 1)]


@pytest.mark.parametrize("seqs", [TOKENS, PROMPTS, LONG], ids=["tokens", "prompts", "long"])
@pytest.mark.parametrize("fmt", [ref.NV, ref.MX])
@pytest.mark.parametrize("q,k,scale", [(-98, 114, 2.0 ** -18), (-98, 114, -2.0 ** -18), (-90, 123, 2.0 ** -35), (0, 110, 0.0),
                                       (100, -97, 2.0 ** -4), (-60, -60, 2.0 ** 119)])
def test_factors_far_from_one(q, k, scale, fmt, seqs):
    """Scores of order 1 (or all 0) whose factors, taken one after the other, leave float32's range."""
    announce(f"kv attention q 2^{q} k 2^{k} scale {scale} fmt {fmt} {seqs}")
    case = ref.Case(fmt, 1, 64, 16, seqs, seed=256 + q + k, k_std=2.0 ** k)
    case.k_amax = np.float32(0.9 * max(float(np.abs(x).max()) for x in case.k))
    store = case.full_store()
    for dtype in (torch.bfloat16, torch.float32):
        x, x64 = queries(case, 2, dtype, std=2.0 ** q)
        check(case, store, x, x64, scale=scale)
