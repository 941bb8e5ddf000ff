"""GPU: a query row that holds a NaN, or whose scores pass float32, shows it in its output and its log-sum-exp, and
in no other row's."""
import numpy as np
import pytest
import torch

import kv_reference as ref
import micro_scaled_fp4_amd as fp4
from gpu_util import DEV, announce
from test_gpu_kv_attention import queries
from test_gpu_kv_cache import gpu_cache, tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs", [[(70, 1), (0, 1), (300, 1), (33, 1)], [(6000, 1), (2500, 1), (0, 2)], [(400, 9), (60, 12), (5, 8)],
                                  [(2500, 130), (90, 90), (20, 30)]], ids=["tokens", "long", "drafts", "prompts"])
@pytest.mark.parametrize("fmt", [ref.NV, ref.MX])
def test_nan_rows(fmt, seqs):
    announce(f"kv attention NaN rows fmt {fmt} {seqs}")
    for D in (64, 128, 256):
        case = ref.Case(fmt, 1, D, 16, seqs, seed=D)
        cache = gpu_cache(case, case.full_store())
        pos = torch.cat([torch.arange(length - n, length) for length, n in seqs])
        for dtype in (torch.bfloat16, torch.float32):
            q, _ = queries(case, 2, dtype)
            want, wlse = fp4.kv_cache_attention(cache, q, *tables(case), return_lse=True)
            bad = q.clone()
            rows = torch.arange(0, case.T, 3)
            bad[rows, 1, 7] = float("nan")
            got, lse = fp4.kv_cache_attention(cache, bad, *tables(case), return_lse=True)
            hit = torch.zeros(case.T, 2, dtype=torch.bool)
            hit[rows, 1] = pos[rows] >= 0       # (a row that sees nothing has nothing to show)
            hit = hit.to(got.device)
            assert torch.equal(got[~hit], want[~hit]) and torch.equal(lse[~hit], wlse[~hit])
            assert got[hit].isnan().all() and lse[hit].isnan().all()


@pytest.mark.parametrize("fmt", [ref.NV, ref.MX])
def test_scores_past_float32_are_nan(fmt):
    """Not a row of zeros, and not the log-sum-exp of a row that sees nothing."""
    announce(f"kv attention scores past float32 fmt {fmt}")
    for seqs in ([(70, 1), (0, 1)], [(5000, 1), (20, 1)], [(100, 40), (90, 90)]):
        case = ref.Case(fmt, 1, 64, 16, seqs, seed=3)
        for b in range(case.B):
            case.k[b][:] = np.abs(case.k[b]) + 1
        case.k_amax = np.float32(max(x.max(initial=1) for x in case.k))
        cache = gpu_cache(case, case.full_store())
        for dtype in (torch.bfloat16, torch.float32):
            q = torch.full((case.T, 2, 64), 2.0 ** 100, dtype=dtype, device=DEV)
            out, lse = fp4.kv_cache_attention(cache, q, *tables(case), scale=2.0 ** 120, return_lse=True)
            for b in range(case.B):
                rows = slice(int(case.offsets[b]), int(case.offsets[b + 1]))
                if case.lengths[b]:
                    assert out[rows].isnan().all() and lse[rows].isnan().all()
                else:
                    assert (out[rows] == 0).all() and lse[rows].isneginf().all()
