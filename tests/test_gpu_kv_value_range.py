"""GPU: attention over values near both ends of the range that the formats are used in (2^-99 to 2^120): no sum may
pass float32 where the result does not, and no factor of a result may be a subnormal number."""
import numpy as np
import pytest
import torch

import kv_reference as ref
import micro_scaled_fp4_amd as fp4
from gpu_util import DEV, announce
from test_gpu_kv_attention import check, queries
from test_gpu_kv_cache import gpu_cache, tables

pytestmark = pytest.mark.gpu

# one position; short and cut contexts of single tokens; drafts; prompts that are cut and that are not
SEQS = {"one": [(1, 1)], "tokens": [(70, 1), (333, 1)], "long_token": [(6000, 1), (20, 1)], "drafts": [(900, 20), (65, 3)],
        "prompts": [(2500, 130), (70, 70)]}


@pytest.mark.parametrize("seqs", list(SEQS))
@pytest.mark.parametrize("power", [118, 100, -99])
@pytest.mark.parametrize("fmt", [ref.NV, ref.MX])
def test_large_and_small_values(fmt, power, seqs):
    announce(f"kv attention values of 2^{power} fmt {fmt} {seqs}")
    for D in (64, 256):
        case = ref.Case(fmt, 1, D, 16, SEQS[seqs], seed=128 + power + D, v_std=2.0 ** power)
        case.v_amax = np.float32(0.9 * max(float(np.abs(x).max(initial=0)) for x in case.v))
        store = case.full_store()
        for dtype in (torch.bfloat16, torch.float32):
            q, q64 = queries(case, 2, dtype)
            check(case, store, q, q64)


@pytest.mark.parametrize("length,rows,group", [(1, 1, 1), (8191, 1, 1), (700, 1, 2), (7001, 40, 1), (7777, 300, 1), (7001, 7001, 64)])
@pytest.mark.parametrize("power", [120, -99])
@pytest.mark.parametrize("fmt", [ref.NV, ref.MX])
def test_equal_values_come_back(fmt, power, length, rows, group):
    """Keys of 0 and one value everywhere: the value itself.  Every weight is the same power of two, and
    fewer than 2^13 of them times a value of 5 significant bits sum exactly.  Then a factor and its
    reciprocal are rounded, the unit, and the products with both: 4 half steps of 2^-24 for each of the
    three levels (part of a wave, waves, parts) and one for each of at most 2 x 128 parts' sums: 2^-15.8."""
    announce(f"kv attention equal values of 2^{power} fmt {fmt} {length} positions {rows} rows group {group}")
    D = 32
    value = np.float32(1.5 * 2.0 ** power)
    case = ref.Case(fmt, 1, D, 64, [(length, rows)], seed=1, k_std=0.0, v_std=0.0)
    case.v[0][:] = value
    case.v_amax = value
    cache = gpu_cache(case, case.full_store())
    held = float(value)                         # (E2M1 6 x 448 x amax / 2688, or 6 x a power of two)
    for dtype in (torch.bfloat16, torch.float32):
        q = torch.ones(rows, group, D, dtype=dtype, device=DEV)
        got, lse = fp4.kv_cache_attention(cache, q, *tables(case), return_lse=True)
        off = ((got.double() - held).abs().max() / held).item()
        assert off <= 2.0 ** -15.8 + (2.0 ** -8 if dtype == torch.bfloat16 else 0), off
        seen = torch.arange(length - rows + 1, length + 1, device=DEV, dtype=torch.float64)
        # log of an exact sum, one rounding and the multiplication by ln 2
        assert ((lse.double() - seen.log()[:, None]).abs() <= 2.0 ** -21 * (11 + seen.log()[:, None])).all()
