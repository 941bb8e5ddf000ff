"""GPU: attention with scores so large that their float32 steps pass 1: the largest score takes all the weight."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from gpu_util import DEV, announce
from test_gpu_kv_attention import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,power", [(64, p) for p in (18, 21, 23, 25, 26, 29, 60, 110)] + [(128, 24), (128, 30), (256, 24), (256, 30)])
@pytest.mark.parametrize("fmt", [ref.NV, ref.MX])
def test_the_largest_score_takes_all(fmt, D, power):
    """Constant keys of 1, 2 and 4 beside one of 8 (negative scores: 2, 4 and 8 beside one of 1): the
    loudest score is ahead by half of itself (negative ones: by itself), more than 2^14, so the other weights are 0 and the output
    is that position's value.  Its weight cancels but for its rounding to fp16 (2^-11; in two parts 2^-20)."""
    announce(f"kv attention scores of 2^{power} fmt {fmt} D {D}")
    for seqs, places in (([(300, 1), (70, 1)], (0, 150, 299)), ([(1500, 1)], (0, 1499)), ([(400, 12)], (380,)), ([(200, 130)], (60,)),
                         ([(90, 90)], (0,))):
        for at in places:
            for sign in (1, -1):
                case = ref.Case(fmt, 1, D, 16, seqs, seed=at)
                for b in range(case.B):
                    n = len(case.k[b])
                    case.k[b][:] = np.exp2(case.rng.integers(0, 3, (n, 1, 1)) + (sign < 0)).astype(np.float32)
                    case.k[b][min(at, n - 1)] = 8.0 if sign > 0 else 1.0
                case.k_amax = np.float32(8.0)
                store = case.full_store()
                # the largest score in size is 2^power x 1.3 (not a power of two)
                scale = sign * 2.0 ** power * 1.3 / (D * 8)
                for dtype in (torch.bfloat16, torch.float32):
                    q = torch.ones(case.T, 2, D, dtype=dtype, device=DEV)
                    got, _ = check(case, store, q, q.double().cpu().numpy(), scale=float(np.float32(scale)))
                    near = 2.0 ** -11 + 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -20
                    for b in range(case.B):
                        lo, hi = int(case.offsets[b]), int(case.offsets[b + 1])
                        want = case.held(store, b, 1)[0][min(at, int(case.lengths[b]) - 1), 0]
                        off = np.abs(got[lo:hi].double().cpu().numpy() - want)
                        assert (off <= near * np.abs(want)).all()


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 8, 9, 16])
@pytest.mark.parametrize("fmt", [ref.NV, ref.MX])
def test_a_maximum_that_grows_by_a_float32_step(fmt, steps):
    """Scores (times log2(e)) of 2^26 + 8 and 8 `steps` above it, exact, the float32 step being 8 there: the weights
    are as 1 to 2^(8 steps), whichever comes first, in the same wave's steps."""
    announce(f"kv attention maximum grown by {steps} steps of 8 at 2^26, fmt {fmt}")
    D = 64
    for seqs in ([(400, 1)], [(400, 12)], [(400, 70)]):
        for first, second in ((3, 290), (290, 3)):
            case = ref.Case(fmt, 1, D, 16, seqs, seed=steps)
            k = case.k[0]
            k[:] = 0
            # <q, k> = 2^23 + 1 and 2^23 + 1 + steps, in bits of 1, 2, 4, 8 and 16
            k[first, 0, [0, 8]] = 1.0
            k[second, 0, 0] = 1.0
            k[[first, second], 0, 15] = 1.5     # 6 x the block's scale, which is 1/4 then (q is 0 there)
            for bit in range(5):
                k[second, 0, 8 + bit] = float((1 + steps) >> bit & 1)
            case.k_amax = np.float32(2688.0 / 4)        # NVFP4: a tensor scale of 1/4
            store = case.full_store()
            held = case.held(store, 0, 0)[0]
            assert np.array_equal(held[:, 0], k[:, 0])
            for dtype in (torch.bfloat16, torch.float32):
                q = torch.zeros(case.T, 2, D, dtype=dtype, device=DEV)
                q[:, :, 0] = 2.0 ** 23
                for bit in range(5):
                    q[:, :, 8 + bit] = 2.0 ** bit
                got, _ = check(case, store, q, q.double().cpu().numpy(), scale=float(np.float32(8 * np.log(2.0))))
                v = case.held(store, 0, 1)[0][:, 0]
                small = 2.0 ** (-8 * steps)
                want, size = (v[second] + small * v[first]) / (1 + small), (np.abs(v[second]) + small * np.abs(v[first])) / (1 + small)
                near = 2.0 ** -11 + 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -19
                assert (np.abs(got.double().cpu().numpy() - want) <= near * size + 2.0 ** -24 * np.abs(v).max()).all()
