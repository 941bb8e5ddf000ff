"""GPU parity at the edges of expert routing and combining: gradients of dropped
slots, and renormalized weights of scores that float32 cannot hold by themselves.
Tolerances as in test_gpu_moe: a weight is a few float32 operations on exponentials
within 3 ulp, 4e-6 relative."""
import numpy as np
import pytest
import torch

import micro_scaled_fp4_amd as fp4
import moe_reference as ref
from gpu_util import DEV, announce
from test_gpu_moe import check_route, gpu, host

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
TINY = 2.0 ** -126                     # the smallest normal float32


@pytest.mark.parametrize("H", [16, 2056, 7])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_dropped_slots_have_no_weight_gradient(H, dtype):
    """0 for a slot without a row, whatever dy holds."""
    announce(f"combine backward of dropped slots H={H} {dtype}")
    T, k = 6, 3
    slot_rows = np.full((T, k), -1, np.int32)
    slot_rows[:, 1] = np.arange(T)
    row_slots = np.full(T * k, -1, np.int32)
    row_slots[:T] = np.arange(T) * k + 1
    slot_rows[5, 2] = T * k            # past the rows
    dy = torch.ones(T, H, device=DEV).to(dtype)
    for t, v in enumerate((float("inf"), float("-inf"), float("nan"), 3e38, 1.0, float("inf"))):
        dy[t, t % H] = v
    rows = torch.ones(T * k, H, device=DEV).to(dtype)
    w = gpu(np.full((T, k), 0.5, np.float32))
    dr, dw = fp4.moe_combine_backward(dy, rows, w, gpu(slot_rows), gpu(row_slots))
    dw = host(dw)
    assert (dw[:, 0] == 0).all() and (dw[:, 2] == 0).all()
    assert np.isposinf(dw[0, 1]) and np.isneginf(dw[1, 1]) and np.isnan(dw[2, 1]) and dw[4, 1] == H
    assert not dr[T:].float().ne(0).any()


@pytest.mark.parametrize("E", [16, 64, 256, 700])
@pytest.mark.parametrize("groups", [1, 4])
def test_renormalized_softmax_far_below_the_largest_logit(E, groups):
    """A bias that selects experts whose scores are e^-90 to e^-300: their ratios are
    well defined, forward and backward."""
    announce(f"route far below the largest logit E={E} groups={groups}")
    rng = np.random.default_rng(E)
    T, k = 9, 4
    logits = rng.normal(0, 2, (T, E)).astype(np.float32)
    logits[:, : E // 2] -= rng.uniform(90, 300, (T, 1)).astype(np.float32)
    logits[0, : E // 2] = -600.0       # (equal logits, equal weights)
    bias = np.zeros(E, np.float32)
    bias[: E // 2] = 4.0 + np.arange(E // 2) / 64
    t, ids, w = check_route(logits, k, False, bias=bias, groups=groups, top_groups=max(1, groups // 2), scale=2.5)
    assert (ids < E // 2).all() and (ids >= 0).all()
    np.testing.assert_allclose(w.sum(1), 2.5, rtol=4e-6)
    dw = rng.normal(0, 1, (T, k)).astype(np.float32)
    got = host(fp4.moe_route_backward(gpu(dw), t, gpu(ids), scale=2.5))
    want = ref.route_grad(dw, logits, ids, False, True, 2.5)
    np.testing.assert_allclose(got, want, rtol=2e-5, atol=4e-6 * 2.5 * np.abs(dw).max())


@pytest.mark.parametrize("E", [16, 256, 700])
@pytest.mark.parametrize("low,high", [(-88.6, -87.05), (-110.0, -80.0), (-400.0, -395.0)])
def test_renormalized_sigmoid_of_small_scores(E, low, high):
    """All scores at or below float32's smallest normal number."""
    announce(f"route sigmoid scores in e^{low}..e^{high} E={E}")
    rng = np.random.default_rng(E)
    T, k = 7, 5
    logits = rng.uniform(low, high, (T, E)).astype(np.float32)
    logits[-1, 3] = 2.0                # (one ordinary score among them)
    t, ids, w = check_route(logits, k, True, scale=1.5)
    np.testing.assert_allclose(w.sum(1), 1.5, rtol=4e-6)
    dw = rng.normal(0, 1, (T, k)).astype(np.float32)
    got = host(fp4.moe_route_backward(gpu(dw), t, gpu(ids), score=fp4.FP4_SCORE_SIGMOID, scale=1.5))
    want = ref.route_grad(dw, logits, ids, True, True, 1.5)
    np.testing.assert_allclose(got, want, rtol=2e-5, atol=4e-6 * 1.5 * np.abs(dw).max())
    # not renormalized: the scores themselves, those below 2^-126 may be 0
    i2, w2 = fp4.moe_route(t, k, score=fp4.FP4_SCORE_SIGMOID, renormalize=False, scale=1.5)
    want = ref.route_weights(logits, host(i2), True, False, 1.5)
    assert (np.abs(host(w2) - want) <= 4e-6 * want + 1.5 * TINY).all()


def test_selection_by_scores_down_to_the_smallest_normal_number():
    """Scores from 2^-126 on order the selection also where a bias is given."""
    logits = -87.0 - 0.02 * np.random.default_rng(3).permutation(16).astype(np.float32)[None]
    _, ids, _ = check_route(logits, 6, True, bias=np.zeros(16, np.float32))
    assert (ids[0] == np.argsort(-logits[0])[:6]).all()


@pytest.mark.parametrize("renorm", [False, True])
def test_sigmoid_gradient_of_saturated_scores(renorm):
    """1 - s by its own formula: the gradient of large logits is small and exact."""
    logits = np.array([[12.0, 15.0, 9.5, 17.0, 8.0, -3.0, -20.0, 30.0]], np.float32)
    dw = np.array([[1.0, -0.5, 0.25, 2.0]], np.float32)
    ids = np.array([[0, 1, 2, 7]], np.int32)
    got = host(fp4.moe_route_backward(gpu(dw), gpu(logits), gpu(ids), score=fp4.FP4_SCORE_SIGMOID, renormalize=renorm))
    l, g = logits.astype(np.float64)[0, ids[0]], dw.astype(np.float64)[0]
    s, rest = ref.sigmoid(l), ref.sigmoid(-l)            # (1 - s would lose 64-bit digits at 30)
    if renorm:
        q = s / s.sum()
        g = q * (g - (g * q).sum()) / s
    want = np.zeros((1, 8))
    want[0, ids[0]] = g * s * rest
    np.testing.assert_allclose(got, want, rtol=4e-6 if not renorm else 1e-5, atol=1e-30)
