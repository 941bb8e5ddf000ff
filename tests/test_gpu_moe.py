"""GPU parity: expert routing, dispatch and combine against 64-bit plain forms
(moe_reference) and, for quantized rows, the oracle's quantizers bit for bit.

Tolerances.  Routing weights are a few float32 operations on scores whose
exponentials are within 3 ulp: 4e-6 relative to the largest weight's scale.
Sums of n float32 products: n 2^-24 times the sum of their magnitudes, and one
2^-8 relative rounding where the output is bf16 (2^-9 would do).
"""
import numpy as np
import pytest
import torch

import micro_scaled_fp4_amd as fp4
import moe_reference as ref
from oracle import fp4_oracle as o
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
EPS = 2.0 ** -24


def gpu(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(DEV)


def host(t):
    return t.detach().float().cpu().numpy() if t.dtype == BF else t.detach().cpu().numpy()


def separated(v, bias):
    """Rows whose distinct selection values are further apart than float32 resolves:
    a score has a few ulp of relative error and the sum with the bias one of its
    own, so 16 ulp of (value + largest bias) separate two of them."""
    s = np.sort(np.where(np.isfinite(v), v, -1e9), axis=1)
    d = np.diff(s, axis=1)
    most = 0.0 if bias is None else np.abs(bias[np.isfinite(bias)]).max(initial=0.0)
    return ~((d > 0) & (d < 16 * EPS * (np.abs(s[:, 1:]) + most))).any(axis=1)


def check_route(logits, k, sig, dtype=torch.float32, bias=None, **kw):
    t = gpu(logits, dtype)
    l = host(t)
    ids, w = fp4.moe_route(t, k, score=int(sig), bias=None if bias is None else gpu(bias), **{
        "num_groups": kw.get("groups", 1), "top_groups": kw.get("top_groups", 1),
        "group_top": kw.get("group_top", 1), "renormalize": kw.get("renorm", True),
        "scale": kw.get("scale", 1.0)})
    ri, rw, v = ref.route(l, k, sig, bias, **kw)
    ids, w = host(ids), host(w)
    plain = bias is None and not (kw.get("groups", 1) > 1 and kw.get("group_top", 1) == 2)
    ok = np.ones(len(l), bool) if plain else separated(v, bias)
    np.testing.assert_array_equal(ids[ok], ri[ok])
    # elsewhere the ids may differ where their values do not
    most = 0.0 if bias is None else np.abs(bias[np.isfinite(bias)]).max(initial=0.0)
    np.testing.assert_array_equal(ids < 0, ri < 0)
    at, rat = np.maximum(ids, 0), np.maximum(ri, 0)
    got, want = np.take_along_axis(v, at, 1), np.take_along_axis(v, rat, 1)
    live = ri >= 0
    got, want = got[live], want[live]
    apart = got != want                                      # (equal infinities are equal)
    assert (np.abs(got - want)[apart] <= 16 * EPS * (np.abs(want) + most)[apart]).all()
    for row in ids:
        assert len(set(row[row >= 0])) == (row >= 0).sum()
    rw = ref.route_weights(l, ids, sig, kw.get("renorm", True), kw.get("scale", 1.0))
    np.testing.assert_allclose(w, rw, rtol=4e-6, atol=4e-6 * kw.get("scale", 1.0) * 1e-3)
    return t, ids, w


SIZES = [(1, 1, 1), (1, 64, 8), (3, 7, 7), (5, 16, 4), (17, 60, 6), (33, 128, 8), (70, 160, 6), (9, 256, 16),
         (6, 500, 9), (5, 512, 8), (4, 640, 8), (3, 1023, 5), (2, 1024, 16)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("sig", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_route_top_k(T, E, k, sig, dtype):
    announce(f"route T={T} E={E} k={k} sigmoid={sig} {dtype}")
    rng = np.random.default_rng(T * 1000 + E)
    logits = rng.normal(0, 2, (T, E)).astype(np.float32)
    for renorm in (True, False):
        check_route(logits, k, sig, dtype, renorm=renorm, scale=1.0 if renorm else 2.5)


@pytest.mark.parametrize("T,E,k,groups,top_groups,group_top", [
    (19, 256, 8, 8, 4, 2), (7, 64, 6, 4, 2, 1), (13, 60, 5, 12, 3, 2), (4, 64, 2, 64, 5, 2),
    (5, 1024, 16, 64, 9, 2), (6, 512, 8, 2, 1, 1), (8, 20, 4, 4, 4, 2), (3, 6, 4, 3, 2, 1)])
@pytest.mark.parametrize("sig", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_route_groups_and_bias(T, E, k, groups, top_groups, group_top, sig, biased):
    announce(f"route groups T={T} E={E} k={k} groups={groups} sigmoid={sig} bias={biased}")
    rng = np.random.default_rng(E + groups)
    logits = rng.normal(0, 1.5, (T, E)).astype(np.float32)
    bias = (rng.integers(-60, 61, E) * 0.004).astype(np.float32) if biased else None
    for renorm in (True, False):
        check_route(logits, k, sig, bias=bias, groups=groups, top_groups=top_groups, group_top=group_top,
                    renorm=renorm, scale=2.5)


@pytest.mark.parametrize("E", [8, 64, 256, 700])
def test_route_ties_go_to_the_lowest_index(E):
    rng = np.random.default_rng(E)
    logits = rng.integers(-2, 3, (40, E)).astype(np.float32)
    logits[0] = 0.0
    logits[1] = np.where(np.arange(E) % 2, 0.0, -0.0)        # -0 and +0 are equal
    for sig in (False, True):
        check_route(logits, min(8, E), sig)
        check_route(logits, min(8, E), sig, groups=4, top_groups=2)


@pytest.mark.parametrize("E", [16, 64, 200, 1000])
def test_route_masks(E):
    """Rows with few or no experts left, the type's lowest value, NaN and infinities."""
    rng = np.random.default_rng(E)
    k = 6
    logits = rng.normal(0, 1, (12, E)).astype(np.float32)
    logits[0] = -np.inf
    logits[1] = np.nan
    logits[2, 1:] = -np.inf
    logits[3, 3:] = np.nan
    logits[4] = np.finfo(np.float32).min
    logits[5, 2:] = np.finfo(np.float32).min
    logits[6, ::2] = np.nan
    logits[7, 5] = np.inf
    logits[8] = 80.0
    logits[9, :] = -60.0
    logits[9, 4] = 60.0
    logits[10, : E // 2] = -np.inf
    for sig in (False, True):
        for renorm in (True, False):
            _, ids, w = check_route(logits, k, sig, renorm=renorm)
            assert np.isfinite(w).all()
            assert (ids[0] == -1).all() and (ids[1] == -1).all() and (w[:2] == 0).all()
            assert ids[2, 0] == 0 and (ids[2, 1:] == -1).all()
            check_route(logits, k, sig, renorm=renorm, groups=4, top_groups=2)
    bias = np.zeros(E, np.float32)
    bias[: E // 2] = -np.inf                                 # a bias can switch experts off
    _, ids, _ = check_route(logits[6:7] * 0 + 1, k, True, bias=bias)
    assert (ids >= E // 2).all() or (ids == -1).any()


GRAD_SIZES = [(1, 1, 1), (3, 16, 4), (21, 64, 8), (5, 60, 6), (10, 128, 3), (6, 256, 8), (4, 511, 16), (3, 1024, 8)]


@pytest.mark.parametrize("T,E,k", GRAD_SIZES)
@pytest.mark.parametrize("sig", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward(T, E, k, sig, renorm):
    announce(f"route backward T={T} E={E} k={k} sigmoid={sig} renorm={renorm}")
    rng = np.random.default_rng(T + E)
    logits = rng.normal(0, 1.5, (T, E)).astype(np.float32)
    if T > 2:
        logits[0] = -np.inf
        logits[1, 2:] = -np.inf
    t = gpu(logits)
    dw = rng.normal(0, 1, (T, k)).astype(np.float32)
    ids, _ = fp4.moe_route(t, k, score=int(sig), renormalize=renorm, scale=1.5)
    got = host(fp4.moe_route_backward(gpu(dw), t, ids, score=int(sig), renormalize=renorm, scale=1.5))
    want = ref.route_grad(dw, logits, host(ids), sig, renorm, 1.5)
    np.testing.assert_allclose(got, want, rtol=2e-5, atol=4e-6 * 1.5 * np.abs(dw).max())
    # the gradient against central differences of the 64-bit weights
    h = 1e-5
    for _ in range(6):
        a, e = rng.integers(0, T), rng.integers(0, E)
        if not np.isfinite(logits[a, e]):
            assert got[a, e] == 0
            continue
        up, dn = logits.astype(np.float64), logits.astype(np.float64)
        up[a, e] += h
        dn[a, e] -= h
        i = host(ids)
        num = ((ref.route_weights(up, i, sig, renorm, 1.5) - ref.route_weights(dn, i, sig, renorm, 1.5)) * dw).sum() / (2 * h)
        assert abs(num - got[a, e]) < 2e-5 * (1 + abs(num))
    bf = host(fp4.moe_route_backward(gpu(dw), t, ids, score=int(sig), renormalize=renorm, scale=1.5, out_dtype=BF))
    np.testing.assert_allclose(bf, got, rtol=2.0 ** -8, atol=0)


# --------------------------------------------------------------- dispatch ----
def oracle_rows(x, fmt, amax=None):
    if fmt == "nv":
        q, s, G, g = o.nvfp4_quantize(x) if amax is None else o.nvfp4_quantize(x, amax)
        return q, s, G, g
    q, s = o.mxfp4_quantize(x)
    return q, s, None, None


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("T,H,E,k,dtype", [
    (1, 32, 1, 1, torch.float32), (1, 512, 64, 8, BF), (5, 96, 3, 2, torch.float32), (130, 160, 64, 8, BF),
    (1000, 64, 256, 8, BF), (700, 32, 1024, 16, torch.float32), (2049, 32, 7, 4, BF)])
def test_dispatch(fmt, T, H, E, k, dtype):
    announce(f"dispatch {fmt} T={T} H={H} E={E} k={k} {dtype}")
    rng = np.random.default_rng(T + E)
    x = gpu(rng.normal(0, 1, (T, H)).astype(np.float32), dtype)
    ids = rng.integers(-1, E + 1, (T, k)).astype(np.int32)   # -1 and E: dropped slots
    f = fp4.FP4_NVFP4 if fmt == "nv" else fp4.FP4_MXFP4
    q, s, G, g, off, sr, rs = fp4.moe_dispatch(f, x, gpu(ids), E)
    r_off, r_sr, r_rs = ref.sort_slots(ids, E)
    np.testing.assert_array_equal(host(off), r_off)
    np.testing.assert_array_equal(host(sr), r_sr)
    np.testing.assert_array_equal(host(rs), r_rs)
    oq, os_, oG, og = oracle_rows(host(x).astype(np.float32), fmt)
    want_q = np.zeros((T * k, H // 2), np.uint8)
    want_s = np.zeros((T * k, os_.shape[1]), np.uint8)
    live = r_rs >= 0
    want_q[live], want_s[live] = oq[r_rs[live] // k], os_[r_rs[live] // k]
    np.testing.assert_array_equal(host(q), want_q)
    np.testing.assert_array_equal(host(s), want_s)
    if fmt == "nv":
        assert host(G)[0] == np.float32(oG) and host(g)[0] == np.float32(og)


def test_dispatch_given_amax_and_all_dropped():
    rng = np.random.default_rng(3)
    x = gpu(rng.normal(0, 1, (9, 64)).astype(np.float32))
    ids = np.full((9, 2), -1, np.int32)
    q, s, a, g, off, sr, rs = fp4.moe_dispatch(fp4.FP4_NVFP4, x, gpu(ids), 4, amax=6.0)
    assert not host(q).any() and not host(s).any() and not host(off).any()
    assert (host(sr) == -1).all() and (host(rs) == -1).all()
    assert host(g)[0] == np.float32(np.float32(6.0) / np.float32(2688.0))
    ids[:, 0] = 3
    q, s, a, g, off, sr, rs = fp4.moe_dispatch(fp4.FP4_NVFP4, x, gpu(ids), 4, amax=6.0)
    oq, os_, _, _ = oracle_rows(host(x), "nv", np.float32(6.0))
    np.testing.assert_array_equal(host(q)[:9], oq)
    np.testing.assert_array_equal(host(s)[:9], os_)
    np.testing.assert_array_equal(host(off), [0, 0, 0, 0, 9])


def test_dispatch_without_tokens():
    q, s, a, g, off, sr, rs = fp4.moe_dispatch(fp4.FP4_NVFP4, torch.empty(0, 64, device=DEV),
                                               torch.empty(0, 4, dtype=torch.int32, device=DEV), 5)
    assert not host(off).any() and host(a)[0] == 0 and host(g)[0] == 1
    q, s, a, g, off, sr, rs = fp4.moe_dispatch(fp4.FP4_MXFP4, torch.empty(0, 64, device=DEV),
                                               torch.empty(0, 4, dtype=torch.int32, device=DEV), 5)
    assert not host(off).any() and a is None and g is None


def test_dispatch_chunk_boundaries():
    """Slot counts at and around the sort's chunk of 4096 slots, one expert and many."""
    for T, k, E in ((1024, 4, 64), (1025, 4, 64), (2047, 2, 1), (4097, 3, 300)):
        rng = np.random.default_rng(T)
        ids = rng.integers(0, E, (T, k)).astype(np.int32)
        out = fp4.moe_dispatch(fp4.FP4_MXFP4, torch.zeros(T, 32, device=DEV), gpu(ids), E)
        for got, want in zip(out[4:], ref.sort_slots(ids, E)):
            np.testing.assert_array_equal(host(got), want)


# ---------------------------------------------------------------- combine ----
@pytest.mark.parametrize("T,H,k,dtype,out", [
    (1, 1, 1, torch.float32, torch.float32), (3, 7, 2, BF, torch.float32), (5, 8, 8, BF, BF),
    (17, 2056, 3, torch.float32, BF), (33, 512, 16, BF, BF), (2, 4100, 5, torch.float32, torch.float32)])
@pytest.mark.parametrize("with_residual", [False, True])
def test_combine_and_gradients(T, H, k, dtype, out, with_residual):
    announce(f"combine T={T} H={H} k={k} {dtype}->{out} residual={with_residual}")
    rng = np.random.default_rng(T * H + k)
    perm = rng.permutation(T * k).astype(np.int32)
    drop = rng.random(T * k) < 0.2
    # dropped slots have no row: the rows of the others come first
    order = [s for s in perm if not drop[s]]
    rs = np.full(T * k, -1, np.int32)
    rs[:len(order)] = order
    sr = np.full(T * k, -1, np.int32)
    sr[order] = np.arange(len(order))
    sr = sr.reshape(T, k)
    rows = gpu(rng.normal(0, 1, (T * k, H)).astype(np.float32), dtype)
    rows[len(order):] = float("nan")                         # rows of no slot are not read
    w = rng.random((T, k)).astype(np.float32)
    res = gpu(rng.normal(0, 1, (T, H)).astype(np.float32), dtype) if with_residual else None
    y = host(fp4.moe_combine(rows, gpu(w), gpu(sr), residual=res, out_dtype=out))
    R = np.where(np.isnan(host(rows)), 0, host(rows))
    want = ref.combine(R, w, sr, None if res is None else host(res))
    mag = ref.combine(np.abs(R), w, sr, None if res is None else np.abs(host(res)))
    tol = (k + 2) * EPS * mag + (2.0 ** -8 * np.abs(want) if out == BF else 0) + 1e-30
    assert (np.abs(y - want) <= tol).all()

    dy = gpu(rng.normal(0, 1, (T, H)).astype(np.float32), dtype)
    dr, dw = fp4.moe_combine_backward(dy, rows, gpu(w), gpu(sr), gpu(rs), out_dtype=out)
    want_r, want_w = ref.combine_grad(host(dy), R, w, sr)
    _, mag_w = ref.combine_grad(np.abs(host(dy)), np.abs(R), w, sr)
    tol = (EPS + (2.0 ** -8 if out == BF else 0)) * np.abs(want_r)
    assert (np.abs(host(dr) - want_r) <= tol).all()
    assert (np.abs(host(dw) - want_w) <= (H + 2) * EPS * mag_w).all()
    # differences: y is linear in the weights and the rows
    if out == torch.float32 and len(order):
        s = order[0]
        t, j, r = s // k, s % k, 0
        w2 = w.copy()
        w2[t, j] += 1.0
        num = ((ref.combine(R, w2, sr) - ref.combine(R, w, sr)) * host(dy)).sum()
        assert abs(num - host(dw)[t, j]) <= (H + 2) * EPS * mag_w[t, j] + 1e-9


# ---------------------------------------------------- streams, determinism ----
def test_routing_on_another_stream_and_in_a_graph():
    """Route, dispatch and combine on a side stream, then captured and replayed with
    eager work between the replays; every replay equals the eager result."""
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    T, H, E, k = 600, 256, 64, 8
    logits = torch.randn(T, E, generator=g, device=DEV)
    x = torch.randn(T, H, generator=g, device=DEV).to(BF)
    rows = torch.randn(T * k, H, generator=g, device=DEV).to(BF)

    def step():
        ids, w = fp4.moe_route(logits, k)
        out = fp4.moe_dispatch(fp4.FP4_NVFP4, x, ids, E)
        y = fp4.moe_combine(rows, w, out[5])
        dr, dw = fp4.moe_combine_backward(y, rows, w, out[5], out[6])
        dl = fp4.moe_route_backward(dw, logits, ids)
        return [ids, w, *out, y, dr, dw, dl]

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(3):
        g.manual_seed(50 + seed)
        logits.copy_(torch.randn(T, E, generator=g, device=DEV))
        x.copy_(torch.randn(T, H, generator=g, device=DEV).to(BF))
        want = [t.clone() for t in step()]
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b)
