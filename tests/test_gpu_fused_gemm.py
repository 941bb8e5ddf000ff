"""GPU parity: FP4 products with bias, activation and residual in the epilogue,
dense and grouped, and the epilogue's backward pass, against 64-bit plain forms.

Tolerances.  z: the product rule of the GEMM, 1e-5 |g_d| sum |a w|, and the
rounding of the sum with the bias, 2^-23 (|z| + |bias|).  Through an activation
(slope at most 1.2) that error grows by at most 1.2, and the activation adds its
own: its exponential's argument is rounded once or twice, 4e-6 (1 + |x|) relative.
The residual's sum adds 2^-23 of its terms, a bf16 output 2^-8 relative.
"""
import numpy as np
import pytest
import torch

import micro_scaled_fp4_amd as fp4
import moe_reference as ref
import workloads
from oracle import fp4_oracle as o
from gpu_util import DEV, announce, to_gpu_u8

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
E23 = 2.0 ** -23


def gpu(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32))
    return (t if dtype is None else t.to(dtype)).to(DEV)


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def operand(fmt, rows, K, seed, groups=0):
    """Random codes and scale bytes (values of order 1 after the tensor scale)."""
    n = rows * max(groups, 1)
    q = workloads.random_codes((n, K // 2), seed)
    if fmt == "nv":
        s = workloads.random_bytes((n, K // 16), 0x20, 0x40, seed + 1)
        g = np.random.default_rng(seed).uniform(0.02, 0.1, max(groups, 1)).astype(np.float32)
    else:
        s = workloads.random_bytes((n, K // 32), 120, 124, seed + 1)
        g = None
    return q, s, g


def values(fmt, q, s, g, K):
    return o.nv_operand_f64(q, s, g, K) if fmt == "nv" else o.mx_operand_f64(q, s, K)


def check(D, z_ref, z_err, bias, act, gated, residual, out):
    """D against the epilogue of z_ref, z off by at most z_err."""
    z_err = z_err + E23 * (np.abs(z_ref) + (0 if bias is None else np.abs(bias)))
    want = ref.epilogue(z_ref, act, gated, residual)
    own = lambda x: 4e-6 * (1 + np.abs(x)) * np.abs(ref.act(x, act)) + 1e-12  # noqa: E731
    if gated:
        g, u = z_ref[..., 0::2], z_ref[..., 1::2]
        eg, eu = z_err[..., 0::2], z_err[..., 1::2]
        fg = ref.act(g, act)
        tol = (1.2 * eg + own(g)) * (np.abs(u) + eu) + np.abs(fg) * eu + E23 * np.abs(fg * u)
    else:
        tol = 1.2 * z_err + own(z_ref)
    tol = tol + E23 * (np.abs(want) + (0 if residual is None else np.abs(residual)))
    if out == BF:
        tol = tol + 2.0 ** -8 * np.abs(want)
    bad = ~(np.abs(D - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], D[bad][:5], want[bad][:5], tol[bad][:5])


def run_dense(fmt, M, N, K, act, gated, bias_t, res_t, out, pre_t, seed, g_d=1.0):
    f = fp4.FP4_NVFP4 if fmt == "nv" else fp4.FP4_MXFP4
    qa, sa, ga = operand(fmt, M, K, seed)
    qw, sw, gw = operand(fmt, N, K, seed + 10)
    rng = np.random.default_rng(seed)
    bias = None if bias_t is None else gpu(rng.normal(0, 1, N), bias_t)
    No = N // 2 if gated else N
    res = None if res_t is None else gpu(rng.normal(0, 1, (M, No)), res_t)
    t = lambda g: None if g is None else torch.from_numpy(g).to(DEV)  # noqa: E731
    got = fp4.fp4_scaled_gemm_fused(f, to_gpu_u8(qa), to_gpu_u8(sa), t(ga), to_gpu_u8(qw), to_gpu_u8(sw), t(gw), K,
                                    g_d, activation=act, gated=gated, bias=bias, residual=res, preact_dtype=pre_t,
                                    out_dtype=out)
    D, z = got if pre_t is not None else (got, None)
    A = values(fmt, qa, sa, None if ga is None else ga[0], K)
    W = values(fmt, qw, sw, None if gw is None else gw[0], K)
    b = None if bias is None else host(bias)
    z_ref = g_d * (A @ W.T) + (0 if b is None else b)
    z_err = 1e-5 * abs(g_d) * (np.abs(A) @ np.abs(W).T)
    check(host(D), z_ref, z_err, b, act, gated, None if res is None else host(res), out)
    if z is not None:
        tol = z_err + E23 * (np.abs(z_ref) + (0 if b is None else np.abs(b))) + (2.0 ** -8 * np.abs(z_ref) if pre_t == BF else 0)
        assert (np.abs(host(z) - z_ref) <= tol).all()


ACTS = sorted(ref.ACTS.items())


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("name,act", ACTS)
@pytest.mark.parametrize("gated", [False, True])
def test_every_activation(fmt, name, act, gated):
    announce(f"fused gemm {fmt} {name} gated={gated}")
    run_dense(fmt, 70, 96, 288, act, gated, F32, BF, F32, F32, 7, -0.5)
    run_dense(fmt, 70, 96, 256, act, gated, None, None, BF, None, 8)


SHAPES = [(1, 1, 32), (1, 16, 64), (2, 27, 96), (3, 130, 512), (5, 1000, 1056), (16, 272, 2048), (17, 515, 320),
          (31, 64, 7168), (33, 48, 256), (64, 300, 1024), (65, 256, 512), (257, 272, 768), (300, 521, 1056),
          (255, 1030, 288)]


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_sizes(fmt, M, N, K):
    announce(f"fused gemm {fmt} {M}x{N}x{K}")
    run_dense(fmt, M, N, K, ref.SILU, False, BF, F32, F32, BF, M + N)
    run_dense(fmt, M, N, K, ref.GELU, N % 2 == 0, F32, BF, BF, None, M + K, 0.25)
    run_dense(fmt, M, N, K, ref.NONE, False, None, None, F32, None, N + K)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_more_tiles_than_compute_units(fmt):
    """Persistent workgroups: several tiles each, ragged edges, the next tile's
    operands in flight during the epilogue."""
    announce(f"fused gemm {fmt} many tiles")
    run_dense(fmt, 2100, 8496, 256, ref.SILU, True, BF, BF, BF, None, 3)
    run_dense(fmt, 1111, 16404, 288, ref.GELU_TANH, False, F32, F32, F32, F32, 4)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M,N,K,gated,pre", [(3001, 2995, 544, False, BF), (2900, 3008, 1088, True, F32),
                                             (2817, 3010, 800, True, None)])
def test_tile_sizes(fmt, M, N, K, gated, pre):
    """Sizes of many tiles, with edges in every direction."""
    announce(f"fused gemm tiles {fmt} {M}x{N}x{K}")
    run_dense(fmt, M, N, K, ref.SILU, gated, BF, F32, F32, pre, M)
    run_dense(fmt, M, N, K, ref.GELU_TANH, gated, None, BF, BF, None, N)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M,N,K,gated,pre", [(4081, 4001, 1056, False, BF), (4096, 4016, 1280, True, F32)])
def test_large_sizes(fmt, M, N, K, gated, pre):
    """Outputs that fill the device with 256 x 256 tiles."""
    announce(f"fused gemm large {fmt} {M}x{N}x{K}")
    run_dense(fmt, M, N, K, ref.SILU, gated, BF, F32, F32, pre, M)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("N,K", [(16404, 288), (16400, 544), (16400, 512)])
def test_short_contractions_repeat(fmt, N, K):
    """One to three stages per tile, several tiles per compute unit: the same bits
    on every run, with other inputs' tiles in shared memory in between."""
    announce(f"fused gemm short {fmt} N={N} K={K}")
    f, M = (fp4.FP4_NVFP4 if fmt == "nv" else fp4.FP4_MXFP4), 1111
    t = lambda g: None if g is None else torch.from_numpy(g).to(DEV)  # noqa: E731
    args = []
    for seed in (1, 2):
        qa, sa, ga = operand(fmt, M, K, seed)
        qw, sw, gw = operand(fmt, N, K, seed + 10)
        args.append((f, to_gpu_u8(qa), to_gpu_u8(sa), t(ga), to_gpu_u8(qw), to_gpu_u8(sw), t(gw), K))
    want = [fp4.fp4_scaled_gemm(*a, out_dtype=F32) for a in args]
    for i in range(12):
        got = fp4.fp4_scaled_gemm_fused(*args[i & 1], out_dtype=F32)
        assert ((got - want[i & 1]).abs() <= 1e-4 * want[i & 1].abs().max()).all()
        if i < 2:
            first = (got,) if i == 0 else first + (got,)
        assert torch.equal(got, first[i & 1])


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_equals_the_plain_gemm_without_an_epilogue(fmt):
    f = fp4.FP4_NVFP4 if fmt == "nv" else fp4.FP4_MXFP4
    M, N, K = 300, 304, 768
    qa, sa, ga = operand(fmt, M, K, 1)
    qw, sw, gw = operand(fmt, N, K, 2)
    t = lambda g: None if g is None else torch.from_numpy(g).to(DEV)  # noqa: E731
    args = (f, to_gpu_u8(qa), to_gpu_u8(sa), t(ga), to_gpu_u8(qw), to_gpu_u8(sw), t(gw), K, 0.75)
    assert torch.equal(fp4.fp4_scaled_gemm_fused(*args, out_dtype=F32), fp4.fp4_scaled_gemm(*args, out_dtype=F32))
    assert torch.equal(fp4.fp4_scaled_gemm_fused(*args), fp4.fp4_scaled_gemm(*args))


@pytest.mark.parametrize("M", [4, 300])
@pytest.mark.parametrize("out", [BF, F32])
def test_residual_in_place_and_misaligned(M, out):
    """The residual may be the output; pointers aligned to their element only."""
    N, K = 272, 320
    qa, sa, ga = operand("nv", M, K, 5)
    qw, sw, gw = operand("nv", N, K, 6)
    t = lambda g: torch.from_numpy(g).to(DEV)  # noqa: E731
    args = (fp4.FP4_NVFP4, to_gpu_u8(qa), to_gpu_u8(sa), t(ga), to_gpu_u8(qw), to_gpu_u8(sw), t(gw), K)
    rng = np.random.default_rng(5)
    res = gpu(rng.normal(0, 1, (M, N)), out)
    bias = gpu(rng.normal(0, 1, N), out)
    want = fp4.fp4_scaled_gemm_fused(*args, activation=ref.SILU, bias=bias, residual=res, out_dtype=out)
    into = res.clone()
    fp4.fp4_scaled_gemm_fused(*args, activation=ref.SILU, bias=bias, residual=into, out=into)
    assert torch.equal(into, want)
    off = lambda x: torch.cat([x.new_zeros(1), x.flatten()])[1:].view(x.shape)  # noqa: E731
    got = fp4.fp4_scaled_gemm_fused(*args, activation=ref.SILU, bias=off(bias), residual=off(res),
                                    out=off(torch.zeros_like(res)))
    assert torch.equal(got, want)


def test_empty_contraction_and_empty_sizes():
    e = lambda *s: torch.empty(*s, dtype=torch.uint8, device=DEV)  # noqa: E731
    rng = np.random.default_rng(0)
    bias, res = gpu(rng.normal(0, 1, 40)), gpu(rng.normal(0, 1, (7, 40)))
    for fmt, g in ((fp4.FP4_NVFP4, torch.ones(1, device=DEV)), (fp4.FP4_MXFP4, None)):
        D = fp4.fp4_scaled_gemm_fused(fmt, e(7, 0), e(7, 0), g, e(40, 0), e(40, 0), g, 0, activation=ref.SILU,
                                      bias=bias, residual=res, out_dtype=F32)
        want = ref.epilogue(np.broadcast_to(host(bias), (7, 40)), ref.SILU, False, host(res))
        assert np.abs(host(D) - want).max() < 1e-5
        assert fp4.fp4_scaled_gemm_fused(fmt, e(0, 32), e(0, 4), g, e(8, 32), e(8, 4), g, 64).shape == (0, 8)
        off = torch.zeros(4, dtype=torch.int32, device=DEV)
        off[1:] = torch.tensor([3, 3, 7])
        D = fp4.fp4_grouped_gemm_fused(fmt, e(7, 0), e(7, 0), g, e(3, 40, 0), e(3, 40, 0),
                                       None if g is None else torch.ones(3, device=DEV), off, 0,
                                       bias=bias.repeat(3, 1), out_dtype=F32)
        assert np.abs(host(D) - host(bias)).max() < 1e-6


# ---------------------------------------------------------------- grouped ----
GROUPS = [([1], 16, 32), ([0, 1, 3, 0, 16, 17], 130, 320), ([2] * 60, 272, 1024), ([5, 0, 33, 64, 65, 1, 0], 96, 544),
          ([300], 96, 256), ([0, 17, 256, 300], 258, 1056), ([40, 0, 1, 513, 77, 0, 255, 256], 520, 512), ([0, 0], 32, 64),
          ([1] * 100 + [31], 64, 7168), ([700, 0, 1, 513, 900, 255, 256, 300], 3006, 544),
          ([0, 5, 130, 0, 128, 300, 1, 0], 200, 512), ([1800, 1850], 4002, 1056)]


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("case", range(len(GROUPS)))
@pytest.mark.parametrize("tail", [0, 9])
def test_grouped(fmt, case, tail):
    """tail: rows past the last group (dropped slots), which become zeros."""
    sizes, N, K = GROUPS[case]
    announce(f"fused grouped gemm {fmt} E={len(sizes)} N={N} K={K} tail={tail}")
    E, M = len(sizes), int(sum(sizes)) + tail
    if M == 0:
        return
    f = fp4.FP4_NVFP4 if fmt == "nv" else fp4.FP4_MXFP4
    qa, sa, ga = operand(fmt, M, K, case)
    qw, sw, gw = operand(fmt, N, K, case + 20, E)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    rng = np.random.default_rng(case)
    t = lambda g: None if g is None else torch.from_numpy(g).to(DEV)  # noqa: E731
    A = values(fmt, qa, sa, None if ga is None else ga[0], K)
    W = np.stack([values(fmt, qw[e * N:(e + 1) * N], sw[e * N:(e + 1) * N], None if gw is None else gw[e], K)
                  for e in range(E)])
    for act, gated, bias_t, out, pre in ((ref.SILU, True, F32, BF, None), (ref.GELU, False, BF, F32, F32),
                                         (ref.NONE, False, None, BF, BF)):
        bias = None if bias_t is None else gpu(rng.normal(0, 1, (E, N)), bias_t)
        res = gpu(rng.normal(0, 1, (M, N // 2 if gated else N)), out) if act == ref.GELU else None
        got = fp4.fp4_grouped_gemm_fused(f, to_gpu_u8(qa), to_gpu_u8(sa), t(ga), to_gpu_u8(qw).view(E, N, -1),
                                         to_gpu_u8(sw).view(E, N, -1), t(gw), t(off), K, 0.5, activation=act, gated=gated,
                                         bias=bias, residual=res, preact_dtype=pre, out_dtype=out)
        D, z = got if pre is not None else (got, None)
        for e in range(E):
            r = slice(off[e], off[e + 1])
            b = None if bias is None else host(bias)[e]
            z_ref = 0.5 * (A[r] @ W[e].T) + (0 if b is None else b)
            z_err = 0.5e-5 * (np.abs(A[r]) @ np.abs(W[e]).T)
            check(host(D)[r], z_ref, z_err, b, act, gated, None if res is None else host(res)[r], out)
            if z is not None:
                tol = z_err + E23 * (np.abs(z_ref) + (0 if b is None else np.abs(b))) + (2.0 ** -8 * np.abs(z_ref) if pre == BF else 0)
                assert (np.abs(host(z)[r] - z_ref) <= tol).all()
        assert (host(D)[off[-1]:] == 0).all()
        if z is not None:
            assert (host(z)[off[-1]:] == 0).all()


# --------------------------------------------------------------- backward ----
@pytest.mark.parametrize("name,act", ACTS)
@pytest.mark.parametrize("gated", [False, True])
def test_epilogue_backward_matches_formula_and_differences(name, act, gated):
    rng = np.random.default_rng(act)
    M, N = 37, 64
    No = N // 2 if gated else N
    z = rng.normal(0, 2, (M, N)).astype(np.float32)
    z[0, :8] = [0.0, -0.0, 30.0, -30.0, 5.0, -5.0, 9.0, -9.0]
    dD = rng.normal(0, 1, (M, No)).astype(np.float32)
    dz, db = fp4.fp4_epilogue_backward(gpu(dD), gpu(z), act, gated=gated, out_dtype=F32)
    want = ref.epilogue_grad(dD.astype(np.float64), z.astype(np.float64), act, gated)
    # derivative: the activation's own error and 1 - s, s (1 - s): 1e-5 (1 + |z|) of the factors
    fac = np.abs(np.repeat(dD, 2, axis=1) if gated else dD)
    if gated:
        fac = fac * np.maximum(1, np.repeat(np.abs(z[:, 1::2]), 2, axis=1)) * np.maximum(1, np.abs(z))
    tol = 1e-5 * (1 + np.abs(z)) * fac + 1e-9
    assert (np.abs(host(dz) - want) <= tol).all()
    assert (np.abs(host(db) - want.sum(0)) <= tol.sum(0) + M * 2.0 ** -24 * np.abs(want).sum(0)).all()
    # central differences of the 64-bit epilogue
    h = 1e-5
    for _ in range(40):
        i, j = rng.integers(1, M), rng.integers(0, N)
        if act == ref.RELU and abs(z[i, j]) < 1e-3:
            continue
        up, dn = z.astype(np.float64), z.astype(np.float64)
        up[i, j] += h
        dn[i, j] -= h
        num = ((ref.epilogue(up[i], act, gated) - ref.epilogue(dn[i], act, gated)) * dD[i]).sum() / (2 * h)
        assert abs(num - host(dz)[i, j]) <= tol[i, j] + 1e-6 * (1 + abs(num))


@pytest.mark.parametrize("M,N,gated", [(1, 1, False), (3, 2, True), (1000, 17, False), (500, 1030, True),
                                       (4099, 528, True), (129, 4112, False), (0, 48, False)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_epilogue_backward_sizes(M, N, gated, dtype):
    announce(f"epilogue backward {M}x{N} gated={gated} {dtype}")
    rng = np.random.default_rng(M + N)
    z = gpu(rng.normal(0, 2, (M, N)), dtype)
    dD = gpu(rng.normal(0, 1, (M, N // 2 if gated else N)), dtype)
    dz, db = fp4.fp4_epilogue_backward(dD, z, ref.SILU, gated=gated, out_dtype=dtype)
    zh, dh = host(z), host(dD)
    want = ref.epilogue_grad(dh, zh, ref.SILU, gated)
    tol = 4e-5 * (1 + np.abs(zh)) * (np.repeat(np.abs(dh), 2, axis=1) * (1 + np.repeat(np.abs(zh[:, 1::2]), 2, axis=1))
                                     * (1 + np.abs(zh)) if gated else np.abs(dh))
    sum_tol = tol.sum(0) + (M + 8) * 2.0 ** -24 * np.abs(want).sum(0) + 1e-30
    if dtype == BF:
        tol = tol + 2.0 ** -8 * np.abs(want)
    assert (np.abs(host(dz) - want) <= tol).all()
    assert (np.abs(host(db) - want.sum(0)) <= sum_tol).all()
    again = fp4.fp4_epilogue_backward(dD, z, ref.SILU, gated=gated, out_dtype=dtype)
    assert torch.equal(again[0], dz) and torch.equal(again[1], db)


def test_epilogue_backward_grouped():
    sizes = [0, 3, 200, 0, 1, 90, 0]
    E, N, tail = len(sizes), 80, 4
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    M = int(off[-1]) + tail
    rng = np.random.default_rng(9)
    z, dD = gpu(rng.normal(0, 2, (M, N))), gpu(rng.normal(0, 1, (M, N // 2)))
    dz, db = fp4.fp4_epilogue_backward(dD, z, ref.GELU, gated=True, offsets=torch.from_numpy(off).to(DEV), out_dtype=F32)
    want = ref.epilogue_grad(host(dD), host(z), ref.GELU, True)
    r = slice(0, off[-1])
    assert np.abs(host(dz)[r] - want[r]).max() < 1e-4
    for e in range(E):
        w = want[off[e]:off[e + 1]]
        assert (np.abs(host(db)[e] - w.sum(0)) <= 1e-4 * (1 + np.abs(w).sum(0))).all()
        if sizes[e] == 0:
            assert (host(db)[e] == 0).all()


def test_on_another_stream_and_in_a_graph():
    """Dense, grouped and backward calls on a side stream, then captured; three
    replays with new inputs against the eager results."""
    M, N, K, E = 70, 96, 512, 5
    qa, sa, ga = operand("nv", M, K, 1)
    qw, sw, gw = operand("nv", N, K, 2, E)
    t = lambda g: torch.from_numpy(g).to(DEV)  # noqa: E731
    A, SA, W, SW = to_gpu_u8(qa), to_gpu_u8(sa), to_gpu_u8(qw).view(E, N, -1), to_gpu_u8(sw).view(E, N, -1)
    GA, GW = t(ga), t(gw)
    off = torch.tensor([0, 10, 10, 41, 60, 66], dtype=torch.int32, device=DEV)
    res = torch.randn(M, N // 2, device=DEV)

    def step():
        d, z = fp4.fp4_scaled_gemm_fused(fp4.FP4_NVFP4, A, SA, GA, W[0], SW[0], GW[:1], K, activation=ref.SILU, gated=True,
                                         residual=res, preact_dtype=F32, out_dtype=F32)
        e = fp4.fp4_grouped_gemm_fused(fp4.FP4_NVFP4, A, SA, GA, W, SW, GW, off, K, activation=ref.GELU, gated=True)
        dz, db = fp4.fp4_epilogue_backward(d, z, ref.SILU, gated=True)
        return [d, z, e, dz, db]

    want = [x.clone() for x in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(3):
        res.copy_(torch.randn(M, N // 2, device=DEV))
        A.copy_(torch.randint(0, 256, A.shape, dtype=torch.uint8, device=DEV))
        want = [x.clone() for x in step()]
        for x in held:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
