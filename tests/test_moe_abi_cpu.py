"""Host-side checks of the expert-layer entry points (no GPU needed): bad
arguments come back as their status before anything reaches a device, and the
binding refuses wrong types, shapes and host tensors."""
import ctypes
import os

import numpy as np
import pytest
import torch

import micro_scaled_fp4_amd as m
import moe_reference as ref

pytestmark = pytest.mark.skipif(not os.path.exists(m.LIB_PATH), reason="libfp4.so not built")

OK, NULL, SHAPE, DTYPE, ALIGN, ARCH, WORKSPACE, HIP, ALIAS = range(9)
P = ctypes.c_void_p(4096)       # non-NULL, aligned stand-ins (never dereferenced)
Q = ctypes.c_void_p(8192)
ODD = ctypes.c_void_p(4097)


def dense(fmt=0, A=P, sa=P, ga=P, W=P, sw=P, gb=P, M=8, N=8, K=64, act=0, gated=0, bias=None, bt=0, res=None, rt=0, z=None,
          zt=0, D=Q, dt=1):
    return m.load_library().fp4_scaled_gemm_fused(fmt, A, sa, ga, W, sw, gb, 1.0, M, N, K, act, gated, bias, bt, res, rt, z,
                                                  zt, D, dt, None)


def test_fused_gemm_argument_errors():
    assert dense(fmt=2) == DTYPE
    assert dense(act=5) == DTYPE and dense(act=-1) == DTYPE
    assert dense(dt=2) == DTYPE                                # E4M3 is no fused output
    assert dense(bias=P, bt=2) == DTYPE and dense(res=P, rt=3) == DTYPE and dense(z=P, zt=2) == DTYPE
    assert dense(K=48) == SHAPE and dense(M=-1) == SHAPE
    assert dense(gated=1, N=7) == SHAPE and dense(gated=2) == SHAPE
    assert dense(M=(1 << 30) + 1) == SHAPE and dense(K=1 << 23) == SHAPE
    assert dense(M=1 << 30, N=1 << 30) == SHAPE                # tile bound
    assert dense(fmt=1) == DTYPE                               # MXFP4 takes no tensor scales
    assert dense(A=None) == NULL and dense(ga=None) == NULL and dense(D=None) == NULL
    assert dense(A=ctypes.c_void_p(4104)) == ALIGN and dense(D=ODD) == ALIGN
    assert dense(bias=ODD, bt=1) == ALIGN and dense(res=ctypes.c_void_p(4098), rt=0) == ALIGN and dense(z=ODD) == ALIGN
    assert dense(res=Q, rt=0, dt=1) == ALIAS                   # in place needs equal types
    assert dense(z=Q) == ALIAS and dense(z=P, res=P) == ALIAS
    assert dense(A=None, M=0) == OK and dense(A=None, N=0) == OK
    assert dense(A=None, sa=None, W=None, sw=None, ga=None, gb=None, K=0, D=None) == NULL


def test_grouped_fused_argument_errors():
    lib = m.load_library()

    def g(groups=2, off=P, M=8, N=8, K=64):
        return lib.fp4_grouped_gemm_fused(0, P, P, P, P, P, P, 1.0, groups, off, M, N, K, 0, 0, None, 0, None, 0, None, 0, None,
                                          1, None)

    assert g(groups=0) == SHAPE and g(groups=(1 << 20) + 1) == SHAPE
    assert g(off=None) == NULL and g() == NULL                 # D
    assert g(K=40) == SHAPE and g(M=0) == OK


def test_epilogue_backward_argument_errors():
    lib = m.load_library()
    need = lib.fp4_epilogue_backward_workspace_bytes(1, 1000, 64)
    assert need >= 64 * 4
    assert lib.fp4_epilogue_backward_workspace_bytes(0, 10, 64) == 0

    def b(dD=P, dt=1, z=P, zt=1, groups=1, off=None, M=1000, N=64, act=2, gated=0, dz=Q, dzt=1, db=P, ws=P, n=need):
        return lib.fp4_epilogue_backward(dD, dt, z, zt, groups, off, M, N, act, gated, dz, dzt, db, ws, n, None)

    assert b(dt=2) == DTYPE and b(zt=5) == DTYPE and b(act=9) == DTYPE
    assert b(M=-1) == SHAPE and b(gated=1, N=63) == SHAPE and b(groups=2) == SHAPE and b(groups=0) == SHAPE
    assert b(dD=None) == NULL and b(z=None) == NULL and b(dz=None) == NULL
    assert b(ws=None) == WORKSPACE and b(n=need - 1) == WORKSPACE
    assert b(dD=ODD) == ALIGN and b(db=ctypes.c_void_p(4098)) == ALIGN
    assert b(dz=P, dD=P) == ALIAS and b(dz=P, z=P, dD=Q, dzt=0) == ALIAS
    assert b(N=0) == OK and b(M=0, db=None) == OK


def test_routing_argument_errors():
    lib = m.load_library()

    def r(l=P, lt=0, T=4, E=64, k=8, score=0, bias=None, G=1, tg=1, gt=1, ids=P, w=P):
        return lib.moe_route(l, lt, T, E, k, score, bias, G, tg, gt, 1, 1.0, ids, w, None)

    assert r(lt=2) == DTYPE and r(score=2) == DTYPE
    assert r(E=0) == SHAPE and r(E=1025) == SHAPE and r(k=0) == SHAPE and r(k=17) == SHAPE and r(E=4, k=5) == SHAPE
    assert r(G=0) == SHAPE and r(G=3) == SHAPE and r(G=65, E=65 * 2) == SHAPE and r(G=4, tg=5) == SHAPE
    assert r(G=4, tg=0) == SHAPE and r(gt=3) == SHAPE and r(T=-1) == SHAPE and r(T=(1 << 26) + 1) == SHAPE
    assert r(l=None) == NULL and r(ids=None) == NULL and r(w=None) == NULL
    assert r(l=ODD) == ALIGN and r(bias=ODD) == ALIGN
    assert r(l=None, T=0) == OK

    def rb(dw=P, l=P, lt=0, ids=P, T=4, E=64, k=8, dl=P, dt=0):
        return lib.moe_route_backward(dw, l, lt, ids, T, E, k, 0, 1, 1.0, dl, dt, None)

    assert rb(lt=2) == DTYPE and rb(dt=2) == DTYPE and rb(k=65) == SHAPE
    assert rb(dw=None) == NULL and rb(dl=None) == NULL and rb(ids=ODD) == ALIGN and rb(T=0) == OK


def test_dispatch_and_combine_argument_errors():
    lib = m.load_library()
    need = lib.moe_dispatch_workspace_bytes(4096, 8, 64)
    assert need >= 4096 and lib.moe_dispatch_workspace_bytes(4096, 17, 64) == 0

    def d(fmt=0, x=P, xt=1, T=4096, H=64, ids=P, k=8, E=64, q=P, s=P, a=P, given=0, g=Q, off=P, sr=P, rs=P, ws=P, n=need):
        return lib.moe_dispatch(fmt, x, xt, T, H, ids, k, E, q, s, a, given, g, off, sr, rs, ws, n, None)

    assert d(fmt=3) == DTYPE and d(xt=2) == DTYPE and d(fmt=1) == DTYPE
    assert d(H=48) == SHAPE and d(E=2000) == SHAPE and d(k=0) == SHAPE and d(T=-1) == SHAPE
    assert d(x=None) == NULL and d(ids=None) == NULL and d(off=None) == NULL and d(g=None) == NULL
    assert d(a=None, given=1) == NULL and d(sr=None) == NULL
    assert d(ws=None) == WORKSPACE and d(n=need - 1) == WORKSPACE
    assert d(q=ctypes.c_void_p(4104)) == ALIGN and d(x=ODD) == ALIGN
    assert d(g=P) == ALIAS

    def c(rows=P, rt=1, M=8, H=64, w=P, sr=P, T=4, k=2, res=None, rst=0, y=Q, yt=1):
        return lib.moe_combine(rows, rt, M, H, w, sr, T, k, res, rst, y, yt, None)

    assert c(rt=2) == DTYPE and c(res=P, rst=2) == DTYPE and c(k=17) == SHAPE and c(M=-1) == SHAPE and c(H=-1) == SHAPE
    assert c(rows=None) == NULL and c(w=None) == NULL and c(y=None) == NULL
    assert c(y=ODD) == ALIGN and c(y=P) == ALIAS and c(res=Q, rst=0, yt=1) == ALIAS
    assert c(T=0) == OK and c(H=0) == OK

    def cb(dy=P, rows=P, w=P, sr=P, rs=P, T=4, k=2, H=64, dr=Q, dw=P):
        return lib.moe_combine_backward(dy, 1, rows, 1, w, sr, rs, T, k, H, dr, 1, dw, None)

    assert cb(k=0) == SHAPE and cb(dy=None) == NULL and cb(rs=None) == NULL and cb(dw=None) == NULL
    assert cb(dr=P) == ALIAS and cb(dw=ODD) == ALIGN and cb(T=0) == OK


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64)
    for call in (lambda: m.moe_route(x, 2), lambda: m.moe_dispatch(0, x, torch.zeros(4, 2, dtype=torch.int32), 4),
                 lambda: m.moe_combine(x, torch.zeros(2, 2), torch.zeros(2, 2, dtype=torch.int32)),
                 lambda: m.fp4_epilogue_backward(x, x, 0)):
        with pytest.raises(ValueError):
            call()


# ---- the 64-bit forms themselves ----
def test_reference_activations_and_gradients():
    torch_act = {ref.RELU: torch.relu, ref.SILU: torch.nn.functional.silu, ref.GELU: torch.nn.functional.gelu,
                 ref.GELU_TANH: lambda x: torch.nn.functional.gelu(x, approximate="tanh"), ref.NONE: lambda x: x}
    z = torch.linspace(-9, 9, 397, dtype=torch.float64, requires_grad=True)
    for a, f in torch_act.items():
        y = f(z)
        g, = torch.autograd.grad(y.sum(), z)
        np.testing.assert_allclose(ref.act(z.detach().numpy(), a), y.detach().numpy(), rtol=1e-12, atol=1e-15)
        np.testing.assert_allclose(ref.act_grad(z.detach().numpy(), a), g.numpy(), rtol=1e-9, atol=1e-12)


def test_reference_routing_by_hand():
    l = np.array([[0.0, 1.0, 1.0, -np.inf], [np.nan] * 4], np.float32)
    ids, w, _ = ref.route(l, 3, False)
    assert ids.tolist() == [[1, 2, 0], [-1, -1, -1]]
    e = np.exp(-1.0)
    np.testing.assert_allclose(w[0], np.array([1, 1, e]) / (2 + e))
    assert (w[1] == 0).all()
    # groups of two: {0, 1} sums to 1.0 + 0.9, {2, 3} to 1.1 + 0.1
    v = np.log(np.array([[1.0, 0.9, 1.1, 0.1]]) / 4).astype(np.float32)
    assert ref.route(v, 2, False, groups=2, top_groups=1, group_top=2)[0].tolist() == [[0, 1]]
    assert ref.route(v, 2, False, groups=2, top_groups=1, group_top=1)[0].tolist() == [[2, 3]]
    off, sr, rs = ref.sort_slots(np.array([[2, 0], [0, 5], [2, -1]]), 3)
    assert off.tolist() == [0, 2, 2, 4] and sr.tolist() == [[2, 0], [1, -1], [3, -1]] and rs.tolist() == [1, 2, 0, 4, -1, -1]


def test_reference_checks_find_planted_mistakes():
    rng = np.random.default_rng(1)
    l = rng.normal(0, 1, (3, 8))
    ids, w, _ = ref.route(l, 2, False)
    g = ref.route_grad(np.ones_like(w), l, ids, False, False, 1.0)
    h = 1e-6
    up, dn = l.copy(), l.copy()
    up[0, 3] += h
    dn[0, 3] -= h
    num = (ref.route_weights(up, ids, False, False, 1.0) - ref.route_weights(dn, ids, False, False, 1.0)).sum() / (2 * h)
    assert abs(num - g[0, 3]) < 1e-6
    wrong = ref.route_grad(np.ones_like(w), l, ids[:, ::-1][:, :1].repeat(2, 1), False, False, 1.0)
    assert np.abs(wrong - g).max() > 1e-3
