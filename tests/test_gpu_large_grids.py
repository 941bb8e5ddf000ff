"""Calls of 2^24 and more workgroups of 256 threads: a dispatch counts work-items in
32 bits per dimension, so they do not fit one dimension of a grid.  Compared with the
same mathematics in torch where that is exact, else with the rows of a small call."""
import pytest
import torch

import micro_scaled_fp4_amd as fp4
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
WGS = 1 << 24


def needs(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes * 1e9:
        pytest.skip(f"needs {gigabytes} GB of free device memory")


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("H", [8, 7])       # 16-byte accesses, and single elements
def test_combine_and_gradients_of_many_tokens(H):
    T = WGS + 3
    announce(f"combine T={T} H={H}")
    needs(8)
    g = gen(H)
    rows = torch.randn(T, H, generator=g, device=DEV).to(BF)
    w = torch.rand(T, 1, generator=g, device=DEV)
    sr = torch.randperm(T, generator=g, device=DEV).to(torch.int32)
    rs = torch.empty_like(sr)
    rs[sr.long()] = torch.arange(T, dtype=torch.int32, device=DEV)
    sr = sr.view(T, 1)
    y = fp4.moe_combine(rows, w, sr)
    assert torch.equal(y, (w * rows[sr.flatten().long()].float()).to(BF))
    dy = torch.randn(T, H, generator=g, device=DEV).to(BF)
    dr, dw = fp4.moe_combine_backward(dy, rows, w, sr, rs)
    assert torch.equal(dr[sr.flatten().long()], (w * dy.float()).to(BF))
    prod = dy.float() * rows[sr.flatten().long()].float()
    assert ((dw.flatten() - prod.sum(1)).abs() <= 2 * H * 2.0 ** -24 * prod.abs().sum(1)).all()


def test_combine_of_long_rows_by_element():
    """The bound in pieces of a row: 524 288 tokens of 8191 values."""
    T, H = 1 << 19, 8191
    announce(f"combine T={T} H={H}")
    needs(20)
    rows = torch.randn(4, H, generator=gen(1), device=DEV).to(BF)
    sr = (torch.arange(T, device=DEV, dtype=torch.int32) % 4).view(T, 1)
    w = torch.ones(T, 1, device=DEV)
    y = fp4.moe_combine(rows, w, sr)
    for t in (0, 1, T // 2, T - 5, T - 1):
        assert torch.equal(y[t], rows[t % 4])
    assert bool((y.view(T // 4, 4, H) == rows).all())


def test_route_and_gradient_of_the_most_tokens():
    """2^26 tokens of 513 experts: 2^24 workgroups of four tokens."""
    T, E, k = 1 << 26, 513, 1
    announce(f"route T={T} E={E}")
    needs(150)
    base = 1 << 10
    small = torch.randn(base, E, generator=gen(2), device=DEV).to(BF)
    logits = torch.zeros(T, E, dtype=BF, device=DEV)
    at = (0, T // 2, T - base)
    for r in at:
        logits[r:r + base] = small
    ids, w = fp4.moe_route(logits, k, renormalize=False)
    si, sw = fp4.moe_route(small, k, renormalize=False)
    for r in at:
        assert torch.equal(ids[r:r + base], si) and torch.equal(w[r:r + base], sw)
    assert not ids[base:T // 2].any()
    dw = torch.ones(T, k, device=DEV)
    dl = fp4.moe_route_backward(dw, logits, ids, renormalize=False)
    sd = fp4.moe_route_backward(dw[:base], small, si, renormalize=False)
    for r in at:
        assert torch.equal(dl[r:r + base], sd)


def test_epilogue_backward_of_many_groups():
    """2^20 groups of 17 column parts each, most of them empty: bias sums of all."""
    E, N, M = 1 << 20, 2050, 6
    announce(f"epilogue backward E={E} N={N}")
    needs(40)
    z = torch.randn(M, N, generator=gen(3), device=DEV)
    dD = torch.randn(M, N, generator=gen(4), device=DEV)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[1:] = 2
    off[E // 2:] = 3
    off[E:] = 5
    dz, db = fp4.fp4_epilogue_backward(dD, z, fp4.FP4_ACT_NONE, offsets=off, out_dtype=torch.float32)
    assert torch.equal(dz[:5], dD[:5]) and not dz[5:].any()
    assert torch.equal(db[0], dD[0] + dD[1]) and torch.equal(db[E // 2 - 1], dD[2])
    assert torch.equal(db[E - 1], dD[3] + dD[4])
    assert int(torch.count_nonzero(db.abs().amax(1))) == 3


def test_grouped_product_of_many_groups():
    """2^20 groups of 4096 columns, three of them with rows: a launch by the rows, not
    by the 2^24 tiles that as many groups could have."""
    E, N, K, M = 1 << 20, 4096, 32, 5
    announce(f"grouped gemm E={E} N={N} K={K}")
    needs(90)
    A = torch.randint(0, 256, (M, K // 2), dtype=torch.uint8, generator=gen(5), device=DEV)
    sa = torch.full((M, 1), 127, dtype=torch.uint8, device=DEV)
    W = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV)
    sw = torch.full((E, N, 1), 127, dtype=torch.uint8, device=DEV)
    used = (0, E // 2, E - 1)
    for i, e in enumerate(used):
        W[e] = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, generator=gen(6 + i), device=DEV)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[1:] = 2
    off[E // 2 + 1:] = 3
    off[E:] = 5
    rows = ((0, 0, 2), (E // 2, 2, 3), (E - 1, 3, 5))
    D = fp4.fp4_grouped_gemm(fp4.FP4_MXFP4, A, sa, None, W, sw, None, off, K, out_dtype=torch.float32)
    F = fp4.fp4_grouped_gemm_fused(fp4.FP4_MXFP4, A, sa, None, W, sw, None, off, K, out_dtype=torch.float32)
    for e, lo, hi in rows:
        want = fp4.fp4_scaled_gemm(fp4.FP4_MXFP4, A[lo:hi], sa[lo:hi], None, W[e], sw[e], None, K, out_dtype=torch.float32)
        assert torch.equal(D[lo:hi], want) and torch.equal(F[lo:hi], want)
