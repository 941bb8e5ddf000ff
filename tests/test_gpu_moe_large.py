"""Expert-layer operators past 32-bit byte and element offsets: the rows beyond
each boundary equal those of a small call on the same inputs, bit for bit."""
import pytest
import torch

import micro_scaled_fp4_amd as fp4
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rand(seed, *shape):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV)


def test_route_past_32_bit_offsets():
    """4.5 GB of logits: 2.2 M tokens x 1024 experts, and their gradient."""
    base, T, E, k = 64, 64 * 34400, 1024, 8
    announce(f"route {T}x{E}")
    small = rand(1, base, E).to(BF)
    logits = small.repeat(T // base, 1)
    ids, w = fp4.moe_route(logits, k)
    si, sw = fp4.moe_route(small, k)
    dw = rand(2, base, k)
    dl = fp4.moe_route_backward(dw.repeat(T // base, 1), logits, ids)
    sd = fp4.moe_route_backward(dw, small, si)
    for r in (0, T // 2, T - 2 * base, T - base):
        r = r // base * base
        assert torch.equal(ids[r:r + base], si) and torch.equal(w[r:r + base], sw)
        assert torch.equal(dl[r:r + base], sd)


def test_dispatch_and_combine_past_32_bit_offsets():
    """1.1 M rows of 8192 values: 4.6 GB of codes, 18 GB of expert outputs."""
    base, T, H, E, k = 32, 32 * 4400, 8192, 64, 8
    announce(f"dispatch {T}x{H} top {k}")
    small = rand(3, base, H).to(BF)
    x = small.repeat(T // base, 1)
    ids = torch.argsort(rand(4, T, E), dim=1)[:, :k].to(torch.int32)
    q, s, a, g, off, sr, rs = fp4.moe_dispatch(fp4.FP4_NVFP4, x, ids, E)
    qs, ss, _, gs = fp4.nvfp4_quantize(small)
    assert torch.equal(g, gs) and int(off[-1]) == T * k
    assert torch.equal(rs[sr.flatten().long()], torch.arange(T * k, device=DEV, dtype=torch.int32))
    per = torch.bincount(ids.flatten().long(), minlength=E)
    assert torch.equal(off[1:] - off[:-1], per.to(torch.int32))
    for r in (0, 524288, 1048576, T * k - 64):     # both sides of byte 2^31 and 2^32 of the codes
        rows = torch.arange(max(0, r - 32), r + 32, device=DEV)
        tok = rs[rows].long() // k % base
        assert torch.equal(q[rows], qs[tok]) and torch.equal(s[rows], ss[tok])
    del q, s, x
    rows = small.float().to(BF).repeat(T * k // base, 1)   # row r holds row r % base
    w = torch.rand(T, k, device=DEV)
    y = fp4.moe_combine(rows, w, sr)
    dy = small.repeat(T // base, 1)
    dr, dw = fp4.moe_combine_backward(dy, rows, w, sr, rs)
    for t in (0, T // 2, T - 1):
        at = sr[t].long()
        ones = torch.arange(k, dtype=torch.int32, device=DEV)
        ys = fp4.moe_combine(rows[at], w[t:t + 1], ones[None])
        ds, ws = fp4.moe_combine_backward(dy[t:t + 1], rows[at], w[t:t + 1], ones[None], ones)
        assert torch.equal(y[t:t + 1], ys) and torch.equal(dr[at], ds) and torch.equal(dw[t:t + 1], ws)


@pytest.mark.parametrize("rows", [2, 300])
def test_grouped_product_past_32_bit_offsets(rows):
    """300 experts of 4096 x 8192: 5 GB of codes; few rows, and tiles."""
    E, N, K = 300, 4096, 8192
    announce(f"fused grouped gemm E={E} {rows}x{N}x{K}")
    W = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device=DEV)
    sw = torch.randint(0x20, 0x40, (E, N, K // 16), dtype=torch.uint8, device=DEV)
    gw = torch.rand(E, device=DEV) + 0.5
    M = E * rows
    A = torch.randint(0, 256, (M, K // 2), dtype=torch.uint8, device=DEV)
    sa = torch.randint(0x20, 0x40, (M, K // 16), dtype=torch.uint8, device=DEV)
    ga = torch.full((1,), 2.0 ** -9, device=DEV)
    off = torch.arange(0, M + 1, rows, dtype=torch.int32, device=DEV)
    bias = rand(5, E, N)
    D = fp4.fp4_grouped_gemm_fused(fp4.FP4_NVFP4, A, sa, ga, W, sw, gw, off, K, activation=fp4.FP4_ACT_SILU, gated=True,
                                   bias=bias, out_dtype=torch.float32)
    for e in (0, 127, 128, 129, 255, 256, 257, E - 1):
        r = slice(e * rows, (e + 1) * rows)
        one = fp4.fp4_grouped_gemm_fused(fp4.FP4_NVFP4, A[r], sa[r], ga, W[e:e + 1], sw[e:e + 1], gw[e:e + 1],
                                         torch.tensor([0, rows], dtype=torch.int32, device=DEV), K,
                                         activation=fp4.FP4_ACT_SILU, gated=True, bias=bias[e:e + 1],
                                         out_dtype=torch.float32)
        # (another split of K may round differently: the products' float32 rule)
        torch.testing.assert_close(D[r], one, rtol=1e-4, atol=1e-4 * float(D[r].abs().max()))


def test_epilogue_backward_past_32_bit_offsets():
    """2.2 G pre-activations (4.4 GB in bf16)."""
    base, M, N = 64, 64 * 4200, 8192
    announce(f"epilogue backward {M}x{N}")
    z, d = rand(6, base, N).to(BF), rand(7, base, N // 2).to(BF)
    dz, db = fp4.fp4_epilogue_backward(d.repeat(M // base, 1), z.repeat(M // base, 1), fp4.FP4_ACT_SILU, gated=True)
    sz, sb = fp4.fp4_epilogue_backward(d, z, fp4.FP4_ACT_SILU, gated=True)
    for r in (0, M // 2 // base * base, M - base):
        assert torch.equal(dz[r:r + base], sz)
    torch.testing.assert_close(db, sb * (M // base), rtol=1e-3, atol=1e-3 * float(sb.abs().max()) * (M // base))
