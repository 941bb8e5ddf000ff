"""GPU: caches past 2^32 bytes, a context past a million positions, query tensors past 2^31 elements."""
import numpy as np
import pytest
import torch

import kv_reference as ref
import micro_scaled_fp4_amd as fp4
from gpu_util import DEV, announce
from test_gpu_kv_attention import check, queries
from test_gpu_kv_cache import gpu_cache, i32, tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [ref.NV, ref.MX])
def test_pages_past_32_bit_offsets(fmt):
    """Codes of 9 GB: a sequence on the first and the last pages."""
    announce(f"kv cache past 32 bits fmt {fmt}")
    H, D, page, num = 8, 256, 64, 140000        # 65536 bytes of codes a page
    case = ref.Case(fmt, H, D, page, [(300, 300)], seed=1)
    bs = ref.block(fmt)
    cache = fp4.KVCache(fmt, *[torch.zeros(num, H, page, w, dtype=torch.uint8, device=DEV) for w in (D // 2, D // bs, D // 2, D // bs)],
                        *case.amaxes())
    pages = i32([[num - 1, 0, 70000, num - 2, 33333]])
    k, v = (torch.from_numpy(t[0]).to(DEV) for t in (case.k, case.v))
    off, ln = i32([0, 300]), i32([300])
    fp4.kv_cache_write(cache, k, v, off, ln, pages)
    got = fp4.kv_cache_read(cache, off, ln, pages, 300, out_dtype=torch.float32)
    for which, x, amax in ((0, case.k[0], case.k_amax), (1, case.v[0], case.v_amax)):
        codes, scales = case.quantize(x, amax)
        want = case.values(codes.reshape(300 * H, -1), scales.reshape(300 * H, -1), which, f32=True).reshape(300, H, D)
        assert np.array_equal(got[which].cpu().numpy(), np.asarray(want, np.float32))
    # attention over them is that over a small cache of the same bytes
    small = gpu_cache(case, case.full_store())
    for n in (1, 40, 300):
        q = torch.randn(n, 2 * H, D, device=DEV).to(torch.bfloat16)
        o = i32([0, n])
        assert torch.equal(fp4.kv_cache_attention(cache, q, o, ln, pages), fp4.kv_cache_attention(small, q, o, *tables(case)[1:]))


@pytest.mark.parametrize("rows", [1, 12, 70])
def test_a_million_positions(rows):
    announce(f"kv attention over a million positions, {rows} rows")
    case = ref.Case(ref.MX, 1, 32, 256, [(1000003, 0), (5, 0)], seed=2)
    case.rows = [rows, 1]
    case.offsets = np.array([0, rows, rows + 1], np.int32)
    case.T = rows + 1
    bs = ref.block(case.fmt)
    # bytes drawn on the spot: quantizing a million rows on the host is slow
    rng = np.random.default_rng(3)
    store = case.empty_store(0)
    for at in (0, 2):
        store[at][:] = rng.integers(0, 256, store[at].shape, dtype=np.uint8)
        store[at + 1][:] = rng.integers(124, 128, store[at + 1].shape, dtype=np.uint8)
    cache = gpu_cache(case, store)
    q, q64 = queries(case, 2, torch.bfloat16, std=0.5)
    got, lse = fp4.kv_cache_attention(cache, q, *tables(case), return_lse=True)
    p = case.pages[0, np.arange(1000003) // 256]
    s = np.arange(1000003) % 256
    k, v = (case.values(store[2 * w][p, 0, s], store[2 * w + 1][p, 0, s], w) for w in (0, 1))
    for r in {0, rows // 2, rows - 1}:
        n = 1000003 - rows + 1 + r
        for h in range(2):
            x = 32 ** -0.5 * (k[:n] @ q64[r, h])
            A = 32 ** -0.5 * float((np.abs(k[:n]) @ np.abs(q64[r, h])).max())
            e = np.exp(x - x.max())
            want = e @ v[:n] / e.sum()
            # as kv_reference.attention; the sums are joined in parts of at most 2^16 positions and 2^10 parts
            rel = (4 * 48 + 4) * 2.0 ** -24 * A + 2.0 ** -20 + 2 * (2 ** 16 + 2 ** 10) * 2.0 ** -24 + 2.0 ** -11
            tol = rel * (e @ np.abs(v[:n]) / e.sum()) + n * 2.0 ** -36 * np.abs(v).max() * np.exp(0.0)
            assert (np.abs(got[r, h].double().cpu().numpy() - want) <= tol + 2.0 ** -8 * np.abs(want)).all()
            wl = x.max() + np.log(e.sum())
            assert abs(float(lse[r, h]) - wl) <= 96 * 2.0 ** -24 * A + 2.0 ** -20 + 2 * 2 ** 16 * 2.0 ** -24 + 2.0 ** -22 * abs(wl)


def test_query_rows_past_32_bit_offsets():
    """140000 rows of 64 heads x 256 channels (2.3e9 elements), a window of 16: single rows against a call of
    their own, with the positions that they see."""
    announce("kv attention of 140000 x 64 x 256 queries")
    T, H, G, D, page = 140000, 8, 8, 256, 64
    wide = -(-T // page)
    cache = fp4.KVCache.empty(fp4.FP4_NVFP4, wide, H, page, D, 4.0, 4.0, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(4)
    for t in (cache.k_codes, cache.v_codes):
        t.random_(0, 256, generator=g)
    for t in (cache.k_scales, cache.v_scales):
        t.random_(0, 0x60, generator=g)
    pages = torch.randperm(wide, generator=g, device=DEV).reshape(1, wide).to(torch.int32)
    q = torch.randn(T, H * G, D, generator=g, device=DEV, dtype=torch.bfloat16)
    out = fp4.kv_cache_attention(cache, q, i32([0, T]), i32([T]), pages, window=16)
    for r in (0, 15, 70001, 131072, T - 1):
        one = fp4.kv_cache_attention(cache, q[r:r + 1], i32([0, 1]), i32([r + 1]), pages, window=16)
        # another kernel: 2^-11 of sum p |v| for the weights of each, 2^-8 of the value for each rounding; |v| <= 4.1
        assert (out[r].double() - one[0].double()).abs().max() <= 2 * (2.0 ** -11 * 4.1 + 2.0 ** -8 * float(one.abs().max()))
        assert float(one.abs().max()) > 0
