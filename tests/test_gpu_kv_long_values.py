"""GPU: the outputs of attention over a million positions and of calls past 2^31 query elements, with bounds well
below the outputs, and with planted mistakes that the bounds have to show."""
import numpy as np
import pytest
import torch

import kv_reference as ref
import micro_scaled_fp4_amd as fp4
from gpu_util import DEV, announce
from test_gpu_kv_cache import gpu_cache, i32, tables

pytestmark = pytest.mark.gpu

L, PAGE, D = 1000003, 256, 32
LOUD = (1000, 500000, 999000)                   # positions with some 5% of the weight each


def weights_and_mean(k, v, q, seen):
    x = D ** -0.5 * (k[:seen] @ q)
    e = np.exp(x - x.max())
    return x, e / e.sum(), x.max() + np.log(e.sum())


@pytest.mark.parametrize("fmt", [ref.NV, ref.MX])
@pytest.mark.parametrize("rows", [1, 12, 70])
def test_a_million_positions_with_a_signal(fmt, rows):
    """Values of one sign that grow 2^8-fold along the sequence, and three loud positions with values of their own.

    Tolerance as in kv_reference.attention, but for the sums: 512 parts and more fill the card, for two tiles at
    most, so a part has fewer than 2^12 positions, whose terms (all of one sign here) are added one after
    another at most, and fewer than 2^11 parts and waves follow: 2 (2^12 + 2^11) 2^-24 for sum and weights."""
    announce(f"kv attention over a million positions with a signal, fmt {fmt}, {rows} rows")
    case = ref.Case(fmt, 1, D, PAGE, [(L, 0), (5, 0)], seed=12)
    case.rows, case.offsets, case.T = [rows, 1], np.array([0, rows, rows + 1], np.int32), rows + 1
    case.k_amax = case.v_amax = np.float32(2688.0)      # NVFP4: tensor scales of 1
    rng = np.random.default_rng(13)
    t = np.arange(L)
    page, slot = case.pages[0, t // PAGE], t % PAGE
    store = case.empty_store(0)
    sign = rng.integers(0, 2, D)
    # NVFP4: E4M3 bytes of powers of two, 0x38 = 1; MXFP4: 0x7f = 1
    power = (lambda e: (0x38 + 8 * e).astype(np.uint8)) if fmt == ref.NV else (lambda e: (127 + e).astype(np.uint8))
    blocks = D // ref.block(fmt)
    def put(at, codes, exponents):
        store[at][page, 0, slot] = codes[:, 0::2] | codes[:, 1::2] << 4
        store[at + 1][page, 0, slot] = power(exponents)[:, None].repeat(blocks, 1)
    codes = rng.integers(0, 16, (L, D)).astype(np.uint8)
    exponents = rng.integers(-3, 1, L)
    codes[list(LOUD)], exponents[list(LOUD)] = 6 | sign.astype(np.uint8) << 3, 0     # 4 with q's signs
    put(0, codes, exponents)
    codes = rng.integers(1, 8, (L, D)).astype(np.uint8)
    exponents = -5 + 8 * t // L
    exponents[list(LOUD)] = 4
    put(2, codes, exponents)
    k, v = (case.values(store[2 * w][page, 0, slot], store[2 * w + 1][page, 0, slot], w) for w in (0, 1))
    cache = gpu_cache(case, store)
    q = torch.from_numpy((np.where(sign, -0.5, 0.5) + 0.05 * rng.standard_normal((case.T, 2, D))).astype(np.float32)).to(torch.bfloat16)
    q64 = q.double().numpy()
    for dtype in (torch.bfloat16, torch.float32):
        got, lse = fp4.kv_cache_attention(cache, q.to(dtype).to(DEV), *tables(case), return_lse=True)
        for r in sorted({0, rows // 2, rows - 1}):
            seen = L - rows + 1 + r
            for h in range(2):
                x, w, wl = weights_and_mean(k, v, q64[r, h], seen)
                want = w @ v[:seen]
                A = D ** -0.5 * float((np.abs(k[:seen]) @ np.abs(q64[r, h])).max())
                sums = 2 * (2 ** 12 + 2 ** 11) * 2.0 ** -24
                rel = (4 * (D + 16) + 4) * 2.0 ** -24 * A + 2.0 ** -20 + sums
                rel += 2.0 ** -11 + 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -21 + 4 * 2.0 ** -22 * A + 2.0 ** -24
                tol = rel * want + seen * 2.0 ** -36 * v.max()       # (want = sum p |v|)
                off = np.abs(got[r, h].double().cpu().numpy() - want)
                assert (off <= tol).all(), float((off / tol).max())
                assert abs(float(lse[r, h]) - wl) <= (2 * (D + 16) * 2.0 ** -24 + 2.0 ** -22) * A + 2.0 ** -20 + sums + 2.0 ** -22 * abs(wl)
                # mistakes that have to show: nothing, half of the positions, in float32 a part's less, the
                # loud positions' values from a neighbour page or with a neighbour block scale
                half = w[:seen // 2]
                wrong = [np.zeros(D), half @ v[:seen // 2] / half.sum()]
                if dtype == torch.float32:
                    part = slice(seen // 2 + 1, seen // 2 + 4097)
                    wrong.append((want - w[part] @ v[part]) / (1 - w[part].sum()))
                wrong += [want + w[at] * (value - v[at]) for at in LOUD for value in (v[at + PAGE], v[at] / 2)]
                assert all((np.abs(p - want) > 2 * tol).any() for p in wrong), [float((np.abs(p - want) / tol).max()) for p in wrong]


def test_query_rows_past_32_bit_offsets_against_64_bits():
    """140000 rows of 64 heads x 256 channels, a window of 16: rows against 64 bits on the 16 positions that they see
    (tolerance as in kv_reference.attention)."""
    announce("kv attention of 140000 x 64 x 256 queries against 64 bits")
    T, H, G, C, page = 140000, 8, 8, 256, 64
    wide = -(-T // page)
    cache = fp4.KVCache.empty(fp4.FP4_NVFP4, wide, H, page, C, 4.0, 4.0, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(14)
    for t in (cache.k_codes, cache.v_codes):
        t.random_(0, 256, generator=g)
    for t in (cache.k_scales, cache.v_scales):
        t.random_(0x48, 0x60, generator=g)
    pages = torch.randperm(wide, generator=g, device=DEV).reshape(1, wide).to(torch.int32)
    q = torch.randn(T, H * G, C, generator=g, device=DEV, dtype=torch.bfloat16)
    out = fp4.kv_cache_attention(cache, q, i32([0, T]), i32([T]), pages, window=16)
    for r in (0, 15, 70001, 131072, T - 1):
        lo = max(0, r - 15)
        n = r + 1 - lo
        k, v = (x.double().cpu().numpy() for x in fp4.kv_cache_read(cache, i32([0, n]), i32([T]), pages, n, starts=i32([lo]),
                                                                    out_dtype=torch.float32))
        # (read back in float32: each value within 2^-24 of scale x code, in the tolerance's 2^-20)
        wrong = out[(r + 77777) % T].double().cpu().numpy()
        for h in range(0, H * G, 5):
            kh, vh, x = k[:, h // G], v[:, h // G], q[r, h].double().cpu().numpy()
            s = C ** -0.5 * (kh @ x)
            A = C ** -0.5 * float((np.abs(kh) @ np.abs(x)).max())
            w = np.exp(s - s.max())
            w /= w.sum()
            rel = (4 * (C + 16) + 4) * 2.0 ** -24 * A + 2.0 ** -20 + 2 * (n + 64) * 2.0 ** -24 + 2.0 ** -11
            tol = rel * (w @ np.abs(vh)) + n * 2.0 ** -36 * np.abs(vh).max() + 2.0 ** -8 * np.abs(w @ vh)
            assert (np.abs(out[r, h].double().cpu().numpy() - w @ vh) <= tol).all()
            # another row's outputs, and zeros, show in most channels (row 0's: an eighth of the codes is +-0)
            for planted in (wrong[h], 0.0):
                shown = float((np.abs(planted - w @ vh) > 4 * tol).mean())
                assert shown > 0.75
