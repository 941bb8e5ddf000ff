"""GPU: writing and reading a paged FP4 cache against the CPU oracle, bit for bit."""
import numpy as np
import pytest
import torch

import kv_reference as ref
import micro_scaled_fp4_amd as fp4
from gpu_util import DEV, announce
from oracle import fp4_oracle as o

pytestmark = pytest.mark.gpu

SEQS = {
    "single_tokens": [(1, 1), (17, 1), (300, 1), (16, 1), (33, 1)],
    "prompts": [(70, 70), (1, 1), (33, 20), (129, 5)],
    "more_rows_than_positions": [(3, 7), (0, 4), (20, 20)],
    "empty_ones": [(0, 0), (40, 0), (25, 3), (0, 0), (50, 0)],
}


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)


def gpu_cache(case, store):
    return fp4.KVCache(case.fmt, *[torch.from_numpy(t).to(DEV) for t in store], *case.amaxes())


def tables(case):
    return i32(case.offsets), i32(case.lengths), i32(case.pages)


def store_of(cache):
    return [t.cpu().numpy() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]


def rows_of(case, spare=0.0):
    """The k and v rows of the call, [T, H, D] float32 (rows before position 0: drawn)."""
    k = np.full((case.T, case.H, case.D), spare, np.float32)
    v = k.copy()
    for b in range(case.B):
        lo, n, L = int(case.offsets[b]), case.rows[b], int(case.lengths[b])
        for i in range(n):
            t = L - n + i
            k[lo + i], v[lo + i] = (case.k[b][t], case.v[b][t]) if t >= 0 else (7.0, 8.0)
    return k, v


def expected_write(case, store, k, v):
    for b in range(case.B):
        lo, n, L = int(case.offsets[b]), case.rows[b], int(case.lengths[b])
        case.put(store, b, [L - n + i for i in range(n)], k[lo:lo + n], v[lo:lo + n])
    return store


@pytest.mark.parametrize("seqs", list(SEQS))
@pytest.mark.parametrize("fmt", [ref.NV, ref.MX])
@pytest.mark.parametrize("H,D,page", [(1, 32, 16), (8, 128, 16), (3, 96, 64), (5, 256, 32), (2, 160, 128)])
def test_write_and_read_bytes(seqs, fmt, H, D, page):
    announce(f"kv write/read {seqs} fmt {fmt} H {H} D {D} page {page}")
    case = ref.Case(fmt, H, D, page, SEQS[seqs], seed=H * D + page, spare_rows=2)
    k, v = rows_of(case)
    for dtype in (torch.bfloat16, torch.float32):
        cache = gpu_cache(case, case.empty_store(0xa5))
        fp4.kv_cache_write(cache, torch.from_numpy(k).to(DEV).to(dtype), torch.from_numpy(v).to(DEV).to(dtype), *tables(case))
        want = expected_write(case, case.empty_store(0xa5), k, v)
        for got, w, name in zip(store_of(cache), want, ("k codes", "k scales", "v codes", "v scales")):
            assert np.array_equal(got, w), name
    # read back every row (bf16 values of the float32 ones; rows past the last sequence stay)
    for dtype, mark in ((torch.float32, 123.0), (torch.bfloat16, -77.0)):
        out = [torch.full((case.T, H, D), mark, dtype=dtype, device=DEV) for _ in range(2)]
        got = fp4.kv_cache_read(cache, *tables(case), case.T, out=out)
        want = [np.full((case.T, H, D), mark, np.float32) for _ in range(2)]
        for b in range(case.B):
            lo, n, L = int(case.offsets[b]), case.rows[b], int(case.lengths[b])
            for i in range(n):
                t = L - n + i
                for which in (0, 1):
                    want[which][lo + i] = 0
                    if t >= 0:
                        p, s = case.pages[b, t // page], t % page
                        st = store_of(cache)
                        want[which][lo + i] = case.values(st[2 * which][p, :, s], st[2 * which + 1][p, :, s], which, f32=True)
        for which in (0, 1):
            w = torch.from_numpy(want[which]).to(dtype)
            bits = torch.int32 if dtype == torch.float32 else torch.int16
            assert torch.equal(got[which].cpu().view(bits), w.view(bits)), which


def test_write_takes_views_of_a_joint_projection_and_odd_places():
    """Keys and values read in place out of [T, heads, D] rows of a projection; copied where heads are not
    contiguous; at addresses that are not 16-byte aligned; the same bytes each time."""
    announce("kv write of views")
    case = ref.Case(ref.NV, 2, 64, 16, [(40, 40), (21, 5)], seed=5)
    k, v = rows_of(case)
    want = expected_write(case, case.empty_store(), k, v)
    for dtype in (torch.bfloat16, torch.float32):
        joint = torch.zeros(case.T, 9, 64, dtype=dtype, device=DEV)
        joint[:, 4:6], joint[:, 7:9] = torch.from_numpy(k).to(DEV).to(dtype), torch.from_numpy(v).to(DEV).to(dtype)
        flat = torch.zeros(2 * case.T * 128 + 1, dtype=dtype, device=DEV)
        odd = [flat[1:][j * case.T * 128:(j + 1) * case.T * 128].view(case.T, 2, 64) for j in (0, 1)]
        odd[0].copy_(joint[:, 4:6])
        odd[1].copy_(joint[:, 7:9])
        head_major = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (joint[:, 4:6], joint[:, 7:9])]
        for pair in ((joint[:, 4:6], joint[:, 7:9]), odd, head_major):
            cache = gpu_cache(case, case.empty_store())
            fp4.kv_cache_write(cache, *pair, *tables(case))
            assert all(np.array_equal(g, w) for g, w in zip(store_of(cache), want))


def test_holes_are_not_written_and_read_as_zeros():
    announce("kv holes")
    case = ref.Case(ref.MX, 2, 64, 16, [(64, 64), (30, 30)], seed=6)
    case.pages[0, 1], case.pages[0, 3], case.pages[1, 0] = -1, case.num_pages, 2 ** 30
    k, v = rows_of(case)
    cache = gpu_cache(case, case.empty_store())
    fp4.kv_cache_write(cache, torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV), *tables(case))
    want = expected_write(case, case.empty_store(), k, v)
    assert all(np.array_equal(g, w) for g, w in zip(store_of(cache), want))
    got = fp4.kv_cache_read(cache, *tables(case), case.T, out_dtype=torch.float32)
    for b in range(2):
        for which in (0, 1):
            vals, hole = case.held(want, b, which)
            g = got[which][int(case.offsets[b]):int(case.offsets[b + 1])].cpu().numpy()
            assert (g[hole] == 0).all() and np.array_equal(g[~hole], vals[~hole].astype(np.float32))


def test_read_from_given_starts():
    """starts before 0, past the length and inside; a sequence read in part."""
    announce("kv read starts")
    case = ref.Case(ref.NV, 2, 96, 32, [(100, 40), (50, 9), (3, 6), (0, 2)], seed=7)
    store = case.full_store()
    cache = gpu_cache(case, store)
    starts = np.array([17, -4, 1, 0], np.int32)
    got = fp4.kv_cache_read(cache, *tables(case), case.T, starts=i32(starts), out_dtype=torch.float32)
    for b in range(case.B):
        for i in range(case.rows[b]):
            t = int(starts[b]) + i
            for which in (0, 1):
                g = got[which][int(case.offsets[b]) + i].cpu().numpy()
                if not 0 <= t < case.lengths[b]:
                    assert (g == 0).all()
                else:
                    p, s = case.pages[b, t // case.page], t % case.page
                    w = case.values(store[2 * which][p, :, s], store[2 * which + 1][p, :, s], which, f32=True)
                    assert np.array_equal(g.view(np.int32), np.asarray(w, np.float32).view(np.int32))


def test_starts_near_the_ends_of_int32():
    announce("kv read starts at int32's ends")
    case = ref.Case(ref.NV, 1, 32, 16, [(20, 5), (20, 5)], seed=8)
    cache = gpu_cache(case, case.full_store())
    got = fp4.kv_cache_read(cache, *tables(case), case.T, starts=i32([2 ** 31 - 2, -2 ** 31]))
    assert all((g == 0).all() for g in got)


def test_same_bytes_as_the_tensor_quantizers():
    """A prompt's rows hold what nvfp4_quantize / mxfp4_quantize give for them, zeros and subnormals included."""
    announce("kv write against the tensor quantizers")
    T, H, D = 48, 4, 128
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(T, H, D, generator=g, device=DEV)
    x[3] = 0
    x[4, 1, :32] = -0.0
    x[5] *= 1e-6
    x[6] *= 1e4
    pages = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    off, ln = i32([0, T]), i32([T])
    for dtype in (torch.bfloat16, torch.float32):
        y = x.to(dtype)
        for fmt in (fp4.FP4_NVFP4, fp4.FP4_MXFP4):
            nv = fmt == fp4.FP4_NVFP4
            cache = fp4.KVCache.empty(fmt, 3, H, 16, D, 37.0 if nv else None, 37.0 if nv else None, device=DEV)
            fp4.kv_cache_write(cache, y, y, off, ln, pages)
            q, s = (fp4.nvfp4_quantize(y.reshape(T * H, D), amax=37.0) if nv else fp4.mxfp4_quantize(y.reshape(T * H, D)))[:2]
            for t, want in ((cache.k_codes, q), (cache.k_scales, s), (cache.v_codes, q), (cache.v_scales, s)):
                got = t[pages[0].long()].transpose(1, 2).reshape(T * H, -1)
                assert torch.equal(got, want)


def test_offsets_and_lengths_outside_their_range_touch_nothing_else():
    """Clamped: the call stays inside its tensors (here: guard bytes around the cache hold)."""
    announce("kv clamps")
    H, D, page, T = 2, 64, 16, 12
    for fmt in (ref.NV, ref.MX):
        case = ref.Case(fmt, H, D, page, [(20, 6), (30, 6)], seed=9)
        big = [torch.full((t.size + 8192,), 0x5a, dtype=torch.uint8, device=DEV) for t in case.empty_store()]
        inner = [b[4096:4096 + t.size].view(t.shape) for b, t in zip(big, case.empty_store())]
        cache = fp4.KVCache(fmt, *inner, *case.amaxes())
        x = torch.randn(T, H, D, device=DEV)
        for off, ln in (([-5, 6, 2 ** 31 - 1], [20, 2 ** 31 - 1]), ([0, 2 ** 30, 12], [-7, 1000]), ([3, 1, 9], [5, 6])):
            pg = i32(case.pages)
            fp4.kv_cache_write(cache, x, x, i32(off), i32(ln), pg)
            fp4.kv_cache_read(cache, i32(off), i32(ln), pg, T)
            fp4.kv_cache_attention(cache, x, i32(off), i32(ln), pg)
        for b, t in zip(big, case.empty_store()):
            assert (b[:4096] == 0x5a).all() and (b[4096 + t.size:] == 0x5a).all()


def test_nothing_to_do():
    announce("kv no rows, no sequences, no pages")
    cache = fp4.KVCache.empty(fp4.FP4_MXFP4, 0, 2, 16, 64, device=DEV)
    none = torch.empty(0, 2, 64, device=DEV)
    fp4.kv_cache_write(cache, none, none, i32([0]), i32([]), torch.empty(0, 0, dtype=torch.int32, device=DEV))
    assert fp4.kv_cache_read(cache, i32([0, 0]), i32([0]), i32([[0]]), 0)[0].shape == (0, 2, 64)
    assert fp4.kv_cache_attention(cache, none, i32([0, 0]), i32([0]), i32([[0]])).shape == (0, 2, 64)
    # rows of a sequence without any page: nothing to see
    x = torch.randn(3, 2, 64, device=DEV)
    table = torch.empty(1, 0, dtype=torch.int32, device=DEV)
    out, lse = fp4.kv_cache_attention(cache, x, i32([0, 3]), i32([0]), table, return_lse=True)
    assert (out == 0).all() and (lse == -float("inf")).all()
    k, v = fp4.kv_cache_read(cache, i32([0, 3]), i32([3]), table, 3)
    assert (k == 0).all() and (v == 0).all()
    fp4.kv_cache_write(cache, x, x, i32([0, 3]), i32([3]), table)
