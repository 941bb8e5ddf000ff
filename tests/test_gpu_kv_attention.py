"""GPU: attention over a paged FP4 cache against the definition in 64 bits, on the cache's own
dequantized values; tolerances are derived in kv_reference.attention."""
import numpy as np
import pytest
import torch

import kv_reference as ref
import micro_scaled_fp4_amd as fp4
from gpu_util import DEV, announce
from test_gpu_kv_cache import gpu_cache, i32, tables

pytestmark = pytest.mark.gpu


def queries(case, Hq, dtype, std=1.5):
    x = torch.from_numpy((case.rng.standard_normal((case.T, Hq, case.D)) * std).astype(np.float32)).to(dtype)
    return x.to(DEV), x.double().numpy()


def check(case, store, q, q64, out_dtype=None, causal=True, window=0, scale=None, cache=None):
    s = case.D ** -0.5 if scale is None else scale
    out_dtype = out_dtype or q.dtype
    T, Hq, D = q.shape
    cache = cache or gpu_cache(case, store)
    out = torch.full((T, Hq, D), 55.0, dtype=out_dtype, device=DEV)
    got, lse = fp4.kv_cache_attention(cache, q, *tables(case), scale=s, causal=causal, window=window, out=out,
                                      return_lse=True)
    assert got is out
    f32 = q.dtype == torch.float32 or out_dtype == torch.float32
    want, wlse, tol, ltol = ref.attention(case, store, q64, s, causal, window, f32)
    inside = np.arange(T) < case.offsets[-1]
    g, gl = got.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (g[~inside] == 55.0).all()
    g, gl, want, wlse, tol, ltol = (a[inside] for a in (g, gl, want, wlse, tol, ltol))
    half_step = 2.0 ** (-8 if out_dtype == torch.bfloat16 else -24)
    off = np.abs(g - want) - (tol * (1 + half_step) + half_step * np.abs(want) + 1e-38)
    assert np.isfinite(g).all() and off.max(initial=-1) <= 0, float(off.max())
    empty = np.isneginf(wlse)
    assert np.isneginf(gl[empty]).all() and (g[empty] == 0).all()
    assert (np.abs(gl[~empty] - wlse[~empty]) <= ltol[~empty]).all()
    return got, lse


DECODE = [(1, 1), (64, 1), (65, 1), (300, 1), (0, 1), (17, 0), (129, 1)]
DRAFTS = [(5, 5), (70, 4), (200, 7), (3, 6), (0, 2), (128, 8)]
PROMPTS = [(150, 150), (1, 1), (200, 33), (64, 64), (90, 0), (20, 25)]


@pytest.mark.parametrize("seqs", [DECODE, DRAFTS, PROMPTS], ids=["decode", "drafts", "prompts"])
@pytest.mark.parametrize("fmt", [ref.NV, ref.MX])
@pytest.mark.parametrize("H,G,D,page", [(1, 1, 32, 16), (2, 4, 128, 16), (1, 3, 96, 32), (2, 1, 64, 64), (1, 16, 128, 128),
                                        (1, 2, 256, 16), (1, 5, 192, 64), (1, 20, 160, 16), (3, 2, 224, 16)])
def test_against_64_bits(seqs, fmt, H, G, D, page):
    announce(f"kv attention fmt {fmt} H {H} G {G} D {D} page {page} seqs {seqs}")
    case = ref.Case(fmt, H, D, page, seqs, seed=G * D + page + len(seqs), spare_rows=1)
    store = case.full_store()
    for dtype in (torch.bfloat16, torch.float32):
        q, q64 = queries(case, H * G, dtype)
        check(case, store, q, q64)


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 7), (True, 64), (True, 100), (True, 1 << 40)])
@pytest.mark.parametrize("seqs", [DECODE, PROMPTS], ids=["decode", "prompts"])
def test_masks(seqs, causal, window):
    announce(f"kv attention mask causal {causal} window {window} seqs {seqs}")
    for fmt, D, G in ((ref.NV, 128, 4), (ref.MX, 64, 2)):
        case = ref.Case(fmt, 1, D, 16, seqs, seed=window % 1000 + D)
        store = case.full_store()
        q, q64 = queries(case, G, torch.bfloat16)
        check(case, store, q, q64, causal=causal, window=window)


@pytest.mark.parametrize("fmt", [ref.NV, ref.MX])
def test_holes_and_rows_that_see_nothing(fmt):
    announce(f"kv attention holes fmt {fmt}")
    case = ref.Case(fmt, 2, 128, 16, [(100, 100), (48, 1), (80, 9), (33, 1)], seed=21)
    case.pages[0, 0] = -1                       # the first 16 rows see only a hole
    case.pages[0, 3] = case.num_pages
    case.pages[1, :3] = -5                      # a sequence of holes
    case.pages[2, 2] = -1
    case.pages[3, 2] = -1                       # the last position, its own
    store = case.full_store()
    for dtype in (torch.bfloat16, torch.float32):
        q, q64 = queries(case, 6, dtype)
        check(case, store, q, q64)
        check(case, store, q, q64, causal=False)
        check(case, store, q, q64, window=16)


@pytest.mark.parametrize("q_dtype,out_dtype", [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
def test_types_of_queries_and_outputs(q_dtype, out_dtype):
    announce(f"kv attention {q_dtype} -> {out_dtype}")
    for seqs in (DECODE, PROMPTS):
        case = ref.Case(ref.NV, 2, 128, 32, seqs, seed=31)
        q, q64 = queries(case, 8, q_dtype)
        check(case, case.full_store(), q, q64, out_dtype=out_dtype)


@pytest.mark.parametrize("fmt", [ref.NV, ref.MX])
def test_ranges_of_queries_keys_and_values(fmt):
    """Large and small magnitudes, sharp and flat softmaxes, negative and zero scales."""
    for q_std, k_std, v_std, scale in ((1e-20, 1.0, 1.0, 1.0), (300.0, 1.0, 1e-6, 0.01), (1e6, 1e-7, 1e5, 0.5), (1.0, 3e4, 2.0, 1e-5),
                                       (2.0, 1.0, 1.0, -0.2), (3.0, 2.0, 1.0, 0.0), (6.0, 5.0, 1.0, 1.0), (1e-30, 1e-3, 1.0, 1e30)):
        announce(f"kv attention ranges fmt {fmt} q {q_std} k {k_std} v {v_std} scale {scale}")
        for seqs in ([(200, 1), (77, 1)], [(90, 90), (130, 20)]):
            case = ref.Case(fmt, 1, 64, 16, seqs, seed=41, k_std=k_std, v_std=v_std)
            store = case.full_store()
            for dtype in (torch.bfloat16, torch.float32):
                q, q64 = queries(case, 2, dtype, std=q_std)
                check(case, store, q, q64, scale=scale)


@pytest.mark.parametrize("fmt", [ref.NV, ref.MX])
def test_a_loud_key_with_a_quiet_value(fmt):
    """Most of the weight on a position whose value is small, as first tokens have it: the others' small
    weights decide the output.  And magnitudes that change by 2^24 along the sequence."""
    announce(f"kv attention sink fmt {fmt}")
    for seqs in ([(700, 1), (333, 1)], [(400, 60)]):
        for order in (1, -1):
            case = ref.Case(fmt, 1, 128, 32, seqs, seed=51)
            for b in range(case.B):
                case.k[b][0] = 3.0
                case.v[b][0] *= np.float32(2.0 ** -8)
                if fmt == ref.MX:
                    n = len(case.v[b])
                    step = np.exp2(np.round(np.linspace(-12, 12, n)[::order])).astype(np.float32)[:, None, None]
                    case.v[b] *= step
            store = case.full_store()
            for dtype in (torch.bfloat16, torch.float32):
                q, q64 = queries(case, 2, dtype, std=0.3)
                q = (q.float() + 0.25).to(dtype)
                check(case, store, q, q.double().cpu().numpy())


def test_views_and_odd_places():
    """q out of a joint projection, with heads apart, at addresses that are not 16-byte aligned."""
    announce("kv attention q views")
    for seqs in (DECODE, PROMPTS):
        for dtype in (torch.bfloat16, torch.float32):
            case = ref.Case(ref.NV, 2, 64, 16, seqs, seed=61)
            store = case.full_store()
            cache = gpu_cache(case, store)
            q, q64 = queries(case, 4, dtype)
            want, wlse = check(case, store, q, q64, cache=cache)
            joint = torch.zeros(case.T, 9, 64, dtype=dtype, device=DEV)
            joint[:, 3:7] = q
            flat = torch.zeros(q.numel() + 1, dtype=dtype, device=DEV)
            flat[1:] = q.flatten()
            for view in (joint[:, 3:7], flat[1:].view(q.shape), q.transpose(0, 1).contiguous().transpose(0, 1)):
                got, lse = fp4.kv_cache_attention(cache, view, *tables(case), return_lse=True)
                assert torch.equal(got, want) and torch.equal(lse, wlse)
            # an output that starts at an odd place
            room = torch.zeros(q.numel() + 1, dtype=dtype, device=DEV)
            got = fp4.kv_cache_attention(cache, q, *tables(case), out=room[1:].view(q.shape))
            assert torch.equal(got, want)


def test_a_long_context_in_parts():
    """Contexts long enough to be split, next to short and empty ones; positions' order does not matter to a
    query that sees all of them."""
    announce("kv attention long")
    for fmt, G, rows in ((ref.NV, 4, 1), (ref.MX, 8, 1), (ref.MX, 2, 40), (ref.NV, 8, 130)):
        case = ref.Case(fmt, 1, 128, 64, [(6000, rows), (10, min(rows, 10)), (0, 1), (2500, 1)], seed=71)
        store = case.full_store()
        for dtype in (torch.bfloat16, torch.float32):
            q, q64 = queries(case, G, dtype)
            check(case, store, q, q64)
            check(case, store, q, q64, window=3000)


def test_many_sequences():
    """More sequences than a round of the search takes, most without rows."""
    announce("kv attention many sequences")
    rng = np.random.default_rng(81)
    seqs = [(int(rng.integers(0, 40)), int(rng.integers(0, 3)) if rng.random() < 0.3 else 0) for _ in range(200)]
    case = ref.Case(ref.MX, 1, 32, 16, seqs, seed=82, spare_rows=5)
    q, q64 = queries(case, 2, torch.bfloat16)
    check(case, case.full_store(), q, q64)


@pytest.mark.parametrize("fmt", [ref.NV, ref.MX])
@pytest.mark.parametrize("seqs", [[(400, 1), (170, 1)], [(300, 4), (65, 3)], [(500, 130), (90, 90)]], ids=["decode", "drafts", "prompts"])
def test_positions_before_every_window_may_hold_anything(fmt, seqs):
    """A window has left pages behind whose table entries still stand: their bytes are NaN and the largest scales."""
    announce(f"kv attention garbage before the window fmt {fmt} {seqs}")
    for D, page, window in ((128, 16, 20), (64, 64, 33), (256, 16, 64)):
        case = ref.Case(fmt, 2, D, page, seqs, seed=window)
        store = case.full_store()
        for junk in (0xff, 0x7f, 0xfe):
            mine = [t.copy() for t in store]
            for b, (length, n) in enumerate(seqs):
                for t in range(max(0, length - n - window + 1)):
                    for a in mine:
                        a[case.pages[b, t // page], :, t % page] = junk
            for dtype in (torch.bfloat16, torch.float32):
                q, q64 = queries(case, 4, dtype)
                got = fp4.kv_cache_attention(gpu_cache(case, mine), q, *tables(case), window=window)
                want = fp4.kv_cache_attention(gpu_cache(case, store), q, *tables(case), window=window)
                assert torch.equal(got, want)
        check(case, store, q, q64, window=window)


@pytest.mark.parametrize("fmt", [ref.NV, ref.MX])
def test_far_more_rows_than_positions(fmt):
    """Whole row tiles before position 0, in the first sequence and a later one."""
    announce(f"kv attention rows before position 0 fmt {fmt}")
    case = ref.Case(fmt, 1, 64, 16, [(20, 300), (0, 200), (33, 1), (5, 140)], seed=9)
    store = case.full_store()
    for dtype in (torch.bfloat16, torch.float32):
        q, q64 = queries(case, 2, dtype)
        check(case, store, q, q64)
        check(case, store, q, q64, window=4)
    # and on the kernels for few rows
    case = ref.Case(fmt, 1, 64, 16, [(2, 30)] + [(40, 1)] * 9, seed=10)
    q, q64 = queries(case, 4, torch.bfloat16)
    check(case, case.full_store(), q, q64)


@pytest.mark.parametrize("fmt", [ref.NV, ref.MX])
@pytest.mark.parametrize("B,most_rows,long", [(64, 1, 5000), (65, 1, 5000), (65, 80, 700), (130, 3, 2100), (1030, 1, 3000),
                                             (2500, 2, 400)])
def test_more_sequences_than_lanes(fmt, B, most_rows, long):
    """Around and past the sequences that a wave lays out by itself: short ones, empty ones, one long one that is cut."""
    announce(f"kv attention of {B} sequences, up to {most_rows} rows, one of {long}, fmt {fmt}")
    rng = np.random.default_rng(B + most_rows)
    seqs = [(int(rng.integers(0, 30)), int(rng.integers(most_rows // 3, most_rows + 1))) for _ in range(B)]
    seqs[B // 2] = (long, most_rows)
    seqs[0], seqs[B - 1] = (0, 1), (9, 0)
    case = ref.Case(fmt, 1, 32, 16, seqs, seed=B, spare_rows=3)
    store = case.full_store()
    q, q64 = queries(case, 2, torch.bfloat16)
    check(case, store, q, q64)
    if B == 130:
        check(case, store, q, q64, window=50)
        check(case, store, q, q64, causal=False)


def test_layout_of_many_sequences_in_a_graph():
    announce("kv attention of 300 sequences, captured, replayed with other lengths")
    case = ref.Case(ref.NV, 2, 64, 16, [(90, 1)] * 300, seed=5)
    cache = gpu_cache(case, case.full_store())
    q, _ = queries(case, 8, torch.bfloat16)
    offsets, lengths, pages = tables(case)
    fp4.kv_cache_attention(cache, q, offsets, lengths, pages)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = fp4.kv_cache_attention(cache, q, offsets, lengths, pages, return_lse=True)
    rng = np.random.default_rng(6)
    for _ in range(4):
        lengths.copy_(i32(rng.integers(0, 91, 300)))
        graph.replay()
        want, wlse = fp4.kv_cache_attention(cache, q, offsets, lengths, pages, return_lse=True)
        assert torch.equal(out, want) and torch.equal(lse, wlse)


@pytest.mark.parametrize("fmt", [ref.NV, ref.MX])
def test_largest_factors_with_scores_of_zero(fmt):
    """|scale| and q so large that their product is past float32, keys of 0: the mean of the values."""
    announce(f"kv attention of scores of zero fmt {fmt}")
    case = ref.Case(fmt, 1, 64, 16, [(70, 1), (100, 40)], seed=3, k_std=0.0)
    store = case.full_store()
    for dtype in (torch.bfloat16, torch.float32):
        for group in (1, 4):
            q = torch.full((case.T, group, 64), 2.0 ** 120, dtype=dtype, device=DEV)
            check(case, store, q, q.double().cpu().numpy(), scale=2.0 ** 120)
