"""GPU: the cache calls' execution model: graphs, streams, repeated calls, a whole conversation, and many random
batches against 64 bits."""
import threading

import numpy as np
import pytest
import torch

import kv_reference as ref
import micro_scaled_fp4_amd as fp4
from gpu_util import DEV, announce
from test_gpu_kv_attention import check, queries
from test_gpu_kv_cache import gpu_cache, i32, store_of, tables

pytestmark = pytest.mark.gpu


def same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


def step(cache, qkv, offsets, lengths, pages, workspace=None):
    """One pass: write, attend, read back."""
    H = cache.num_heads
    fp4.kv_cache_write(cache, qkv[:, -2 * H:-H], qkv[:, -H:], offsets, lengths, pages)
    out, lse = fp4.kv_cache_attention(cache, qkv[:, :-2 * H], offsets, lengths, pages, return_lse=True, workspace=workspace)
    return [out, lse, *fp4.kv_cache_read(cache, offsets, lengths, pages, qkv.shape[0])]


@pytest.mark.parametrize("fmt", [ref.NV, ref.MX])
@pytest.mark.parametrize("rows", [1, 3, 40])
def test_replays_with_other_contents(fmt, rows):
    """Captured once; replayed with other tokens, lengths, offsets and pages, eager work in between."""
    announce(f"kv graph fmt {fmt} rows {rows}")
    B, H, G, D, page, wide = 5, 2, 4, 128, 16, 200
    g = torch.Generator(device=DEV).manual_seed(rows)
    def cache():
        c = fp4.KVCache.empty(fmt, B * wide, H, page, D, *((5.0, 5.0) if fmt == ref.NV else ()), device=DEV)
        for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales):
            t.fill_(0x37)
        return c
    a, b = cache(), cache()
    inputs = []
    for k in range(4):
        pages = torch.randperm(B * wide, generator=g, device=DEV).reshape(B, wide).to(torch.int32)
        lens = torch.randint(rows, wide * page + 1, (B,), generator=g, device=DEV).to(torch.int32)
        if k == 2:
            lens[1:] = rows                     # one long sequence
        off = torch.arange(B + 1, device=DEV).to(torch.int32) * rows
        if k == 3:
            off[-1] = off[-2]                   # a sequence without rows: rows behind the last one
        inputs.append((torch.randn(B * rows, H * G + 2 * H, D, generator=g, device=DEV).to(torch.bfloat16), off, lens, pages))
    static = [t.clone() for t in inputs[0]]
    step(a, *static)                            # first calls outside the capture
    step(b, *inputs[0])                         # (both caches see the same calls)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(a, *static)
    for k in (1, 2, 0, 3, 1):
        for t, new in zip(static, inputs[k]):
            t.copy_(new)
        n = int(inputs[k][1][-1])
        junk = torch.randn(1 << 20, device=DEV).sum()
        graph.replay()
        torch.cuda.synchronize()
        eager = step(b, *inputs[k])
        torch.cuda.synchronize()
        assert same([t[:n] for t in out], [t[:n] for t in eager]), f"replay {k}"
        assert same(*([getattr(c, name) for name in ("k_codes", "k_scales", "v_codes", "v_scales")] for c in (a, b)))
        del junk


def test_two_graphs_share_a_workspace():
    """The workspace's contents matter only within a call."""
    announce("kv graphs with one workspace")
    cases = [ref.Case(ref.NV, 2, 128, 64, [(5000, 1), (70, 1)], seed=1), ref.Case(ref.NV, 2, 128, 64, [(3000, 40), (900, 40)], seed=2)]
    caches = [gpu_cache(c, c.full_store()) for c in cases]
    qs = [queries(c, 8, torch.bfloat16)[0] for c in cases]
    wheres = [tables(c) for c in cases]
    lib = fp4.load_library()
    need = max(lib.kv_cache_attention_workspace_bytes(c._address, q.shape[0], 2, 8) for c, q in zip(caches, qs))
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    want = [fp4.kv_cache_attention(c, q, *w) for c, q, w in zip(caches, qs, wheres)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c, q, w in zip(caches, qs, wheres):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(fp4.kv_cache_attention(c, q, *w, workspace=ws))
        graphs.append(graph)
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for t in outs:
            t.zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in set(order):
            assert torch.equal(outs[i], want[i])
    with pytest.raises(fp4.FP4Error):
        fp4.kv_cache_attention(caches[0], qs[0], *wheres[0], workspace=ws[:16])


def test_same_bits_every_time():
    """Sums are taken in a fixed order."""
    announce("kv attention repeated")
    for seqs, G in (([(6000, 1), (100, 1)], 4), ([(4000, 9)], 2), ([(3000, 200), (500, 100)], 2)):
        for fmt in (ref.NV, ref.MX):
            case = ref.Case(fmt, 2, 128, 16, seqs, seed=3)
            cache = gpu_cache(case, case.full_store())
            for dtype in (torch.bfloat16, torch.float32):
                q, _ = queries(case, 2 * G, dtype)
                first = fp4.kv_cache_attention(cache, q, *tables(case), return_lse=True)
                for _ in range(3):
                    assert same(first, fp4.kv_cache_attention(cache, q, *tables(case), return_lse=True))


def test_two_threads_on_two_streams():
    announce("kv two threads, two streams")
    cases = [ref.Case(ref.NV, 2, 64, 16, [(2000, 1), (300, 1)], seed=4), ref.Case(ref.MX, 2, 128, 32, [(900, 100), (40, 1)], seed=5)]
    caches = [gpu_cache(c, c.full_store()) for c in cases]
    g = torch.Generator(device=DEV).manual_seed(1)
    qkvs = [torch.randn(c.T, 12, c.D, generator=g, device=DEV).to(torch.bfloat16) for c in cases]
    wheres = [tables(c) for c in cases]
    serial = [step(c, x, *w) for c, x, w in zip(caches, qkvs, wheres)]
    torch.cuda.synchronize()
    streams, results, errors = [torch.cuda.Stream() for _ in range(2)], [None, None], []
    barrier = threading.Barrier(2, timeout=30)

    def run(i):
        try:
            torch.cuda.set_device(0)
            barrier.wait()
            with torch.cuda.stream(streams[i]):
                for _ in range(8):
                    results[i] = step(caches[i], qkvs[i], *wheres[i])
            streams[i].synchronize()
        except Exception as e:          # reported on the main thread
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,), daemon=True) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=60)
    assert not errors and all(not t.is_alive() for t in threads), errors
    assert all(same(r, s) for r, s in zip(results, serial))


@pytest.mark.parametrize("fmt", [ref.NV, ref.MX])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_conversation(fmt, dtype):
    """Prompts in two chunks, drafts of which some are taken back and written again, single tokens: after each
    call the cache holds the oracle's bytes and attention is that of 64 bits on them."""
    announce(f"kv conversation fmt {fmt} {dtype}")
    H, G, D, page, B = 2, 3, 64, 16, 3
    full = ref.Case(fmt, H, D, page, [(170, 0), (90, 0), (33, 0)], seed=6)
    store = full.empty_store()
    cache = gpu_cache(full, store)
    lens = [0] * B
    # rows of each sequence, and how many positions are taken back before them
    for rows, back in (([100, 64, 0], 0), ([60, 1, 31], 0), ([4, 4, 1], 0), ([3, 4, 1], 2), ([1, 1, 1], 1), ([1, 0, 1], 0)):
        lens = [min(int(full.lengths[b]), max(0, lens[b] - (back if rows[b] else 0)) + rows[b]) for b in range(B)]
        case = ref.Case(fmt, H, D, page, [(n, min(r, n)) for n, r in zip(lens, rows)], seed=7)
        case.pages, case.max_pages, case.num_pages = full.pages, full.max_pages, full.num_pages
        case.k_amax, case.v_amax = full.k_amax, full.v_amax
        k = np.zeros((case.T, H, D), np.float32)
        v = k.copy()
        for b in range(B):
            lo, n = int(case.offsets[b]), case.rows[b]
            k[lo:lo + n], v[lo:lo + n] = full.k[b][lens[b] - n:lens[b]], full.v[b][lens[b] - n:lens[b]]
            case.put(store, b, range(lens[b] - n, lens[b]), k[lo:lo + n], v[lo:lo + n])
        fp4.kv_cache_write(cache, torch.from_numpy(k).to(DEV).to(dtype), torch.from_numpy(v).to(DEV).to(dtype), *tables(case))
        assert all(np.array_equal(g, w) for g, w in zip(store_of(cache), store))
        q, q64 = queries(case, H * G, dtype)
        check(case, store, q, q64, cache=cache)


@pytest.mark.parametrize("seed", range(24))
def test_random_batches(seed):
    """Ragged batches of every kind: rows, lengths, heads, pages, windows, holes, more sequences than lanes."""
    rng = np.random.default_rng(1000 + seed)
    B = int(rng.choice([1, 2, 5, 17, 70, 130]))
    H, G, D = int(rng.choice([1, 2, 3])), int(rng.choice([1, 2, 5, 8])), int(rng.choice([32, 64, 96, 128, 192, 256]))
    page, fmt = int(rng.choice([16, 32, 64, 256])), int(rng.integers(0, 2))
    budget = 500 // (H * G) + 1                  # rows in all, for the reference's sake
    kind = rng.choice(["decode", "drafts", "prompts", "mixed"])
    seqs = []
    for b in range(B):
        length = int(np.exp(rng.uniform(0, np.log(3000 if b < 3 else 200)))) - 1
        most = {"decode": 1, "drafts": 6, "prompts": 300, "mixed": int(rng.choice([1, 4, 150]))}[kind]
        n = int(rng.integers(0, most + 1)) if kind != "decode" else 1
        n = min(n, budget)
        budget -= n
        seqs.append((length, n if rng.random() < 0.1 else min(n, length)))
    announce(f"kv random {seed}: {kind} B {B} H {H} G {G} D {D} page {page} fmt {fmt}")
    case = ref.Case(fmt, H, D, page, seqs, seed=2000 + seed, spare_rows=int(rng.integers(0, 3)), wide=int(rng.integers(0, 300)))
    for b in range(B):
        if rng.random() < 0.15 and seqs[b][0] > 0:
            case.pages[b, rng.integers(0, -(-seqs[b][0] // page))] = -1
    store = case.full_store()
    cache = gpu_cache(case, store)
    causal = bool(rng.random() < 0.8)
    window = int(rng.integers(1, 500)) if causal and rng.random() < 0.4 else 0
    for dtype in (torch.bfloat16, torch.float32):
        q, q64 = queries(case, H * G, dtype)
        check(case, store, q, q64, causal=causal, window=window, cache=cache)
