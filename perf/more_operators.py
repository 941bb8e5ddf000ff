"""A paged key/value cache held in FP4 as measured cases: tokens quantized as they
are written into their pages, positions read back, and attention over the cache
for prompts, prompt chunks, drafted tokens and single tokens.

`run` computes a case either in plain torch operations in 32 bits (own = False)
or through micro_scaled_fp4_amd (own = True), on the inputs that `prepare` makes
from a seed.  `exact` computes the same outputs from the definitions in 64 bits.

Definitions
-----------
Cache.  Keys and values of H heads of D channels.  Position t of sequence b sits
  in page pages[b][t // page_size] at slot t % page_size; a page holds
  [H, page_size, D / 2] packed E2M1 codes and [H, page_size, D / bs] scale bytes for
  keys and as much for values (bs = 16 E4M3 bytes under one given tensor amax, or
  32 E8M0 bytes).  Rows offsets[b] .. offsets[b + 1] of the [T, heads, D] operands
  belong to sequence b.
Write.  The n rows of sequence b are its last n positions before lengths[b].
Read.  Row r holds position starts[b] + r - offsets[b].
Attention.  Query row i of n sits at position p = lengths[b] - n + i and sees the
  positions t < lengths[b], t <= p where causal, t > p - window where a window is
  given.  Query head h reads key/value head h // group.
  out = sum_t softmax_t(scale * <q, k_t>) v_t;  lse = log(sum_t exp(scale * <q, k_t>));
  0 and -inf where nothing is seen.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases ----
def _case(name, op, fmt, H, D, page, dtype, seqs, lengths, rows=(1, 1), group=1, causal=True,
          window=0, lse=False, padded=0):
    return {"name": name, "op": op, "fmt": fmt, "H": H, "D": D, "page": page, "dtype": dtype,
            "seqs": seqs, "len_lo": lengths[0], "len_hi": lengths[1], "rows_lo": rows[0],
            "rows_hi": rows[1], "group": group, "causal": causal, "window": window, "lse": lse,
            "padded": padded}


def listed():
    return [
        # one decoding step's token of each of 32 sequences enters the cache
        _case("append_decode", "append", "nv", 8, 128, 16, "bf16", 32, (900, 8000)),
        # four prompts of 16384 tokens in all enter the cache
        _case("append_prompts", "append", "mx", 8, 128, 32, "bf16", 4, (6500, 6500), rows=(1692, 6500)),
        # a cached conversation of 65536 tokens read out, to move it or to compute on it
        _case("read_long", "read", "nv", 8, 128, 64, "bf16", 1, (65536, 65536), rows=(65536, 65536)),
        # the tails of 7 short sequences read out in float32, heads of 96 channels
        _case("read_ragged", "read", "mx", 5, 96, 16, "f32", 7, (301, 2111), rows=(33, 300)),
        # one token of one short conversation: latency only
        _case("decode_one", "attend", "nv", 8, 128, 16, "bf16", 1, (1000, 1000), group=4),
        # a decoding batch of ragged lengths; the last two places of the batch are empty
        _case("decode_batch", "attend", "nv", 8, 128, 64, "bf16", 32, (1000, 16000), group=8, padded=2),
        # one token over a context of 131072
        _case("decode_long", "attend", "mx", 8, 128, 64, "bf16", 1, (131072, 131072), group=4),
        # a small model in float32 with a head of keys per query head and a sliding window
        _case("decode_window", "attend", "mx", 12, 64, 16, "f32", 8, (777, 12345), window=4096, lse=True),
        # five drafted tokens per sequence are checked at once
        _case("verify_drafts", "attend", "nv", 8, 128, 32, "bf16", 16, (2500, 9001), rows=(5, 5), group=5),
        # a whole prompt
        _case("prefill", "attend", "nv", 8, 128, 64, "bf16", 1, (8192, 8192), rows=(8192, 8192), group=4),
        # the next chunk of two long prompts
        _case("prefill_chunk", "attend", "mx", 8, 128, 64, "bf16", 2, (16384, 32768), rows=(512, 512), group=8),
        # short prompts of odd lengths, heads of 256 channels, a sliding window
        _case("prefill_ragged", "attend", "nv", 4, 256, 16, "bf16", 5, (333, 3001), rows=(333, 3001), group=2,
              window=1024, lse=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "attend"])
    fmt, dtype = rng.choice(["nv", "mx"]), rng.choice(["bf16", "bf16", "f32"])
    D = 32 * rng.choice([1, 2, 2, 3, 4, 4, 4, 5, 6, 8])
    H, page = _log_int(rng, 1, 16), 16 << rng.randint(0, 4)
    seqs = _log_int(rng, 1, 64)
    if op != "attend":
        rows = _log_int(rng, 1, max(1, 65536 * 8 * 128 // (seqs * H * D)))
        return _case("", op, fmt, H, D, page, dtype, seqs, (rows, rows + _log_int(rng, 1, 4096)),
                     rows=(max(1, rows // 3), rows))
    group = rng.choice([1, 1, 2, 3, 4, 5, 8, 16])
    lo = _log_int(rng, 1, max(2, min(131072, 131072 * 8 * 128 // (seqs * H * D))))
    hi = min(131072, rng.randint(lo, 4 * lo))
    # a draw's scores stay within a quarter of the largest listed case's
    most = max(1, min(lo, 2 ** 29 // (seqs * H * group * hi)))
    rows = rng.choice([1, 1, min(most, rng.randint(2, 8)), _log_int(rng, 1, most), most])
    causal = rng.random() < 0.8
    return _case("", op, fmt, H, D, page, dtype, seqs, (lo, hi), rows=(max(1, rows // 2), rows), group=group,
                 causal=causal, window=_log_int(rng, 1, 2 * hi) if causal and rng.random() < 0.3 else 0,
                 lse=rng.random() < 0.5, padded=rng.choice([0, 0, min(2, seqs - 1)]))


def _sizes(case):
    """(length, rows) of each sequence, before the seed orders them."""
    n, got = case["seqs"], []
    for b in range(n):
        f = b / max(1, n - 1) if n > 1 else 1.0
        length = int(round(case["len_lo"] * (case["len_hi"] / case["len_lo"]) ** f))
        rows = min(length, int(round(case["rows_lo"] + (case["rows_hi"] - case["rows_lo"]) * f)))
        got.append((0 if b < case["padded"] else length, rows))
    return got


# ----------------------------------------------------------------- formats ----
def _f32(v):
    return torch.full((1,), v, dtype=torch.float32, device=DEV)


def _e2m1_codes(q):
    """Codes of the nearest E2M1 magnitudes (ties to the even code), sign kept."""
    m = q.abs()
    c = (m > 0.25).to(torch.uint8)
    c += m >= 0.75
    c += m > 1.25
    c += m >= 1.75
    c += m > 2.5
    c += m >= 3.5
    c += m > 5.0
    return c | (torch.signbit(q).to(torch.uint8) << 3)


def _tensor_scale(amax):
    return torch.where(amax != 0, amax / _f32(2688.0), _f32(1.0))


def _quantize(x, fmt, amax):
    """x [..., D] -> (packed codes [..., D/2], scale bytes [..., D/bs])."""
    x = x.float()
    if fmt == "nv":
        sg = _tensor_scale(amax)
        xb = x.unflatten(-1, (-1, 16))
        e4 = (xb.abs().amax(-1) / _f32(6.0) / sg).clamp(max=448.0).to(torch.float8_e4m3fn)
        sb = sg * e4.float()
        r, bytes_ = torch.where(sb != 0, _f32(1.0) / sb, _f32(0.0)), e4.view(torch.uint8)
    else:
        xb = x.unflatten(-1, (-1, 32))
        a = xb.abs().amax(-1).view(torch.int32)
        byte = ((a >> 23) - 2 + ((a & 0x7FFFFF) > 0x400000).int()).clamp(min=0)
        r, bytes_ = ((254 - byte) << 23).view(torch.float32), byte.to(torch.uint8)
    c = _e2m1_codes(xb * r[..., None]).flatten(-2).unflatten(-1, (-1, 2))
    return c[..., 0] | (c[..., 1] << 4), bytes_


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _dequantize(pairs, packed, scales, fmt, amax):
    """Packed codes [..., D/2] and scale bytes -> float32 values [..., D]; pairs: the two
    values of each byte, [256, 2]."""
    v = pairs[packed.int()].flatten(-2)
    if fmt == "nv":
        s = _tensor_scale(amax) * scales.view(torch.float8_e4m3fn).float()
    else:
        s = (scales.int() << 23).view(torch.float32)
    return (v.unflatten(-1, (-1, 16 if fmt == "nv" else 32)) * s[..., None]).flatten(-2)


# ------------------------------------------------------------------ inputs ----
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _keys(g, n, H, D):
    """N(0, 1) with one channel in 32 five times as large, as keys have them."""
    k = _randn(g, n, H, D)
    k[..., torch.randperm(D, generator=g, device=DEV)[: D // 32]] *= 5.0
    return k


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    fmt, H, D, ps, op = case["fmt"], case["H"], case["D"], case["page"], case["op"]
    sizes = _sizes(case)
    order = torch.randperm(len(sizes), generator=g, device=DEV).tolist()
    lens, rows = [sizes[b][0] for b in order], [sizes[b][1] for b in order]
    B, T, most = len(sizes), sum(rows), max(lens)
    wide = max(1, -(-most // ps))
    num = B * wide
    s = {"case": case, "T": T, "most_rows": max(rows), "most": most,
         "lengths": torch.tensor(lens, dtype=torch.int32, device=DEV),
         "offsets": torch.tensor([0] + rows, device=DEV).cumsum(0).to(torch.int32),
         # pages in the order in which a running server hands them out
         "pages": torch.randperm(num, generator=g, device=DEV).reshape(B, wide).to(torch.int32),
         "pairs": torch.tensor([[E2M1[b & 15], E2M1[b >> 4]] for b in range(256)], device=DEV),
         "amax": (None, None)}
    dt = TYPES[case["dtype"]]
    if op == "append":
        # keys and values lie behind the queries in one projection's rows
        qkv = torch.empty(T, 2 * H * case["group"] + 2 * H, D, dtype=dt, device=DEV)
        s["k"], s["v"] = qkv[:, -2 * H:-H], qkv[:, -H:]
        s["k"].copy_(_keys(g, T, H, D))
        s["v"].copy_(_randn(g, T, H, D))
        if fmt == "nv":
            # calibrated on other tokens: a few values lie above
            s["amax"] = (s["k"].abs().amax().float().reshape(1) * 0.97, s["v"].abs().amax().float().reshape(1) * 0.97)
        bs = 16 if fmt == "nv" else 32
        store = [torch.zeros(num, H, ps, w, dtype=torch.uint8, device=DEV) for w in (D // 2, D // bs, D // 2, D // bs)]
    else:
        k, v = _keys(g, num * ps, H, D), _randn(g, num * ps, H, D)
        if fmt == "nv":
            s["amax"] = (k.abs().amax().reshape(1), v.abs().amax().reshape(1))
        store = []
        for x, a in ((k, s["amax"][0]), (v, s["amax"][1])):
            for t in _quantize(x, fmt, a):
                store.append(t.reshape(num, ps, H, -1).transpose(1, 2).contiguous())
        del k, v
        if op == "read":
            s["starts"] = s["lengths"] - (s["offsets"][1:] - s["offsets"][:-1])
        else:
            heads = H * case["group"]
            s["q"] = torch.empty(T, heads + 2 * H, D, dtype=dt, device=DEV)[:, :heads]
            s["q"].copy_(1.5 * _randn(g, T, heads, D))
    s["store"] = store
    if own:
        import micro_scaled_fp4_amd as fp4

        s["cache"] = fp4.KVCache(fp4.FP4_NVFP4 if fmt == "nv" else fp4.FP4_MXFP4, *store, *s["amax"])
    return s


# -------------------------------------------------------------- plain forms ----
def _rows(state):
    """Sequence of each row, and its place among the sequence's rows."""
    off = state["offsets"].long()
    r = torch.arange(state["T"], device=DEV)
    b = torch.searchsorted(off[1:].contiguous(), r, right=True)
    return b, r - off[b]


def _values(state, which, page, slot):
    """Float32 values at the given pages and slots, [..., H, D]."""
    codes, scales = state["store"][2 * which:2 * which + 2]
    return _dequantize(state["pairs"], codes[page, :, slot], scales[page, :, slot], state["case"]["fmt"],
                       state["amax"][which])


def _read_at(state, b, pos):
    ps = state["case"]["page"]
    page, slot = state["pages"][b, pos // ps].long(), pos % ps
    dt = TYPES[state["case"]["dtype"]]
    return {"k": _values(state, 0, page, slot).to(dt), "v": _values(state, 1, page, slot).to(dt)}


def _plain_append(state):
    case, (b, i) = state["case"], _rows(state)
    off = state["offsets"].long()
    pos = state["lengths"].long()[b] - (off[b + 1] - off[b]) + i
    page, slot = state["pages"][b, pos // case["page"]].long(), pos % case["page"]
    kc, ks = _quantize(state["k"], case["fmt"], state["amax"][0])
    vc, vs = _quantize(state["v"], case["fmt"], state["amax"][1])
    store = state["store"]
    store[0][page, :, slot] = kc
    store[1][page, :, slot] = ks
    store[2][page, :, slot] = vc
    store[3][page, :, slot] = vs
    return _read_at(state, b, pos)


def _plain_read(state):
    b, i = _rows(state)
    return _read_at(state, b, state["starts"].long()[b] + i)


def _plain_attend(state):
    """Every sequence padded to the longest and to the most rows, dense scores."""
    case = state["case"]
    H, G, D, ps = case["H"], case["group"], case["D"], case["page"]
    off, L = state["offsets"].long(), state["lengths"].long()
    B, n, most = L.numel(), state["most_rows"], state["most"]
    t = torch.arange(most, device=DEV)
    page, slot = state["pages"][:, t // ps].long(), (t % ps).expand(B, most)
    k = _values(state, 0, page, slot).permute(0, 2, 3, 1).contiguous()      # [B, H, D, L]
    v = _values(state, 1, page, slot).transpose(1, 2).contiguous()         # [B, H, L, D]
    i = torch.arange(n, device=DEV)
    at = off[:-1, None] + i
    inside = at < off[1:, None]
    q = state["q"][at.clamp(max=state["T"] - 1)].float().reshape(B, n, H, G, D)
    q = q.permute(0, 2, 3, 1, 4).reshape(B, H, G * n, D)
    s = torch.matmul(q, k).mul_(1.0 / math.sqrt(D)).view(B, H, G, n, most)
    p = (L - (off[1:] - off[:-1]))[:, None] + i
    seen = (t < L[:, None])[:, None, :].expand(B, n, most)
    if case["causal"]:
        seen = seen & (t <= p[..., None])
    if case["window"]:
        seen = seen & (t > p[..., None] - case["window"])
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, _f32(0.0), m)
    e = s.sub_(m).exp_()
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, H, G * n, most), v).view(B, H, G, n, D)
    o = torch.where(l > 0, o / l, _f32(0.0))
    out = {"out": o.permute(0, 3, 1, 2, 4).reshape(B, n, H * G, D)[inside].to(state["q"].dtype)}
    if case["lse"]:
        lse = torch.where(l > 0, m + torch.log(l), _f32(-math.inf))[..., 0]
        out["lse"] = lse.permute(0, 3, 1, 2).reshape(B, n, H * G)[inside]
    return out


# ------------------------------------------------------- the framework's own ----
def _own(state):
    import micro_scaled_fp4_amd as fp4

    case, cache = state["case"], state["cache"]
    where = (state["offsets"], state["lengths"], state["pages"])
    dt = TYPES[case["dtype"]]
    if case["op"] == "attend":
        got = fp4.kv_cache_attention(cache, state["q"], *where, scale=1.0 / math.sqrt(case["D"]), causal=case["causal"],
                                     window=case["window"], return_lse=case["lse"])
        return {"out": got[0], "lse": got[1]} if case["lse"] else {"out": got}
    if case["op"] == "append":
        fp4.kv_cache_write(cache, state["k"], state["v"], *where)
        # no starts: a sequence's last rows
        k, v = fp4.kv_cache_read(cache, *where, state["T"], out_dtype=dt)
    else:
        k, v = fp4.kv_cache_read(cache, *where, state["T"], starts=state["starts"], out_dtype=dt)
    return {"k": k, "v": v}


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "read": _plain_read, "attend": _plain_attend}[state["case"]["op"]](state)


# -------------------------------------------------------------------- work ----
def work(case):
    size = {"bf16": 2, "f32": 4}[case["dtype"]]
    H, D, G = case["H"], case["D"], case["group"]
    row = 2 * H * D * (0.5 + (1 / 16 if case["fmt"] == "nv" else 1 / 32))   # a position's bytes in the cache
    T = sum(n for _, n in _sizes(case))
    if case["op"] == "append":
        # read in, written, and read again where the values are returned
        return {"bytes": int(T * (4 * H * D * size + 2 * row)), "flops": 8 * T * H * D}
    if case["op"] == "read":
        return {"bytes": int(T * (2 * H * D * size + row)), "flops": 4 * T * H * D}
    held = pairs = 0
    for length, n in _sizes(case):
        w = case["window"] or length
        first = length - n + 1            # positions that the first row sees, without a window
        if not case["causal"]:
            held, pairs = held + length, pairs + n * length
            continue
        held += max(0, min(length, w + n - 1))
        # sum over i of min(first + i, w), rows before the sequence's start seeing nothing
        low, count = max(first, 1), min(n, length)
        short = max(0, min(count, w - low + 1))
        pairs += short * low + short * (short - 1) // 2 + (count - short) * w
    b = held * row + T * H * G * (2 * D * size + (4 if case["lse"] else 0))
    return {"bytes": int(b), "flops": 4 * D * H * G * pairs}


# ------------------------------------------------------- in 64 bits, apart ----
def _exact_values(codes, scales, fmt, amax):
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    exp2, man = ((code >> 1) & 3).double(), (code & 1).double()
    mag = torch.where(exp2 > 0, torch.exp2(exp2 - 1) * (1 + 0.5 * man), 0.5 * man)
    mag = torch.where(code >= 8, -mag, mag)
    s = scales.double()
    if fmt == "nv":
        e, m = torch.floor(s / 8), s % 8
        s = torch.where(e > 0, torch.exp2(e - 7) * (1 + m / 8), m / 512) * (amax.double() / 2688)
    else:
        s = torch.exp2(s - 127)
    return mag * torch.repeat_interleave(s, 16 if fmt == "nv" else 32, dim=-1)


def exact(case, seed):
    if case["op"] == "append":
        # the quantized values are decisions of 32-bit steps: no 64-bit value
        return None
    st = prepare(case, seed)
    ps, fmt, D, G = case["page"], case["fmt"], case["D"], case["group"]
    off, lens = st["offsets"].tolist(), st["lengths"].tolist()

    def held(b, which):
        """Sequence b's positions in order, [H, length, .] bytes."""
        pages = st["pages"][b].long()
        return [st["store"][2 * which + j][pages].transpose(0, 1).flatten(1, 2)[:, :lens[b]] for j in (0, 1)]

    parts = []
    for b in range(len(lens)):
        n, L = off[b + 1] - off[b], lens[b]
        keys, values = held(b, 0), held(b, 1)
        if case["op"] == "read":
            parts.append([_exact_values(c[:, L - n:], s[:, L - n:], fmt, a).transpose(0, 1)
                          for (c, s), a in zip((keys, values), st["amax"])])
            continue
        out = torch.zeros(n, case["H"] * G, D, dtype=torch.float64, device=DEV)
        lse = torch.full((n, case["H"] * G), -math.inf, dtype=torch.float64, device=DEV)
        at = torch.arange(L - n, L, device=DEV)[:, None]
        t = torch.arange(L, device=DEV)
        seen = torch.ones(n, L, dtype=torch.bool, device=DEV)
        if case["causal"]:
            seen &= t <= at
        if case["window"]:
            seen &= at - t < case["window"]
        for h in range(case["H"] if L else 0):
            k = _exact_values(keys[0][h], keys[1][h], fmt, st["amax"][0])
            v = _exact_values(values[0][h], values[1][h], fmt, st["amax"][1])
            for j in range(h * G, h * G + G):
                x = (st["q"][off[b]:off[b + 1], j].double() @ k.T) / math.sqrt(D)
                x = torch.where(seen, x, -math.inf)
                lse[:, j] = torch.logsumexp(x, 1)
                out[:, j] = torch.nan_to_num(torch.softmax(x, 1)) @ v
        parts.append([out, lse])
    if case["op"] == "read":
        return {"k": torch.cat([p[0] for p in parts]), "v": torch.cat([p[1] for p in parts])}
    got = {"out": torch.cat([p[0] for p in parts])}
    if case["lse"]:
        got["lse"] = torch.cat([p[1] for p in parts])
    return got
