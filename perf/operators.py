"""The operators around FP4 expert layers as measured cases: routing tokens to
experts, moving their rows to the experts and back, and the block-scaled FP4
product with bias, activation and residual in its epilogue.

`run` computes a case either in plain torch operations in 32 bits (own = False)
or through micro_scaled_fp4_amd (own = True), on the inputs that `prepare` makes
from a seed.  `exact` computes the same outputs from the definitions in 64 bits.

Definitions
-----------
Routing.  Per token, over its E logits l (NaN and -inf: the expert is masked):
  score s = softmax(l) or sigmoid(l); selection value v = l, or s + bias where a
  bias is given (bias only selects), or s where group scores are sums of two.
  Groups: a group's score is the sum of its group_top largest v; only the experts
  of the top_groups best groups stay.  ids: the k largest v, ties to the lowest
  index; -1 past the unmasked ones.  weights: scale * s, or scale * s / (sum of
  the selected s) when renormalized; 0 where the id is -1.
  Backward: the gradient of the weights with respect to the logits (ids fixed).
Product.  z = alpha * A @ W^T + bias over dequantized FP4 operands, alpha the
  product of the tensor scales; D = act(z) + residual, or, gated,
  act(z[:, 0::2]) * z[:, 1::2] + residual.  Experts: row group e uses W[e], bias[e].
  Backward: dz from dD and z, and the bias gradient sum over rows of dz.
Dispatch.  Rows (token, slot) sorted by expert, stable in t * k + slot; the
  tokens quantized to FP4 (one tensor scale) and laid out in that order.
Combine.  y[t] = sum over slots of weight * row (+ residual); backward: the
  gradients of the rows and of the weights.
"""
import math

import torch

own = False

DEV = "cuda"
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases ----
def _route(name, T, E, k, score, dtype, bias=False, groups=1, top_groups=1, group_top=1,
           renorm=True, scale=1.0, padded=0, backward=False):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "score": score, "dtype": dtype,
            "bias": bias, "groups": groups, "top_groups": top_groups, "group_top": group_top,
            "renorm": renorm, "scale": scale, "padded": padded, "backward": backward}


def _product(name, fmt, M, N, K, act, out, gated=False, bias="", residual="", preact=""):
    return {"name": name, "op": "product", "fmt": fmt, "M": M, "N": N, "K": K, "act": act,
            "out": out, "gated": gated, "bias": bias, "residual": residual, "preact": preact}


def _experts(name, fmt, T, E, k, N, K, act, out, gated=False, bias=""):
    return {"name": name, "op": "experts", "fmt": fmt, "T": T, "E": E, "k": k, "N": N, "K": K,
            "act": act, "out": out, "gated": gated, "bias": bias}


def _epilogue_backward(name, M, N, act, dtype, gated):
    return {"name": name, "op": "epilogue_backward", "M": M, "N": N, "act": act, "dtype": dtype,
            "gated": gated}


def _dispatch(name, fmt, T, H, E, k, dtype):
    return {"name": name, "op": "dispatch", "fmt": fmt, "T": T, "H": H, "E": E, "k": k,
            "dtype": dtype}


def _combine(name, T, H, E, k, dtype, residual, backward):
    return {"name": name, "op": "combine", "T": T, "H": H, "E": E, "k": k, "dtype": dtype,
            "residual": residual, "backward": backward}


def listed():
    return [
        # one decoded token routed to 8 of 64 experts: latency only
        _route("route_token", 1, 64, 8, "softmax", "bf16"),
        # a training batch over 256 experts in 8 groups, sigmoid scores with a balance bias,
        # forward and backward; the last tokens are padding (every logit masked)
        _route("route_train_groups", 32768, 256, 8, "sigmoid", "f32", bias=True, groups=8,
               top_groups=4, group_top=2, scale=2.5, padded=77, backward=True),
        # one decoded token through a dense layer of the decode shape (27648 x 5120)
        _product("product_token", "nv", 1, 27648, 5120, "gelu", "bf16", bias="f32"),
        # a short prompt of odd length through a layer whose sizes fill no tile; the
        # pre-activations are kept for training
        _product("product_ragged", "mx", 1021, 5125, 7200, "silu", "f32", bias="bf16",
                 residual="f32", preact="f32"),
        # a prefill through the first layer of a feed-forward block (8192 x 28672 x 8192)
        _product("product_prefill", "mx", 8192, 28672, 8192, "gelu_tanh", "bf16", bias="bf16",
                 residual="bf16"),
        # 16 decoded tokens through the gate and up projections of 64 experts (top 8)
        _experts("experts_decode", "nv", 16, 64, 8, 4096, 7168, "silu", "bf16", gated=True),
        # 4096 prompt tokens through the same layer: 32768 routed rows
        _experts("experts_prefill", "nv", 4096, 64, 8, 4096, 7168, "silu", "bf16", gated=True,
                 bias="f32"),
        # a training step's way back through a gated activation and its bias
        _epilogue_backward("epilogue_train", 8192, 28672, "silu", "bf16", True),
        # rows of 16 decoded tokens sorted by expert and quantized
        _dispatch("dispatch_decode", "nv", 16, 7168, 64, 8, "bf16"),
        # the same for a prompt of 4096 tokens
        _dispatch("dispatch_prefill", "nv", 4096, 7168, 64, 8, "bf16"),
        # 16 decoded tokens: expert outputs weighted and summed onto the residual stream
        _combine("combine_decode", 16, 7168, 64, 8, "bf16", True, False),
        # a training batch: the sum and both of its gradients
        _combine("combine_train", 4096, 7168, 64, 8, "bf16", False, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "product", "experts", "epilogue_backward", "dispatch", "combine"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log_int(rng, max(2, 8 // groups), 512 // groups)
        top_groups = rng.randint(max(1, groups // 2), groups)
        k = rng.randint(1, min(16, E // groups * top_groups))
        T = _log_int(rng, 1, 32768 * 256 // max(256, E))
        return _route("", T, E, k, rng.choice(["softmax", "sigmoid"]), rng.choice(["bf16", "f32"]),
                      bias=rng.random() < 0.5, groups=groups, top_groups=top_groups,
                      group_top=rng.choice([1, 2]), renorm=rng.random() < 0.7,
                      scale=rng.choice([1.0, 2.5]), padded=rng.choice([0, T // 16]),
                      backward=rng.random() < 0.5)
    if op in ("product", "experts"):
        fmt, act, out = rng.choice(["nv", "mx"]), rng.choice(ACTS), rng.choice(["bf16", "f32"])
        gated = act != "none" and rng.random() < 0.5
        K = 32 * _log_int(rng, 4, 256)
        N = _log_int(rng, 16, 28672)
        N += N % 2 if gated else 0
        bias = rng.choice(["", "f32", "bf16"])
        if op == "product":
            M = _log_int(rng, 1, min(8192, max(1, 2 ** 40 // (N * K))))
            return _product("", fmt, M, N, K, act, out, gated, bias,
                            rng.choice(["", "f32", "bf16"]), rng.choice(["", out]))
        E = _log_int(rng, 2, 128)
        N = min(N, max(16, 2 ** 30 // (E * K) // 2 * 2))
        k = rng.randint(1, min(8, E))
        # the plain form pads every expert to the fullest one: rows per expert stay in reach
        T = _log_int(rng, 1, max(1, min(4096, 2 ** 38 // (N * K * k))))
        return _experts("", fmt, T, E, k, N, K, act, out, gated, bias)
    if op == "epilogue_backward":
        N = 2 * _log_int(rng, 8, 14336)
        return _epilogue_backward("", _log_int(rng, 1, 8192), N, rng.choice(ACTS[1:]),
                                  rng.choice(["bf16", "f32"]), rng.random() < 0.5)
    H = 32 * _log_int(rng, 4, 256)
    E = _log_int(rng, 2, 256)
    k = rng.randint(1, min(8, E))
    T = _log_int(rng, 1, 4096 * 7168 * 8 // (8192 * 8))
    dtype = rng.choice(["bf16", "f32"])
    if op == "dispatch":
        return _dispatch("", rng.choice(["nv", "mx"]), T, H, E, k, dtype)
    return _combine("", T, H, E, k, dtype, rng.random() < 0.5, rng.random() < 0.5)


# ----------------------------------------------------------------- formats ----
def _f32(v):
    return torch.full((1,), v, dtype=torch.float32, device=DEV)


def _e2m1_codes(q):
    """Codes of the nearest E2M1 magnitudes (ties to the even code), sign kept."""
    m = q.abs()
    c = (m > 0.25).to(torch.uint8)
    for above in (m >= 0.75, m > 1.25, m >= 1.75, m > 2.5, m >= 3.5, m > 5.0):
        c += above
    return c | (torch.signbit(q).to(torch.uint8) << 3)


def _pack(codes):
    c = codes.reshape(*codes.shape[:-1], -1, 2)
    return c[..., 0] | (c[..., 1] << 4)


def _quantize(x, fmt):
    """x [..., K] float32 -> (4-bit codes [..., K], scale bytes, tensor scale [1] or None)."""
    if fmt == "nv":
        G = x.abs().amax().reshape(1)
        sg = torch.where(G != 0, G / _f32(2688.0), _f32(1.0))
        xb = x.unflatten(-1, (-1, 16))
        t = xb.abs().amax(-1) / _f32(6.0) / sg
        e4 = t.clamp(max=448.0).to(torch.float8_e4m3fn)
        sb = sg * e4.float()
        r = torch.where(sb != 0, _f32(1.0) / sb, _f32(0.0))
        return _e2m1_codes(xb * r[..., None]).flatten(-2), e4.view(torch.uint8), sg
    xb = x.unflatten(-1, (-1, 32))
    a = xb.abs().amax(-1).view(torch.int32)
    byte = ((a >> 23) - 2 + ((a & 0x7FFFFF) > 0x400000).int()).clamp(min=0)
    r = ((254 - byte) << 23).view(torch.float32)
    return _e2m1_codes(xb * r[..., None]).flatten(-2), byte.to(torch.uint8), None


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _block_scales(scales, fmt, sg):
    """Float32 block scales of scale bytes, the tensor scale included."""
    if fmt == "nv":
        s = scales.view(torch.float8_e4m3fn).float()
        return s if sg is None else s * sg.reshape(-1, *[1] * (s.dim() - 1))
    return (scales.int() << 23).view(torch.float32)


def _dequantize(pairs, packed, scales, fmt, sg=None):
    """Packed codes [..., K/2] and scale bytes -> float32 values [..., K]; pairs: the two
    values of each byte, [256, 2]."""
    v = pairs[packed.int()].flatten(-2)
    block = 16 if fmt == "nv" else 32
    return (v.unflatten(-1, (-1, block)) * _block_scales(scales, fmt, sg)[..., None]).flatten(-2)


# ------------------------------------------------------------------ inputs ----
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _activations(g, rows, cols):
    """N(0, 1) with 0.5% of the channels scaled by 40."""
    x = _randn(g, rows, cols)
    hot = torch.randperm(cols, generator=g, device=DEV)[: max(1, cols // 200)]
    x[:, hot] *= 40.0
    return x


def _expert_ids(g, T, E, k):
    """k distinct experts per token, popularities exp(N(0, 0.5^2))."""
    pop = 0.5 * _randn(g, E)
    u = torch.rand(T, E, generator=g, device=DEV).clamp(min=1e-20)
    return torch.topk(pop - torch.log(-torch.log(u)), k, dim=1).indices.to(torch.int32)


def _bits64(case, logits, bias):
    """Scores and selection values of a routing case in 64 bits."""
    l = logits.double()
    dead = torch.isnan(l) | (l == -math.inf)
    lm = torch.where(dead, torch.full_like(l, -math.inf), l)
    if case["score"] == "softmax":
        top = lm.amax(1, keepdim=True)
        e = torch.where(dead, torch.zeros_like(l), torch.exp(lm - torch.where(top == -math.inf, 0.0, top)))
        tot = e.sum(1, keepdim=True)
        s = torch.where(tot > 0, e / tot, torch.zeros_like(e))
    else:
        s = torch.where(dead, torch.zeros_like(l), torch.sigmoid(lm))
    if bias is not None:
        v = s + bias.double()
    elif case["groups"] > 1 and case["group_top"] == 2:
        v = s
    else:
        v = lm
    return s, torch.where(dead, torch.full_like(l, -math.inf), v), dead


def _prepare_route(case, g):
    T, E = case["T"], case["E"]
    dt = TYPES[case["dtype"]]
    # a balance bias moves in fixed small steps
    bias = None
    if case["bias"]:
        bias = torch.randint(-60, 61, (E,), generator=g, device=DEV).float() * 0.001
    logits = (1.5 * _randn(g, T, E)).to(dt)
    for _ in range(3):
        # Where two selection values differ by less than 32 bits resolve, either order is
        # right: such rows are drawn anew, so that the order is part of the answer.  (Values
        # that are equal stay: ties go to the lowest index.)
        s, v, _ = _bits64(case, logits, bias)
        near = torch.zeros(T, dtype=torch.bool, device=DEV)
        top = torch.sort(v, dim=1, descending=True).values
        gap = top[:, :-1] - top[:, 1:]
        if bias is not None or (case["groups"] > 1 and case["group_top"] == 2):
            near |= ((gap > 0) & (gap < 2e-6)).any(1)
        if case["groups"] > 1 and case["group_top"] == 2:
            gs = torch.sort(v.reshape(T, case["groups"], -1), dim=2, descending=True).values[..., :2].sum(2)
            gs = torch.sort(gs, dim=1, descending=True).values
            gap = gs[:, :-1] - gs[:, 1:]
            near |= ((gap > 0) & (gap < 4e-6)).any(1)
        logits = torch.where(near[:, None], (1.5 * _randn(g, T, E)).to(dt), logits)
    if case["padded"]:
        logits[T - case["padded"]:] = -math.inf
    dw = _randn(g, T, case["k"]) if case["backward"] else None
    return {"logits": logits, "bias": bias, "dw": dw}


def _operand(g, rows, K, fmt, std, experts=0):
    """An FP4 operand: packed codes, scale bytes and tensor scale(s)."""
    shape = (experts, rows, K) if experts else (rows, K)
    x = _randn(g, *shape).mul_(std) if std else _activations(g, rows, K)
    codes, scales, sg = _quantize(x, fmt)
    if experts and fmt == "nv":
        # one tensor scale per expert: experts trained to different magnitudes
        sg = sg * (1.0 + 0.25 * torch.rand(experts, generator=g, device=DEV))
    return _pack(codes), scales, sg


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case, "pairs": torch.tensor([[E2M1[b & 15], E2M1[b >> 4]] for b in range(256)], device=DEV)}
    if op == "route":
        s.update(_prepare_route(case, g))
    elif op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        No = N // 2 if case["gated"] else N
        s["A"] = _operand(g, M, K, case["fmt"], 0.0)
        s["W"] = _operand(g, N, K, case["fmt"], 0.02)
        s["bias"] = (0.5 * _randn(g, N)).to(TYPES[case["bias"]]) if case["bias"] else None
        s["residual"] = _randn(g, M, No).to(TYPES[case["residual"]]) if case["residual"] else None
    elif op == "experts":
        T, E, N, K = case["T"], case["E"], case["N"], case["K"]
        ids = _expert_ids(g, T, E, case["k"])
        sizes = torch.bincount(ids.flatten().long(), minlength=E)
        s["A"] = _operand(g, T * case["k"], K, case["fmt"], 0.0)
        s["W"] = _operand(g, N, K, case["fmt"], 0.02, experts=E)
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), sizes.cumsum(0)]).to(torch.int32)
        s["most"] = int(sizes.max())
        s["bias"] = (0.5 * _randn(g, E, N)).to(TYPES[case["bias"]]) if case["bias"] else None
    elif op == "epilogue_backward":
        dt = TYPES[case["dtype"]]
        s["z"] = (1.5 * _randn(g, case["M"], case["N"])).to(dt)
        s["dD"] = (0.01 * _randn(g, case["M"], case["N"] // 2 if case["gated"] else case["N"])).to(dt)
    elif op == "dispatch":
        s["x"] = _activations(g, case["T"], case["H"]).to(TYPES[case["dtype"]])
        s["ids"] = _expert_ids(g, case["T"], case["E"], case["k"])
    else:
        T, H, k, dt = case["T"], case["H"], case["k"], TYPES[case["dtype"]]
        ids = _expert_ids(g, T, case["E"], k)
        order = torch.argsort(ids.flatten(), stable=True)
        s["row_slots"] = order.to(torch.int32)
        s["slot_rows"] = torch.argsort(order, stable=True).to(torch.int32).reshape(T, k)
        s["rows"] = _randn(g, T * k, H).to(dt)
        s["weights"] = torch.softmax(_randn(g, T, k), 1)
        s["residual"] = _randn(g, T, H).to(dt) if case["residual"] else None
        s["dy"] = (0.01 * _randn(g, T, H)).to(dt) if case["backward"] else None
    return s


# -------------------------------------------------------------- plain forms ----
def _sum_selected(s, ids):
    live = ids >= 0
    picked = torch.gather(s, 1, ids.clamp(min=0).long())
    return torch.where(live, picked, torch.zeros_like(picked)), live


def _plain_route(state):
    case, bias = state["case"], state["bias"]
    l = state["logits"].float()
    T, E = l.shape
    k, G = case["k"], case["groups"]
    minus = _f32(-math.inf)
    dead = torch.isnan(l) | (l == minus)
    lm = torch.where(dead, minus, l)
    if case["score"] == "softmax":
        top = lm.amax(1, keepdim=True)
        e = torch.where(dead, _f32(0.0), torch.exp(lm - torch.where(top == minus, _f32(0.0), top)))
        tot = e.sum(1, keepdim=True)
        s = torch.where(tot > 0, e / tot, _f32(0.0))
    else:
        s = torch.where(dead, _f32(0.0), 1.0 / (1.0 + torch.exp(-lm)))
    two = G > 1 and case["group_top"] == 2
    v = s + bias if bias is not None else s if two else lm
    v = torch.where(dead, minus, v)
    if G > 1:
        members = torch.sort(v.reshape(T, G, E // G), dim=2, descending=True).values[..., : case["group_top"]]
        gs = torch.where(members == minus, _f32(0.0), members).sum(2)
        gs = torch.where(members[..., 0] == minus, minus, gs)
        best = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, : case["top_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=DEV).scatter_(1, best, True)
        v = torch.where(keep[..., None].expand(T, G, E // G).reshape(T, E), v, minus)
    got = torch.sort(v, dim=1, descending=True, stable=True)
    ids = torch.where(got.values[:, :k] == minus, -1, got.indices[:, :k]).to(torch.int32)
    picked, live = _sum_selected(s, ids)
    scale = case["scale"]
    total = picked.sum(1, keepdim=True)
    if case["renorm"]:
        q = torch.where(total > 0, picked / total, _f32(0.0))
    else:
        q = picked
    out = {"ids": ids, "weights": q * scale}
    if case["backward"]:
        dw = torch.where(live, state["dw"], _f32(0.0)) * scale
        softmax = case["score"] == "softmax"
        at = ids.clamp(min=0).long()
        if case["renorm"]:
            inner = dw - (dw * q).sum(1, keepdim=True)
            # softmax: through the selected logits; sigmoid: through s and its derivative
            per = q * inner if softmax else q * inner * (1.0 - picked)
            dl = torch.zeros_like(l).scatter_add_(1, at, torch.where(live, per, _f32(0.0)))
        elif softmax:
            mean = (dw * picked).sum(1, keepdim=True)
            dl = torch.zeros_like(l).scatter_add_(1, at, dw * picked) - s * mean
        else:
            dl = torch.zeros_like(l).scatter_add_(1, at, dw * picked * (1.0 - picked))
        out["d_logits"] = dl.to(state["logits"].dtype)
    return out


def _act(x, act):
    if act == "relu":
        return torch.clamp(x, min=0.0)
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * torch.special.erfc(x * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def _epilogue(z, case, residual):
    d = _act(z[..., 0::2], case["act"]) * z[..., 1::2] if case["gated"] else _act(z, case["act"])
    return (d if residual is None else d + residual.float()).to(TYPES[case["out"]])


def _plain_product(state):
    case = state["case"]
    A = _dequantize(state["pairs"], *state["A"][:2], case["fmt"])
    W = _dequantize(state["pairs"], *state["W"][:2], case["fmt"])
    z = A @ W.T
    if case["fmt"] == "nv":
        z = z * (state["A"][2] * state["W"][2])
    if state["bias"] is not None:
        z = z + state["bias"].float()
    out = {"D": _epilogue(z, case, state["residual"])}
    if case["preact"]:
        out["z"] = z.to(TYPES[case["preact"]])
    return out


def _plain_experts(state):
    """Every expert's rows padded to the fullest expert's, one batched product."""
    case, most = state["case"], state["most"]
    A = _dequantize(state["pairs"], *state["A"][:2], case["fmt"])
    W = _dequantize(state["pairs"], *state["W"][:2], case["fmt"])
    lo, hi = state["offsets"][:-1].long(), state["offsets"][1:].long()
    at = lo[:, None] + torch.arange(most, device=DEV)
    inside = at < hi[:, None]
    z = torch.bmm(A[at.clamp(max=A.shape[0] - 1)], W.transpose(1, 2))
    if case["fmt"] == "nv":
        z = z * (state["A"][2] * state["W"][2])[:, None, None]
    if state["bias"] is not None:
        z = z + state["bias"].float()[:, None, :]
    return {"D": _epilogue(z[inside], case, None)}


def _act_grad(x, act):
    if act == "relu":
        return (x > 0).float()
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-x))
        return s * (1.0 + x * (1.0 - s))
    if act == "gelu":
        return 0.5 * torch.special.erfc(x * -math.sqrt(0.5)) + x * torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (x + 0.044715 * x * x * x))
        return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * x * x)
    return torch.ones_like(x)


def _plain_epilogue_backward(state):
    case = state["case"]
    z, d = state["z"].float(), state["dD"].float()
    if case["gated"]:
        gate, up = z[:, 0::2], z[:, 1::2]
        dz = torch.stack([d * up * _act_grad(gate, case["act"]), d * _act(gate, case["act"])], 2).flatten(1)
    else:
        dz = d * _act_grad(z, case["act"])
    return {"dz": dz.to(state["z"].dtype), "dbias": dz.sum(0)}


def _plain_dispatch(state):
    case = state["case"]
    T, k, E = case["T"], case["k"], case["E"]
    flat = state["ids"].flatten()
    order = torch.argsort(flat, stable=True)
    slot_rows = torch.argsort(order, stable=True).reshape(T, k)
    ends = torch.searchsorted(flat[order].contiguous(), torch.arange(E + 1, device=DEV, dtype=torch.int32))
    codes, scales, sg = _quantize(state["x"].float(), case["fmt"])
    token = order // k
    values = _dequantize(state["pairs"], _pack(codes)[token], scales[token], case["fmt"], sg)
    return {"values": values.to(torch.bfloat16), "offsets": ends.to(torch.int32),
            "slot_rows": slot_rows.to(torch.int32), "row_slots": order.to(torch.int32)}


def _plain_combine(state):
    case, w = state["case"], state["weights"]
    at = state["slot_rows"].long()
    r = state["rows"].float()[at]
    y = (r * w[..., None]).sum(1)
    if state["residual"] is not None:
        y = y + state["residual"].float()
    out = {"y": y.to(TYPES[case["dtype"]])}
    if case["backward"]:
        dy = state["dy"].float()
        d = torch.empty_like(state["rows"])
        d[at.flatten()] = (w[..., None] * dy[:, None, :]).flatten(0, 1).to(d.dtype)
        out["d_rows"] = d
        out["d_weights"] = (r * dy[:, None, :]).sum(2)
    return out


# ------------------------------------------------------- the framework's own ----
def _own(state):
    import micro_scaled_fp4_amd as fp4

    case, op = state["case"], state["case"]["op"]
    if op == "route":
        score = fp4.FP4_SCORE_SOFTMAX if case["score"] == "softmax" else fp4.FP4_SCORE_SIGMOID
        ids, weights = fp4.moe_route(state["logits"], case["k"], score=score, bias=state["bias"],
                                     num_groups=case["groups"], top_groups=case["top_groups"],
                                     group_top=case["group_top"], renormalize=case["renorm"],
                                     scale=case["scale"])
        out = {"ids": ids, "weights": weights}
        if case["backward"]:
            out["d_logits"] = fp4.moe_route_backward(state["dw"], state["logits"], ids, score=score,
                                                     renormalize=case["renorm"], scale=case["scale"])
        return out
    if op == "combine":
        out = {"y": fp4.moe_combine(state["rows"], state["weights"], state["slot_rows"],
                                    residual=state["residual"], out_dtype=TYPES[case["dtype"]])}
        if case["backward"]:
            out["d_rows"], out["d_weights"] = fp4.moe_combine_backward(
                state["dy"], state["rows"], state["weights"], state["slot_rows"], state["row_slots"])
        return out
    if op == "epilogue_backward":
        dz, dbias = fp4.fp4_epilogue_backward(state["dD"], state["z"], ACTS.index(case["act"]),
                                              gated=case["gated"], out_dtype=TYPES[case["dtype"]])
        return {"dz": dz, "dbias": dbias}
    fmt = fp4.FP4_NVFP4 if case["fmt"] == "nv" else fp4.FP4_MXFP4
    if op == "dispatch":
        codes, scales, _, sg, offsets, slot_rows, row_slots = fp4.moe_dispatch(
            fmt, state["x"], state["ids"], case["E"])
        return {"values": fp4.fp4_dequantize(fmt, codes, scales, sg, case["H"], torch.bfloat16),
                "offsets": offsets, "slot_rows": slot_rows, "row_slots": row_slots}
    (A, sa, ga), (W, sw, gw) = state["A"], state["W"]
    how = dict(activation=ACTS.index(case["act"]), gated=case["gated"], bias=state["bias"],
               out_dtype=TYPES[case["out"]])
    if op == "experts":
        return {"D": fp4.fp4_grouped_gemm_fused(fmt, A, sa, ga, W, sw, gw, state["offsets"],
                                                case["K"], **how)}
    got = fp4.fp4_scaled_gemm_fused(fmt, A, sa, ga, W, sw, gw, case["K"], residual=state["residual"],
                                    preact_dtype=TYPES.get(case["preact"]), **how)
    return {"D": got[0], "z": got[1]} if case["preact"] else {"D": got}


def run(state):
    if own:
        return _own(state)
    plain = {"route": _plain_route, "product": _plain_product, "experts": _plain_experts,
             "epilogue_backward": _plain_epilogue_backward, "dispatch": _plain_dispatch,
             "combine": _plain_combine}
    return plain[state["case"]["op"]](state)


# -------------------------------------------------------------------- work ----
def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4, "": 0}
    if op == "route":
        T, E, k, e = case["T"], case["E"], case["k"], size[case["dtype"]]
        b = T * E * e + T * k * 8 + (4 * E if case["bias"] else 0)
        if case["backward"]:
            b += T * E * e + T * k * 4
        return {"bytes": b, "flops": 4 * T * E}
    if op in ("product", "experts"):
        N, K = case["N"], case["K"]
        per = 0.5 + (1 / 16 if case["fmt"] == "nv" else 1 / 32)
        No = N // 2 if case["gated"] else N
        if op == "product":
            M, E, used = case["M"], 1, 1
            extra = M * No * size[case["residual"]] + M * N * size[case["preact"]]
        else:
            # experts that a draw of T * k slots over E is expected to reach
            M, E = case["T"] * case["k"], case["E"]
            used = E * (1 - (1 - case["k"] / E) ** case["T"])
            extra = 0
        b = (M * K + used * N * K) * per + M * No * size[case["out"]] + used * N * size[case["bias"]] + extra
        return {"bytes": int(b), "flops": 2 * M * N * K}
    if op == "epilogue_backward":
        M, N, e = case["M"], case["N"], size[case["dtype"]]
        return {"bytes": M * N * 2 * e + M * (N // 2 if case["gated"] else N) * e + 4 * N, "flops": 10 * M * N}
    T, H, k, e = case["T"], case["H"], case["k"], size[case["dtype"]]
    if op == "dispatch":
        # the codes are written, and read again where their values are returned in bf16
        per = 0.5 + (1 / 16 if case["fmt"] == "nv" else 1 / 32)
        return {"bytes": int(T * H * e + T * k * (H * (2 * per + 2) + 12) + 4 * (case["E"] + 1)),
                "flops": 4 * T * H}
    b = T * k * (H * e + 8) + T * H * e + (T * H * e if case["residual"] else 0)
    if case["backward"]:
        b += T * k * (2 * H * e + 12) + T * H * e
    return {"bytes": b, "flops": 2 * T * k * H}


# ------------------------------------------------------- in 64 bits, apart ----
def _exact_values(packed, scales, fmt):
    """Dequantized operand in 64 bits, without its tensor scale."""
    low, high = packed & 15, packed >> 4
    code = torch.stack([low, high], -1).flatten(-2)
    exp2, man = ((code >> 1) & 3).double(), (code & 1).double()
    mag = torch.where(exp2 > 0, torch.exp2(exp2 - 1) * (1 + 0.5 * man), 0.5 * man)
    mag = torch.where(code >= 8, -mag, mag)
    s = scales.double()
    if fmt == "nv":
        e, m = torch.floor(s / 8), s % 8
        s = torch.where(e > 0, torch.exp2(e - 7) * (1 + m / 8), m / 512)
    else:
        s = torch.exp2(s - 127)
    return mag * torch.repeat_interleave(s, 16 if fmt == "nv" else 32, dim=-1)


def _exact_act(x, act):
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return x * torch.special.ndtr(x)
    if act == "gelu_tanh":
        return x * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))
    return torch.relu(x) if act == "relu" else x


def _exact_route(case, st):
    l, bias, k, G = st["logits"], st["bias"], case["k"], case["groups"]
    T, E = l.shape
    s, v, dead = _bits64(case, l, bias)
    if G > 1:
        per = v.reshape(T, G, E // G)
        first = per.amax(2)
        gs = first
        if case["group_top"] == 2 and E // G > 1:
            second = torch.sort(per, dim=2).values[..., -2]
            gs = torch.where(second == -math.inf, first, first + second)
        # rank of a group: how many are better, or equal and earlier
        better = (gs[:, None, :] > gs[:, :, None]) | (
            (gs[:, None, :] == gs[:, :, None]) & (torch.arange(G, device=DEV)[None, :] < torch.arange(G, device=DEV)[:, None]))
        keep = better.sum(2) < case["top_groups"]
        v = torch.where(keep.repeat_interleave(E // G, dim=1), v, torch.full_like(v, -math.inf))
    ids, left = [], v.clone()
    for _ in range(k):
        best = left.amax(1)
        at = (left == best[:, None]).to(torch.int8).argmax(1)
        ids.append(torch.where(best == -math.inf, -1, at))
        left[torch.arange(T, device=DEV), at] = -math.inf
    ids = torch.stack(ids, 1)
    live = ids >= 0
    picked = torch.where(live, torch.gather(s, 1, ids.clamp(min=0)), 0.0)
    if case["renorm"]:
        tot = picked.sum(1, keepdim=True)
        w = torch.where(tot > 0, picked / tot, torch.zeros_like(picked)) * case["scale"]
    else:
        w = picked * case["scale"]
    out = {"ids": ids.to(torch.int32), "weights": w}
    if case["backward"]:
        # the weights again as a function of the logits, differentiated by torch
        leaf = torch.where(dead, torch.zeros_like(l.double()), l.double()).requires_grad_(True)
        if case["score"] == "softmax":
            lv = torch.where(dead, torch.full_like(leaf, -1e9), leaf)
            sc = torch.softmax(lv, 1)
        else:
            sc = torch.sigmoid(leaf)
        sel = torch.where(live, torch.gather(sc, 1, ids.clamp(min=0)), 0.0)
        if case["renorm"]:
            t = sel.sum(1, keepdim=True)
            sel = sel / torch.where(t > 0, t, torch.ones_like(t))
        (sel * case["scale"] * torch.where(live, st["dw"].double(), 0.0)).sum().backward()
        out["d_logits"] = torch.where(dead, torch.zeros_like(leaf), leaf.grad).detach()
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(case, st)
    if op in ("product", "experts"):
        fmt = case["fmt"]
        A = _exact_values(*st["A"][:2], fmt)

        def finish(z, residual):
            d = _exact_act(z[:, 0::2], case["act"]) * z[:, 1::2] if case["gated"] else _exact_act(z, case["act"])
            return d if residual is None else d + residual.double()

        if op == "product":
            z = A @ _exact_values(*st["W"][:2], fmt).T
            if fmt == "nv":
                z = z * (st["A"][2].double() * st["W"][2].double())
            if st["bias"] is not None:
                z = z + st["bias"].double()
            out = {"D": finish(z, st["residual"])}
            if case["preact"]:
                out["z"] = z
            return out
        offs, parts = st["offsets"].tolist(), []
        for e in range(case["E"]):
            if offs[e + 1] == offs[e]:
                continue
            z = A[offs[e]:offs[e + 1]] @ _exact_values(st["W"][0][e], st["W"][1][e], fmt).T
            if fmt == "nv":
                z = z * (st["A"][2].double() * st["W"][2][e].double())
            if st["bias"] is not None:
                z = z + st["bias"][e].double()
            parts.append(finish(z, None))
        return {"D": torch.cat(parts)}
    if op == "epilogue_backward":
        z = st["z"].double().requires_grad_(True)
        d = _exact_act(z[:, 0::2], case["act"]) * z[:, 1::2] if case["gated"] else _exact_act(z, case["act"])
        d.backward(st["dD"].double())
        return {"dz": z.grad, "dbias": z.grad.sum(0)}
    if op == "dispatch":
        # the quantized values are decisions of 32-bit steps: no 64-bit value
        return None
    w, at = st["weights"].double(), st["slot_rows"].long()
    y = st["residual"].double() if st["residual"] is not None else torch.zeros(case["T"], case["H"], dtype=torch.float64, device=DEV)
    for j in range(case["k"]):
        y = y + w[:, j:j + 1] * st["rows"][at[:, j]].double()
    out = {"y": y}
    if case["backward"]:
        dy = st["dy"].double()
        d = torch.zeros(st["rows"].shape, dtype=torch.float64, device=DEV)
        dw = torch.zeros_like(w)
        for j in range(case["k"]):
            d[at[:, j]] = w[:, j:j + 1] * dy
            dw[:, j] = (dy * st["rows"][at[:, j]].double()).sum(1)
        out["d_rows"], out["d_weights"] = d, dw
    return out
