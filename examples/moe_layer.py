"""A mixture-of-experts feed-forward layer on FP4 experts.

    python examples/moe_layer.py [--tokens 4096] [--format nvfp4|mxfp4] [--check]

Per token: route (moe_route) -> rows sorted by expert and quantized
(moe_dispatch) -> gate and up products with the gated activation
(fp4_grouped_gemm_fused) -> quantize -> down product -> weighted sum onto the
residual stream (moe_combine).  Weights are quantized and interleaved once, in
the constructor.  `backward` returns the gradients that flow past the FP4 products
(to the down product's output and input activations, the biases and the router).

--check compares the layer with the same computation in plain float32 torch on
dequantized operands.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import micro_scaled_fp4_amd as fp4  # noqa: E402


class MoELayer:
    def __init__(self, hidden, inner, experts, top_k, fmt=fp4.FP4_NVFP4, groups=1, top_groups=1, seed=0,
                 device="cuda:0"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.fmt, self.hidden, self.inner, self.experts, self.top_k = fmt, hidden, inner, experts, top_k
        self.groups, self.top_groups = groups, top_groups
        self.router = (rand(experts, hidden) * hidden ** -0.5).to(torch.bfloat16)
        self.balance = torch.zeros(experts, device=device)     # moved by the trainer, only selects
        gate_up = fp4.interleave_gate_up(rand(experts, inner, hidden) * 0.02, rand(experts, inner, hidden) * 0.02)
        self.gate_up = self._quantize(gate_up)
        self.down = self._quantize(rand(experts, hidden, inner) * 0.02)
        self.bias = rand(experts, 2 * inner) * 0.01

    def _quantize(self, w):
        """Expert weights [E, N, K]: codes, scale bytes and (NVFP4) one tensor scale per expert."""
        if self.fmt == fp4.FP4_MXFP4:
            parts = [fp4.mxfp4_quantize(e) + (None,) for e in w]
        else:
            parts = [(q, s, g) for q, s, _, g in (fp4.nvfp4_quantize(e) for e in w)]
        scale = None if parts[0][2] is None else torch.cat([p[2] for p in parts])
        return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts]), scale

    def _rows(self, x):
        """Rows quantized as a GEMM operand: codes, scale bytes, tensor scale or None."""
        if self.fmt == fp4.FP4_MXFP4:
            return fp4.mxfp4_quantize(x) + (None,)
        q, s, _, g = fp4.nvfp4_quantize(x)
        return q, s, g

    def forward(self, x, keep=None):
        """x [T, hidden] bf16 -> x + the experts' output.  keep: a dict that receives
        what backward needs."""
        logits = x @ self.router.T
        ids, weights = fp4.moe_route(logits, self.top_k, score=fp4.FP4_SCORE_SIGMOID, bias=self.balance,
                                     num_groups=self.groups, top_groups=self.top_groups,
                                     group_top=2 if self.groups > 1 else 1)
        q, s, _, g, offsets, slot_rows, row_slots = fp4.moe_dispatch(self.fmt, x, ids, self.experts)
        w, sw, gw = self.gate_up
        h = fp4.fp4_grouped_gemm_fused(self.fmt, q, s, g, w, sw, gw, offsets, self.hidden,
                                       activation=fp4.FP4_ACT_SILU, gated=True, bias=self.bias,
                                       preact_dtype=None if keep is None else torch.bfloat16)
        if keep is not None:
            h, z = h
            keep.update(logits=logits, ids=ids, weights=weights, offsets=offsets, slot_rows=slot_rows,
                        row_slots=row_slots, z=z)
        hq, hs, hg = self._rows(h)
        w, sw, gw = self.down
        out = fp4.fp4_grouped_gemm_fused(self.fmt, hq, hs, hg, w, sw, gw, offsets, self.inner)
        if keep is not None:
            keep["rows"] = out
        return fp4.moe_combine(out, weights, slot_rows, residual=x)

    def backward(self, dy, keep, d_hidden):
        """From dy [T, hidden]: the gradients of the expert outputs and of the router's
        logits; from d_hidden [rows, inner], the gradient of the gated activation's
        output, those of its pre-activations and of the biases."""
        d_rows, d_weights = fp4.moe_combine_backward(dy, keep["rows"], keep["weights"], keep["slot_rows"],
                                                     keep["row_slots"])
        d_logits = fp4.moe_route_backward(d_weights, keep["logits"], keep["ids"], score=fp4.FP4_SCORE_SIGMOID)
        dz, d_bias = fp4.fp4_epilogue_backward(d_hidden, keep["z"], fp4.FP4_ACT_SILU, gated=True,
                                               offsets=keep["offsets"])
        return {"rows": d_rows, "logits": d_logits, "z": dz, "bias": d_bias}

    # ---- the same in plain torch, for --check ----
    def _dequantize(self, w, K):
        q, s, g = w
        return torch.stack([fp4.fp4_dequantize(self.fmt, q[e], s[e], None if g is None else g[e:e + 1], K)
                            for e in range(self.experts)])

    def plain_forward(self, x):
        logits = (x @ self.router.T).float()
        score = torch.sigmoid(logits)
        v = score + self.balance
        if self.groups > 1:
            per = v.view(-1, self.groups, self.experts // self.groups)
            best = per.topk(2, dim=2).values.sum(2).topk(self.top_groups, dim=1).indices
            mask = torch.zeros(per.shape[:2], dtype=torch.bool, device=x.device).scatter_(1, best, True)
            v = torch.where(mask[..., None].expand_as(per).reshape(v.shape), v, float("-inf"))
        ids = v.topk(self.top_k, dim=1).indices
        weights = score.gather(1, ids)
        weights = weights / weights.sum(1, keepdim=True)
        q, s, g = self._rows(x)
        xq = fp4.fp4_dequantize(self.fmt, q, s, g, self.hidden)
        gate_up, down = self._dequantize(self.gate_up, self.hidden), self._dequantize(self.down, self.inner)
        T, k = ids.shape
        h = torch.zeros(T, k, self.inner, device=x.device)
        for e in range(self.experts):
            t, j = (ids == e).nonzero(as_tuple=True)
            z = xq[t] @ gate_up[e].T + self.bias[e]
            h[t, j] = torch.nn.functional.silu(z[:, 0::2]) * z[:, 1::2]
        q, s, g = self._rows(h.to(torch.bfloat16).view(T * k, self.inner))
        hq = fp4.fp4_dequantize(self.fmt, q, s, g, self.inner).view(T, k, self.inner)
        y = x.float()
        for e in range(self.experts):
            t, j = (ids == e).nonzero(as_tuple=True)
            y.index_add_(0, t, weights[t, j, None] * (hq[t, j] @ down[e].T).to(torch.bfloat16).float())
        return y


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--inner", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--top-k", type=int, default=8)
    ap.add_argument("--groups", type=int, default=8)
    ap.add_argument("--top-groups", type=int, default=4)
    ap.add_argument("--format", choices=["nvfp4", "mxfp4"], default="nvfp4")
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args()
    fmt = fp4.FP4_NVFP4 if a.format == "nvfp4" else fp4.FP4_MXFP4
    layer = MoELayer(a.hidden, a.inner, a.experts, a.top_k, fmt, a.groups, a.top_groups)
    x = torch.randn(a.tokens, a.hidden, device="cuda:0").to(torch.bfloat16)
    y = layer.forward(x)
    if a.check:
        want = layer.plain_forward(x)
        err = float((y.float() - want).norm() / (want - x.float()).norm())
        print(f"relative difference from plain torch: {err:.2e}")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(10):
        layer.forward(x)
    end.record()
    torch.cuda.synchronize()
    print(f"{a.tokens} tokens, {a.experts} experts, top {a.top_k}: {start.elapsed_time(end) * 100:.1f} us per forward")
    keep = {}
    layer.forward(x, keep)
    dy = torch.randn_like(x)
    grads = layer.backward(dy, keep, torch.randn(keep["z"].shape[0], a.inner, device=x.device).to(torch.bfloat16))
    print("gradients:", ", ".join(f"{n} {tuple(t.shape)}" for n, t in grads.items()))


if __name__ == "__main__":
    main()
