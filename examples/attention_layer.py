"""An attention layer on FP4 projections and a paged FP4 key/value cache.

    python examples/attention_layer.py [--format nvfp4|mxfp4] [--tokens 200] [--steps 8] [--check]

Per call: one FP4 product for queries, keys and values (fp4_scaled_gemm) -> keys and values into
their pages (kv_cache_write, read in place out of the product's rows) -> attention over the cache
(kv_cache_attention) -> output projection onto the residual stream (fp4_scaled_gemm_fused).  A
prompt and a single token take the same calls; the decoding step is captured in a graph once and
replayed with other tokens and lengths.

--check compares every call with plain float64 torch on the dequantized weights and cache.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import micro_scaled_fp4_amd as fp4  # noqa: E402


class AttentionLayer:
    def __init__(self, hidden, q_heads, kv_heads, head_dim, seqs, max_len, fmt=fp4.FP4_NVFP4, page=16, seed=0,
                 device="cuda:0"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.fmt, self.hidden, self.q_heads, self.kv_heads, self.dim = fmt, hidden, q_heads, kv_heads, head_dim
        self.wqkv = self._quantize(rand((q_heads + 2 * kv_heads) * head_dim, hidden) * hidden ** -0.5)
        self.wo = self._quantize(rand(hidden, q_heads * head_dim) * (q_heads * head_dim) ** -0.5)
        wide = -(-max_len // page)
        nv = fmt == fp4.FP4_NVFP4
        # amax of keys and values: calibrated in earnest, here a bound for unit inputs
        self.cache = fp4.KVCache.empty(fmt, seqs * wide, kv_heads, page, head_dim, 6.0 if nv else None,
                                       6.0 if nv else None, device)
        self.pages = torch.randperm(seqs * wide, generator=g, device=device).reshape(seqs, wide).to(torch.int32)

    def _quantize(self, x):
        """Codes, scale bytes, tensor scale or None."""
        if self.fmt == fp4.FP4_MXFP4:
            return fp4.mxfp4_quantize(x) + (None,)
        q, s, _, g = fp4.nvfp4_quantize(x)
        return q, s, g

    def forward(self, x, offsets, lengths, keep=None):
        """x [T, hidden] bf16: rows offsets[b] .. offsets[b + 1] are sequence b's last ones of lengths[b]."""
        qkv = fp4.fp4_scaled_gemm(self.fmt, *self._quantize(x), *self.wqkv, self.hidden)
        qkv = qkv.view(x.shape[0], self.q_heads + 2 * self.kv_heads, self.dim)
        q, k, v = qkv.split([self.q_heads, self.kv_heads, self.kv_heads], dim=1)
        where = (offsets, lengths, self.pages)
        fp4.kv_cache_write(self.cache, k, v, *where)
        attended = fp4.kv_cache_attention(self.cache, q, *where)
        rows = self._quantize(attended.view(x.shape[0], -1))
        y = fp4.fp4_scaled_gemm_fused(self.fmt, *rows, *self.wo, self.q_heads * self.dim, residual=x)
        if keep is not None:
            keep.update(q=q, attended=attended)
        return y

    def plain_attention(self, q, offsets, lengths):
        """What kv_cache_attention gives, in float64 on the cache's values."""
        offs, lens = offsets.tolist(), lengths.tolist()
        starts = torch.zeros_like(lengths)
        every = torch.tensor([0] + lens, device=q.device).cumsum(0).to(torch.int32)
        k, v = fp4.kv_cache_read(self.cache, every, lengths, self.pages, int(every[-1]), starts=starts,
                                 out_dtype=torch.float32)
        out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
        for b, length in enumerate(lens):
            n, at = offs[b + 1] - offs[b], int(every[b])
            kb, vb = (t[at:at + length].double().repeat_interleave(self.q_heads // self.kv_heads, 1).transpose(0, 1).contiguous()
                      for t in (k, v))
            s = q[offs[b]:offs[b + 1]].double().transpose(0, 1).contiguous() @ kb.transpose(1, 2).contiguous() * self.dim ** -0.5
            late = torch.arange(length, device=q.device) > torch.arange(length - n, length, device=q.device)[:, None]
            out[offs[b]:offs[b + 1]] = (torch.softmax(s.masked_fill(late, -torch.inf), -1) @ vb).transpose(0, 1)
        return out


def difference(layer, keep, offsets, lengths):
    want = layer.plain_attention(keep["q"], offsets, lengths)
    return float((keep["attended"].double() - want).norm() / want.norm())


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--format", choices=("nvfp4", "mxfp4"), default="nvfp4")
    ap.add_argument("--tokens", type=int, default=200)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    dev, seqs = "cuda:0", 4
    fmt = fp4.FP4_NVFP4 if a.format == "nvfp4" else fp4.FP4_MXFP4
    layer = AttentionLayer(1024, 16, 4, 128, seqs, a.tokens + a.steps, fmt)
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device=dev)  # noqa: E731
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    # prompts of different lengths, then one token of each sequence a step
    lens = [max(1, a.tokens - 13 * b) for b in range(seqs)]
    offsets, lengths, keep, off = i32([0] + lens).cumsum(0).to(torch.int32), i32(lens), {}, []
    layer.forward(torch.randn(sum(lens), 1024, generator=g, device=dev).to(torch.bfloat16), offsets, lengths, keep)
    if a.check:
        off.append(difference(layer, keep, offsets, lengths))
    x = torch.randn(seqs, 1024, generator=g, device=dev).to(torch.bfloat16)
    one = torch.arange(seqs + 1, dtype=torch.int32, device=dev)
    lengths += 1
    layer.forward(x, one, lengths, keep)        # first calls outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.forward(x, one, lengths, keep)
    for _ in range(a.steps - 1):
        x.copy_(torch.randn(seqs, 1024, generator=g, device=dev))
        lengths += 1
        graph.replay()
        if a.check:
            off.append(difference(layer, keep, one, lengths))
    torch.cuda.synchronize()
    print(f"{a.format}: {sum(lens)} prompt tokens, {a.steps} steps of {seqs}; |y| {float(y.float().norm()):.3f}")
    if a.check:
        print("relative differences of attention from float64:", " ".join(f"{d:.1e}" for d in off))
    return off


if __name__ == "__main__":
    main()
