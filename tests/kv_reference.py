"""Plain 64-bit reference of the paged FP4 cache and of attention over it, for the tests.

A case is a set of sequences (length, rows) with shuffled pages.  The cache's bytes come from
the CPU oracle's quantizers; every byte that no position was written to is 0xff (a NaN scale in
both formats), so a kernel that uses one shows it."""
import numpy as np

from oracle import fp4_oracle as o

NV, MX = 0, 1


def block(fmt):
    return 16 if fmt == NV else 32


class Case:
    def __init__(self, fmt, H, D, page, seqs, seed, k_std=1.0, v_std=1.0, spare_pages=3, spare_rows=0, wide=0):
        """seqs: (length, rows) of each sequence; spare_rows: rows behind the last sequence."""
        rng = np.random.default_rng(seed)
        self.rng, self.fmt, self.H, self.D, self.page = rng, fmt, H, D, page
        self.lengths = np.array([s[0] for s in seqs], np.int32)
        self.rows = [s[1] for s in seqs]
        self.B = len(seqs)
        self.offsets = np.concatenate([[0], np.cumsum(self.rows)]).astype(np.int32)
        self.T = int(self.offsets[-1]) + spare_rows
        need = [-(-int(length) // page) for length in self.lengths]
        self.max_pages = max(1, wide, *need) if self.B else 1
        self.num_pages = sum(need) + spare_pages
        ids = rng.permutation(self.num_pages).astype(np.int32)
        # entries past a sequence's length: other sequences' pages and holes
        self.pages = rng.integers(-2, self.num_pages + 2, (self.B, self.max_pages)).astype(np.int32)
        at = 0
        for b, n in enumerate(need):
            self.pages[b, :n] = ids[at:at + n]
            at += n
        # all positions' keys and values, [length, H, D] per sequence, bf16 values
        def draw(std):
            return [o.bf16_bits_to_f32(o.f32_to_bf16_bits((rng.standard_normal((int(n), H, D)) * std).astype(np.float32)))
                    for n in self.lengths]
        self.k, self.v = draw(k_std), draw(v_std)
        self.k_amax = np.float32(max([1e-3] + [float(np.abs(x).max()) for x in self.k if x.size]) * 0.9)
        self.v_amax = np.float32(max([1e-3] + [float(np.abs(x).max()) for x in self.v if x.size]) * 0.9)

    # ---- bytes ----
    def empty_store(self, fill=0xff):
        bs = block(self.fmt)
        return [np.full((self.num_pages, self.H, self.page, w), fill, np.uint8)
                for w in (self.D // 2, self.D // bs, self.D // 2, self.D // bs)]

    def quantize(self, x, amax):
        """[n, H, D] -> (codes [n, H, D/2], scale bytes [n, H, D/bs])."""
        n = x.shape[0]
        flat = np.ascontiguousarray(x, np.float32).reshape(n * self.H, self.D)
        if n == 0:
            return np.zeros((0, self.H, self.D // 2), np.uint8), np.zeros((0, self.H, self.D // block(self.fmt)), np.uint8)
        q, s = (o.nvfp4_quantize(flat, amax=amax)[:2] if self.fmt == NV else o.mxfp4_quantize(flat)[:2])
        return q.reshape(n, self.H, -1), s.reshape(n, self.H, -1)

    def put(self, store, b, positions, k, v):
        """Writes rows k, v [n, H, D] to positions of sequence b (skipping holes and negative ones)."""
        for x, amax, at in ((k, self.k_amax, 0), (v, self.v_amax, 2)):
            q, s = self.quantize(x, amax)
            for i, t in enumerate(positions):
                if t < 0:
                    continue
                p = self.pages[b, t // self.page]
                if 0 <= p < self.num_pages:
                    store[at][p, :, t % self.page] = q[i]
                    store[at + 1][p, :, t % self.page] = s[i]

    def full_store(self):
        store = self.empty_store()
        for b in range(self.B):
            self.put(store, b, range(int(self.lengths[b])), self.k[b], self.v[b])
        return store

    # ---- values ----
    def held(self, store, b, which):
        """(values [length, H, D] float64, in_hole [length]) of sequence b; which: 0 keys, 1 values."""
        n = int(self.lengths[b])
        out, hole = np.zeros((n, self.H, self.D)), np.zeros(n, bool)
        for t in range(n):
            p = self.pages[b, t // self.page]
            if not 0 <= p < self.num_pages:
                hole[t] = True
                continue
            out[t] = self.values(store[2 * which][p, :, t % self.page], store[2 * which + 1][p, :, t % self.page], which)
        return out, hole

    def values(self, codes, scales, which, f32=False):
        amax = (self.k_amax, self.v_amax)[which]
        if self.fmt == NV:
            g = o.nv_global_scale(amax)
            return (o.nvfp4_dequantize(codes, scales, g, self.D) if f32 else
                    o.nv_operand_f64(codes, scales, 1.0, self.D) * (float(amax) / 2688.0))
        return o.mxfp4_dequantize(codes, scales, self.D) if f32 else o.mx_operand_f64(codes, scales, self.D)

    def amaxes(self):
        return (float(self.k_amax), float(self.v_amax)) if self.fmt == NV else (None, None)


def attention(case, store, q, scale, causal=True, window=0, f32=False):
    """(out [T, Hq, D], lse [T, Hq], tolerance of out, tolerance of lse) in float64 for q [T, Hq, D]
    (values as given, exact); rows behind the last sequence are NaN.

    Tolerances, per row and head, before the output's own rounding.  A = max over the seen t of
    scale * sum |q k| bounds the scores.  Float32 accumulation of D products and the scaling:
    (D + 16) 2^-24 A per score; in a weight p = exp(s - m) / l both s and m carry it, and l once
    more: 4 times.  exp and log: 2^-21 of their result (a float32 exponent argument of up to 2 A
    included: 2 A 2^-24).  Sums over L weights, joined in parts: (L + 64) 2^-24.  Weights as fp16
    2^-11 (half a step 2^-12, and the same for l's), or, from float32 operands, in two fp16 parts:
    2^-21, and q in two fp16 parts: 2^-22 A per score.  All of them multiply sum p |v|.  Weights
    are stored as P = 2^11 w 2^d at the least, w relative to the largest and d >= 0: where P is below
    2^-14 fp16's steps are 2^-24 and half a step 2^-25 is 2^-36 of the largest weight, so 2^-36 of
    the largest |v| per position."""
    T, Hq, D = q.shape
    G = Hq // case.H
    out, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    tol, ltol = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for b in range(case.B):
        (k, hole), (v, _) = case.held(store, b, 0), case.held(store, b, 1)
        L, lo, hi = int(case.lengths[b]), int(case.offsets[b]), int(case.offsets[b + 1])
        t = np.arange(L)
        for r in range(lo, hi):
            p = L - (hi - r)
            seen = ~hole
            if causal:
                seen = seen & (t <= p)
            if window:
                seen = seen & (t > p - window)
            n = int(seen.sum())
            if n == 0:
                out[r], lse[r] = 0.0, -np.inf
                continue
            for h in range(Hq):
                kh, vh = k[seen, h // G], v[seen, h // G]
                s = scale * (kh @ q[r, h])
                A = abs(scale) * float((np.abs(kh) @ np.abs(q[r, h])).max())
                m = s.max()
                e = np.exp(s - m)
                w = e / e.sum()
                out[r, h], lse[r, h] = w @ vh, m + np.log(e.sum())
                rel = (4 * (D + 16) + 4) * 2.0 ** -24 * A + 2.0 ** -20 + 2 * (n + 64) * 2.0 ** -24
                if f32:
                    rel += 2.0 ** -21 + 4 * 2.0 ** -22 * A
                else:
                    rel += 2.0 ** -11
                tol[r, h] = rel * (w @ np.abs(vh)) + n * 2.0 ** -36 * np.abs(vh).max()
                ltol[r, h] = (2 * (D + 16) * 2.0 ** -24 + (2.0 ** -22 if f32 else 0)) * A + 2.0 ** -20 + \
                    (n + 64) * 2.0 ** -24 + 2.0 ** -22 * abs(lse[r, h])
    return out, lse, tol, ltol
