"""Plain 64-bit forms of the paged 8-bit KV cache and of attention over it, on the CPU."""
import math

import torch

BLOCK = 64
F64 = torch.float64


class Cache:
    """Codes and scales [P, Hkv, BLOCK, D] and [P, Hkv] of K and V in their plain order."""

    def __init__(self, P, Hkv, D):
        self.codes = {n: torch.zeros(P, Hkv, BLOCK, D, dtype=torch.int8) for n in "kv"}
        self.scale = {n: torch.full((P, Hkv), math.nan) for n in "kv"}

    def write(self, k, v, seqs, table):
        """k, v [T, Hkv, D] CPU tensors; seqs (first row, pos, tokens)."""
        for row, pos, n in seqs:
            i = seqs.index((row, pos, n))
            at = pos
            while at < pos + n:
                page, off = int(table[i][at // BLOCK]), at % BLOCK
                m = min(BLOCK - off, pos + n - at)
                if 0 <= page < self.scale["k"].shape[0]:
                    for name, x in (("k", k), ("v", v)):
                        self._page(name, page, off, x[row + at - pos: row + at - pos + m].float())
                at += m

    def _page(self, name, page, off, x):
        x = x.transpose(0, 1)  # [Hkv, m, D]
        m = x.shape[1]
        codes, scale = self.codes[name][page], self.scale[name][page]
        # binary32 throughout: torch on the CPU divides as IEEE does
        s = torch.maximum(x.abs().amax((1, 2)) / torch.tensor(127.0), torch.tensor(2.0 ** -64))
        if off:
            s = torch.maximum(s, scale)
            old = codes[:, :off].float() * scale[:, None, None]
            codes[:, :off] = (old / s[:, None, None]).round().clamp(-127, 127).to(torch.int8)
        codes[:, off:off + m] = (x / s[:, None, None]).round().clamp(-127, 127).to(torch.int8)
        self.scale[name][page] = s

    def rows(self, name, i, pos, n, table):
        """Values [n, Hkv, D] in 64 bits of positions pos .. pos + n - 1 of sequence i; None
        in place of those whose page is none."""
        out = []
        for t in range(pos, pos + n):
            page = int(table[i][t // BLOCK])
            if 0 <= page < self.scale["k"].shape[0]:
                out.append(self.codes[name][page, :, t % BLOCK].to(F64) * self.scale[name][page].to(F64)[:, None])
            else:
                out.append(None)
        return out


def attention(cache, q, seqs, table, window, sm_scale):
    """(y, lse, tol, lse_tol) in 64 bits, rows of no sequence NaN.

    tol, for bf16 outputs: half a step of the output, 2^-8 |y|; a weight's rounding to
    float16, 2^-11 of it, and 2^-25 of the largest weight times scale for the smallest ones, against
    codes of up to 127; the relative error of a weight from its score, ln 2 times
    delta, for numerator and denominator, with delta (in powers of two) from the float32 sums of the
    dot product (2^-23 a term), the scales (four roundings), and the hardware's logarithm and
    exponential (2^-22 each, relative to the arguments involved); and float32 sums over the tokens."""
    T, Hq, D = q.shape
    Hkv = cache.scale["k"].shape[1]
    y = torch.full((T, Hq, D), math.nan, dtype=F64)
    lse = torch.full((T, Hq), math.nan, dtype=F64)
    tol, ltol = torch.zeros(T, Hq, D, dtype=F64), torch.zeros(T, Hq, dtype=F64)
    G = Hq // Hkv
    for i, (row, pos, n) in enumerate(seqs):
        if n == 0:
            continue
        total = pos + n
        ks, vs = cache.rows("k", i, 0, total, table), cache.rows("v", i, 0, total, table)
        there = torch.tensor([t is not None for t in ks])
        zero = torch.zeros(Hkv, D, dtype=F64)
        K = torch.stack([zero if t is None else t for t in ks])
        V = torch.stack([zero if t is None else t for t in vs])
        vscale = torch.stack([cache.scale["v"][max(0, min(int(table[i][t // BLOCK]), cache.scale["v"].shape[0] - 1))]
                              for t in range(total)]).to(F64)  # [total, Hkv]
        at = torch.arange(total)
        for j in range(n):
            p = pos + j
            see = there & (at <= p) & ((at > p - window) if window else torch.ones(total, dtype=torch.bool))
            if not see.any():
                y[row + j], lse[row + j] = 0.0, -math.inf
                continue
            for h in range(Hq):
                kh, vh, sv = K[see][:, h // G], V[see][:, h // G], vscale[see][:, h // G]
                qv = q[row + j, h].to(F64)
                s = kh @ qv * sm_scale
                m = s.max()
                w = torch.exp(s - m)
                l = w.sum()
                w = w / l
                y[row + j, h] = w @ vh
                lse[row + j, h] = m + math.log(l)
                size = (kh.abs() @ qv.abs()).max().item() * sm_scale * 1.4427
                big = s.abs().max().item() * 1.4427 + sv.log2().abs().max().item()
                delta = size * 2.0 ** -23 * (D + 4) + big * 2.0 ** -21
                rel = 2 * (math.log(2) * delta + 2.0 ** -22) + 2.0 ** -11 + len(s) * 2.0 ** -24
                tol[row + j, h] = (2.0 ** -8 * y[row + j, h].abs() + rel * (w @ vh.abs())
                                   + len(s) * 2.0 ** -25 * 127 * (w * sv).max())
                ltol[row + j, h] = delta + 2.0 ** -21 * (1 + big) + len(s) * 2.0 ** -24
    return y, lse, tol, ltol
