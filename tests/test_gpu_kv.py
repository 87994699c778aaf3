"""The paged 8-bit KV cache and attention over it, against the plain 64-bit forms."""
import math

import pytest
import torch

import activation_quantized_linear_amd as aql
from kv_reference import BLOCK, Cache, attention

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def gen(seed):
    return torch.Generator().manual_seed(seed)


class Step:
    """Sequences of (past, new) with pages shuffled over a cache, and their K, V and queries."""

    def __init__(self, seqs, Hq, Hkv, D, seed=0, window=0, pad=0, dtype=torch.bfloat16, P=None,
                 pages=None):
        g = gen(seed)
        self.Hq, self.Hkv, self.D, self.window = Hq, Hkv, D, window
        need = [(p + n + BLOCK - 1) // BLOCK for p, n in seqs]
        self.P = P or sum(need) + 2
        order = torch.randperm(self.P, generator=g).tolist() if pages is None else pages
        self.W = max(need + [1]) + 1
        self.table, at = [], 0
        for m in need:
            self.table.append(order[at:at + m] + [2 ** 31 - 1] * (self.W - m))
            at += m
        self.pasts, self.news = [p for p, _ in seqs], [n for _, n in seqs]
        self.cu = [0]
        for n in self.news:
            self.cu.append(self.cu[-1] + n)
        self.T = self.cu[-1] + pad
        self.seqs = [(c, p, n) for c, (p, n) in zip(self.cu, seqs)]

        def draw(T, heads):
            x = torch.randn(T, heads, D, generator=g)
            x[:, :, :max(1, D // 16)] *= 6.0
            x *= torch.exp(0.7 * torch.randn(T, 1, 1, generator=g))  # tokens of very different size
            return x.to(dtype)

        # the tokens before the step, written as one, and those of the step
        self.past = [(0, 0, p) for p in self.pasts]
        c = 0
        for i, p in enumerate(self.pasts):
            self.past[i] = (c, 0, p)
            c += p
        self.pk, self.pv = draw(c, Hkv), draw(c, Hkv)
        self.k, self.v = draw(self.T, Hkv), draw(self.T, Hkv)
        self.q = torch.randn(self.T, Hq, D, generator=g).to(torch.bfloat16)
        self.ref = Cache(self.P, Hkv, D)
        self.cache = aql.aql_kv_cache(self.P, Hkv, D, DEV)
        self.cache.kq.fill_(-128)  # what was there before
        self.cache.vq.fill_(-128)
        self.cache.ks.fill_(math.nan)
        self.cache.vs.fill_(math.nan)
        self.dev_table = i32(self.table)

    def plan(self, **kw):
        return aql.aql_kv_plan(i32(self.cu), i32(self.pasts), self.T, max(self.news + [1]), self.Hq, self.Hkv,
                               self.W, self.window, **kw)

    def write_past(self):
        T = len(self.pk)
        if T:
            cu = [r for r, _, _ in self.past] + [T]
            plan = aql.aql_kv_plan(i32(cu), i32([0] * len(self.past)), T, max(self.pasts), self.Hq, self.Hkv, self.W)
            assert plan.info.item() == 0
            aql.aql_kv_cache_write(self.pk.to(DEV), self.pv.to(DEV), self.cache, self.dev_table, plan)
            self.ref_write(self.pk, self.pv, self.past)

    def ref_write(self, k, v, seqs):
        for i, s in enumerate(seqs):
            self.ref.write(k, v, [s], [self.table[i]])

    def write(self):
        plan = self.plan()
        aql.aql_kv_cache_write(self.k.to(DEV), self.v.to(DEV), self.cache, self.dev_table, plan)
        self.ref_write(self.k, self.v, self.seqs)
        return plan

    def codes(self, name):
        """The cache's codes [P, Hkv, 64, DP] in plain order."""
        if name == "k":
            c = self.cache.kq.transpose(2, 3)
            return c.reshape(self.P, self.Hkv, BLOCK, -1).cpu()
        return self.cache.vq.transpose(2, 3).cpu()

    def check_cache(self):
        for name, scale in (("k", self.cache.ks), ("v", self.cache.vs)):
            codes, want = self.codes(name), self.ref.codes[name]
            for i, (p, n) in enumerate(zip(self.pasts, self.news)):
                for b in range((p + n + BLOCK - 1) // BLOCK):
                    page, live = self.table[i][b], min(BLOCK, p + n - b * BLOCK)
                    if not 0 <= page < self.P:
                        continue
                    assert torch.equal(scale[page].cpu(), self.ref.scale[name][page]), (name, i, b)
                    assert torch.equal(codes[page, :, :live, :self.D], want[page, :, :live]), (name, i, b)
                    assert not codes[page, :, :live, self.D:].any()

    def attend(self, plan, lse=True, **kw):
        y = torch.full((self.T, self.Hq, self.D), 77.0, dtype=torch.bfloat16, device=DEV)
        out = torch.full((self.T, self.Hq), 77.0, device=DEV) if lse else None
        aql.aql_attention_kv8(self.q.to(DEV), self.cache, self.dev_table, plan, y=y, lse=out, **kw)
        return y, out

    def check_attention(self, y, lse, sm_scale=None):
        want, wl, tol, ltol = attention(self.ref, self.q, self.seqs, self.table, self.window,
                                        self.D ** -0.5 if sm_scale is None else sm_scale)
        y, n = y.cpu().double(), self.cu[-1]
        assert (y[n:] == 77).all(), "rows of no sequence were written"
        err = (y[:n] - want[:n]).abs()
        bad = ~(err <= tol[:n])
        assert not bad.any(), (bad.nonzero()[0].tolist(), (err / tol[:n].clamp(min=1e-30)).max().item())
        if lse is not None:
            lse = lse.cpu().double()
            assert (lse[n:] == 77).all()
            none = torch.isinf(wl[:n])
            assert torch.equal(none, torch.isinf(lse[:n]))
            bad = ~(none | ((lse[:n] - wl[:n]).abs() <= ltol[:n]))
            assert not bad.any(), ((lse[:n] - wl[:n]).abs() / ltol[:n])[bad].max().item()


DECODE = [(0, 1), (62, 1), (63, 1), (64, 1), (65, 1), (333, 1), (1000, 1)]
CASES = [
    # seqs, Hq, Hkv, D, window
    (DECODE, 15, 5, 64, 0),
    (DECODE, 8, 2, 128, 0),
    (DECODE, 4, 4, 80, 70),
    (DECODE, 6, 1, 256, 1),
    (DECODE, 3, 1, 192, 64),
    (DECODE, 2, 2, 8, 0),
    ([(500, 1)], 32, 1, 128, 0),           # 32 rows of one kv head
    ([(500, 1), (3, 1)], 40, 1, 64, 0),    # 40
    ([(130, 3), (0, 0), (7, 5), (70, 1)], 8, 2, 128, 0),
    ([(130, 3), (0, 2), (61, 7), (70, 1)], 4, 2, 96, 65),
    ([(0, 130), (63, 66), (200, 1), (1, 64)], 4, 2, 64, 0),
    ([(0, 200), (90, 97)], 6, 3, 128, 0),
    ([(0, 150), (300, 70)], 4, 1, 256, 100),
    ([(0, 97)], 2, 2, 120, 13),
    ([(0, 40)] * 9, 2, 1, 72, 0),
    ([(4000, 1), (1, 1)], 4, 2, 128, 0),   # one long sequence: spread over several units
    ([(2100, 20)], 2, 1, 64, 0),
    ([(1500, 70)], 2, 1, 128, 900),
    ([(0, 150), (100, 33), (5, 1)], 3, 1, 192, 0),
    ([(0, 90), (700, 1), (0, 0), (63, 1), (2000, 64)], 12, 4, 128, 0),   # a chunk among decoding sequences
    ([(0, 260), (40, 100)], 2, 2, 256, 0),
    ([(3000, 300)], 2, 2, 64, 0),
]


@pytest.mark.parametrize("seqs,Hq,Hkv,D,window", CASES)
def test_write_and_attention(seqs, Hq, Hkv, D, window):
    s = Step(seqs, Hq, Hkv, D, seed=Hq * D + window, window=window, pad=3)
    s.write_past()
    plan = s.write()
    assert plan.info.item() == 0
    s.check_cache()
    y, lse = s.attend(plan)
    s.check_attention(y, lse)
