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
    ([(0, 150), (700, 1)], 2, 1, 200, 80),
    ([(400, 30), (10, 2)], 2, 1, 256, 0),  # 60 rows of a wide head
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


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("new", [6, 12, 25, 70])  # 12, 24, 50 and 140 rows
@pytest.mark.parametrize("window", [0, 1200])
def test_divided_units(D, new, window):
    """Long sequences whose blocks are divided over units, of every number of rows and head size."""
    s = Step([(1900, new), (900, max(1, new // 3)), (0, 2)], 4, 2, D, seed=D + new, window=window, pad=1)
    s.write_past()
    plan = s.write()
    y, lse = s.attend(plan)
    s.check_attention(y, lse)


@pytest.mark.parametrize("D", [64, 128, 184, 256])
@pytest.mark.parametrize("Hq,Hkv,window", [(4, 2, 0), (16, 1, 0), (3, 3, 500)])
def test_few_rows_among_many(D, Hq, Hkv, window):
    """Decoding sequences, divided and whole, beside a prefill and a short chunk."""
    s = Step([(3000, 1), (0, 200), (700, 1), (130, 1), (63, 3), (0, 1), (1000, 17)], Hq, Hkv, D, seed=D + Hq,
             window=window, pad=2)
    s.write_past()
    plan = s.write()
    y, lse = s.attend(plan)
    s.check_attention(y, lse)


@pytest.mark.parametrize("Hq,D", [(129, 64), (200, 128), (1024, 8)])
@pytest.mark.parametrize("window", [0, 100])
def test_many_heads_of_one_kv_head(Hq, D, window):
    """A token's heads fill more than one unit."""
    s = Step([(700, 1), (63, 2), (0, 1)], Hq, 1, D, seed=Hq, window=window)
    s.write_past()
    plan = s.write()
    y, lse = s.attend(plan)
    s.check_attention(y, lse)


def test_scale_of_softmax_and_no_lse():
    s = Step([(70, 3), (0, 70), (200, 1)], 4, 2, 64, seed=3)
    s.write_past()
    plan = s.write()
    y, _ = s.attend(plan, lse=False, sm_scale=0.05)
    s.check_attention(y, None, sm_scale=0.05)


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 64), (3, 1, 72)])
def test_token_by_token(Hq, Hkv, D):
    """A sequence grows a token a step over page ends, its pages' scales with it, is taken
    back and grows again; every step's cache and attention against the plain form."""
    past = 61
    g = gen(17)
    s = Step([(past, 1)], Hq, Hkv, D, seed=17, P=6, pages=[4, 1, 3, 0, 2, 5])
    s.W = 3
    s.table = [[4, 1, 3]]
    s.dev_table = i32(s.table)
    s.write_past()
    positions = [61, 62, 63, 64, 65, 66, 62, 63, 64, 65, 126, 127, 128]
    at = 61
    for step, p in enumerate(positions):
        n = max(1, p - at + 1) if p > at else 1  # (a jump writes several tokens)
        pos = p - n + 1
        size = 10.0 ** torch.empty(1).uniform_(-1, 1, generator=g).item()  # some raise the scale, some do not
        k, v = [(torch.randn(n, Hkv, D, generator=g) * size).to(torch.bfloat16) for _ in range(2)]
        s.k, s.v, s.T, s.news, s.pasts = k, v, n, [n], [pos]
        s.q = torch.randn(n, Hq, D, generator=g).to(torch.bfloat16)
        s.cu, s.seqs = [0, n], [(0, pos, n)]
        plan = s.write()
        s.check_cache()
        y, lse = s.attend(plan)
        s.check_attention(y, lse)
        at = p + 1


@pytest.mark.parametrize("D", [64, 128, 200])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_read_back(D, dtype):
    """float32 K and V too; rows of any range, rounded once; rows of no sequence stay."""
    s = Step([(130, 5), (0, 64), (63, 2), (0, 0)], 2, 2, D, seed=D, pad=2, dtype=torch.float32)
    s.write_past()
    s.write()
    s.check_cache()
    ranges = [(100, 35), (1, 60), (60, 5), (0, 0)]
    cu = [0]
    for _, n in ranges:
        cu.append(cu[-1] + n)
    T = cu[-1] + 3
    plan = aql.aql_kv_plan(i32(cu), i32([p for p, _ in ranges]), T, 40 + 20, s.Hq, s.Hkv, s.W)
    k, v = [torch.full((T, s.Hkv, D), 5.0, dtype=dtype, device=DEV) for _ in range(2)]
    aql.aql_kv_cache_read(s.cache, s.dev_table, plan, dtype, k=k, v=v)
    for name, x in (("k", k), ("v", v)):
        want = []
        for i, (p, n) in enumerate(ranges):
            for t in range(p, p + n):
                page = s.table[i][t // BLOCK]
                want.append(s.ref.codes[name][page, :, t % BLOCK].float() * s.ref.scale[name][page][:, None])
        want = torch.stack(want).to(dtype)
        assert torch.equal(x[:cu[-1]].cpu(), want)
        assert (x[cu[-1]:] == 5).all()


def test_slices_of_one_projection():
    """q, k and v as slices of one tensor; the same bits as from copies."""
    s = Step([(70, 40), (5, 1), (0, 130)], 6, 2, 64, seed=5)
    s.write_past()
    plan = s.plan()
    qkv = torch.cat([s.q.flatten(1), s.k.flatten(1), s.v.flatten(1)], 1).to(DEV)
    q, k, v = qkv[:, :384].unflatten(1, (6, 64)), qkv[:, 384:512].unflatten(1, (2, 64)), qkv[:, 512:].unflatten(1, (2, 64))
    assert not (q.is_contiguous() or k.is_contiguous() or v.is_contiguous())
    aql.aql_kv_cache_write(k, v, s.cache, s.dev_table, plan)
    s.ref_write(s.k, s.v, s.seqs)
    s.check_cache()
    y = aql.aql_attention_kv8(q, s.cache, s.dev_table, plan)
    s.check_attention(y, None)
    with pytest.raises(ValueError):  # heads apart
        aql.aql_attention_kv8(torch.empty(s.T, 64, 6, dtype=torch.bfloat16, device=DEV).transpose(1, 2), s.cache,
                              s.dev_table, plan)
    with pytest.raises(ValueError):
        aql.aql_attention_kv8(q[:-1], s.cache, s.dev_table, plan)
    with pytest.raises(TypeError):
        aql.aql_kv_cache_write(k, v.float(), s.cache, s.dev_table, plan)
    with pytest.raises(aql.AqlError):  # rows that overlap
        aql.aql_kv_cache_write(k[:1].expand(s.T, 2, 64), v, s.cache, s.dev_table, plan)
    with pytest.raises(aql.AqlError):
        aql.aql_attention_kv8(q, s.cache, s.dev_table, plan, sm_scale=-1.0)


@pytest.mark.parametrize("seqs", [[(300, 1), (64, 1), (10, 1)], [(300, 100), (64, 70), (10, 1)]])
def test_page_numbers_that_are_none(seqs):
    """Not written, read back as zeros, not seen; a row that sees nothing gets zeros."""
    s = Step(seqs, 4, 2, 64, seed=9)
    s.table[0][1] = -1
    s.table[0][(seqs[0][0]) // BLOCK] = s.P       # where the first sequence's new tokens begin
    s.table[1] = [-7] * len(s.table[1])           # a sequence without any page
    s.dev_table = i32(s.table)
    s.write_past()
    plan = s.write()
    s.check_cache()
    y, lse = s.attend(plan)
    s.check_attention(y, lse)
    row, _, n = s.seqs[1]
    assert (y[row:row + n] == 0).all() and torch.isinf(lse[row:row + n]).all()
    k, v = aql.aql_kv_cache_read(s.cache, s.dev_table, plan)
    assert not k[row:row + n].any() and not v[row:row + n].any()


@pytest.mark.parametrize("seqs", [[(100, 1), (30, 1)], [(0, 200), (30, 1)], [(100, 40), (30, 1)]])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_pages_without_finite_values(seqs, bad):
    """Tokens of another page, rows that see none of its tokens and other sequences keep their
    values; rows that see the page get none."""
    s = Step(seqs, 4, 2, 64, seed=11)
    s.write_past()
    (_, past, n), total = s.seqs[0], sum(seqs[0])
    t = total - 1                                 # the last token, in the last page
    s.k[n - 1, 1, 3] = bad
    s.v[n - 1, 1, 5] = bad
    plan = s.write()
    y, lse = s.attend(plan)
    y, lse = y.cpu(), lse.cpu()
    first = t // BLOCK * BLOCK                    # rows from here on see a token of that page
    # heads of kv head 0, rows before the page and other sequences: as without the bad values
    for name in "kv":
        page = s.table[0][t // BLOCK]
        s.ref.scale[name][page, 1] = 1.0
        s.ref.codes[name][page, 1] = 0
    want, wl, tol, ltol = attention(s.ref, s.q, s.seqs, s.table, 0, 64 ** -0.5)
    row = torch.arange(len(y))
    own = row < n
    sees = own & (past + row >= first)
    ok = torch.ones(len(y), 4, dtype=torch.bool)
    ok[sees, 2:] = False
    err = (y.double() - want).abs()
    assert (err <= tol)[ok].all() and ((lse.double() - wl).abs() <= ltol)[ok].all()
    assert not torch.isfinite(y[sees][:, 2:]).any()
    k, v = aql.aql_kv_cache_read(s.cache, s.dev_table, plan, torch.float32)
    lo = max(0, first - past)
    assert not torch.isfinite(k[lo:n, 1]).any() and not torch.isfinite(v[lo:n, 1]).any()
    assert torch.isfinite(k[:lo]).all() and torch.isfinite(k[n:]).all() and torch.isfinite(k[:, 0]).all()


def test_sequences_that_cannot_be_served():
    """Each is left out, its rows stay, the plan says which; the others are served."""
    def plan_of(cu, pos, most, W=4, T=12):
        return aql.aql_kv_plan(i32(cu), i32(pos), T, most, 4, 2, W)

    assert plan_of([0, 2, 5, 12], [0, 3, 9], 7).info.item() == 0
    assert plan_of([0, 2, 5, 12], [0, 3, 9], 6).info.item() == 3      # more than `most`
    assert plan_of([0, 2, 1, 12], [0, 3, 9], 12).info.item() == 2     # not ascending
    assert plan_of([0, 2, 5, 13], [0, 3, 9], 12).info.item() == 3     # past T
    assert plan_of([-1, 2, 5, 12], [0, 3, 9], 12).info.item() == 1
    assert plan_of([0, 2, 5, 12], [0, -1, 9], 12).info.item() == 2
    assert plan_of([0, 2, 5, 12], [0, 254, 9], 12).info.item() == 2   # past the table
    assert plan_of([0, 2, 5, 12], [0, 253, 9], 12).info.item() == 0
    assert plan_of([0, 2, 2, 12], [0, 1 << 30, 9], 12).info.item() == 0   # no tokens: wherever it is
    # overlapping to more rows than the step has
    big = aql.aql_kv_plan(i32([0, 600, 0, 600, 0, 600, 0, 600]), i32([0] * 7), 600, 600, 4, 2, 16)
    assert big.info.item() in (2, 8)
    s = Step([(70, 3), (20, 2), (0, 90)], 4, 2, 64, seed=13)
    s.write_past()
    s.ref_write(s.k, s.v, [s.seqs[0], (0, 0, 0), s.seqs[2]])
    plan = aql.aql_kv_plan(i32(s.cu), i32([70, -20, 0]), s.T, 90, 4, 2, s.W)
    assert plan.info.item() == 2
    aql.aql_kv_cache_write(s.k.to(DEV), s.v.to(DEV), s.cache, s.dev_table, plan)
    y, lse = s.attend(plan)
    assert (y[3:5] == 77).all() and (lse[3:5] == 77).all()
    want, _, tol, _ = attention(s.ref, s.q, [s.seqs[0], (3, 20, 0), s.seqs[2]], s.table, 0, 64 ** -0.5)
    keep = torch.ones(s.T, dtype=torch.bool)
    keep[3:5] = False
    assert ((y.cpu().double() - want).abs() <= tol)[keep].all()


def test_many_sequences():
    """More sequences, pieces and tiles than the plan's workgroup has threads."""
    g = gen(23)
    seqs = [(int(torch.randint(0, 90, (1,), generator=g)), int(torch.randint(0, 3, (1,), generator=g)))
            for _ in range(2300)]
    s = Step(seqs, 2, 1, 8, seed=23)
    s.write_past()
    plan = s.write()
    assert plan.info.item() == 0
    s.check_cache()
    y, lse = s.attend(plan)
    pick = [i for i in range(0, 2300, 19)]
    want, wl, tol, ltol = attention(s.ref, s.q, [s.seqs[i] if i in set(pick) else (0, 0, 0) for i in range(2300)],
                                    s.table, 0, 8 ** -0.5)
    keep = ~torch.isnan(want[:, 0, 0])
    assert keep.sum() > 50
    assert ((y.cpu().double() - want).abs() <= tol)[keep].all()
    assert ((lse.cpu().double() - wl).abs() <= ltol)[keep].all()


@pytest.mark.parametrize("new", [1, 40])
def test_offsets_past_32_bits(new):
    """Pages that lie more than 2^32 bytes into the cache."""
    P = 36000  # 131072 bytes a page and array
    pages = [P - 1, 3, P - 2, P - 700, 0, 33000]
    s = Step([(200, new), (100, 1)], 8, 8, 256, seed=29, P=6, pages=[5, 0, 4, 3, 1, 2])
    cache = aql.aql_kv_cache(P, 8, 256, DEV)
    assert cache.kq.numel() > 2 ** 32
    remap = dict(zip([5, 0, 4, 3, 1, 2], pages))
    s.cache, s.table = cache, [[remap.get(p, p) for p in r] for r in s.table]
    s.dev_table = i32(s.table)
    s.P = P
    s.ref = Cache(6, 8, 256)  # (under the pages' small numbers)
    back = {v: k for k, v in remap.items()}
    s.table = [[back.get(p, p) for p in r] for r in s.table]
    s.write_past()
    plan = s.write()
    y, lse = s.attend(plan)
    s.P = 6
    s.check_attention(y, lse)


def test_very_different_scales():
    """Pages of V (and K) from 1e-18 to 1e18, rows of q from 1e-30 up: weights are taken relative
    to the page that counts most, so none overflows or is lost."""
    for new in (1, 70):
        s = Step([(400, new)], 4, 2, 64, seed=31)
        f = 10.0 ** torch.linspace(-18, 18, 7)
        at = torch.arange(len(s.pk)) // BLOCK
        s.pv = (s.pv.float() * f[at][:, None, None]).to(torch.bfloat16)
        s.pk = (s.pk.float() * 10.0 ** (at % 3 - 3)[:, None, None]).to(torch.bfloat16)
        s.q = (s.q.float() * 10.0 ** (torch.arange(4) * 10 - 30)[None, :, None]).to(torch.bfloat16)
        s.write_past()
        plan = s.write()
        s.check_cache()
        y, lse = s.attend(plan)
        s.check_attention(y, lse)


def test_same_bits_every_time():
    """Atomics in the plan order the work, not any sum."""
    for seqs in ([(3000, 1), (700, 1), (900, 1)], [(1000, 300), (700, 1), (900, 20)]):
        s = Step(seqs, 4, 2, 128, seed=37)
        s.write_past()
        first = None
        for _ in range(4):
            plan = s.write()
            ws = torch.empty(aql.aql_attention_kv8_bytes(s.T, len(seqs), 4, 2, 128, s.W, max(s.news)), dtype=torch.uint8,
                             device=DEV).fill_(255)
            y, lse = s.attend(plan, workspace=ws)
            if first is None:
                first = (y, lse, s.cache.kq.clone(), s.cache.vq.clone())
            assert torch.equal(y, first[0]) and torch.equal(lse, first[1])
            assert torch.equal(s.cache.kq, first[2]) and torch.equal(s.cache.vq, first[3])
    with pytest.raises(aql.AqlError):
        s.attend(plan, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


def test_two_streams_and_other_sizes():
    """Two batches on two streams at once, each with its own plan, cache and workspace."""
    a = Step([(900, 1)] * 3, 8, 2, 64, seed=41)
    b = Step([(0, 300), (50, 1)], 4, 4, 128, seed=43)
    for s in (a, b):
        s.write_past()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(3):
        for s, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                outs.append(s.attend(s.write()))
    torch.cuda.synchronize()
    for (y, lse), s in zip(outs, (a, b) * 3):
        s.check_attention(y, lse)


def test_captured_decode_step():
    """Plan, write and attention in one captured graph: the positions move on the device, and
    every replay serves the next token, eager work and other steps going on between."""
    Hq, Hkv, D, steps = 6, 2, 64, 5
    s = Step([(126, 1), (30, 1), (700, 1)], Hq, Hkv, D, seed=47)
    s.write_past()
    S, g = 3, gen(53)
    W = s.W
    free = [p for p in range(s.P) if all(p not in r for r in s.table)]
    s.table[0][2] = free[0]  # the first sequence begins a page on the way
    s.dev_table = i32(s.table)
    pos, cu = i32(s.pasts), i32(s.cu)
    q, k, v = [torch.empty(S, h, D, dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hkv)]
    y = torch.empty(S, Hq, D, dtype=torch.bfloat16, device=DEV)
    plan = aql.aql_kv_plan(cu, pos, S, 1, Hq, Hkv, W)
    ws = torch.empty(max(1, aql.aql_attention_kv8_bytes(S, S, Hq, Hkv, D, W, 1)), dtype=torch.uint8, device=DEV)

    def step():
        aql.aql_kv_plan(cu, pos, S, 1, Hq, Hkv, W, plan=plan)
        aql.aql_kv_cache_write(k, v, s.cache, s.dev_table, plan)
        aql.aql_attention_kv8(q, s.cache, s.dev_table, plan, y=y, workspace=ws)
        pos.add_(1)

    keep = [t.clone() for t in (s.cache.kq, s.cache.vq, s.cache.ks, s.cache.vs)]
    k.zero_(), v.zero_(), q.zero_()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, o in zip((s.cache.kq, s.cache.vq, s.cache.ks, s.cache.vs), keep):
        t.copy_(o)
    pos.copy_(i32(s.pasts))
    for i in range(steps):
        s.q, s.k, s.v = [torch.randn(S, h, D, generator=g).to(torch.bfloat16) for h in (Hq, Hkv, Hkv)]
        for d, h in ((q, s.q), (k, s.k), (v, s.v)):
            d.copy_(h)
        graph.replay()
        s.pasts = [126 + i, 30 + i, 700 + i]
        s.seqs = [(c, p, 1) for c, p in zip(s.cu, s.pasts)]
        s.ref_write(s.k, s.v, s.seqs)
        torch.cuda.synchronize()
        assert plan.info.item() == 0
        s.check_cache()
        got = y.clone()
        s.check_attention(got, None)
        # the same step without the graph, and work of another size between the replays
        eager = aql.aql_attention_kv8(q, s.cache, s.dev_table, plan)
        assert torch.equal(eager, got)
        other = Step([(70, 3)], 2, 1, 64, seed=i)
        other.write_past()
        other.attend(other.write())
