"""Attention over the 8-bit cache where its numbers leave their ordinary range, against the definition in 64
bits on the codes that the cache holds."""
import math

import pytest
import torch

import activation_quantized_linear_amd as aql

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64
BLOCK = 64
LOG2E = 1.0 / math.log(2.0)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Filled:
    """A cache of given codes [P, Hkv, 64, D] and scales [P, Hkv], pages in reverse order, for
    sequences (past, new) whose tokens are all in it."""

    def __init__(self, seqs, Hq, Hkv, D, window=0):
        self.seqs, self.Hq, self.Hkv, self.D, self.window = seqs, Hq, Hkv, D, window
        need = [(p + n + BLOCK - 1) // BLOCK for p, n in seqs]
        self.P, self.W = sum(need), max(need)
        order = list(range(self.P))[::-1]
        self.pages, at = [], 0
        for n in need:
            self.pages.append(order[at:at + n])
            at += n
        self.table = i32([p + [-1] * (self.W - len(p)) for p in self.pages])
        self.T = sum(n for _, n in seqs)

    def fill(self, k, ks, v, vs):
        self.k, self.ks, self.v, self.vs = k, ks, v, vs
        pad = (self.D + 63) // 64 * 64
        self.cache = aql.aql_kv_cache(self.P, self.Hkv, self.D, DEV)
        wide = torch.zeros(self.P, self.Hkv, BLOCK, pad, dtype=torch.int8, device=DEV)
        wide[..., :self.D] = k
        self.cache.kq.copy_(wide.view(self.P, self.Hkv, BLOCK, pad // 64, 64).transpose(2, 3))
        wide[..., :self.D] = v
        self.cache.vq.copy_(wide.transpose(2, 3))
        self.cache.ks.copy_(ks)
        self.cache.vs.copy_(vs)

    def run(self, q, sm):
        cu = [0]
        for _, n in self.seqs:
            cu.append(cu[-1] + n)
        plan = aql.aql_kv_plan(i32(cu), i32([p for p, _ in self.seqs]), self.T, max(n for _, n in self.seqs), self.Hq,
                               self.Hkv, self.W, self.window)
        lse = torch.empty(self.T, self.Hq, device=DEV)
        y = aql.aql_attention_kv8(q, self.cache, self.table, plan, sm_scale=sm, lse=lse)
        assert plan.info.item() == 0
        return y, lse

    def check(self, q, sm):
        """One half step of the output, 2^-8 of it. A weight's rounding to float16: 2^-11 of it, or 2^-25 of
        2^-7 of the largest weight times scale, against codes of up to 127. A score's error
        delta, in powers of two: the float32 sum of its dot product (2^-23 a term and four
        scales), the hardware's logarithm and exponential and the differences to the maximum (2^-21 of the
        arguments); as relative error of a weight ln 2 times that, for numerator and denominator. Float32
        sums over the tokens, 2^-24 each."""
        y, lse = self.run(q, sm)
        G, row = self.Hq // self.Hkv, 0
        for (past, new), pages in zip(self.seqs, self.pages):
            n = past + new
            for h in range(self.Hkv):
                at = torch.tensor(pages, device=DEV)
                k = (self.k[at, h].to(F64) * self.ks[at, h].to(F64)[:, None, None]).view(-1, self.D)[:n]
                v = (self.v[at, h].to(F64) * self.vs[at, h].to(F64)[:, None, None]).view(-1, self.D)[:n]
                sv = self.vs[at, h].to(F64).repeat_interleave(BLOCK)[:n]
                rows = q[row:row + new, h * G:(h + 1) * G].to(F64).reshape(-1, self.D)
                p = torch.arange(past, n, device=DEV).repeat_interleave(G)[:, None]
                t = torch.arange(n, device=DEV)[None, :]
                hidden = t > p
                if self.window:
                    hidden = hidden | (t <= p - self.window)
                s = torch.mm(rows, k.T) * sm
                size = torch.mm(rows.abs(), k.abs().T) * sm * LOG2E
                size = size.masked_fill(hidden, 0.0).amax(1, keepdim=True)
                big = s.masked_fill(hidden, 0.0).abs().amax(1, keepdim=True) * LOG2E + sv.log2().abs().max()
                s = s.masked_fill(hidden, -math.inf)
                want_lse = torch.logsumexp(s, 1, keepdim=True)
                w = torch.exp(s - want_lse)
                want = torch.mm(w, v)
                delta = size * 2.0 ** -23 * (self.D + 4) + big * 2.0 ** -21
                rel = 2 * (math.log(2) * delta + 2.0 ** -22) + 2.0 ** -11 + n * 2.0 ** -24
                tol = (2.0 ** -8 * want.abs() + rel * torch.mm(w, v.abs())
                       + n * 2.0 ** -32 * 127 * (w * sv).amax(1, keepdim=True))
                got = y[row:row + new, h * G:(h + 1) * G].reshape(-1, self.D).to(F64)
                err = (got - want).abs()
                assert (err <= tol).all(), (past, new, h, (err / tol).max().item())
                ltol = delta + 2.0 ** -21 * (1 + big) + n * 2.0 ** -24
                got = lse[row:row + new, h * G:(h + 1) * G].reshape(-1, 1).to(F64)
                assert ((got - want_lse).abs() <= ltol).all(), (past, new, h)
            row += new


def offset_case(seqs, D, offset, window=0, seed=0):
    """Scores of a few units around a common offset (what a bias in K's projection gives); the first
    page of the first sequence has V of zero, whose scale is the smallest."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = Filled(seqs, 4, 2, D, window)
    k = torch.randint(-32, 33, (c.P, 2, BLOCK, D), generator=g, device=DEV, dtype=torch.int8)
    v = torch.randint(-127, 128, (c.P, 2, BLOCK, D), generator=g, device=DEV, dtype=torch.int8)
    k[..., 0] = 127
    ks = torch.full((c.P, 2), 2.0 ** -5, device=DEV)
    vs = torch.rand(c.P, 2, generator=g, device=DEV) + 0.5
    v[c.pages[0][0]] = 0
    vs[c.pages[0][0]] = 2.0 ** -64
    c.fill(k, ks, v, vs)
    q = torch.randn(c.T, 4, D, generator=g, device=DEV)
    sm = D ** -0.5
    q[..., 0] = offset / (127 * 2.0 ** -5 * sm)
    return c, q.to(torch.bfloat16), sm


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 40, 70, 300])
@pytest.mark.parametrize("past", [70, 1900])  # one unit a tile, and blocks divided over several
@pytest.mark.parametrize("offset", [-60, -100, -200, 200])
def test_common_offset(D, new, past, offset):
    c, q, sm = offset_case([(past, new), (0, new), (past // 2, 1)], D, offset, seed=D + new)
    c.check(q, sm)


@pytest.mark.parametrize("D", [64, 192])
@pytest.mark.parametrize("new", [1, 90])
def test_common_offset_in_a_window(D, new):
    c, q, sm = offset_case([(1000, new), (0, new)], D, -150, window=100, seed=D)
    c.check(q, sm)


@pytest.mark.parametrize("new", [1, 6, 70])  # streams of 16 and 32 rows, tiles
@pytest.mark.parametrize("past", [300, 2100])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_most_of_the_weight_without_values(new, past, D):
    """In every page one token has nearly all of the weight and a V of zero; the others, 14.5 2^-24
    of its weight each, are all that the outputs are made of."""
    g = torch.Generator(device=DEV).manual_seed(D + new)
    c = Filled([(past, new), (past // 2, 1)], 4, 1, D)
    k = torch.zeros(c.P, 1, BLOCK, D, dtype=torch.int8, device=DEV)
    v = torch.randint(30, 128, (c.P, 1, BLOCK, D), generator=g, device=DEV, dtype=torch.int8)
    k[:, :, 0, 0] = 127
    v[:, :, 0] = 0
    c.fill(k, torch.full((c.P, 1), 1 / 127, device=DEV), v, torch.full((c.P, 1), 0.03, device=DEV))
    q = torch.randn(c.T, 4, D, generator=g, device=DEV)
    q[..., 0] = 1.0
    c.check(q.to(torch.bfloat16), -math.log(14.5 * 2.0 ** -24))


@pytest.mark.parametrize("new,Hkv", [(1, 1), (6, 1), (70, 1), (1, 256), (40, 256)])
def test_one_token_with_most_of_the_weight(new, Hkv, D=64):
    """The first of 131072 tokens has 90% of every row's weight and a V of zero; divided and whole."""
    g = torch.Generator(device=DEV).manual_seed(D + new)
    c = Filled([(131072 - new, new)], 4 * Hkv, Hkv, D)
    k = torch.zeros(c.P, Hkv, BLOCK, D, dtype=torch.int8, device=DEV)
    v = torch.randint(30, 128, (c.P, Hkv, BLOCK, D), generator=g, device=DEV, dtype=torch.int8)
    k[c.pages[0][0], :, 0, 0] = 127
    v[c.pages[0][0], :, 0] = 0
    c.fill(k, torch.full((c.P, Hkv), 1 / 127, device=DEV), v, torch.full((c.P, Hkv), 0.03, device=DEV))
    q = torch.randn(c.T, 4 * Hkv, D, generator=g, device=DEV)
    q[..., 0] = 1.0
    c.check(q.to(torch.bfloat16), -math.log(14.5 * 2.0 ** -24))


@pytest.mark.parametrize("new", [1, 6, 70])
@pytest.mark.parametrize("D", [64, 128, 200])
def test_small_elements_of_a_query(new, D):
    """A query whose largest element meets a channel without K, and whose other elements, down to 2^-32
    of it, meet channels that run as hot: each counts with all of its bits."""
    g = torch.Generator(device=DEV).manual_seed(D + new)
    c = Filled([(700, new), (40, 1)], 4, 2, D)
    k = torch.randint(-127, 128, (c.P, 2, BLOCK, D), generator=g, device=DEV, dtype=torch.int8)
    v = torch.randint(-127, 128, (c.P, 2, BLOCK, D), generator=g, device=DEV, dtype=torch.int8)
    k[..., 0] = 0
    down = torch.tensor([22.0, 24.0, 28.0, 30.0], device=DEV)  # of each head
    ks = torch.tensor([2.0 ** 16, 2.0 ** 22], device=DEV).expand(c.P, 2).contiguous()
    c.fill(k, ks, v, torch.rand(c.P, 2, generator=g, device=DEV) + 0.5)
    q = torch.rand(c.T, 4, D, generator=g, device=DEV) * 2 + 0.25
    q = torch.where(torch.rand(c.T, 4, D, generator=g, device=DEV) < 0.5, q, -q) * (2.0 ** -down)[None, :, None]
    q[..., 0] = 1.0
    c.check(q.to(torch.bfloat16), 0.25)


@pytest.mark.parametrize("new", [1, 6, 70])
@pytest.mark.parametrize("D", [64, 192])
@pytest.mark.parametrize("up", [0, 46])
def test_scales_of_v_far_apart(new, D, up):
    """Every other page has V of zero under the smallest scale, 2^-64, the rest V of 2^up: the tokens
    of both count alike in the denominator."""
    g = torch.Generator(device=DEV).manual_seed(D + new)
    c = Filled([(700, new), (100, 1)], 4, 2, D)
    k = torch.randint(-32, 33, (c.P, 2, BLOCK, D), generator=g, device=DEV, dtype=torch.int8)
    v = torch.randint(-127, 128, (c.P, 2, BLOCK, D), generator=g, device=DEV, dtype=torch.int8)
    vs = torch.full((c.P, 2), 2.0 ** up, device=DEV)
    for p in (p for s in c.pages for p in s[::2]):
        v[p], vs[p] = 0, 2.0 ** -64
    c.fill(k, torch.full((c.P, 2), 2.0 ** -5, device=DEV), v, vs)
    c.check(torch.randn(c.T, 4, D, generator=g, device=DEV).to(torch.bfloat16), D ** -0.5)
