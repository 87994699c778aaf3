"""A decoder layer served in 8 bits, end to end: fused projection, cache write, attention, output
projection onto the residual stream and a gated MLP, and the gradients of that MLP's frozen
linears; against the same layer in 64 bits."""
import math

import pytest
import torch

import activation_quantized_linear_amd as aql
from kv_reference import Cache, attention

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64


def weights(g, n, k):
    w = torch.randn(n, k, generator=g) * 0.5 / math.sqrt(k)
    q, s, _ = aql.aql_quantize_weight_int8(w.to(DEV))
    return q, s, q.cpu().to(F64) * s.cpu().to(F64)[:, None]


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def bf(x):
    """What a bf16 tensor holds of 64-bit values."""
    return x.to(torch.bfloat16).to(F64)


@pytest.mark.parametrize("steps", [[(0, 70), (0, 3), (0, 130)], [(0, 1), (0, 1), (0, 1)]])
@pytest.mark.parametrize("H,Hq,Hkv,D,FF", [(192, 6, 2, 64, 320), (256, 4, 4, 72, 512)])
def test_layer(steps, H, Hq, Hkv, D, FF):
    """A prefill (or first tokens) and two decode steps behind it. Each rounding of the served layer
    to bf16 is one of the 64-bit layer too, so what is left are those at other values:
    errors stay below 2^-6 of the residual stream's norm, where a layer rounds five times by 2^-8."""
    g = torch.Generator().manual_seed(H + D)
    wqkv, wo = weights(g, (Hq + 2 * Hkv) * D, H), weights(g, H, (Hq * D + 15) // 16 * 16)
    assert (Hq * D) % 16 == 0
    wu, wg, wd = weights(g, FF, H), weights(g, FF, H), weights(g, H, FF)
    S, W = len(steps), 4
    table = [[0, 7, 2, 9], [3, 4, 10, 11], [6, 5, 1, 8]]
    cache, ref = aql.aql_kv_cache(12, Hkv, D, DEV), Cache(12, Hkv, D)
    dev_table = i32(table)
    pasts = [0] * S
    for turn in range(3):
        news = [n for _, n in steps] if turn == 0 else [1] * S
        cu = [0]
        for n in news:
            cu.append(cu[-1] + n)
        T = cu[-1]
        seqs = [(c, p, n) for c, p, n in zip(cu, pasts, news)]
        x = torch.randn(T, H, generator=g).to(torch.bfloat16)
        plan = aql.aql_kv_plan(i32(cu), i32(pasts), T, max(news), Hq, Hkv, W)

        def mine(x):
            qkv = aql.aql_linear_w8a16(x, *wqkv[:2])
            q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
            aql.aql_kv_cache_write(k, v, cache, dev_table, plan)
            y = aql.aql_attention_kv8(q, cache, dev_table, plan)
            x = aql.aql_linear_w8a16_act(y.reshape(T, Hq * D), *wo[:2], residual=x)
            up = aql.aql_linear_w8a16(x, *wu[:2])
            h = aql.aql_linear_w8a16_act(x, *wg[:2], act=aql.AQL_ACT_SILU, mul=up)
            return aql.aql_linear_w8a16_act(h, *wd[:2], residual=x), k, v

        got, k, v = mine(x.to(DEV))
        for i, s in enumerate(seqs):  # the cache takes what the projection gave
            ref.write(k.cpu(), v.cpu(), [s], [table[i]])
        x64 = x.to(F64)
        qkv = bf(x64 @ wqkv[2].T)
        y = bf(attention(ref, qkv[:, :Hq * D].reshape(T, Hq, D), seqs, table, 0, D ** -0.5)[0])
        r = bf(y.reshape(T, -1) @ wo[2].T + x64)
        gate = r @ wg[2].T
        want = bf(bf(gate * torch.sigmoid(gate) * bf(r @ wu[2].T)) @ wd[2].T + r)
        err = (got.cpu().to(F64) - want).norm() / want.norm()
        assert err < 2.0 ** -6, err
        pasts = [p + n for p, n in zip(pasts, news)]


def test_gradients_of_a_gated_mlp():
    """x -> silu(x Wg) * (x Wu) -> Wd, its input's gradient through the frozen int8 weights, with
    each step's gradient from the framework; against autograd in 64 bits."""
    g = torch.Generator().manual_seed(3)
    H, FF, M = 128, 256, 70
    wu, wg, wd = weights(g, FF, H), weights(g, FF, H), weights(g, H, FF)
    x = torch.randn(M, H, generator=g).to(torch.bfloat16)
    dy = torch.randn(M, H, generator=g).to(torch.bfloat16)
    xd = x.to(DEV)
    up = aql.aql_linear_w8a16(xd, *wu[:2])
    pre = torch.empty_like(up)
    h = aql.aql_linear_w8a16_act(xd, *wg[:2], act=aql.AQL_ACT_SILU, mul=up, pre=pre)
    out = aql.aql_linear_w8a16_act(h, *wd[:2], residual=xd)
    dh = aql.aql_linear_w8a16_dgrad(dy.to(DEV), *wd[:2])
    dv, dup = aql.aql_act_mul_backward(dh, pre, aql.AQL_ACT_SILU, up)
    dx = (dy.to(DEV).float() + aql.aql_linear_w8a16_dgrad(dv, *wg[:2]).float()
          + aql.aql_linear_w8a16_dgrad(dup, *wu[:2]).float())
    x64 = x.to(F64).requires_grad_()
    gate = x64 @ wg[2].T
    y = (gate * torch.sigmoid(gate) * (x64 @ wu[2].T)) @ wd[2].T + x64
    y.backward(dy.to(F64))
    # five roundings by 2^-8 on the way there, as many back
    assert (out.cpu().to(F64) - y.detach()).norm() / y.norm() < 2.0 ** -6
    assert (dx.cpu().to(F64) - x64.grad).norm() / x64.grad.norm() < 2.0 ** -6
