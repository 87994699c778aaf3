"""The linear with an epilogue where its contraction is split and a second kernel sums the parts:
rows that end inside that kernel's groups of four outputs."""
import pytest
import torch

import activation_quantized_linear_amd as aql
from test_gpu_act import ACTS, BF16, DEV, F64, HALF, act64, check, linear

pytestmark = pytest.mark.gpu

# the skinny tile's split and the tiles', every remainder of N by 4, rows of fewer than four
SIZES = [(13, 8192, 261), (27, 8192, 262), (27, 14336, 1003), (63, 8192, 1), (27, 8192, 3), (27, 8192, 260),
         (130, 8192, 265), (130, 8192, 266), (65, 14336, 519), (64, 8192, 7), (130, 8192, 264)]


@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("name,b,m,r", [("silu", 0, 1, 0), ("none", 1, 0, 1), ("gelu", 1, 1, 1), ("gelu_tanh", 0, 0, 0)])
def test_split(M, K, N, name, b, m, r):
    assert aql.aql_workspace_bytes(aql.AQL_OP_W8A16, M, N, K) > 0  # (this size splits)
    x, q, scale, bias, mul, res, v, ev = linear(M, K, N, M + K + N)
    bias, mul, res = bias if b else None, mul if m else None, res if r else None
    if not b:
        v = torch.mm(x.to(F64), q.to(F64).T) * scale.to(F64)
    pre = torch.full((M, N), torch.nan, dtype=BF16, device=DEV)
    y = aql.aql_linear_w8a16_act(x, q, scale, bias, act=ACTS[name], mul=mul, residual=res, pre=pre)
    f = mul.to(F64) if m else torch.ones_like(v)
    a = act64(name, v)
    want = a * f + (res.to(F64) if r else 0.0)
    # slopes are at most 1.13; the hardware's exponential and reciprocal leave 2^-16 of the value
    check(y, want, HALF * want.abs() + (1.13 * ev + 2.0 ** -16 * a.abs()) * f.abs() + 2.0 ** -22 * want.abs() + 1e-30)
    check(pre, v, HALF * v.abs() + ev)
    for t in (mul, res):  # y in mul's or residual's own memory
        if t is None:
            continue
        args = {"mul": mul if mul is None else mul.clone(), "residual": res if res is None else res.clone()}
        own = args["mul" if t is mul else "residual"]
        p2 = torch.full_like(pre, torch.nan)
        got = aql.aql_linear_w8a16_act(x, q, scale, bias, act=ACTS[name], pre=p2, y=own, **args)
        assert got is own and torch.equal(got, y) and torch.equal(p2, pre)
