"""The int8 linear with activation, product and residual in its epilogue, and the gradients of
that epilogue, against their 64-bit forms."""
import math

import pytest
import torch

import activation_quantized_linear_amd as aql

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64
BF16 = torch.bfloat16
ACTS = {"none": aql.AQL_ACT_NONE, "relu": aql.AQL_ACT_RELU, "gelu": aql.AQL_ACT_GELU,
        "gelu_tanh": aql.AQL_ACT_GELU_TANH, "silu": aql.AQL_ACT_SILU}
HALF = 2.0 ** -8  # half a bf16 step, relative


def act64(name, z):
    """The activation in 64 bits."""
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z * math.sqrt(0.5))  # (keeps its left tail: Phi(-12) = 1.8e-33)
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z * 1


def grad64(name, z):
    z = z.clone().requires_grad_()
    act64(name, z).sum().backward()
    return z.grad


def bf16(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(BF16).to(DEV)


def linear(M, K, N, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = bf16(g, M, K, std=std)
    q = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8).to(DEV)
    scale = (torch.rand(N, generator=g) * 2 / (74 * math.sqrt(K))).to(DEV)
    bias, mul, res = bf16(g, N), bf16(g, M, N), bf16(g, M, N, std=3.0)
    v = (x.to(F64) @ q.to(F64).T) * scale.to(F64) + bias.to(F64)
    # float32 sums of exact products: 2^-23 a term at most, with the scale's and bias's roundings
    size = (x.to(F64).abs() @ q.to(F64).abs().T) * scale.to(F64) + bias.to(F64).abs()
    return x, q, scale, bias, mul, res, v, size * (min(K, 1024) + 8) * 2.0 ** -23


def check(y, want, tol):
    err = (y.to(F64) - want).abs()
    assert (err <= tol).all(), (err / tol.clamp(min=1e-30)).max().item()


# a size of every kernel that the linear takes: the single-row ones, a few rows, the
# skinny tile (2, 3 rows too), its shared form and its split, the tiles and their split
SIZES = [(1, 960, 2560), (1, 4096, 520), (1, 2560, 961), (1, 8192, 136), (2, 2048, 130), (3, 960, 77),
         (2, 64, 40), (4, 4096, 256), (5, 960, 2560), (27, 8192, 260), (13, 4096, 8200), (9, 4112, 12300),
         (63, 1040, 100), (64, 960, 2560), (65, 72 * 16, 333), (130, 8192, 264), (300, 256, 4100),
         (500, 320, 11007), (257, 192, 16500), (1100, 64, 16390)]


@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("name,m,r,p", [("silu", 1, 0, 0), ("none", 0, 1, 1), ("gelu", 1, 1, 1), ("gelu_tanh", 0, 0, 1),
                                       ("relu", 0, 1, 0)])
def test_linear(M, K, N, name, m, r, p):
    x, q, scale, bias, mul, res, v, ev = linear(M, K, N, M + K + N)
    pre = torch.empty(M, N, dtype=BF16, device=DEV) if p else None
    y = aql.aql_linear_w8a16_act(x, q, scale, bias if p else None, act=ACTS[name], mul=mul if m else None,
                                 residual=res if r else None, pre=pre)
    if not p:
        v = v - bias.to(F64)
    f, rr = mul.to(F64) if m else 1.0, res.to(F64) if r else 0.0
    a = act64(name, v)
    want = a * f + rr
    # slopes are at most 1.13; the hardware's exponential and reciprocal leave 2^-16 of the value
    tol = HALF * want.abs() + (1.13 * ev + 2.0 ** -16 * a.abs()) * abs(f) + 2.0 ** -22 * want.abs() + 1e-30
    check(y, want, tol)
    if p:
        check(pre, v, HALF * v.abs() + ev)


def test_linear_in_place_and_plain():
    """y in residual's or mul's own memory; without act, mul and residual the linear itself."""
    for M, K, N in [(1, 960, 2560), (27, 8192, 260), (300, 256, 4100), (500, 320, 11007), (130, 8192, 264)]:
        x, q, scale, bias, mul, res, _, _ = linear(M, K, N, 3)
        want = aql.aql_linear_w8a16_act(x, q, scale, bias, act=aql.AQL_ACT_SILU, mul=mul, residual=res)
        for which in (0, 1):
            a, b = mul.clone(), res.clone()
            y = (a, b)[which]
            got = aql.aql_linear_w8a16_act(x, q, scale, bias, act=aql.AQL_ACT_SILU, mul=a, residual=b, y=y)
            assert got is y and torch.equal(y, want)
        assert torch.equal(aql.aql_linear_w8a16_act(x, q, scale, bias), aql.aql_linear_w8a16(x, q, scale, bias))


@pytest.mark.parametrize("name", list(ACTS))
def test_far_values(name):
    """Values whose exponentials leave float32, through a linear of one channel."""
    x = torch.zeros(8, 16, dtype=BF16, device=DEV)
    x[:, 0] = torch.tensor([-1e30, -300.0, -89.0, -12.0, 12.0, 89.0, 300.0, 1e30])
    q = torch.ones(1, 16, dtype=torch.int8, device=DEV)
    scale = torch.ones(1, device=DEV)
    y = aql.aql_linear_w8a16_act(x, q, scale, act=ACTS[name])
    z = x[:, :1].to(F64)
    want = act64(name, z)
    check(y, want, (HALF + 2.0 ** -16) * want.abs() + 1e-35)
    dv, _ = aql.aql_act_mul_backward(torch.ones_like(y), x[:, :1].contiguous(), ACTS[name])
    wide = z.abs() > 50  # (the cube's own gradient is no number there)
    d = torch.where(wide, (z > 0).to(F64) if name != "none" else torch.ones_like(z), grad64(name, z.clamp(-50, 50)))
    check(dv, d, HALF * d.abs() + 2.0 ** -20)


@pytest.mark.parametrize("M,N", [(1, 1), (3, 5), (63, 2560), (1, 4095), (7, 1001), (130, 8200), (1, 8), (2, 4096)])
@pytest.mark.parametrize("name", list(ACTS))
@pytest.mark.parametrize("m", [0, 1])
def test_backward(M, N, name, m):
    g = torch.Generator().manual_seed(M * N)
    dy, pre, mul = bf16(g, M, N), bf16(g, M, N, std=2.5), bf16(g, M, N)
    dv, dmul = aql.aql_act_mul_backward(dy, pre, ACTS[name], mul if m else None)
    z, f = pre.to(F64), mul.to(F64) if m else torch.ones(M, N, dtype=F64, device=DEV)
    d, a = grad64(name, z), act64(name, z)
    # act' is a sum of terms up to 1.2: 2^-20 absolute where they cancel
    check(dv, dy.to(F64) * f * d, (dy.to(F64) * f).abs() * ((HALF + 2.0 ** -15) * d.abs() + 2.0 ** -20))
    if m:
        check(dmul, dy.to(F64) * a, dy.to(F64).abs() * (HALF + 2.0 ** -15) * a.abs() + 1e-30)
        # in place, and without dmul
        d2 = dy.clone()
        m2 = mul.clone()
        o1, o2 = aql.aql_act_mul_backward(d2, pre, ACTS[name], m2, dv=d2, dmul=m2)
        assert torch.equal(o1, dv) and torch.equal(o2, dmul)
        o1, o2 = aql.aql_act_mul_backward(dy, pre, ACTS[name], mul, need_dmul=False)
        assert torch.equal(o1, dv) and o2 is None
    else:
        assert dmul is None


@pytest.mark.parametrize("name", list(ACTS))
def test_backward_against_differences(name):
    """dv against central differences of the 64-bit forward form (relu away from its corner)."""
    g = torch.Generator().manual_seed(5)
    dy, pre = bf16(g, 8, 64), bf16(g, 8, 64, std=2.0)
    pre = torch.where(pre.abs() < 0.01, torch.ones_like(pre), pre)
    dv, _ = aql.aql_act_mul_backward(dy, pre, ACTS[name])
    h, z = 1e-4, pre.to(F64)
    d = (act64(name, z + h) - act64(name, z - h)) / (2 * h)
    # the difference's own error: h^2 / 6 of a third derivative below 3
    check(dv, dy.to(F64) * d, dy.to(F64).abs() * ((HALF + 2.0 ** -15) * d.abs() + 2.0 ** -20 + 3 * h * h))
