"""Low-rank adapters beside the W8A16 linear, their gradients, and 8-bit
activation checkpoints, against plain 64-bit forms on the CPU.

Tolerances. With u = 2^-24, a float32 sum of n terms in any order is off by at
most (n + 1) u T, T the sum of the terms' magnitudes (products of bf16 or int8
values are exact in float32; one rounding more for a scale). Then
  h, u     (K + 3) u T                     (N for u; + alpha's rounding)
  y        2^-8 |y| (rounding to bf16) + (K + R + 4) u T
           + (|h|'s own error + 2^-16 |h|, its two-part split) . |B|
  dx       2^-8 |dx| + (N + R + 4) u T + (|u|'s own error + 2^-16 |u|) . |A|
           + sum |error of (dy scale)| |q|: 2^-11 of it, its rounding to float16
           (and 2^-38 of its row's largest, the half step of float16's subnormals
           2^-25 under a largest value of at least 2^13)
  dA, dB   (m + 4) u T + 2^-23 T (three-part split, the product with a scale)
           + u's own error . |x'|,  m the adapter's rows
and over the whole of a bf16 output the norm of the error is at most 4e-3 of
the output's: one rounding of relative size 2^-8 / sqrt(3) at most, 2.3e-3."""
import numpy as np
import pytest
import torch

import activation_quantized_linear_amd as aql
import workloads

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
GROUP = 128


def say(*a):
    print(*a, flush=True)


def make(M, K, N, L, R, mix="random", bias=False, seed=0):
    g = workloads.gen(1000 + seed + 7 * M + 11 * K + 13 * N + L + R)
    w = workloads.randn(g, N, K, std=0.02)
    scale = w.abs().amax(1).clamp_min(1e-9) / 127.0 if N else torch.empty(0)
    c = {
        "q": torch.round(w / scale[:, None]).clamp(-127, 127).to(torch.int8),
        "scale": scale,
        "bias": workloads.randn(g, N, std=0.1).to(torch.bfloat16) if bias else None,
        "x": workloads.randn(g, M, K).to(torch.bfloat16),
        "dy": (workloads.randn(g, M, N, std=1e-3)
               * torch.exp(workloads.randn(g, M, 1))).to(torch.bfloat16),
        "A": workloads.randn(g, L, R, K, std=K ** -0.5).to(torch.bfloat16),
        "B": workloads.randn(g, L, N, R, std=0.02).to(torch.bfloat16),
        "alpha": 0.5 + torch.rand(L, generator=g),
    }
    if mix == "random":
        idx = torch.randint(-1, L + 1, (M,), generator=g)  # -1 and L: none
        idx[idx == L] = 2 ** 31 - 1
    elif mix == "runs":
        idx = (torch.arange(M) * L) // max(M, 1)
    elif mix == "none":
        idx = torch.full((M,), -5)
    else:
        idx = torch.full((M,), int(mix))
    c["idx"] = idx.to(torch.int32)
    return c


def dev(c):
    return {k: (v.contiguous().to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in c.items()}


def f64(t):
    return t.double()


def rows_of(c, a):
    return (c["idx"] == a).nonzero()[:, 0]


def ref_forward(c):
    x, q, s = f64(c["x"]), f64(c["q"]), f64(c["scale"])
    M, K = x.shape
    N, (L, R) = q.shape[0], c["A"].shape[:2]
    y, T = (x @ q.T) * s, (x.abs() @ q.abs().T) * s
    h, hT = torch.zeros(M, R).double(), torch.zeros(M, R).double()
    tol = torch.zeros(M, N).double()
    for a in range(L):
        r = rows_of(c, a)
        if len(r) == 0:
            continue
        A, B, al = f64(c["A"][a]), f64(c["B"][a]), float(c["alpha"][a])
        h[r] = al * (x[r] @ A.T)
        hT[r] = al * (x[r].abs() @ A.abs().T)
        y[r] += h[r] @ B.T
        T[r] += h[r].abs() @ B.abs().T
        tol[r] += ((K + 3) * U * hT[r] + 2.0 ** -16 * h[r].abs()) @ B.abs().T
    if c["bias"] is not None:
        y, T = y + f64(c["bias"]), T + f64(c["bias"]).abs()
    tol += 2.0 ** -8 * y.abs() + (K + R + 4) * U * T
    return y, tol, h, (K + 3) * U * hT


def checkpoint_ref(x):
    """Codes and scales in the definition's own float32 steps."""
    x = x.float()
    M, K = x.shape
    G = (K + GROUP - 1) // GROUP
    p = torch.zeros(M, G * GROUP)
    p[:, :K] = x
    p = p.view(M, G, GROUP)
    s = p.abs().amax(2) / np.float32(127.0)
    s = torch.where(s > 0, s, torch.ones_like(s))
    codes = torch.round(p / s[:, :, None]).clamp(-127, 127)
    return codes.view(M, -1)[:, :K].to(torch.int8), s


def decoded(xq, xs):
    K = xq.shape[1]
    return f64(xq) * f64(xs).repeat_interleave(GROUP, 1)[:, :K]


def ref_dgrad(c):
    """dx = (dy scale) q, the magnitudes of its terms, and what float16 takes of dy scale."""
    d, q = f64(c["dy"]) * f64(c["scale"]), f64(c["q"])
    off = 2.0 ** -11 * d.abs()
    if d.numel():
        off = off + 2.0 ** -38 * d.abs().amax(1, keepdim=True)
    return d @ q, d.abs() @ q.abs(), off @ q.abs()


def ref_backward(c, h, xq, xs):
    dy, x = f64(c["dy"]), decoded(xq, xs)
    N, K = c["q"].shape
    L, R = c["A"].shape[:2]
    dx, T, tol = ref_dgrad(c)
    dA, dB = torch.zeros(L, R, K).double(), torch.zeros(L, N, R).double()
    tA, tB = torch.zeros_like(dA), torch.zeros_like(dB)
    for a in range(L):
        r = rows_of(c, a)
        m = len(r)
        if m == 0:
            continue
        A, B, al = f64(c["A"][a]), f64(c["B"][a]), float(c["alpha"][a])
        u = al * (dy[r] @ B)
        ue = (N + 3) * U * al * (dy[r].abs() @ B.abs())
        dx[r] += u @ A
        T[r] += u.abs() @ A.abs()
        tol[r] += (ue + 2.0 ** -16 * u.abs()) @ A.abs()
        dA[a] = u.T @ x[r]
        tA[a] = ((m + 4) * U + 2.0 ** -23) * (u.abs().T @ x[r].abs()) + ue.T @ x[r].abs()
        hr = f64(h[r])
        dB[a] = dy[r].T @ hr
        tB[a] = ((m + 4) * U + 2.0 ** -23) * (dy[r].abs().T @ hr.abs())
    tol += 2.0 ** -8 * dx.abs() + (N + R + 4) * U * T
    return (dx, tol), (dA, tA), (dB, tB)


def close(got, ref, tol, what, norm=None):
    got = got.double().cpu()
    assert got.shape == ref.shape, what
    assert torch.isfinite(got).all(), f"{what}: not finite"
    err = (got - ref).abs()
    bad = err > tol
    if bad.any():
        i = torch.argmax(err - tol)
        at = np.unravel_index(int(i), tuple(err.shape))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst at {at}: got "
                             f"{got[at].item()!r} want {ref[at].item()!r} tol {tol[at].item()!r}")
    if norm is not None and ref.numel():
        assert err.norm() <= norm * ref.norm() + 1e-300, f"{what}: norm {err.norm() / ref.norm()}"


def forward(d, plan=None, **kw):
    if plan is None:
        plan = aql.aql_lora_plan(d["idx"], d["A"].shape[0])
    y, h = aql.aql_linear_w8a16_lora(d["x"], d["q"], d["scale"], d["A"], d["B"], d["alpha"], plan,
                                     d["bias"], **kw)
    return y, h, plan


def backward(d, plan, h, xq, xs, **kw):
    return aql.aql_linear_w8a16_lora_backward(d["dy"], d["q"], d["scale"], d["A"], d["B"],
                                              d["alpha"], plan, h, xq, xs, **kw)


# ------------------------------------------------------------------- the plan


@pytest.mark.parametrize("M,L", [(1, 1), (1, 7), (5, 2), (16, 3), (17, 1), (64, 64), (500, 3),
                                 (1023, 9), (1024, 1), (1025, 33), (3000, 1024), (5000, 200)])
@pytest.mark.parametrize("mix", ["random", "runs", "none"])
def test_plan(M, L, mix):
    say("plan", M, L, mix)
    g = workloads.gen(M + L)
    if mix == "random":
        idx = torch.randint(-2, L + 2, (M,), generator=g).to(torch.int32)
    elif mix == "runs":
        idx = ((torch.arange(M) * L) // M).to(torch.int32)
    else:
        idx = torch.full((M,), -1, dtype=torch.int32)
    p = aql.aql_lora_plan(idx.to(DEV), L)
    torch.cuda.synchronize()
    assert (p.M, p.L) == (M, L)
    b = p.buffer.cpu().view(torch.int32)
    tiles = M // 16 + min(M, L + 1)
    up = lambda v: (v + 15) // 16 * 16
    o_idx, o_perm = 16, 16 + up(M)
    o_own = o_perm + 16 * tiles
    o_first = o_own + up(tiles)
    valid = torch.where((idx >= 0) & (idx < L), idx, torch.full_like(idx, -1))
    assert torch.equal(b[o_idx:o_idx + M], valid)
    perm, own, first = b[o_perm:o_own], b[o_own:o_own + tiles], b[o_first:o_first + L + 1]
    t = 0
    for a in list(range(L)) + [-1]:
        rows = (valid == a).nonzero()[:, 0].to(torch.int32)
        n = (len(rows) + 15) // 16
        assert int(first[a if a >= 0 else L]) == t
        want = torch.full((16 * n,), -1, dtype=torch.int32)
        want[:len(rows)] = rows
        assert torch.equal(perm[16 * t:16 * (t + n)], want), (a, rows)
        assert (own[t:t + n] == a).all()
        t += n
    assert int(b[0]) == t and (own[t:] == -2).all() and (perm[16 * t:] == -1).all()
    # groups of 128 rows: more than 4 adapters or not
    mixed = b[o_first + up(L + 1):]
    for i in range((M + 127) // 128):
        here = valid[128 * i:128 * (i + 1)]
        assert int(mixed[i]) == (len(set(here[here >= 0].tolist())) > 4)


# -------------------------------------------------------------------- forward

FORWARD = [
    # one row: single-row tile (K outside 2048..8192), contiguous form, x past the LDS budget
    (1, 16, 1, 1, 8, "0"), (1, 960, 2560, 4, 8, "random"), (1, 2048, 40, 2, 16, "0"),
    (1, 4096, 2056, 3, 64, "1"), (1, 8192, 24, 2, 128, "0"), (1, 17408, 24, 2, 16, "1"),
    (1, 960, 77, 3, 24, "none"),
    # two to four rows: skinny tile, few-row form
    (2, 256, 50, 3, 16, "random"), (3, 2048, 33, 4, 40, "random"), (4, 4096, 64, 2, 8, "runs"),
    (2, 16384, 9, 2, 16, "runs"), (3, 16400, 9, 2, 16, "runs"),
    # skinny tile, shared-x tile, split K with the workspace
    (5, 960, 2560, 8, 16, "random"), (16, 976, 65, 3, 32, "random"), (27, 512, 131, 27, 16, "runs"),
    (63, 2560, 960, 5, 128, "random"), (33, 64, 8200, 4, 16, "random"),
    (17, 4096, 12290, 2, 8, "random"), (16, 8192, 72, 3, 64, "random"), (63, 9232, 40, 1, 16, "0"),
    # tiled GEMM: ragged and whole K, 64 x 128, 128 x 128, wide with 4 and 2 stages, split K
    (64, 48, 130, 3, 8, "random"), (65, 64, 127, 64, 16, "random"), (200, 320, 257, 3, 64, "runs"),
    (129, 1024, 264, 2, 128, "random"), (2048, 64, 2048, 5, 24, "runs"),
    (70, 64, 40960, 3, 16, "random"), (1024, 80, 16384, 2, 40, "runs"),
    (100, 8192, 72, 3, 16, "random"), (257, 8192, 1024, 1, 64, "0"), (150, 96, 64, 2, 16, "none"),
    # rows that begin at any even address, in every tile form
    (70, 64, 40957, 3, 16, "random"), (1024, 80, 16381, 2, 40, "runs"), (2048, 64, 2043, 1, 8, "0"),
    (500, 64, 11005, 3, 16, "runs"), (77, 128, 6, 2, 8, "random"), (65, 64, 3, 1, 8, "0"),
    (129, 64, 1, 1, 8, "0"),
    # many adapters in a tile, in every tile form; products given to the sum of a split
    (64, 4096, 1000, 64, 16, "random"), (300, 128, 515, 300, 8, "runs"),
    (150, 64, 20480, 9, 40, "random"), (1024, 80, 16381, 12, 8, "random"),
    (2048, 64, 2043, 20, 16, "random"), (300, 8192, 1000, 7, 64, "random"),
    (513, 8192, 1001, 5, 128, "runs"),
]


@pytest.mark.parametrize("M,K,N,L,R,mix", FORWARD)
@pytest.mark.parametrize("bias", [False, True])
def test_forward(M, K, N, L, R, mix, bias):
    say("forward", M, K, N, L, R, mix, bias)
    c = make(M, K, N, L, R, mix, bias)
    y, h, _ = forward(dev(c))
    torch.cuda.synchronize()
    yr, ytol, hr, htol = ref_forward(c)
    close(h, hr, htol, "h")
    close(y, yr, ytol, "y", norm=4e-3)


def test_forward_without_adapters_is_the_plain_linear():
    for M, K, N in ((1, 960, 2560), (1, 4096, 520), (3, 4096, 40), (20, 512, 96), (40, 64, 8200),
                    (128, 256, 512)):
        say("plain", M, K, N)
        d = dev(make(M, K, N, 2, 16, "none", True))
        y, h, _ = forward(d)
        assert torch.equal(h, torch.zeros_like(h))
        if M in (1, 20, 40, 128):  # the same kernels serve both calls
            assert torch.equal(y, aql.aql_linear_w8a16(d["x"], d["q"], d["scale"], d["bias"]))


@pytest.mark.parametrize("M", [9, 27, 150, 300])
def test_adapters_do_not_reach_each_other(M):
    """NaN and infinities in one adapter's matrices, and in its rows, stay in its rows."""
    say("isolation", M)
    c = make(M, 512, 320, 3, 16, "random")
    y0, h0, _ = forward(dev(c))
    c["A"][1], c["B"][1, ::2], c["B"][1, 1::2] = float("nan"), float("inf"), float("nan")
    c["x"][c["idx"] == 1] = float("inf")
    y1, h1, plan = forward(dev(c))
    torch.cuda.synchronize()
    other = (c["idx"] != 1).to(DEV)
    assert torch.equal(y0[other], y1[other]) and torch.equal(h0[other], h1[other])
    assert not torch.isfinite(h1[~other]).any()
    # the gradients too: rows of adapter 1, and rows without one, hold NaN
    c = make(M, 512, 320, 3, 16, "random")
    d = dev(c)
    y, h, plan = forward(d)
    xq, xs = aql.aql_act_checkpoint(d["x"])
    dx0, dA0, dB0 = backward(d, plan, h, xq, xs)
    for bad in (1, -1, 2 ** 31 - 1):
        rows = (c["idx"] == bad).to(DEV)
        d["dy"][rows], h[rows], xs[rows] = float("nan"), float("inf"), float("nan")
    d["A"][1], d["B"][1] = float("nan"), float("inf")
    dx1, dA1, dB1 = backward(d, plan, h, xq, xs)
    torch.cuda.synchronize()
    ok = ((c["idx"] == 0) | (c["idx"] == 2)).to(DEV)
    assert torch.equal(dx0[ok], dx1[ok])
    assert torch.equal(dA0[::2], dA1[::2]) and torch.equal(dB0[::2], dB1[::2])


@pytest.mark.parametrize("K,N", [(512, 320), (64, 20480), (2560, 264)])
def test_groups_of_many_and_of_few_adapters(K, N):
    """One batch with rows of nine adapters at random, of one, of two and of none; a
    NaN in one adapter's matrices, and in its rows, stays in its rows."""
    M, L, R = 700, 9, 24
    c = make(M, K, N, L, R, "random")
    c["idx"][128:256], c["idx"][256:400] = 3, -1
    c["idx"][400:640] = torch.arange(240).to(torch.int32) // 130
    say("groups", K, N)

    def run():
        d = dev(c)
        y, h, plan = forward(d)
        xq, xs = aql.aql_act_checkpoint(d["x"])
        out = (y, h, *backward(d, plan, h, xq, xs))
        torch.cuda.synchronize()
        return out

    y, h, dx, dA, dB = run()
    yr, ytol, hr, htol = ref_forward(c)
    close(h, hr, htol, "h")
    close(y, yr, ytol, "y", norm=4e-3)
    rows = c["idx"] == 3
    c["A"][3], c["B"][3], c["x"][rows], c["dy"][rows] = (float("nan"),) * 4
    y1, h1, dx1, dA1, dB1 = run()
    ok, others = (~rows).to(DEV), [a for a in range(L) if a != 3]
    for a, b in ((y, y1), (h, h1), (dx, dx1)):
        assert torch.equal(a[ok], b[ok]) and torch.isnan(b[~ok]).all()
    assert torch.equal(dA[others], dA1[others]) and torch.equal(dB[others], dB1[others])


# ------------------------------------------------------------------- backward

BACKWARD = [
    (1, 16, 8, 1, 8, "0"), (1, 960, 2560, 2, 16, "1"), (2, 144, 24, 3, 24, "runs"),
    (15, 128, 128, 2, 32, "random"), (16, 272, 136, 1, 40, "0"), (17, 256, 264, 4, 64, "random"),
    (31, 2560, 960, 3, 128, "runs"), (63, 960, 2560, 2, 8, "runs"), (64, 64, 4096, 64, 16, "runs"),
    (130, 4096, 72, 3, 16, "random"), (257, 304, 200, 5, 48, "runs"), (500, 1024, 520, 3, 64, "runs"),
    (300, 80, 1048, 1, 16, "none"), (1000, 512, 640, 7, 128, "random"),
    (2100, 2560, 192, 2, 16, "runs"), (1100, 16384, 64, 1, 8, "0"), (33, 12288, 1032, 33, 8, "runs"),
    (200, 4096, 1024, 8, 16, "runs"), (1100, 320, 136, 1, 40, "0"), (2200, 144, 72, 2, 128, "runs"),
    (1100, 16384, 64, 9, 24, "random"), (198, 5120, 80, 16, 32, "random"),
    (300, 4096, 1040, 6, 64, "random"), (130, 272, 136, 130, 8, "runs"),
    (1200, 256, 2048, 2, 16, "runs"), (90, 4096, 1024, 64, 32, "random"),
]


@pytest.mark.parametrize("M,K,N,L,R,mix", BACKWARD)
def test_backward(M, K, N, L, R, mix):
    say("backward", M, K, N, L, R, mix)
    c = make(M, K, N, L, R, mix)
    d = dev(c)
    _, h, plan = forward(d)
    xq, xs = aql.aql_act_checkpoint(d["x"])
    dx, dA, dB = backward(d, plan, h, xq, xs)
    torch.cuda.synchronize()
    (rx, tx), (rA, tA), (rB, tB) = ref_backward(c, h.cpu(), xq.cpu(), xs.cpu())
    close(dx, rx, tx, "dx", norm=4e-3)
    close(dA, rA, tA, "dA")
    close(dB, rB, tB, "dB")


@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (1, 4096, 2048), (7, 72, 48), (64, 64, 128),
                                   (65, 136, 400), (333, 2560, 960), (200, 200, 12304),
                                   (128, 11008, 256), (2500, 128, 2064), (1300, 64, 16384),
                                   (40, 0, 64), (3, 16456, 64), (2, 16384, 32), (300, 1032, 96)])
def test_dgrad(M, N, K):
    say("dgrad", M, N, K)
    c = make(M, K, N, 1, 8, "0")
    d = dev(c)
    dx = aql.aql_linear_w8a16_dgrad(d["dy"], d["q"], d["scale"])
    torch.cuda.synchronize()
    ref, T, off = ref_dgrad(c)
    close(dx, ref, 2.0 ** -8 * ref.abs() + (N + 4) * U * T + off, "dx", norm=4e-3)


def test_dgrad_of_rows_of_any_size():
    """Rows from 1e-38 to 1e38, zero rows, values 2^30 apart in a row."""
    M, N, K = 70, 264, 48
    c = make(M, K, N, 1, 8, "0")
    p = torch.linspace(-38, 33, M, dtype=torch.float64)
    dy = f64(workloads.randn(workloads.gen(9), M, N)) * 10.0 ** p[:, None]
    dy[::7] *= 2.0 ** torch.linspace(-30, 0, N, dtype=torch.float64)
    dy[5], dy[6, 1:] = 0.0, 0.0
    c["dy"] = dy.to(torch.float32).to(torch.bfloat16)
    d = dev(c)
    dx = aql.aql_linear_w8a16_dgrad(d["dy"], d["q"], d["scale"])
    torch.cuda.synchronize()
    ref, T, off = ref_dgrad(c)
    # plus bf16's subnormals (2^-134 the half step), and float32's in dy scale and the result
    tiny = 2.0 ** -134 + N * 127 * 2.0 ** -150 + 2.0 ** -149
    close(dx, ref, 2.0 ** -8 * ref.abs() + (N + 4) * U * T + off + tiny, "dx")


def test_dgrad_keeps_what_is_not_finite():
    """NaN of any payload and infinities in dy's rows, or in a scale, reach every dx
    they enter, and no other row."""
    for M, N, K in ((40, 264, 320), (600, 256, 16640)):
        c = make(M, K, N, 1, 8, "0")
        c["q"][c["q"] == 0] = 1
        d = dev(c)
        dx0 = aql.aql_linear_w8a16_dgrad(d["dy"], d["q"], d["scale"])
        d["dy"][3, 7], d["dy"][17, 200], d["dy"][M - 1, N - 1] = float("nan"), float("inf"), 1e38
        d["dy"].view(torch.int16)[5, 0] = 2 ** 15 - 1
        d["dy"].view(torch.int16)[6, 1] = -1
        d["dy"][20, :] = 0.0
        dx1 = aql.aql_linear_w8a16_dgrad(d["dy"], d["q"], d["scale"])
        bad = torch.zeros(M, dtype=torch.bool, device=DEV)
        bad[torch.tensor([3, 5, 6, 17], device=DEV)] = True
        assert not torch.isfinite(dx1[bad]).any()
        assert torch.isfinite(dx1[~bad]).all() and not dx1[20].any()
        same = ~bad
        same[20] = same[M - 1] = False
        assert torch.equal(dx0[same], dx1[same])
        for payload in (0x7fffffff, -1, 0x7f800001):
            d["scale"].view(torch.int32)[9] = payload
            assert torch.isnan(aql.aql_linear_w8a16_dgrad(d["dy"], d["q"], d["scale"])).all()


@pytest.mark.parametrize("M", [1, 5, 30, 100, 700])
def test_forward_keeps_what_is_not_finite(M):
    """A NaN of any payload in a row of x, in a scale or in alpha shows in every output."""
    c = make(M, 1024, 520, 3, 16, "runs")
    c["q"][c["q"] == 0] = 1
    for name, dt, payloads in (("x", torch.int16, (0x7fff, -1, 0x7f81)),
                               ("scale", torch.int32, (0x7fffffff, -1, 0x7f800001)),
                               ("alpha", torch.int32, (0x7fffffff, -1, 0x7f800001))):
        for p in payloads:
            d = dev(c)
            d[name].view(dt).view(-1)[0] = p
            y, h, _ = forward(d)
            torch.cuda.synchronize()
            if name == "scale":
                assert torch.isnan(y[:, 0]).all() and torch.isfinite(y[:, 1:]).all()
            else:
                rows = torch.zeros(M, dtype=torch.bool, device=DEV)
                rows[0 if name == "x" else slice(None)] = True
                if name == "alpha":
                    rows = d["idx"] == 0
                assert torch.isnan(y[rows]).all() and torch.isfinite(y[~rows]).all()
                assert torch.isnan(h[rows]).all() and torch.isfinite(h[~rows]).all()


def test_two_streams_share_a_plan():
    """Forward and backward of two layers on two streams at once, one plan."""
    c1, c2 = make(90, 2560, 960, 3, 16, "random", seed=1), make(90, 960, 2560, 3, 16, "random", seed=2)
    c2["idx"] = c1["idx"]
    ds = [dev(c1), dev(c2)]
    plan = aql.aql_lora_plan(ds[0]["idx"], 3)

    def step(d):
        y, h, _ = forward(d, plan)
        xq, xs = aql.aql_act_checkpoint(d["x"])
        return (y, h, *backward(d, plan, h, xq, xs))

    want = [step(d) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = step(ds[i])
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, g))


def test_backward_accumulates_and_leaves_out():
    c = make(100, 256, 136, 4, 16, "runs")
    c["idx"][c["idx"] == 2] = 1  # adapter 2: no rows
    d = dev(c)
    _, h, plan = forward(d)
    xq, xs = aql.aql_act_checkpoint(d["x"])
    dx, dA, dB = backward(d, plan, h, xq, xs)
    assert torch.equal(dA[2], torch.zeros_like(dA[2])) and torch.equal(dB[2], torch.zeros_like(dB[2]))
    a0, b0 = torch.randn_like(dA), torch.randn_like(dB)
    a1, b1 = a0.clone(), b0.clone()
    none, a2, b2 = backward(d, plan, h, xq, xs, dA=a1, dB=b1, accumulate=True, need_dx=False)
    assert none is None and a2 is a1 and b2 is b1
    assert torch.equal(a1, a0 + dA) and torch.equal(b1, b0 + dB)
    with pytest.raises(ValueError):
        backward(d, plan, h, xq, xs, accumulate=True)
    with pytest.raises(ValueError):
        backward(d, plan, h, xq, xs, dx=dx, need_dx=False)


def test_gradients_against_differences():
    """Central differences of sum(dy y) in 64 bits, x as its checkpoint holds it,
    along random directions: the function is linear in A, in B and in x, so a
    difference is exact up to rounding; the kernels' gradients agree within
    their tolerances summed against the direction's magnitudes."""
    c = make(48, 144, 72, 3, 16, "random")
    d = dev(c)
    xq, xs = aql.aql_act_checkpoint(d["x"])
    c["x"] = decoded(xq.cpu(), xs.cpu())
    plan = aql.aql_lora_plan(d["idx"], 3)
    h = torch.zeros(48, 16)
    al = [float(v) for v in c["alpha"]]

    def loss(x, A, B):
        y = (x @ f64(c["q"]).T) * f64(c["scale"])
        for a in range(3):
            r = rows_of(c, a)
            y[r] += al[a] * (x[r] @ A[a].T) @ B[a].T
        return float((y * f64(c["dy"])).sum())

    p = {"x": c["x"], "A": f64(c["A"]), "B": f64(c["B"])}
    for a in range(3):
        r = rows_of(c, a)
        h[r] = (al[a] * (p["x"][r] @ p["A"][a].T)).float()
    dx, dA, dB = backward(d, plan, h.to(DEV), xq, xs)
    (_, tx), (_, tA), (_, tB) = ref_backward(c, h, xq.cpu(), xs.cpu())
    g = workloads.gen(5)
    for name, got, tol in (("x", dx, tx), ("A", dA, tA), ("B", dB, tB)):
        v = torch.randn(p[name].shape, generator=g).double()
        up, down = dict(p), dict(p)
        up[name], down[name] = p[name] + 1e-3 * v, p[name] - 1e-3 * v
        diff = (loss(**up) - loss(**down)) / 2e-3
        slack = float((tol * v.abs()).sum()) + 1e-9 * abs(diff)
        # dB's reference h was rounded to float32 once
        slack += 2.0 ** -24 * float((f64(got.cpu()).abs() * v.abs()).sum()) * 48
        assert abs(float((got.double().cpu() * v).sum()) - diff) <= slack, name


# ---------------------------------------------------------------- checkpoints


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,K", [(1, 4), (3, 128), (5, 132), (1, 260), (37, 960), (64, 1020),
                                 (2, 14336), (1000, 512)])
def test_checkpoint(M, K, dt):
    say("checkpoint", M, K, dt)
    g = workloads.gen(M + K)
    x = workloads.randn(g, M, K)
    x[:, K // 2] *= 100.0
    x[M // 2, : min(K, 128)] = 0.0
    if M > 4:
        x[0] *= 1e-38   # subnormal scales
        x[1] *= 1e-44   # scales that round to 0 or to the smallest subnormal
        x[2] *= 1e36 if dt == torch.float32 else 1e34
    x = x.to(dt)
    xq, xs = aql.aql_act_checkpoint(x.to(DEV))
    out = aql.aql_act_restore(xq, xs, dt)
    other = aql.aql_act_restore(xq, xs, torch.bfloat16 if dt == torch.float32 else torch.float32)
    torch.cuda.synchronize()
    rq, rs = checkpoint_ref(x)
    assert torch.equal(xs.cpu(), rs)
    assert torch.equal(xq.cpu(), rq)
    exact = decoded(rq, rs).float()  # a product of 8 and 24 bits: one float32 rounding
    assert torch.equal((out if dt == torch.float32 else other).cpu(), exact)
    assert torch.equal((other if dt == torch.float32 else out).cpu(), exact.to(torch.bfloat16))


def test_checkpoint_past_32_bits():
    M, K = 528000, 4096  # 2.16e9 values
    x = torch.empty(M, K, dtype=torch.bfloat16, device=DEV)
    x.normal_(generator=torch.Generator(device=DEV).manual_seed(3))
    xq, xs = aql.aql_act_checkpoint(x)
    back = aql.aql_act_restore(xq, xs)
    for r in (0, 262143, 524287, 524289, M - 3):
        q1, s1 = aql.aql_act_checkpoint(x[r:r + 3].clone())
        assert torch.equal(xq[r:r + 3], q1) and torch.equal(xs[r:r + 3], s1)
        assert torch.equal(back[r:r + 3], aql.aql_act_restore(q1, s1))


def test_checkpoint_of_values_that_are_no_numbers():
    """A group with a NaN (of any payload) or an infinity restores without a finite
    value; every other group restores as without it."""
    for dt in (torch.float32, torch.bfloat16):
        x = workloads.randn(workloads.gen(4), 9, 400).to(dt)
        q0, s0 = aql.aql_act_checkpoint(x.to(DEV))
        b0, f0 = aql.aql_act_restore(q0, s0), aql.aql_act_restore(q0, s0, torch.float32)
        x[1, 5], x[2, 200], x[3, 399] = float("nan"), float("inf"), float("-inf")
        x[4, 128:256] = float("inf")
        i = x.view(torch.int32 if dt == torch.float32 else torch.int16)
        i[5, 0], i[6, 390] = (2 ** 31 - 1, -1) if dt == torch.float32 else (2 ** 15 - 1, -1)
        q1, s1 = aql.aql_act_checkpoint(x.to(DEV))
        b1, f1 = aql.aql_act_restore(q1, s1), aql.aql_act_restore(q1, s1, torch.float32)
        torch.cuda.synchronize()
        bad = torch.zeros(9, 512, dtype=torch.bool)
        for m, g in ((1, 0), (2, 1), (3, 3), (4, 1), (5, 0), (6, 3)):
            bad[m, 128 * g:128 * (g + 1)] = True
        bad = bad[:, :400].to(DEV)
        for v0, v1 in ((b0, b1), (f0, f1)):
            assert not torch.isfinite(v1[bad]).any()
            assert torch.equal(v0[~bad], v1[~bad])


# ------------------------------------------------------------ past 32 bits


def cut(c, rows, cols=None, ks=None):
    """The problem of some rows and of some output channels or inputs, on the CPU."""
    r = {"bias": None, "alpha": c["alpha"].cpu()}
    r["x"], r["dy"], r["idx"] = c["x"][rows].cpu(), c["dy"][rows].cpu(), c["idx"][rows].cpu()
    n = slice(None) if cols is None else cols
    k = slice(None) if ks is None else ks
    r["q"], r["scale"] = c["q"][n][:, k].cpu(), c["scale"][n].cpu()
    r["B"], r["A"] = c["B"][:, n].cpu(), c["A"][:, :, k].cpu()
    return r


def big(M, K, N, L, R):
    g = torch.Generator(device=DEV).manual_seed(M + K + N)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=DEV) * std).to(torch.bfloat16)
    return {"x": rnd(M, K), "dy": rnd(M, N, std=1e-2),
            "q": torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8),
            "scale": 1e-3 + 1e-3 * torch.rand(N, generator=g, device=DEV), "bias": None,
            "A": rnd(L, R, K, std=K ** -0.5), "B": rnd(L, N, R, std=0.02),
            "alpha": torch.ones(L, device=DEV),
            "idx": torch.randint(-1, L, (M,), generator=g, device=DEV, dtype=torch.int32)}


@pytest.mark.parametrize("L", [3, 6])  # walked in the tiles, and products given
def test_outputs_past_32_bits(L):
    M, K, N, R = 2100, 16, 1050001, 8  # y: 2.2e9 values
    say("outputs", L)
    d = big(M, K, N, L, R)
    y, h, _ = forward(d)
    torch.cuda.synchronize()
    rows = torch.tensor([0, 1, 1022, 1023, 1024, 2047, M - 1], device=DEV)
    cols = torch.cat([torch.arange(40), torch.arange(N - 300, N)]).to(DEV)
    c = cut(d, rows, cols)
    yr, ytol, hr, htol = ref_forward(c)
    close(h[rows], hr, htol, "h")
    close(y[rows][:, cols], yr, ytol, "y", norm=4e-3)


def test_weights_past_32_bits():
    M, K, N, L, R = 70, 65552, 65600, 2, 8  # q: 4.3e9 bytes
    say("weights")
    d = big(M, K, N, L, R)
    _, h, plan = forward(d)
    xq, xs = aql.aql_act_checkpoint(d["x"])
    dx, dA, dB = backward(d, plan, h, xq, xs)
    alone = aql.aql_linear_w8a16_dgrad(d["dy"], d["q"], d["scale"])
    torch.cuda.synchronize()
    rows = torch.tensor([0, 63, 64, M - 1], device=DEV)
    ks = torch.cat([torch.arange(16), torch.arange(K - 128, K)]).to(DEV)
    c = cut(d, rows, ks=ks)
    ref, T, off = ref_dgrad(c)
    close(alone[rows][:, ks], ref, 2.0 ** -8 * ref.abs() + (N + 4) * U * T + off, "dx", norm=4e-3)
    tol = torch.zeros_like(ref)
    for i, a in enumerate(c["idx"].tolist()):
        if a < 0:
            continue
        A, B, dy = f64(c["A"][a]), f64(c["B"][a]), f64(c["dy"][i])
        u, ue = dy @ B, (N + 3) * U * (dy.abs() @ B.abs())
        ref[i] += u @ A
        T[i] += u.abs() @ A.abs()
        tol[i] += (ue + 2.0 ** -16 * u.abs()) @ A.abs()
    tol += off + 2.0 ** -8 * ref.abs() + (N + R + 4) * U * T
    close(dx[rows][:, ks], ref, tol, "dx with adapters", norm=4e-3)


def test_most_rows():
    M, K, N, L, R = 1048560, 16, 24, 1024, 8
    say("rows")
    d = big(M, K, N, L, R)
    y, h, plan = forward(d)
    xq, xs = aql.aql_act_checkpoint(d["x"])
    dx, dA, dB = backward(d, plan, h, xq, xs)
    torch.cuda.synchronize()
    rows = torch.cat([torch.arange(200), torch.arange(M - 200, M)]).to(DEV)
    c = cut(d, rows)
    yr, ytol, hr, htol = ref_forward(c)
    close(h[rows], hr, htol, "h")
    close(y[rows], yr, ytol, "y", norm=4e-3)
    (rx, tx), _, _ = ref_backward(c, h[rows].cpu(), xq[rows].cpu(), xs[rows].cpu())
    close(dx[rows], rx, tx, "dx", norm=4e-3)
    for a in (0, 511, 1023):  # every row of these adapters
        one = (d["idx"] == a).nonzero()[:, 0]
        c = cut(d, one)
        _, (rA, tA), (rB, tB) = ref_backward(c, h[one].cpu(), xq[one].cpu(), xs[one].cpu())
        close(dA[a], rA[a], tA[a], "dA")
        close(dB[a], rB[a], tB[a], "dB")


# ------------------------------------------------------------------- together


def test_training_step_of_an_mlp():
    """Checkpoint, forward and backward of a SmolVLM-size up projection feeding a
    down projection, three adapters in the batch, then one update of them: the
    chain's gradients against 64 bits on the same intermediate values."""
    M, L, R = 200, 3, 16
    up = make(M, 960, 2560, L, R, "runs", seed=1)
    down = make(M, 2560, 960, L, R, "runs", seed=2)
    u, d = dev(up), dev(down)
    plan = aql.aql_lora_plan(u["idx"], L)
    ck1 = aql.aql_act_checkpoint(u["x"])
    y1, h1, _ = forward(u, plan)
    act = torch.relu(y1)
    d["x"] = act
    down["x"] = act.cpu()
    ck2 = aql.aql_act_checkpoint(act)
    y2, h2, _ = forward(d, plan)
    d["dy"] = (y2.float() * 1e-3).to(torch.bfloat16)
    down["dy"] = d["dy"].cpu()
    da, dA2, dB2 = backward(d, plan, h2, *ck2)
    u["dy"] = torch.where(act > 0, da, torch.zeros_like(da))
    up["dy"] = u["dy"].cpu()
    dx, dA1, dB1 = backward(u, plan, h1, *ck1)
    new = [(p.float() - 0.1 * g).to(torch.bfloat16)
           for p, g in ((u["A"], dA1), (u["B"], dB1), (d["A"], dA2), (d["B"], dB2))]
    torch.cuda.synchronize()
    y, ytol, h, htol = ref_forward(down)
    close(y2, y, ytol, "y2", norm=4e-3)
    for c, h, ck, got in ((down, h2, ck2, (da, dA2, dB2)), (up, h1, ck1, (dx, dA1, dB1))):
        refs = ref_backward(c, h.cpu(), ck[0].cpu(), ck[1].cpu())
        for name, g, (ref, tol) in zip(("dx", "dA", "dB"), got, refs):
            close(g, ref, tol, name, norm=4e-3)
    assert all(torch.isfinite(t).all() for t in new)


@pytest.mark.parametrize("M", [1, 20, 200])
def test_repeats_bit_for_bit_and_on_a_side_stream(M):
    c = make(M, 2560, 960, 4, 32, "random")
    d = dev(c)
    y, h, plan = forward(d)
    xq, xs = aql.aql_act_checkpoint(d["x"])
    g = backward(d, plan, h, xq, xs)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y2, h2, plan2 = forward(d)
        xq2, xs2 = aql.aql_act_checkpoint(d["x"])
        g2 = backward(d, plan2, h2, xq2, xs2)
    s.synchronize()
    for a, b in zip((y, h, xq, xs, *g), (y2, h2, xq2, xs2, *g2)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M", [3, 150])
def test_graph_replays_with_a_new_batch(M):
    """One captured graph of plan, forward, checkpoint and backward, replayed with
    new rows, adapters and gradients in its inputs, eager work between."""
    L, R = 4, 16
    c = make(M, 512, 264, L, R, "random")
    d = dev(c)
    plan = aql.aql_lora_plan(d["idx"], L)
    kw = dict(y=torch.empty(M, 264, dtype=torch.bfloat16, device=DEV),
              h=torch.empty(M, R, device=DEV))
    out = dict(dx=torch.empty(M, 512, dtype=torch.bfloat16, device=DEV),
               dA=torch.empty(L, R, 512, device=DEV), dB=torch.empty(L, 264, R, device=DEV),
               workspace=torch.empty(aql.aql_lora_backward_bytes(M, 264, 512, L, R), dtype=torch.uint8,
                                     device=DEV))
    xq, xs = aql.aql_act_checkpoint(d["x"])

    def step():
        aql.aql_lora_plan(d["idx"], L, plan)
        forward(d, plan, **kw)
        aql.aql_act_checkpoint(d["x"], xq, xs)
        backward(d, plan, kw["h"], xq, xs, **out)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        n = dev(make(M, 512, 264, L, R, "random", seed=10 + i))
        for k in ("x", "dy", "idx"):
            d[k].copy_(n[k])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (kw["y"], kw["h"], xq, xs, out["dx"], out["dA"], out["dB"])]
        y, h, p = forward(d)
        eq, es = aql.aql_act_checkpoint(d["x"])
        for a, b in zip(got, (y, h, eq, es, *backward(d, p, h, eq, es))):
            assert torch.equal(a, b), i


def test_a_plan_serves_only_its_batch():
    d = dev(make(8, 64, 32, 2, 8, "runs"))
    plan = aql.aql_lora_plan(d["idx"], 2)
    d2 = dev(make(9, 64, 32, 2, 8, "runs"))
    with pytest.raises(ValueError):
        forward(d2, plan)
    with pytest.raises(ValueError):
        aql.aql_lora_plan(d2["idx"], 2, plan)
    with pytest.raises(TypeError):
        forward(d, plan.buffer)


def test_empty_batches():
    d = dev(make(0, 64, 32, 2, 8, "none"))
    y, h, plan = forward(d)
    assert y.shape == (0, 32) and h.shape == (0, 8)
    xq, xs = aql.aql_act_checkpoint(d["x"])
    dx, dA, dB = backward(d, plan, h, xq, xs)
    assert dx.shape == (0, 64) and not dA.any() and not dB.any()
    a, b = torch.ones_like(dA), torch.ones_like(dB)
    backward(d, plan, h, xq, xs, dA=a, dB=b, accumulate=True)
    assert (a == 1).all() and (b == 1).all()
    # no output channels: the input's gradient is zero, dA too
    d = dev(make(5, 64, 0, 2, 8, "runs"))
    plan = aql.aql_lora_plan(d["idx"], 2)
    xq, xs = aql.aql_act_checkpoint(d["x"])
    dx, dA, dB = backward(d, plan, torch.zeros(5, 8, device=DEV), xq, xs)
    assert not dx.any() and not dA.any() and dB.shape == (2, 0, 8)
    for M, K in ((5, 64), (20, 8192), (100, 512), (100, 8192)):  # h has a value all the same
        c = make(M, K, 0, 2, 8, "runs")
        y, h, _ = forward(dev(c))
        torch.cuda.synchronize()
        _, _, hr, htol = ref_forward(c)
        assert y.shape == (M, 0)
        close(h, hr, htol, "h")


def test_one_workspace_serves_smaller_batches():
    """Buffers sized for the largest batch, filled with what no sum may take in, under
    batches on both sides of the forms' edges; K and N split at some of them."""
    N, K, L, R, most = 4096, 8192, 5, 8, 2048
    full = dev(make(most, K, N, L, R, "random"))
    fw = torch.empty(aql.aql_lora_forward_bytes(most, N, K, L, R), dtype=torch.uint8, device=DEV)
    bw = torch.empty(aql.aql_lora_backward_bytes(most, N, K, L, R), dtype=torch.uint8, device=DEV)
    dw = torch.empty(aql.aql_workspace_bytes(aql.AQL_OP_W8A16_DGRAD, most, N, K), dtype=torch.uint8,
                     device=DEV)
    for M in (2048, 1100, 512, 300, 130, 64, 63, 20, 1):
        say("M", M)
        d = dict(full, **{k: full[k][:M].contiguous() for k in ("x", "dy", "idx")})
        y, h, plan = forward(d)
        xq, xs = aql.aql_act_checkpoint(d["x"])
        want = (y, h, *backward(d, plan, h, xq, xs), aql.aql_linear_w8a16_dgrad(d["dy"], d["q"], d["scale"]))
        for w in (fw, bw, dw):
            w.fill_(0xff)
        y, h, _ = forward(d, plan, workspace=fw)
        got = (y, h, *backward(d, plan, h, xq, xs, workspace=bw),
               aql.aql_linear_w8a16_dgrad(d["dy"], d["q"], d["scale"], workspace=dw))
        for a, b in zip(got, want):
            assert torch.equal(a, b), M


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_checkpoint_of_more_groups_than_a_launch_takes(dt):
    """2^30 + 5 rows of 4: more threads than a grid may have. Blocks of 2^20 rows hold
    the same numbers times a power of two, so codes repeat and scales follow it."""
    n, reps, tail = 1 << 20, 1 << 10, 5
    M = n * reps + tail
    g = torch.Generator(device=DEV).manual_seed(5)
    block = torch.randn(n, 4, generator=g, device=DEV).to(dt)
    bq, bs = aql.aql_act_checkpoint(block)
    power = (2.0 ** (torch.arange(reps, device=DEV) % 16))
    x = torch.empty(M, 4, dtype=dt, device=DEV)
    for i in range(reps):
        torch.mul(block, float(2 ** (i % 16)), out=x[i * n:(i + 1) * n])
    x[n * reps:] = block[:tail]
    xq, xs = aql.aql_act_checkpoint(x)
    say("saved", M)
    body = n * reps
    assert (xq[:body].view(reps, -1) == bq.view(1, -1)).all() and torch.equal(xq[body:], bq[:tail])
    assert (xs[:body].view(reps, n) == bs.view(1, n) * power[:, None]).all()
    assert torch.equal(xs[body:], bs[:tail])
    want = aql.aql_act_restore(bq, bs, dt)
    x.zero_()
    aql.aql_act_restore(xq, xs, dt, x)
    say("restored")
    for i in range(0, reps, 31):
        assert torch.equal(x[i * n:(i + 1) * n], want * float(2 ** (i % 16))), i
    assert torch.equal(x[(reps - 1) * n:body], want * float(2 ** ((reps - 1) % 16)))
    assert torch.equal(x[body:], want[:tail])


def test_products_of_more_tiles_than_a_launch_takes():
    """1089 tiles of the plan by 15470 blocks of columns are more threads than one grid
    may have (1024 adapters of 8 ranks, 3.96e6 channels: B holds 65 GB)."""
    M, K, N, L, R = 1025, 16, 3960001, 1024, 8
    g = torch.Generator(device=DEV).manual_seed(8)
    B = torch.empty(L, N, R, dtype=torch.bfloat16, device=DEV).normal_(0, 0.02, generator=g)
    c = make(M, K, 8, L, R, "random")
    perm = torch.randperm(M, generator=workloads.gen(6))
    c["idx"] = (perm - 1).to(torch.int32)  # an adapter for every row but one
    d = dev(c)
    d["q"] = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    d["scale"] = torch.rand(N, generator=g, device=DEV) * 1e-3
    d["B"] = B
    say("start", M, N, L)
    y, h, _ = forward(d)
    torch.cuda.synchronize()
    cols = torch.cat([torch.randint(0, N, (60,), generator=workloads.gen(7)),
                      torch.tensor([0, 255, 256, N - 257, N - 2, N - 1])])
    at = cols.to(DEV)
    part = dict(c, q=d["q"][at].cpu(), scale=d["scale"][at].cpu(), B=B[:, at].cpu())
    ry, tol, rh, htol = ref_forward(part)
    close(h, rh, htol, "h")
    close(y[:, at], ry, tol, "y", norm=4e-3)


# a sum of splits beside the weight gradients, alone and with the products given
# ahead; no split
SUBSETS = [(63, 960, 2560, 2, 8), (300, 4096, 1040, 6, 64), (100, 256, 136, 4, 16)]


@pytest.mark.parametrize("M,K,N,L,R", SUBSETS)
def test_backward_of_some_outputs(M, K, N, L, R):
    """Each subset of dx, dA and dB. dx does not depend on the others to the bit; the
    weight gradients' sums may take another order, so they go by their bounds."""
    c = make(M, K, N, L, R, "random")
    d = dev(c)
    _, h, plan = forward(d)
    xq, xs = aql.aql_act_checkpoint(d["x"])
    dx, _, _ = backward(d, plan, h, xq, xs)
    refs = ref_backward(c, h.cpu(), xq.cpu(), xs.cpu())
    for bits in range(8):
        need = dict(need_dx=bool(bits & 1), need_dA=bool(bits & 2), need_dB=bool(bits & 4))
        say(M, K, N, L, R, need)
        ck = (xq, xs) if need["need_dA"] else (None, None)
        got = backward(d, plan, h, *ck, **need)
        for name, g, (ref, tol) in zip(("dx", "dA", "dB"), got, refs):
            assert (g is not None) == need["need_" + name]
            if g is not None:
                close(g, ref, tol, name)
        assert got[0] is None or torch.equal(got[0], dx)
    a = torch.empty(L, R, K, device=DEV)
    for kw in (dict(need_dA=False, dA=a), dict(need_dB=False, dB=torch.empty(L, N, R, device=DEV)),
               dict(accumulate=True, dA=a), dict(accumulate=True, need_dA=False)):
        with pytest.raises(ValueError):
            backward(d, plan, h, xq, xs, **kw)
    with pytest.raises(TypeError):
        backward(d, plan, h, None, None)


@pytest.mark.parametrize("M,K,N,L,R", SUBSETS)
def test_backward_accumulates_in_every_form(M, K, N, L, R):
    c = make(M, K, N, L, R, "random")
    c["idx"][c["idx"] == 1] = -1  # adapter 1: no rows
    d = dev(c)
    _, h, plan = forward(d)
    xq, xs = aql.aql_act_checkpoint(d["x"])
    dx, dA, dB = backward(d, plan, h, xq, xs)
    assert not dA[1].any() and not dB[1].any()
    a0, b0 = torch.randn_like(dA), torch.randn_like(dB)
    for need_dx in (True, False):
        _, sA, sB = backward(d, plan, h, xq, xs, need_dx=need_dx)
        a, b = a0.clone(), b0.clone()
        got = backward(d, plan, h, xq, xs, dA=a, dB=b, accumulate=True, need_dx=need_dx)
        assert got[1] is a and got[2] is b
        assert torch.equal(a, a0 + sA) and torch.equal(b, b0 + sB)
        assert torch.equal(got[0], dx) if need_dx else got[0] is None
    _, onlyA, _ = backward(d, plan, h, xq, xs, need_dx=False, need_dB=False)
    a = a0.clone()
    backward(d, plan, h, xq, xs, dA=a, accumulate=True, need_dx=False, need_dB=False)
    assert torch.equal(a, a0 + onlyA)


def test_empty_backward_of_some_outputs():
    d = dev(make(0, 64, 32, 2, 8, "none"))
    _, h, plan = forward(d)
    dx, dA, dB = backward(d, plan, h, None, None, need_dA=False)
    assert dx.shape == (0, 64) and dA is None and not dB.any()
    assert backward(d, plan, h, None, None, need_dA=False, need_dB=False, need_dx=False) == (None,) * 3
