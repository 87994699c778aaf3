"""Refusals of the low-rank adapter and 8-bit checkpoint entry points without a
GPU: every invalid argument gets the documented status before any HIP call
(fake device addresses are never touched), and empty problems launch nothing."""
import ctypes as C

import pytest
import torch

import activation_quantized_linear_amd as aql

P = C.c_void_p(0x10000)    # fake, 16-byte aligned, never dereferenced
MIS = C.c_void_p(0x10004)  # misaligned
L = aql._lib
BIG = 1 << 40

OK, NULL, SHAPE, ALIGN, PARAM, WS = (aql.AQL_OK, aql.AQL_ERR_NULL, aql.AQL_ERR_SHAPE,
                                     aql.AQL_ERR_ALIGN, aql.AQL_ERR_PARAM, aql.AQL_ERR_WORKSPACE)


def call(fn, defaults, **kw):
    args = dict(defaults)
    for k, v in kw.items():
        assert k in args, k
        args[k] = v
    return fn(*args.values())


def plan(**kw):
    return call(L.aql_lora_plan, dict(idx=P, M=5, L=3, plan=P, plan_bytes=BIG, stream=None), **kw)


def test_plan_bytes():
    b = aql.aql_lora_plan_bytes
    assert b(0, 1) > 0 and b(1, 1) > 0
    # idx, 16 positions and an owner a tile: M / 16 + min(M, L + 1) tiles
    assert b(1000, 7) >= 4 * (1000 + 17 * (1000 // 16 + 8) + 8)
    for M, A in ((-1, 1), (1, 0), (1, 1025), (1048561, 1)):
        assert b(M, A) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), SHAPE), (dict(M=1048561), SHAPE), (dict(L=0), SHAPE), (dict(L=1025), SHAPE),
    (dict(idx=None), NULL), (dict(plan=None), NULL), (dict(idx=MIS), ALIGN),
    (dict(plan=MIS), ALIGN), (dict(plan_bytes=64), WS)])
def test_plan_refusals(kw, code):
    assert plan(**kw) == code
    assert "aql_lora_plan" in aql.aql_last_error()


FWD = dict(x=P, M=5, K=64, q=P, scale=P, bias=None, N=24, A=P, B=P, alpha=P, L=3, R=8, plan=P, y=P,
           h=P, ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=8), SHAPE), (dict(K=40), SHAPE),
    (dict(R=0), SHAPE), (dict(R=12), SHAPE), (dict(R=136), SHAPE), (dict(L=0), SHAPE),
    (dict(L=1025), SHAPE)]
    + [({k: None}, NULL) for k in ("x", "q", "scale", "A", "B", "alpha", "plan", "y", "h")]
    + [({k: MIS}, ALIGN) for k in ("x", "q", "scale", "bias", "A", "B", "alpha", "plan", "y", "h",
                                   "ws")])
def test_forward_refusals(kw, code):
    assert call(L.aql_linear_w8a16_lora, FWD, **kw) == code


def test_forward_workspace():
    wb = aql.aql_lora_forward_bytes
    assert wb(1, 4096, 4096, 2, 16) == 0                      # one row: nothing to split
    need = wb(100, 72, 8192, 3, 16)
    assert need >= aql.aql_workspace_bytes(aql.AQL_OP_W8A16, 100, 72, 8192) > 0
    big = dict(M=100, N=72, K=8192, R=16)
    assert call(L.aql_linear_w8a16_lora, FWD, **big) == WS
    assert call(L.aql_linear_w8a16_lora, FWD, ws=P, ws_bytes=need - 1, **big) == WS
    for bad in ((0, 72, 64, 3, 16), (5, -1, 64, 3, 16), (5, 72, 8, 3, 16), (5, 72, 64, 0, 16),
                (5, 72, 64, 3, 12)):
        assert wb(*bad) == 0


def test_forward_empty():
    none = {k: None for k in ("x", "y", "h")}
    assert call(L.aql_linear_w8a16_lora, FWD, M=0, **none) == OK
    # no output channels: h is still to be computed
    assert call(L.aql_linear_w8a16_lora, FWD, N=0, q=None, scale=None, y=None, B=None,
                x=None) == NULL
    assert call(L.aql_linear_w8a16_lora, FWD, N=0, q=None, scale=None, y=None, B=None,
                h=None) == NULL


DG = dict(dy=P, M=5, N=24, q=P, scale=P, K=64, dx=P, ws=P, ws_bytes=BIG, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), SHAPE), (dict(M=1048561), SHAPE), (dict(N=-8), SHAPE), (dict(N=12), SHAPE),
    (dict(N=(1 << 22) + 8), SHAPE), (dict(K=0), SHAPE), (dict(K=24), SHAPE),
    (dict(K=(1 << 24) + 16), SHAPE), (dict(ws=None), WS), (dict(ws_bytes=5 * 64 * 2), WS)]
    + [({k: None}, NULL) for k in ("dy", "q", "scale", "dx")]
    + [({k: MIS}, ALIGN) for k in ("dy", "q", "scale", "dx", "ws")])
def test_dgrad_refusals(kw, code):
    assert call(L.aql_linear_w8a16_dgrad, DG, **kw) == code


def test_dgrad_empty_and_workspace():
    assert call(L.aql_linear_w8a16_dgrad, DG, M=0, dy=None, dx=None) == OK
    wb = lambda M, N, K: L.aql_workspace_bytes(aql.AQL_OP_W8A16_DGRAD, M, N, K)
    # the scaled dy in float16 and an exponent a row, nothing else where no sum is split
    assert wb(2048, 11008, 4096) == 2048 * 11008 * 2 + 2048 * 4
    assert wb(64, 4096, 4096) > 64 * 4096 * 2 + 64 * 4 + 64 * 4096 * 4
    assert wb(-1, 16, 16) == 0 and wb(0, 16, 16) == 0 and wb(1 << 21, 16, 16) == 0


BWD = dict(dy=P, M=5, N=24, q=P, scale=P, K=64, A=P, B=P, alpha=P, L=3, R=8, plan=P, h=P, xq=P,
           xs=P, accumulate=0, dx=P, dA=P, dB=P, ws=P, ws_bytes=BIG, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), SHAPE), (dict(N=12), SHAPE), (dict(K=24), SHAPE), (dict(R=4), SHAPE),
    (dict(R=132), SHAPE), (dict(L=0), SHAPE), (dict(L=1025), SHAPE), (dict(ws=None), WS),
    (dict(ws_bytes=16), WS)]
    + [({k: None}, NULL) for k in ("dy", "q", "scale", "A", "B", "alpha", "plan", "h", "xq", "xs")]
    + [({k: MIS}, ALIGN) for k in ("dy", "q", "scale", "A", "B", "alpha", "plan", "h", "xq", "xs",
                                   "dx", "dA", "dB", "ws")])
def test_backward_refusals(kw, code):
    assert call(L.aql_linear_w8a16_lora_backward, BWD, **kw) == code


def test_backward_nothing_asked_for():
    assert call(L.aql_linear_w8a16_lora_backward, BWD, dx=None, dA=None, dB=None) == OK
    assert aql.aql_lora_backward_bytes(0, 24, 64, 3, 8) == 0
    assert aql.aql_lora_backward_bytes(5, 24, 64, 3, 8) >= 5 * 8 * 4 + 5 * 64 * 2


CK = dict(x=P, dtype=0, M=5, K=64, xq=P, xs=P, stream=None)
RS = dict(xq=P, xs=P, M=5, K=64, x=P, dtype=0, stream=None)


@pytest.mark.parametrize("fn,base", [("aql_act_checkpoint", CK), ("aql_act_restore", RS)])
def test_checkpoint_refusals(fn, base):
    f = getattr(L, fn)
    assert call(f, base, dtype=2) == PARAM
    for kw in (dict(M=-1), dict(K=0), dict(K=6), dict(M=1 << 37)):
        assert call(f, base, **kw) == SHAPE
    for k in ("x", "xq", "xs"):
        assert call(f, base, **{k: None}) == NULL
        assert call(f, base, **{k: MIS}) == ALIGN
    assert call(f, base, M=0, x=None, xq=None, xs=None) == OK


def test_binding_refuses_host_tensors():
    idx = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        aql.aql_lora_plan(idx, 2)
    with pytest.raises(TypeError):
        aql.aql_lora_plan(idx.long(), 2)
    with pytest.raises(ValueError):
        aql.aql_act_checkpoint(torch.zeros(4, 16))
    with pytest.raises(TypeError):
        aql.aql_act_checkpoint(torch.zeros(4, 16, dtype=torch.float16))


def test_arguments_that_are_no_tensors():
    x = torch.zeros(2, 16, dtype=torch.bfloat16)
    for f in (lambda: aql.aql_act_checkpoint(None), lambda: aql.aql_act_restore(None, None),
              lambda: aql.aql_lora_plan([0, 1], 2),
              lambda: aql.aql_linear_w8a16_dgrad(None, None, None),
              lambda: aql.aql_linear_w8a16_lora(None, *[None] * 6)):
        with pytest.raises(TypeError):
            f()
    for f in (lambda: aql.aql_act_checkpoint(x), lambda: aql.aql_lora_plan(x[0].int(), 2),
              lambda: aql.aql_linear_w8a16_dgrad(x, x, x)):
        with pytest.raises(ValueError, match="device tensor"):
            f()


# Rows at and around every change of tiles, splits and forms.
EDGES = sorted({m + d for m in (1, 12, 16, 32, 48, 64, 128, 192, 256, 320, 384, 448, 512, 576, 640,
                                768, 1024, 1280, 2048, 2560, 4096, 8192) for d in (-1, 0, 1)
                if m + d > 0} | set(range(1, 300, 7)) | {5000, 20480, 1048560})
SIZES = [(4096, 14336, 1, 16), (4096, 4096, 1, 16), (14336, 4096, 8, 16), (4096, 14336, 3, 64),
         (2560, 960, 2, 8), (960, 2560, 5, 128), (16, 8192, 1, 8), (64, 65536, 64, 32),
         (4096, 4096, 1024, 128), (4096, 16, 6, 8), (12288, 1 << 23, 5, 8)]


@pytest.mark.parametrize("N,K,A,R", SIZES)
def test_a_workspace_of_a_large_batch_serves_smaller_ones(N, K, A, R):
    """Sized once, for the most rows: no smaller batch may need more."""
    fwd = [aql.aql_lora_forward_bytes(M, N, K, A, R) for M in EDGES]
    dg = [aql.aql_workspace_bytes(aql.AQL_OP_W8A16_DGRAD, M, N, K) for M in EDGES]
    bwd = [aql.aql_lora_backward_bytes(M, N, K, A, R) for M in EDGES]
    for need in (fwd, dg, bwd):
        assert need == sorted(need)
    for top in (len(EDGES) - 1, EDGES.index(2048)):
        for i in range(top + 1):
            kw = dict(M=EDGES[i], N=N, K=K)
            assert call(L.aql_linear_w8a16_lora, FWD, L=A, R=R, ws=P, ws_bytes=fwd[top], **kw) != WS
            assert call(L.aql_linear_w8a16_dgrad, DG, ws_bytes=dg[top], **kw) != WS
            assert call(L.aql_linear_w8a16_lora_backward, BWD, L=A, R=R, ws_bytes=bwd[top],
                        **kw) != WS


def test_forward_channels():
    """More channels than one grid of the streaming kernels holds are refused."""
    wide = dict(N=(1 << 26) + 1)
    assert aql.aql_lora_forward_bytes(5, 1 << 26, 64, 3, 8) == 0  # few rows need none
    assert aql.aql_lora_forward_bytes(64, 1 << 26, 64, 5, 8) > 0
    assert aql.aql_lora_forward_bytes(64, wide["N"], 64, 5, 8) == 0
    assert call(L.aql_linear_w8a16_lora, FWD, **wide) == SHAPE
    assert "N <= 67108864" in aql.aql_last_error()
    assert call(L.aql_linear_w8a16_lora, FWD, N=1 << 26) != SHAPE
