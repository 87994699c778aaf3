"""Refusals of the KV cache, attention and activation-epilogue entry points without a GPU:
every invalid argument gets the documented status before any HIP call (fake device
addresses are never touched), and empty problems launch nothing."""
import ctypes as C
import math

import pytest
import torch

import activation_quantized_linear_amd as aql

P = C.c_void_p(0x10000)    # fake, 16-byte aligned, never dereferenced
P2 = C.c_void_p(0x20000)
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


SIZES = [dict(T=-1), dict(T=(1 << 20) + 1), dict(S=-1), dict(S=4097), dict(W=0), dict(W=(1 << 20) + 1),
         dict(Hkv=0), dict(Hkv=3), dict(Hq=0), dict(Hq=1025, Hkv=1), dict(Hkv=16), dict(most=0),
         dict(most=(1 << 20) + 1)]
PLAN = dict(cu=P, pos=P, T=9, S=3, Hq=8, Hkv=2, W=5, most=4, window=0, plan=P, plan_bytes=BIG, stream=None)


@pytest.mark.parametrize("kw,code", [(k, SHAPE) for k in SIZES] + [
    (dict(window=-1), SHAPE), (dict(window=(1 << 30) + 1), SHAPE), (dict(cu=None), NULL),
    (dict(pos=None), NULL), (dict(plan=None), NULL), (dict(cu=MIS), ALIGN), (dict(pos=MIS), ALIGN),
    (dict(plan=MIS), ALIGN), (dict(plan_bytes=64), WS)])
def test_plan_refusals(kw, code):
    assert call(L.aql_kv_plan, PLAN, **kw) == code
    assert "aql_kv_plan" in aql.aql_last_error()


def test_bytes():
    b, w = aql.aql_kv_plan_bytes, aql.aql_attention_kv8_bytes
    assert b(0, 0, 8, 2, 5, 4) > 0
    # a piece of 32 bytes for each page that new tokens touch, a unit for each 128 rows
    assert b(1 << 16, 7, 8, 2, 5000, 1 << 14) >= 32 * ((1 << 16) // 64 + 2 * 7) + 32 * (1 << 16) * 4 // 128
    for bad in SIZES:
        z = dict(T=9, S=3, Hq=8, Hkv=2, W=5, most=4)
        z.update(bad)
        assert b(*z.values()) == 0
        assert w(z["T"], z["S"], z["Hq"], z["Hkv"], 64, z["W"], z["most"]) == 0
    for D in (0, 4, 12, 264):
        assert w(9, 3, 8, 2, D, 50, 4) == 0
    assert w(1, 1, 8, 2, 64, 4, 1) == 0       # nothing to spread over several units
    assert w(1, 1, 8, 2, 64, 400, 1) > 0


CACHE = dict(kq=P, vq=P, ks=P, vs=P, P=10)
WRITE = dict(k=P, krow=128, v=P, vrow=128, dtype=aql.AQL_BF16, T=9, S=3, Hq=8, Hkv=2, D=64, table=P, W=5, most=4,
             plan=P, kq=P, vq=P, ks=P, vs=P, P=10, stream=None)
READ = dict(kq=P, vq=P, ks=P, vs=P, P=10, T=9, S=3, Hq=8, Hkv=2, D=64, table=P, W=5, most=4, plan=P, k=P, v=P,
            dtype=aql.AQL_BF16, stream=None)
ATT = dict(q=P, qrow=512, T=9, S=3, Hq=8, Hkv=2, D=64, sm_scale=0.1, window=0, kq=P, vq=P, ks=P, vs=P, P=10, table=P,
           W=5, most=4, plan=P, y=P, lse=None, ws=P, ws_bytes=BIG, stream=None)
COMMON = ([(k, SHAPE) for k in SIZES]
          + [(dict(D=d), SHAPE) for d in (0, 4, 12, 264)] + [(dict(P=0), SHAPE), (dict(P=1 << 31), SHAPE)]
          + [({k: None}, NULL) for k in ("kq", "vq", "ks", "vs", "table", "plan")]
          + [({k: MIS}, ALIGN) for k in ("kq", "vq", "ks", "vs", "table", "plan")])


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(dtype=2), PARAM), (dict(krow=120), SHAPE), (dict(vrow=120), SHAPE), (dict(krow=132), SHAPE),
    (dict(krow=130, dtype=aql.AQL_F32), SHAPE), (dict(k=None), NULL), (dict(v=None), NULL), (dict(k=MIS), ALIGN),
    (dict(v=MIS), ALIGN)])
def test_write_refusals(kw, code):
    assert call(L.aql_kv_cache_write, WRITE, **kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(dtype=2), PARAM), (dict(k=None), NULL), (dict(v=None), NULL), (dict(k=MIS), ALIGN), (dict(v=MIS), ALIGN)])
def test_read_refusals(kw, code):
    assert call(L.aql_kv_cache_read, READ, **kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(sm_scale=0.0), PARAM), (dict(sm_scale=-1.0), PARAM), (dict(sm_scale=math.inf), PARAM),
    (dict(sm_scale=math.nan), PARAM), (dict(window=-1), SHAPE), (dict(qrow=504), SHAPE), (dict(qrow=516), SHAPE),
    (dict(q=None), NULL), (dict(y=None), NULL), (dict(q=MIS), ALIGN), (dict(y=MIS), ALIGN), (dict(lse=MIS), ALIGN),
    (dict(ws=MIS), ALIGN), (dict(ws=None, W=500), WS), (dict(ws_bytes=64, W=500), WS)])
def test_attention_refusals(kw, code):
    assert call(L.aql_attention_kv8, ATT, **kw) == code


@pytest.mark.parametrize("kw", [dict(T=0), dict(S=0)])
def test_empty_steps(kw):
    none = dict(kq=None, vq=None, ks=None, vs=None, table=None, plan=None, **kw)
    assert call(L.aql_kv_cache_write, WRITE, k=None, v=None, **none) == OK
    assert call(L.aql_kv_cache_read, READ, k=None, v=None, **none) == OK
    assert call(L.aql_attention_kv8, ATT, q=None, y=None, ws=None, ws_bytes=0, **none) == OK


LIN = dict(x=P, M=5, K=64, q=P, scale=P, bias=None, N=24, act=4, mul=None, residual=None, pre=None, y=P, ws=None,
           ws_bytes=0, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=8), SHAPE), (dict(K=40), SHAPE), (dict(act=-1), PARAM),
    (dict(act=5), PARAM), (dict(pre=P), PARAM)]
    + [({k: None}, NULL) for k in ("x", "q", "scale", "y")]
    + [({k: MIS}, ALIGN) for k in ("x", "q", "scale", "bias", "mul", "residual", "pre", "y", "ws")])
def test_linear_refusals(kw, code):
    assert call(L.aql_linear_w8a16_act, LIN, **kw) == code


BWD = dict(dy=P, pre=P, act=4, mul=P, M=5, N=24, dv=P, dmul=P2, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(M=1 << 21, N=1 << 20), SHAPE), (dict(act=-1), PARAM),
    (dict(act=5), PARAM), (dict(mul=None), PARAM), (dict(dmul=P), PARAM)]
    + [({k: None}, NULL) for k in ("dy", "pre", "dv")]
    + [({k: MIS}, ALIGN) for k in ("dy", "pre", "mul", "dv", "dmul")])
def test_backward_refusals(kw, code):
    assert call(L.aql_act_mul_backward, BWD, **kw) == code


def test_empty_linears():
    assert call(L.aql_linear_w8a16_act, LIN, M=0, x=None, y=None) == OK
    assert call(L.aql_linear_w8a16_act, LIN, N=0, q=None, scale=None, y=None) == OK
    assert call(L.aql_act_mul_backward, BWD, M=0, dy=None, pre=None, dv=None, mul=None, dmul=None) == OK


def test_binding_refusals():
    """Host tensors, wrong types and shapes: refused by the binding, nothing called."""
    cpu = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        aql.aql_kv_plan(cpu, cpu[:3], 4, 1, 8, 2, 4)
    with pytest.raises(TypeError):
        aql.aql_kv_plan(cpu.long(), cpu[:3].long(), 4, 1, 8, 2, 4)
    for bad in ((0, 2, 64), (4, 0, 64), (4, 2, 12), (4, 2, 264), (4, 2, 0)):
        with pytest.raises(ValueError):
            aql.aql_kv_cache(*bad, device="cpu")
    cache = aql.aql_kv_cache(4, 2, 64, "cpu")
    assert cache.kq.shape == (4, 2, 1, 64, 64) and cache.vq.shape == (4, 2, 64, 64) and cache.ks.shape == (4, 2)
    plan = aql.KvPlan(4, 3, 8, 2, 4, 1, 0, torch.zeros(64, dtype=torch.uint8))
    table, x = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    for f in (lambda: aql.aql_kv_cache_write(x, x, cache, table, plan), lambda: aql.aql_kv_cache_read(cache, table, plan),
              lambda: aql.aql_attention_kv8(torch.zeros(4, 8, 64, dtype=torch.bfloat16), cache, table, plan),
              lambda: aql.aql_linear_w8a16_act(x[:, 0], cpu, cpu), lambda: aql.aql_act_mul_backward(x[:, 0], x[:, 0], 1)):
        with pytest.raises((ValueError, TypeError)):
            f()
    for bad in (None, 3, x[0]):
        with pytest.raises((ValueError, TypeError)):
            aql.aql_attention_kv8(bad, cache, table, plan)
        with pytest.raises((ValueError, TypeError)):
            aql.aql_kv_cache_write(bad, x, cache, table, plan)
