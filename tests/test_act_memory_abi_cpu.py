"""Outputs of the linear with an epilogue in memory of its operands, without a GPU: refused before any HIP
call (fake device addresses are never touched)."""
import ctypes as C

import pytest

import activation_quantized_linear_amd as aql

M, N = 70, 264
SIZE = 2 * M * N  # bytes of a matrix
A, B, Y, PRE = 0x1000000, 0x2000000, 0x3000000, 0x4000000  # mul, residual, y, pre


def call(mul=A, residual=B, pre=PRE, y=Y):
    p = C.c_void_p(0x10000)
    ptr = [C.c_void_p(v) if v else None for v in (mul, residual, pre, y)]
    return aql._lib.aql_linear_w8a16_act(p, M, 64, p, p, None, N, aql.AQL_ACT_SILU, *ptr, None, 0, None)


@pytest.mark.parametrize("kw", [dict(pre=A), dict(pre=B), dict(pre=Y), dict(pre=A + 16), dict(pre=B - SIZE + 16),
                                dict(pre=Y + SIZE - 16), dict(y=A + 16), dict(y=B - 16), dict(y=A - SIZE + 16),
                                dict(pre=A, y=A), dict(pre=B, y=B), dict(pre=A, residual=None), dict(pre=B, mul=None)])
def test_shared_memory_is_refused(kw):
    assert call(**kw) == aql.AQL_ERR_PARAM
    assert "memory" in aql.aql_last_error()


@pytest.mark.parametrize("kw", [{}, dict(y=A), dict(y=B), dict(mul=B), dict(mul=None, residual=None), dict(pre=None),
                                dict(pre=A + SIZE), dict(pre=B - SIZE), dict(y=A + SIZE), dict(y=A - SIZE)])
def test_separate_memory_is_not(kw):
    """These pass the checks of the arguments (and end at the device's, where there is none)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are no device's")
    assert call(**kw) not in (aql.AQL_ERR_PARAM, aql.AQL_OK)


def gradients(dy=A, pre=B, mul=Y, dv=PRE, dmul=0x5000000):
    ptr = [C.c_void_p(v) if v else None for v in (dy, pre, mul, dv, dmul)]
    return aql._lib.aql_act_mul_backward(ptr[0], ptr[1], aql.AQL_ACT_SILU, ptr[2], M, N, ptr[3], ptr[4], None)


@pytest.mark.parametrize("kw", [dict(dv=A + 16), dict(dv=B - 16), dict(dv=Y + SIZE - 16), dict(dmul=A - 16),
                                dict(dmul=B + 16), dict(dmul=Y - SIZE + 16), dict(dmul=PRE), dict(dmul=PRE + 16)])
def test_gradients_across_memory_are_refused(kw):
    assert gradients(**kw) == aql.AQL_ERR_PARAM
    assert "memory" in aql.aql_last_error()


@pytest.mark.parametrize("kw", [{}, dict(dv=A), dict(dv=B, dmul=Y), dict(dv=Y, dmul=A), dict(dmul=B), dict(dv=A + SIZE),
                                dict(mul=None, dmul=None, dv=A), dict(dmul=PRE - SIZE)])
def test_gradients_in_memory_of_their_own_or_an_input(kw):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are no device's")
    assert gradients(**kw) not in (aql.AQL_ERR_PARAM, aql.AQL_OK)
