"""Sizes whose grids would hold 2^32 threads or more: the runtime starts a part of such
a grid without an error, so the entry points refuse them and write nothing."""
import pytest
import torch

import activation_quantized_linear_amd as aql

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def refused(fn, *outs):
    for o in outs:
        o.fill_(77)
    with pytest.raises(aql.AqlError, match="launch failed") as e:
        fn()
    assert e.value.code == aql.AQL_ERR_HIP
    torch.cuda.synchronize()
    for o in outs:
        assert (o[:4096] == 77).all() and (o[-4096:] == 77).all()


@pytest.mark.parametrize("M", [1, 2])
def test_w8a16_of_more_channels_than_a_grid_holds(M):
    N, K = (1 << 29) + 64, 16
    print("w8a16", M, N, K, flush=True)
    q = torch.ones(N, K, dtype=torch.int8, device=DEV)
    scale = torch.ones(N, device=DEV)
    x = torch.ones(M, K, dtype=torch.bfloat16, device=DEV)
    y = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    refused(lambda: aql.aql_linear_w8a16(x, q, scale, y=y), y.view(-1))
    if M == 1:
        host, dev = aql.aql_w8a16_group_plan([(x, q, scale, None, y)])
        refused(lambda: aql.aql_linear_w8a16_grouped(host, dev), y.view(-1))
    n = N // 2  # and half of them run
    aql.aql_linear_w8a16(x, q[:n], scale[:n], y=y.view(-1)[:M * n].view(M, n))
    assert (y.view(-1)[:M * n] == 16).all()


@pytest.mark.parametrize("K", [4, 1028])
def test_quantizers_of_more_rows_than_a_grid_holds(K):
    rows = (1 << 26) + 4 if K == 4 else (1 << 24) + 1
    print("quantizers", rows, K, flush=True)
    x = torch.ones(rows, K, device=DEV)
    q = torch.empty(rows, K, dtype=torch.int8, device=DEV)
    s = torch.empty(rows, device=DEV)
    i = torch.empty(rows, dtype=torch.int32, device=DEV)
    refused(lambda: aql.aql_quantize_weight_int8(x, q=q, scale=s, wsum=i), q.view(-1), s, i)
    refused(lambda: aql.aql_choose_qparams_rows(x, scale=s, zp=i, xq=q), q.view(-1), s, i)
    aql.aql_quantize_weight_int8(x[8:], q=q[8:], scale=s[8:], wsum=i[8:])
    assert (q[8:] == 127).all() and (i[8:] == 127 * K).all()


@pytest.mark.parametrize("M,N,K", [(2, (1 << 26) + 64, 2048), (4, (1 << 29) + 64, 16)])
def test_w8a16_below_the_limit_of_its_own_grid(M, N, K):
    """Grids of fewer threads a channel go further: 32 for two rows, 4 for four."""
    print("w8a16", M, N, K, flush=True)
    q = torch.ones(N, K, dtype=torch.int8, device=DEV)
    scale = torch.ones(N, device=DEV)
    x = torch.ones(M, K, dtype=torch.bfloat16, device=DEV)
    y = aql.aql_linear_w8a16(x, q, scale)
    assert (y == K).all()
