"""The plan of a step on the 8-bit cache: sequences that overlap, and plans of two streams at once."""
import pytest
import torch

import activation_quantized_linear_amd as aql
from test_gpu_kv import Step

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("cu,T,most", [([0, 600, 0, 600, 0, 600, 0, 600], 600, 600), ([0, 300, 0, 300, 0, 300, 0, 300], 300, 300)])
def test_sequences_that_overlap_to_more_rows(cu, T, most):
    """1 + S, whatever else is wrong with a sequence; nothing is written or attended."""
    S, Hq, Hkv, D, W, P = len(cu) - 1, 4, 2, 64, 16, 200
    plan = aql.aql_kv_plan(i32(cu), i32([0] * S), T, most, Hq, Hkv, W)
    assert plan.info.item() == 1 + S
    cache = aql.aql_kv_cache(P, Hkv, D, DEV)
    for t in (cache.kq, cache.vq, cache.ks, cache.vs):
        t.fill_(77)
    table = torch.arange(S * W, dtype=torch.int32, device=DEV).view(S, W)
    k = torch.ones(T, Hkv, D, dtype=torch.bfloat16, device=DEV)
    aql.aql_kv_cache_write(k, k, cache, table, plan)
    y = torch.full((T, Hq, D), 77.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, Hq), 77.0, device=DEV)
    aql.aql_attention_kv8(torch.ones_like(y), cache, table, plan, y=y, lse=lse)
    a, b = aql.aql_kv_cache_read(cache, table, plan, k=torch.full_like(k, 77.0), v=torch.full_like(k, 77.0))
    for t in (cache.kq, cache.vq, cache.ks, cache.vs, y, lse, a, b):
        assert (t == 77).all()
    # the same buffer serves the next step
    aql.aql_kv_plan(i32([0] + [T] * S), i32([0] * S), T, most, Hq, Hkv, W, plan=plan)
    assert plan.info.item() == 0


@pytest.mark.parametrize("T,D,fits", [(1 << 20, 256, False), (1 << 20, 136, False), (1 << 19, 256, True), (1 << 20, 128, True)])
def test_units_past_one_grid(T, D, fits):
    """Heads past 128 run in workgroups of 512 threads, of which a grid holds half as many. The plan
    has room for as many units as a step of these sizes could have and holds none."""
    Hq, Hkv, W = 1024, 1, 8
    print("attention", T, D, flush=True)
    room = torch.zeros(aql.aql_kv_plan_bytes(T, 1, Hq, Hkv, W, T), dtype=torch.uint8, device=DEV)
    assert aql.aql_attention_kv8_bytes(T, 1, Hq, Hkv, D, W, T) == 0
    any16 = torch.zeros(1 << 16, dtype=torch.uint8, device=DEV)
    p = any16.data_ptr()
    rc = aql._lib.aql_attention_kv8(p, Hq * D, T, 1, Hq, Hkv, D, 0.1, 0, p, p, p, p, 1, p, W, T, room.data_ptr(), p, None,
                                    None, 0, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == (aql.AQL_OK if fits else aql.AQL_ERR_HIP), aql.aql_last_error()
    assert not any16.any()


def test_two_streams_with_work_in_flight():
    """Writes and attention of two batches queued on two streams, everything made before: divided
    units, so that both keep partial results, of decoding sequences and of a chunk."""
    batches = [Step([(3000, 1), (2500, 1), (700, 1)], 8, 2, 64, seed=41), Step([(2600, 40), (900, 1)], 4, 2, 128, seed=43)]
    work = []
    for s in batches:
        s.write_past()
        plan = s.write()
        assert aql.aql_attention_kv8_bytes(s.T, len(s.seqs), s.Hq, s.Hkv, s.D, s.W, max(s.news)) > 0
        want = s.attend(plan)
        s.check_attention(*want)
        work.append((s, plan, want, s.q.to(DEV), s.k.to(DEV), s.v.to(DEV)))
    turns = 60
    outs = [[(torch.full_like(w[2][0], 77.0), torch.full_like(w[2][1], 77.0)) for _ in range(turns)] for w in work]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for t in range(turns):
        for (s, plan, _, q, k, v), out, st in zip(work, outs, streams):
            with torch.cuda.stream(st):
                aql.aql_kv_cache_write(k, v, s.cache, s.dev_table, plan)  # (the same tokens: the same codes)
                aql.aql_attention_kv8(q, s.cache, s.dev_table, plan, y=out[t][0], lse=out[t][1])
    torch.cuda.synchronize()
    for (s, _, want, *_), out in zip(work, outs):
        s.check_cache()
        for y, lse in out:
            assert torch.equal(y, want[0]) and torch.equal(lse, want[1])
