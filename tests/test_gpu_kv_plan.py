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


@pytest.mark.parametrize("D", [64, 200, 256])
def test_captured_chunks(D):
    """Plan, write, attention and read of a chunk beside decoding sequences in one graph: its positions move on
    the device, replays alternate with eager work, and each equals the eager step and the plain form."""
    Hq, Hkv, new, turns = 4, 2, 48, 3
    s = Step([(900, new), (700, 1), (60, 1)], Hq, Hkv, D, seed=D)
    s.write_past()
    free = [p for p in range(s.P) if all(p not in r for r in s.table)]
    need = [(p + turns * n + 63) // 64 for p, n in zip(s.pasts, s.news)]
    W = max(need) + 2
    P = s.P + sum(need)
    wide = aql.aql_kv_cache(P, Hkv, D, DEV)  # room for the pages to come
    for a, b in ((wide.kq, s.cache.kq), (wide.vq, s.cache.vq), (wide.ks, s.cache.ks), (wide.vs, s.cache.vs)):
        a[:s.P] = b
    s.cache, fresh = wide, iter(free + list(range(s.P, P)))
    have = [(p + n + 63) // 64 for p, n in zip(s.pasts, s.news)]
    s.table = [[r[b] if b < h else next(fresh) if b < m else -1 for b in range(W)] for r, h, m in zip(s.table, have, need)]
    s.dev_table, s.W = i32(s.table), W
    ref = s.ref
    s.ref = type(ref)(P, Hkv, D)
    for name in "kv":
        s.ref.codes[name][:s.P], s.ref.scale[name][:s.P] = ref.codes[name], ref.scale[name]
    s.P = P
    cu, pos, grow = i32(s.cu), i32(s.pasts), i32(s.news)
    q, k, v = [torch.zeros(s.T, h, D, dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hkv)]
    plan = aql.aql_kv_plan(cu, pos, s.T, new, Hq, Hkv, W)
    y, kb, vb = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    lse = torch.empty(s.T, Hq, device=DEV)
    keep = [t.clone() for t in (wide.kq, wide.vq, wide.ks, wide.vs)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        aql.aql_kv_plan(cu, pos, s.T, new, Hq, Hkv, W, plan=plan)
        aql.aql_kv_cache_write(k, v, wide, s.dev_table, plan)
        aql.aql_attention_kv8(q, wide, s.dev_table, plan, y=y, lse=lse)
        aql.aql_kv_cache_read(wide, s.dev_table, plan, k=kb, v=vb)
        pos.add_(grow)
    for a, b in zip((wide.kq, wide.vq, wide.ks, wide.vs), keep):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))  # (nothing ran in the capture)
    g = torch.Generator().manual_seed(D)
    for t in range(turns):
        s.q, s.k, s.v = [torch.randn(s.T, h, D, generator=g).to(torch.bfloat16) for h in (Hq, Hkv, Hkv)]
        for a, b in ((q, s.q), (k, s.k), (v, s.v)):
            a.copy_(b)
        graph.replay()
        s.seqs = [(c, p, n) for c, p, n in zip(s.cu, s.pasts, s.news)]
        s.ref_write(s.k, s.v, s.seqs)
        torch.cuda.synchronize()
        assert plan.info.item() == 0
        s.check_cache()
        s.check_attention(y, lse)
        eager = aql.aql_attention_kv8(q, wide, s.dev_table, plan)
        assert torch.equal(eager, y)
        a, b = aql.aql_kv_cache_read(wide, s.dev_table, plan)
        assert torch.equal(a, kb) and torch.equal(b, vb)
        other = Step([(70, 40)], 2, 1, 64, seed=t)
        other.write_past()
        other.attend(other.write())
        s.pasts = [p + n for p, n in zip(s.pasts, s.news)]
