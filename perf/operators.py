"""Low-rank adapters beside the frozen int8 linear: what is measured.

Four operators, each in its plain form (elementary torch operations in 32 bits)
and as the framework's call:

  lora        y = scale * (x . q^T) + bias + h . B_a^T,  h = alpha_a * (x . A_a^T), a = idx[row]
              (rows whose idx lies outside [0, L) have no adapter: h = 0)
  checkpoint  activations in 8 bits, groups of 128 along a row, and their restoration
  dgrad       dx = (dy * scale) . q, the frozen linear's gradient to its input
  backward    dx, dA, dB of the linear with adapters, from the 8-bit checkpoint of x

Shapes: x [M, K] bf16, q [N, K] int8, scale [N], A [L, R, K] bf16, B [L, N, R]
bf16, alpha [L], idx [M] int32. The sizes are the MLP linears of the
repository's workloads (960 x 2560, 4096 x 14336, 4096 x 11008).
"""
import math

import torch

own = False

GROUP = 128  # values of a row that share one checkpoint scale


def listed():
    return [
        # one request of a small model's decode step: the least work, latency counts
        dict(name="lora_small_m1", op="lora", M=1, K=960, N=2560, L=4, R=8, mix="random", bias=False),
        # one request of a 7B model's decode step
        dict(name="lora_7b_m1", op="lora", M=1, K=4096, N=14336, L=8, R=16, mix="random", bias=False),
        # 27 requests of one decode step, each with an adapter of its own or none
        dict(name="lora_7b_m27", op="lora", M=27, K=14336, N=4096, L=32, R=16, mix="random", bias=True),
        # a ragged prefill of three requests, larger rank, odd channel count
        dict(name="lora_prefill_m500", op="lora", M=500, K=4096, N=11007, L=3, R=64, mix="runs", bias=True),
        # a training forward: one adapter, 2048 tokens
        dict(name="lora_7b_m2048", op="lora", M=2048, K=4096, N=14336, L=1, R=16, mix="runs", bias=False),
        # activations of a small model's layer, odd row count
        dict(name="ckpt_small_bf16", op="checkpoint", M=509, K=2560, dtype="bf16"),
        # activations of a 7B model's down projection
        dict(name="ckpt_7b_bf16", op="checkpoint", M=8192, K=14336, dtype="bf16"),
        # the gradient through a layer that carries no adapter: small and 7B
        dict(name="dgrad_small_m333", op="dgrad", M=333, K=960, N=2560),
        dict(name="dgrad_7b_m2048", op="dgrad", M=2048, K=4096, N=11008),
        # training steps: a short sequence of a small model, a ragged batch of
        # three adapters, a 7B model's up projection
        dict(name="bwd_small_m63", op="backward", M=63, K=960, N=2560, L=2, R=8, mix="runs"),
        dict(name="bwd_7b_m500", op="backward", M=500, K=14336, N=4096, L=3, R=64, mix="runs"),
        dict(name="bwd_7b_m2048", op="backward", M=2048, K=4096, N=14336, L=1, R=16, mix="runs"),
    ]


def _cost(c):
    if c["op"] == "checkpoint":
        return 0
    rank = c.get("L", 0) * c.get("R", 0)
    return c["M"] * (c["N"] * c["K"] + rank * (c["N"] + c["K"])) * (2 if c["op"] == "backward" else 1)


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["lora", "lora", "checkpoint", "dgrad", "backward"])
    if op == "checkpoint":
        M, K = log_int(1, 8192), 4 * log_int(1, 3584)
        # bf16 rows of 14336 are the largest; float32 rows cost twice the bytes
        dtype = rng.choice(["bf16", "f32"])
        return dict(op=op, M=min(M, 4096) if dtype == "f32" else M, K=K, dtype=dtype)
    K = 16 * log_int(4, 896)
    if op == "lora":
        M = log_int(1, 63) if rng.random() < 0.5 else log_int(64, 2048)
        N = log_int(64, 14336)
    else:
        M, N = log_int(1, 2048), 8 * log_int(8, 1792)
    c = dict(op=op, M=M, K=K, N=N)
    if op != "dgrad":
        R = rng.choice([8, 16, 24, 32, 64, 128])
        c.update(L=max(1, min(log_int(1, 32), 512 // R)), R=R, mix=rng.choice(["random", "runs"]))
    if op == "lora":
        c["bias"] = rng.random() < 0.5
    top = max(_cost(d) for d in listed())
    if _cost(c) > top:
        c["M"] = max(1, int(c["M"] * top / _cost(c)))
    return c


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std


def _weights(g, N, K):
    """A linear's int8 weights as a program holds them: codes and one scale per channel."""
    w = _randn(g, N, K, std=0.02)
    w[torch.randperm(N, generator=g, device="cuda")[: N // 100]] *= 8.0  # outlier channels
    scale = w.abs().amax(1) / 127.0
    return torch.round(w / scale[:, None]).clamp(-127, 127).to(torch.int8), scale


def _adapters(g, N, K, L, R):
    A = _randn(g, L, R, K, std=K ** -0.5).to(torch.bfloat16)
    B = _randn(g, L, N, R, std=0.02).to(torch.bfloat16)
    alpha = 0.5 + 3.5 * torch.rand(L, generator=g, device="cuda")
    return A, B, alpha


def _index(g, M, L, mix):
    """Each row's adapter: whole sequences in a row ("runs"), or every row its own."""
    if mix == "random":
        return (torch.randint(0, L + 1, (M,), generator=g, device="cuda") - 1).to(torch.int32)  # -1: none
    cuts = torch.rand(max(L - 1, 0), generator=g, device="cuda").mul(M).long()
    at = torch.arange(M, device="cuda")
    return (at[:, None] >= cuts[None, :]).sum(1).to(torch.int32)


def _activations(g, M, K):
    x = _randn(g, M, K)
    x[:, torch.randperm(K, generator=g, device="cuda")[: max(1, K // 512)]] *= 30.0  # channels that run hot
    x[0] *= 50.0  # the position that attention sinks into
    return x


def _pad(x):
    M, K = x.shape
    G = (K + GROUP - 1) // GROUP
    padded = torch.zeros(M, G * GROUP, device=x.device, dtype=x.dtype)
    padded[:, :K] = x
    return padded.view(M, G, GROUP)


def _codes(x):
    """The checkpoint's codes and scales: the float32 quotient x / scale, rounded half to even."""
    p = _pad(x.float())
    scale = p.abs().amax(2) / 127.0
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    quotient = (p.double() / scale.double()[:, :, None]).float()
    codes = torch.round(quotient).clamp(-127, 127)
    return codes.view(x.shape[0], -1)[:, : x.shape[1]].contiguous(), scale


def _decoded(codes, scale):
    return codes * scale.repeat_interleave(GROUP, dim=1)[:, : codes.shape[1]]


def _one_hot(idx, L, dtype):
    return (idx[:, None].long() == torch.arange(L, device=idx.device)[None, :]).to(dtype)


def _shrink(x, W, alpha, hot):
    """alpha_a * (x . W_a^T) of each row's adapter, W [L, R, K]; zero without one."""
    L, R, K = W.shape
    every = (x @ W.reshape(L * R, K).T).view(-1, L, R)
    return (every * (hot * alpha)[:, :, None]).sum(1)


def _spread(h, hot):
    """h [M, R] in its adapter's place of [M, L * R], zero elsewhere."""
    return (hot[:, :, None] * h[:, None, :]).reshape(h.shape[0], -1)


def prepare(case, seed):
    g = _gen(seed)
    M, K = case["M"], case["K"]
    s = dict(case)
    if case["op"] == "checkpoint":
        s["x"] = _activations(g, M, K).to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        return s
    N = case["N"]
    s["q"], s["scale"] = _weights(g, N, K)
    if case["op"] != "lora":
        # gradients: small, rows of very different size (token losses)
        s["dy"] = (_randn(g, M, N, std=1e-3) * torch.exp(_randn(g, M, 1))).to(torch.bfloat16)
    if case["op"] == "dgrad":
        return s
    L, R = case["L"], case["R"]
    s["A"], s["B"], s["alpha"] = _adapters(g, N, K, L, R)
    s["idx"] = _index(g, M, L, case["mix"])
    x = _activations(g, M, K).to(torch.bfloat16) if case["op"] == "backward" else _randn(g, M, K).to(torch.bfloat16)
    if case["op"] == "lora":
        s["x"] = x
        s["bias"] = _randn(g, N, std=0.1).to(torch.bfloat16) if case["bias"] else None
    else:
        # what the forward pass of a training step left: the checkpoint of x, and h
        codes, s["xs"] = _codes(x)
        s["xq"] = codes.to(torch.int8)
        s["h"] = _shrink(x.float(), s["A"].float(), s["alpha"], _one_hot(s["idx"], L, torch.float32))
    if own:
        import activation_quantized_linear_amd as aql

        # one plan for a batch: every layer's linears and both directions use it
        s["plan"] = aql.aql_lora_plan(s["idx"], L)
    return s


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "checkpoint":
        codes, scale = _codes(s["x"])
        return {"scale": scale, "restored": _decoded(codes, scale).to(s["x"].dtype)}
    w = s["q"].float() * s["scale"][:, None]
    if s["op"] == "dgrad":
        return {"dx": (s["dy"].float() @ w).to(torch.bfloat16)}
    hot = _one_hot(s["idx"], s["L"], torch.float32)
    A, B = s["A"].float(), s["B"].float()
    if s["op"] == "lora":
        x = s["x"].float()
        h = _shrink(x, A, s["alpha"], hot)
        y = x @ w.T + _spread(h, hot) @ B.transpose(1, 2).reshape(-1, B.shape[1])
        if s["bias"] is not None:
            y = y + s["bias"].float()
        return {"y": y.to(torch.bfloat16), "h": h}
    dy = s["dy"].float()
    u = _shrink(dy, B.transpose(1, 2), s["alpha"], hot)
    spread = _spread(u, hot)
    dx = dy @ w + spread @ A.reshape(-1, A.shape[2])
    x = _decoded(s["xq"].float(), s["xs"])
    dA = (spread.T @ x).view(A.shape)
    dB = (_spread(s["h"], hot).T @ dy).view(s["L"], s["R"], -1).transpose(1, 2).contiguous()
    return {"dx": dx.to(torch.bfloat16), "dA": dA, "dB": dB}


def _run_own(s):
    import activation_quantized_linear_amd as aql

    if s["op"] == "lora":
        y, h = aql.aql_linear_w8a16_lora(s["x"], s["q"], s["scale"], s["A"], s["B"], s["alpha"], s["plan"], s["bias"])
        return {"y": y, "h": h}
    if s["op"] == "checkpoint":
        xq, xs = aql.aql_act_checkpoint(s["x"])
        return {"scale": xs, "restored": aql.aql_act_restore(xq, xs, s["x"].dtype)}
    if s["op"] == "dgrad":
        return {"dx": aql.aql_linear_w8a16_dgrad(s["dy"], s["q"], s["scale"])}
    dx, dA, dB = aql.aql_linear_w8a16_lora_backward(s["dy"], s["q"], s["scale"], s["A"], s["B"], s["alpha"],
                                                    s["plan"], s["h"], s["xq"], s["xs"])
    return {"dx": dx, "dA": dA, "dB": dB}


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "checkpoint":
        wide, scales = (2 if case["dtype"] == "bf16" else 4) * M * K, 4 * M * ((K + GROUP - 1) // GROUP)
        # x in, codes and scales out; codes and scales in, restored values out
        return {"bytes": 2 * (wide + M * K + scales), "flops": 4 * M * K}
    N = case["N"]
    if case["op"] == "dgrad":
        return {"bytes": N * K + 4 * N + 2 * M * N + 2 * M * K, "flops": 2 * M * N * K}
    L, R = case["L"], case["R"]
    live = min(L, M)  # adapters that rows can name
    adapters = 2 * live * R * (N + K) + 4 * L + 4 * M
    if case["op"] == "lora":
        return {"bytes": N * K + 4 * N + 2 * M * K + 2 * M * N + 4 * M * R + adapters + (2 * N if case["bias"] else 0),
                "flops": 2 * M * N * K + 2 * M * R * (N + K)}
    return {"bytes": N * K + 4 * N + 2 * M * N + 2 * M * K + M * K + 4 * M * ((K + GROUP - 1) // GROUP) + 4 * M * R
            + adapters + 4 * L * R * (N + K),
            "flops": 2 * M * N * K + 4 * M * R * (N + K)}


def exact(case, seed):
    """The definitions, adapter by adapter, in 64 bits."""
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "checkpoint":
        x = s["x"].to(f)
        scales, restored = [], []
        for k in range(0, case["K"], GROUP):
            part = x[:, k : k + GROUP]
            scale = (part.abs().max(1, keepdim=True).values / 127).to(torch.float32).to(f)
            scale[scale == 0] = 1
            code = (part / scale).to(torch.float32).to(f).round()  # a float32 quotient, half to even
            scales.append(scale)
            restored.append(code * scale)
        return {"scale": torch.cat(scales, 1), "restored": torch.cat(restored, 1)}
    q, scale = s["q"].to(f), s["scale"].to(f)
    if case["op"] == "dgrad":
        return {"dx": torch.mm(s["dy"].to(f) * scale, q)}
    A, B, alpha = s["A"].to(f), s["B"].to(f), s["alpha"].to(f)
    if case["op"] == "lora":
        x = s["x"].to(f)
        y, h = torch.mm(x, q.T) * scale, torch.zeros(case["M"], case["R"], dtype=f, device=x.device)
        for a in range(case["L"]):
            rows = (s["idx"] == a).nonzero()[:, 0]
            h[rows] = alpha[a] * torch.mm(x[rows], A[a].T)
            y[rows] += torch.mm(h[rows], B[a].T)
        return {"y": y if s["bias"] is None else y + s["bias"].to(f), "h": h}
    dy = s["dy"].to(f)
    dx, dA, dB = torch.mm(dy * scale, q), torch.zeros_like(A), torch.zeros_like(B)
    at = torch.arange(case["K"], device=dy.device) // GROUP
    for a in range(case["L"]):
        rows = (s["idx"] == a).nonzero()[:, 0]
        u = alpha[a] * torch.mm(dy[rows], B[a])
        dx[rows] += torch.mm(u, A[a])
        dA[a] = torch.mm(u.T, s["xq"][rows].to(f) * s["xs"][rows].to(f)[:, at])
        dB[a] = torch.mm(dy[rows].T, s["h"][rows].to(f))
    return {"dx": dx, "dA": dA, "dB": dB}
