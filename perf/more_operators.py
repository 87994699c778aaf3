"""A decoder layer served in 8 bits: what is measured.

Four operators, each in its plain form (elementary torch operations in 32 bits)
and as the framework's call:

  cache     K and V of new tokens quantised into a paged 8-bit cache, and the pages
            that they touched read back. A page holds 64 tokens; each page and kv head has
            one scale for K and one for V: s = max(max |x| / 127, 2^-64). A write behind live
            tokens of a page raises the scale where it has to and rounds their codes anew.
  attend    attention of new tokens over such a cache, their own K and V in it: a token
            at position p sees positions max(0, p - window + 1) .. p (window 0: all)
  linear    y = act(scale * (x . q^T) + bias) * mul + residual, int8 weights
  act_grad  the gradients of that epilogue to its product and to mul

Shapes: k, v [T, Hkv, D] and query [T, Hq, D], slices of one fused projection's
output; x [M, K], mul, residual, y [M, N] bf16, q [N, K] int8, scale [N]. The sizes are those of the
repository's workloads (hidden 960 with 2560, 4096 with 14336 and 11008 channels), with
head layouts to match and generic ones.
"""
import math
import random

import torch

own = False

BLOCK = 64  # tokens of a page
FLOOR = 2.0 ** -64  # the smallest scale


def listed():
    return [
        # 27 sequences of a small model each write the token of a decode step
        dict(name="cache_small_m27", op="cache", heads="15/5", D=64, decode=27, past=1000, prefill=0, new=0),
        # a prefill of five ragged prompts into a 7B model's cache, behind shared beginnings
        dict(name="cache_7b_prefill", op="cache", heads="32/8", D=128, decode=0, past=701, prefill=5, new=2730),
        # one request of a small model: the least work, latency counts
        dict(name="attend_small_m1", op="attend", heads="15/5", D=64, decode=1, past=333, prefill=0, new=0, window=0),
        # a decode step of 64 ragged requests
        dict(name="attend_7b_m64", op="attend", heads="32/8", D=128, decode=64, past=8191, prefill=0, new=0, window=0),
        # one request with a very long context
        dict(name="attend_7b_long", op="attend", heads="32/8", D=128, decode=1, past=131070, prefill=0, new=0, window=0),
        # one step that serves 16 decoding requests and a chunk of a long prompt
        dict(name="attend_7b_mixed", op="attend", heads="32/8", D=128, decode=16, past=6007, prefill=1, new=509,
             window=0),
        # the prefill of three ragged prompts
        dict(name="attend_7b_prefill", op="attend", heads="32/8", D=128, decode=0, past=0, prefill=3, new=4096,
             window=0),
        # gate projection of a small model's decode step: silu(gate) * up
        dict(name="linear_small_m1", op="linear", M=1, K=960, N=2560, act="silu", bias=False, mul=True, residual=False,
             pre=False),
        # down projection of 27 requests, added to the residual stream
        dict(name="linear_7b_m27", op="linear", M=27, K=14336, N=4096, act="none", bias=True, mul=False, residual=True,
             pre=False),
        # gate projection of a training forward, ragged rows: the product is kept for the backward pass
        dict(name="linear_7b_m500", op="linear", M=500, K=4096, N=11007, act="gelu", bias=True, mul=True,
             residual=False, pre=True),
        # gradients of a small model's short sequence, and of a 7B model's 2048 tokens
        dict(name="act_grad_small_m63", op="act_grad", M=63, N=2560, act="gelu_tanh", mul=True),
        dict(name="act_grad_7b_m2048", op="act_grad", M=2048, N=14336, act="silu", mul=True),
    ]


# ------------------------------------------------------------------ sequences


def _heads(case):
    hq, hkv = case["heads"].split("/")
    return int(hq), int(hkv)


def _sequences(case):
    """(past, new) of every sequence: tokens that its cache holds, and tokens of this step."""
    r = random.Random("%(heads)s %(D)d %(decode)d %(past)d %(prefill)d %(new)d" % case)
    out = [(case["past"] if i == 0 else r.randint(0, case["past"]), 1) for i in range(case["decode"])]
    for i in range(case["prefill"]):
        new = case["new"] if i == 0 else r.randint(max(1, case["new"] // 4), case["new"])
        out.append((case["past"] if i == 0 else r.randint(0, case["past"]), new))
    return out


def _visible(case):
    """(pairs of a new token and one that it sees, tokens of the cache that any sees)."""
    pairs = tokens = 0
    w = case.get("window", 0)
    for past, new in _sequences(case):
        first = past + 1  # tokens that the first new one sees without a window
        if w == 0:
            pairs += new * first + new * (new - 1) // 2
            tokens += past + new
        else:
            full = max(0, min(new, w - first))  # tokens whose window is not full yet
            pairs += full * first + full * (full - 1) // 2 + (new - full) * w
            tokens += past + new - max(0, first - w)
    return pairs, tokens


def _new_tokens(case):
    return sum(new for _, new in _sequences(case))


# ----------------------------------------------------------------------- draw


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = ("15/5", "32/8", "32/32", "16/2", "8/1", "40/10", "12/4", "64/8")


def draw(rng):
    op = rng.choice(["cache", "attend", "attend", "linear", "act_grad"])
    while True:
        if op in ("cache", "attend"):
            c = dict(op=op, heads=rng.choice(HEADS), D=rng.choice([64, 64, 80, 96, 128, 128, 256]))
            kind = rng.choice(["decode", "decode", "prefill", "mixed"])
            c["decode"] = 0 if kind == "prefill" else _log_int(rng, 1, 64)
            c["prefill"] = 0 if kind == "decode" else rng.randint(1, 5)
            c["new"] = _log_int(rng, 2, 4096) if c["prefill"] else 0
            c["past"] = _log_int(rng, 1, 131072 if c["decode"] == 1 else 8192) - 1
            if op == "attend":
                c["window"] = rng.choice([0, 0, _log_int(rng, 1, 4096)])
        else:
            M = _log_int(rng, 1, 63) if rng.random() < 0.5 else _log_int(rng, 64, 2048)
            c = dict(op=op, M=M, N=_log_int(rng, 64, 14336), act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                     mul=rng.random() < 0.5)
            if op == "linear":
                c.update(K=16 * _log_int(rng, 4, 896), bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                         pre=rng.random() < 0.3)
        if all(_cost(c)[i] <= max(_cost(d)[i] for d in listed() if d["op"] == op) for i in (0, 1)):
            return c


def _cost(case):
    w = work(case)
    return w["bytes"], w["flops"]


# -------------------------------------------------------------------- prepare


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


def _over(x, s):
    """The binary32 quotient."""
    return (x.double() / s.double()).float()


def _quantise(x):
    """[pages, Hkv, BLOCK, D] -> codes and the scale of each page and head."""
    s = _over(x.abs().amax((2, 3)), torch.full((), 127.0, device=x.device)).clamp(min=FLOOR)
    return torch.round(_over(x, s[:, :, None, None])).clamp(-127, 127).to(torch.int8), s


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _prepare_cache(s, g, case, seed):
    hq, hkv = _heads(case)
    D, seqs = case["D"], _sequences(case)
    s["seqs"] = seqs
    T = _new_tokens(case)
    need = [(past + new + BLOCK - 1) // BLOCK for past, new in seqs]
    pages, wide = sum(need) + 3, max(need)
    order = list(range(pages))
    random.Random(seed).shuffle(order)  # pages as an allocator hands them out
    table, at = [], 0
    for n in need:
        table.append(order[at : at + n] + [-1] * (wide - n))
        at += n
    s["rows"], s["table"] = table, _int32(table)
    hot = 1.0 + 7.0 * (torch.rand(hkv, 1, D, generator=g, device="cuda") < 0.03)  # K channels that run hot
    # the fused projection's output of this step, of which query, k and v are slices
    qkv = _randn(g, T, (hq + 2 * hkv) * D)
    qkv[:, : hq * D] *= 1.5
    qkv[:, hq * D : (hq + hkv) * D].unflatten(1, (hkv, D)).mul_(hot[:, 0])
    qkv = qkv.to(torch.bfloat16)
    s["q"] = qkv[:, : hq * D].unflatten(1, (hq, D))
    s["k"] = qkv[:, hq * D : (hq + hkv) * D].unflatten(1, (hkv, D))
    s["v"] = qkv[:, (hq + hkv) * D :].unflatten(1, (hkv, D))
    for name in ("K", "V"):
        codes = torch.empty(pages, hkv, BLOCK, D, dtype=torch.int8, device="cuda")
        scale = torch.empty(pages, hkv, device="cuda")
        for a in range(0, pages, 256):
            x = _randn(g, min(256, pages - a), hkv, BLOCK, D)
            codes[a : a + 256], scale[a : a + 256] = _quantise(x * hot if name == "K" else x)
        s[name], s[name + "s"] = codes, scale
    cu = [0]
    for _, new in seqs:
        cu.append(cu[-1] + new)
    s["cu"] = cu
    if not own:
        return
    import activation_quantized_linear_amd as aql

    # the cache as the library lays it out: head sizes padded to 64, K in slices of 64, V transposed
    pad = (D + 63) // 64 * 64
    cache = aql.aql_kv_cache(pages, hkv, D, "cuda")
    kq = torch.zeros(pages, hkv, BLOCK, pad, dtype=torch.int8, device="cuda")
    kq[..., :D] = s["K"]
    cache.kq.copy_(kq.view(pages, hkv, BLOCK, pad // 64, 64).transpose(2, 3))
    kq[..., :D] = s["V"]
    cache.vq.copy_(kq.transpose(2, 3))
    cache.ks.copy_(s["Ks"])
    cache.vs.copy_(s["Vs"])
    s["cache"] = cache
    most = max(new for _, new in seqs)
    # one plan for a step: every layer's write and attention use it
    s["plan"] = aql.aql_kv_plan(_int32(cu), _int32([past for past, _ in seqs]), T, most, hq, hkv, wide,
                                window=case.get("window", 0))
    if case["op"] == "cache":
        back = [0]
        for past, new in seqs:
            back.append(back[-1] + past % BLOCK + new)
        s["back"] = aql.aql_kv_plan(_int32(back), _int32([past - past % BLOCK for past, _ in seqs]), back[-1],
                                    most + BLOCK - 1, hq, hkv, wide)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] in ("cache", "attend"):
        _prepare_cache(s, g, case, seed)
        if case["op"] == "cache":
            _prepare_touched(s, case)  # (new tokens that attend are in the cache already)
        return s
    M, N = case["M"], case["N"]
    if case["mul"]:
        s["mul"] = _randn(g, M, N).to(torch.bfloat16)
    if case["op"] == "act_grad":
        # gradients: small, rows of very different size (token losses)
        s["dy"] = (_randn(g, M, N, std=1e-3) * torch.exp(_randn(g, M, 1))).to(torch.bfloat16)
        s["z"] = _randn(g, M, N, std=2.0).to(torch.bfloat16)
        return s
    K = case["K"]
    s["w"], s["scale"] = _weights(g, N, K)
    s["x"] = _randn(g, M, K).to(torch.bfloat16)
    if case["bias"]:
        s["b"] = _randn(g, N, std=0.1).to(torch.bfloat16)
    if case["residual"]:
        s["r"] = _randn(g, M, N, std=4.0).to(torch.bfloat16)
    return s


def _prepare_touched(s, case):
    """Index tensors of the pages that a write touches, for the plain form."""
    page, live, token, back = [], [], [], []
    for i, (past, new) in enumerate(s["seqs"]):
        for b in range(past // BLOCK, (past + new - 1) // BLOCK + 1):
            first = b * BLOCK
            n = len(page)
            page.append(s["rows"][i][b])
            live.append(max(0, past - first))  # tokens of the page that were there before
            token.append([s["cu"][i] + first + j - past if past <= first + j < past + new else -1 for j in range(BLOCK)])
            back += [n * BLOCK + j for j in range(min(BLOCK, past + new - first))]
    s["page"], s["live"] = _int32(page).long(), _int32(live)
    s["token"], s["order"] = _int32(token).long(), _int32(back).long()


# ------------------------------------------------------------------------ run


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "cache":
        return {"k": _write(s, s["k"], "K"), "v": _write(s, s["v"], "V")}
    if s["op"] == "attend":
        return {"y": _attend(s)}
    if s["op"] == "act_grad":
        z, dy = s["z"].float(), s["dy"].float()
        a, d = _act(s["act"], z)
        if s["mul"] is not False:
            return {"dv": (dy * s["mul"].float() * d).to(torch.bfloat16), "dmul": (dy * a).to(torch.bfloat16)}
        return {"dv": (dy * d).to(torch.bfloat16)}
    z = s["x"].float() @ (s["w"].float() * s["scale"][:, None]).T
    if s["bias"]:
        z = z + s["b"].float()
    y = _act(s["act"], z)[0]
    if s["mul"] is not False:
        y = y * s["mul"].float()
    if s["residual"]:
        y = y + s["r"].float()
    out = {"y": y.to(torch.bfloat16)}
    if s["pre"]:
        out["pre"] = z.to(torch.bfloat16)
    return out


def _act(name, z):
    """The activation and its derivative."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        on = (z > 0).to(z.dtype)
        return z * on, on
    if name == "silu":
        g = 1.0 / (1.0 + torch.exp(-z))
        return z * g, g * (1.0 + z * (1.0 - g))
    if name == "gelu":
        c = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return z * c, c + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    r = math.sqrt(2.0 / math.pi)
    t = torch.tanh(r * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * r * (1.0 + 3 * 0.044715 * z * z)


def _write(s, x, name):
    """Quantises the new tokens into their pages; the touched pages' live tokens as bf16."""
    codes, scales = s[name], s[name + "s"]
    page, live, token = s["page"], s["live"], s["token"]
    here = torch.arange(BLOCK, device=page.device)[None, :] < live[:, None]
    old = torch.where((live > 0)[:, None], scales[page], torch.zeros_like(scales[page]))
    values = codes[page].float() * old[:, :, None, None]
    fresh = x[token.clamp(min=0)].float() * (token >= 0)[:, :, None, None]  # [n, BLOCK, Hkv, D]
    fresh = fresh.transpose(1, 2)
    top = _over(fresh.abs().amax((2, 3)), torch.full((), 127.0, device=x.device)).clamp(min=FLOOR)
    scale = torch.maximum(old, top)
    values = torch.where(here[:, None, :, None], values, fresh)
    new = torch.round(_over(values, scale[:, :, None, None])).clamp(-127, 127)
    codes[page], scales[page] = new.to(torch.int8), scale
    out = (new * scale[:, :, None, None]).transpose(1, 2).flatten(0, 1)
    return out[s["order"]].to(torch.bfloat16)


def _attend(s):
    q = s["q"]
    T, hq, D = q.shape
    hkv = s["K"].shape[1]
    out = torch.empty(T, hq, D, dtype=torch.bfloat16, device=q.device)
    for i, (past, new) in enumerate(s["seqs"]):
        n = past + new
        pages = s["table"][i, : (n + BLOCK - 1) // BLOCK].long()
        k = (s["K"][pages].float() * s["Ks"][pages][:, :, None, None]).transpose(0, 1).reshape(hkv, -1, D)[:, :n]
        v = (s["V"][pages].float() * s["Vs"][pages][:, :, None, None]).transpose(0, 1).reshape(hkv, -1, D)[:, :n]
        a = s["cu"][i]
        rows = q[a : a + new].float().view(new, hkv, hq // hkv, D).permute(1, 2, 0, 3).reshape(hkv, -1, D)
        p = (rows @ k.transpose(1, 2)) * D ** -0.5
        p = p.view(hkv, -1, new, n)
        at, to = torch.arange(past, n, device=q.device)[:, None], torch.arange(n, device=q.device)[None, :]
        hidden = to > at
        if s["window"]:
            hidden = hidden | (to <= at - s["window"])
        p = p.masked_fill(hidden, -math.inf)
        p = torch.exp(p - p.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        y = p.reshape(hkv, -1, n) @ v
        out[a : a + new] = y.view(hkv, -1, new, D).permute(2, 0, 1, 3).reshape(new, hq, D).to(torch.bfloat16)
    return out


def _run_own(s):
    import activation_quantized_linear_amd as aql

    if s["op"] == "cache":
        aql.aql_kv_cache_write(s["k"], s["v"], s["cache"], s["table"], s["plan"])
        k, v = aql.aql_kv_cache_read(s["cache"], s["table"], s["back"], torch.bfloat16)
        return {"k": k, "v": v}
    if s["op"] == "attend":
        return {"y": aql.aql_attention_kv8(s["q"], s["cache"], s["table"], s["plan"])}
    act = {"none": aql.AQL_ACT_NONE, "relu": aql.AQL_ACT_RELU, "gelu": aql.AQL_ACT_GELU,
           "gelu_tanh": aql.AQL_ACT_GELU_TANH, "silu": aql.AQL_ACT_SILU}[s["act"]]
    mul = None if s["mul"] is False else s["mul"]
    if s["op"] == "act_grad":
        dv, dmul = aql.aql_act_mul_backward(s["dy"], s["z"], act, mul)
        return {"dv": dv} if dmul is None else {"dv": dv, "dmul": dmul}
    pre = torch.empty(s["M"], s["N"], dtype=torch.bfloat16, device=s["x"].device) if s["pre"] else None
    y = aql.aql_linear_w8a16_act(s["x"], s["w"], s["scale"], s.get("b"), act=act, mul=mul, residual=s.get("r"), pre=pre)
    return {"y": y} if pre is None else {"y": y, "pre": pre}


def work(case):
    if case["op"] in ("cache", "attend"):
        hq, hkv = _heads(case)
        D, seqs = case["D"], _sequences(case)
        T = _new_tokens(case)
        if case["op"] == "cache":
            pages = sum((past + new - 1) // BLOCK - past // BLOCK + 1 for past, new in seqs)
            back = sum(past % BLOCK + new for past, new in seqs)  # tokens read back
            # K and V: tokens in, codes and scales out; codes and scales in, values out
            return {"bytes": 2 * hkv * (3 * T * D + 3 * back * D + 8 * pages), "flops": 2 * hkv * D * 4 * (T + back)}
        pairs, tokens = _visible(case)
        return {"bytes": 2 * hkv * D * tokens + 8 * hkv * ((tokens + BLOCK - 1) // BLOCK) + 4 * T * hq * D,
                "flops": 4 * pairs * hq * D}
    M, N = case["M"], case["N"]
    if case["op"] == "act_grad":
        return {"bytes": 2 * M * N * (5 if case["mul"] else 3), "flops": 12 * M * N}
    K = case["K"]
    sides = 1 + case["mul"] + case["residual"] + case["pre"]
    return {"bytes": N * K + 4 * N + 2 * M * K + 2 * M * N * sides + (2 * N if case["bias"] else 0),
            "flops": 2 * M * N * K}


# ---------------------------------------------------------------------- exact


def exact(case, seed):
    """The definitions, sequence by sequence and head by head, in 64 bits."""
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "cache":
        return {"k": _exact_write(s, s["k"], "K"), "v": _exact_write(s, s["v"], "V")}
    if case["op"] == "attend":
        return {"y": _exact_attend(s)}
    name = case["act"]
    mul = s["mul"].to(f) if case["mul"] else None
    if case["op"] == "act_grad":
        dy, z = s["dy"].to(f), s["z"].to(f).requires_grad_()
        a = _exact_act(name, z)
        d, = torch.autograd.grad(a.sum(), z)
        dv = dy * d if mul is None else dy * d * mul
        return {"dv": dv} if mul is None else {"dv": dv, "dmul": dy * a.detach()}
    z = torch.mm(s["x"].to(f), s["w"].to(f).T) * s["scale"].to(f)
    if case["bias"]:
        z += s["b"].to(f)
    y = _exact_act(name, z)
    y = y if mul is None else y * mul
    y = y + s["r"].to(f) if case["residual"] else y
    return {"y": y, "pre": z} if case["pre"] else {"y": y}


def _exact_act(name, z):
    if name == "none":
        return z * 1
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))


def _round32(x):
    return x.to(torch.float32).to(torch.float64)


def _exact_write(s, x, name):
    out = []
    for i, (past, new) in enumerate(s["seqs"]):
        at = past
        while at < past + new:  # page by page
            page, live = s["rows"][i][at // BLOCK], at % BLOCK
            n = min(BLOCK - live, past + new - at)
            row = s["cu"][i] + at - past
            fresh = x[row : row + n].to(torch.float64)  # [n, Hkv, D]
            scale = _round32(fresh.abs().amax((0, 2)) / 127).clamp(min=FLOOR)
            values = fresh
            if live:
                old = s[name + "s"][page].to(torch.float64)
                scale = torch.maximum(scale, old)
                values = torch.cat([_round32(s[name][page, :, :live].to(torch.float64) * old[:, None, None]).transpose(0, 1),
                                    fresh])
            code = _round32(values / scale[:, None]).round()  # a binary32 quotient, half to even
            out.append(code * scale[:, None])
            at += n
    return torch.cat(out)


def _exact_attend(s):
    q = s["q"].to(torch.float64)
    T, hq, D = q.shape
    hkv = s["K"].shape[1]
    out = torch.empty(T, hq, D, dtype=torch.float64, device=q.device)
    for i, (past, new) in enumerate(s["seqs"]):
        n = past + new
        pages = s["table"][i, : (n + BLOCK - 1) // BLOCK].long()
        a = s["cu"][i]
        for j in range(hkv):
            k = (s["K"][pages, j].to(torch.float64) * s["Ks"][pages, j].to(torch.float64)[:, None, None]).view(-1, D)[:n]
            v = (s["V"][pages, j].to(torch.float64) * s["Vs"][pages, j].to(torch.float64)[:, None, None]).view(-1, D)[:n]
            for h in range(j * (hq // hkv), (j + 1) * (hq // hkv)):
                score = torch.mm(q[a : a + new, h], k.T) / math.sqrt(D)
                age = torch.arange(past, n, device=q.device)[:, None] - torch.arange(n, device=q.device)
                score[age < 0] = -math.inf
                if s["window"]:
                    score[age >= s["window"]] = -math.inf
                out[a : a + new, h] = torch.mm(torch.softmax(score, -1), v)
    return out
