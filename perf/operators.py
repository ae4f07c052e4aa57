"""What the 4-bit cache and sampling operators are measured on.

Three operators, each in a plain form (elementary torch operations) and through
the framework's own calls:

  append     quantise new K and V rows into a 4-bit cache and read them back
  attention  attention of one or more new tokens per request over a 4-bit cache
  sample     a token per row of logits by temperature, top-k, top-p and min-p
             from given random numbers

``own`` selects the framework's calls; everything else is the same.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"fp16": 2, "bf16": 2, "fp32": 4}
# share of the full length that request b of a ragged batch has
SHARE = (1.0, 0.37, 0.81, 0.06, 0.93, 0.59, 0.22, 0.48)


# ---- cases ---------------------------------------------------------------------------------------
def _attention(name, batch, heads, kv_heads, dim, group, ctx, queries=1, window=0, ragged=False, dtype="fp16"):
    return {"name": name, "op": "attention", "batch": batch, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "group": group, "ctx": ctx, "queries": queries, "window": window, "ragged": ragged, "dtype": dtype}


def _append(name, batch, kv_heads, dim, group, ctx, tokens, ragged=False, dtype="fp16"):
    return {"name": name, "op": "append", "batch": batch, "kv_heads": kv_heads, "dim": dim, "group": group,
            "ctx": ctx, "tokens": tokens, "ragged": ragged, "dtype": dtype}


def _sample(name, rows, vocab, top_k=True, top_p=True, min_p=True, dtype="fp32"):
    return {"name": name, "op": "sample", "rows": rows, "vocab": vocab, "top_k": top_k, "top_p": top_p,
            "min_p": min_p, "dtype": dtype}


def listed():
    return [
        # a small model's step, a few dozen tokens in: latency alone counts
        _attention("att_tiny", 1, 4, 4, 64, 32, 47),
        # one decode step of a 1.8B model at a 2,048-token prompt, in the engine's fp32 activations
        _attention("att_2k_fp32", 1, 16, 16, 128, 32, 2300, dtype="fp32"),
        # one decode step of the same model at the end of a 32K context
        _attention("att_32k", 1, 16, 16, 128, 64, 32768),
        # eight requests of uneven length, shared K/V heads
        _attention("att_gqa_ragged", 8, 32, 8, 128, 128, 8191, ragged=True, dtype="bf16"),
        # eight long requests: the largest stream of cache bytes
        _attention("att_8x32k", 8, 16, 16, 128, 32, 32768, dtype="bf16"),
        # five drafted tokens per request checked at once, within a sliding window
        _attention("att_draft", 4, 16, 4, 64, 32, 4096, queries=5, window=1500, ragged=True, dtype="bf16"),
        # a 1,024-token chunk of a prompt over a 7B model's 4,096-token context
        _attention("att_chunk", 1, 32, 32, 128, 64, 4096, queries=1024, dtype="bf16"),
        # the K and V of one step of eight requests, stored
        _append("append_step", 8, 16, 128, 32, 2304, 1),
        # the K and V of one layer of two uneven prompts, stored
        _append("append_prompt", 2, 32, 128, 64, 4096, 4001, ragged=True, dtype="bf16"),
        # the token after one decode step
        _sample("sample_1", 1, 32000),
        # the tokens of a small batch, odd vocabulary, 16-bit logits
        _sample("sample_8", 8, 50001, min_p=False, dtype="bf16"),
        # the tokens of a large batch over a large vocabulary
        _sample("sample_64", 64, 131072),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attention", "attention", "chunk", "append", "sample"])
    dim = rng.choice([64, 128])
    group = rng.choice([g for g in (32, 64, 128) if g <= dim])
    if kind == "attention":
        kv_heads = rng.choice([1, 2, 4, 5, 8, 16, 32])
        heads = kv_heads * rng.choice([g for g in (1, 2, 3, 4, 7, 8) if g * kv_heads <= 64])
        batch = rng.choice([1, 1, 2, 3, 5, 8])
        ctx = _log(rng, 1, min(32768, 8 * 16 * 32768 // (batch * kv_heads)))
        queries = rng.choice([1, 1, 1, 2, 3, 8])
        queries = min(queries, ctx)
        window = rng.choice([0, 0, 0, _log(rng, 1, ctx)])
        return _attention("", batch, heads, kv_heads, dim, group, ctx, queries, window, rng.random() < 0.5,
                          rng.choice(["fp16", "bf16", "fp32"]))
    if kind == "chunk":
        kv_heads = rng.choice([1, 4, 8, 16])
        heads = kv_heads * rng.choice([1, 2, 4])
        heads = min(heads, 32)
        heads -= heads % kv_heads
        ctx = _log(rng, 100, 4096)
        queries = min(ctx, _log(rng, 17, 1024))
        return _attention("", rng.choice([1, 1, 2]) if heads <= 16 else 1, heads, kv_heads, dim, group, ctx, queries,
                          rng.choice([0, 0, _log(rng, 1, ctx)]), rng.random() < 0.3, "bf16")
    if kind == "append":
        batch, kv_heads = rng.choice([1, 2, 3, 8]), rng.choice([1, 4, 8, 16, 32])
        tokens = _log(rng, 1, min(4000, 250000 // (batch * kv_heads)))
        return _append("", batch, kv_heads, dim, group, tokens + _log(rng, 1, 300), tokens, rng.random() < 0.5,
                       rng.choice(["fp16", "bf16", "fp32"]))
    vocab = _log(rng, 100, 131072)
    rows = _log(rng, 1, min(256, 64 * 131072 // vocab))
    return _sample("", rows, vocab, rng.random() < 0.7, rng.random() < 0.7, rng.random() < 0.7,
                   rng.choice(["fp32", "fp32", "fp16", "bf16"]))


def _lens(c):
    """(keys, new tokens) of every request of an attention case."""
    lens, news = [], []
    for b in range(c["batch"]):
        r = SHARE[b % 8] if c["ragged"] else 1.0
        lens.append(max(1, int(c["ctx"] * r)))
        news.append(max(1, min(lens[-1], int(c["queries"] * (SHARE[(b + 4) % 8] if c["ragged"] else 1.0)))))
    return lens, news


def _places(c):
    """(start, new tokens) of every request of an append case."""
    news = [max(1, int(c["tokens"] * (SHARE[b % 8] if c["ragged"] else 1.0))) for b in range(c["batch"])]
    return [(c["ctx"] - n) * (b + 1) // (c["batch"] + 1) for b, n in enumerate(news)], news


def work(case):
    c = case
    if c["op"] == "sample":
        n = c["rows"] * c["vocab"]
        return {"bytes": n * SIZE[c["dtype"]] + c["rows"] * 28, "flops": 12 * n}
    row = c["dim"] // 2 + 4 * (c["dim"] // c["group"])     # bytes of one stored K or V row of a head
    if c["op"] == "append":
        n = sum(_places(c)[1]) * c["kv_heads"]
        # stored from the inputs, and read back into fp16
        return {"bytes": 2 * n * (c["dim"] * (SIZE[c["dtype"]] + 2) + 2 * row), "flops": 2 * n * c["dim"] * 8}
    keys = pairs = rows = 0
    for n, t in zip(*_lens(c)):
        w = c["window"] or n
        first = max(0, n - t + 1 - w)
        keys += n - first
        pairs += sum(min(w, n - t + 1 + i) for i in range(t))
        rows += t
    return {"bytes": 2 * keys * c["kv_heads"] * row + 2 * rows * c["heads"] * c["dim"] * SIZE[c["dtype"]],
            "flops": 4 * pairs * c["heads"] * c["dim"]}


# ---- inputs --------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(0x5eed + seed)
    return g


def _kv(shape, dtype, g):
    """K or V as it comes: N(0, 1) with 0.1 % of the entries at +-20."""
    x = torch.randn(shape, generator=g, device="cuda")
    big = torch.rand(shape, generator=g, device="cuda") < 1e-3
    return torch.where(big, torch.copysign(torch.tensor(20.0, device="cuda"), x), x).to(DTYPES[dtype])


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _inputs(c, seed):
    g = _gen(seed)
    if c["op"] == "sample":
        n, v = c["rows"], c["vocab"]
        # logits of a peaked head (a few likely tokens) over a broad one
        x = torch.randn(n, v, generator=g, device="cuda") * 1.8
        x += 6.0 * torch.rand(n, v, generator=g, device="cuda").pow(40)
        pick = torch.rand(4, n, generator=g, device="cuda")
        t = torch.where(pick[0] < 0.1, torch.zeros_like(pick[0]), 0.6 + 0.8 * pick[0])
        k = torch.where(pick[1] < 0.3, torch.zeros_like(pick[1]), (10 + 400 * pick[1]).floor())
        p = torch.where(pick[2] < 0.2, torch.ones_like(pick[2]), 0.5 + 0.49 * pick[2])
        m = torch.where(pick[3] < 0.3, torch.zeros_like(pick[3]), 0.1 * pick[3])
        u = torch.rand(n, generator=g, device="cuda")
        return {"logits": x.to(DTYPES[c["dtype"]]), "u": u, "temperature": t,
                "top_k": k.to(torch.int32) if c["top_k"] else None,
                "top_p": p if c["top_p"] else None, "min_p": m if c["min_p"] else None}
    b, h, d = c["batch"], c["kv_heads"], c["dim"]
    if c["op"] == "append":
        # K and V as slices of one fused projection's output
        qkv = _kv((b, c["tokens"], 3 * h, d), c["dtype"], g)
        return {"k": qkv[:, :, h:2 * h], "v": qkv[:, :, 2 * h:]}
    q = (torch.randn(b, c["queries"], c["heads"], d, generator=g, device="cuda") * 1.5).to(DTYPES[c["dtype"]])
    return {"q": q, "k": _kv((b, c["ctx"], h, d), "fp16", g), "v": _kv((b, c["ctx"], h, d), "fp16", g)}


def prepare(case, seed):
    c = case
    state = {"case": c, **_inputs(c, seed)}
    if c["op"] == "sample":
        return state
    b, h, d, g = c["batch"], c["kv_heads"], c["dim"], c["group"]
    if c["op"] == "append":
        start, news = _places(c)
        state["start"], state["news"] = _i32(start), _i32(news) if c["ragged"] else None
        state["out"] = [torch.zeros(b, c["tokens"], h, d, dtype=torch.float16, device="cuda") for _ in range(2)]
        if own:
            from autoregressive_decode_gb300 import kie
            state["cache"] = kie.KV4Cache(b, h, c["ctx"], d, g)
            return state
        state["rows"] = torch.tensor([i for i, n in enumerate(news) for _ in range(n)], device="cuda")
        state["cols"] = torch.tensor([t for n in news for t in range(n)], device="cuda")
        state["cache"] = [_empty(b, h, c["ctx"], d, g) for _ in range(2)]
        return state
    lens, news = _lens(c)
    state["lens"], state["news"] = _i32(lens), _i32(news) if c["ragged"] else None
    state["out"] = torch.zeros_like(state["q"])
    k, v = state.pop("k"), state.pop("v")
    if own:
        from autoregressive_decode_gb300 import kie
        state["cache"] = kie.KV4Cache(b, h, c["ctx"], d, g)
        state["cache"].append(k, v, _i32([0] * b))
    else:
        state["cache"] = [tuple(x.transpose(1, 2).contiguous() for x in _quantise(y, g)) for y in (k, v)]
        state["new"] = _i32(news)
    return state


# ---- plain forms ---------------------------------------------------------------------------------
def _empty(b, h, n, d, g):
    return (torch.zeros(b, h, n, d // g, g, dtype=torch.uint8, device="cuda"),
            torch.zeros(b, h, n, d // g, 1, dtype=torch.float16, device="cuda"),
            torch.zeros(b, h, n, d // g, 1, dtype=torch.float16, device="cuda"))


def _quantise(x, g):
    """(codes, scale, zero) of each group of g channels."""
    x = x.float().clamp(-65504.0, 65504.0).half().float()
    x = x.reshape(*x.shape[:-1], x.shape[-1] // g, g)
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = ((hi - lo) / 15.0).half()
    sf = s.float()
    code = torch.round((x - lo) / torch.where(sf == 0, torch.ones_like(sf), sf)).clamp(0, 15)
    code = torch.where(sf == 0, torch.zeros_like(code), code)
    return code.to(torch.uint8), s, lo.half()


def _values(code, s, z):
    x = code.float() * s.float() + z.float()
    return x.reshape(*x.shape[:-2], x.shape[-2] * x.shape[-1])


def _run_append(st):
    c, rows, cols = st["case"], st["rows"], st["cols"]
    at = (st["start"][rows] + cols).long()
    for x, cache, out in zip((st["k"], st["v"]), st["cache"], st["out"]):
        for kept, new in zip(cache, _quantise(x[rows, cols], c["group"])):
            kept[rows, :, at] = new
        out[rows, cols] = _values(*(kept[rows, :, at] for kept in cache)).half()
    return st["out"]


def _run_attention(st):
    c, q, new = st["case"], st["q"].float(), st["new"]
    k, v = (_values(*x) for x in st["cache"])                              # [b, h, ctx, d]
    b, t, hq, d = q.shape
    h = k.shape[1]
    q = q.transpose(1, 2).reshape(b, h, (hq // h) * t, d)
    s = (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    s = s.reshape(b, h, hq // h, t, -1)
    j = torch.arange(c["ctx"], device="cuda")
    i = torch.arange(t, device="cuda")
    last = (st["lens"] - new)[:, None] + i                                 # the last key each query sees
    seen = j <= last[:, :, None]
    if c["window"]:
        seen &= j > last[:, :, None] - c["window"]
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp_min(-3.0e38)
    p = torch.exp(s.sub_(m))
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(b, h, (hq // h) * t, -1) @ v).reshape(b, h, hq // h, t, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.reshape(b, hq, t, d).transpose(1, 2)
    there = (i < new[:, None])[:, :, None, None]
    return torch.where(there, o.to(st["q"].dtype), st["out"])


def _run_sample(st):
    x = st["logits"].double()
    n, v = x.shape
    temperature = st["temperature"].double()[:, None]
    best = x.amax(1, keepdim=True)
    w = torch.exp((x - best) / torch.where(temperature > 0, temperature, torch.ones_like(temperature)))
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    ranked = w.gather(1, order)
    keep = torch.ones_like(ranked, dtype=torch.bool)
    if st["top_k"] is not None:
        k = st["top_k"][:, None]
        keep &= (k <= 0) | (torch.arange(v, device="cuda") < k)
    if st["top_p"] is not None:
        p = st["top_p"].double()[:, None]
        mass = torch.where(keep, ranked, torch.zeros_like(ranked))
        before = mass.cumsum(1) - mass
        keep &= (p >= 1) | (before < p * mass.sum(1, keepdim=True))
        keep[:, 0] = True
    if st["min_p"] is not None:
        keep &= ranked >= st["min_p"].double()[:, None]
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(keep, ranked, torch.zeros_like(ranked)))
    run_ = kept.cumsum(1)
    total = run_[:, -1:]
    token = (run_ <= st["u"].double()[:, None] * total).sum(1).clamp_max(v - 1)
    greedy = ~(temperature[:, 0] > 0)
    # the first of the largest logits
    first = (x == best).to(torch.uint8).argmax(1)
    prob = kept.gather(1, token[:, None])[:, 0] / total[:, 0]
    return (torch.where(greedy, first, token).to(torch.int32),
            torch.where(greedy, torch.ones_like(prob), prob).float())


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"append": _run_append, "attention": _run_attention, "sample": _run_sample}[op](state)
    if op == "append":
        cache, out = state["cache"], state["out"]
        cache.append(state["k"], state["v"], state["start"], n_tok=state["news"])
        cache.read(state["start"], out[0].shape[1], n_tok=state["news"], out=out)
        return out
    if op == "attention":
        return state["cache"].attention(state["q"], state["lens"], n_tok=state["news"],
                                        window=state["case"]["window"], out=state["out"])
    from autoregressive_decode_gb300 import kie
    return kie.sample(state["logits"], state["u"], temperature=state["temperature"], top_k=state["top_k"],
                      top_p=state["top_p"], min_p=state["min_p"])


# ---- in 64 bits, from the definitions ----------------------------------------------------------------
def _stored(x, g):
    """The values a 4-bit group stands for, in 64 bits.  The stored scale and
    the code are defined with fp32 differences and quotients: a 64-bit one,
    rounded, is the same number."""
    f = x.double().cpu().numpy()
    f = np.clip(f, -65504.0, 65504.0).astype(np.float16).astype(np.float64)
    f = f.reshape(*f.shape[:-1], -1, g)
    low = f.min(-1, keepdims=True)
    span = (f.max(-1, keepdims=True) - low).astype(np.float32).astype(np.float64)
    s = (span / 15.0).astype(np.float32).astype(np.float16).astype(np.float64)
    diff = (f - low).astype(np.float32).astype(np.float64)
    code = np.rint(np.divide(diff, s, out=np.zeros_like(diff), where=s > 0).astype(np.float32))
    out = np.clip(code, 0, 15).astype(np.float64) * s + low
    return out.reshape(x.shape)


def exact(case, seed):
    c = case
    x = _inputs(c, seed)
    if c["op"] == "append":
        out = []
        for y in (x["k"], x["v"]):
            o = np.zeros(y.shape)
            full = _stored(y, c["group"])
            for b, n in enumerate(_places(c)[1]):
                o[b, :n] = full[b, :n]
            out.append(torch.from_numpy(o))
        return out
    if c["op"] == "attention":
        if c["batch"] * c["kv_heads"] * c["ctx"] * c["dim"] > 2 ** 28:   # a minute of host work
            return None
        q = x["q"].double()
        out = torch.zeros_like(q)
        k, v = (torch.from_numpy(_stored(y, c["group"])).cuda() for y in (x["k"], x["v"]))
        each = c["heads"] // c["kv_heads"]
        for b, (n, t) in enumerate(zip(*_lens(c))):
            for head in range(c["heads"]):
                kk, vv = k[b, :n, head // each], v[b, :n, head // each]
                for t0 in range(0, t, 256):
                    t1 = min(t, t0 + 256)
                    s = torch.einsum("td,jd->tj", q[b, t0:t1, head], kk) / math.sqrt(c["dim"])
                    far = torch.arange(n - t + t0, n - t + t1, device=s.device)[:, None] - torch.arange(n, device=s.device)
                    s = torch.where((far < 0) | (far >= (c["window"] or n + 1)), -math.inf, s)
                    out[b, t0:t1, head] = torch.softmax(s, -1) @ vv
        return out
    rows = []
    for i in range(c["rows"]):
        lg = x["logits"][i].double().cpu().numpy()
        t = float(x["temperature"][i])
        if t <= 0:
            rows.append((int(np.argmax(lg)), 1.0))
            continue
        w = np.exp((lg - lg.max()) / t)
        order = np.argsort(-lg, kind="stable")
        if x["top_k"] is not None and int(x["top_k"][i]) > 0:
            order = order[:int(x["top_k"][i])]
        if x["top_p"] is not None and float(x["top_p"][i]) < 1:
            run_ = np.cumsum(w[order])
            order = order[:1 + int(np.searchsorted(run_, float(x["top_p"][i]) * run_[-1]))]
        if x["min_p"] is not None:
            order = order[w[order] >= float(x["min_p"][i])]
        ids = np.sort(order)
        run_ = np.cumsum(w[ids])
        at = min(int(np.searchsorted(run_, float(x["u"][i]) * run_[-1], side="right")), len(ids) - 1)
        rows.append((int(ids[at]), w[ids[at]] / run_[-1]))
    return (torch.tensor([r[0] for r in rows], dtype=torch.int32),
            torch.tensor([r[1] for r in rows], dtype=torch.float64))
