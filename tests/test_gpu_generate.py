"""The operators together, as a decode loop uses them: an engine's sampled
generation against its own steps and kie.sample, and a layer's step of append,
attention and sampling, captured once and replayed over growing lengths."""
import numpy as np
import pytest

import synthetic as S
from _common import engine_for
from autoregressive_decode_gb300 import kie

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TINY = S.WORKLOADS["tiny"]
MEDIUM = S.Workload("medium", 5, 2, 1024, 8, 128, 4608, 10007, prompt_len=100, decode_steps=24)


def params(b, **kw):
    types = {"temperature": torch.float32, "top_k": torch.int32, "top_p": torch.float32, "min_p": torch.float32}
    return {n: torch.full((b,), v, dtype=types[n], device="cuda") for n, v in kw.items()}


def batched(w, weights, b):
    e = kie.Engine(kie.make_config(w.n_layers, w.d_model, w.n_heads, w.head_dim, w.ffn_dim, w.vocab, w.max_ctx,
                                   w.rms_eps, w.rope_theta, batch=b))
    e.load_weights(weights)
    for r in range(b):
        e.select_request(r)
        e.prefill(S.gen_prompt(w, n=w.prompt_len - 3 * r, seed=11 + r), want_logits=False)
    return e


@pytest.mark.parametrize("w", [TINY, MEDIUM], ids=lambda w: w.name)
@pytest.mark.parametrize("mode", ["persistent", "graph"])
@pytest.mark.parametrize("kw", [dict(), dict(temperature=0.7, top_k=40), dict(top_p=0.9, min_p=0.01)],
                         ids=["plain", "k", "p"])
def test_sampled_generation_is_steps_and_draws(w, mode, kw):
    """Tokens and probabilities equal those of decode_step and kie.sample in turn."""
    weights = S.gen_weights(w)
    prompt = S.gen_prompt(w)
    n = 8
    u = torch.rand(n, 1, generator=torch.Generator().manual_seed(3)).cuda()
    p = params(1, **kw)
    e = engine_for(w, weights, mode)
    e.prefill(prompt, want_logits=False)
    toks = torch.full((n, 1), -7, dtype=torch.int32, device="cuda")
    probs = torch.zeros(n, 1, device="cuda")
    torch.cuda.synchronize()
    e.generate_sampled_device(5, u, toks, probs, **p)
    e.sync()
    assert e.pos == len(prompt) + n
    r = engine_for(w, weights, mode)
    r.prefill(prompt, want_logits=False)
    tok = 5
    for t in range(n):
        _, lg = r.decode_step(tok)
        got, prob = kie.sample(torch.tensor(lg[None]).cuda(), u[t], **p)
        tok = int(got)
        assert tok == int(toks[t]) and float(prob) == float(probs[t])
    # the engine goes on from there
    assert e.decode_step(tok, want_logits=False)[0] == r.decode_step(tok, want_logits=False)[0]


@pytest.mark.parametrize("mode", ["persistent", "graph"])
def test_temperature_zero_is_greedy(mode):
    weights = S.gen_weights(MEDIUM)
    prompt = S.gen_prompt(MEDIUM)
    out = []
    for sampled in (False, True):
        e = engine_for(MEDIUM, weights, mode)
        e.prefill(prompt, want_logits=False)
        if sampled:
            toks = torch.zeros(10, 1, dtype=torch.int32, device="cuda")
            u = torch.rand(10, 1, device="cuda")
            torch.cuda.synchronize()
            e.generate_sampled_device([9], u, toks, **params(1, temperature=0.0))
            e.sync()
            out.append(toks.cpu().numpy()[:, 0])
        else:
            out.append(np.array(step_by_step(e, 9, 10)))
    np.testing.assert_array_equal(out[0], out[1])


def step_by_step(e, tok, n):
    """Greedy tokens of n single steps."""
    got = []
    for _ in range(n):
        tok, _ = e.decode_step(tok, want_logits=False)
        got.append(tok)
    return got


def test_batched_sampled_generation():
    """Requests at different positions with parameters of their own."""
    w, b, n = MEDIUM, 5, 6
    weights = S.gen_weights(w)
    u = torch.rand(n, b, generator=torch.Generator().manual_seed(4)).cuda()
    p = {"temperature": torch.tensor([0.0, 1.0, 0.5, 2.0, 1.0], device="cuda"),
         "top_k": torch.tensor([0, 5, 100, 0, 2000], dtype=torch.int32, device="cuda"),
         "top_p": torch.tensor([0.5, 1.0, 0.8, 0.9, 0.99], device="cuda")}
    firsts = [1, 2, 3, 4, 5]
    e = batched(w, weights, b)
    toks = torch.zeros(n, b, dtype=torch.int32, device="cuda")
    probs = torch.zeros(n, b, device="cuda")
    torch.cuda.synchronize()
    e.generate_sampled_device(firsts, u, toks, probs, **p)
    e.sync()
    r = batched(w, weights, b)
    cur = firsts
    for t in range(n):
        _, lg = r.decode_batch(cur)
        got, prob = kie.sample(torch.tensor(lg).cuda(), u[t], **p)
        assert torch.equal(got, toks[t]) and torch.equal(prob, probs[t])
        cur = got.cpu().numpy()
    for q in range(b):
        e.select_request(q)
        assert e.pos == w.prompt_len - 3 * q + n


def test_sampled_generation_refusals():
    w = TINY
    e = engine_for(w, S.gen_weights(w))
    toks = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    u = torch.zeros(4, 1, device="cuda")
    with pytest.raises(ValueError):
        e.generate_sampled_device([1, 2], u, toks)
    with pytest.raises(ValueError):
        e.generate_sampled_device(1, u, toks[:3])
    with pytest.raises(ValueError):
        e.generate_sampled_device(1, u.double(), toks)
    with pytest.raises(ValueError):
        e.generate_sampled_device(1, u, toks, top_k=torch.zeros(1, device="cuda"))
    with pytest.raises(kie.KieError):
        e.generate_sampled_device(w.vocab, u, toks)
    e.set_pos(w.max_ctx - 3)
    with pytest.raises(kie.KieError):
        e.generate_sampled_device(1, u, toks)
    assert e.pos == w.max_ctx - 3 and int(toks.abs().sum()) == 0
    e.generate_sampled_device(1, u[:0], toks[:0])
    assert e.pos == w.max_ctx - 3


def test_append_attention_sample_in_one_graph():
    """A step of one layer: the new K and V are appended, the new query attends to
    all, a projection of the result is sampled, the lengths advance.  One graph,
    captured at the first step and replayed, gives what the calls give one by one,
    and what they give agrees with the formula over the values read back."""
    b, hq, hkv, hd, ctx, steps, vocab = 3, 8, 2, 128, 300, 6, 700
    g = torch.Generator(device="cuda").manual_seed(5)

    def rand(*s):
        return torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    qkv = rand(steps, b, 1, (hq + 2 * hkv) * hd)             # of a fused projection: strided parts
    pk, pv = rand(b, 250, hkv, hd), rand(b, 250, hkv, hd)
    proj = (rand(hq * hd, vocab).float() * 0.2)
    start_len = torch.tensor([250, 1, 64], dtype=torch.int32, device="cuda")
    u = torch.rand(steps, b, generator=g, device="cuda")
    top_k = torch.tensor([20, 0, 300], dtype=torch.int32, device="cuda")
    top_p = torch.tensor([0.95, 0.9, 1.0], device="cuda")

    def fresh():
        c = kie.KV4Cache(b, hkv, ctx, hd)
        c.append(pk, pv, torch.zeros(b, dtype=torch.int32, device="cuda"), start_len)
        return c

    def step(c, x, un, pos, out, toks, probs):
        q = x[..., :hq * hd].view(b, 1, hq, hd)
        k = x[..., hq * hd:(hq + hkv) * hd].view(b, 1, hkv, hd)
        v = x[..., (hq + hkv) * hd:].view(b, 1, hkv, hd)
        c.append(k, v, pos)
        pos += 1
        c.attention(q, pos, out=out)
        kie.sample(out.view(b, hq * hd).float() @ proj, un, top_k=top_k, top_p=top_p, tokens=toks, probs=probs)

    def buffers():
        return (torch.zeros(b, 1, hq, hd, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(b, dtype=torch.int32, device="cuda"), torch.zeros(b, device="cuda"))
    plain, c, pos = [], fresh(), start_len.clone()
    out, toks, probs = buffers()
    for t in range(steps):
        step(c, qkv[t], u[t], pos, out, toks, probs)
        plain.append((out.clone(), toks.clone(), probs.clone()))
    # against the formula in 64 bits
    kk, vv = c.read(torch.zeros(b, dtype=torch.int32, device="cuda"), ctx, n_tok=pos, dtype=torch.float32)
    for t in range(steps):
        for r in range(b):
            n = int(start_len[r]) + t + 1
            q = qkv[t, r, 0, :hq * hd].double().view(hkv, hq // hkv, hd)
            s = torch.einsum("hgd,nhd->hgn", q, kk[r, :n].double()) * hd ** -0.5
            o = torch.einsum("hgn,nhd->hgd", torch.softmax(s, -1), vv[r, :n].double()).reshape(hq, hd)
            # o is sum p (s code) + sum p z, each of whose terms is at most 3 times the head's
            # largest |v| between them (s code = v - z), not the channel's; p is rounded by
            # 2^-11 above and below the division; the result is rounded to bf16
            lim = vv[r, :n].double().abs().amax((0, 2)).repeat_interleave(hq // hkv)[:, None]
            assert ((plain[t][0][r, 0].double() - o).abs() <= 2.0 ** -8 * o.abs() + 6 * 2.0 ** -11 * lim).all()
    c, pos = fresh(), start_len.clone()
    out, toks, probs = buffers()
    x, un = qkv[0].clone(), u[0].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):                               # warm up on other data, then start over
        step(c, x, un, pos, out, toks, probs)
    torch.cuda.synchronize()
    c2 = fresh()
    pos.copy_(start_len)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(c2, x, un, pos, out, toks, probs)
    for t in range(steps):
        x.copy_(qkv[t])
        un.copy_(u[t])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, plain[t][0]) and torch.equal(toks, plain[t][1]) and torch.equal(probs, plain[t][2])
    assert pos.tolist() == (start_len + steps).tolist()
