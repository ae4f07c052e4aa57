"""Sampling on the GPU against its definition in 64 bits: tokens equal, the
probabilities to fp32 rounding."""
import math

import numpy as np
import pytest

from autoregressive_decode_gb300 import kie

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def reference(logits, u, t=1.0, k=0, p=1.0, min_p=0.0):
    """(token, probability) of one row, in fp64."""
    l = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    m = l.max()
    if m == -np.inf:
        return -1, 0.0
    if not t > 0:
        return int(np.argmax(l)), 1.0
    if m == np.inf:
        l, m = np.where(l == np.inf, 0.0, -np.inf), 0.0
    far = m - l > np.finfo(np.float32).max               # beyond fp32's range: infinite
    w = np.where(far, 0.0, np.exp(np.where(far, 0.0, l - m) / float(t)))
    order = np.argsort(-l, kind="stable")
    if 0 < k < len(l):
        order = order[:k]
    if p < 1:
        run = np.cumsum(w[order])
        order = order[:1 + min(int(np.searchsorted(run, max(float(p), 0.0) * run[-1])), len(order) - 1)]
    if min_p > 0:
        order = order[w[order] >= min(float(min_p), 1.0)]
    ids = np.sort(order[w[order] > 0])
    run = np.cumsum(w[ids])
    x = min(max(float(u), 0.0), 1.0 - 2.0 ** -53)
    at = min(int(np.searchsorted(run, x * run[-1], side="right")), len(ids) - 1)
    return int(ids[at]), w[ids[at]] / run[-1]


def run_and_check(x, u, t=None, k=None, p=None, m=None, **kw):
    n = x.shape[0]

    def dev(a, dtype):
        return None if a is None else torch.tensor(np.broadcast_to(np.asarray(a), (n,)).copy(), dtype=dtype, device="cuda")
    tu, tt, tk = dev(u, torch.float32), dev(t, torch.float32), dev(k, torch.int32)
    tp, tm = dev(p, torch.float32), dev(m, torch.float32)
    tok, prob = kie.sample(x, tu, tt, tk, tp, tm, **kw)
    rows = x.float().cpu().numpy()
    tok, prob = tok.cpu().numpy(), prob.cpu().numpy()
    val = lambda a, i, d: d if a is None else a[i].item()  # noqa: E731
    for i in range(n):
        rt, rp = reference(rows[i], tu[i].item(), val(tt, i, 1.0), val(tk, i, 0), val(tp, i, 1.0), val(tm, i, 0.0))
        assert tok[i] == rt, (i, tok[i], rt)
        # the mass ratio is good to 2^-37, then rounded to fp32
        assert abs(prob[i] - rp) <= rp * 2.0 ** -23, (i, prob[i], rp)
    return tok, prob


def logits(rows, vocab, seed, dtype="fp32", std=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, vocab, generator=g) * std + 5.0 * torch.rand(rows, vocab, generator=g).pow(30)
    return x.to(TYPES[dtype]).cuda()


def uniform(n, seed):
    return torch.rand(n, generator=torch.Generator().manual_seed(seed)).numpy()


@pytest.mark.parametrize("vocab", [1, 2, 31, 1000, 4096, 32000, 50001, 131072, 262144])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_no_filter(vocab, dtype):
    run_and_check(logits(5, vocab, vocab, dtype), uniform(5, 1), t=[1.0, 0.3, 2.0, 0.0, 1e-6])


@pytest.mark.parametrize("rows,vocab", [(1, 32000), (3, 777), (40, 5000), (170, 2049)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("which", ["k", "p", "m", "kp", "km", "pm", "kpm"])
def test_filters(rows, vocab, dtype, which):
    g = np.random.default_rng(rows * 7 + vocab)
    kw = {"t": g.uniform(0.4, 1.5, rows)}
    if "k" in which:
        kw["k"] = g.choice([0, 1, 2, 5, 40, 300, 5000, -3], rows)
    if "p" in which:
        kw["p"] = g.choice([0.0, 0.01, 0.5, 0.9, 0.999, 1.0], rows)
    if "m" in which:
        kw["m"] = g.choice([0.0, 0.01, 0.2, 0.9, 1.0, 3.0], rows)
    run_and_check(logits(rows, vocab, 3, dtype), g.random(rows), **kw)


@pytest.mark.parametrize("vocab", [50, 1500, 40000])
def test_equal_logits(vocab):
    """One value, and two: the filters cut inside the crowd, lowest ids first."""
    x = torch.zeros(6, vocab, device="cuda")
    x[3:, ::3] = 1.0
    u = [0.0, 0.5, 0.999999, 0.0, 0.5, 0.999999]
    tok, _ = run_and_check(x, u, k=[7, vocab // 2, vocab - 1, 5, vocab // 2, 3])
    assert tok[0] == 0 and tok[2] == vocab - 2
    run_and_check(x, u, p=[0.25, 0.5, 0.7, 0.25, 0.9, 0.1])
    run_and_check(x, u, k=[7, 9, vocab - 1, 5, 6, 3], p=[0.5] * 6)


def test_near_equal_logits():
    """Neighbouring fp32 values: the order is decided in the last bits."""
    n = 5000
    base = np.full(n, 1.0, np.float32).view(np.int32)
    x = (base + np.random.default_rng(5).integers(0, 700, n)).astype(np.int32).view(np.float32)
    x = torch.tensor(np.stack([x, x, -x, x * 2 ** 20])).cuda()
    run_and_check(x, [0.1, 0.9, 0.5, 0.3], t=[1.0, 1e-3, 1.0, 1.0], k=[1000, 2500, 17, 400])
    run_and_check(x, [0.1, 0.9, 0.5, 0.3], p=[0.3, 0.5, 0.7, 0.2])


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_prefix_ends_near_zero(dtype):
    """Logits around zero, where neighbouring numbers are many: the prefix ends just
    inside a bin that spans zero, and its keys reach into the bin before."""
    rows, vocab = 76, 8200
    g = np.random.default_rng(8)
    x = logits(rows, vocab, 4, dtype, std=0.01)
    for p in (None, 0.85, 0.9, 0.97):
        run_and_check(x, g.random(rows), k=g.integers(2000, 6000, rows), p=p)
    run_and_check(x, g.random(rows), p=g.uniform(0.3, 0.99, rows))


def test_masks_and_extremes():
    v = 3000
    inf, low = math.inf, torch.finfo(torch.float32).min
    x = logits(12, v, 9)
    x[0] = -inf
    x[1] = -inf
    x[1, 17] = -4.0
    x[2, 5:] = low
    x[3] = low
    x[4] = math.nan
    x[5, ::2] = math.nan
    x[6, [3, 900, 2999]] = inf
    x[7] = -inf
    x[7, [100, 200]] = inf
    x[8, :] = low
    x[8, 9] = torch.finfo(torch.float32).max
    x[9, 10:] = -inf
    x[10] = 1e-42
    x[11, ::5] = 65504.0
    u = uniform(12, 4)
    for kw in ({}, {"k": 4}, {"p": 0.6}, {"m": 0.5}, {"k": 2000, "p": 0.99, "m": 1e-6}, {"t": 0.0}, {"t": -1.0},
               {"t": math.nan}, {"t": 1e30}, {"t": 1e-42}, {"t": math.inf}):
        tok, _ = run_and_check(x, u, **kw)
        assert tok[0] == -1 and tok[4] == -1 and tok[1] == 17


def test_random_numbers_at_the_ends():
    x = logits(8, 500, 12)
    x[:, 0] = -math.inf
    x[:, -1] = -math.inf
    tok, _ = run_and_check(x, [0.0, -1.0, 1.0, 2.0, 1.0 - 2.0 ** -24, 2.0 ** -60, math.inf, -math.inf])
    assert list(tok[:2]) == [1, 1] and tok[2] == tok[3] == tok[6] == 498


def test_strides_outputs_and_streams():
    big = logits(7, 4001, 21)
    x = big[:, 1:3908]                                    # rows that start on odd addresses
    tok = torch.full((7,), -9, dtype=torch.int32, device="cuda")
    prob = torch.zeros(7, device="cuda")
    run_and_check(x, uniform(7, 2), k=50, tokens=tok, probs=prob)
    s = torch.cuda.Stream()
    u = torch.tensor(uniform(7, 2), device="cuda")
    k = torch.full((7,), 50, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t2, p2 = kie.sample(x, u, top_k=k, stream=s)
    s.synchronize()
    assert torch.equal(t2, tok) and torch.equal(p2, prob)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        kie.sample(x, u, top_k=k, tokens=t2, probs=p2)
    t2.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(t2, tok)
    wide = logits(1, 1000, 3).expand(6, 1000)             # one row of logits, six draws
    run_and_check(wide, uniform(6, 8), p=0.8)


def test_distribution():
    """20,000 draws from one row: frequencies within six standard deviations."""
    n = 20000
    x = torch.tensor([[1.0, 0.0, 2.0, -1.0, 1.5]], device="cuda")
    u = torch.rand(n, generator=torch.Generator().manual_seed(77)).cuda()
    tok, _ = kie.sample(x.expand(n, 5), u)
    p = torch.softmax(x[0].double(), 0).cpu().numpy()
    f = np.bincount(tok.cpu().numpy(), minlength=5) / n
    assert (np.abs(f - p) <= 6 * np.sqrt(p * (1 - p) / n)).all()
