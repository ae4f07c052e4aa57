"""The 4-bit K/V cache on the GPU: storing and reading against the format's
definition bit for bit, attention against a plain one in 64 bits."""
import math

import numpy as np
import pytest

from autoregressive_decode_gb300 import kie

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def gen(shape, seed, dtype="fp16", std=1.0, outliers=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * std
    if outliers:
        x = torch.where(torch.rand(shape, generator=g) < 2e-3, 20.0 * std * torch.sign(x), x)
    return x.to(TYPES[dtype]).cuda()


def stored(x, group):
    """Values that the cache stands for, in fp64, from the definition."""
    f = np.nan_to_num(x.double().cpu().numpy(), nan=0.0, posinf=65504.0, neginf=-65504.0)
    f = np.clip(f, -65504.0, 65504.0).astype(np.float32).astype(np.float16).astype(np.float32)
    g = f.reshape(*f.shape[:-1], -1, group)
    z = g.min(-1, keepdims=True)
    s = ((g.max(-1, keepdims=True) - z).astype(np.float32) / np.float32(15)).astype(np.float16).astype(np.float32)
    q = np.divide((g - z).astype(np.float32), s, out=np.zeros_like(g), where=s > 0)
    code = np.clip(np.rint(q), 0, 15)
    return (code.astype(np.float64) * s + z).reshape(f.shape)


def reference(q, k, v, lens, news, causal=True, window=0, scale=None):
    """softmax(scale q k^T) v in fp64; q torch [b, t, hq, d], k, v numpy [b, n, h, d].
    Returns (out, largest sum |q k|, largest |v|)."""
    q = q.double().cpu().numpy()
    b_, t_, hq, d = q.shape
    per = hq // k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    out = np.zeros_like(q)
    smax = vmax = 0.0
    for b in range(b_):
        n = lens[b]
        for t in range(news[b]):
            hi = min(n, max(0, n - news[b] + t + 1)) if causal else n
            lo = max(0, n - news[b] + t + 1 - window) if window else 0
            if hi <= lo:
                continue
            for h in range(hq):
                kk, vv = k[b, lo:hi, h // per], v[b, lo:hi, h // per]
                s = kk @ q[b, t, h] * scale
                p = np.exp(s - s.max())
                out[b, t, h] = p @ vv / p.sum()
                smax = max(smax, float((np.abs(kk) @ np.abs(q[b, t, h])).max()) * abs(scale))
                vmax = max(vmax, float(np.abs(vv).max()))
    return out, smax, vmax


def tolerance(dtype, ref, smax, vmax):
    """Scores carry 2^-20 of their sum of magnitudes (q in two fp16 parts, 2^-22;
    fp32 products and sums), so each probability 2^-20 smax relative, twice for
    the normalisation; probabilities 2^-20 more from exp and their two fp16
    parts, or 2^-11 in bf16's one; then the result's own rounding."""
    p = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -20
    return (2 * 2.0 ** -20 * smax + 2 * p) * vmax + np.abs(ref) * torch.finfo(TYPES[dtype]).eps / 2 + 1e-30


def check(out, q, k, v, lens, news, dtype, **kw):
    ref, smax, vmax = reference(q, k, v, lens, news, **kw)
    got = out.double().cpu().numpy()
    err = np.abs(got - ref)
    for b, n in enumerate(news):
        bad = err[b, :n] > tolerance(dtype, ref[b, :n], smax, vmax)
        assert not bad.any(), (b, float(err[b, :n].max()), smax, vmax)


# ---- store and read ------------------------------------------------------------------------------
@pytest.mark.parametrize("dim,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_append_and_read_bit_exact(dim, group, dtype):
    b, h, n, ctx = 3, 5, 37, 101
    k, v = gen((b, n, h, dim), 1, dtype), gen((b, n, h, dim), 2, dtype, std=1e-2)
    k[0, 0, 0] = 0.25                                     # constant
    k[0, 1, 0] = 0.0
    k[0, 2, 0, ::2] = -0.0
    k[0, 3, 0] = torch.linspace(-65504, 65504, dim).to(k.dtype)
    k[0, 4, 0, 3], k[0, 4, 0, 5] = math.inf, -math.inf
    k[0, 5, 0, 7] = math.nan
    k[0, 6, 0] = torch.arange(dim).to(k.dtype) * 2.0 ** -24      # fp16 subnormals
    k[0, 7, 0] = torch.arange(dim).to(k.dtype) * 0.5             # exact halves between codes
    cache = kie.KV4Cache(b, h, ctx, dim, group)
    start, news = i32(0, 60, 90), i32(n, n - 5, 20)
    cache.append(k, v, start, n_tok=news)
    out = [torch.full((b, n, h, dim), 7.0, device="cuda") for _ in range(2)]
    cache.read(start, n, n_tok=news, out=out)
    # request 2's tokens from position 101 on are outside the cache, rows past n_tok are left alone
    count = [n, n - 5, 11]
    for x, y in zip((k, v), out):
        ref = stored(x, group)
        for i, m in enumerate(count):
            np.testing.assert_array_equal(y[i, :m].cpu().numpy(), ref[i, :m].astype(np.float32))
            assert (y[i, m:] == 7.0).all()
    for t in ("fp16", "bf16"):
        got = cache.read(start, n, n_tok=news, dtype=TYPES[t])
        for x, y in zip(out, got):
            for i, m in enumerate(count):
                lim = 65504.0 if t == "fp16" else math.inf
                assert torch.equal(x[i, :m].clamp(-lim, lim).to(TYPES[t]), y[i, :m])


def test_append_keeps_other_positions_and_takes_any_strides():
    b, h, dim, ctx = 2, 3, 128, 70
    full = gen((b, ctx, h, dim), 5)
    cache = kie.KV4Cache(b, h, ctx, dim, 64)
    cache.append(full, full, i32(0, 0))
    fused = gen((b, 9, 4 * h + 1, dim + 3), 6)            # odd rows: no 16-byte alignment
    k, v = fused[:, :, 1:1 + h, :dim], fused[:, :, 1 + h:1 + 2 * h, 1:dim + 1]
    one = gen((1, 9, 1, dim), 7).expand(b, 9, h, dim)     # broadcast
    cache.append(k, one, i32(-4, 65))                     # 4 tokens before the start, 4 past the end
    kk, vv = cache.read(i32(0, 0), ctx, dtype=torch.float32)
    want = [stored(full, 64) for _ in range(2)]
    for w, x in zip(want, (k, one)):
        s = stored(x, 64)
        w[0, 0:5], w[1, 65:70] = s[0, 4:], s[1, :5]
    np.testing.assert_array_equal(kk.cpu().numpy(), want[0].astype(np.float32))
    np.testing.assert_array_equal(vv.cpu().numpy(), want[1].astype(np.float32))


# ---- attention ------------------------------------------------------------------------------------
def filled(b, h, ctx, dim, group, lens, seed=11, kstd=1.0, vstd=1.0):
    """A cache over memory of all ones (NaN scales) with the first lens[b]
    positions stored, and their values."""
    cache = kie.KV4Cache(b, h, ctx, dim, group)
    cache.data.fill_(255)
    n = max(max(lens), 1)
    k, v = gen((b, n, h, dim), seed, std=kstd), gen((b, n, h, dim), seed + 1, std=vstd)
    cache.append(k, v, i32(*[0] * b), n_tok=i32(*lens))
    return cache, stored(k, group), stored(v, group)


@pytest.mark.parametrize("dim,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("heads,kv_heads", [(4, 4), (14, 2), (3, 1), (24, 2)])
def test_single_tokens(dim, group, dtype, heads, kv_heads):
    lens = [1, 0, 33, 517, 64, 1000]
    cache, k, v = filled(6, kv_heads, 1000, dim, group, lens)
    q = gen((6, 1, heads, dim), 3, dtype, std=1.5, outliers=False)
    out = cache.attention(q, i32(*lens))
    assert (out[1] == 0).all()
    check(out, q, k, v, lens, [1] * 6, dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("n_q,causal,window", [(2, True, 0), (5, True, 40), (37, True, 0), (37, False, 0),
                                               (70, True, 33), (131, True, 1), (300, True, 0)])
@pytest.mark.parametrize("dim,group", [(64, 32), (128, 64)])
def test_several_tokens(dtype, n_q, causal, window, dim, group):
    lens, news = [311, 4, 150, 0], [n_q, min(n_q, 9), max(1, n_q - 3), n_q]      # request 1 has empty rows
    cache, k, v = filled(4, 2, 311, dim, group, lens)
    q = gen((4, n_q, 6, dim), 4, dtype, std=1.5, outliers=False)
    out = torch.full_like(q, 3.0)
    cache.attention(q, i32(*lens), n_tok=i32(*news), causal=causal, window=window, out=out)
    for b, n in enumerate(news):
        assert (out[b, n:] == 3.0).all()
    check(out, q, k, v, lens, news, dtype, causal=causal, window=window)


@pytest.mark.parametrize("vstd", [1e-4, 1e-2, 300.0])
@pytest.mark.parametrize("qstd", [1e-3, 4.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_magnitudes(vstd, qstd, dtype):
    """Small and large values keep their relative accuracy."""
    lens = [700]
    cache, k, v = filled(1, 2, 700, 128, 32, lens, vstd=vstd)
    q = gen((1, 1, 4, 128), 8, dtype, std=qstd)
    check(cache.attention(q, i32(700)), q, k, v, lens, [1], dtype)


def test_growing_values_along_the_cache():
    """Scores and V scales that grow from tile to tile: every rescale runs."""
    n = 900
    k, v = gen((1, n, 1, 64), 21, outliers=False), gen((1, n, 1, 64), 22, outliers=False)
    ramp = torch.linspace(0.01, 8.0, n, device="cuda").view(1, n, 1, 1)
    k, v = (k * ramp).half(), (v * ramp ** 3).half()
    cache = kie.KV4Cache(1, 1, n, 64, 32)
    cache.append(k, v, i32(0))
    q = gen((1, 1, 1, 64), 23, "fp32")
    check(cache.attention(q, i32(n)), q, stored(k, 32), stored(v, 32), [n], [1], "fp32")


def test_strides_scale_and_lengths_past_the_cache():
    lens = [200, 77]
    cache, k, v = filled(2, 2, 200, 128, 128, lens)
    big = gen((2, 3, 11, 131), 9, "bf16", outliers=False)
    q = big[:, :, 2:8, 1:129]
    hold = torch.full((2, 6, 3, 130), 5.0, dtype=torch.bfloat16, device="cuda")
    out = hold.transpose(1, 2)[..., :128]
    cache.attention(q, i32(1 << 30, 77), n_tok=i32(1 << 30, -5), scale=0.3, out=out)     # clamped to 200 keys, 3 and 0 tokens
    assert (out[1] == 5.0).all() and (hold[..., 128:] == 5.0).all()
    check(out, q, k, v, [200, 77], [3, 0], "bf16", scale=0.3)


def test_nan_query_reaches_its_row_only():
    cache, k, v = filled(1, 1, 64, 64, 32, [64])
    q = gen((1, 2, 4, 64), 5, "fp32", outliers=False)
    q[0, 1, 2, 5] = math.nan
    out = cache.attention(q, i32(64))
    assert torch.isnan(out[0, 1, 2]).all()
    ok = torch.ones(1, 2, 4, dtype=torch.bool, device="cuda")
    ok[0, 1, 2] = False
    assert torch.isfinite(out[ok]).all()


def test_repeat_gives_the_same_bits():
    lens = [3000, 1111]
    cache, _, _ = filled(2, 4, 3000, 128, 64, lens)
    q = gen((2, 1, 8, 128), 6, "fp32")
    first = cache.attention(q, i32(*lens))
    for _ in range(3):
        assert torch.equal(first, cache.attention(q, i32(*lens)))


def test_far_positions():
    """Codes and parameters more than 2^31 bytes into the cache."""
    ctx, dim = (1 << 25) + 777, 128
    cache = kie.KV4Cache(1, 2, ctx, dim, 128)
    n = 300
    k, v = gen((1, n, 2, dim), 31), gen((1, n, 2, dim), 32)
    cache.append(k, v, i32(ctx - n))
    kk, vv = cache.read(i32(ctx - n), n, dtype=torch.float32)
    np.testing.assert_array_equal(kk.cpu().numpy(), stored(k, 128).astype(np.float32))
    np.testing.assert_array_equal(vv.cpu().numpy(), stored(v, 128).astype(np.float32))
    q = gen((1, 2, 4, dim), 33, "fp32")
    out = cache.attention(q, i32(ctx), window=n - 1)
    check(out, q, stored(k, 128), stored(v, 128), [n], [2], "fp32", window=n - 1)


def test_decode_in_a_graph():
    """Append and attention captured once and replayed as the lengths move on,
    on a stream of its own, equal to eager calls."""
    b, h, dim, ctx = 2, 2, 64, 128
    caches = [kie.KV4Cache(b, h, ctx, dim, 32) for _ in range(2)]
    ks, vs = gen((b, ctx, h, dim), 41), gen((b, ctx, h, dim), 42)
    qs = gen((b, ctx, 4, dim), 43)
    k, v, q = ks[:, :1].contiguous(), vs[:, :1].contiguous(), qs[:, :1].contiguous()
    start = i32(0, 0)
    out = torch.zeros_like(q)
    lens = start + 1

    def step(c):
        c.append(k, v, start)
        torch.add(start, 1, out=lens)
        c.attention(q, lens, out=out)
        start.copy_(lens)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(caches[0])                                   # loads the kernels
    side.synchronize()
    start.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(caches[0])
    start.zero_()
    got, want = [], []
    for t in range(100):
        k.copy_(ks[:, t:t + 1]); v.copy_(vs[:, t:t + 1]); q.copy_(qs[:, t:t + 1])
        graph.replay()
        got.append(out.clone())
    start.zero_()
    for t in range(100):
        k.copy_(ks[:, t:t + 1]); v.copy_(vs[:, t:t + 1]); q.copy_(qs[:, t:t + 1])
        step(caches[1])
        want.append(out.clone())
    assert torch.equal(torch.cat(got, 1), torch.cat(want, 1))
    check(torch.cat(got[-1:], 1), qs[:, 99:100], stored(ks[:, :100], 32), stored(vs[:, :100], 32), [100] * 2, [1] * 2, "fp16")


def test_calls_on_two_streams():
    lens = [1500]
    cache, k, v = filled(1, 4, 1500, 128, 32, lens)
    qs = [gen((1, 1, 4, 128), 50 + i, "fp32") for i in range(8)]
    want = [cache.attention(q, i32(1500)) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    lengths = i32(1500)
    torch.cuda.synchronize()
    got = []
    for i, q in enumerate(qs):
        got.append(cache.attention(q, lengths, stream=streams[i % 2]))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dim,group,heads,kv_heads,n_q,window", [(128, 64, 4, 4, 300, 0), (64, 32, 8, 2, 129, 0),
                                                                (128, 128, 2, 1, 200, 900), (64, 64, 16, 1, 33, 0),
                                                                (128, 32, 4, 2, 128, 0)])
def test_many_tokens_over_a_long_cache(dim, group, heads, kv_heads, n_q, window):
    """Many key tiles per row tile, one and two row tiles, the keys split over CTAs."""
    lens, news = [5000, 2977], [n_q, n_q - 1]
    cache, k, v = filled(2, kv_heads, 5000, dim, group, lens)
    q = gen((2, n_q, heads, dim), 61, "bf16", std=1.5, outliers=False)
    out = cache.attention(q, i32(*lens), n_tok=i32(*news), window=window)
    rows = [0, 1, n_q // 2, n_q - 2]                      # a few rows of each request against 64 bits
    for b in range(2):
        for t in rows:
            if t >= news[b]:
                continue
            n = lens[b] - news[b] + t + 1
            check(out[b:b + 1, t:t + 1], q[b:b + 1, t:t + 1], k[b:b + 1, :n], v[b:b + 1, :n], [n], [1], "bf16",
                  window=window)
    assert torch.isfinite(out[0]).all()
    again = cache.attention(q, i32(*lens), n_tok=i32(*news), window=window)
    assert torch.equal(out[0], again[0])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [3, 40, 200])
def test_window_of_the_largest_number(dtype, n):
    """A window of 2^31 - 1 is no window, also for queries before the first key."""
    b, hkv, hq, dim, ctx = 2, 2, 16, 128, 150
    c = kie.KV4Cache(b, hkv, ctx, dim)
    k, v, q = gen((b, ctx, hkv, dim), 1, dtype), gen((b, ctx, hkv, dim), 2, dtype), gen((b, n, hq, dim), 3, dtype)
    c.append(k, v, torch.zeros(b, dtype=torch.int32, device="cuda"))
    lens = torch.tensor([2, 130], dtype=torch.int32, device="cuda")
    assert torch.equal(c.attention(q, lens, window=2 ** 31 - 1), c.attention(q, lens))


@pytest.mark.parametrize("dim,n", [(64, 100), (128, 2300), (128, 40000)])
def test_fp32_stays_fp32_over_long_contexts(dim, n):
    """A probability carries a few 2^-22 (scores and their splits, exp, the split of
    p s), a sum of 16 terms 2^-22 of the largest; all independent from key to key, so
    over n keys they add up like the result itself, as the root of n, and stay within
    2^-19 of its norm.  (What is cut to one side would grow with n against it.)"""
    h = 4
    c = kie.KV4Cache(1, h, n, dim)
    q, k, v = gen((1, 1, h, dim), 1, "fp32"), gen((1, n, h, dim), 2, "fp32"), gen((1, n, h, dim), 3, "fp32")
    zero, lens = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((1,), n, dtype=torch.int32, device="cuda")
    c.append(k, v, zero)
    kk, vv = (x[0].double() for x in c.read(zero, n, dtype=torch.float32))
    p = torch.softmax(torch.einsum("hd,nhd->hn", q[0, 0].double(), kk) * dim ** -0.5, -1)
    ref = torch.einsum("hn,nhd->hd", p, vv)
    assert (c.attention(q, lens)[0, 0].double() - ref).norm() <= 2.0 ** -19 * ref.norm()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_16_bit_results_over_long_contexts(dtype):
    """The result's own rounding, at most half a step for each element, and as much
    again for p's and the sums', over so many keys that each warp adds many tiles."""
    h, dim, n = 1, 128, 600000
    c = kie.KV4Cache(1, h, n, dim, 128)
    q, k, v = gen((1, 1, h, dim), 1, dtype), gen((1, n, h, dim), 2, dtype), gen((1, n, h, dim), 3, dtype)
    zero, lens = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((1,), n, dtype=torch.int32, device="cuda")
    c.append(k, v, zero)
    kk, vv = (x[0].double() for x in c.read(zero, n, dtype=torch.float32))
    p = torch.softmax(torch.einsum("hd,nhd->hn", q[0, 0].double(), kk) * dim ** -0.5, -1)
    ref = torch.einsum("hn,nhd->hd", p, vv)
    assert (c.attention(q, lens)[0, 0].double() - ref).norm() <= torch.finfo(TYPES[dtype]).eps * ref.norm()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [1, 100])
def test_values_at_the_end_of_fp16(dtype, n):
    """Values stored at +-65504 (infinities among them) round to 65,536 with their
    scale: finite results for one token and for many."""
    b, hkv, hq, dim, ctx = 1, 2, 8, 128, 200
    c = kie.KV4Cache(b, hkv, ctx, dim, 64)
    k, v, q = gen((b, ctx, hkv, dim), 1, dtype), gen((b, ctx, hkv, dim), 2, dtype), gen((b, n, hq, dim), 3, dtype)
    v[0, ::7, :, 3] = math.inf
    v[0, ::7, :, 5] = -math.inf
    v[0, 3::11, :, 70] = 65504.0
    v[0, 3::11, :, 71] = -65504.0
    lens = torch.full((b,), ctx, dtype=torch.int32, device="cuda")
    c.append(k, v, torch.zeros(b, dtype=torch.int32, device="cuda"))
    check(c.attention(q, lens), q, stored(k, 64), stored(v, 64), [ctx], [n], dtype)
    # the greatest key alone decides
    k[0, 50] = math.inf
    k[0, 50, :, 1] = -math.inf
    q[..., :] = 1.0
    c.append(k, v, torch.zeros(b, dtype=torch.int32, device="cuda"))
    out = c.attention(q, lens, causal=False)
    want = stored(v, 64)[0, 50].repeat(hq // hkv, 0)
    # p s code and p z, each at most 3 of the largest |v| together, with p s rounded by 2^-11 twice
    assert np.allclose(out[0, -1].double().cpu().numpy(), want, rtol=2.0 ** -8, atol=6 * 2.0 ** -11 * np.abs(want).max())
