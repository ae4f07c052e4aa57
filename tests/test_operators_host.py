"""Refusals of the operators on device tensors, before anything reaches a GPU."""
import ctypes as C

import pytest

from autoregressive_decode_gb300 import kie

BAD, UNSUPPORTED, OOM = kie.KIE_ERR_INVALID_ARG, kie.KIE_ERR_UNSUPPORTED, kie.KIE_ERR_OOM
P = 1 << 20      # stands for a device address; nothing here reads it


def cache(**kw):
    a = dict(data=P, batch=2, n_kv_heads=4, max_ctx=100, head_dim=128, group=32, device=0)
    a.update(kw)
    return kie.kie_kv4_cache(*(a[n] for n, _ in kie.kie_kv4_cache._fields_))


def query(**kw):
    a = dict(q=P, out=P, q_strides=None, out_strides=None, kv_len=P, n_tok=None, dtype=0, n_tokens=1, n_heads=8,
             causal=1, window=0, scale=0.1)
    a.update(kw)
    return kie.kie_kv4_query(*(a[n] for n, _ in kie.kie_kv4_query._fields_))


def test_cache_bytes():
    lib = kie.load()
    # 128 positions (100 padded to 64s), 2 x 4 heads, K and V: 64 bytes of codes and 4 (scale, zero) pairs
    assert lib.kie_kv4_bytes(C.byref(cache())) == 2 * 8 * 128 * (64 + 16)
    assert lib.kie_kv4_bytes(C.byref(cache(max_ctx=64, head_dim=64, group=64))) == 2 * 8 * 64 * (32 + 4)
    assert lib.kie_kv4_bytes(C.byref(cache(batch=8, n_kv_heads=16, max_ctx=1 << 24))) == 2 * 128 * (1 << 24) * 80


@pytest.mark.parametrize("kw", [dict(batch=0), dict(n_kv_heads=0), dict(max_ctx=0), dict(head_dim=96),
                                dict(group=16), dict(group=128, head_dim=64), dict(max_ctx=(1 << 30) + 1),
                                dict(batch=1 << 20, n_kv_heads=32)])
def test_bad_caches(kw):
    lib = kie.load()
    c = cache(**kw)
    assert lib.kie_kv4_bytes(C.byref(c)) == 0
    assert lib.kie_kv4_append(C.byref(c), P, P, 0, None, None, 1, P, None, None) == BAD
    assert lib.kie_kv4_read(C.byref(c), P, P, 0, None, None, 1, P, None, None) == BAD
    assert lib.kie_kv4_attention(C.byref(c), C.byref(query()), P, 1 << 40, None) == BAD
    assert lib.kie_kv4_attention_workspace(C.byref(c), C.byref(query())) == 0
    assert lib.kie_last_error(None)


def test_bad_rows():
    lib = kie.load()
    for f in (lib.kie_kv4_append, lib.kie_kv4_read):
        ok = C.byref(cache())
        assert f(None, P, P, 0, None, None, 1, P, None, None) == BAD
        assert f(C.byref(cache(data=None)), P, P, 0, None, None, 1, P, None, None) == BAD
        assert f(C.byref(cache(data=P + 16)), P, P, 0, None, None, 1, P, None, None) == BAD
        assert f(ok, None, P, 0, None, None, 1, P, None, None) == BAD
        assert f(ok, P, None, 0, None, None, 1, P, None, None) == BAD
        assert f(ok, P, P, 0, None, None, 1, None, None, None) == BAD
        assert f(ok, P, P, 3, None, None, 1, P, None, None) == BAD
        assert f(ok, P, P, -1, None, None, 1, P, None, None) == BAD
        assert f(ok, P + 1, P, 0, None, None, 1, P, None, None) == BAD
        assert f(ok, P, P + 2, 2, None, None, 1, P, None, None) == BAD
        assert f(ok, P, P, 0, None, None, -1, P, None, None) == BAD
        assert f(ok, P, P, 0, None, None, 0, None, None, None) == kie.KIE_OK      # nothing to do
        assert f(C.byref(cache(batch=1 << 10, n_kv_heads=1 << 10)), P, P, 0, None, None, 1 << 15, P, None,
                 None) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(q=None), dict(out=None), dict(kv_len=None), dict(dtype=7), dict(n_tokens=-1),
                                dict(n_heads=6), dict(n_heads=0), dict(causal=2), dict(window=-1),
                                dict(causal=0, window=4), dict(scale=float("inf")), dict(scale=float("nan")),
                                dict(q=P + 1), dict(dtype=2, out=P + 2), dict(n_tokens=1 << 30)])
def test_bad_queries(kw):
    lib = kie.load()
    assert lib.kie_kv4_attention(C.byref(cache()), C.byref(query(**kw)), P, 1 << 40, None) == BAD


def test_empty_query_and_nulls():
    lib = kie.load()
    assert lib.kie_kv4_attention(C.byref(cache()), C.byref(query(n_tokens=0)), None, 0, None) == kie.KIE_OK
    assert lib.kie_kv4_attention(C.byref(cache()), None, P, 1 << 40, None) == BAD
    assert lib.kie_kv4_attention(None, C.byref(query()), P, 1 << 40, None) == BAD
    assert lib.kie_kv4_bytes(None) == 0
    assert lib.kie_sample(None, None) == BAD


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), BAD), (dict(u=None), BAD), (dict(tokens=None), BAD), (dict(dtype=3), BAD), (dict(rows=-1), BAD),
    (dict(vocab=0), BAD), (dict(vocab=(1 << 18) + 1), UNSUPPORTED), (dict(rows=(1 << 24) + 1), UNSUPPORTED),
    (dict(logits=P + 2), BAD), (dict(u=P + 1), BAD), (dict(top_k=P + 2), BAD), (dict(rows=0), kie.KIE_OK)])
def test_bad_samples(kw, status):
    a = dict(logits=P, dtype=2, rows=3, vocab=100, row_stride=100, temperature=None, top_k=None, top_p=None,
             min_p=None, u=P, tokens=P, probs=None, device=0)
    a.update(kw)
    s = kie.kie_sample_args(*(a[n] for n, _ in kie.kie_sample_args._fields_))
    assert kie.load().kie_sample(C.byref(s), None) == status


def test_python_checks():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        kie.sample(x, torch.zeros(2))                     # host tensors
    with pytest.raises(ValueError):
        kie._dtype(torch.zeros(1, dtype=torch.float64))
    with pytest.raises(ValueError):
        kie._written(x[:1].expand(2, 8), "out")
    with pytest.raises(ValueError):
        kie._vector(x, 2, torch.int32, 0, "start")


def test_sampled_generation_refuses_on_the_host():
    lib = kie.load()
    s = kie.kie_sampling(None, None, None, None, P)
    assert lib.kie_generate_sampled_device(None, P, 1, C.byref(s), P, None) == BAD
    assert lib.kie_last_error(None)
