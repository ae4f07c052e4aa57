"""Thin ctypes binding of libkie.so (argument marshalling only).

Every entry point of include/kie.h is exposed under the same name on ``lib``;
``Engine`` wraps one engine handle.  All computation happens in the CUDA
library: if the library cannot be loaded this module raises instead of falling
back to anything else.

Arrays may be numpy arrays (host memory) or torch tensors; torch CUDA tensors
are passed as device pointers where the C entry point takes device pointers
(kie_generate_greedy_device, kie_load_weights with on_device = 1, the
workspace of kie_create).
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np

from . import _build

KIE_OK, KIE_ERR_INVALID_ARG, KIE_ERR_OOM, KIE_ERR_CUDA = 0, -1, -2, -3
KIE_ERR_NOT_LOADED, KIE_ERR_CTX_OVERFLOW, KIE_ERR_DEVICE_TIMEOUT = -4, -5, -6
KIE_ERR_LAUNCH, KIE_ERR_UNSUPPORTED = -7, -8
KV_DTYPES = {"fp16": 0, "fp8_e5m2": 1, "u8": 2, "fp8_e5m2_scaled": 3}
W_DTYPES = {"fp16": 0, "int4_g128": 1, "fp8_e4m3": 2, "nvfp4": 3}
MODES = {"persistent": 0, "graph": 1}

STATUS_NAMES = {0: "KIE_OK", -1: "KIE_ERR_INVALID_ARG", -2: "KIE_ERR_OOM", -3: "KIE_ERR_CUDA",
                -4: "KIE_ERR_NOT_LOADED", -5: "KIE_ERR_CTX_OVERFLOW", -6: "KIE_ERR_DEVICE_TIMEOUT",
                -7: "KIE_ERR_LAUNCH", -8: "KIE_ERR_UNSUPPORTED"}


class KieError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class kie_config(C.Structure):
    _fields_ = [("n_layers", C.c_int32), ("d_model", C.c_int32), ("n_heads", C.c_int32),
                ("head_dim", C.c_int32), ("ffn_dim", C.c_int32), ("vocab", C.c_int32),
                ("max_ctx", C.c_int32), ("rms_eps", C.c_float), ("rope_theta", C.c_float),
                ("kv_dtype", C.c_int32), ("ffn_wdtype", C.c_int32), ("mode", C.c_int32),
                ("device", C.c_int32), ("attn_wdtype", C.c_int32), ("batch", C.c_int32),
                ("kv_scale_k", C.c_float), ("kv_scale_v", C.c_float)]


class kie_layer_weights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("attn_norm", "wq", "wk", "wv", "wo", "ffn_norm",
                                         "w_gate", "w_up", "w_down")]


class kie_weights(C.Structure):
    _fields_ = [("tok_emb", C.c_void_p), ("final_norm", C.c_void_p), ("lm_head", C.c_void_p),
                ("layers", C.POINTER(kie_layer_weights)), ("on_device", C.c_int32)]


class kie_kv4_cache(C.Structure):
    _fields_ = [("data", C.c_void_p), ("batch", C.c_int32), ("n_kv_heads", C.c_int32), ("max_ctx", C.c_int32),
                ("head_dim", C.c_int32), ("group", C.c_int32), ("device", C.c_int32)]


class kie_kv4_query(C.Structure):
    _fields_ = [("q", C.c_void_p), ("out", C.c_void_p), ("q_strides", C.c_void_p), ("out_strides", C.c_void_p),
                ("kv_len", C.c_void_p), ("n_tok", C.c_void_p), ("dtype", C.c_int32), ("n_tokens", C.c_int32),
                ("n_heads", C.c_int32), ("causal", C.c_int32), ("window", C.c_int32), ("scale", C.c_float)]


class kie_sample_args(C.Structure):
    _fields_ = [("logits", C.c_void_p), ("dtype", C.c_int32), ("rows", C.c_int32), ("vocab", C.c_int32),
                ("row_stride", C.c_int64), ("temperature", C.c_void_p), ("top_k", C.c_void_p), ("top_p", C.c_void_p),
                ("min_p", C.c_void_p), ("u", C.c_void_p), ("tokens", C.c_void_p), ("probs", C.c_void_p),
                ("device", C.c_int32)]


class kie_sampling(C.Structure):
    _fields_ = [("temperature", C.c_void_p), ("top_k", C.c_void_p), ("top_p", C.c_void_p), ("min_p", C.c_void_p),
                ("u", C.c_void_p)]


EXPORTS = {
    # name: (restype, argtypes)
    "kie_workspace_bytes": (C.c_size_t, [C.POINTER(kie_config)]),
    "kie_create": (C.c_int, [C.POINTER(kie_config), C.c_void_p, C.c_size_t, C.c_void_p, C.POINTER(C.c_void_p)]),
    "kie_load_weights": (C.c_int, [C.c_void_p, C.POINTER(kie_weights)]),
    "kie_prefill": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.c_void_p]),
    "kie_decode_step": (C.c_int, [C.c_void_p, C.c_int32, C.POINTER(C.c_int32), C.c_void_p]),
    "kie_generate_greedy": (C.c_int, [C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p]),
    "kie_generate_greedy_device": (C.c_int, [C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p]),
    "kie_sync": (C.c_int, [C.c_void_p]),
    "kie_decode_step_static_scratch": (C.c_int, [C.c_void_p, C.c_int32, C.c_void_p, C.c_void_p]),
    "kie_trace_decode": (C.c_int, [C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_size_t]),
    "kie_select_request": (C.c_int, [C.c_void_p, C.c_int32]),
    "kie_decode_batch": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]),
    "kie_generate_greedy_batch": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.c_void_p, C.c_void_p]),
    "kie_generate_greedy_batch_device": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.c_void_p, C.c_void_p]),
    "kie_generate_sampled_device": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.POINTER(kie_sampling), C.c_void_p,
                                              C.c_void_p]),
    "kie_reset": (C.c_int, [C.c_void_p]),
    "kie_get_pos": (C.c_int32, [C.c_void_p]),
    "kie_set_pos": (C.c_int, [C.c_void_p, C.c_int32]),
    "kie_set_timeout_ms": (C.c_int, [C.c_void_p, C.c_int32]),
    "kie_debug_skip_grid_arrival": (C.c_int, [C.c_void_p, C.c_int32]),
    "kie_get_stream": (C.c_void_p, [C.c_void_p]),
    "kie_grid_size": (C.c_int32, [C.c_void_p]),
    "kie_last_error": (C.c_char_p, [C.c_void_p]),
    "kie_destroy": (None, [C.c_void_p]),
    "kie_set_kv": (C.c_int, [C.c_void_p, C.c_int32, C.c_void_p, C.c_void_p, C.c_int32]),
    "kie_read_kv": (C.c_int, [C.c_void_p, C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_void_p,
                              C.c_void_p, C.c_void_p, C.c_void_p]),
    "kie_quantize_kv_u8": (C.c_int, [C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p, C.c_void_p]),
    "kie_quantize_int4_g128": (C.c_int, [C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p]),
    "kie_quantize_fp8_rows": (C.c_int, [C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p]),
    "kie_quantize_nvfp4_rows": (C.c_int, [C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p, C.c_void_p]),
    "kie_convert_fp8_e5m2": (C.c_int, [C.c_void_p, C.c_size_t, C.c_void_p]),
    "kie_kv4_bytes": (C.c_size_t, [C.POINTER(kie_kv4_cache)]),
    "kie_kv4_append": (C.c_int, [C.POINTER(kie_kv4_cache), C.c_void_p, C.c_void_p, C.c_int32, C.c_void_p, C.c_void_p,
                                 C.c_int32, C.c_void_p, C.c_void_p, C.c_void_p]),
    "kie_kv4_read": (C.c_int, [C.POINTER(kie_kv4_cache), C.c_void_p, C.c_void_p, C.c_int32, C.c_void_p, C.c_void_p,
                               C.c_int32, C.c_void_p, C.c_void_p, C.c_void_p]),
    "kie_kv4_attention_workspace": (C.c_size_t, [C.POINTER(kie_kv4_cache), C.POINTER(kie_kv4_query)]),
    "kie_kv4_attention": (C.c_int, [C.POINTER(kie_kv4_cache), C.POINTER(kie_kv4_query), C.c_void_p, C.c_size_t,
                                    C.c_void_p]),
    "kie_sample": (C.c_int, [C.POINTER(kie_sample_args), C.c_void_p]),
}

_lib = None


def load(build: bool = True):
    """Load libkie.so (building it first if missing or stale)."""
    global _lib
    if _lib is None:
        path = _build.build() if build else _build.LIB
        if not os.path.exists(path):
            raise OSError(f"libkie.so not found at {path}")
        lib = C.CDLL(path)
        for name, (res, args) in EXPORTS.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _lib = lib
    return _lib


def _ptr(a):
    """Address of a numpy array or torch tensor (None -> NULL)."""
    if a is None:
        return None
    if isinstance(a, np.ndarray):
        if not a.flags["C_CONTIGUOUS"]:
            raise ValueError("array must be C-contiguous")
        return a.ctypes.data
    if hasattr(a, "data_ptr"):
        if not a.is_contiguous():
            raise ValueError("tensor must be contiguous")
        return a.data_ptr()
    raise TypeError(f"unsupported buffer type {type(a)}")


def _check(st, eng=None):
    if st != KIE_OK:
        msg = load().kie_last_error(eng)
        raise KieError(st, msg.decode() if msg else "")


def make_config(n_layers, d_model, n_heads, head_dim, ffn_dim, vocab, max_ctx, rms_eps=1e-5, rope_theta=10000.0,
                kv_dtype="fp16", ffn_wdtype="fp16", mode="persistent", device=0, attn_wdtype="fp16",
                batch=1, kv_scale=(0.0, 0.0)) -> kie_config:
    return kie_config(n_layers, d_model, n_heads, head_dim, ffn_dim, vocab, max_ctx, rms_eps, rope_theta,
                      KV_DTYPES[kv_dtype], W_DTYPES[ffn_wdtype], MODES[mode], device, W_DTYPES[attn_wdtype],
                      int(batch), float(kv_scale[0]), float(kv_scale[1]))


class Engine:
    """One engine handle (kie_create .. kie_destroy)."""

    def __init__(self, cfg: kie_config, stream=None, workspace=None):
        lib = load()
        self.cfg = cfg
        self._ws = workspace                 # kept alive for the engine's lifetime
        h = C.c_void_p()
        ws_ptr = _ptr(workspace)
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        st_ptr = None if stream is None else (stream if isinstance(stream, int) else stream.cuda_stream)
        _check(lib.kie_create(C.byref(cfg), ws_ptr, ws_bytes, st_ptr, C.byref(h)))
        self.h = h
        self.vocab = cfg.vocab
        self.batch = max(1, cfg.batch)

    # -- lifetime -------------------------------------------------------------------------
    def close(self):
        if getattr(self, "h", None):
            load().kie_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    # -- API --------------------------------------------------------------------------------
    def load_weights(self, w: dict):
        """w: dict as from synthetic.gen_weights (numpy fp16 arrays, or torch CUDA fp16 tensors)."""
        layers = w["layers"]
        on_dev = int(not isinstance(w["tok_emb"], np.ndarray) and getattr(w["tok_emb"], "is_cuda", False))
        arr = (kie_layer_weights * len(layers))()
        keep = []
        for i, lw in enumerate(layers):
            for n in ("attn_norm", "wq", "wk", "wv", "wo", "ffn_norm", "w_gate", "w_up", "w_down"):
                setattr(arr[i], n, _ptr(lw[n]))
                keep.append(lw[n])
        kw = kie_weights(_ptr(w["tok_emb"]), _ptr(w["final_norm"]), _ptr(w["lm_head"]),
                         C.cast(arr, C.POINTER(kie_layer_weights)), on_dev)
        _check(load().kie_load_weights(self.h, C.byref(kw)), self.h)

    def prefill(self, tokens, want_logits: bool = True):
        toks = np.ascontiguousarray(tokens, dtype=np.int32)
        out = np.empty(self.vocab, np.float32) if want_logits else None
        _check(load().kie_prefill(self.h, _ptr(toks), len(toks), _ptr(out)), self.h)
        return out

    def decode_step(self, token: int, want_logits: bool = True):
        nxt = C.c_int32()
        out = np.empty(self.vocab, np.float32) if want_logits else None
        _check(load().kie_decode_step(self.h, int(token), C.byref(nxt), _ptr(out)), self.h)
        return nxt.value, out

    def generate_greedy(self, first_token: int, n: int, want_logits: bool = False):
        toks = np.empty(n, np.int32)
        logs = np.empty((n, self.vocab), np.float32) if want_logits else None
        _check(load().kie_generate_greedy(self.h, int(first_token), int(n), _ptr(toks), _ptr(logs)), self.h)
        return toks, logs

    def generate_greedy_device(self, first_token: int, n: int, d_tokens, d_logits=None):
        _check(load().kie_generate_greedy_device(self.h, int(first_token), int(n), _ptr(d_tokens), _ptr(d_logits)),
               self.h)

    def trace_decode(self, first_token: int, n: int):
        """n greedy steps with per-phase stamps: (uint64 [n, 5L+1, 6, grid],
        ring trace of CTA 0 [32768, 4]) in ns."""
        shape = (n, 5 * self.cfg.n_layers + 1, 6, self.grid)
        nph = int(np.prod(shape))
        buf = np.zeros(nph + 32768 * 4, np.uint64)
        _check(load().kie_trace_decode(self.h, int(first_token), int(n), _ptr(buf), buf.size), self.h)
        return buf[:nph].reshape(shape), buf[nph:].reshape(32768, 4)

    def decode_step_static_scratch(self, token: int, d_next_token, d_logits=None):
        """kie_decode_step_static_scratch: device outputs, no allocation, no sync."""
        _check(load().kie_decode_step_static_scratch(self.h, int(token), _ptr(d_next_token), _ptr(d_logits)), self.h)

    # -- batched engines --------------------------------------------------------------------
    def select_request(self, b: int):
        """Address request b with prefill / set_kv / read_kv / set_pos / pos."""
        _check(load().kie_select_request(self.h, int(b)), self.h)

    def decode_batch(self, tokens, want_logits: bool = True):
        """One step of every request: (next tokens [batch], logits [batch, vocab] or None)."""
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        nxt = np.empty(self.batch, np.int32)
        out = np.empty((self.batch, self.vocab), np.float32) if want_logits else None
        _check(load().kie_decode_batch(self.h, _ptr(t), _ptr(nxt), _ptr(out)), self.h)
        return nxt, out

    def generate_greedy_batch(self, first_tokens, n: int, want_logits: bool = False):
        """n greedy steps of every request: (tokens [n, batch], logits [n, batch, vocab] or None)."""
        f = np.ascontiguousarray(first_tokens, dtype=np.int32)
        toks = np.empty((n, self.batch), np.int32)
        logs = np.empty((n, self.batch, self.vocab), np.float32) if want_logits else None
        _check(load().kie_generate_greedy_batch(self.h, _ptr(f), int(n), _ptr(toks), _ptr(logs)), self.h)
        return toks, logs

    def generate_greedy_batch_device(self, first_tokens, n: int, d_tokens, d_logits=None):
        f = np.ascontiguousarray(first_tokens, dtype=np.int32)
        _check(load().kie_generate_greedy_batch_device(self.h, _ptr(f), int(n), _ptr(d_tokens), _ptr(d_logits)),
               self.h)

    # -- sampling ---------------------------------------------------------------------------
    def generate_sampled_device(self, first_tokens, u, d_tokens, d_probs=None, temperature=None, top_k=None,
                                top_p=None, min_p=None):
        """kie_generate_sampled_device: len(u) steps of every request, tokens drawn
        with the random numbers u (CUDA fp32 [n, batch]) into d_tokens (CUDA int32
        [n, batch]) and their probabilities into d_probs (fp32); the parameters are
        CUDA tensors [batch].  Enqueued on the engine's stream without
        synchronising: that stream must see the tensors written, and they must
        live until it is done."""
        torch = _need_torch()
        f = np.ascontiguousarray(first_tokens, dtype=np.int32).reshape(-1)
        if f.size != self.batch:
            raise ValueError(f"first_tokens must hold {self.batch} tokens")
        n, b, dev, i32, f32 = len(u), self.batch, self.cfg.device, torch.int32, torch.float32
        for t, dtype, what in ((u, f32, "u"), (d_tokens, i32, "d_tokens"), (d_probs, f32, "d_probs")):
            if t is None and what == "d_probs":
                continue
            _on(t, dev, what)
            if t.dtype is not dtype or t.shape != (n, b) or not t.is_contiguous():
                raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape ({n}, {b})")
        s = kie_sampling(_vector(temperature, b, f32, dev, "temperature"), _vector(top_k, b, i32, dev, "top_k"),
                         _vector(top_p, b, f32, dev, "top_p"), _vector(min_p, b, f32, dev, "min_p"), u.data_ptr())
        _check(load().kie_generate_sampled_device(self.h, _ptr(f), n, C.byref(s), d_tokens.data_ptr(),
                                                  _ptr(d_probs)), self.h)

    def sync(self):
        _check(load().kie_sync(self.h), self.h)

    def reset(self):
        _check(load().kie_reset(self.h), self.h)

    @property
    def pos(self) -> int:
        return load().kie_get_pos(self.h)

    def set_pos(self, pos: int):
        _check(load().kie_set_pos(self.h, int(pos)), self.h)

    def set_timeout_ms(self, ms: int):
        _check(load().kie_set_timeout_ms(self.h, int(ms)), self.h)

    def debug_skip_grid_arrival(self, cta: int):
        """Failure injection (tests): CTA `cta` skips its first grid-barrier
        arrival in the next persistent launch of several steps."""
        _check(load().kie_debug_skip_grid_arrival(self.h, int(cta)), self.h)

    @property
    def stream(self) -> int:
        return load().kie_get_stream(self.h) or 0

    @property
    def grid(self) -> int:
        return load().kie_grid_size(self.h)

    def set_kv(self, layer: int, k16: np.ndarray, v16: np.ndarray):
        k = np.ascontiguousarray(k16, dtype=np.float16)
        v = np.ascontiguousarray(v16, dtype=np.float16)
        _check(load().kie_set_kv(self.h, int(layer), _ptr(k), _ptr(v), k.shape[0]), self.h)

    def read_kv(self, layer: int, which: int, p0: int, n: int):
        """Raw storage of K (which=0) or V (1): (data [H, n, h], tail fp16 or None,
        scale [H, nseg] (uint8) / [nslices] (scaled E5M2) or None, zp [H, nseg] or None)."""
        H, h = self.cfg.n_heads, self.cfg.head_dim
        kv = self.cfg.kv_dtype
        data = np.empty((H, n, h), np.uint16 if kv == 0 else np.uint8)
        tail = sc = zp = None
        if kv == 3:   # scaled E5M2: the scales of the slices the range meets
            sc = np.zeros((p0 + n + 255) // 256 - p0 // 256, np.float32)
        if kv == 2:
            tail = np.zeros((H, n, h), np.uint16)
            nseg = (p0 + n + 127) // 128 - p0 // 128
            sc = np.zeros((H, nseg), np.float32)
            zp = np.zeros((H, nseg), np.int32)
        _check(load().kie_read_kv(self.h, int(layer), int(which), int(p0), int(n), _ptr(data), _ptr(tail), _ptr(sc),
                                  _ptr(zp)), self.h)
        return data, tail, sc, zp


# ---- stateless routines ----------------------------------------------------------------------
def quantize_kv_u8(x16: np.ndarray, n_seg: int):
    x = np.ascontiguousarray(x16, dtype=np.float16).reshape(-1)
    seg = x.size // n_seg
    codes = np.empty(x.size, np.uint8)
    scale = np.empty(n_seg, np.float32)
    zp = np.empty(n_seg, np.int32)
    _check(load().kie_quantize_kv_u8(_ptr(x), n_seg, seg, _ptr(codes), _ptr(scale), _ptr(zp)))
    return codes.reshape(n_seg, seg), scale, zp


def quantize_int4_g128(w16: np.ndarray):
    w = np.ascontiguousarray(w16, dtype=np.float16)
    rows, cols = w.shape
    codes = np.empty((rows, cols), np.int8)
    sc = np.empty((rows, cols // 128), np.uint16)
    _check(load().kie_quantize_int4_g128(_ptr(w), rows, cols, _ptr(codes), _ptr(sc)))
    return codes, sc.view(np.float16)


def quantize_fp8_rows(w16: np.ndarray):
    """kie_quantize_fp8_rows: (codes uint8 [rows, cols], scales fp32 [rows])."""
    w = np.ascontiguousarray(w16, dtype=np.float16)
    rows, cols = w.shape
    codes = np.empty((rows, cols), np.uint8)
    sc = np.empty(rows, np.float32)
    _check(load().kie_quantize_fp8_rows(_ptr(w), rows, cols, _ptr(codes), _ptr(sc)))
    return codes, sc


def quantize_nvfp4_rows(w16: np.ndarray):
    """kie_quantize_nvfp4_rows: (E2M1 codes uint8 [rows, cols] in 0..15,
    E4M3 block-scale bytes uint8 [rows, cols/16], row scales fp32 [rows])."""
    w = np.ascontiguousarray(w16, dtype=np.float16)
    rows, cols = w.shape
    codes = np.empty((rows, cols), np.uint8)
    bs = np.empty((rows, cols // 16), np.uint8)
    rs = np.empty(rows, np.float32)
    _check(load().kie_quantize_nvfp4_rows(_ptr(w), rows, cols, _ptr(codes), _ptr(bs), _ptr(rs)))
    return codes, bs, rs


def convert_fp8_e5m2(x16: np.ndarray) -> np.ndarray:
    x = np.ascontiguousarray(x16, dtype=np.float16).reshape(-1)
    out = np.empty(x.size, np.uint8)
    _check(load().kie_convert_fp8_e5m2(_ptr(x), x.size, _ptr(out)))
    return out


# ---- operators on device tensors ---------------------------------------------------------------
# torch CUDA tensors in and out, enqueued on torch's current stream of their
# device (or on `stream`, a torch.cuda.Stream).  Results are allocated by torch
# where `out` is not given.
_torch = None
_raw_stream = None
DTYPES = {}      # torch dtype -> kie_dtype


def _need_torch():
    global _torch, _raw_stream
    if _torch is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # what current_stream() wraps
        DTYPES.update({torch.float16: 0, torch.bfloat16: 1, torch.float32: 2})
        _torch = torch
    return _torch


def _dtype(t):
    _need_torch()
    d = DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"tensors must be float16, bfloat16 or float32, not {t.dtype}")
    return d


def _on(t, device, what):
    if not t.is_cuda or t.get_device() != device:
        raise ValueError(f"{what} must be a CUDA tensor on device {device}")


def _vector(t, n, dtype, device, what):
    """Address of a contiguous [n] tensor of `dtype`; None stays None."""
    if t is None:
        return None
    _on(t, device, what)
    if t.dtype is not dtype or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape ({n},)")
    return t.data_ptr()


def _rows(t, shape, device, what):
    """(address, strides or None) of a 4-D tensor whose channels are contiguous."""
    _on(t, device, what)
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.is_contiguous():
        return t.data_ptr(), None
    s = t.stride()
    if s[3] != 1:
        raise ValueError(f"{what} must have contiguous channels")
    return t.data_ptr(), (C.c_int64 * 3)(*s[:3])


def _written(t, what):
    """A tensor that a kernel writes must not hold one element twice."""
    if any(n > 1 and s == 0 for n, s in zip(t.shape, t.stride())):
        raise ValueError(f"{what} must not be broadcast")


def _stream(stream, device):
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(device) if _raw_stream is not None else _torch.cuda.current_stream(device).cuda_stream


class KV4Cache:
    """A 4-bit K/V cache of one layer (kie_kv4_cache): `batch` requests of up to
    max_ctx positions, n_kv_heads heads of head_dim 64 or 128, a scale and a zero
    per `group` channels.  Its memory is a torch tensor (`data`)."""

    def __init__(self, batch: int, n_kv_heads: int, max_ctx: int, head_dim: int, group: int = 32, device=None):
        torch = _need_torch()
        device = torch.device("cuda" if device is None else device)
        index = torch.cuda.current_device() if device.index is None else device.index
        self.desc = kie_kv4_cache(None, batch, n_kv_heads, max_ctx, head_dim, group, index)
        n = load().kie_kv4_bytes(C.byref(self.desc))
        if n == 0:
            raise ValueError(f"no 4-bit cache of shape batch {batch}, heads {n_kv_heads}, max_ctx {max_ctx}, "
                             f"head_dim {head_dim}, group {group}")
        self.data = torch.empty(n, dtype=torch.uint8, device=f"cuda:{index}")
        self.desc.data = self.data.data_ptr()
        self.batch, self.n_kv_heads, self.max_ctx, self.head_dim = batch, n_kv_heads, max_ctx, head_dim
        self.group, self.device = group, index
        self._ws_bytes = {}      # (tokens, heads, dtype, window) -> kie_kv4_attention_workspace

    def append(self, k, v, start, n_tok=None, stream=None):
        """kie_kv4_append: store k, v [batch, tokens, n_kv_heads, head_dim] (any
        strides with contiguous channels) at positions start[b] + t, t < n_tok[b]."""
        if k.dim() != 4 or k.dtype is not v.dtype:
            raise ValueError("k and v must be 4-D tensors of one type")
        b, n, dev = self.batch, k.shape[1], self.device
        shape = (b, n, self.n_kv_heads, self.head_dim)
        kp, ks = _rows(k, shape, dev, "k")
        vp, vs = _rows(v, shape, dev, "v")
        i32 = _torch.int32
        _check(_lib.kie_kv4_append(self.desc, kp, vp, _dtype(k), ks, vs, n, _vector(start, b, i32, dev, "start"),
                                   _vector(n_tok, b, i32, dev, "n_tok"), _stream(stream, dev)))

    def read(self, start, tokens: int, n_tok=None, out=None, dtype=None, stream=None):
        """kie_kv4_read: the values at positions start[b] + t, t < n_tok[b], as
        (k, v) [batch, tokens, n_kv_heads, head_dim]: `out`, or new tensors of
        `dtype` (float16) with zeros in the rows that are not read."""
        b, dev = self.batch, self.device
        shape = (b, tokens, self.n_kv_heads, self.head_dim)
        if out is None:
            with _torch.cuda.stream(stream):
                out = [_torch.zeros(shape, dtype=dtype or _torch.float16, device=self.data.device) for _ in range(2)]
        k, v = out
        if k.dtype is not v.dtype:
            raise ValueError("the two outputs must be of one type")
        kp, ks = _rows(k, shape, dev, "out[0]")
        vp, vs = _rows(v, shape, dev, "out[1]")
        if ks is not None:
            _written(k, "out[0]")
        if vs is not None:
            _written(v, "out[1]")
        i32 = _torch.int32
        _check(_lib.kie_kv4_read(self.desc, kp, vp, _dtype(k), ks, vs, tokens, _vector(start, b, i32, dev, "start"),
                                 _vector(n_tok, b, i32, dev, "n_tok"), _stream(stream, dev)))
        return k, v

    def attention(self, q, kv_len, n_tok=None, causal=True, window: int = 0, scale=None, out=None, stream=None):
        """kie_kv4_attention of q [batch, tokens, n_heads, head_dim] over the
        stored positions: `out`, or a new tensor like q with zeros in the rows
        from n_tok[b] on.  scale: 1/sqrt(head_dim) unless given."""
        if stream is not None:
            # what is allocated here belongs to the stream that the kernels run on
            with _torch.cuda.stream(stream):
                return self.attention(q, kv_len, n_tok, causal, window, scale, out)
        if q.dim() != 4:
            raise ValueError("q must be a 4-D tensor")
        b, dev = self.batch, self.device
        n, heads = q.shape[1], q.shape[2]
        shape = (b, n, heads, self.head_dim)
        qp, qs = _rows(q, shape, dev, "q")
        if out is None:
            out = (_torch.empty if n_tok is None else _torch.zeros)(shape, dtype=q.dtype, device=q.device)
        elif out.dtype is not q.dtype:
            raise ValueError("out must have q's type")
        op, os_ = _rows(out, shape, dev, "out")
        if os_ is not None:
            _written(out, "out")
        dt, i32 = _dtype(q), _torch.int32
        a = kie_kv4_query(qp, op, None if qs is None else C.addressof(qs), None if os_ is None else C.addressof(os_),
                          _vector(kv_len, b, i32, dev, "kv_len"), _vector(n_tok, b, i32, dev, "n_tok"), dt, n, heads,
                          bool(causal), window, self.head_dim ** -0.5 if scale is None else scale)
        key = (n, heads, dt, window)
        need = self._ws_bytes.get(key)
        if need is None:
            if len(self._ws_bytes) > 1000:
                self._ws_bytes.clear()
            need = self._ws_bytes[key] = _lib.kie_kv4_attention_workspace(self.desc, a)
        if need > 16:
            # of this call: the allocator gives it to no one else before the stream
            # is done with it, and a captured graph keeps its own
            ws = _torch.empty(need, dtype=_torch.uint8, device=q.device)
            _check(_lib.kie_kv4_attention(self.desc, a, ws.data_ptr(), need, _stream(None, dev)))
        else:
            _check(_lib.kie_kv4_attention(self.desc, a, None, 0, _stream(None, dev)))
        return out


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, probs=None, stream=None):
    """kie_sample: a token per row of logits [rows, vocab] (contiguous within a
    row) from the random numbers u [rows], and its probability: (int32 [rows],
    fp32 [rows]), written to `tokens` and `probs` where given."""
    torch = _need_torch()
    load()
    if stream is not None:
        with torch.cuda.stream(stream):
            return sample(logits, u, temperature, top_k, top_p, min_p, tokens, probs)
    if logits.dim() != 2 or not logits.is_cuda:
        raise ValueError("logits must be a 2-D CUDA tensor")
    rows, vocab = logits.shape
    stride, last = logits.stride()
    if vocab > 1 and last != 1:
        raise ValueError("logits must be contiguous within a row")
    dev, i32, f32 = logits.get_device(), torch.int32, torch.float32
    if tokens is None:
        tokens = torch.empty(rows, dtype=i32, device=logits.device)
    if probs is None:
        probs = torch.empty(rows, dtype=f32, device=logits.device)
    a = kie_sample_args(logits.data_ptr(), _dtype(logits), rows, vocab, stride,
                        _vector(temperature, rows, f32, dev, "temperature"), _vector(top_k, rows, i32, dev, "top_k"),
                        _vector(top_p, rows, f32, dev, "top_p"), _vector(min_p, rows, f32, dev, "min_p"),
                        _vector(u, rows, f32, dev, "u"), _vector(tokens, rows, i32, dev, "tokens"),
                        _vector(probs, rows, f32, dev, "probs"), dev)
    _check(_lib.kie_sample(a, _stream(None, dev)))
    return tokens, probs
