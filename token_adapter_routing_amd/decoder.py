"""ctypes binding of the decoder's operators (include/molora_decoder.h) with the C entry points'
names: routing by scores, causal attention forward and backward, the paged key-value cache and the
attention of one new token over it.

As in ``binding``: arguments are checked and marshalled, missing outputs and workspaces come from
torch, nothing is computed here.  Tensors have to be on the current device.  Work goes to ``stream``
(default: the current one); what a call allocates belongs to that stream.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional, Tuple

import torch

from . import binding as _b
from .binding import BF16, _c_f, _c_i, _c_p, _c_sz, _check

E4M3 = 2
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1


class MoloraRows(ctypes.Structure):
    _fields_ = [("p", _c_p), ("token", ctypes.c_longlong), ("head", ctypes.c_longlong)]


class MoloraAttnShape(ctypes.Structure):
    _fields_ = [("n_seq", _c_i), ("n_heads", _c_i), ("n_kv_heads", _c_i), ("head_dim", _c_i), ("Tq", _c_i), ("Tkv", _c_i),
                ("q_off", _c_p), ("kv_off", _c_p), ("window", _c_i), ("sinks", _c_i), ("scale", _c_f)]


class MoloraKvCache(ctypes.Structure):
    _fields_ = [("k", _c_p), ("v", _c_p), ("k_scale", _c_p), ("v_scale", _c_p), ("n_pages", _c_i), ("n_kv_heads", _c_i),
                ("page_size", _c_i), ("head_dim", _c_i), ("dtype", _c_i)]


_SIGS = {
    "molora_route_scores": (_c_i, [_c_p, _c_p, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i, _c_f, _c_p, _c_p, _c_p]),
    "molora_route_scores_backward": (_c_i, [_c_p, _c_p, _c_p, _c_i, _c_i, _c_i, _c_i, _c_i, _c_f, _c_p, _c_p]),
    "molora_attn_forward_workspace": (_c_i, [_c_p, _c_p]),
    "molora_attn_forward": (_c_i, [_c_p] * 7 + [_c_sz, _c_p]),
    "molora_attn_backward_workspace": (_c_i, [_c_p, _c_p]),
    "molora_attn_backward": (_c_i, [_c_p] * 11 + [_c_sz, _c_p]),
    "molora_kv_append": (_c_i, [_c_p, _c_p, _c_p, _c_i, _c_i, _c_p, _c_p, _c_i, _c_p, _c_p]),
    "molora_attn_decode_workspace": (_c_i, [_c_p, _c_i, _c_i, _c_i, _c_p]),
    "molora_attn_decode": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_i, _c_i, _c_p, _c_i, _c_p, _c_i, _c_i, _c_f, _c_p, _c_sz,
                                  _c_p]),
    "molora_xf_serve_workspace": (_c_i, [_c_i, _c_i, _c_i, _c_p, _c_p, _c_i, _c_i, _c_i, _c_i, _c_p]),
    "molora_xf_prefill": (_c_i, [_c_i, _c_i, _c_i, _c_p, _c_p, _c_i, _c_i, _c_p, _c_p, _c_i, _c_p, _c_i, _c_i,  # .. sinks
                                 _c_p, _c_p, _c_i, _c_p, _c_p, _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "molora_xf_decode": (_c_i, [_c_i, _c_i, _c_i, _c_p, _c_p, _c_i, _c_p, _c_i, _c_p, _c_i, _c_i,  # .. sinks
                                _c_p, _c_p, _c_i, _c_p, _c_p, _c_p, _c_p, _c_p, _c_sz, _c_p]),
}
_lib = None


def _library() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        lib = _b.load_library()
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def decoder_symbols() -> Tuple[str, ...]:
    return tuple(_SIGS)


def _on_stream(fn):
    """Runs a call with ``stream=`` (a torch stream or a raw handle) as the current stream, so that what
    it allocates belongs to the stream that uses it."""
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream))
        if stream.device.index != torch.cuda.current_device():
            raise ValueError("stream belongs to another device than the current one")
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    call.__name__, call.__doc__, call.__wrapped__ = fn.__name__, fn.__doc__, fn
    return call


# The current device and stream by torch's short way where this torch has it (a call's marshalling is a
# good part of a small call's time: 2.8 us for torch.cuda.current_stream(), 0.1 us for this).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _here(t: torch.Tensor, name: str):
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    if d != _current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{_current_device()}")


def _flat(t: Optional[torch.Tensor], dtype, shape, name: str) -> Optional[int]:
    """Pointer of a contiguous tensor of exactly this type and shape (a tuple)."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} of shape {list(shape)}, got {t.dtype} of {list(t.shape)}")
    _here(t, name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t: torch.Tensor, shape, name: str) -> MoloraRows:
    """Rows [T][H][D] bf16 with any token and head strides."""
    if t.dtype != torch.bfloat16 or t.shape != shape:
        raise ValueError(f"{name} must be torch.bfloat16 of shape {list(shape)}, got {t.dtype} of {list(t.shape)}")
    _here(t, name)
    token, head, value = t.stride()
    if value != 1 and t.numel():
        raise ValueError(f"{name}: the values of a head must be contiguous")
    # a stride over one token or one head is never used: torch may give it any value
    return MoloraRows(t.data_ptr(), token if shape[0] > 1 else 0, head if shape[1] > 1 else 0)


def _stream() -> int:
    return _raw_stream(_current_device()) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream


def _workspace(ws: Optional[torch.Tensor], need: int, device):
    """Pointer and size of the caller's workspace (uint8, checked by the library) or of a new one, and it."""
    if ws is None:
        if need == 0:
            return None, 0, None
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    else:
        if ws.dtype != torch.uint8 or not ws.is_contiguous():
            raise ValueError("ws must be contiguous torch.uint8")
        _here(ws, "ws")
    return ws.data_ptr(), ws.numel(), ws


# ----------------------------------------------------------------------------------- routing

@_on_stream
def molora_route_scores(logits: torch.Tensor, k: int, bias: Optional[torch.Tensor] = None, score: int = SCORE_SOFTMAX,
                        n_group: int = 1, topk_group: int = 1, renorm: bool = True, factor: float = 1.0,
                        idx: Optional[torch.Tensor] = None, w: Optional[torch.Tensor] = None):
    """Top-k routing by softmax or sigmoid scores of logits [N][K] fp32, with a balance bias [K] for the
    selection and adapter groups: (idx int32 [N][k], w fp32 [N][k]), ready for molora_dispatch."""
    N, K = logits.shape
    if idx is None:
        idx = torch.empty(N, max(k, 0), dtype=torch.int32, device=logits.device)
    if w is None:
        w = torch.empty(N, max(k, 0), dtype=torch.float32, device=logits.device)
    _check(_library().molora_route_scores(
        _flat(logits, torch.float32, (N, K), "logits"), _flat(bias, torch.float32, (K,), "bias"), N, K, int(k), int(score),
        int(n_group), int(topk_group), int(bool(renorm)), float(factor), _flat(idx, torch.int32, (N, k), "idx"),
        _flat(w, torch.float32, (N, k), "w"), _stream()))
    return idx, w


@_on_stream
def molora_route_scores_backward(logits: torch.Tensor, idx: torch.Tensor, dw: torch.Tensor, score: int = SCORE_SOFTMAX,
                                 renorm: bool = True, factor: float = 1.0, dlogits: Optional[torch.Tensor] = None):
    """dL/dlogits [N][K] fp32 of molora_route_scores, its selection idx [N][k] held fixed; dw fp32 [N][k]."""
    N, K = logits.shape
    k = idx.shape[1]
    if dlogits is None:
        dlogits = torch.empty(N, K, dtype=torch.float32, device=logits.device)
    _check(_library().molora_route_scores_backward(
        _flat(logits, torch.float32, (N, K), "logits"), _flat(idx, torch.int32, (N, k), "idx"),
        _flat(dw, torch.float32, (N, k), "dw"), N, K, int(k), int(score), int(bool(renorm)), float(factor),
        _flat(dlogits, torch.float32, (N, K), "dlogits"), _stream()))
    return dlogits


# ----------------------------------------------------------------------------------- attention

@functools.lru_cache(maxsize=256)
def _attn_bytes(backward: bool, n_seq: int, Hq: int, Hkv: int, D: int, Tq: int, Tkv: int, window: int, sinks: int) -> int:
    """A call's workspace, which goes by these numbers alone (the address stands for offsets)."""
    lib, n = _library(), _c_sz()
    fn = lib.molora_attn_backward_workspace if backward else lib.molora_attn_forward_workspace
    _check(fn(ctypes.byref(MoloraAttnShape(n_seq, Hq, Hkv, D, Tq, Tkv, 256, None, window, sinks, 1.0)),
              ctypes.byref(n)))
    return n.value


@functools.lru_cache(maxsize=256)
def _decode_bytes(n_pages: int, heads: int, page: int, D: int, n_seq: int, n_heads: int, width: int) -> int:
    n = _c_sz()
    _check(_library().molora_attn_decode_workspace(
        ctypes.byref(MoloraKvCache(None, None, None, None, n_pages, heads, page, D, BF16)), n_seq, n_heads, width,
        ctypes.byref(n)))
    return n.value


def _shape(q, k, q_off, kv_off, scale, window, sinks) -> MoloraAttnShape:
    Tq, Hq, D = q.shape
    Tkv, Hkv, _ = k.shape
    n = q_off.numel() - 1
    if n < 0:
        raise ValueError("q_off needs n_seq + 1 entries")
    return MoloraAttnShape(n, Hq, Hkv, D, Tq, Tkv, _flat(q_off, torch.int32, (n + 1,), "q_off"),
                           _flat(kv_off, torch.int32, (n + 1,), "kv_off"), int(window), int(sinks),
                           1.0 / math.sqrt(D) if scale is None else float(scale))


@_on_stream
def molora_attn_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_off: torch.Tensor,
                        kv_off: Optional[torch.Tensor] = None, scale: Optional[float] = None, window: int = 0,
                        sinks: int = 0, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        ws: Optional[torch.Tensor] = None):
    """Causal attention of packed sequences: q bf16 [Tq][Hq][D], k and v bf16 [Tkv][Hkv][D] (any token and
    head strides), q_off and kv_off int32 [n_seq + 1] on the GPU; window 0: none.  Returns (o, lse), o
    bf16 [Tq][Hq][D], lse fp32 [Hq][Tq].  scale defaults to 1 / sqrt(D)."""
    Tq, Hq, D = q.shape
    kv = (k.shape[0], k.shape[1], D)
    if out is None:
        out = torch.empty(Tq, Hq, D, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty(Hq, Tq, dtype=torch.float32, device=q.device)
    s = _shape(q, k, q_off, kv_off, scale, window, sinks)
    lib, ref = _library(), ctypes.byref
    wp, wn, ws = _workspace(ws, _attn_bytes(False, s.n_seq, Hq, kv[1], D, Tq, kv[0], s.window, s.sinks), q.device)
    _check(lib.molora_attn_forward(
        ref(s), ref(_rows(q, (Tq, Hq, D), "q")), ref(_rows(k, kv, "k")), ref(_rows(v, kv, "v")),
        ref(_rows(out, (Tq, Hq, D), "out")), _flat(lse, torch.float32, (Hq, Tq), "lse"), wp, wn, _stream()))
    return out, lse


def molora_attn_forward_workspace(q: torch.Tensor, k: torch.Tensor, q_off: torch.Tensor, window: int = 0,
                                  sinks: int = 0) -> int:
    """Bytes of molora_attn_forward's ``ws`` for these shapes."""
    return _attn_bytes(False, q_off.numel() - 1, q.shape[1], k.shape[1], q.shape[2], q.shape[0], k.shape[0], int(window),
                       int(sinks))


def molora_attn_backward_workspace(q: torch.Tensor, k: torch.Tensor, q_off: torch.Tensor, window: int = 0,
                                   sinks: int = 0) -> int:
    """Bytes of molora_attn_backward's ``ws`` for these shapes."""
    return _attn_bytes(True, q_off.numel() - 1, q.shape[1], k.shape[1], q.shape[2], q.shape[0], k.shape[0], int(window),
                       int(sinks))


@_on_stream
def molora_attn_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                         lse: torch.Tensor, q_off: torch.Tensor, kv_off: Optional[torch.Tensor] = None,
                         scale: Optional[float] = None, window: int = 0, sinks: int = 0,
                         dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                         dv: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """Gradients (dq, dk, dv), bf16 and shaped like q, k, v, from dL/do and molora_attn_forward's o and lse."""
    Tq, Hq, D = q.shape
    qs, kv = (Tq, Hq, D), (k.shape[0], k.shape[1], D)
    if dq is None:
        dq = torch.empty(qs, dtype=torch.bfloat16, device=q.device)
    if dk is None:
        dk = torch.empty(kv, dtype=torch.bfloat16, device=q.device)
    if dv is None:
        dv = torch.empty(kv, dtype=torch.bfloat16, device=q.device)
    s = _shape(q, k, q_off, kv_off, scale, window, sinks)
    lib, ref = _library(), ctypes.byref
    wp, wn, ws = _workspace(ws, _attn_bytes(True, s.n_seq, Hq, kv[1], D, Tq, kv[0], s.window, s.sinks), q.device)
    _check(lib.molora_attn_backward(
        ref(s), ref(_rows(dout, qs, "dout")), ref(_rows(q, qs, "q")), ref(_rows(k, kv, "k")), ref(_rows(v, kv, "v")),
        ref(_rows(o, qs, "o")), _flat(lse, torch.float32, (Hq, Tq), "lse"), ref(_rows(dq, qs, "dq")),
        ref(_rows(dk, kv, "dk")), ref(_rows(dv, kv, "dv")), wp, wn, _stream()))
    return dq, dk, dv


# ----------------------------------------------------------------------------------- cache

class KvCache:
    """A paged key-value cache over the caller's tensors: k and v [n_pages][Hkv][page_size][D], bf16 or
    torch.float8_e4m3fn, the latter with uint8 scale bytes [n_pages][Hkv][page_size]."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None):
        if k.dim() != 4:
            raise ValueError("k must be [n_pages][n_kv_heads][page_size][head_dim]")
        n_pages, heads, page, D = k.shape
        if k.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise ValueError(f"cache dtype {k.dtype}: torch.bfloat16 or torch.float8_e4m3fn")
        e4m3 = k.dtype == torch.float8_e4m3fn
        if e4m3 != (k_scale is not None) or e4m3 != (v_scale is not None):
            raise ValueError("k_scale and v_scale go with an e4m3 cache, and only with one")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim, self.dtype = n_pages, heads, page, D, k.dtype
        self._c = MoloraKvCache(_flat(k, k.dtype, k.shape, "k"), _flat(v, k.dtype, k.shape, "v"),
                                _flat(k_scale, torch.uint8, k.shape[:3], "k_scale"),
                                _flat(v_scale, torch.uint8, k.shape[:3], "v_scale"), n_pages, heads, page, D,
                                E4M3 if e4m3 else BF16)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, n_pages: int, n_kv_heads: int, page_size: int, head_dim: int, dtype=torch.bfloat16, device="cuda"):
        """A new cache of zeros."""
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        k, v = (torch.zeros(shape, dtype=torch.uint8 if dtype == torch.float8_e4m3fn else dtype, device=device)
                for _ in range(2))
        if dtype != torch.float8_e4m3fn:
            return cls(k, v)
        ks, vs = (torch.full(shape[:3], 127, dtype=torch.uint8, device=device) for _ in range(2))
        return cls(k.view(dtype), v.view(dtype), ks, vs)


@_on_stream
def molora_kv_append(cache: KvCache, k: torch.Tensor, v: torch.Tensor, q_off: Optional[torch.Tensor],
                     table: torch.Tensor, lens: torch.Tensor):
    """Writes the newest rows of every sequence: rows [q_off[b], q_off[b+1]) of k and v (bf16 [T][Hkv][D])
    become the last ones of lens[b] tokens; q_off None: one row per sequence.  table int32
    [n_seq][width], lens int32 [n_seq], on the GPU."""
    _here(cache.k, "cache")
    n, width = table.shape
    shape = (k.shape[0], cache.n_kv_heads, cache.head_dim)
    ref = ctypes.byref
    _check(_library().molora_kv_append(
        cache._ref, ref(_rows(k, shape, "k")), ref(_rows(v, shape, "v")), shape[0], n,
        _flat(q_off, torch.int32, (n + 1,), "q_off"), _flat(table, torch.int32, (n, width), "table"), width,
        _flat(lens, torch.int32, (n,), "lens"), _stream()))


def molora_attn_decode_workspace(cache: KvCache, n_seq: int, n_heads: int, table_width: int) -> int:
    """Bytes of molora_attn_decode's ``ws``."""
    return _decode_bytes(cache.n_pages, cache.n_kv_heads, cache.page_size, cache.head_dim, int(n_seq), int(n_heads),
                         int(table_width))


@_on_stream
def molora_attn_decode(q: torch.Tensor, cache: KvCache, table: torch.Tensor, lens: torch.Tensor,
                       scale: Optional[float] = None, window: int = 0, sinks: int = 0,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       ws: Optional[torch.Tensor] = None):
    """Attention of one new token per sequence over the cache: q bf16 [n_seq][Hq][D], table int32
    [n_seq][width], lens int32 [n_seq] (with the new token).  Returns (o, lse), lse fp32 [n_seq][Hq]."""
    _here(cache.k, "cache")
    n, Hq, D = q.shape
    width = table.shape[1]
    if out is None:
        out = torch.empty(n, Hq, D, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty(n, Hq, dtype=torch.float32, device=q.device)
    lib, ref = _library(), ctypes.byref
    wp, wn, ws = _workspace(ws, molora_attn_decode_workspace(cache, n, Hq, width), q.device)
    qs = (n, Hq, cache.head_dim)
    _check(lib.molora_attn_decode(
        cache._ref, ref(_rows(q, qs, "q")), ref(_rows(out, qs, "out")), _flat(lse, torch.float32, (n, Hq), "lse"), n, Hq,
        _flat(table, torch.int32, (n, width), "table"), width, _flat(lens, torch.int32, (n,), "lens"), int(window),
        int(sinks), 1.0 / math.sqrt(D) if scale is None else float(scale), wp, wn, _stream()))
    return out, lse


# ----------------------------------------------------------------------------------- the decoder, serving

def _caches(model, caches):
    if len(caches) != len(model.layers):
        raise ValueError(f"{len(model.layers)} layers need as many caches, got {len(caches)}")
    for c in caches:
        _here(c.k, "cache")
    return (MoloraKvCache * len(caches))(*[c._c for c in caches])


def molora_xf_serve_workspace(model, caches, n_seq: int, N: int, table_width: int, k: int = 1) -> int:
    n = _c_sz()
    _check(_library().molora_xf_serve_workspace(model.d, model.f, len(model.layers), model._arr, _caches(model, caches),
                                                int(n_seq), int(N), int(table_width), int(k), ctypes.byref(n)))
    return n.value


def _serve(model, caches, x, q_off, table, lens, window, sinks, route, k, out, ws):
    N, (n, width) = x.shape[0], table.shape
    if q_off is None and N != n:
        raise ValueError(f"one token per sequence: {N} rows for {n} sequences")
    if out is None:
        out = torch.empty_like(x)
    arr = _caches(model, caches)
    lib = _library()
    need = _c_sz()
    _check(lib.molora_xf_serve_workspace(model.d, model.f, len(model.layers), model._arr, arr, n, N, width, int(k),
                                         ctypes.byref(need)))
    wp, wn, ws = _workspace(ws, need.value, x.device)
    K = next((L["lora"].K for L in model.layers if L.get("lora") is not None), 0)
    r = (None,) * 4
    if route is not None:
        P = N * int(k)
        r = tuple(_flat(t[:P] if name != "offsets" else t, dt, (K + 1,) if name == "offsets" else (P,), name)
                  for t, dt, name in zip(route, (torch.int32, torch.int32, torch.float32, torch.int32),
                                         ("offsets", "perm", "perm_w", "inv")))
    head = (model.d, model.f, len(model.layers), model._arr, arr, n)
    tail = (_flat(table, torch.int32, (n, width), "table"), width, _flat(lens, torch.int32, (n,), "lens"), int(window),
            int(sinks), _flat(x, torch.bfloat16, (N, model.d), "x"), _flat(out, torch.bfloat16, (N, model.d), "out"), int(k),
            *r, wp, wn, _stream())
    if q_off is None:
        _check(lib.molora_xf_decode(*head, *tail))
    else:
        _check(lib.molora_xf_prefill(*head, N, _flat(q_off, torch.int32, (n + 1,), "q_off"), *tail))
    return out


@_on_stream
def molora_xf_prefill(model, caches, x: torch.Tensor, q_off: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
                      window: int = 0, sinks: int = 0, route=None, k: int = 1, out: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None):
    """The decoder (an XfModel) over prompts that open their sequences: x bf16 [N][d] packed rows, one KvCache
    per layer, route = (offsets, perm, perm_w, inv) of molora_dispatch for the N tokens."""
    return _serve(model, caches, x, q_off, table, lens, window, sinks, route, k, out, ws)


@_on_stream
def molora_xf_decode(model, caches, x: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, window: int = 0,
                     sinks: int = 0, route=None, k: int = 1, out: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None):
    """The decoder over one new token per sequence, x bf16 [n_seq][d]; lens with the new tokens."""
    return _serve(model, caches, x, None, table, lens, window, sinks, route, k, out, ws)
