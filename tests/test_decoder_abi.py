"""CPU checks of the decoder operators' C ABI (include/molora_decoder.h): exports, workspace
arithmetic and the refusals, none of which launches anything (no GPU)."""
import ctypes
import os
import re

import pytest
import torch

import token_adapter_routing_amd as m
from token_adapter_routing_amd import decoder as D

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "molora_decoder.h")
FAKE = 0x10000  # an aligned address that nothing dereferences
EINVAL, ENOTSUP, ENOSPC = m.MOLORA_EINVAL, m.MOLORA_ENOTSUP, m.MOLORA_ENOSPC


def lib():
    if not os.path.exists(m.LIB_PATH):
        pytest.skip("library not built")
    return D._library()


def last():
    return lib().molora_last_error().decode()


def test_every_declared_symbol_is_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(molora_\w+)\s*\(", text)))
    assert names == sorted(m.decoder_symbols())
    for n in names:
        assert hasattr(lib(), n) and hasattr(m, n), n


ROUTE = dict(logits=FAKE, bias=None, N=4, K=16, k=2, score=0, n_group=1, topk_group=1, renorm=1, factor=1.0, idx=FAKE,
             w=FAKE, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(N=-1), EINVAL), (dict(K=0), ENOTSUP), (dict(K=65), ENOTSUP), (dict(k=0), ENOTSUP), (dict(k=9), ENOTSUP),
    (dict(K=4, k=5), ENOTSUP), (dict(score=2), EINVAL), (dict(score=-1), EINVAL), (dict(factor=float("nan")), EINVAL),
    (dict(factor=float("inf")), EINVAL), (dict(n_group=0), ENOTSUP), (dict(n_group=3), ENOTSUP),
    (dict(n_group=4, topk_group=5), ENOTSUP), (dict(n_group=4, topk_group=0), ENOTSUP),
    (dict(n_group=16, topk_group=1), ENOTSUP), (dict(logits=None), EINVAL), (dict(idx=None), EINVAL),
    (dict(w=None), EINVAL), (dict(logits=FAKE + 4), EINVAL), (dict(idx=FAKE + 2), EINVAL), (dict(bias=FAKE + 1), EINVAL),
    (dict(N=1 << 30), ENOTSUP), (dict(N=1 << 29, K=1, k=1), ENOTSUP)])
def test_route_scores_refusals(change, code):
    a = dict(ROUTE, **change)
    assert lib().molora_route_scores(*a.values()) == code, last()
    assert last()


def test_route_scores_of_no_tokens():
    a = dict(ROUTE, N=0, logits=None, idx=None, w=None)
    assert lib().molora_route_scores(*a.values()) == 0
    assert lib().molora_route_scores_backward(None, None, None, 0, 16, 2, 0, 1, 1.0, None, None) == 0


@pytest.mark.parametrize("change,code", [
    (dict(K=0), ENOTSUP), (dict(k=17), ENOTSUP), (dict(score=7), EINVAL), (dict(logits=None), EINVAL),
    (dict(idx=None), EINVAL), (dict(dw=None), EINVAL), (dict(dl=None), EINVAL), (dict(dl=FAKE + 8), EINVAL)])
def test_route_scores_backward_refusals(change, code):
    a = dict(logits=FAKE, idx=FAKE, dw=FAKE, N=4, K=16, k=2, score=0, renorm=1, factor=1.0, dl=FAKE, stream=None)
    a.update(change)
    assert lib().molora_route_scores_backward(*a.values()) == code, last()


def rows(token, head, p=FAKE):
    return D.MoloraRows(p, token, head)


def shape(**kw):
    a = dict(n_seq=2, n_heads=8, n_kv_heads=2, head_dim=64, Tq=10, Tkv=12, q_off=FAKE, kv_off=FAKE, window=0, sinks=0,
             scale=0.125)
    a.update(kw)
    return D.MoloraAttnShape(*a.values())


def attn(s=None, q=None, k=None, v=None, o=None, lse=FAKE, ws=None, size=0):
    r = ctypes.byref
    return lib().molora_attn_forward(r(s or shape()), r(q or rows(512, 64)), r(k or rows(128, 64)),
                                     r(v or rows(128, 64)), r(o or rows(512, 64)), lse, ws, size, None)


@pytest.mark.parametrize("change,code", [
    (dict(head_dim=96), ENOTSUP), (dict(head_dim=0), ENOTSUP), (dict(n_kv_heads=0), ENOTSUP), (dict(n_kv_heads=3), ENOTSUP),
    (dict(n_heads=0), ENOTSUP), (dict(n_heads=2048), ENOTSUP), (dict(n_seq=-1), EINVAL), (dict(Tq=-1), EINVAL),
    (dict(Tkv=-1), EINVAL), (dict(Tq=1 << 24), ENOTSUP), (dict(Tq=1 << 23, n_heads=1024), ENOTSUP),
    (dict(n_seq=1 << 21), ENOTSUP), (dict(n_seq=(1 << 24) - 1, n_heads=1024), ENOTSUP),
    (dict(window=-1), EINVAL), (dict(sinks=-1), EINVAL), (dict(sinks=(1 << 24) + 1), ENOTSUP), (dict(scale=0.0), EINVAL),
    (dict(scale=-1.0), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL),
    (dict(q_off=None), EINVAL), (dict(q_off=FAKE + 2), EINVAL), (dict(kv_off=FAKE + 1), EINVAL)])
def test_attention_shape_refusals(change, code):
    assert attn(shape(**change)) == code, last()
    n = ctypes.c_size_t()
    assert lib().molora_attn_backward_workspace(ctypes.byref(shape(**change)), ctypes.byref(n)) == code
    assert lib().molora_attn_forward_workspace(ctypes.byref(shape(**change)), ctypes.byref(n)) == code


@pytest.mark.parametrize("which,bad,code", [
    ("q", rows(512, 64, None), EINVAL), ("q", rows(512, 64, FAKE + 8), EINVAL), ("q", rows(-512, 64), EINVAL),
    ("k", rows(130, 64), EINVAL), ("v", rows(128, 60), EINVAL), ("q", rows(1 << 23, 64), ENOTSUP),
    ("k", rows(128, 1 << 40), ENOTSUP), ("o", rows(0, 64), EINVAL), ("o", rows(512, 32), EINVAL),
    ("o", rows(504, 64), EINVAL), ("o", rows(64, 632), EINVAL)])
def test_attention_rows_refusals(which, bad, code):
    assert attn(**{which: bad}) == code, last()
    assert last()


def test_attention_misaligned_lse_and_empty_calls():
    assert attn(lse=FAKE + 2) == EINVAL
    assert attn(shape(Tq=0), q=rows(512, 64, None), o=rows(512, 64, None)) == 0
    assert attn(shape(n_seq=0, q_off=None)) == 0


def test_attention_forward_workspace():
    r, n = ctypes.byref, ctypes.c_size_t()
    assert lib().molora_attn_forward_workspace(r(shape()), None) == EINVAL
    assert lib().molora_attn_forward_workspace(r(shape()), r(n)) == 0 and n.value == 0  # few keys: nothing to split
    few = shape(Tkv=5000)
    assert lib().molora_attn_forward_workspace(r(few), r(n)) == 0 and n.value > 0 and n.value % 256 == 0
    assert attn(few) == ENOSPC and attn(few, ws=FAKE, size=n.value - 1) == ENOSPC
    assert attn(few, ws=FAKE + 64, size=n.value) == ENOSPC
    assert lib().molora_attn_forward_workspace(r(shape(Tkv=5000, Tq=100000)), r(n)) == 0 and n.value == 0


def test_attention_backward_workspace_and_refusals():
    r, n = ctypes.byref, ctypes.c_size_t()
    L = lib()
    assert L.molora_attn_backward_workspace(r(shape()), None) == EINVAL
    assert L.molora_attn_backward_workspace(r(shape()), r(n)) == 0 and n.value >= 10 * 8 * 4 and n.value % 256 == 0
    q, k = rows(512, 64), rows(128, 64)

    def call(lse=FAKE, ws=FAKE, size=None, dq=q, dk=k, dv=k, dout=q):
        return L.molora_attn_backward(r(shape()), r(dout), r(q), r(k), r(k), r(q), lse, r(dq), r(dk), r(dv), ws,
                                      n.value if size is None else size, None)
    assert call(lse=None) == EINVAL
    assert call(ws=None) == ENOSPC and call(ws=FAKE + 16) == ENOSPC and call(size=n.value - 1) == ENOSPC
    assert call(dq=rows(0, 64)) == EINVAL and call(dk=rows(64, 64)) == EINVAL and call(dv=rows(128, 0)) == EINVAL
    assert call(dout=rows(512, 64, None)) == EINVAL


def cache(**kw):
    a = dict(k=FAKE, v=FAKE, ks=None, vs=None, n_pages=4, heads=2, page=16, dim=64, dtype=m.BF16)
    a.update(kw)
    return D.MoloraKvCache(*a.values())


BAD_CACHES = [(dict(n_pages=0), ENOTSUP), (dict(heads=0), ENOTSUP), (dict(page=8), ENOTSUP), (dict(page=48), ENOTSUP),
              (dict(page=512), ENOTSUP), (dict(dim=80), ENOTSUP), (dict(dtype=m.F32), EINVAL), (dict(k=None), EINVAL),
              (dict(v=FAKE + 8), EINVAL), (dict(dtype=m.E4M3), EINVAL), (dict(dtype=m.E4M3, ks=FAKE, vs=FAKE + 4), EINVAL)]


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_cache_refusals(change, code):
    r = ctypes.byref
    c = cache(**change)
    heads = max(1, c.n_kv_heads)
    assert lib().molora_kv_append(r(c), r(rows(128, 64)), r(rows(128, 64)), 3, 3, None, FAKE, 2, FAKE, None) == code, last()
    assert lib().molora_attn_decode(r(c), r(rows(128, 64)), r(rows(128, 64)), None, 3, heads, FAKE, 2, FAKE, 0, 0, 0.1,
                                    FAKE, 1 << 30, None) == code, last()


def append(c=None, k=None, v=None, T=3, n_seq=3, q_off=None, table=FAKE, width=2, lens=FAKE):
    r = ctypes.byref
    return lib().molora_kv_append(r(c or cache()), r(k or rows(128, 64)), r(v or rows(128, 64)), T, n_seq, q_off, table,
                                  width, lens, None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), EINVAL), (dict(T=1 << 24, q_off=FAKE), ENOTSUP), (dict(T=4), EINVAL), (dict(n_seq=-1), EINVAL),
    (dict(width=-1), EINVAL), (dict(width=1 << 26), ENOTSUP), (dict(table=None), EINVAL), (dict(lens=None), EINVAL),
    (dict(lens=FAKE + 1), EINVAL), (dict(q_off=FAKE + 2), EINVAL), (dict(k=rows(128, 64, None)), EINVAL),
    (dict(v=rows(127, 64)), EINVAL), (dict(T=0), 0), (dict(T=0, n_seq=0), 0), (dict(width=0), 0)])
def test_append_refusals(change, code):
    assert append(**change) == code, last()


def decode(c=None, q=None, o=None, lse=None, n_seq=3, heads=4, table=FAKE, width=64, lens=FAKE, window=0, sinks=0,
           scale=0.1, ws=FAKE, ws_bytes=1 << 30):
    r = ctypes.byref
    return lib().molora_attn_decode(r(c or cache()), r(q or rows(256, 64)), r(o or rows(256, 64)), lse, n_seq, heads, table,
                                    width, lens, window, sinks, scale, ws, ws_bytes, None)


@pytest.mark.parametrize("change,code", [
    (dict(heads=3), ENOTSUP), (dict(heads=0), ENOTSUP), (dict(n_seq=-1), EINVAL), (dict(n_seq=1 << 22), ENOTSUP),
    (dict(width=1 << 26), ENOTSUP), (dict(window=-1), EINVAL), (dict(sinks=-2), EINVAL), (dict(scale=0.0), EINVAL),
    (dict(q=rows(256, 64, None)), EINVAL), (dict(o=rows(128, 64)), EINVAL), (dict(lse=FAKE + 2), EINVAL),
    (dict(table=None), EINVAL), (dict(lens=None), EINVAL), (dict(ws=None), ENOSPC), (dict(ws=FAKE + 64), ENOSPC),
    (dict(ws_bytes=16), ENOSPC), (dict(n_seq=0), 0)])
def test_decode_refusals(change, code):
    assert decode(**change) == code, last()


def test_decode_workspace():
    n = ctypes.c_size_t()
    r = ctypes.byref
    L = lib()
    assert L.molora_attn_decode_workspace(r(cache()), 3, 4, 64, None) == EINVAL
    assert L.molora_attn_decode_workspace(r(cache()), 3, 5, 64, r(n)) == ENOTSUP
    assert L.molora_attn_decode_workspace(r(cache()), 3, 4, 1, r(n)) == 0 and n.value == 0  # 16 positions: one part
    assert L.molora_attn_decode_workspace(r(cache()), 3, 4, 64, r(n)) == 0 and n.value > 0
    assert L.molora_attn_decode_workspace(r(cache()), 0, 4, 64, r(n)) == 0 and n.value == 0


def test_binding_refuses_wrong_tensors():
    lib()
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="GPU"):
        m.molora_route_scores(x, 2)
    with pytest.raises(ValueError, match="float32"):
        m.molora_route_scores(x.double(), 2)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    off = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        m.molora_attn_forward(q, q, q, off)
    with pytest.raises(ValueError, match="e4m3"):
        m.KvCache(torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16),
                  torch.zeros(1, 1, 16, dtype=torch.uint8), torch.zeros(1, 1, 16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="dtype"):
        m.KvCache(torch.zeros(1, 1, 16, 64), torch.zeros(1, 1, 16, 64))
