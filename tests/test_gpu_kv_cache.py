"""The paged cache: molora_kv_append and molora_attn_decode against the fp64 oracle.

Appending is exact: 16-bit rows are copied, 8-bit rows are the oracle's e4m3 values and scale bytes.
Decode errs as the packed attention does (see test_gpu_attn.py): weights rounded to bf16 (2^-8 of
sum p |v|), the result rounded once (2^-8), fp32 sums within 2^-12; the cache's values enter exactly,
since an e4m3 value times a power of two is a bf16 value."""
import math

import numpy as np
import pytest
import torch

from gpu_util import host, need_gpu
from oracle import decoder_ops as O

pytestmark = pytest.mark.gpu
HALF, FINE = 2.0 ** -8, 2.0 ** -12
E4M3 = torch.float8_e4m3fn


def normal(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def values(x, scale):
    v = f64(x.float() if x.dtype == E4M3 else x)
    return v if scale is None else v * 2.0 ** (f64(scale)[..., None] - 127)


def pages(lens, page, seed, spare=3, width=None):
    need = [-(-max(n, 0) // page) for n in lens]
    n_pages = sum(need) + spare
    order = np.random.default_rng(seed).permutation(n_pages)
    table = np.full((len(lens), width or max(max(need), 1) + 1), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, n_pages


def filled(m, lens, Hkv, D, page, dtype, seed, junk=float("nan")):
    """A cache whose sequences hold random rows and whose other rows hold `junk`."""
    table, n_pages = pages(lens, page, seed)
    shape = (n_pages, Hkv, page, D)
    ks, vs = normal(seed, *shape), normal(seed + 1, *shape)
    used = np.zeros((n_pages, page), bool)
    for b, n in enumerate(lens):
        for j in range(n):
            used[table[b, j // page], j % page] = True
    used = torch.from_numpy(used)[:, None, :, None]
    if dtype == torch.bfloat16:
        k, v = (torch.where(used, x, torch.full_like(x, junk)).cuda() for x in (ks, vs))
        return m.KvCache(k, v), torch.from_numpy(table).cuda()
    out = []
    for x in (ks, vs):
        q = x.float().mul(40).clamp(-448, 448)
        q = torch.where(used, q, torch.full_like(q, junk)).to(E4M3).cuda()
        out.append((q, torch.randint(110, 125, shape[:3], dtype=torch.uint8, generator=torch.Generator().manual_seed(seed)).cuda()))
    (k, a), (v, b) = out
    return m.KvCache(k, v, a, b), torch.from_numpy(table).cuda()


def clean(x):
    return np.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0)


def check(m, cache, table, lens, q, window=0, sinks=0, **kw):
    o, lse = m.molora_attn_decode(q.cuda(), cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                  window=window, sinks=sinks, **kw)
    scale = kw.get("scale") or 1 / math.sqrt(q.shape[2])
    kc, vc = clean(values(cache.k, cache.k_scale)), clean(values(cache.v, cache.v_scale))
    ro, rl, mag = O.decode(f64(q), kc, vc, host(table), lens, scale, window, sinks)
    go, gl = f64(o), f64(lse)
    bad = ~(np.abs(go - ro) <= HALF * (mag + np.abs(ro)) + FINE * mag + 1e-30)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3])
    assert (np.isneginf(gl) == np.isneginf(rl)).all()
    fin = np.isfinite(rl)
    assert (np.abs(gl - rl)[fin] <= 2.0 ** -14 * (1 + np.abs(rl[fin]))).all()
    return o, lse


DTYPES = [torch.bfloat16, E4M3]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_lengths_and_pages(dtype, D, page):
    m = need_gpu()
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 513]
    cache, table = filled(m, lens, 2, D, page, dtype, page)
    o, lse = check(m, cache, table, lens, normal(1, len(lens), 4, D))
    assert (o[0] == 0).all() and torch.isneginf(lse[0]).all()


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 5), (8, 2), (15, 3), (16, 1), (17, 1), (48, 2), (40, 1)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_heads(Hq, Hkv, dtype):
    m = need_gpu()
    lens = [70, 5, 0, 400]
    cache, table = filled(m, lens, Hkv, 64, 16, dtype, Hq)
    check(m, cache, table, lens, normal(2, 4, Hq, 64))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("window", [1, 2, 16, 31, 33, 64, 100, 2000])
@pytest.mark.parametrize("sinks", [0, 1, 4, 32, 40, 1500])
def test_window_and_sinks_with_freed_pages(dtype, window, sinks):
    """The pages that nothing sees any more are gone from the table, or hold NaN."""
    m = need_gpu()
    lens = [1, 31, 97, 600, 1203]
    page = 16
    cache, table = filled(m, lens, 1, 64, page, dtype, window + sinks)
    t = host(table).copy()
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            if i * page >= sinks and (i + 1) * page <= n - window:
                cache.k.view(torch.uint8)[t[b, i]] = 0x7f
                cache.v.view(torch.uint8)[t[b, i]] = 0x7f
                t[b, i] = -1 if (i + b) % 2 else t[b, i]
    check(m, cache, torch.from_numpy(t).cuda(), lens, normal(3, 5, 4, 64), window=window, sinks=sinks)


def test_bad_pages_and_lengths():
    """Entries outside the pool are not visible, lengths past the table are limited, negative ones 0."""
    m = need_gpu()
    lens = [100, 64, 40, 10]
    cache, table = filled(m, lens, 2, 64, 16, torch.bfloat16, 5, junk=0.0)
    t = host(table).copy()
    t[0, 1], t[0, 6], t[1, :] = cache.n_pages, -7, 2 ** 30
    t[2, 3:] = t[2, 0]
    o, lse = check(m, cache, torch.from_numpy(t).cuda(), [100, 64, 10 ** 9, -3], normal(4, 4, 4, 64))
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all() and (o[3] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_long_sequences_in_many_parts(dtype):
    m = need_gpu()
    lens = [5000, 257, 3, 9001]
    cache, table = filled(m, lens, 1, 128, 64, dtype, 6)
    assert m.molora_attn_decode_workspace(cache, 4, 4, table.shape[1]) > 0
    check(m, cache, table, lens, normal(5, 4, 4, 128))
    check(m, cache, table, lens, normal(6, 4, 4, 128), window=4097, sinks=33)


def test_one_part_and_many_parts_agree():
    """A table one page wide leaves nothing to split; a wide one splits by the length alone."""
    m = need_gpu()
    lens = [200, 13]
    cache, table = filled(m, lens, 2, 64, 256, torch.bfloat16, 7)
    narrow, wide = table[:, :1].contiguous(), torch.full((2, 500), -1, dtype=torch.int32, device="cuda")
    wide[:, :1] = narrow
    assert m.molora_attn_decode_workspace(cache, 2, 4, 1) == 0
    q = normal(7, 2, 4, 64)
    a, b = check(m, cache, narrow, lens, q), check(m, cache, wide, lens, q)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])  # 200 positions are one part either way


def test_many_sequences():
    m = need_gpu()
    lens = [(i * 37) % 90 for i in range(700)]
    cache, table = filled(m, lens, 1, 64, 16, torch.bfloat16, 8)
    check(m, cache, table, lens, normal(8, 700, 2, 64))


def test_large_scores():
    m = need_gpu()
    lens = [300, 300]
    cache, table = filled(m, lens, 1, 64, 16, torch.bfloat16, 9)
    q = (normal(9, 2, 2, 64).float() * torch.tensor([8.0, 0.0])[:, None, None]).to(torch.bfloat16)
    check(m, cache, table, lens, q)
    check(m, cache, table, lens, q, scale=0.01)


def test_page_past_4_gb():
    m = need_gpu()
    n_pages = 150000  # 150000 x 2 x 128 x 64 x 2 bytes = 4.9 GB each
    k = torch.zeros(n_pages, 2, 128, 64, dtype=torch.bfloat16, device="cuda")
    cache = m.KvCache(k, torch.zeros_like(k))
    table = torch.tensor([[149999, 140001, 3]], dtype=torch.int32, device="cuda")
    new_k, new_v = normal(10, 300, 2, 64), normal(11, 300, 2, 64)
    off, lens = torch.tensor([0, 300], dtype=torch.int32, device="cuda"), torch.tensor([300], dtype=torch.int32, device="cuda")
    m.molora_kv_append(cache, new_k.cuda(), new_v.cuda(), off, table, lens)
    assert torch.equal(cache.k[149999, :, 7].cpu(), new_k[7]) and torch.equal(cache.v[140001, 1, 3].cpu(), new_v[131, 1])
    q = normal(12, 1, 4, 64)
    o, _ = m.molora_attn_decode(q.cuda(), cache, table, lens)
    ro, _, mag = O.attn(f64(q), f64(new_k), f64(new_v), np.array([0, 1]), np.array([0, 300]), 0.125)
    assert (np.abs(f64(o) - ro) <= HALF * (mag + np.abs(ro)) + FINE * mag).all()


def test_strides_and_in_place():
    m = need_gpu()
    lens = [90, 0, 33]
    cache, table = filled(m, lens, 2, 64, 16, torch.bfloat16, 13)
    q = normal(13, 3, 4, 64)
    ref, _ = check(m, cache, table, lens, q)
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    wide = torch.full((3, 6, 72), 9.0, dtype=torch.bfloat16, device="cuda")
    view = wide[:, 1:5, :64]
    view.copy_(q)
    o, _ = m.molora_attn_decode(view, cache, table, L, out=view)  # into q itself
    assert o is view and torch.equal(view.contiguous(), ref)
    assert (wide[:, 0] == 9).all() and (wide[:, 5] == 9).all() and (wide[:, :, 64:] == 9).all()


# ------------------------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Hkv,D,page", [(1, 64, 16), (3, 128, 32), (8, 64, 256), (16, 128, 64)])
def test_append(dtype, Hkv, D, page):
    m = need_gpu()
    new, past = [5, 0, 1, 70, 130], [0, 9, 16, 31, 200]
    lens = [a + b for a, b in zip(new, past)]
    table, n_pages = pages(lens, page, 20)
    shape = (n_pages, Hkv, page, D)
    T = sum(new)
    k, v = normal(21, T, Hkv, D), normal(22, T, Hkv, D)
    k[3] *= 1e4
    v[4] = 0
    k[7, 0, 0] = 448.0
    v[9] *= 2.0 ** -60
    if dtype == torch.bfloat16:
        cache = m.KvCache(normal(23, *shape).cuda(), normal(24, *shape).cuda())
    else:
        cache = m.KvCache(*(normal(s, *shape).cuda().to(E4M3) for s in (23, 24)),
                          *(torch.full(shape[:3], 9, dtype=torch.uint8, device="cuda") for _ in range(2)))
    before = [x.clone() for x in (cache.k, cache.v)]
    off = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    # k and v as parts of one buffer
    both = torch.cat([k, v], 1).cuda()
    m.molora_kv_append(cache, both[:, :Hkv], both[:, Hkv:], off, torch.from_numpy(table).cuda(),
                       torch.tensor(lens, dtype=torch.int32, device="cuda"))
    for x, old, scale, rows in ((cache.k, before[0], cache.k_scale, k), (cache.v, before[1], cache.v_scale, v)):
        want, byte = f64(old.float()), np.full(shape[:3], 9)
        quant = O.e4m3_rows(f64(rows)) if dtype == E4M3 else (f64(rows), None)
        t = 0
        for b, n in enumerate(new):
            for j in range(past[b], lens[b]):
                p, row = O.place(table, page, b, j, n_pages)
                want[p, :, row] = quant[0][t]
                if byte is not None and quant[1] is not None:
                    byte[p, :, row] = quant[1][t]
                t += 1
        np.testing.assert_array_equal(f64(x.float()), want)
        if scale is not None:
            np.testing.assert_array_equal(host(scale), byte)


def test_append_every_bf16_value():
    """e4m3 of every finite bf16 as the only value of its row, and as one beside a larger one; non-finite."""
    m = need_gpu()
    bits = torch.arange(0, 65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    fin = bits[torch.isfinite(bits)]
    x = torch.zeros(fin.numel(), 2, 64, dtype=torch.bfloat16)
    x[:, 0, 17] = fin
    x[:, 1, 5] = fin
    x[:, 1, 63] = 1.0
    T = x.shape[0]
    page = 256
    n_pages = -(-T // page)
    cache = m.KvCache.empty(n_pages, 2, page, 64, dtype=E4M3)
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None]
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    m.molora_kv_append(cache, x.cuda(), (-x).cuda(), off, table, off[1:].contiguous())
    rows = cache.k.float().transpose(1, 2).reshape(-1, 2, 64)[:T].cpu()
    byte = cache.k_scale.transpose(1, 2).reshape(-1, 2)[:T].cpu()
    n = (byte.int() - 127)[..., None]
    y = torch.ldexp(x.double(), -n).float()
    assert torch.equal(rows, y.clamp(-448, 448).to(E4M3).float())
    big = x.double().abs().amax(-1)
    ceil = 448 * torch.ldexp(torch.ones((), dtype=torch.float64), n[..., 0])
    assert (big <= ceil).all() and ((big > ceil / 2) | (n[..., 0] == -112)).all()
    assert torch.equal(cache.v.float().transpose(1, 2).reshape(-1, 2, 64)[:T].cpu(), -rows)
    odd = torch.ones(3, 2, 64, dtype=torch.bfloat16)
    odd[0, 0, 3], odd[1, 1, 4], odd[2, 0, 5] = math.inf, -math.inf, math.nan
    m.molora_kv_append(cache, odd.cuda(), odd.cuda(), torch.tensor([0, 3], dtype=torch.int32, device="cuda"), table,
                       torch.tensor([3], dtype=torch.int32, device="cuda"))
    got = cache.k[0, :, :3].float().cpu()
    one = 256.0  # 1 = 256 x 2^-8
    assert got[0, 0, 3] == 448 and got[1, 1, 4] == -448 and torch.isnan(got[0, 2, 5])
    assert got[0, 0, 0] == one and got[0, 2, 0] == one and (cache.k_scale[0, :, :3] == 127 - 8).all()


def test_append_one_row_per_sequence():
    m = need_gpu()
    B, page = 130, 16
    lens = [(7 * i) % 50 + 1 for i in range(B)]
    lens[3], lens[4], lens[5] = 0, -2, 10 ** 6  # nowhere to write
    table, n_pages = pages([max(min(n, 64), 1) for n in lens], page, 30, width=4)
    table[6] = n_pages + 2
    table[7] = -1
    cache = m.KvCache.empty(n_pages, 2, page, 64)
    k, v = normal(31, B, 2, 64), normal(32, B, 2, 64)
    m.molora_kv_append(cache, k.cuda(), v.cuda(), None, torch.from_numpy(table).cuda(),
                       torch.tensor(lens, dtype=torch.int32, device="cuda"))
    want = torch.zeros_like(cache.k, device="cpu")
    for b in range(B):
        at = O.place(table, page, b, lens[b] - 1, n_pages)
        if at is not None:
            want[at[0], :, at[1]] = k[b]
    assert torch.equal(cache.k.cpu(), want)
    assert int((want != 0).any(-1).sum()) == 2 * (B - 5)


def test_append_rows_outside_sequences_and_bad_offsets():
    m = need_gpu()
    cache = m.KvCache.empty(4, 1, 16, 64)
    table = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    k = normal(33, 12, 1, 64).cuda()
    off = torch.tensor([2, 5, 9], dtype=torch.int32, device="cuda")  # rows 0, 1 and 9.. belong to nobody
    m.molora_kv_append(cache, k, k, off, table, torch.tensor([3, 6], dtype=torch.int32, device="cuda"))
    want = torch.zeros_like(cache.k)
    want[0, 0, :3], want[1, 0, 2:6] = k[2:5, 0], k[5:9, 0]
    assert torch.equal(cache.k, want)
    # more rows than the sequence is long: the first ones have no position
    m.molora_kv_append(cache, k, k, torch.tensor([0, 6, 12], dtype=torch.int32, device="cuda"), table,
                       torch.tensor([2, 40], dtype=torch.int32, device="cuda"))
    want[0, 0, :2] = k[4:6, 0]  # sequence 1: positions 34.. are past its table
    assert torch.equal(cache.k, want)


def test_decoding_step_by_step_equals_the_packed_attention():
    """Append a token, attend, 40 times over; the rows are those of one causal call."""
    m = need_gpu()
    T, Hq, Hkv, D, page = 40, 4, 2, 128, 16
    q, k, v = normal(40, T, Hq, D).cuda(), normal(41, T, Hkv, D).cuda(), normal(42, T, Hkv, D).cuda()
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    for window, sinks in ((0, 0), (9, 3)):
        ref, rl = m.molora_attn_forward(q, k, v, off, window=window, sinks=sinks)
        cache = m.KvCache.empty(5, Hkv, page, D)
        table = torch.tensor([[4, 0, 2]], dtype=torch.int32, device="cuda")
        lens = torch.zeros(1, dtype=torch.int32, device="cuda")
        for t in range(T):
            lens += 1
            m.molora_kv_append(cache, k[t:t + 1], v[t:t + 1], None, table, lens)
            o, lse = m.molora_attn_decode(q[t:t + 1], cache, table, lens, window=window, sinks=sinks)
            assert (lse[0] - rl[:, t]).abs().max() < 1e-4
            # both round the same weights to bf16 and the result once
            assert (o.float() - ref[t:t + 1].float()).abs().max() <= 4 * HALF * v.float().abs().max()


@pytest.mark.parametrize("dtype", DTYPES)
def test_captured_decode_loop_replays(dtype):
    m = need_gpu()
    B, Hq, Hkv, D, page = 6, 8, 2, 64, 16
    cache = m.KvCache.empty(6 * 40, Hkv, page, D, dtype=dtype)
    table = torch.randperm(6 * 40)[:6 * 38].view(6, 38).to(torch.int32).cuda()
    start = torch.tensor([0, 3, 15, 100, 500, 31], dtype=torch.int32, device="cuda")
    lens = start.clone()
    q, k, v = (torch.empty(B, h, D, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))
    one = torch.ones(B, dtype=torch.int32, device="cuda")

    def step():
        lens.add_(one)
        m.molora_kv_append(cache, k, v, None, table, lens)
        return m.molora_attn_decode(q, cache, table, lens, window=60, sinks=4)
    for x in (q, k, v):
        x.normal_()
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = step()
    state = [x.clone() for x in (cache.k, cache.v)]
    lens.copy_(start)
    for i in range(20):
        for x in (q, k, v):
            x.normal_()
        at = lens.clone()
        cache.k.copy_(state[0]), cache.v.copy_(state[1])
        g.replay()
        torch.cuda.synchronize()
        got, after = (o.clone(), lse.clone()), [x.clone() for x in (cache.k, cache.v)]
        lens.copy_(at)
        cache.k.copy_(state[0]), cache.v.copy_(state[1])
        eager = step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], eager[0]) and torch.equal(got[1], eager[1])
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(after, (cache.k, cache.v)))
        state = after


def test_streams():
    m = need_gpu()
    lens = [3000, 17]
    sets = [(filled(m, lens, 2, 64, 16, torch.bfloat16, s), normal(s, 2, 4, 64)) for s in (50, 51)]
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ins = [q.cuda() for _, q in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[m.molora_attn_decode(q, c, t, L, stream=s) for _ in range(5)] for ((c, t), _), q, s in zip(sets, ins, streams)]
    torch.cuda.synchronize()
    for ((c, t), q), got in zip(sets, outs):
        ref = check(m, c, t, lens, q)
        assert all(torch.equal(o, ref[0]) and torch.equal(l, ref[1]) for o, l in got)


def test_binding_refusals():
    m = need_gpu()
    cache = m.KvCache.empty(4, 2, 16, 64)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    t, n = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        m.molora_attn_decode(q, cache, t.long(), n)
    with pytest.raises(ValueError):
        m.molora_attn_decode(q, cache, t[:1], n)
    with pytest.raises(ValueError):
        m.molora_attn_decode(q, cache, t, n.cpu())
    with pytest.raises(ValueError):
        m.molora_attn_decode(q[..., :32], cache, t, n)
    with pytest.raises(m.MoloraError, match="workspace"):
        m.molora_attn_decode(q, cache, torch.zeros(2, 300, dtype=torch.int32, device="cuda"), n,
                             ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(m.MoloraError, match="page_size"):
        m.molora_attn_decode(q, m.KvCache.empty(4, 2, 24, 64), t, n)
    with pytest.raises(ValueError):
        m.molora_kv_append(cache, q, q, None, t, n)  # 4 heads into a cache of 2
    with pytest.raises(m.MoloraError, match="rows"):
        x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
        m.molora_kv_append(cache, x, x, None, t, n)
