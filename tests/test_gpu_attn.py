"""Causal attention of packed sequences, forward and backward, against the fp64 oracle on the same
bf16 inputs.

Bounds, element by element.  bf16 rounds by at most 2^-8 of a value.  Forward: the weights enter the
second product rounded to bf16 (2^-8 of sum p |v|) and o is rounded once (2^-8 |o|); the fp32 part
(scores summed over D terms, exp, the running sum) errs by less than 2^-12 of the same sums for the
score sizes used here (|scale q.k| < 2^6: D 2^-24 2^6 < 2^-11 relative in the worst order, and sums
of random signs stay far below that).  lse: fp32 throughout, D 2^-24 times the magnitudes of the
largest score, below 2^-14.  Backward, from the same o and lse: P and dS are rounded to bf16 (2^-8 of
the sums of |dS| |k| and so on) and the result is rounded (2^-8); dS = P (dP - delta) is formed in
fp32 from sums whose magnitudes (the oracle's `wide`) it keeps to 2^-12."""
import math

import numpy as np
import pytest
import torch

from gpu_util import host, need_gpu
from oracle import decoder_ops as O

pytestmark = pytest.mark.gpu
HALF, FINE = 2.0 ** -8, 2.0 ** -12


def normal(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def offs(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


class Case:
    def __init__(self, q_lens, kv_lens, Hq, Hkv, D, window=0, sinks=0, seed=0, scale=None):
        self.q_off, self.kv_off = offs(q_lens), offs(kv_lens)
        Tq, Tk = int(self.q_off[-1]), int(self.kv_off[-1])
        self.q, self.do = normal(seed, Tq, Hq, D), normal(seed + 1, Tq, Hq, D)
        self.k, self.v = normal(seed + 2, Tk, Hkv, D), normal(seed + 3, Tk, Hkv, D)
        self.kw = dict(window=window, sinks=sinks)
        self.scale = scale

    def off(self):
        return torch.from_numpy(self.q_off).cuda(), torch.from_numpy(self.kv_off).cuda()

    def oracle(self):
        s = self.scale or 1 / math.sqrt(self.q.shape[2])
        return O.attn(f64(self.q), f64(self.k), f64(self.v), self.q_off, self.kv_off, s, **self.kw)


def check_forward(c, o, lse):
    ro, rl, mag = c.oracle()
    go, gl = f64(o), f64(lse)
    bad = np.abs(go - ro) > HALF * (mag + np.abs(ro)) + FINE * mag + 1e-30
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], np.abs(go - ro).max())
    inside = np.zeros(ro.shape[0], bool)
    inside[c.q_off[0]:c.q_off[-1]] = True
    none = np.isneginf(rl)
    assert (np.isneginf(gl) == none)[:, inside].all()
    fin = ~none & inside[None]
    assert (np.abs(gl - rl)[fin] <= 2.0 ** -14 * (1 + np.abs(rl[fin]))).all()
    return ro


def check_backward(c, o, lse, got):
    s = c.scale or 1 / math.sqrt(c.q.shape[2])
    ref, mag, wide = O.attn_backward(f64(c.do), f64(c.q), f64(c.k), f64(c.v), f64(o), f64(lse), c.q_off, c.kv_off, s, **c.kw)
    for name, g, r, a, w in zip(("dq", "dk", "dv"), got, ref, mag, wide):
        err, bound = np.abs(f64(g) - r), HALF * (a + np.abs(r)) + FINE * w + 1e-30
        assert (err <= bound).all(), (name, int((err > bound).sum()), (err / bound).max())


def run(m, c, backward=True):
    q, k, v, do = (x.cuda() for x in (c.q, c.k, c.v, c.do))
    q_off, kv_off = c.off()
    o, lse = m.molora_attn_forward(q, k, v, q_off, kv_off, scale=c.scale, **c.kw)
    check_forward(c, o, lse)
    if backward:
        got = m.molora_attn_backward(do, q, k, v, o, lse, q_off, kv_off, scale=c.scale, **c.kw)
        check_backward(c, o, lse, got)
        return o, lse, got
    return o, lse


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("L", [1, 2, 15, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 257, 400])
def test_lengths(L, D):
    run(need_gpu(), Case([L], [L], 2, 1, D, seed=L))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (8, 8), (6, 2), (4, 1), (16, 1), (24, 8)])
def test_heads(Hq, Hkv):
    run(need_gpu(), Case([70, 5], [70, 5], Hq, Hkv, 64, seed=Hq))


@pytest.mark.parametrize("lens", [[3, 0, 130, 1, 64, 0], [0, 0], [1] * 70, [128, 128, 128], [200, 1, 1, 200], [0, 300]])
def test_packed_sequences(lens):
    run(need_gpu(), Case(lens, lens, 4, 2, 64, seed=len(lens)))


@pytest.mark.parametrize("q_lens,kv_lens", [([1], [300]), ([5, 40], [200, 41]), ([130, 1, 0], [150, 64, 30]),
                                            ([64], [65]), ([10, 0, 3], [10, 7, 130])])
def test_queries_behind_earlier_keys(q_lens, kv_lens):
    run(need_gpu(), Case(q_lens, kv_lens, 4, 2, 128, seed=9))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_lens,kv_lens,window,sinks", [
    ([1], [2000], 0, 0), ([20], [1500], 0, 0), ([130, 0, 7], [1000, 50, 2100], 0, 0), ([800], [800], 0, 0),
    ([33], [1700], 900, 0), ([33], [1700], 500, 70), ([900, 40], [20, 1600], 0, 0)])
def test_keys_split_over_workgroups(q_lens, kv_lens, window, sinks, D):
    """Few query rows before many keys: parts and their join, forward and backward."""
    m = need_gpu()
    c = Case(q_lens, kv_lens, 4, 2, D, window=window, sinks=sinks, seed=30)
    assert m.molora_attn_forward_workspace(c.q.cuda(), c.k.cuda(), c.off()[0], window, sinks) > 0
    a, b = run(m, c), run(m, c)
    for x, y in zip((a[0], a[1], *a[2]), (b[0], b[1], *b[2])):
        assert torch.equal(x, y)


@pytest.mark.parametrize("n_seq", [15, 16, 17, 63, 64, 65, 200])
def test_numbers_of_sequences(n_seq):
    """Tiles are found in three ways, by the number of sequences."""
    lens = [(i * 53) % 190 for i in range(n_seq)]
    kv = [n + (i * 31) % 70 if n else 0 for i, n in enumerate(lens)]
    run(need_gpu(), Case(lens, kv, 2, 1, 64, window=40, sinks=3, seed=n_seq))
    run(need_gpu(), Case(lens, kv, 1, 1, 64, seed=n_seq))


def test_key_tiles_split_into_chunks():
    """Long sequences of few heads: the backward's key tiles in chunks, a window's sinks apart."""
    run(need_gpu(), Case([2500, 0, 1100], [2500, 9, 1300], 2, 1, 64, seed=31))
    run(need_gpu(), Case([2500, 0, 1100], [2500, 9, 1300], 4, 1, 64, window=200, sinks=150, seed=32))
    run(need_gpu(), Case([1600], [1600], 4, 1, 128, window=300, sinks=5, seed=33))


def test_sinks_of_many_sequences():
    """So many sink tiles that they are not taken apart: a long one still runs as a whole."""
    lens = [400] + [3] * 300 + [700] + [2] * 300
    run(need_gpu(), Case(lens, lens, 8, 2, 64, window=64, sinks=2, seed=35))


def test_no_keys_with_window_and_sinks():
    m = need_gpu()
    q = torch.ones(9, 2, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    off, none = torch.tensor([0, 4, 9], dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    o, lse = m.molora_attn_forward(q, k, k, off, none, window=2, sinks=3)
    assert (o == 0).all() and torch.isneginf(lse).all()
    dq, dk, dv = m.molora_attn_backward(q, q, k, k, o, lse, off, none, window=2, sinks=3)
    assert (dq == 0).all() and dk.numel() == 0 and dv.numel() == 0


def test_workspace_given():
    m = need_gpu()
    c = Case([20], [1500], 4, 2, 64, seed=34)
    q, k, v, do = (x.cuda() for x in (c.q, c.k, c.v, c.do))
    q_off, kv_off = c.off()
    ws = torch.full((m.molora_attn_forward_workspace(q, k, q_off) + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    o, lse = m.molora_attn_forward(q, k, v, q_off, kv_off, ws=ws)  # whatever it holds
    check_forward(c, o, lse)
    assert (ws[-512:] == 0xFF).all()
    n = m.molora_attn_backward_workspace(q, k, q_off)
    wb = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    check_backward(c, o, lse, m.molora_attn_backward(do, q, k, v, o, lse, q_off, kv_off, ws=wb))
    assert (wb[n:] == 0xFF).all()
    with pytest.raises(m.MoloraError, match="workspace"):
        m.molora_attn_forward(q, k, v, q_off, kv_off, ws=ws[:256])
    with pytest.raises(m.MoloraError, match="workspace"):
        m.molora_attn_backward(do, q, k, v, o, lse, q_off, kv_off, ws=wb[:256])


@pytest.mark.parametrize("q_lens,kv_lens", [([40], [10]), ([200, 5], [3, 0]), ([130], [129]), ([300], [140])])
@pytest.mark.parametrize("window", [0, 7])
def test_rows_that_see_nothing(q_lens, kv_lens, window):
    m = need_gpu()
    c = Case(q_lens, kv_lens, 2, 1, 64, window=window, seed=10)
    o, lse, (dq, dk, dv) = run(m, c)
    for b, (a, n) in enumerate(zip(q_lens, kv_lens)):
        lo = int(c.q_off[b])
        empty = max(a - n, 0)
        assert (o[lo:lo + empty] == 0).all() and torch.isneginf(lse[:, lo:lo + empty]).all()
        assert (dq[lo:lo + empty] == 0).all()


@pytest.mark.parametrize("window", [1, 2, 31, 32, 64, 65, 100, 128, 1000])
@pytest.mark.parametrize("sinks", [0, 1, 4, 33, 64, 70, 500])
def test_window_and_sinks(window, sinks):
    run(need_gpu(), Case([333, 40], [333, 90], 2, 1, 64, window=window, sinks=sinks, seed=window))


def test_window_and_sinks_wide_heads():
    run(need_gpu(), Case([700], [700], 8, 2, 128, window=130, sinks=5, seed=3))
    run(need_gpu(), Case([64, 700, 3], [700, 701, 500], 4, 4, 128, window=65, sinks=129, seed=4))


def test_largest_window_and_sinks():
    run(need_gpu(), Case([150], [150], 2, 1, 64, window=2 ** 31 - 1, sinks=2 ** 24, seed=5))


@pytest.mark.parametrize("size", [0.0, 1e-3, 8.0])
def test_sizes_of_scores(size):
    """Equal scores (all zero), tiny ones, and ones that leave a single key standing."""
    m = need_gpu()
    c = Case([150], [150], 2, 2, 64, seed=6)
    c.q = normal(6, 150, 2, 64, scale=size)
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    q_off, kv_off = c.off()
    o, lse = m.molora_attn_forward(q, k, v, q_off, kv_off)
    check_forward(c, o, lse)
    check_backward(c, o, lse, m.molora_attn_backward(c.do.cuda(), q, k, v, o, lse, q_off, kv_off))


def test_growing_scores():
    """Keys that grow along the sequence move the running maximum in every tile."""
    m = need_gpu()
    c = Case([520], [520], 2, 1, 64, seed=7)
    c.k = (c.k.float() * torch.linspace(0.1, 6, 520)[:, None, None]).to(torch.bfloat16)
    run(m, c)
    c.k = c.k.flip(0)
    run(m, c)


def test_scale():
    run(need_gpu(), Case([100], [100], 2, 1, 64, scale=0.5, seed=8))
    run(need_gpu(), Case([100], [100], 2, 1, 128, scale=1e-6, seed=8))


@pytest.mark.parametrize("D", [64, 128])
def test_strides(D):
    """q, k, v as parts of one buffer, heads outside tokens, a shared (broadcast) key-value row; every
    output into a wider buffer whose other values stay."""
    m = need_gpu()
    c = Case([90, 45], [90, 45], 4, 2, D, window=50, sinks=2, seed=11)
    T = 135
    one = torch.full((T, 8 * D + 8), 99.0, dtype=torch.bfloat16, device="cuda")
    q, k, v = (one[:, a * D:b * D].view(T, b - a, D) for a, b in ((0, 4), (4, 6), (6, 8)))
    q.copy_(c.q), k.copy_(c.k), v.copy_(c.v)
    q_off, kv_off = c.off()
    wide = torch.full((4, T + 3, D + 8), 7.0, dtype=torch.bfloat16, device="cuda")  # heads outside tokens
    out = wide[:, :T, :D].transpose(0, 1)
    o, lse = m.molora_attn_forward(q, k, v, q_off, kv_off, out=out, **c.kw)
    assert o is out
    check_forward(c, o, lse)
    assert (wide[:, T:] == 7).all() and (wide[:, :, D:] == 7).all() and (one[:, 8 * D:] == 99).all()
    do = c.do.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    grads = torch.full((T, 8 * D + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    dq, dk, dv = (grads[:, a * D:b * D].view(T, b - a, D) for a, b in ((0, 4), (4, 6), (6, 8)))
    got = m.molora_attn_backward(do, q, k, v, o, lse, q_off, kv_off, dq=dq, dk=dk, dv=dv, **c.kw)
    check_backward(c, o, lse, got)
    assert (grads[:, 8 * D:] == 5).all()


def test_broadcast_inputs():
    m = need_gpu()
    c = Case([70], [70], 4, 2, 64, seed=12)
    row = normal(13, 1, 1, 64)
    c.v = row.expand(70, 2, 64)
    q, k, v = c.q.cuda(), c.k.cuda(), row.cuda().expand(70, 2, 64)
    q_off, kv_off = c.off()
    o, lse = m.molora_attn_forward(q, k, v, q_off, kv_off)
    check_forward(c, o, lse)
    check_backward(c, o, lse, m.molora_attn_backward(c.do.cuda(), q, k, v, o, lse, q_off, kv_off))


def test_rows_outside_sequences():
    """Tokens before the first and behind the last sequence: never used, never written."""
    m = need_gpu()
    c = Case([60, 30], [80, 30], 4, 2, 64, seed=14)
    ro = c.oracle()[0]

    def pad(x, n):
        y = torch.full((n,) + x.shape[1:], float("nan"), dtype=x.dtype)
        y[5:5 + x.shape[0]] = x
        return y.cuda()
    q, do, k, v = pad(c.q, 120), pad(c.do, 120), pad(c.k, 130), pad(c.v, 130)
    q_off, kv_off = (x + 5 for x in c.off())
    out = torch.full((120, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 120), 3.0, device="cuda")
    m.molora_attn_forward(q, k, v, q_off, kv_off, out=out, lse=lse)
    check_forward(c, out[5:95], lse[:, 5:95])
    assert (out[:5] == 3).all() and (out[95:] == 3).all() and (lse[:, :5] == 3).all() and (lse[:, 95:] == 3).all()
    dq, dk, dv = (torch.full((n, h, 64), 3.0, dtype=torch.bfloat16, device="cuda") for n, h in ((120, 4), (130, 2), (130, 2)))
    m.molora_attn_backward(do, q, k, v, out, lse, q_off, kv_off, dq=dq, dk=dk, dv=dv)
    check_backward(c, out[5:95], lse[:, 5:95], (dq[5:95], dk[5:115], dv[5:115]))
    for t, n in ((dq, 90), (dk, 110), (dv, 110)):
        assert (t[:5] == 3).all() and (t[5 + n:] == 3).all()
    assert ro.shape[0] == 90


def test_offsets_past_the_tensors_are_limited():
    m = need_gpu()
    c = Case([64], [64], 2, 1, 64, seed=15)
    off = torch.tensor([0, 1000], dtype=torch.int32, device="cuda")
    o, lse = m.molora_attn_forward(c.q.cuda(), c.k.cuda(), c.v.cuda(), off)
    check_forward(c, o, lse)


def test_no_rows():
    m = need_gpu()
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    q = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(9, 1, 64, dtype=torch.bfloat16, device="cuda")
    kv_off = torch.tensor([0, 4, 9], dtype=torch.int32, device="cuda")
    o, lse = m.molora_attn_forward(q, k, k, off, kv_off)
    dq, dk, dv = m.molora_attn_backward(q, q, k, k, o, lse, off, kv_off,
                                        dk=torch.full_like(k, 2.0), dv=torch.full_like(k, 2.0))
    assert dq.numel() == 0 and (dk == 0).all() and (dv == 0).all()
    q9 = torch.ones(9, 2, 64, dtype=torch.bfloat16, device="cuda")
    k0 = torch.zeros(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = m.molora_attn_forward(q9, k0, k0, kv_off, off)
    assert (o == 0).all() and torch.isneginf(lse).all()
    dq, _, _ = m.molora_attn_backward(q9, q9, k0, k0, o, lse, kv_off, off, dq=torch.full_like(q9, 2.0))
    assert (dq == 0).all()


def test_rows_past_32_bits():
    """A token stride of 2^23 - 8 elements: row 300 lies 5 GB into the buffer."""
    m = need_gpu()
    c = Case([300], [300], 1, 1, 64, seed=16)
    stride = 2 ** 23 - 8
    buf = torch.empty(299 * stride + 64, dtype=torch.bfloat16, device="cuda")
    k = buf.as_strided((300, 1, 64), (stride, 64, 1))
    k.copy_(c.k)
    q, v, do = c.q.cuda(), c.v.cuda(), c.do.cuda()
    q_off, kv_off = c.off()
    o, lse = m.molora_attn_forward(q, k, v, q_off, kv_off)
    check_forward(c, o, lse)
    check_backward(c, o, lse, m.molora_attn_backward(do, q, k, v, o, lse, q_off, kv_off))
    o2 = buf.as_strided((300, 1, 64), (stride, 64, 1))
    m.molora_attn_forward(q, c.k.cuda(), v, q_off, kv_off, out=o2)
    assert torch.equal(o2.contiguous(), o)


def test_gradients_against_differences():
    """dL/dx along random directions: (L(x + h d) - L(x - h d)) / 2h of the oracle's forward."""
    m = need_gpu()
    c = Case([50, 33], [60, 33], 4, 2, 64, window=20, sinks=3, seed=17)
    _, _, got = run(m, c)
    x = [f64(c.q), f64(c.k), f64(c.v)]
    do = f64(c.do)
    r = np.random.default_rng(18)
    h = 1e-5
    for i in range(3):
        d = r.normal(size=x[i].shape)
        vals = []
        for sign in (1, -1):
            y = list(x)
            y[i] = x[i] + sign * h * d
            vals.append((O.attn(*y, c.q_off, c.kv_off, 0.125, 20, 3)[0] * do).sum())
        want, have = (vals[0] - vals[1]) / (2 * h), (f64(got[i]) * d).sum()
        # the gradient's roundings (2^-8 each, and of o in delta) along a random direction add up as a random walk
        assert abs(want - have) <= 4 * 2.0 ** -7 * np.linalg.norm(f64(got[i]) * d)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,kv_lens,window,sinks,keys,queries", [
    ([200], [200], 0, 0, [150, 199], [60]),          # later tokens
    ([300], [300], 40, 3, [100, 170], [5, 220]),     # behind the window, between sinks and window
    ([150, 90], [150, 95], 33, 0, [0, 149, 200], [149]),
    ([24], [1500], 300, 20, [600, 1490], [3]),       # keys split over workgroups
    ([1700], [1700], 200, 5, [900, 1301], [777]),    # key tiles split into chunks
    ([60], [20], 5, 0, [19], [10, 59]),              # a bad row that sees nothing
])
def test_rows_that_are_not_finite_reach_only_what_sees_them(lens, kv_lens, window, sinks, keys, queries, D):
    """NaN and infinities in tokens: whatever does not see them is as if they were not there."""
    m = need_gpu()
    c = Case(lens, kv_lens, 4, 2, D, window=window, sinks=sinks, seed=40)
    for x, rows in ((c.k, keys), (c.v, keys), (c.q, queries), (c.do, queries)):
        x[rows] = 0
    ref = c.oracle()
    q, k, v, do = (x.cuda() for x in (c.q, c.k, c.v, c.do))
    for i, j in enumerate(keys):  # in turn: only the key, only one value, both
        if i != 1:
            k[j] = float("nan")
        if i != 0:
            v[j, :, 3] = float("inf")
            v[j, :, 40:] = float("nan")
    for i, j in enumerate(queries):
        if i != 0:
            q[j] = float("nan")
        do[j, :, 7:] = float("-inf")
    q_off, kv_off = c.off()
    o, lse = m.molora_attn_forward(q, k, v, q_off, kv_off, **c.kw)
    see = np.zeros((c.q.shape[0], c.k.shape[0]), bool)
    for (a, b), (s, e) in zip(zip(c.q_off, c.q_off[1:]), zip(c.kv_off, c.kv_off[1:])):
        see[a:b, s:e] = O.visible(b - a, e - s, window, sinks)
    lost = see[:, keys].any(1)          # rows of o
    lost[queries[1:]] |= see[queries[1:]].any(1)
    held = o.cpu()
    assert not torch.isfinite(held[lost]).all(-1).any()
    held[lost], lse_h = torch.from_numpy(ref[0][lost]).to(torch.bfloat16), lse.cpu()
    lse_h[:, lost] = torch.from_numpy(ref[1][:, lost]).float()
    check_forward(c, held, lse_h)
    got = m.molora_attn_backward(do, q, k, v, o, lse, q_off, kv_off, **c.kw)
    s = 1 / math.sqrt(D)
    want, mag, wide = O.attn_backward(f64(c.do), f64(c.q), f64(c.k), f64(c.v), f64(held), f64(lse_h), c.q_off, c.kv_off, s,
                                      **c.kw)
    bad = lost.copy()
    bad[queries] |= see[queries].any(1)
    gone = see[bad].any(0)              # keys that a bad row sees
    assert (~bad).any()
    for name, g, r, a, w, out in zip(("dq", "dk", "dv"), got, want, mag, wide, (bad, gone, gone)):
        g = f64(g)
        if name != "dv":                  # (P dO may be finite where dS is not)
            assert not np.isfinite(g[out]).all(-1).any(), name
        err, bound = np.abs(g - r)[~out], (HALF * (a + np.abs(r)) + FINE * w + 1e-30)[~out]
        assert (err <= bound).all(), (name, int((~(err <= bound)).sum()))


def test_repeats_are_equal_bit_for_bit():
    m = need_gpu()
    c = Case([400, 77], [400, 77], 8, 2, 128, window=90, sinks=4, seed=19)
    a, b = run(m, c), run(m, c)
    for x, y in zip((a[0], a[1], *a[2]), (b[0], b[1], *b[2])):
        assert torch.equal(x, y)


def test_captured_training_step_replays():
    m = need_gpu()
    c = Case([200, 56], [200, 56], 4, 2, 64, seed=20)
    q, k, v, do = (x.cuda() for x in (c.q, c.k, c.v, c.do))
    q_off, kv_off = c.off()

    def step():
        o, lse = m.molora_attn_forward(q, k, v, q_off, kv_off, window=64, sinks=2)
        return (o, lse) + m.molora_attn_backward(do, q, k, v, o, lse, q_off, kv_off, window=64, sinks=2)
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step()
    g2 = torch.cuda.CUDAGraph()  # a second graph, its own workspace
    with torch.cuda.graph(g2):
        held2 = step()
    for i in range(3):
        for j, x in enumerate((q, k, v, do)):
            x.copy_(normal(100 + 10 * i + j, *x.shape).cuda())
        for t in held + held2:
            t.zero_()
        g.replay()
        g2.replay()
        torch.cuda.synchronize()
        for a, b, d in zip(held, held2, step()):
            assert torch.equal(a, d) and torch.equal(b, d)


def test_two_streams_at_once():
    m = need_gpu()
    cs = [Case([300], [300], 4, 2, 64, seed=s) for s in (21, 22)]
    ins = [[x.cuda() for x in (c.q, c.k, c.v, c.do)] for c in cs]
    off = [c.off() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    outs = []
    for (q, k, v, do), (a, b), s in zip(ins, off, streams):
        o, lse = m.molora_attn_forward(q, k, v, a, b, stream=s)
        outs.append((o, lse, m.molora_attn_backward(do, q, k, v, o, lse, a, b, stream=s)))
    torch.cuda.synchronize()
    for c, (o, lse, got) in zip(cs, outs):
        check_forward(c, o, lse)
        check_backward(c, o, lse, got)


def test_binding_refusals():
    m = need_gpu()
    q = torch.zeros(8, 2, 64, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="bfloat16"):
        m.molora_attn_forward(q.float(), q, q, off)
    with pytest.raises(ValueError, match="shape"):
        m.molora_attn_forward(q, q, q[:7], off)
    with pytest.raises(ValueError, match="contiguous"):
        m.molora_attn_forward(q.transpose(1, 2).contiguous().transpose(1, 2), q, q, off)
    with pytest.raises(ValueError, match="int32"):
        m.molora_attn_forward(q, q, q, off.long())
    with pytest.raises(ValueError):
        m.molora_attn_forward(q, q, q, off.cpu())
    with pytest.raises(m.MoloraError):
        m.molora_attn_forward(q, q, q, off, out=torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda").expand(8, 2, 64))
    with pytest.raises(m.MoloraError, match="head_dim"):
        x = torch.zeros(8, 2, 96, dtype=torch.bfloat16, device="cuda")
        m.molora_attn_forward(x, x, x, off)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,kv_lens,Hq,Hkv", [([2048], [2048], 16, 2), ([2304], [2500], 13, 1), ([1500, 3, 1300], [1500, 900, 1400], 3, 3)])
def test_long_tiles_split_among_many(lens, kv_lens, Hq, Hkv, D):
    """As many queries as keys: the long tiles are split into chunks of one length, short ones stay whole."""
    m = need_gpu()
    c = Case(lens, kv_lens, Hq, Hkv, D, seed=50)
    assert m.molora_attn_forward_workspace(c.q.cuda(), c.k.cuda(), c.off()[0]) > 0
    run(m, c)


def test_many_sequences_with_split_keys():
    """More sequences than a wave has lanes, each with few queries before many keys."""
    m = need_gpu()
    lens = [1 + i % 3 for i in range(70)]
    kv = [700 + (i * 37) % 300 for i in range(70)]
    c = Case(lens, kv, 2, 1, 64, seed=51)
    assert m.molora_attn_forward_workspace(c.q.cuda(), c.k.cuda(), c.off()[0]) > 0
    run(m, c)
