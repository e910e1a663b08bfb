"""Pins of the decoder operators' oracle (oracle/decoder_ops.py): hand-worked examples, closed forms,
torch's own softmax, attention and autograd, central differences, and torch's e4m3 rounding."""
import itertools
import math

import numpy as np
import pytest
import torch

from oracle import decoder_ops as O


def rng(seed):
    return np.random.default_rng([77, seed])


def test_route_hand_worked():
    # sigmoid of 0 is 1/2, of ln 3 is 3/4; the bias moves the choice, not the weight
    l = np.array([[0.0, math.log(3.0), 0.0, math.log(3.0)]])
    idx, w = O.route_scores(l, 2, score="sigmoid")
    assert idx.tolist() == [[1, 3]] and np.allclose(w, [[0.5, 0.5]])
    idx, w = O.route_scores(l, 2, bias=np.array([0.3, 0, 0, 0]), score="sigmoid", renorm=False, factor=2.0)
    assert idx.tolist() == [[0, 1]] and np.allclose(w, [[1.0, 1.5]])
    # ties go to the lowest index; groups of two: marks 5/4, 5/4, so group 0 alone
    idx, _ = O.route_scores(l, 2, score="sigmoid", n_group=2, topk_group=1)
    assert idx.tolist() == [[0, 1]]


def test_route_softmax_is_torch_softmax():
    l = rng(1).normal(size=(20, 12)) * 3
    idx, w = O.route_scores(l, 12, renorm=False)
    assert (idx == np.arange(12)).all()
    assert np.allclose(w, torch.softmax(torch.from_numpy(l), -1).numpy(), rtol=1e-14)
    idx, w = O.route_scores(l, 5)
    top = torch.topk(torch.from_numpy(l), 5).indices.sort(-1).values.numpy()
    assert (idx == top).all() and np.allclose(w.sum(1), 1.0)


def test_route_groups_against_brute_force():
    r = rng(2)
    for _ in range(50):
        l, b = np.round(r.normal(size=(1, 8)), 1), np.round(r.normal(size=8) * 0.3, 1)
        idx, _ = O.route_scores(l, 3, bias=b, score="sigmoid", n_group=4, topk_group=2)
        c = 1 / (1 + np.exp(-l[0])) + b
        best = max(itertools.combinations(range(4), 2), key=lambda gs: (sum(c[2 * g] + c[2 * g + 1] for g in gs),
                                                                        [-g for g in gs]))
        pool = [e for e in range(8) if e // 2 in best]
        pick = max(itertools.combinations(pool, 3), key=lambda es: (sum(c[list(es)]), [-e for e in es]))
        assert idx[0].tolist() == list(pick)


def test_route_absent():
    l = np.array([[-np.inf, 1.0, np.nan, -np.inf], [-np.inf] * 4, [np.inf, np.inf, 0.0, 1.0]])
    idx, w = O.route_scores(l, 2)
    assert idx.tolist() == [[1, -1], [-1, -1], [0, 1]]
    assert w.tolist() == [[1.0, 0.0], [0.0, 0.0], [0.5, 0.5]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_against_autograd_and_differences(score, renorm):
    r = rng(3)
    l, dw = r.normal(size=(6, 9)), r.normal(size=(6, 3))
    l[2, 4] = -np.inf
    idx, _ = O.route_scores(l, 3, score=score, renorm=renorm, factor=1.7)
    got, mag = O.route_scores_backward(l, idx, dw, score, renorm, 1.7)
    t = torch.from_numpy(l).requires_grad_(True)
    s = torch.softmax(t, -1) if score == "softmax" else torch.sigmoid(t)
    p = s.gather(1, torch.from_numpy(idx))
    w = 1.7 * (p / p.sum(-1, keepdim=True) if renorm else p)
    ref, = torch.autograd.grad((w * torch.from_numpy(dw)).sum(), t)
    assert np.allclose(got, np.nan_to_num(ref.numpy()), atol=1e-12)
    assert (np.abs(got) <= mag + 1e-15).all()
    h = 1e-6
    for e in range(9):
        if not np.isfinite(l[0, e]):
            continue
        up, dn = l.copy(), l.copy()
        up[0, e] += h
        dn[0, e] -= h
        d = [(O.route_scores(x, 3, score=score, renorm=renorm, factor=1.7)[1][0] * dw[0]).sum() for x in (up, dn)]
        assert abs((d[0] - d[1]) / (2 * h) - got[0, e]) < 1e-7


def test_visible_by_words():
    see = O.visible(3, 5, 2, 1)  # positions 2, 3, 4; the last two keys, and key 0
    assert see.astype(int).tolist() == [[1, 1, 1, 0, 0], [1, 0, 1, 1, 0], [1, 0, 0, 1, 1]]
    assert O.visible(3, 1, 0, 0).astype(int).tolist() == [[0], [0], [1]]
    assert O.visible(2, 4, 1, 0).astype(int).tolist() == [[0, 0, 1, 0], [0, 0, 0, 1]]
    assert (O.visible(6, 6, 6, 0) == O.visible(6, 6, 0, 0)).all()


@pytest.mark.parametrize("window,sinks,Lk", [(0, 0, 7), (0, 0, 12), (3, 0, 12), (3, 2, 12), (4, 20, 9)])
def test_attention_against_torch(window, sinks, Lk):
    r = rng(4)
    q, k, v, do = (r.normal(size=s) for s in ((7, 4, 16), (Lk, 2, 16), (Lk, 2, 16), (7, 4, 16)))
    see = torch.from_numpy(O.visible(7, Lk, window, sinks))
    t = [torch.from_numpy(x).requires_grad_(True) for x in (q, k, v)]
    kk, vv = (x.repeat_interleave(2, 1).transpose(0, 1) for x in t[1:])
    ref = torch.nn.functional.scaled_dot_product_attention(t[0].transpose(0, 1), kk, vv, attn_mask=see).transpose(0, 1)
    off = [np.array([0, 7]), np.array([0, Lk])]
    o, lse, mag = O.attn(q, k, v, *off, 0.25, window, sinks)
    assert np.allclose(o, ref.detach().numpy(), atol=1e-12) and (np.abs(o) <= mag + 1e-15).all()
    z = 0.25 * torch.einsum("qhd,hkd->hqk", t[0], kk.detach()).masked_fill(~see, -math.inf)
    assert np.allclose(lse, torch.logsumexp(z, -1).detach().numpy(), atol=1e-12)
    grads = torch.autograd.grad((ref * torch.from_numpy(do)).sum(), t)
    got, m, wide = O.attn_backward(do, q, k, v, o, lse, *off, 0.25, window, sinks)
    for g, x, a, b in zip(grads, got, m, wide):
        assert np.allclose(x, g.numpy(), atol=1e-12)
        assert (np.abs(x) <= a + 1e-15).all() and (a <= b + 1e-15).all()


def test_attention_empty_rows_and_sequences():
    r = rng(5)
    q, k, v = r.normal(size=(5, 1, 4)), r.normal(size=(3, 1, 4)), r.normal(size=(3, 1, 4))
    q_off, kv_off = np.array([0, 0, 3, 5]), np.array([0, 1, 2, 3])  # no query; 3 queries of 1 key; 2 of 1
    o, lse, _ = O.attn(q, k, v, q_off, kv_off, 0.5)
    assert (o[[0, 1, 3]] == 0).all() and np.isneginf(lse[0, [0, 1, 3]]).all()
    assert np.allclose(o[2, 0], v[1, 0]) and np.allclose(o[4, 0], v[2, 0])
    g, _, _ = O.attn_backward(np.ones_like(q), q, k, v, o, lse, q_off, kv_off, 0.5)
    assert (g[0] == 0).all() and (g[1] == 0).all() and (g[2][0] == 0).all() and np.allclose(g[2][1:], 1.0)


def test_attention_gradient_against_differences():
    r = rng(6)
    q, k, v, do = (r.normal(size=(5, 2, 4)) for _ in range(4))
    off = np.array([0, 2, 5])
    o, lse, _ = O.attn(q, k, v, off, off, 0.5, 2, 1)
    got, _, _ = O.attn_backward(do, q, k, v, o, lse, off, off, 0.5, 2, 1)
    h = 1e-6
    for i, x in enumerate((q, k, v)):
        for at in ((0, 0, 1), (3, 1, 2), (4, 0, 3)):
            d = []
            for sign in (1, -1):
                y = [q.copy(), k.copy(), v.copy()]
                y[i][at] += sign * h
                d.append((O.attn(*y, off, off, 0.5, 2, 1)[0] * do).sum())
            assert abs((d[0] - d[1]) / (2 * h) - got[i][at]) < 1e-7


def test_decode_is_the_last_row_of_attention():
    r = rng(7)
    page, n = 4, 11
    k, v, q = r.normal(size=(n, 2, 8)), r.normal(size=(n, 2, 8)), r.normal(size=(1, 4, 8))
    kc, vc = np.zeros((6, 2, page, 8)), np.zeros((6, 2, page, 8))
    table = np.array([[5, 0, 3]])
    for j in range(n):
        p, row = O.place(table, page, 0, j, 6)
        kc[p, :, row], vc[p, :, row] = k[j], v[j]
    for window, sinks in ((0, 0), (3, 0), (3, 2)):
        o, lse, _ = O.decode(q, kc, vc, table, np.array([n]), 0.3, window, sinks)
        ro, rl, _ = O.attn(q, k, v, np.array([0, 1]), np.array([0, n]), 0.3, window, sinks)
        assert np.allclose(o, ro) and np.allclose(lse[0], rl[:, 0])
    gone = table.copy()
    gone[0, 1] = -1  # positions 4..7 are not there
    o, _, _ = O.decode(q, kc, vc, gone, np.array([n]), 0.3)
    keep = [0, 1, 2, 3, 8, 9, 10]
    ro, _, _ = O.attn(q, k[keep], v[keep], np.array([0, 1]), np.array([0, 7]), 0.3)
    assert np.allclose(o, ro)


def test_e4m3_rounding_is_torchs():
    x = np.concatenate([rng(8).normal(size=(40, 16)) * 10.0 ** rng(9).integers(-6, 6, size=(40, 1)),
                        np.zeros((1, 16)), np.linspace(-448, 448, 16)[None]])
    x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    q, byte = O.e4m3_rows(x)
    y = torch.from_numpy(x / 2.0 ** (byte[:, None] - 127.0))
    assert np.array_equal(q, y.to(torch.float32).to(torch.float8_e4m3fn).double().numpy())
    big = np.abs(q).max(1)
    assert ((big >= 448 / 2) | (byte == 15)).all() and (big <= 448).all() and byte[-2] == 15 and byte[-1] == 127
