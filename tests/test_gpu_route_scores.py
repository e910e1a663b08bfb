"""Routing by scores (molora_route_scores and its backward) against the fp64 oracle.

The selection has to be the oracle's, index for index: without a bias and with one group it is the
order of the logits, else that of s + bias in 64 bits, and the inputs hold no two values nearer than
64-bit exp's error unless they are equal.  Weights: l - top is rounded once (|l - top| 2^-24 in the
exponent), exp and the division err by a few units of 2^-24, a sum of K terms by at most K more:
relative error at most (2 max|l| + K + 16) 2^-24.  Gradients: the same, relative to the sum of the
magnitudes of the terms, and twice for the product of two such scores."""
import numpy as np
import pytest
import torch

from gpu_util import dev, host, need_gpu
from oracle import decoder_ops as O

pytestmark = pytest.mark.gpu
SCORES = ["softmax", "sigmoid"]


def run(m, l, k, bias=None, score="softmax", **kw):
    idx, w = m.molora_route_scores(dev(l), k, bias=None if bias is None else dev(bias),
                                   score=m.SCORE_SIGMOID if score == "sigmoid" else m.SCORE_SOFTMAX, **kw)
    return host(idx), host(w).astype(np.float64)


def rel_bound(l):
    # a logit more than 128 below the top has a weight below 2^-126 on both sides, so larger ones do
    # not count (in fp32 the product below would overflow for them)
    fin = np.minimum(np.abs(l[np.isfinite(l)]).astype(np.float64), 128.0)
    return (2 * (fin.max() if fin.size else 0.0) + l.shape[1] + 16) * 2.0 ** -24


def check(m, l, k, **kw):
    idx, w = run(m, l, k, **kw)
    ri, rw = O.route_scores(l, k, **kw)
    np.testing.assert_array_equal(idx, ri)
    assert (np.abs(w - rw) <= rel_bound(l) * np.abs(rw) + 2.0 ** -126).all(), np.abs(w - rw).max()
    return idx, w


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("K,k,n_group,topk_group", [
    (1, 1, 1, 1), (2, 1, 1, 1), (7, 3, 1, 1), (8, 8, 1, 1), (13, 4, 1, 1), (16, 2, 1, 1), (16, 4, 4, 2), (17, 5, 1, 1),
    (24, 6, 8, 3), (30, 4, 5, 2), (32, 8, 2, 1), (33, 3, 3, 2), (48, 8, 6, 6), (63, 7, 9, 4), (64, 8, 8, 4), (64, 1, 64, 2),
    (64, 8, 16, 5), (60, 8, 60, 9)])
def test_selection_and_weights(score, K, k, n_group, topk_group):
    m = need_gpu()
    r = np.random.default_rng(K * 100 + k)
    l = (2 * r.normal(size=(203, K))).astype(np.float32)
    for bias in (None, (0.3 * r.normal(size=K)).astype(np.float32)):
        for renorm in (True, False):
            check(m, l, k, bias=bias, score=score, n_group=n_group, topk_group=topk_group, renorm=renorm, factor=1.5)


@pytest.mark.parametrize("N", [0, 1, 7, 8, 9, 31, 32, 33, 257])
def test_numbers_of_tokens_and_what_lies_behind(N):
    m = need_gpu()
    l = np.random.default_rng(N).normal(size=(N, 20)).astype(np.float32)
    idx = torch.full((N + 5, 3), 77, dtype=torch.int32, device="cuda")
    w = torch.full((N + 5, 3), 7.0, device="cuda")
    m.molora_route_scores(dev(l), 3, idx=idx[:N], w=w[:N])
    ri, rw = O.route_scores(l, 3)
    np.testing.assert_array_equal(host(idx)[:N], ri)
    assert (host(idx)[N:] == 77).all() and (host(w)[N:] == 7.0).all()
    np.testing.assert_allclose(host(w)[:N], rw, rtol=(2 * 6 + 36) * 2.0 ** -24)


@pytest.mark.parametrize("score", SCORES)
def test_equal_values_go_to_the_lowest_index(score):
    m = need_gpu()
    r = np.random.default_rng(5)
    l = r.integers(-2, 3, size=(300, 24)).astype(np.float32)  # few values: ties everywhere
    check(m, l, 5, score=score)
    bias = np.zeros(24, np.float32)
    check(m, l, 5, score=score, bias=bias, n_group=6, topk_group=3)
    check(m, np.zeros((9, 64), np.float32), 8, score=score, bias=np.zeros(64, np.float32), n_group=8, topk_group=2)


def test_decisions_nearer_than_32_bits():
    """s + bias of two adapters apart by less than fp32 keeps: the 64-bit order decides."""
    m = need_gpu()
    r = np.random.default_rng(6)
    K, N = 16, 512
    l = np.full((N, K), -3.0, np.float32)
    base = r.normal(size=N).astype(np.float32)
    up = r.integers(-3, 4, size=N)  # units in the last place
    l[:, 4] = base
    l[:, 11] = np.where(up >= 0, base + up * np.spacing(base), base - (-up) * np.spacing(base)).astype(np.float32)
    bias = np.full(K, 0.25, np.float32)
    check(m, l, 1, score="sigmoid", bias=bias)
    check(m, l, 1, score="softmax", bias=bias)
    check(m, l, 2, score="sigmoid", bias=bias, n_group=8, topk_group=1)


@pytest.mark.parametrize("score", SCORES)
def test_absent_adapters_and_extreme_values(score):
    m = need_gpu()
    r = np.random.default_rng(7)
    l = r.normal(size=(200, 21)).astype(np.float32)
    l[r.random(l.shape) < 0.6] = -np.inf
    l[r.random(l.shape) < 0.1] = np.nan
    l[3] = -np.inf
    l[4] = np.nan
    l[5] = -np.inf
    l[5, 20] = 1.0
    for kw in (dict(), dict(bias=(0.2 * r.normal(size=21)).astype(np.float32)), dict(n_group=7, topk_group=2),
               dict(renorm=False)):
        idx, w = check(m, l, 4, score=score, **kw)
        assert (idx[3] == -1).all() and (w[3] == 0).all() and (idx[4] == -1).all()
        assert idx[5].tolist() == [20, -1, -1, -1] and (w[5, 1:] == 0).all()
    big = np.zeros((4, 8), np.float32)
    big[0, 3], big[0, 6] = np.inf, np.inf
    big[1, 2] = 3e38
    big[2] = -3e38
    big[3] = [-1e4, -1e4, 0, 1, 2, 3, 4, 5]
    check(m, big, 2, score=score)
    bias = np.zeros(21, np.float32)
    bias[2], bias[3], bias[4] = np.nan, -np.inf, np.inf
    idx, _ = run(m, np.nan_to_num(l, nan=0.0, neginf=0.0), 4, bias=bias, score=score)
    ri, _ = O.route_scores(np.nan_to_num(l, nan=0.0, neginf=0.0), 4, bias=bias, score=score)
    np.testing.assert_array_equal(idx, ri)
    assert (idx != 2).all() and (idx != 3).all() and (idx == 4).any(1).all()


@pytest.mark.parametrize("K,k", [(12, 2), (32, 4), (64, 5)])
def test_chosen_scores_that_are_tiny(K, k):
    """A bias that picks adapters far below the top, sigmoid scores near the smallest numbers: the
    renormalised weights and their gradients stay those of the formula."""
    m = need_gpu()
    r = np.random.default_rng(K)
    N = 70
    low = np.arange(K) % 3 == 1
    bias = np.where(low, 4.0, 0.0).astype(np.float32)
    for score, at in (("softmax", -30.0), ("softmax", -86.0), ("softmax", -100.0), ("softmax", -120.0), ("sigmoid", -86.0),
                      ("sigmoid", -100.0)):
        l = r.normal(size=(N, K)).astype(np.float32)
        l[:, low] += at
        if low.sum() < k:
            l[:, ~low] = -np.inf
        kw = dict(bias=bias, score=score, renorm=True, factor=2.5)
        # the choice among values that differ by far less than the bias's last bit goes by index on both sides
        idx, w = run(m, l, k, **kw)
        ri, rw = O.route_scores(l, k, **kw)
        np.testing.assert_array_equal(idx, ri)
        assert (np.abs(w - rw) <= rel_bound(l) * np.abs(rw) + 2.0 ** -126).all(), (score, at)
        dw = r.normal(size=(N, k)).astype(np.float32)
        got = host(m.molora_route_scores_backward(dev(l), dev(idx.astype(np.int32)), dev(dw),
                                                  score=m.SCORE_SIGMOID if score == "sigmoid" else m.SCORE_SOFTMAX,
                                                  renorm=True, factor=2.5))
        ref, mag = O.route_scores_backward(l, idx, dw, score=score, renorm=True, factor=2.5)
        assert (np.abs(got - ref) <= 3 * rel_bound(l) * mag + 2.0 ** -120).all(), (score, at)


def test_output_of_another_operator_feeds_dispatch():
    m = need_gpu()
    l = np.random.default_rng(8).normal(size=(500, 12)).astype(np.float32)
    l[7] = -np.inf
    idx, w = m.molora_route_scores(dev(l), 3, score=m.SCORE_SIGMOID)
    counts, offsets, perm, perm_w, inv = m.molora_dispatch(idx, w, 12, 3)
    ri, _ = O.route_scores(l, 3, score="sigmoid")
    np.testing.assert_array_equal(host(counts), np.bincount(ri[ri >= 0], minlength=12))
    assert int(host(offsets)[-1]) == 499 * 3 and (host(inv).reshape(500, 3)[7] == -1).all()


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("N,K,k", [(1, 1, 1), (33, 5, 2), (64, 16, 4), (203, 17, 3), (100, 40, 8), (65, 64, 8)])
def test_backward(score, renorm, N, K, k):
    m = need_gpu()
    r = np.random.default_rng(N + K)
    l = (2 * r.normal(size=(N, K))).astype(np.float32)
    if K > 4:
        l[r.random(l.shape) < 0.2] = -np.inf
        l[0] = -np.inf
        l[N - 1, 1] = np.nan
    dw = r.normal(size=(N, k)).astype(np.float32)
    idx, _ = O.route_scores(l, k, score=score)
    if N > 40:
        idx[5, 0], idx[6, k - 1] = -1, K  # receive nothing
    got = host(m.molora_route_scores_backward(dev(l), dev(idx.astype(np.int32)), dev(dw), renorm=renorm, factor=1.5,
                                              score=m.SCORE_SIGMOID if score == "sigmoid" else m.SCORE_SOFTMAX))
    ref, mag = O.route_scores_backward(l, idx, dw, score, renorm, 1.5)
    # mag leaves sigmoid's factor 1 - s at 1, whose error is 2^-24 itself and not a part of it
    bound = 3 * rel_bound(l)
    assert (np.abs(got - ref) <= bound * mag + 2.0 ** -126).all(), (np.abs(got - ref) / (mag + 1e-30)).max()
    assert (got[~(l > -np.inf)] == 0).all()


@pytest.mark.parametrize("score", SCORES)
def test_a_single_renormalised_weight_is_constant(score):
    """k = 1 with renorm: the weight is the factor itself, whatever the logits, and the gradient exactly 0."""
    m = need_gpu()
    r = np.random.default_rng(13)
    l = (3 * r.normal(size=(400, 36))).astype(np.float32)
    idx, w = run(m, l, 1, score=score, factor=2.5)
    assert (w == 2.5).all()
    dw = r.normal(size=(400, 1)).astype(np.float32)
    got = m.molora_route_scores_backward(dev(l), dev(idx.astype(np.int32)), dev(dw), factor=2.5,
                                         score=m.SCORE_SIGMOID if score == "sigmoid" else m.SCORE_SOFTMAX)
    assert (got == 0).all()


def test_backward_against_differences():
    m = need_gpu()
    r = np.random.default_rng(11)
    l = r.normal(size=(8, 10)).astype(np.float32)
    dw = r.normal(size=(8, 3)).astype(np.float32)
    for score in SCORES:
        for renorm in (True, False):
            idx, _ = O.route_scores(l, 3, score=score, renorm=renorm)
            got = host(m.molora_route_scores_backward(
                dev(l), dev(idx.astype(np.int32)), dev(dw), renorm=renorm,
                score=m.SCORE_SIGMOID if score == "sigmoid" else m.SCORE_SOFTMAX))
            h = 1e-5
            for t in range(8):
                for e in range(10):
                    d = []
                    for sign in (1, -1):
                        x = l.astype(np.float64)
                        x[t, e] += sign * h
                        s, _ = O.scores(x[t:t + 1], score)
                        p = s[0, idx[t]]
                        d.append(((p / p.sum() if renorm else p) * dw[t]).sum())
                    assert abs((d[0] - d[1]) / (2 * h) - got[t, e]) < 1e-5


def test_captured_call_replays():
    m = need_gpu()
    r = np.random.default_rng(12)
    l, bias = torch.empty(300, 64, device="cuda"), dev(r.normal(size=64).astype(np.float32))
    idx, w = torch.empty(300, 8, dtype=torch.int32, device="cuda"), torch.empty(300, 8, device="cuda")
    dw, dl = dev(r.normal(size=(300, 8)).astype(np.float32)), torch.empty(300, 64, device="cuda")

    def step():
        m.molora_route_scores(l, 8, bias=bias, score=m.SCORE_SIGMOID, n_group=8, topk_group=3, idx=idx, w=w)
        m.molora_route_scores_backward(l, idx, dw, score=m.SCORE_SIGMOID, dlogits=dl)
    l.zero_()
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(3):
        l.copy_(dev(r.normal(size=(300, 64)).astype(np.float32)))
        g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (idx, w, dl)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (idx, w, dl)))


def test_another_stream():
    m = need_gpu()
    l = np.random.default_rng(13).normal(size=(4096, 32)).astype(np.float32)
    x = dev(l)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = [m.molora_route_scores(x, 4, stream=s) for _ in range(4)]
    outs.append(m.molora_route_scores(x, 4, stream=s.cuda_stream))
    s.synchronize()
    ri, _ = O.route_scores(l[:64], 4)
    for idx, w in outs:
        np.testing.assert_array_equal(host(idx)[:64], ri)
        assert torch.equal(w, outs[0][1])
