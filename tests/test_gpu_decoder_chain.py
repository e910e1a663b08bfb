"""The decoder's operators in a row, as a layer uses them: scores -> dispatch -> q / k / v adapters ->
attention -> its gradient -> the adapters' gradient -> the scores' gradient, captured into one graph,
against the same chain in fp64.

Along it values are rounded to bf16 eight times (q, k, v; P; o; dS and P again; dq, dk, dv), each time by
at most 2^-8 of their size, so gradients are held to 8 x 2^-8 = 2^-5 in the Frobenius norm; a wrong
index, scale or mask moves them by their own size."""
import numpy as np
import pytest
import torch

from gpu_util import dev, dev_bf16, f64, host, need_gpu
from oracle import apply, apply_backward, dispatch
from oracle import decoder_ops as O

pytestmark = pytest.mark.gpu
BAR = 2.0 ** -5


def bits(r, *shape, scale=1.0):
    return torch.from_numpy((scale * r.standard_normal(shape)).astype(np.float32)).to(torch.bfloat16).view(
        torch.int16).numpy().view(np.uint16)


@pytest.mark.parametrize("score,renorm,groups,window", [("sigmoid", True, 2, 0), ("softmax", False, 1, 20)])
def test_training_chain(score, renorm, groups, window):
    m = need_gpu()
    r = np.random.default_rng([91, groups])
    lens, N, d, K, rank, k, H, D = [70, 0, 33], 103, 256, 8, 16, 2, 2, 128
    off = np.array([0, 70, 70, 103], np.int32)
    x, y0, do = bits(r, N, d), [bits(r, N, d) for _ in range(3)], bits(r, N, H, D)
    A = [bits(r, K, d, rank, scale=d ** -0.5) for _ in range(3)]
    B = [bits(r, K, rank, d, scale=rank ** -0.5) for _ in range(3)]
    logits = r.standard_normal((N, K)).astype(np.float32)
    logits[5] = -np.inf  # a token without adapters
    bias = (0.2 * r.standard_normal(K)).astype(np.float32)
    code = m.SCORE_SIGMOID if score == "sigmoid" else m.SCORE_SOFTMAX
    kw = dict(score=code, renorm=renorm)
    pairs = [(dev_bf16(a), dev_bf16(b)) for a, b in zip(A, B)]
    hs, hst = m.molora_hotset_init(pairs, 0.5), m.molora_hotset_init_transposed(pairs, 0.5)
    xd, y0d, dod, ld, bd, offd = dev_bf16(x), [dev_bf16(b) for b in y0], dev_bf16(do), dev(logits), dev(bias), dev(off)

    def step():
        idx, w = m.molora_route_scores(ld, k, bias=bd, n_group=groups, topk_group=1, **kw)
        _, offsets, perm, perm_w, inv = m.molora_dispatch(idx, w, K, k)
        route = (offsets, perm, perm_w, inv)
        q, kk, v = m.molora_apply_multi(hs, [xd] * 3, y0d, *route, k=k, y_dtype=torch.bfloat16)
        rows = [t.view(N, H, D) for t in (q, kk, v)]
        o, lse = m.molora_attn_forward(*rows, offd, window=window, sinks=3)
        grads = m.molora_attn_backward(dod, *rows, o, lse, offd, window=window, sinks=3)
        dw, dA = None, []
        for t, g in enumerate(grads):
            _, da, _, dwt = m.molora_backward(hs, hst, xd, g.view(N, d), *route, k=k, target=t, want=("dA", "dw"))
            dw = dwt if dw is None else dw + dwt
            dA.append(da)
        dl = m.molora_route_scores_backward(ld, idx, dw.view(N, k), **kw)
        return idx, w, o, dl, dA
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step()
    for _ in range(2):
        for t in (held[2], held[3]):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        for a, b in zip((*held[:4], *held[4]), (*eager[:4], *eager[4])):
            assert torch.equal(a, b)

    idx, w, o, dl, dA = eager
    ri, rw = O.route_scores(logits, k, bias=bias, score=score, n_group=groups, topk_group=1, renorm=renorm)
    np.testing.assert_array_equal(host(idx), ri)
    _, offsets, perm, perm_w, _ = dispatch(ri, rw, K)
    qkv = [apply(f64(y0[t]), f64(x), f64(A[t]), f64(B[t]), 0.5, perm, perm_w, offsets, k).reshape(N, H, D) for t in range(3)]
    ro, rl, _ = O.attn(*qkv, off, off, D ** -0.5, window, 3)
    assert np.linalg.norm(host(o) - ro) <= BAR * np.linalg.norm(ro)
    rg, _, _ = O.attn_backward(f64(do), *qkv, ro, rl, off, off, D ** -0.5, window, 3)
    rdw = np.zeros(N * k)
    for t in range(3):
        _, rA, _, dwt = apply_backward(f64(x), rg[t].reshape(N, d), f64(A[t]), f64(B[t]), 0.5, perm, perm_w, offsets, k)
        rdw += dwt
        assert np.linalg.norm(host(dA[t]) - rA) <= BAR * np.linalg.norm(rA)
    rdl, _ = O.route_scores_backward(logits, ri, rdw.reshape(N, k), score, renorm)
    assert np.linalg.norm(host(dl) - rdl) <= BAR * np.linalg.norm(rdl)
    assert (host(dl)[5] == 0).all()
    hs.close()
    hst.close()


def test_serving_chain():
    """Route, dispatch, q / k / v adapters, append and attend for single tokens: the last rows of the same
    chain over whole sequences."""
    m = need_gpu()
    r = np.random.default_rng(92)
    lens, d, K, rank, k, H, D = [40, 3, 18], 256, 4, 16, 2, 2, 128
    N = sum(lens)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    x, y0 = bits(r, N, d), [bits(r, N, d) for _ in range(3)]
    A = [bits(r, K, d, rank, scale=d ** -0.5) for _ in range(3)]
    B = [bits(r, K, rank, d, scale=rank ** -0.5) for _ in range(3)]
    logits = r.standard_normal((N, K)).astype(np.float32)
    hs = m.molora_hotset_init([(dev_bf16(a), dev_bf16(b)) for a, b in zip(A, B)], 0.5)

    def project(rows):
        idx, w = m.molora_route_scores(dev(logits[rows]), k, score=m.SCORE_SIGMOID)
        _, *route = m.molora_dispatch(idx, w, K, k)
        out = m.molora_apply_multi(hs, [dev_bf16(x[rows])] * 3, [dev_bf16(b[rows]) for b in y0], *route, k=k, y_dtype=torch.bfloat16)
        return [t.view(-1, H, D) for t in out]
    whole = project(np.arange(N))
    o, lse = m.molora_attn_forward(*whole, dev(off), window=12, sinks=2)
    cache = m.KvCache.empty(12, H, 16, D)
    table = torch.tensor([[7, 1, 4], [0, -1, -1], [3, 9, -1]], dtype=torch.int32, device="cuda")
    first = np.concatenate([np.arange(off[b], off[b + 1] - 1) for b in range(3)])
    foff = np.concatenate([[0], np.cumsum([n - 1 for n in lens])]).astype(np.int32)
    _, fk, fv = project(first)
    m.molora_kv_append(cache, fk, fv, dev(foff), table, dev(np.array([n - 1 for n in lens], np.int32)))
    last = off[1:] - 1
    q, nk, nv = project(last)
    L = dev(np.array(lens, np.int32))
    m.molora_kv_append(cache, nk, nv, None, table, L)
    got, got_lse = m.molora_attn_decode(q, cache, table, L, window=12, sinks=2)
    # the projections' paths differ with the batch (bf16 results one step apart at most: 2^-7 of a value)
    assert (got.float() - o[last].float()).norm() <= 2.0 ** -6 * o[last].float().norm()
    assert (got_lse - lse[:, last].t()).abs().max() <= 2.0 ** -4
    hs.close()
