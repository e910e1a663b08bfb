"""fp64 oracle of the decoder's operators: routing by scores, causal attention with a window and
sink tokens and its gradients, the paged cache and the attention over it.

Written from the formulas, one token, head or sequence at a time, in NumPy float64.  Each attention
function also returns the sums of magnitudes that a rounding bound needs (``*_mag``)."""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


# ------------------------------------------------------------------------------- routing by scores

def scores(logits, score):
    """Score of every adapter; absent ones (NaN or -inf) 0, +inf as the largest finite fp32."""
    l = np.minimum(np.asarray(logits, np.float64), np.finfo(np.float32).max)
    here = ~np.isnan(l) & (l > -np.inf)
    s = np.zeros_like(l)
    for t in range(l.shape[0]):
        a = here[t]
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                s[t, a] = 1.0 / (1.0 + np.exp(-l[t, a]))
        elif a.any():
            e = np.exp(l[t, a] - l[t, a].max())
            s[t, a] = e / e.sum()
    return s, here


def route_scores(logits, k, bias=None, score="softmax", n_group=1, topk_group=1, renorm=True, factor=1.0):
    """(idx [N][k], w [N][k]): the k largest s + bias of the kept groups, ascending, -1 and 0 where nothing is left."""
    N, K = logits.shape
    s, here = scores(logits, score)
    b = np.zeros(K) if bias is None else np.asarray(bias, np.float64)
    can = here & ~np.isnan(b) & (b > -np.inf)
    idx, w = np.full((N, k), -1, np.int64), np.zeros((N, k))
    gs = K // n_group
    for t in range(N):
        if bias is None and n_group == 1:
            c = np.minimum(np.asarray(logits[t], np.float64), np.finfo(np.float32).max)
        else:
            with np.errstate(invalid="ignore"):
                c = s[t] + b
        marks = []
        for g in range(n_group):
            best = sorted((c[e] for e in range(g * gs, (g + 1) * gs) if can[t, e]), reverse=True)[:2]
            marks.append(sum(best) if best else -np.inf)
        order = sorted((g for g in range(n_group) if marks[g] > -np.inf), key=lambda g: (-marks[g], g))
        kept = set(order[:topk_group])
        pool = sorted((e for e in range(K) if can[t, e] and e // gs in kept), key=lambda e: (-c[e], e))
        chosen = sorted(pool[:k])
        total = sum(s[t, e] for e in chosen)
        for i, e in enumerate(chosen):
            idx[t, i] = e
            w[t, i] = factor * (s[t, e] / total if renorm and total > 0 else 0.0 if renorm else s[t, e])
    return idx, w


def route_scores_backward(logits, idx, dw, score="softmax", renorm=True, factor=1.0):
    """dL/dlogits by the chain rule, and the sums of magnitudes of its terms."""
    N, K = logits.shape
    s, here = scores(logits, score)
    out, mag = np.zeros((N, K)), np.zeros((N, K))
    for t in range(N):
        sel = [(int(e), float(dw[t, i])) for i, e in enumerate(idx[t]) if 0 <= e < K]
        total = sum(s[t, e] for e, _ in sel)
        g, gm = np.zeros(K), np.zeros(K)
        dot = sum(factor * d * s[t, e] for e, d in sel)
        dotm = sum(abs(factor * d) * s[t, e] for e, d in sel)
        for e, d in sel:
            if renorm:
                g[e] = (factor * d - dot / total) / total if total > 0 else 0.0
                gm[e] = (abs(factor * d) + dotm / total) / total if total > 0 else 0.0
            else:
                g[e], gm[e] = factor * d, abs(factor * d)
        if score == "sigmoid":
            out[t], mag[t] = s[t] * (1 - s[t]) * g, s[t] * gm
        else:
            out[t] = s[t] * (g - (s[t] * g).sum())
            mag[t] = s[t] * (gm + (s[t] * gm).sum())
        out[t, ~here[t]] = 0.0
    return out, mag


# ------------------------------------------------------------------------------- attention

def visible(Lq, Lk, window, sinks):
    """[Lq][Lk]: query i stands at position i + Lk - Lq."""
    see = np.zeros((Lq, Lk), bool)
    for i in range(Lq):
        p = i + Lk - Lq
        if p < 0:
            continue
        see[i, :p + 1] = True
        if window:
            see[i, :max(p - window + 1, 0)] = False
            see[i, :min(sinks, p + 1)] = True
    return see


def _weights(q, k, see, scale):
    z = np.where(see, scale * (q @ k.T), -np.inf)
    top = z.max(1, initial=-np.inf)
    p = np.exp(z - np.where(np.isfinite(top), top, 0.0)[:, None])
    p[~see] = 0.0
    l = p.sum(1)
    with np.errstate(divide="ignore"):
        lse = np.where(l > 0, np.where(np.isfinite(top), top, 0.0) + np.log(l), -np.inf)
    return p / np.where(l > 0, l, 1.0)[:, None], lse


def attn(q, k, v, q_off, kv_off, scale, window=0, sinks=0):
    """o [Tq][Hq][D], lse [Hq][Tq], and sum_j p_j |v_j|; rows outside every sequence stay 0."""
    Tq, Hq, D = q.shape
    g = Hq // k.shape[1]
    o, mag, lse = np.zeros(q.shape), np.zeros(q.shape), np.zeros((Hq, Tq))
    for b in range(len(q_off) - 1):
        a, c = slice(q_off[b], q_off[b + 1]), slice(kv_off[b], kv_off[b + 1])
        see = visible(a.stop - a.start, c.stop - c.start, window, sinks)
        for h in range(Hq):
            p, lse[h, a] = _weights(q[a, h], k[c, h // g], see, scale)
            o[a, h] = p @ v[c, h // g]
            mag[a, h] = p @ np.abs(v[c, h // g])
    return o, lse, mag


def attn_backward(dout, q, k, v, o, lse, q_off, kv_off, scale, window=0, sinks=0):
    """dq, dk, dv from the forward's o and lse, and for each (rounding, cancelling): the sums of
    magnitudes of its terms, and those of the differences dP - delta written out."""
    Hq, g = q.shape[1], q.shape[1] // k.shape[1]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    mag = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)]
    wide = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)]
    for b in range(len(q_off) - 1):
        a, c = slice(q_off[b], q_off[b + 1]), slice(kv_off[b], kv_off[b + 1])
        see = visible(a.stop - a.start, c.stop - c.start, window, sinks)
        for h in range(Hq):
            kh = h // g
            z = scale * (q[a, h] @ k[c, kh].T)
            with np.errstate(invalid="ignore", over="ignore"):
                p = np.where(see, np.exp(z - lse[h, a][:, None]), 0.0)
            delta = (dout[a, h] * o[a, h]).sum(1)[:, None]
            dp = dout[a, h] @ v[c, kh].T
            ds = p * (dp - delta)
            dpm = np.abs(dout[a, h]) @ np.abs(v[c, kh]).T + (np.abs(dout[a, h]) * np.abs(o[a, h])).sum(1)[:, None]
            dsm, dsw = np.abs(ds), p * dpm
            dq[a, h] = scale * (ds @ k[c, kh])
            dk[c, kh] += scale * (ds.T @ q[a, h])
            dv[c, kh] += p.T @ dout[a, h]
            mag[0][a, h] = scale * (dsm @ np.abs(k[c, kh]))
            mag[1][c, kh] += scale * (dsm.T @ np.abs(q[a, h]))
            mag[2][c, kh] += p.T @ np.abs(dout[a, h])
            wide[0][a, h] = scale * (dsw @ np.abs(k[c, kh]))
            wide[1][c, kh] += scale * (dsw.T @ np.abs(q[a, h]))
            wide[2][c, kh] += p.T @ np.abs(dout[a, h])
    return (dq, dk, dv), mag, wide


# ------------------------------------------------------------------------------- paged cache

def e4m3_rows(x):
    """Rows of finite values as (e4m3 values, scale bytes): value * 2^(byte - 127) stands for x."""
    x = np.asarray(x, np.float64)
    q, byte = np.zeros_like(x), np.zeros(x.shape[:-1], np.int64)
    for at in np.ndindex(*x.shape[:-1]):
        big = np.abs(x[at]).max()
        n = -112
        while big > E4M3_MAX * 2.0 ** n:
            n += 1
        y = x[at] / 2.0 ** n
        with np.errstate(divide="ignore"):
            e = np.maximum(np.floor(np.log2(np.abs(y))), -6.0)  # below 2^-6 the steps stay 2^-9
        step = 2.0 ** (np.where(np.isfinite(e), e, -6.0) - 3)
        q[at] = np.clip(np.round(y / step) * step, -E4M3_MAX, E4M3_MAX)  # np.round: half to even
        byte[at] = n + 127
    return q, byte


def place(table, page_size, b, j, n_pages):
    """(page, row) of position j of sequence b, or None."""
    if j < 0 or j // page_size >= table.shape[1]:
        return None
    p = int(table[b, j // page_size])
    return (p, j % page_size) if 0 <= p < n_pages else None


def decode(q, kc, vc, table, lens, scale, window=0, sinks=0):
    """o [B][Hq][D], lse [B][Hq], sum p |v|; kc and vc the cache's values [n_pages][Hkv][page][D]."""
    B, Hq, D = q.shape
    n_pages, Hkv, page, _ = kc.shape
    g = Hq // Hkv
    o, mag, lse = np.zeros(q.shape), np.zeros(q.shape), np.full((B, Hq), -np.inf)
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * page)
        at = [place(table, page, b, j, n_pages) for j in range(n) if not window or j >= n - window or j < sinks]
        at = [x for x in at if x is not None]
        if not at:
            continue
        pg, row = np.array([x[0] for x in at]), np.array([x[1] for x in at])
        for h in range(Hq):
            k, v = kc[pg, h // g, row], vc[pg, h // g, row]
            p, l = _weights(q[b, h][None], k, np.ones((1, len(at)), bool), scale)
            o[b, h], lse[b, h], mag[b, h] = (p @ v)[0], l[0], (p @ np.abs(v))[0]
    return o, lse, mag
