"""Cases and plain forms of the decoder's operators: routing by scores, causal attention with a
window and sink tokens (forward and backward), the paged key-value cache and the attention of one
new token over it.

`run` computes a case either with the framework's entry points (`own` true) or in plain torch
operations, in 32 bits (64 for the routing decision, where a rounding would pick another adapter).
`exact` is the same from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
SOFTMAX, SIGMOID = "softmax", "sigmoid"


# ------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # routing of one decode step: 256 sequences, top-2 of 16 adapters (the decode stack's gate)
        {"name": "route decode step", "kind": "route", "N": 256, "K": 16, "k": 2, "score": SOFTMAX, "bias": False,
         "groups": 1, "keep": 1, "renorm": True, "factor": 1.0, "absent": 0.0},
        # routing of a full batch over a full hot set: balanced sigmoid gate, adapters in groups, a few not loaded
        {"name": "route full batch", "kind": "route", "N": 16384, "K": 64, "k": 8, "score": SIGMOID, "bias": True,
         "groups": 8, "keep": 4, "renorm": True, "factor": 2.5, "absent": 0.03},
        # the gate's gradient at the same batch, softmax over every adapter
        {"name": "route grad", "kind": "route_grad", "N": 16384, "K": 64, "k": 4, "score": SOFTMAX, "bias": False,
         "groups": 1, "keep": 1, "renorm": False, "factor": 1.0, "absent": 0.0},
        # a mixed batch of prompts of up to 512 tokens (one of them empty), the decoder's 16 heads of 128
        {"name": "prompt batch", "kind": "attn", "seqs": 16, "len": 512, "past": 0, "ragged": True, "Hq": 16, "Hkv": 16,
         "D": 128, "window": 0, "sinks": 0},
        # one long prompt, grouped heads
        {"name": "long prompt", "kind": "attn", "seqs": 1, "len": 8192, "past": 0, "ragged": False, "Hq": 32, "Hkv": 8,
         "D": 128, "window": 0, "sinks": 0},
        # training on packed sequences of up to 2048 tokens
        {"name": "train batch", "kind": "attn_grad", "seqs": 8, "len": 2048, "past": 0, "ragged": True, "Hq": 16,
         "Hkv": 16, "D": 128, "window": 0, "sinks": 0},
        # training on one long sequence with a window of 1024 and 16 first tokens that stay visible
        {"name": "train long window", "kind": "attn_grad", "seqs": 1, "len": 8192, "past": 0, "ragged": False, "Hq": 32,
         "Hkv": 8, "D": 64, "window": 1024, "sinks": 16},
        # one user, a long context of odd length
        {"name": "decode one", "kind": "decode", "seqs": 1, "len": 32771, "ragged": False, "Hq": 32, "Hkv": 8, "D": 128,
         "window": 0, "sinks": 0, "page": 64, "cache": "bf16"},
        # serving 64 users with contexts of up to 8192 tokens, small pages
        {"name": "decode batch", "kind": "decode", "seqs": 64, "len": 8192, "ragged": True, "Hq": 32, "Hkv": 8, "D": 128,
         "window": 0, "sinks": 0, "page": 16, "cache": "bf16"},
        # 256 users, 8-bit cache, window with sinks: the pages between them are freed
        {"name": "decode 8 bit window", "kind": "decode", "seqs": 256, "len": 4096, "ragged": True, "Hq": 16, "Hkv": 16,
         "D": 128, "window": 2048, "sinks": 4, "page": 32, "cache": "e4m3"},
        # the new tokens of a decode step into an 8-bit cache
        {"name": "append step", "kind": "append", "seqs": 256, "new": 1, "past": 700, "ragged": True, "Hkv": 8, "D": 128,
         "page": 32, "cache": "e4m3"},
        # prompts into a 16-bit cache
        {"name": "append prompts", "kind": "append", "seqs": 16, "new": 2048, "past": 0, "ragged": True, "Hkv": 8,
         "D": 128, "page": 16, "cache": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["route", "route_grad", "attn", "attn_grad", "decode", "append"])
    if kind in ("route", "route_grad"):
        group = rng.choice([1, 1, 2, 4, 8])
        size = rng.randint(1 if group == 1 else 2, 64 // group)
        K = max(2, group * size)
        group = group if K == group * size else 1
        keep = rng.randint(1, group)
        k = rng.randint(1, min(8, max(1, keep * (K // group))))
        return {"kind": kind, "N": _log(rng, 1, 16384), "K": K, "k": k, "score": rng.choice([SOFTMAX, SIGMOID]),
                "bias": rng.random() < 0.5, "groups": group, "keep": keep, "renorm": rng.random() < 0.5,
                "factor": rng.choice([1.0, 2.5]), "absent": rng.choice([0.0, 0.05, 0.4])}
    Hkv = rng.choice([1, 2, 4, 8, 16])
    Hq = Hkv * rng.choice([g for g in (1, 2, 3, 4, 8, 16) if g * Hkv <= 32])
    D = rng.choice([64, 128])
    window = rng.choice([0, 0, _log(rng, 1, 2048)])
    sinks = rng.choice([0, rng.randint(1, 70)]) if window else 0
    if kind in ("attn", "attn_grad"):
        seqs = _log(rng, 1, 16)
        most = math.sqrt(8192.0 * 8192 * 32 / 2 / (seqs * Hq))
        n = _log(rng, 1, min(8192, most))
        past = rng.choice([0, _log(rng, 1, max(1, int(most) - n) or 1)]) if n < most - 1 else 0
        return {"kind": kind, "seqs": seqs, "len": n, "past": past, "ragged": seqs > 1, "Hq": Hq, "Hkv": Hkv, "D": D,
                "window": window, "sinks": sinks}
    cache = rng.choice(["bf16", "e4m3"])
    page = rng.choice([16, 32, 64, 128])
    if kind == "decode":
        seqs = _log(rng, 1, 256)
        n = _log(rng, 1, min(32768, 8192 * 64 * 4 // (seqs * Hkv)))
        return {"kind": kind, "seqs": seqs, "len": n, "ragged": seqs > 1, "Hq": Hq, "Hkv": Hkv, "D": D, "window": window,
                "sinks": sinks, "page": page, "cache": cache}
    seqs = _log(rng, 1, 256)
    return {"kind": kind, "seqs": seqs, "new": _log(rng, 1, max(1, 16384 // seqs)), "past": rng.choice([0, rng.randint(1, 700)]),
            "ragged": seqs > 1, "Hkv": Hkv, "D": D, "page": page, "cache": cache}


def _lengths(n, seqs, ragged, least=1):
    """Lengths spread over [least, n], the first one n; of four or more sequences one is empty."""
    if not ragged:
        return [n] * seqs
    got = [n] + [max(least, int(n * ((0.5 + 0.6180339887 * i) % 1.0))) for i in range(1, seqs)]
    if seqs >= 4:
        got[2] = 0
    return got


def _pairs(q_len, kv_len, window, sinks):
    """Visible (query, key) pairs of one causal sequence whose last query sees its last key."""
    total = 0
    first = kv_len - q_len
    if not window:
        lo, hi = max(first, 0), kv_len - 1  # positions
        return (hi + 1) * (hi + 2) // 2 - lo * (lo + 1) // 2 if kv_len and q_len else 0
    for p in range(max(first, 0), kv_len):
        start = max(0, p - window + 1)
        total += p + 1 - start + min(sinks, start)
    return total


def _attn_lengths(c):
    q = _lengths(c["len"], c["seqs"], c["ragged"])
    return q, [n + c["past"] if n else 0 for n in q]


def work(case):
    c = case
    kind = c["kind"]
    if kind == "route":
        return {"bytes": c["N"] * (4 * c["K"] + 8 * c["k"]) + 4 * c["K"] * c["bias"], "flops": c["N"] * c["K"] * 10}
    if kind == "route_grad":
        return {"bytes": c["N"] * (8 * c["K"] + 8 * c["k"]), "flops": c["N"] * c["K"] * 10}
    if kind in ("attn", "attn_grad"):
        ql, kl = _attn_lengths(c)
        tq, tk = sum(ql), sum(kl)
        pairs = sum(_pairs(a, b, c["window"], c["sinks"]) for a, b in zip(ql, kl))
        q, kv = 2 * tq * c["Hq"] * c["D"], 4 * tk * c["Hkv"] * c["D"]
        if kind == "attn":
            return {"bytes": 2 * q + kv + 4 * tq * c["Hq"], "flops": 4 * pairs * c["Hq"] * c["D"]}
        return {"bytes": 4 * q + 2 * kv + 4 * tq * c["Hq"], "flops": 10 * pairs * c["Hq"] * c["D"]}
    if kind == "decode":
        keys = sum(_pairs(1, n, c["window"], c["sinks"]) for n in _lengths(c["len"], c["seqs"], c["ragged"]) if n)
        row = 2 * (2 * c["D"] if c["cache"] == "bf16" else c["D"] + 1)
        return {"bytes": keys * c["Hkv"] * row + c["seqs"] * c["Hq"] * (4 * c["D"] + 4),
                "flops": 4 * keys * c["Hq"] * c["D"]}
    rows = sum(_lengths(c["new"], c["seqs"], c["ragged"])) * c["Hkv"]
    return {"bytes": rows * 2 * (2 * c["D"] + (2 * c["D"] if c["cache"] == "bf16" else c["D"] + 1)), "flops": rows * 2 * c["D"]}


# ------------------------------------------------------------------------------------ the inputs

def _offsets(lens):
    t = torch.zeros(len(lens) + 1, dtype=torch.int32)
    t[1:] = torch.tensor(lens, dtype=torch.int32).cumsum(0)
    return t.to(DEV)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _powers(e):
    """2^(e - 127) of scale bytes."""
    return torch.ldexp(torch.ones((), device=e.device), e.to(torch.int32) - 127)


def _quantise(x):
    """e4m3 rows and their scale bytes: the smallest power of two, 2^-112 at least, that brings the row within 448."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(m == 0, torch.full_like(e, -112), e).clamp(-112, 120)
    rows = torch.ldexp(x, -e[..., None]).clamp(-448.0, 448.0)
    return rows.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _cache(c, g, lens):
    """A cache that holds `lens` tokens, each sequence's pages anywhere in the pool."""
    page = c["page"]
    need = [-(-n // page) for n in lens]
    n_pages, width = sum(need) + 3, max(1, max(need)) + 1
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    index = torch.zeros(len(lens), width, dtype=torch.int64)
    used = torch.arange(width)[None, :] < torch.tensor(need)[:, None]
    index[used] = torch.arange(sum(need))
    table = torch.where(used.to(DEV), order[index.to(DEV)], torch.full((), -1, dtype=torch.int32, device=DEV))
    shape = (n_pages, c["Hkv"], page, c["D"])
    k, v = _normal(g, *shape), _normal(g, *shape)
    k_scale = v_scale = None
    if c["cache"] == "e4m3":
        (k, k_scale), (v, v_scale) = _quantise(k), _quantise(v)
    return {"k": k, "v": v, "k_scale": k_scale, "v_scale": v_scale, "table": table.contiguous(),
            "lens": torch.tensor(lens, dtype=torch.int32, device=DEV)}


def _own_cache(s):
    import token_adapter_routing_amd as m
    return m.KvCache(s["k"], s["v"], s["k_scale"], s["v_scale"])


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": c}
    if c["kind"] in ("route", "route_grad"):
        N, K = c["N"], c["K"]
        s["logits"] = 1.5 * torch.randn(N, K, generator=g, device=DEV)
        if c["absent"]:
            gone = torch.rand(N, K, generator=g, device=DEV) < c["absent"]
            s["logits"].masked_fill_(gone, -math.inf)
        s["bias"] = 0.2 * torch.randn(K, generator=g, device=DEV) if c["bias"] else None
        if c["kind"] == "route_grad":
            s["idx"], _ = _route(s)
            s["dw"] = torch.randn(N, c["k"], generator=g, device=DEV)
        return s
    if c["kind"] in ("attn", "attn_grad"):
        ql, kl = _attn_lengths(c)
        tq, tk = sum(ql), sum(kl)
        s["q"], s["k"], s["v"] = _normal(g, tq, c["Hq"], c["D"]), _normal(g, tk, c["Hkv"], c["D"]), _normal(g, tk, c["Hkv"], c["D"])
        s["q_off"], s["kv_off"] = _offsets(ql), _offsets(kl)
        s["max_q"], s["max_kv"] = max(ql), max(kl)
        if c["kind"] == "attn_grad":
            s["do"] = _normal(g, tq, c["Hq"], c["D"])
            s["o"], s["lse"] = _attn(s)
        return s
    if c["kind"] == "decode":
        lens = _lengths(c["len"], c["seqs"], c["ragged"])
        s.update(_cache(c, g, lens))
        if c["window"]:  # pages that no later token will see are freed
            first = torch.arange(s["table"].shape[1], device=DEV)[None, :] * c["page"]
            freed = (first >= c["sinks"]) & (first + c["page"] <= s["lens"][:, None] - c["window"])
            s["table"] = torch.where(freed, torch.full_like(s["table"], -1), s["table"])
        s["q"] = _normal(g, c["seqs"], c["Hq"], c["D"])
        return s
    new = _lengths(c["new"], c["seqs"], c["ragged"])
    past = [(37 * i) % (c["past"] + 1) for i in range(c["seqs"])]
    s.update(_cache(c, g, [a + b for a, b in zip(new, past)]))
    s["q_off"] = _offsets(new)
    s["new_k"], s["new_v"] = _normal(g, sum(new), c["Hkv"], c["D"]), _normal(g, sum(new), c["Hkv"], c["D"])
    return s


# ------------------------------------------------------------------------------------ routing

def _route(s):
    """Scores, the selection in 64 bits (ties to the lowest index), weights in 32 bits."""
    c, l = s["case"], s["logits"]
    N, K, k, G = c["N"], c["K"], c["k"], c["groups"]
    there = l > -math.inf
    l64 = l.double()
    if c["score"] == SIGMOID:
        s64, s32 = 1 / (1 + torch.exp(-l64)), 1 / (1 + torch.exp(-l))
    else:
        top = torch.where(there, l, torch.full_like(l, -1e30)).amax(-1, keepdim=True)
        e64, e32 = torch.exp(l64 - top.double()), torch.exp(l - top)
        s64, s32 = e64 / e64.sum(-1, keepdim=True).clamp_min(1e-300), e32 / e32.sum(-1, keepdim=True).clamp_min(1e-37)
    pick = s64 if s["bias"] is None else s64 + s["bias"].double()
    pick = torch.where(there, pick, torch.full_like(pick, -math.inf))
    if G > 1:
        best = torch.sort(pick.view(N, G, K // G), dim=-1, descending=True).values[..., :2]
        some = best[..., 0] > -math.inf
        mark = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(-1)
        mark = torch.where(some, mark, torch.full_like(mark, -math.inf))
        order = torch.sort(mark, dim=-1, descending=True, stable=True).indices[:, :c["keep"]]
        kept = torch.zeros(N, G, dtype=torch.bool, device=l.device).scatter_(1, order, True)
        pick = torch.where(kept.repeat_interleave(K // G, 1), pick, torch.full_like(pick, -math.inf))
    value, idx = torch.sort(pick, dim=-1, descending=True, stable=True)
    idx = torch.where(value[:, :k] > -math.inf, idx[:, :k], torch.full_like(idx[:, :k], K)).sort(-1).values
    real = idx < K
    w = torch.where(real, s32.gather(1, idx.clamp_max(K - 1)), torch.zeros((), device=l.device))
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True).clamp_min(1e-37)
    return torch.where(real, idx, torch.full_like(idx, -1)).to(torch.int32), w * c["factor"]


def _route_grad(s):
    c, l, idx, dw = s["case"], s["logits"], s["idx"].long(), s["dw"]
    real = idx >= 0
    there = l > -math.inf
    if c["score"] == SIGMOID:
        p = 1 / (1 + torch.exp(-l))
    else:
        e = torch.exp(l - torch.where(there, l, torch.full_like(l, -1e30)).amax(-1, keepdim=True))
        p = e / e.sum(-1, keepdim=True).clamp_min(1e-37)
    sel = torch.where(real, p.gather(1, idx.clamp_min(0)), torch.zeros((), device=l.device))
    ds = torch.where(real, dw, torch.zeros_like(dw)) * c["factor"]
    if c["renorm"]:
        total = sel.sum(-1, keepdim=True).clamp_min(1e-37)
        ds = torch.where(real, ds - (ds * sel).sum(-1, keepdim=True) / total, torch.zeros_like(ds)) / total
    dp = torch.zeros_like(l).scatter_add_(1, idx.clamp_min(0), ds)
    if c["score"] == SIGMOID:
        return torch.where(there, dp * p * (1 - p), torch.zeros_like(l))
    return p * (dp - (dp * p).sum(-1, keepdim=True))


# ------------------------------------------------------------------------------------ attention

def _padded(x, off, most):
    """[T][H][D] rows of sequences as fp32 [S][H][most][D], zeros behind each sequence; and where the rows are."""
    at = off[:-1, None].long() + torch.arange(most, device=x.device)
    there = at < off[1:, None]
    rows = x[at.clamp_max(max(x.shape[0] - 1, 0))].float()
    return (rows * there[..., None, None]).transpose(1, 2), there


def _packed(x, there):
    """Back from [S][H][most][D] to [T][H][D]."""
    return x.transpose(1, 2)[there]


def _visible(c, q_len, kv_len, most_q, most_k):
    """[S][1][most_q][most_k]: whether query i (position kv_len - q_len + i) sees key j."""
    i = torch.arange(most_q, device=q_len.device)[:, None]
    j = torch.arange(most_k, device=q_len.device)[None, :]
    p = (kv_len - q_len)[:, None, None] + i
    seen = (j <= p) & (i < q_len[:, None, None])
    if c["window"]:
        seen &= (j > p - c["window"]) | (j < c["sinks"])
    return seen[:, None]


def _scores(s):
    """Scaled scores with -inf where nothing is seen, [S][Hkv][g * Lq][Lk], and the padded operands."""
    c = s["case"]
    S, g, D = c["seqs"], c["Hq"] // c["Hkv"], c["D"]
    q, there_q = _padded(s["q"], s["q_off"], s["max_q"])
    k, there_k = _padded(s["k"], s["kv_off"], s["max_kv"])
    v, _ = _padded(s["v"], s["kv_off"], s["max_kv"])
    q = q.reshape(S, c["Hkv"], g * s["max_q"], D)
    scores = torch.matmul(q, k.transpose(-1, -2).contiguous()) / math.sqrt(D)
    seen = _visible(c, s["q_off"].diff(), s["kv_off"].diff(), s["max_q"], s["max_kv"])
    scores.view(S, c["Hq"], s["max_q"], s["max_kv"]).masked_fill_(~seen, -math.inf)
    return scores, q, k, v, there_q, there_k


def _attn(s):
    c = s["case"]
    scores, _, _, v, there_q, _ = _scores(s)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total)).view(c["seqs"], c["Hq"], s["max_q"], 1)
    o = o.view(c["seqs"], c["Hq"], s["max_q"], c["D"])
    return _packed(o, there_q).to(torch.bfloat16), _packed(lse, there_q)[..., 0].t().contiguous()


def _attn_grad(s):
    c = s["case"]
    S, D = c["seqs"], c["D"]
    scores, q, k, v, there_q, there_k = _scores(s)
    lse, _ = _padded(s["lse"].t()[..., None], s["q_off"], s["max_q"])
    lse = torch.where(lse > -math.inf, lse, torch.zeros_like(lse)).nan_to_num(0.0)
    do, _ = _padded(s["do"], s["q_off"], s["max_q"])
    o, _ = _padded(s["o"], s["q_off"], s["max_q"])
    merged = (S, c["Hkv"], -1, D)
    delta = (do * o).sum(-1, keepdim=True).reshape(S, c["Hkv"], -1, 1)
    do = do.reshape(merged)
    p = scores.sub_(lse.reshape(S, c["Hkv"], -1, 1)).exp_()
    dv = torch.matmul(p.transpose(-1, -2), do)
    ds = torch.matmul(do, v.transpose(-1, -2).contiguous()).sub_(delta).mul_(p).mul_(1 / math.sqrt(D))
    dq = torch.matmul(ds, k).view(S, c["Hq"], s["max_q"], D)
    dk = torch.matmul(ds.transpose(-1, -2), q)
    return (_packed(dq, there_q).to(torch.bfloat16), _packed(dk, there_k).to(torch.bfloat16),
            _packed(dv, there_k).to(torch.bfloat16))


def _read(s, name):
    """The cache's rows by sequence and position, fp32 [S][Hkv][width * page][D]."""
    c = s["case"]
    x = s[name].float()
    if s[name + "_scale"] is not None:
        x = x * _powers(s[name + "_scale"])[..., None]
    x = x[s["table"].clamp_min(0).long()]
    return x.transpose(1, 2).reshape(c["seqs"], c["Hkv"], -1, c["D"])


def _decode(s):
    c = s["case"]
    S, D = c["seqs"], c["D"]
    k, v = _read(s, "k"), _read(s, "v")
    q = s["q"].float().view(S, c["Hkv"], -1, D)
    j = torch.arange(k.shape[2], device=q.device)[None, :]
    n = s["lens"][:, None]
    seen = j < n
    if c["window"]:
        seen &= (j >= n - c["window"]) | (j < c["sinks"])
    scores = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(D)
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o.reshape(S, c["Hq"], D).to(torch.bfloat16), (top + torch.log(total)).reshape(S, c["Hq"])


def _places(s):
    """Page and row of every new token."""
    T = s["new_k"].shape[0]
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(s["q_off"][1:].long(), t, right=True)
    pos = s["lens"].long()[b] - s["q_off"][1:].long()[b] + t
    return s["table"].long()[b, pos // s["case"]["page"]], pos % s["case"]["page"]


def _append(s):
    page, row = _places(s)
    for name in ("k", "v"):
        new = s["new_" + name]
        if s["case"]["cache"] == "e4m3":
            new, scale = _quantise(new)
            s[name + "_scale"][page, :, row] = scale
            s[name].view(torch.uint8)[page, :, row] = new.view(torch.uint8)
        else:
            s[name][page, :, row] = new
    return [x for x in (s["k"], s["v"], s["k_scale"], s["v_scale"]) if x is not None]


def run(state):
    s, c = state, state["case"]
    kind = c["kind"]
    if own:
        import token_adapter_routing_amd as m
        if kind in ("route", "route_grad"):
            score = m.SCORE_SIGMOID if c["score"] == SIGMOID else m.SCORE_SOFTMAX
            if kind == "route":
                return m.molora_route_scores(s["logits"], c["k"], bias=s["bias"], score=score, n_group=c["groups"],
                                             topk_group=c["keep"], renorm=c["renorm"], factor=c["factor"])
            return m.molora_route_scores_backward(s["logits"], s["idx"], s["dw"], score=score, renorm=c["renorm"],
                                                  factor=c["factor"])
        if kind == "attn":
            return m.molora_attn_forward(s["q"], s["k"], s["v"], s["q_off"], s["kv_off"], window=c["window"],
                                         sinks=c["sinks"])
        if kind == "attn_grad":
            return m.molora_attn_backward(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["q_off"], s["kv_off"],
                                          window=c["window"], sinks=c["sinks"])
        if kind == "decode":
            return m.molora_attn_decode(s["q"], _own_cache(s), s["table"], s["lens"], window=c["window"],
                                        sinks=c["sinks"])
        m.molora_kv_append(_own_cache(s), s["new_k"], s["new_v"], s["q_off"], s["table"], s["lens"])
        return [x for x in (s["k"], s["v"], s["k_scale"], s["v_scale"]) if x is not None]
    return {"route": _route, "route_grad": _route_grad, "attn": _attn, "attn_grad": _attn_grad, "decode": _decode,
            "append": _append}[kind](s)


# ------------------------------------------------------------------------------------ in 64 bits

def _exact_weights(c, logits, idx):
    """Weights of the chosen adapters as a differentiable function of the logits, 64 bits."""
    if c["score"] == SIGMOID:
        chance = torch.sigmoid(logits)
    else:
        chance = torch.softmax(logits, -1)
    chance = torch.where(torch.isfinite(logits), chance, torch.zeros_like(chance))
    picked = torch.stack([torch.where(idx[:, j] >= 0, chance[torch.arange(len(idx)), idx[:, j].clamp(min=0)],
                                      torch.zeros(len(idx), dtype=torch.float64)) for j in range(idx.shape[1])], 1)
    if c["renorm"]:
        whole = picked.sum(1, keepdim=True)
        picked = picked / torch.where(whole > 0, whole, torch.ones_like(whole))
    return picked * c["factor"]


def _exact_head(q, k, v, c):
    """One head of one sequence: output, log of the sum, in 64 bits."""
    L, M = q.shape[0], k.shape[0]
    z = q @ k.T * c["D"] ** -0.5
    where = torch.arange(M - L, M, device=q.device)[:, None]
    back = where - torch.arange(M, device=q.device)[None, :]
    hide = back < 0
    if c["window"]:
        hide |= (back >= c["window"]) & (where - back >= c["sinks"])
    z = z.masked_fill(hide, -math.inf)
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - torch.where(torch.isfinite(lse), lse, torch.zeros_like(lse))[:, None])
    return p @ v, lse


def exact(case, seed):
    c, s = case, prepare(case, seed)
    kind = c["kind"]
    if kind == "route":
        idx = _route(s)[0].long().cpu()  # the choice is compared as it is: here it names the weights' adapters
        l = s["logits"].double().cpu()
        l = torch.where((l == -math.inf).all(1, keepdim=True), torch.zeros_like(l), l)
        return None, _exact_weights(c, l, idx)
    if kind == "route_grad":
        l = s["logits"].double().cpu()
        l = torch.where((l == -math.inf).all(1, keepdim=True), torch.zeros_like(l), l).requires_grad_(True)
        w = _exact_weights(c, l, s["idx"].long().cpu())
        grad, = torch.autograd.grad((w * s["dw"].double().cpu()).sum(), l)
        return torch.nan_to_num(grad, nan=0.0)
    if kind in ("attn", "attn_grad"):
        ql, kl = _attn_lengths(c)
        g = c["Hq"] // c["Hkv"]
        q, k, v = (s[n].double() for n in "qkv")
        out = torch.zeros_like(q)
        lse = torch.zeros(c["Hq"], q.shape[0], dtype=torch.float64, device=DEV)
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        a = b = 0
        for n, m in zip(ql, kl):
            for h in range(c["Hq"]):
                ops = [q[a:a + n, h], k[b:b + m, h // g], v[b:b + m, h // g]]
                if n == 0:
                    continue
                if kind == "attn":
                    out[a:a + n, h], lse[h, a:a + n] = _exact_head(*ops, c)
                else:
                    ops = [x.clone().requires_grad_(True) for x in ops]
                    y, _ = _exact_head(*ops, c)
                    d = torch.autograd.grad((y * s["do"][a:a + n, h].double()).sum(), ops)
                    dq[a:a + n, h] = d[0]
                    dk[b:b + m, h // g] += d[1]
                    dv[b:b + m, h // g] += d[2]
            a, b = a + n, b + m
        return (out, lse) if kind == "attn" else (dq, dk, dv)
    if kind == "decode":
        lens = _lengths(c["len"], c["seqs"], c["ragged"])
        g, page = c["Hq"] // c["Hkv"], c["page"]
        out = torch.zeros(c["seqs"], c["Hq"], c["D"], dtype=torch.float64, device=DEV)
        lse = torch.full((c["seqs"], c["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
        for b, n in enumerate(lens):
            see = [j for j in range(n) if not c["window"] or j >= n - c["window"] or j < c["sinks"]]
            if not see:
                continue
            j = torch.tensor(see, device=DEV)
            at, row = s["table"][b].long()[j // page], j % page
            kv = []
            for name in ("k", "v"):
                x = s[name][at, :, row].double()
                if c["cache"] == "e4m3":
                    x = x * 2.0 ** (s[name + "_scale"][at, :, row].double() - 127)[..., None]
                kv.append(x)
            q = s["q"][b].double().view(c["Hkv"], g, c["D"])
            z = torch.einsum("hgd,jhd->hgj", q, kv[0]) * c["D"] ** -0.5
            lse[b] = torch.logsumexp(z, 2).reshape(-1)
            out[b] = torch.einsum("hgj,jhd->hgd", torch.softmax(z, 2), kv[1]).reshape(c["Hq"], c["D"])
        return out, lse
    got = [s["k"].double(), s["v"].double()]
    off, lens = s["q_off"].tolist(), s["lens"].tolist()
    for b in range(c["seqs"]):
        T = off[b + 1] - off[b]
        pos = torch.arange(lens[b] - T, lens[b], device=DEV)
        at = s["table"][b].long()[pos // c["page"]]
        for x, name in zip(got, ("new_k", "new_v")):
            new = s[name][off[b]:off[b + 1]].double()
            if c["cache"] == "e4m3":  # the row over its scale, before it is rounded to 8 bits
                big = new.abs().amax(2, keepdim=True).clamp(min=448 * 2.0 ** -112)
                new = new / 2.0 ** torch.ceil(torch.log2(big / 448))
            x[at, :, pos % c["page"]] = new
    return got if c["cache"] == "bf16" else got + [None, None]
