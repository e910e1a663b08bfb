"""The decoder's serving form (molora_xf_prefill, molora_xf_decode over paged caches) against the fp64
decoder of oracle/transformer.py, and the two against each other.

Bars as in test_gpu_xf.py: every intermediate is stored in bf16, so the GPU and the oracle (rounding at
the same points) differ by one-ulp flips that the layers carry along: relative Frobenius error <= 1e-2,
elements within 0.1 of the rms.  An 8-bit cache moves keys and values by up to 2^-4 of themselves, at
random: its bar is 0.1."""
import numpy as np
import pytest
import torch

import synth
from gpu_util import dev, dev_bf16, host, need_gpu
from oracle import route_topk, route_vocab
from oracle import transformer as T
from test_gpu_xf import _compare, _model, _oracle_layers, f64

pytestmark = pytest.mark.gpu


class Setup:
    def __init__(self, m, cid, d, L, K, r, n_seq, seq_len, k=1, lora=True, cache=torch.bfloat16, page=16, scale=0.5):
        self.m, self.n_seq, self.seq_len, self.d, self.k, self.K, self.scale = m, n_seq, seq_len, d, k, K, scale
        f = synth.xf_mlp_width(d)
        lb = synth.xf_layers(cid, d, L, K, r)
        self.x, ids, bounds, _ = synth.xf_batch(cid, n_seq, seq_len, d, K, mean_run=7.0)
        N = n_seq * seq_len
        if k == 1:
            idx, w = route_vocab(ids, bounds)
            self.idx, self.w = idx.astype(np.int32).reshape(N, 1), w.astype(np.float32).reshape(N, 1)
        else:
            i2, w2, _ = route_topk(np.random.default_rng(cid).standard_normal((N, K)), k)
            self.idx, self.w = i2.astype(np.int32), w2.astype(np.float32)
        self.lora = lora
        self.model = _model(m, lb, d, f, scale, lora)
        self.oracle_layers = _oracle_layers(lb, lora)
        width = -(-seq_len // page) + 1
        self.caches = [m.KvCache.empty(n_seq * width, d // 128, page, 128, dtype=cache) for _ in range(L)]
        self.table = torch.randperm(n_seq * width, generator=torch.Generator().manual_seed(cid)).view(n_seq, width)
        self.table = self.table.to(torch.int32).cuda()

    def route(self, rows):
        if not self.lora:
            return None
        _, *rest = self.m.molora_dispatch(dev(self.idx[rows].reshape(-1)), dev(self.w[rows].reshape(-1)), self.K, self.k)
        return tuple(rest)

    def rows(self, lens):
        """Packed rows of the first lens[b] tokens of every sequence."""
        return np.concatenate([np.arange(n) + b * self.seq_len for b, n in enumerate(lens)]).astype(np.int64)

    def prefill(self, lens, **kw):
        at = self.rows(lens)
        off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        return self.m.molora_xf_prefill(self.model, self.caches, dev_bf16(self.x[at]), off, self.table,
                                        torch.tensor(lens, dtype=torch.int32, device="cuda"), route=self.route(at),
                                        k=self.k, **kw), at

    def decode(self, lens, **kw):
        """Token lens[b] - 1 of every sequence."""
        at = np.array([b * self.seq_len + n - 1 for b, n in enumerate(lens)])
        return self.m.molora_xf_decode(self.model, self.caches, dev_bf16(self.x[at]), self.table,
                                       torch.tensor(lens, dtype=torch.int32, device="cuda"), route=self.route(at),
                                       k=self.k, **kw), at

    def reference(self):
        idx = self.idx if self.k > 1 else self.idx[:, 0]
        w = (self.w if self.k > 1 else self.w[:, 0]).astype(np.float64)
        return T.forward(f64(self.x), self.oracle_layers, self.scale, idx, w, self.K, self.n_seq, self.seq_len,
                         store=T.bf16_store)


@pytest.mark.parametrize("d,L,k,lora", [(256, 2, 1, True), (256, 1, 2, True), (512, 2, 1, False)])
def test_prompts_then_tokens_match_the_oracle(d, L, k, lora):
    m = need_gpu()
    s = Setup(m, 300 + d + k, d, L, 3, 8, 3, 45, k=k, lora=lora)
    ref = s.reference()
    lens = [33, 1, 40]
    y, at = s.prefill(lens)
    _compare(host(y), ref[at])
    for step in range(5):
        lens = [n + 1 for n in lens]
        y, at = s.decode(lens)
        _compare(host(y), ref[at])


def test_prefill_equals_forward():
    """Equal lengths: molora_xf_forward's result up to the attention's own rounding."""
    m = need_gpu()
    s = Setup(m, 310, 256, 2, 4, 16, 2, 70)
    y, at = s.prefill([70, 70])
    z = m.molora_xf_forward(s.model, dev_bf16(s.x), 2, 70, route=s.route(at))
    _compare(host(y), host(z))


@pytest.mark.parametrize("window,sinks", [(6, 0), (10, 3)])
def test_window_prompts_and_tokens_agree(window, sinks):
    m = need_gpu()
    s = Setup(m, 320 + window, 256, 2, 2, 8, 2, 50)
    whole, at = s.prefill([50, 30], window=window, sinks=sinks)
    whole = {int(a): host(whole)[i] for i, a in enumerate(at)}
    lens = [30, 5]
    s.prefill(lens, window=window, sinks=sinks)
    for _ in range(12):
        lens = [n + 1 for n in lens]
        y, at = s.decode(lens, window=window, sinks=sinks)
        _compare(host(y), np.stack([whole[int(a)] for a in at]))
    full, at = s.prefill([50, 30])
    full = {int(a): host(full)[i] for i, a in enumerate(at)}
    far = np.stack([full[49]]) - np.stack([whole[49]])
    assert np.abs(far).max() > 1e-3  # the window does something


def test_8_bit_cache():
    m = need_gpu()
    s = Setup(m, 330, 256, 2, 2, 8, 2, 60, cache=torch.float8_e4m3fn, page=32)
    ref = s.reference()
    s.prefill([40, 55])
    lens = [40, 55]
    for _ in range(4):
        lens = [n + 1 for n in lens]
        y, at = s.decode(lens)
        err = np.linalg.norm(host(y) - ref[at]) / np.linalg.norm(ref[at])
        assert err < 0.1, err


def test_empty_slots_and_in_place():
    """A batch slot without a sequence (length 0) changes nothing else; x_out may be x_in."""
    m = need_gpu()
    s = Setup(m, 340, 256, 1, 2, 8, 3, 30)
    s.prefill([20, 0, 9])
    before = s.caches[0].k.clone()
    lens = torch.tensor([21, 0, 10], dtype=torch.int32, device="cuda")
    at = np.array([20, 30, 69])
    x = dev_bf16(s.x[at])
    y = m.molora_xf_decode(s.model, s.caches, x, s.table, lens, route=s.route(at))
    ref = s.reference()
    _compare(host(y)[[0, 2]], ref[[20, 69]])
    assert int((s.caches[0].k != before).any(-1).sum()) <= 2 * 2
    z = m.molora_xf_decode(s.model, s.caches, x, s.table, lens, route=s.route(at), out=x)
    assert z is x and torch.equal(z, y)


def test_captured_decode_step_replays():
    m = need_gpu()
    s = Setup(m, 350, 256, 2, 2, 8, 2, 40)
    s.prefill([11, 20])
    lens = torch.tensor([12, 21], dtype=torch.int32, device="cuda")
    x = dev_bf16(s.x[np.array([11, 60])])
    route = s.route(np.array([11, 60]))
    ws = torch.empty(m.molora_xf_serve_workspace(s.model, s.caches, 2, 2, s.table.shape[1]), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(x)

    def step():
        m.molora_xf_decode(s.model, s.caches, x, s.table, lens, route=route, out=out, ws=ws)
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        x.copy_(dev_bf16(s.x[np.array([12 + i, 61 + i])]))
        lens.copy_(torch.tensor([13 + i, 22 + i], dtype=torch.int32))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out)


def test_refusals():
    m = need_gpu()
    s = Setup(m, 360, 256, 2, 2, 8, 2, 20)
    x, lens = dev_bf16(s.x[:2]), torch.ones(2, dtype=torch.int32, device="cuda")
    route = s.route(np.array([0, 1]))

    def go(**kw):
        a = dict(model=s.model, caches=s.caches, x=x, table=s.table, lens=lens, route=route)
        rest = {k: v for k, v in kw.items() if k not in a}
        a.update(kw)
        return m.molora_xf_decode(a["model"], a["caches"], a["x"], a["table"], a["lens"], route=a["route"], **rest)
    go()
    with pytest.raises(ValueError, match="caches"):
        go(caches=s.caches[:1])
    with pytest.raises(m.MoloraError, match="heads"):
        go(caches=[m.KvCache.empty(4, 1, 16, 128)] * 2)
    with pytest.raises(m.MoloraError, match="heads"):
        go(caches=[m.KvCache.empty(4, 2, 16, 64)] * 2)
    with pytest.raises(m.MoloraError, match="page_size"):
        go(caches=[s.caches[0], m.KvCache.empty(8, 2, 32, 128)])
    with pytest.raises(m.MoloraError, match="required"):
        go(route=None)
    with pytest.raises(m.MoloraError, match="workspace"):
        go(ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(m.MoloraError, match="window"):
        go(window=-1)
    with pytest.raises(ValueError, match="one token"):
        go(x=dev_bf16(s.x[:3]))
    other = synth.xf_layers(361, 256, 1, 2, 24)[0]
    s.model.layers[1]["lora"] = m.molora_hotset_init([(dev_bf16(a), dev_bf16(b)) for a, b in zip(other["A"], other["B"])], 0.5)
    mixed = m.XfModel(256, s.model.f, s.model.layers)
    with pytest.raises(m.MoloraError, match="rank"):
        go(model=mixed)
