"""The cache and the attention over it as a model runs them: a gated recurrence, then
an attention layer on its output (normed queries and keys, rotation on the way into
the cache).  Padded prompts, prompts in pieces, token by token, and drafted tokens
several at once, against the whole computed in 64 bits (fp32 inputs).

Bounds: 1e-4 * (1 + |ref|) as in the test of the layer of recurrence, norm and scan:
every stage loses 1e-6 relative or less, and scores of order one pass that on as it is."""
import numpy as np
import pytest
import torch

import attn_ref
import glr_ref
import norm_rotate_ref
from mamba_ssd_scan_05_amd import ssd

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = 1e-4


class Layer:
    def __init__(self, b, T, D, Hq, Hk, N, window, seed):
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.b, self.T, self.D, self.Hq, self.Hk, self.N, self.window = b, T, D, Hq, Hk, N, window
        H = Hq + 2 * Hk
        self.t = dict(x=n(b, T, D), r=n(b, T, D), i=n(b, T, D), A=-torch.rand(D, generator=g) - 0.3, rb=n(D), ib=n(D),
                      W=n(D, H * N) / D ** 0.5, qw=1 + 0.1 * n(N), kw=1 + 0.1 * n(N),
                      freqs=(10000.0 ** (-torch.arange(N // 2) / (N // 2))).float())
        self.d = {k: v.to(DEV) for k, v in self.t.items()}
        self.eps, self.scale = float(np.float32(1e-6)), float(np.float32(N ** -0.5))

    def expect(self, i, order):
        """Output [n, Hq, N] and last state of row i over the tokens `order`."""
        a = {k: v.double().numpy() for k, v in self.t.items()}
        x, r, gi = (a[k][i:i + 1, order] for k in ("x", "r", "i"))
        f = glr_ref.forward(x, r, gi, a["A"], a["rb"], a["ib"], None, None, np.zeros((1, self.D)))
        p = (f["h"] @ a["W"]).reshape(1, len(order), -1, self.N)
        pos = np.arange(len(order))[None]
        q, _ = norm_rotate_ref.forward(p[:, :, :self.Hq], a["qw"], pos, a["freqs"], self.eps, False)
        k, _ = norm_rotate_ref.forward(p[:, :, self.Hq:self.Hq + self.Hk], a["kw"], pos, a["freqs"], self.eps, False)
        v = p[0, :, self.Hq + self.Hk:]
        G = self.Hq // self.Hk
        out = np.stack([attn_ref.attend(q[0, :, h], k[0, :, h // G], v[:, h // G], pos[0], self.scale, self.window, 0.0)[0]
                        for h in range(self.Hq)], 1)
        return out, f["fin"][0]

    def cache(self, page, capacity):
        width = -(-capacity // page)
        order = torch.randperm(self.b * width, generator=torch.Generator().manual_seed(1)).to(torch.int32)
        self.table = order.view(self.b, width).to(DEV)
        kv = torch.full((self.b * width, 2, page, self.Hk, self.N), float("nan"), device=DEV)
        self.kc, self.vc = kv[:, 0], kv[:, 1]
        self.state = torch.zeros(self.b, self.D, device=DEV)
        self.start = torch.zeros(self.b, dtype=torch.int32, device=DEV)

    def attention(self, h, tokens, step=False):
        """The attention layer on h [b, L, D]; tokens: how many of them each row has."""
        b, L = h.shape[:2]
        p = torch.matmul(h, self.d["W"]).view(b, L, -1, self.N)
        q, k = ssd.ssd_norm_rotate_fwd(p[:, :, :self.Hq], p[:, :, self.Hq:self.Hq + self.Hk], self.d["qw"], self.d["kw"],
                                       eps=self.eps)
        q = ssd.ssd_kv_append(k, p[:, :, self.Hq + self.Hk:], self.kc, self.vc, self.table, self.start, q=q,
                              freqs=self.d["freqs"], tokens=tokens)
        if step:
            out = ssd.ssd_attn_step(q[:, 0], self.kc, self.vc, self.table, self.start, scale=self.scale, window=self.window)
        else:
            out, _ = ssd.ssd_attn_fwd(q, self.kc, self.vc, self.table, self.start, tokens=tokens, scale=self.scale,
                                      window=self.window)
        self.start += L if tokens is None else tokens
        return out

    def gates(self, cols):
        return [self.d[k][:, cols].contiguous() for k in ("x", "r", "i")] + [self.d[k] for k in ("A", "rb", "ib")]


def close(got, ref, what):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - ref) <= TOL * (1 + np.abs(ref)))
    assert not bad.any(), "%s: worst %.3g of the bound" % (what, np.nanmax(np.abs(got - ref) / (TOL * (1 + np.abs(ref)))))


@pytest.mark.parametrize("page,window", [(16, 0), (5, 0), (16, 24)])
def test_padded_prompts_then_token_by_token(page, window):
    L, K, lens = 70, 9, [70, 41, 0, 1]
    t = Layer(4, L + K, 96, 4, 2, 32, window, seed=3)
    t.cache(page, L + K)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    h, t.state = ssd.ssd_glr_fwd(*t.gates(slice(0, L)), lengths=n, init_state=t.state)
    out = t.attention(h, n)
    ref = [t.expect(i, list(range(lens[i])) + list(range(L, L + K))) for i in range(4)]
    for i in range(4):
        close(out[i, :lens[i]], ref[i][0][:lens[i]], "prompt %d" % i)
    for s in range(K):
        x = [v[:, 0].contiguous() if v.dim() == 3 else v for v in t.gates(slice(L + s, L + s + 1))]
        h = ssd.ssd_glr_step(t.state, *x)
        out = t.attention(h[:, None], None, step=True)
        for i in range(4):
            close(out[i], ref[i][0][lens[i] + s], "row %d token %d" % (i, s))
    for i in range(4):
        close(t.state[i], ref[i][1], "state")


@pytest.mark.parametrize("pieces", [[100], [30, 30, 40], [1, 4, 1, 5, 89], [64, 17, 19]])
def test_prompt_in_pieces_and_drafts(pieces):
    t = Layer(2, 100, 64, 6, 1, 64, 0, seed=5)
    t.cache(16, 100)
    ref = [t.expect(i, list(range(100)))[0] for i in range(2)]
    at = 0
    for n in pieces:
        h, t.state = ssd.ssd_glr_fwd(*t.gates(slice(at, at + n)), init_state=t.state)
        out = t.attention(h, None)
        for i in range(2):
            close(out[i], ref[i][at:at + n], "piece at %d" % at)
        at += n


def test_a_layers_step_in_a_graph():
    # recurrence, norm, append and attention of one token, replayed while the rows grow
    t = Layer(3, 60, 64, 4, 2, 32, 0, seed=7)
    t.cache(8, 60)
    ref = [t.expect(i, list(range(60)))[0] for i in range(3)]
    h, t.state = ssd.ssd_glr_fwd(*t.gates(slice(0, 40)), init_state=t.state)
    t.attention(h, None)
    x, r, i = (torch.empty(3, 64, device=DEV) for _ in range(3))
    start0, state0 = t.start.clone(), t.state.clone()

    def step():
        h = ssd.ssd_glr_step(t.state, x, r, i, t.d["A"], t.d["rb"], t.d["ib"])
        return t.attention(h[:, None], None, step=True)
    for v, k in ((x, "x"), (r, "r"), (i, "i")):
        v.copy_(t.d[k][:, 40])
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    t.start.copy_(start0), t.state.copy_(state0)
    for s in range(40, 60):
        for v, k in ((x, "x"), (r, "r"), (i, "i")):
            v.copy_(t.d[k][:, s])
        graph.replay()
        torch.cuda.synchronize()
        for j in range(3):
            close(out[j], ref[j][s], "token %d" % s)
    assert t.start.tolist() == [60] * 3
