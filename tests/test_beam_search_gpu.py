"""A whole beam search: the choice of beams, pages forked, given out and copied, keys and values appended, attention over the
shared prompt and over each beam's own pages, joined; eager, and as one captured graph.

Beams' histories are followed on the host; a step's attention is held to the plain form over a beam's history.  Softmax
weights are rounded to BF16 (2^-8 each), a part's output (2^-8), the joined one (2^-8): with 32-bit sums beside them, 3.1 * 2^-8 of the largest value."""
import math

import pytest
import torch

import lossless_float_compression_amd as zx
from pages_util import i32
from test_beam_select_gpu import check as check_choice

pytestmark = pytest.mark.gpu


class Search:
    """`layers` attention layers over one pool; each token's query, key and value are rows of fixed tables."""

    def __init__(self, G, K, prompt, T, H, Q, D, V, steps, dtype=zx.BF16, layers=2, C=None, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.G, self.K, self.T, self.D, self.V = G, K, T, D, V
        e = lambda *s: (torch.randn(s, generator=g, device="cuda") * 0.8).to(torch.bfloat16)   # noqa: E731
        self.eq, self.ek, self.ev = ([e(V, h, D) for _ in range(layers)] for h in (Q, H, H))
        self.w = torch.randn((layers * Q * D, V), generator=g, device="cuda") * 0.3
        self.prompt = [torch.randint(0, V, (n,), generator=g, device="cuda") for n in prompt]
        shared = [n // T * T for n in prompt]
        n_pages = sum(shared) // T + G * K * (2 + steps // T) + 7
        self.pool, self.err = zx.PagePool(n_pages, T), i32([0])
        self.caches = [zx.PagedKVCache(n_pages, H, D, T, dtype, block_tokens=C, k_scale=0.02 if dtype == zx.FP8_E4M3FN else None,
                                       v_scale=0.02 if dtype == zx.FP8_E4M3FN else None) for _ in range(layers)]
        self.all = zx.PagedLayers(self.caches)
        # the prompts' whole pages, as rows of their own
        start = [0]
        for n in shared:
            start.append(start[-1] + n)
        table, held, kv = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((G, max(shared) // T + 1), (G,), (G,)))
        b = zx.PagedBatch(i32(start), kv, table)
        self.pool.extend(b, held, err=self.err)
        self.put(torch.cat([p[:n] for p, n in zip(self.prompt, shared)]), b)
        self.before = zx.PagedBatch(i32([i * K for i in range(G + 1)]), held, table, max_q=K)
        # what is left of them, as the beams' first tokens
        n = G * K
        self.table, self.held, self.kv = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((n, 2 + steps // T), (n,), (n,)))
        left = [p.numel() - s for p, s in zip(self.prompt, shared)]
        start = [0]
        for i in range(n):
            start.append(start[-1] + (left[i // K] if i % K == 0 else 0))
        b = zx.PagedBatch(i32(start), self.kv, self.table)
        self.pool.extend(b, self.held, err=self.err)
        self.put(torch.cat([p[s:] for p, s in zip(self.prompt, shared)]), b)
        self.own = zx.PagedBatch(i32(list(range(n + 1))), self.kv, self.table, max_q=1)
        self.copies = zx.PageCopies(n)
        self.scores = torch.full((G, K), -math.inf, device="cuda")
        self.scores[:, 0] = 0.0
        self.fin = torch.zeros((G, K), dtype=torch.bool, device="cuda")
        self.choice = zx.Beams(self.scores, torch.zeros((G, K), dtype=torch.int32, device="cuda"), torch.ones((G, K), dtype=torch.int32, device="cuda"), self.fin)

    def put(self, tokens, batch):
        for c, k, v in zip(self.caches, self.ek, self.ev):
            c.append(k[tokens], v[tokens], batch, err=self.err)

    def step(self):
        """One token more for every beam, from the last choice on, and the next choice in its place."""
        self.pool.fork(self.table, self.held, self.choice.parents, err=self.err)
        self.pool.extend(self.own, self.held, copies=self.copies, err=self.err)
        self.all.copy_pages(self.copies, err=self.err)
        t = self.choice.tokens.view(-1).clamp(min=0).long()
        self.put(t, self.own)
        x = []
        for c, e in zip(self.caches, self.eq):
            q = e[t]
            lses = [torch.full(q.shape[:2], -math.inf, device="cuda") for _ in range(2)]
            outs = [c.attend(q, self.before, causal=False, lse=lses[0], err=self.err), c.attend(q, self.own, lse=lses[1], err=self.err)]
            x.append(zx.merge_attention(outs, lses))
        logits = (torch.cat([y.flatten(1) for y in x], 1).float() @ self.w).view(self.G, self.K, self.V).to(torch.bfloat16)
        before = self.scores.clone(), self.fin.clone()
        zx.beam_select(logits, self.scores, finished=self.fin, end=0, out=self.choice, err=self.err)
        return x, logits, before


CASES = [dict(G=1, K=4, prompt=[50], T=16, H=2, Q=8, D=64, V=500, steps=40), dict(G=3, K=5, prompt=[16, 7, 133], T=16, H=1, Q=4, D=128, V=333, steps=24, C=16),
         dict(G=5, K=3, prompt=[1, 200, 64, 63, 65], T=64, H=2, Q=2, D=64, V=97, steps=20, dtype=zx.FP8_E4M3FN),
         dict(G=2, K=16, prompt=[300, 31], T=32, H=2, Q=6, D=128, V=4001, steps=10)]


@pytest.mark.parametrize("case", CASES)
def test_a_beam_search(case):
    s = Search(**case)
    G, K = s.G, s.K
    hist = [p.tolist() for p in s.prompt for _ in range(K)]
    for i in range(case["steps"]):
        par, tok = s.choice.parents.tolist(), s.choice.tokens.tolist()
        hist = [hist[g * K + par[g][b]] + [max(tok[g][b], 0)] if par[g][b] >= 0 else None for g in range(G) for b in range(K)]
        x, logits, (scores, fin) = s.step()
        assert int(s.err) == 0
        for r, h in enumerate(hist):
            if h is None:
                continue
            for c, y, eq, ek, ev in zip(s.caches, x, s.eq, s.ek, s.ev):
                k, v = (t[h].float() for t in (ek, ev))
                if c.k_scale is not None:
                    k, v = ((t / z[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).float() * z[:, None] for t, z in ((k, c.k_scale), (v, c.v_scale)))
                k, v = (t.double().repeat_interleave(case["Q"] // case["H"], 1) for t in (k, v))
                w = torch.softmax(torch.einsum("hd,thd->ht", eq[h[-1]].double(), k) / math.sqrt(s.D), 1)
                off = (y[r].double() - torch.einsum("ht,thd->hd", w, v)).abs().max()
                assert float(off) <= 3.1 * 2.0 ** -8 * float(v.abs().max()), (i, r, float(off))
        check_choice(s.choice, logits, scores, K, finished=fin, end=0)
        live = sum(-(-int(h) // s.T) for h in s.held) + sum(-(-int(h) // s.T) for h in s.before.kv_len)
        assert int(s.pool.refs.sum()) == live        # every page is held by as many rows as say so
    # the end: all pages come back
    s.pool.trim(s.table, s.held)
    s.pool.trim(s.before.page_table, s.before.kv_len)
    assert not bool(s.pool.refs.any())


@pytest.mark.parametrize("case", CASES[:3])
def test_as_a_graph(case):
    """The step captured once and replayed gives the eager search, bit for bit."""
    a, b = Search(**case), Search(**case)
    kept = [t.clone() for t in (b.pool.refs, b.table, b.held, b.kv, *b.choice)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.step()                                     # (libraries set themselves up outside of captures)
    torch.cuda.current_stream().wait_stream(side)
    for t, k in zip((b.pool.refs, b.table, b.held, b.kv, *b.choice), kept):
        t.copy_(k)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x, logits, _ = b.step()
    for i in range(case["steps"] - 1):
        y, want, _ = a.step()
        g.replay()
        assert torch.equal(logits, want) and all(torch.equal(p, q) for p, q in zip(x, y)), i
        for p, q in zip((*a.choice, a.table, a.held, a.pool.refs), (*b.choice, b.table, b.held, b.pool.refs)):
            assert torch.equal(p, q), i
    assert int(b.err) == 0
