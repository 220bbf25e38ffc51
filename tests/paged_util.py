"""Plain 64-bit forms of the paged K/V cache operators, and how far a kernel may be from them.

Roundings counted: a BF16 value is off by at most 2^-8 of itself (half a step), a 32-bit one by
2^-24; E4M3 by 2^-4 of itself, or 2^-10 below its smallest normal value."""
import math

import torch

import lossless_float_compression_amd as zx

RAW = {zx.BF16: torch.int16, zx.FP8_E4M3FN: torch.uint8}
TDT = {zx.BF16: torch.bfloat16, zx.FP8_E4M3FN: torch.float8_e4m3fn}


class Scene:
    """Sequences with `new` new and `total` total tokens in a shuffled paged cache on the GPU.  What no
    sequence owns holds NaN; unused table entries are no page ids at all."""

    def __init__(self, dtype, H, G, D, T, new, total, C=None, seed=0, pad=0, layout="heads", scales=True, spread=1.0, width=1):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.dtype, self.H, self.G, self.D, self.T, self.C = dtype, H, G, D, T, C
        self.new, self.total = list(new), list(total)
        per = [-(-y // T) for y in total]
        W = max(per + [0]) + width
        n = sum(per) + 2
        self.n_pages = n
        perm = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((len(new), W), -7, dtype=torch.int32, device="cuda")
        self.table[:, -1] = 0x7FFFFFF0
        at = 0
        for b, m in enumerate(per):
            self.table[b, :m] = perm[at:at + m]
            at += m
        self.N = sum(new)
        self.rows = self.N + pad
        self.q_start = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor(total, dtype=torch.int32, device="cuda")
        fp8 = dtype == zx.FP8_E4M3FN
        sc = lambda: (0.02 + 0.05 * torch.rand(H, generator=g, device="cuda")) if fp8 and scales else None   # noqa: E731
        self.ks, self.vs = sc(), sc()
        pages = []
        for s in (self.ks, self.vs):
            x = spread * torch.randn((n, H, T, D), generator=g, device="cuda")
            x[..., 3] *= 5.0
            if s is not None:
                x = x / s[None, :, None, None]
            x = x.clamp(-448, 448)
            if layout == "tokens":
                p = torch.empty((n, T, H, D), dtype=RAW[dtype], device="cuda").transpose(1, 2)
            elif layout == "joint":     # keys and values of a page side by side
                if not pages:
                    self.both = torch.zeros((n, 2, H, T, D), dtype=RAW[dtype], device="cuda")
                p = self.both[:, len(pages)]
            else:
                p = torch.empty((n, H, T, D), dtype=RAW[dtype], device="cuda")
            p.copy_(x.to(TDT[dtype]).view(RAW[dtype]))
            pages.append(p)
        self.kraw, self.vraw = pages
        nan = 0x7FC0 if dtype == zx.BF16 else 0x7F
        dead = torch.ones((n, T), dtype=torch.bool, device="cuda")
        for b, y in enumerate(total):
            t = torch.arange(y, device="cuda")
            dead[self.table[b][t // T].long(), t % T] = False
        for p in pages:
            p.masked_fill_(dead[:, None, :, None], nan)
        self.bounds = None
        if C:
            x = self.kraw.view(TDT[dtype]).float().reshape(n, H, T // C, C, D)
            ok = ~torch.isnan(x)
            lo = torch.where(ok, x, torch.full_like(x, math.inf)).amin(3)
            hi = torch.where(ok, x, torch.full_like(x, -math.inf)).amax(3)
            self.bounds = torch.stack((lo, hi), 3).to(torch.bfloat16)
        self.q = torch.randn((self.rows, H * G, D), generator=g, device="cuda").to(torch.bfloat16)
        self.gen = g

    def cache(self):
        return zx.PagedKVCache(self.n_pages, self.H, self.D, self.T, self.dtype, block_tokens=self.C,
                               k=self.kraw.view(TDT[self.dtype]), v=self.vraw.view(TDT[self.dtype]), bounds=self.bounds,
                               k_scale=self.ks, v_scale=self.vs)

    def batch(self, **kw):
        return zx.PagedBatch(self.q_start, self.kv_len, self.table, **kw)

    def tokens(self, b, which):
        """The K or V rows of sequence b, [tokens, H, D] in 64 bits."""
        p, s = (self.kraw, self.ks) if which == "k" else (self.vraw, self.vs)
        t = torch.arange(self.total[b], device="cuda")
        x = p[self.table[b][t // self.T].long(), :, t % self.T].view(TDT[self.dtype]).float().double()
        return x if s is None else x * s.double()[None, :, None]


def see_mask(scene, b, causal=True, window=0):
    """[new, total]: which tokens each new token sees."""
    n, y = scene.new[b], scene.total[b]
    p = y - n + torch.arange(n, device="cuda")[:, None]
    t = torch.arange(y, device="cuda")[None, :]
    see = (p >= 0).expand(n, y).clone()
    if causal:
        see &= t <= p
    if window:
        see &= t > p - window
    return see


def reference(scene, see, scale=None, weight=None):
    """(out, lse, tolerance of out, tolerance of lse) of all packed rows, NaN behind the last
    sequence; `see` gives [new, H, total] truth values (or [new, total]) per sequence."""
    H, G, D = scene.H, scene.G, scene.D
    scale = D ** -0.5 if scale is None else scale
    shape = (scene.rows, H * G, D)
    out = torch.full(shape, math.nan, dtype=torch.float64, device="cuda")
    tol = torch.full(shape, math.nan, dtype=torch.float64, device="cuda")
    lse = torch.full(shape[:2], math.nan, dtype=torch.float64, device="cuda")
    ltol = torch.full(shape[:2], math.nan, dtype=torch.float64, device="cuda")
    for b in range(len(scene.new)):
        n, y = scene.new[b], scene.total[b]
        if n == 0:
            continue
        r = slice(int(sum(scene.new[:b])), int(sum(scene.new[:b])) + n)
        k, v = scene.tokens(b, "k"), scene.tokens(b, "v")
        m = see(b)
        if m.dim() == 2:
            m = m[:, None, :].expand(n, H, y)
        q = scene.q[r].double().view(n, H, G, D)
        for h in range(H):
            mh = m[:, h][:, None, :]
            mult = None if weight is None else weight(b)[:, h][:, None, :]
            for g in range(G):
                qh = q[:, h, g]
                s = (qh @ k[:, h].T) * scale                                       # [n, y]
                big = (qh.abs() @ k[:, h].abs().T) * scale
                s, big = s[:, None], big[:, None]
                s = torch.where(mh, s, torch.full_like(s, -math.inf))
                if y == 0:
                    out[r, h * G + g], lse[r, h * G + g], tol[r, h * G + g], ltol[r, h * G + g] = 0, -math.inf, 0, 0
                    continue
                mx = s.amax(-1, keepdim=True)
                e = torch.exp(s - torch.where(mx == -math.inf, torch.zeros_like(mx), mx))
                if mult is not None:
                    e = e * mult
                l = e.sum(-1, keepdim=True)
                w = e / torch.where(l > 0, l, torch.ones_like(l))
                vv = torch.where(mh.any(0).T, v[:, h], torch.zeros_like(v[:, h]))   # [y, D]: unseen values count for nothing
                o = (w[:, 0] @ vv)
                a = (w[:, 0] @ vv.abs())
                # scores: D products and sums in 32 bits, two scalings; weights: exp2 of 32-bit
                # arguments (as large as the score, in powers of two), one BF16 rounding
                ds = (torch.where(mh, big, torch.zeros_like(big)).amax(-1) * (D + 8) * 2.0 ** -24)      # [n, 1]
                dw = 2 * ds + (y + 64) * 2.0 ** -24 + 2.0 ** -21
                tol[r, h * G + g] = 2.0 ** -8 * o.abs() * 1.01 + (2.0 ** -8 * 1.01 + dw) * a + 1e-30
                out[r, h * G + g] = o
                x = (mx + torch.log(l))[:, 0, 0]
                lse[r, h * G + g] = x
                ltol[r, h * G + g] = torch.where(torch.isfinite(x), dw[:, 0] + x.abs() * 2.0 ** -21, torch.zeros_like(x))
    return out, lse, tol, ltol


def check_out(scene, got, lse, ref, before=None):
    out, rl, tol, ltol = ref
    n = scene.N
    d = (got[:n].double() - out[:n]).abs()
    bad = ~(d <= tol[:n])
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float((d / tol[:n].clamp(min=1e-30)).nan_to_num(9e9).max()))
    if lse is not None:
        inf = rl[:n] == -math.inf
        assert torch.equal(lse[:n] == -math.inf, inf)
        dl = torch.where(inf, torch.zeros_like(rl[:n]), lse[:n].double() - rl[:n]).abs()
        assert (dl <= ltol[:n]).all(), float((dl / ltol[:n].clamp(min=1e-30)).max())
    if before is not None:
        assert torch.equal(got[n:], before[n:])


def blocks_reference(scene, top_k, keep_first, keep_last):
    """int32 [rows, H, top_k] from the bounds, summed in 64 bits; -1 behind each list."""
    H, G, D, C, T = scene.H, scene.G, scene.D, scene.C, scene.T
    res = torch.full((scene.rows, H, top_k), -1, dtype=torch.int32)
    for b in range(len(scene.new)):
        r0 = sum(scene.new[:b])
        for i in range(scene.new[b]):
            p = scene.total[b] - scene.new[b] + i
            if p < 0:
                continue
            last = p // C
            j = torch.arange(last + 1, device="cuda")
            bd = scene.bounds[scene.table[b][j // (T // C)].long(), :, j % (T // C)].double()      # [blocks, H, 2, D]
            q = scene.q[r0 + i].double().view(H, G, D)
            for h in range(H):
                z = torch.maximum(q[h][:, None] * bd[None, :, h, 0], q[h][:, None] * bd[None, :, h, 1]).sum((0, 2))
                z[:keep_first] = math.inf
                if keep_last:
                    z[max(0, last + 1 - keep_last):] = math.inf
                top = torch.sort(z, descending=True, stable=True)[1][:top_k].sort()[0]
                res[r0 + i, h, :top.numel()] = top.to(torch.int32).cpu()
    return res


def listed_mask(scene, blocks):
    """see() for attention over block lists, and how often each token counts."""
    C = scene.C

    def count(b):
        n, y = scene.new[b], scene.total[b]
        r0 = sum(scene.new[:b])
        m = torch.zeros((n, scene.H, y), dtype=torch.float64, device="cuda")
        for i in range(n):
            for h in range(scene.H):
                for e in blocks[r0 + i, h].tolist():
                    if e < 0:
                        break
                    if e * C < y:
                        m[i, h, e * C:(e + 1) * C] += 1
        return m

    return (lambda b: (count(b) > 0) & see_mask(scene, b)[:, None, :]), count
