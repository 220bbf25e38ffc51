"""The choice of the next beams against its definition in 64 bits.

How far a score may be off.  An exponential's argument (x - top, times a rounded constant, rounded) is off by 3 |d| 2^-24, the
exponential by one step more (2^-23).  Weighted by the probabilities p, sum p |d| = H(p) - ln sum e^d <= ln vocab <= 17.  A thread adds up in 32 bits:
ten roundings a tile and two of the rescaled sum, eight tiles at most, each 2^-24 of the sum; so the ln of the sum is off by less than (3 * 17 + 2 + 96) 2^-24.  The
cases here are held to half of that, 72 * 2^-24 (their sums have one or two tiles a thread, 24 roundings).  What is in 64 bits adds nothing to that; the score
itself is rounded to 32 bits (2^-24 of itself)."""
import math

import pytest
import torch

import lossless_float_compression_amd as zx

pytestmark = pytest.mark.gpu
LSE = 72 * 2.0 ** -24
TYPES = (torch.bfloat16, torch.float16, torch.float32)


def totals(logits, scores, finished=None, end=None, allowed=None, scale=1.0):
    """Every candidate's score, [groups, beams, vocab] in 64 bits on the CPU; -inf: none."""
    x = logits.detach().cpu().double() * scale
    V = x.shape[2]
    if allowed is not None:
        t = torch.arange(V)
        bit = (allowed.cpu().long()[:, :, t // 32] >> (t % 32)) & 1
        x[bit == 0] = -math.inf
    s = scores.cpu().double()
    lse = torch.logsumexp(x, 2)
    x = torch.where((lse == -math.inf)[..., None], -math.inf, x - lse[..., None]) + s[..., None]
    if finished is not None:
        f = finished.cpu()
        x[f] = -math.inf
        x[..., end] = torch.where(f, s, x[..., end])
    x[(s == -math.inf) | s.isnan() | (s == math.inf)] = -math.inf
    x[x.isnan().any(2)] = -math.inf                  # NaN or +inf among the logits: no distribution
    return x


def check(r, logits, scores, M, weights=None, finished=None, end=None, allowed=None, scale=1.0, exact=False):
    """`exact`: equal candidates are equal in the kernel's arithmetic too, so the order is the definition's to the last place."""
    G, K, V = logits.shape
    tot = totals(logits, scores, finished, end, allowed, scale).view(G, K * V)
    w = torch.ones(G, K, dtype=torch.float64) if weights is None else weights.cpu().double()
    key = tot * w.repeat_interleave(V, 1)
    key[tot == -math.inf] = -math.inf
    order = torch.sort(key, dim=1, descending=True, stable=True)
    best, at = order[0][:, :M], order[1][:, :M]
    n = min(M, K * V)
    sc, par, tok, fin = (t.cpu() for t in r)
    assert sc.shape == par.shape == tok.shape == fin.shape == (G, M)
    some = torch.zeros((G, M), dtype=torch.bool)
    some[:, :n] = best > -math.inf
    assert torch.equal(par >= 0, some) and torch.equal(tok >= 0, some)
    assert bool((sc[~some] == -math.inf).all()) and bool((par[~some] == -1).all()) and bool((tok[~some] == -1).all()) and not bool(fin[~some].any())
    mine = (par.clamp(min=0) * V + tok.clamp(min=0)).long()
    for g in range(G):
        assert len(set(mine[g][some[g]].tolist())) == int(some[g].sum())
    mine = mine[:, :n]
    some, want = some[:, :n], torch.gather(tot, 1, mine)
    off = (sc[:, :n].double() - want)[some].abs()
    assert bool((off <= LSE + want[some].abs() * 2.0 ** -24).all()), off.max()
    if exact:
        assert torch.equal(mine[some], at[some])
    # the key at each place is the one that belongs there, as far as the kernel can tell
    wide = w.max(1)[0][:, None].expand(G, n)
    off = (torch.gather(key, 1, mine) - best)[some].abs()
    assert bool((off <= 2 * LSE * wide[some] + 1e-12).all()), off.max()
    done = torch.zeros_like(some) if end is None else tok[:, :n] == end
    if finished is not None:
        done = done | torch.gather(finished.cpu(), 1, par[:, :n].clamp(min=0).long())
    assert torch.equal(fin[:, :n], done & some)


def made(G, K, V, dtype, seed=0, pad=0, start=0, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn((G, K, V + pad + start), generator=g, device="cuda") * spread).to(dtype)
    x[:, :, :start] = math.nan
    x[:, :, start + V:] = math.nan
    return x[:, :, start:start + V], -10.0 * torch.rand((G, K), generator=g, device="cuda")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("G,K,V,M", [(1, 1, 1, 1), (1, 1, 1, 5), (2, 3, 1, 4), (1, 4, 3, 8), (3, 2, 31, 64), (1, 1, 64, 64), (2, 5, 513, 10), (1, 4, 4097, 8),
                                     (3, 7, 2047, 13), (1, 64, 700, 64), (5, 3, 50001, 6), (1, 2, 128256, 4), (40, 8, 9001, 16), (700, 2, 999, 3),
                                     (1, 1, 1 << 20, 64), (150, 8, 8191, 8), (33, 30, 2222, 60), (9000, 2, 5, 3), (1, 3, 70000, 64)])
def test_sizes(dtype, G, K, V, M):
    x, s = made(G, K, V, dtype, seed=V)
    check(zx.beam_select(x, s, M), x, s, M)


def test_default_number_of_candidates():
    x, s = made(2, 5, 100, torch.float32)
    r = zx.beam_select(x, s)
    assert r.scores.shape == (2, 5)
    check(r, x, s, 5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,start", [(1, 0), (3, 1), (0, 7), (8, 3)])
def test_rows_anywhere(dtype, pad, start):
    """Rows that begin at any element, with NaN between them."""
    x, s = made(3, 4, 5003, dtype, seed=pad, pad=pad, start=start)
    check(zx.beam_select(x, s, 9), x, s, 9)


@pytest.mark.parametrize("dtype", TYPES)
def test_strides(dtype):
    """Beams ahead of groups, one row for all beams, groups far apart."""
    x, s = made(4, 3, 1000, dtype)
    y = x.transpose(0, 1)
    assert not y.is_contiguous()
    check(zx.beam_select(y, s.view(3, 4), 5), y, s.view(3, 4), 5)
    y = x[:, :1].expand(4, 3, 1000)
    check(zx.beam_select(y, s, 5), y, s, 5)


def test_groups_beyond_32_bits():
    """Rows whose offsets pass 2^32 elements."""
    far = (1 << 31) + 4096 + 3
    big = torch.empty(2 * far + 3 * 3000, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((3, 2, 2900), (far, 3000, 1))
    y, s = made(3, 2, 2900, torch.bfloat16, seed=9)
    x.copy_(y)
    check(zx.beam_select(x, s, 7), y, s, 7)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("value", [0.0, -3.5])
@pytest.mark.parametrize("G,K,V,M", [(1, 1, 9000, 64), (2, 3, 20000, 17), (1, 64, 5000, 64), (300, 4, 700, 8)])
def test_all_equal(dtype, value, G, K, V, M):
    """Every candidate ties: the first tokens of the first beam; far more of them than the lists hold."""
    x = torch.full((G, K, V), value, dtype=dtype, device="cuda")
    s = torch.zeros((G, K), device="cuda")
    check(zx.beam_select(x, s, M), x, s, M, exact=True)


@pytest.mark.parametrize("dtype", TYPES)
def test_ties(dtype):
    """Few different values, zeros of both signs, equal rows."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randint(-2, 3, (6, 1, 7001), generator=g, device="cuda").to(dtype)
    x[(x == 0) & (torch.rand(x.shape, generator=g, device="cuda") < 0.5)] = -0.0
    x = x.expand(6, 4, 7001).contiguous()
    s = torch.full((6, 4), -1.5, device="cuda")
    check(zx.beam_select(x, s, 50), x, s, 50, exact=True)
    s[:, 2] = -1.0
    check(zx.beam_select(x, s, 50), x, s, 50, exact=True)
    # equal rows that begin at different offsets from 16 bytes
    y = torch.empty((6, 4, 7003), dtype=dtype, device="cuda")[:, :, 1:7002]
    y.copy_(x)
    s[:, 2] = -1.5
    check(zx.beam_select(y, s, 50), y, s, 50, exact=True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("up", [True, False])
def test_sorted_logits(dtype, up):
    """Runs of growing and falling values: the largest ones side by side."""
    V = 30000
    x = torch.linspace(-20, 20, V, device="cuda")
    x = (x if up else x.flip(0)).to(dtype).expand(2, 3, V).contiguous()
    s = torch.tensor([[0.0, -1.0, -2.0], [-5.0, -5.0, -1.0]], device="cuda")
    check(zx.beam_select(x, s, 64), x, s, 64, exact=True)


def test_many_equal_totals():
    """All 64 beams tie, with 64 candidates each in every part: more than the joining list holds."""
    x, _ = made(2, 1, 6000, torch.bfloat16, seed=3, spread=0.2)
    x = x.expand(2, 64, 6000).contiguous()
    s = torch.full((2, 64), -2.0, device="cuda")
    check(zx.beam_select(x, s, 64), x, s, 64, exact=True)


def bits_of(mask):
    G, K, V = mask.shape
    m = torch.nn.functional.pad(mask, (0, -V % 32)).view(G, K, -1, 32).long()
    w = (m << torch.arange(32, device=m.device)).sum(3)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32).contiguous()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("G,K,V,M", [(2, 4, 1000, 8), (3, 5, 4099, 11), (1, 2, 33, 40), (60, 8, 5000, 16)])
def test_masks(dtype, G, K, V, M):
    """NaN and infinities in masked places; beams with one token left, and with none."""
    x, s = made(G, K, V, dtype, seed=V)
    g = torch.Generator(device="cuda").manual_seed(1)
    mask = torch.rand((G, K, V), generator=g, device="cuda") < torch.rand((G, K, 1), generator=g, device="cuda")
    mask[0, 0] = False
    mask[0, 1] = False
    mask[0, 1, V - 1] = True
    odd = torch.tensor([math.nan, math.inf, -math.inf], device="cuda").to(dtype)
    x = torch.where(mask, x, odd[torch.randint(0, 3, x.shape, generator=g, device="cuda")])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = zx.beam_select(x, s, M, allowed=bits_of(mask), err=err)
    check(r, x, s, M, allowed=bits_of(mask))
    assert int(err) == 0
    # the same by -inf
    y = torch.where(mask, x, -math.inf)
    q = zx.beam_select(y, s, M, err=err)
    assert all(torch.equal(a, b) for a, b in zip(r, q)) and int(err) == 0


def test_nothing_to_choose_from():
    x = torch.full((2, 3, 777), -math.inf, device="cuda")
    s = torch.zeros((2, 3), device="cuda")
    x[1, 2, 5] = 1.0
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = zx.beam_select(x, s, 4, err=err)
    check(r, x, s, 4)
    assert r.parents.tolist() == [[-1] * 4, [2, -1, -1, -1]] and int(err) == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_beams_that_are_not_there(dtype):
    """A search begins with one beam; logits of the others are not looked at."""
    x, s = made(3, 4, 2000, dtype)
    x[:, 1:] = math.nan
    s[:, 1:] = -math.inf
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = zx.beam_select(x, s, 8, err=err, weights=torch.tensor([[1.0, 0.0, -1.0, math.nan]] * 3, device="cuda"))
    check(r, x, s, 8)
    assert int(err) == 0 and not bool(r.parents.any())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [1, 6, 13])
def test_finished_beams(dtype, M):
    x, s = made(9, 6, 1501, dtype, seed=M)
    g = torch.Generator(device="cuda").manual_seed(2)
    f = torch.rand((9, 6), generator=g, device="cuda") < 0.4
    f[0], f[1] = True, False
    x[f] = math.nan                                  # not looked at
    x[:, :, 7] = torch.where(f, x[:, :, 7].float(), 12.0).to(dtype)      # others want to end
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    check(zx.beam_select(x, s, M, finished=f, end=7, err=err), x, s, M, finished=f, end=7)
    w = torch.rand((9, 6), generator=g, device="cuda") + 0.1
    check(zx.beam_select(x, s, M, finished=f, end=7, weights=w, err=err), x, s, M, finished=f, end=7, weights=w)
    assert int(err) == 0
    y = torch.where(f[..., None], 0.0, x.float()).to(dtype)
    check(zx.beam_select(y, s, M, end=7), y, s, M, end=7)


@pytest.mark.parametrize("scale", [0.3, 1.0, 1.7, 1e-6, 1e6])
@pytest.mark.parametrize("dtype", TYPES)
def test_scale(dtype, scale):
    x, s = made(2, 4, 3001, dtype)
    if scale == 1e6:                                 # one logit takes all; the others' candidates are at -1e6 and beyond
        r = zx.beam_select(x, s, 4, scale=scale)
        tot = totals(x, s, scale=scale).view(2, -1)
        want = torch.gather(tot, 1, (r.parents.cpu() * 3001 + r.tokens.cpu()).long())
        assert torch.allclose(r.scores.cpu().double(), want, rtol=2.0 ** -22, atol=LSE) and torch.equal(want.max(1)[0], want[:, 0])
        return
    check(zx.beam_select(x, s, 8, scale=scale), x, s, 8, scale=scale)


@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float32))
def test_extreme_logits(dtype):
    """Values up to the type's largest: differences that pass it, one token that has all the probability."""
    top = torch.finfo(dtype).max
    x = torch.tensor([[[top, -top, 0.0, top, 1.0], [-top, -top, -top, -top, -top]]], device="cuda").to(dtype)
    s = torch.tensor([[-1.0, -2.0]], device="cuda")
    r = zx.beam_select(x, s, 7)
    assert r.parents.tolist() == [[0, 0, 1, 1, 1, 1, 1]] and r.tokens.tolist() == [[0, 3, 0, 1, 2, 3, 4]]
    want = torch.tensor([-1 - math.log(2)] * 2 + [-2 - math.log(5)] * 5)
    assert torch.allclose(r.scores.cpu()[0], want, rtol=0, atol=LSE + 4 * 2.0 ** -24)


@pytest.mark.parametrize("what", ["nan", "inf", "score nan", "score inf", "weight 0", "weight -1", "weight nan", "weight inf"])
def test_beams_that_are_left_out(what):
    x, s = made(3, 4, 3000, torch.bfloat16)
    w = torch.rand((3, 4), device="cuda") + 0.5
    good = zx.beam_select(x, s, 6, weights=w)
    if what in ("nan", "inf"):
        x[1, 2, 2999] = float(what)
    elif what.startswith("score"):
        s[1, 2] = float(what.split()[1])
    else:
        w[1, 2] = float(what.split()[1])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = zx.beam_select(x, s, 6, weights=w, err=err)
    assert int(err) == 4
    s2, w2 = s.clone(), w.clone()
    s2[1, 2], w2[1, 2] = -math.inf, 1.0
    check(r, x.nan_to_num(0, 0), s2, 6, weights=w2)
    assert all(torch.equal(a[[0, 2]], b[[0, 2]]) for a, b in zip(r, good))
    assert 2 not in r.parents[1].tolist()


def test_no_groups():
    r = zx.beam_select(torch.empty((0, 4, 100), device="cuda"), torch.empty((0, 4), device="cuda"), 8)
    assert r.parents.shape == (0, 8)


def test_in_place():
    """Scores and flags written over those that were read."""
    x, s = made(5, 6, 4000, torch.float16)
    f = torch.zeros((5, 6), dtype=torch.bool, device="cuda")
    f[:, 1] = True
    want = zx.beam_select(x, s, 6, finished=f, end=3)
    out = zx.Beams(s, torch.empty((5, 6), dtype=torch.int32, device="cuda"), torch.empty((5, 6), dtype=torch.int32, device="cuda"), f)
    r = zx.beam_select(x, s, 6, finished=f, end=3, out=out)
    assert r.scores is s and all(torch.equal(a, b) for a, b in zip(r, want))


def test_the_same_bits_every_time():
    x, s = made(16, 8, 40000, torch.bfloat16)
    a = zx.beam_select(x, s, 16)
    for _ in range(5):
        assert all(torch.equal(p, q) for p, q in zip(a, zx.beam_select(x, s, 16)))


def test_streams():
    """Behind work on the current stream, on another one, and on two at a time."""
    x, s = made(8, 8, 60000, torch.bfloat16)
    y, t = made(8, 8, 60000, torch.bfloat16, seed=5)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    w = torch.randn(4096, 4096, device="cuda")
    for _ in range(3):
        w = (w @ w).mul_(0.01)
    late = y + 0.0 * w[0, 0].clamp(0, 0).to(torch.bfloat16)
    p = zx.beam_select(x, s, 16, stream=a)
    q = zx.beam_select(late, t, 16, stream=b)
    torch.cuda.current_stream().wait_stream(a)
    torch.cuda.current_stream().wait_stream(b)
    check(p, x, s, 16)
    check(q, y, t, 16)


def test_graph():
    """Captured once, replayed on other logits, with eager calls between; two graphs at a time."""
    x, s = made(4, 4, 20000, torch.bfloat16)
    f = torch.zeros((4, 4), dtype=torch.bool, device="cuda")
    zx.beam_select(x, s, 8, finished=f, end=1)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = zx.beam_select(x, s, 8, finished=f, end=1)
        graphs.append((g, r))
    for i in range(4):
        y, t = made(4, 4, 20000, torch.bfloat16, seed=10 + i)
        x.copy_(y)
        s.copy_(t)
        f[:, 0] = i % 2 == 1
        for g, _ in graphs:
            g.replay()
        want = zx.beam_select(x, s, 8, finished=f, end=1)
        torch.cuda.synchronize()
        for _, r in graphs:
            assert all(torch.equal(a, b) for a, b in zip(r, want))
        check(want, x, s, 8, finished=f, end=1)


def test_outputs_are_written_whole():
    x, s = made(3, 4, 500, torch.bfloat16)
    out = zx.Beams(torch.full((3, 20), math.nan, device="cuda"), torch.full((3, 20), 99, dtype=torch.int32, device="cuda"),
                   torch.full((3, 20), 99, dtype=torch.int32, device="cuda"), torch.ones((3, 20), dtype=torch.bool, device="cuda"))
    x[1, :, 3:] = -math.inf                          # 12 candidates
    check(zx.beam_select(x, s, 20, out=out), x, s, 20)


def test_refusals():
    x, s = made(2, 4, 100, torch.bfloat16)
    i32 = dict(dtype=torch.int32, device="cuda")
    f = torch.zeros((2, 4), dtype=torch.bool, device="cuda")
    mk = lambda m: zx.Beams(torch.empty((2, m), device="cuda"), torch.empty((2, m), **i32), torch.empty((2, m), **i32),   # noqa: E731
                            torch.empty((2, m), dtype=torch.bool, device="cuda"))
    o = mk(4)
    bad = [lambda: zx.beam_select(x[0], s), lambda: zx.beam_select(x.double(), s), lambda: zx.beam_select(x.cpu(), s), lambda: zx.beam_select(x, s.cpu()),
           lambda: zx.beam_select(x, s.double()), lambda: zx.beam_select(x, s[:, :3]), lambda: zx.beam_select(x, s.t().contiguous().t()),
           lambda: zx.beam_select(x, s, 0), lambda: zx.beam_select(x, s, 65), lambda: zx.beam_select(x.transpose(1, 2), torch.zeros((2, 100), device="cuda")),
           lambda: zx.beam_select(x[:, :, :0], s), lambda: zx.beam_select(x[:, :0], s[:, :0]), lambda: zx.beam_select(x[:, :, ::2], s),
           lambda: zx.beam_select(x, s, finished=f), lambda: zx.beam_select(x, s, finished=f.int(), end=1), lambda: zx.beam_select(x, s, end=100),
           lambda: zx.beam_select(x, s, end=-1), lambda: zx.beam_select(x, s, weights=s.double()), lambda: zx.beam_select(x, s, scale=0.0),
           lambda: zx.beam_select(x, s, scale=math.nan), lambda: zx.beam_select(x, s, scale=math.inf), lambda: zx.beam_select(x, s, scale=-1.0),
           lambda: zx.beam_select(x, s, allowed=torch.zeros((2, 4, 3), **i32)), lambda: zx.beam_select(x, s, allowed=torch.zeros((2, 4, 4), device="cuda")),
           lambda: zx.beam_select(x, s, out=mk(5)), lambda: zx.beam_select(x, s, 5, out=o), lambda: zx.beam_select(x, s, out=o._replace(tokens=o.parents)),
           lambda: zx.beam_select(x, s, weights=s, out=o._replace(scores=s)), lambda: zx.beam_select(x, s, err=torch.zeros(1, device="cuda")),
           lambda: zx.beam_select(x.clone().requires_grad_(), s), lambda: zx.beam_select(x, s.clone().requires_grad_()),
           lambda: zx.beam_select(x, s, weights=s.clone().requires_grad_()),
           lambda: zx.beam_select(x, s, stream=0x1000)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    with torch.no_grad():
        zx.beam_select(x.clone().requires_grad_(), s)


@pytest.mark.parametrize("dtype", TYPES)
def test_the_smallest_scale(dtype):
    """All that may be taken are equal but for 1e-36 of their logits: logits of -inf and masked tokens have no share, any finite one has."""
    x, s = made(2, 3, 2501, dtype)
    x[0, 1, 5:] = -math.inf
    if dtype is not torch.float16:
        x[1, 1, ::2], x[1, 1, 1::2] = torch.finfo(dtype).max, -torch.finfo(dtype).max    # e^-680 apart
    mask = torch.ones((2, 3, 2501), dtype=torch.bool, device="cuda")
    mask[1, 2, :2400] = False
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = zx.beam_select(x, s, 12, allowed=bits_of(mask), scale=1e-36, err=err)
    assert int(err) == 0
    check(r, x, s, 12, allowed=bits_of(mask), scale=1e-36)
