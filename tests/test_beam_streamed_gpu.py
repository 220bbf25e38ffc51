"""The choice of the next beams where rows are streamed, in parts of 2 to 8 tiles, against its definition in 64 bits (on the GPU, by
sorting whole rows: the sizes are a serving batch's).

How far a score may be off, in units of 2^-24: the argument of an exponential (x - top, times a rounded constant, rounded) 3 |d|, with sum p |d| <=
ln vocab < 12 whatever way it takes over the running maxima; the exponential 2 (a step of the type); for each of up to eight tiles ten sums, a rescaling
exponential (2) and its product (1); the last rescaling 3.  So 3 * 12 + 2 + 8 * 13 + 3 = 145 units for the ln of the sum; what follows is in 64
bits, and the score is rounded to 32 (a unit of itself).  Which tokens a beam gives, and their order, does not depend on the sum: that is exact."""
import math

import pytest
import torch

import lossless_float_compression_amd as zx
from beam_shapes import STREAMED
from test_beam_select_gpu import TYPES, bits_of, made

pytestmark = pytest.mark.gpu
LSE = 145 * 2.0 ** -24
ALL = [(t, s[:4]) for t in TYPES for s in STREAMED[t]]
SOME = [(t, STREAMED[t][i][:4]) for t in TYPES for i in (0, 1, 4, 6, 8, 9)]       # 2, 2 (two parts), 5, 7, 8, 8 tiles
NAMES = dict(ids=lambda a: "x".join(map(str, a[:3])) if isinstance(a, tuple) else str(a).replace("torch.", ""))


def check(r, x, s, M, weights=None, finished=None, end=None, mask=None, scale=1.0, exact=False):
    """`exact`: beams that are equal are equal in the kernel's arithmetic too, so parents are the definition's to the last place."""
    G, K, V = x.shape
    n = min(M, V)
    y = x if mask is None else torch.where(mask, x, -math.inf)
    gone = y.isnan().any(2) | (y == math.inf).any(2) | (s == -math.inf)
    if finished is not None:
        gone |= finished
    y = torch.where(gone[..., None], -math.inf, y)
    top, at = torch.sort(y.float(), dim=2, descending=True, stable=True)
    top, at = top[..., :n].double() * scale, at[..., :n].clone()
    tot = s.double()[..., None] + (top - torch.logsumexp(y.double() * scale, 2)[..., None])
    tot[gone] = -math.inf
    tot = torch.where(tot.isnan(), -math.inf, tot)                       # nothing may be taken
    if finished is not None:
        tot[..., 0] = torch.where(finished, s.double(), tot[..., 0])
        at[..., 0] = torch.where(finished, end, at[..., 0])
    w = torch.ones_like(s, dtype=torch.float64) if weights is None else weights.double()
    key = torch.where(tot == -math.inf, -math.inf, tot * w[..., None]).view(G, K * n)
    best, order = torch.sort(key, dim=1, descending=True, stable=True)
    m = min(M, K * n)
    best, order = best[:, :m], order[:, :m]
    some = torch.nn.functional.pad(best > -math.inf, (0, M - m))
    sc, par, tok, fin = r
    assert torch.equal(par >= 0, some) and torch.equal(tok >= 0, some)
    assert bool((sc[~some] == -math.inf).all()) and not bool(fin[~some].any())
    sc, par, tok, fin, some = sc[:, :m], par[:, :m].clamp(min=0).long(), tok[:, :m].long(), fin[:, :m], some[:, :m]
    nth = (par[:, :, None] == par[:, None, :]).tril(-1).sum(2)           # a candidate's place among its beam's
    assert bool((nth[some] < n).all())
    flat = par * n + nth.clamp(max=n - 1)
    want = torch.gather(at.view(G, -1), 1, flat)
    assert torch.equal(tok[some], want[some])
    if exact:
        assert torch.equal(flat[some], order[some])
    total = torch.gather(tot.view(G, -1), 1, flat)
    off = (sc.double() - total)[some].abs()
    assert bool((off <= LSE + total[some].abs() * 2.0 ** -24).all()), off.max()
    off = (torch.gather(key, 1, flat) - best)[some].abs()
    assert bool((off <= 2 * LSE * w.max(1)[0][:, None].expand(G, m)[some] + 1e-12).all()), off.max()
    done = torch.zeros_like(some) if end is None else tok == end
    if finished is not None:
        done = done | torch.gather(finished, 1, par)
    assert torch.equal(fin[some], done[some])


@pytest.mark.parametrize("dtype,shape", ALL, **NAMES)
def test_sizes(dtype, shape):
    G, K, V, M = shape
    x, s = made(G, K, V, dtype, seed=V)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    check(zx.beam_select(x, s, M, err=err), x, s, M)
    assert int(err) == 0


@pytest.mark.parametrize("dtype,shape", SOME, **NAMES)
def test_masks(dtype, shape):
    """NaN and infinities in masked places; beams with one token left at an end of a part, and with none."""
    G, K, V, M = shape
    x, s = made(G, K, V, dtype, seed=V)
    g = torch.Generator(device="cuda").manual_seed(1)
    mask = torch.rand((G, K, V), generator=g, device="cuda") < torch.rand((G, K, 1), generator=g, device="cuda") ** 4
    for i, t in enumerate((V - 1, 0, V // 2, V - 2, min(V - 1, 16384), min(V - 1, 8191))):
        mask[i] = False
        mask[i, K - 1, t] = True
    mask[6] = False
    odd = torch.tensor([math.nan, math.inf, -math.inf], device="cuda").to(dtype)
    x = torch.where(mask, x, odd[torch.randint(0, 3, x.shape, generator=g, device="cuda")])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = zx.beam_select(x, s, M, allowed=bits_of(mask), err=err)
    check(r, x, s, M, mask=mask)
    assert int(err) == 0 and r.tokens[0, 0] == V - 1 and r.parents[6, 0] == -1
    y = torch.where(mask, x, -math.inf)                                  # the same by -inf
    q = zx.beam_select(y, s, M, err=err)
    assert all(torch.equal(a, b) for a, b in zip(r, q)) and int(err) == 0


@pytest.mark.parametrize("value", [0.0, -3.5])
@pytest.mark.parametrize("dtype,shape", SOME, **NAMES)
def test_all_equal(dtype, shape, value):
    """Every thread of every tile reaches the edge: the first tokens of the first beam."""
    G, K, V, M = shape
    x = torch.full((G, K, V), value, dtype=dtype, device="cuda")
    s = torch.zeros((G, K), device="cuda")
    check(zx.beam_select(x, s, M), x, s, M, exact=True)


@pytest.mark.parametrize("up", [True, False])
@pytest.mark.parametrize("dtype,shape", SOME, **NAMES)
def test_sorted_logits(dtype, shape, up):
    """Growing and falling values, in runs of equal ones in 16 bits; 64 candidates."""
    G, K, V, _ = shape
    x = torch.linspace(-20, 20, V, device="cuda")
    x = (x if up else x.flip(0)).to(dtype).expand(G, K, V).contiguous()
    s = -10.0 * torch.rand((G, K), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    check(zx.beam_select(x, s, 64), x, s, 64)


@pytest.mark.parametrize("length,count", [(1, 300), (32, 40), (3000, 1), (700, 7), (9000, 1)])
@pytest.mark.parametrize("dtype,shape", SOME, **NAMES)
def test_plateaus(dtype, shape, length, count):
    """Stretches of one largest value anywhere, over the ends of pieces, tiles and parts: more of them than lists hold, in few threads'
    shares or in many; zeros of both signs."""
    G, K, V, _ = shape
    x, s = made(G, K, V, dtype, seed=length, spread=0.5)
    x = x.clamp(max=2.0) - 3.0
    g = torch.Generator(device="cuda").manual_seed(count)
    step = torch.zeros((G, K, V + 1), dtype=torch.int32, device="cuda")
    start = torch.randint(0, V, (G, K, count), generator=g, device="cuda")
    start[0, 0, 0] = 0
    start[0, 1 % K, 0] = V - 1
    one = torch.ones_like(start, dtype=torch.int32)
    step.scatter_add_(2, start, one)
    step.scatter_add_(2, (start + length).clamp(max=V), -one)
    high = step.cumsum(2)[..., :V] > 0
    zero = torch.where(torch.rand((V,), generator=g, device="cuda") < 0.5, 0.0, -0.0).to(dtype)
    x = torch.where(high, zero, x)
    check(zx.beam_select(x, s, 64), x, s, 64)


@pytest.mark.parametrize("pad,start", [(1, 0), (2, 5)])
@pytest.mark.parametrize("dtype,shape", SOME, **NAMES)
def test_finished_absent_and_weighted(dtype, shape, pad, start):
    """Rows that begin at any element with NaN between them; beams that are finished or not there (their logits are not looked at), weights, a scale."""
    G, K, V, M = shape
    x, s = made(G, K, V, dtype, seed=V, pad=pad, start=start)
    g = torch.Generator(device="cuda").manual_seed(2)
    f = torch.rand((G, K), generator=g, device="cuda") < 0.3
    s[torch.rand((G, K), generator=g, device="cuda") < 0.3] = -math.inf
    x[f | (s == -math.inf)] = math.nan
    end = V - 3
    x[..., end] = torch.where(x[..., end].isnan(), x[..., end].float(), 12.0).to(dtype)         # others want to end
    w = torch.rand((G, K), generator=g, device="cuda") + 0.1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = zx.beam_select(x, s, M, finished=f, end=end, weights=w, scale=0.7, err=err)
    assert int(err) == 0
    check(r, x, s, M, finished=f & (s > -math.inf), end=end, weights=w, scale=0.7)


@pytest.mark.parametrize("what", [math.nan, math.inf])
@pytest.mark.parametrize("dtype,shape", SOME, **NAMES)
def test_beams_that_are_left_out(dtype, shape, what):
    """One NaN or +inf anywhere in a row: the beam is left out and reported, the others are as they were."""
    G, K, V, M = shape
    x, s = made(G, K, V, dtype, seed=5)
    good = zx.beam_select(x, s, M)
    for i, t in enumerate((0, V - 1, V // 2, V - 9, V // 3)):
        x[i, i % K, t] = what
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = zx.beam_select(x, s, M, err=err)
    assert int(err) == 4
    check(r, x, s, M)
    assert all(torch.equal(a[5:], b[5:]) for a, b in zip(r, good))


@pytest.mark.parametrize("dtype", TYPES)
def test_graph(dtype):
    """Captured once, replayed on other logits, with eager calls between."""
    G, K, V, M, _, _ = STREAMED[dtype][6]
    x, s = made(G, K, V, dtype)
    zx.beam_select(x, s, M)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = zx.beam_select(x, s, M)
    for i in range(3):
        y, t = made(G, K, V, dtype, seed=20 + i)
        x.copy_(y)
        s.copy_(t)
        g.replay()
        want = zx.beam_select(x, s, M)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(r, want))
        check(r, x, s, M)


@pytest.mark.parametrize("scale,spread", [(1e-30, 3.0), (1.0, 1e-25)])
@pytest.mark.parametrize("shape", [(2, 64, 6000, 64), (1, 3, 70000, 64), (300, 4, 700, 8), (5, 40, 20000, 33), (64, 8, 64128, 16)])
@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float32))
def test_scores_that_are_equal_in_64_bits(dtype, shape, scale, spread):
    """Logits differ, scores do not: the earlier beam, then the larger logit; as many candidates as there are, though none of them stands out."""
    G, K, V, M = shape
    x, _ = made(G, K, V, dtype, seed=V, spread=spread)
    s = torch.zeros((G, K), device="cuda")
    s[::2, 0] = -1.0
    check(zx.beam_select(x, s, M, scale=scale), x, s, M, scale=scale, exact=True)
