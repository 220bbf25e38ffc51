"""Infinities, NaN and extreme scales in what the paged K/V cache's operators are given."""
import math
import sys

import pytest
import torch

import lossless_float_compression_amd as zx
from paged_util import Scene, check_out, reference, see_mask

pytestmark = pytest.mark.gpu
BF16, FP8 = zx.BF16, zx.FP8_E4M3FN
INF, NAN = math.inf, math.nan


@pytest.fixture(autouse=True)
def gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print(request.node.name, file=sys.stderr, flush=True)
    yield
    torch.cuda.synchronize()


def ranked(s, b, i, h, top_k, keep_first, keep_last):
    """The blocks of one new token and head by the definition in 64 bits, on the host: sum over heads and channels of
    max(q lo, q hi), NaN last, ties to the earlier block."""
    p = s.total[b] - s.new[b] + i
    last, per = p // s.C, s.T // s.C
    j = torch.arange(last + 1)
    bd = s.bounds.cpu()[s.table[b].cpu()[j // per].long(), h, j % per].double()                  # [blocks, 2, D]
    q = s.q[sum(s.new[:b]) + i].cpu().double().view(s.H, s.G, s.D)[h]
    z = torch.maximum(q[None] * bd[:, None, 0], q[None] * bd[:, None, 1]).sum((1, 2)).tolist()
    kept = lambda x: x < keep_first or x > last - keep_last   # noqa: E731
    order = sorted(range(last + 1), key=lambda x: (not kept(x), math.isnan(z[x]), 0.0 if math.isnan(z[x]) else -z[x], x))
    got = sorted(order[:top_k])
    return got + [-1] * (top_k - len(got))


def check_select(s, top_k, keep_first=1, keep_last=1, **kw):
    got = s.cache().select(s.q, s.batch(**kw), top_k, keep_first, keep_last).cpu()
    for b in range(len(s.new)):
        for i in range(s.new[b]):
            for h in range(s.H):
                want = ranked(s, b, i, h, top_k, keep_first, keep_last)
                assert got[sum(s.new[:b]) + i, h].tolist() == want, (b, i, h)


# what a channel's bounds become (smallest, largest): an overflowed key, two of them, nothing but NaN, nothing but infinities
ODD_BOUNDS = [(None, INF), (-INF, None), (-INF, INF), (INF, -INF), (INF, INF), (-INF, -INF), (None, NAN), (0.0, INF)]
# what the queries of the channel are in all heads of the group: one sign, the other, both, none, and odd ones
QUERIES = {"positive": lambda q: q.abs() + 0.125, "negative": lambda q: -q.abs() - 0.125, "both": lambda q: q, "zero": lambda q: q * 0.0,
           "infinite": lambda q: q * 0.0 + INF, "NaN": lambda q: q * NAN}


@pytest.mark.parametrize("queries", list(QUERIES))
@pytest.mark.parametrize("G,D,width,new", [(1, 128, 1, [1, 2]), (4, 64, 1, [1, 6]), (3, 256, 1, [1, 1]), (2, 128, 2600, [1, 1]), (4, 128, 2600, [5, 2]),
                                           (1, 256, 2600, [9, 1])])
def test_select_of_infinite_bounds(queries, G, D, width, new):
    s = Scene(BF16, 2, G, D, 32, new, [900, 333], C=16, seed=70, width=width)
    s.q[..., 5] = QUERIES[queries](s.q[..., 5])
    for n, (lo, hi) in enumerate(ODD_BOUNDS):
        for page in s.table[0, 3 + n:20:8].tolist() + s.table[1, n:n + 1].tolist():
            if lo is not None:
                s.bounds[page, :, n % 2, 0, 5] = lo
            if hi is not None:
                s.bounds[page, :, n % 2, 1, 5] = hi
    for top_k in (2, 9, 20, 40):
        check_select(s, top_k, max_q=max(new))
    check_select(s, 9, 0, 0, max_q=max(new))
    # the queries' other channels one way too, so that finite sums and their order are left to tell the blocks apart
    s.q[..., 6:] = s.q[..., 6:].abs()
    check_select(s, 12, max_q=max(new))


def test_appended_infinite_key_keeps_its_block():
    """A key that overflowed in one channel does not hide its block from queries that are negative there."""
    s = Scene(BF16, 1, 4, 128, 64, [1], [64 * 12], C=64, seed=71)
    c, b = s.cache(), s.batch()
    k = torch.zeros((12 * 64, 1, 128), dtype=torch.bfloat16, device="cuda")
    k[5 * 64 + 7, 0, 3] = INF
    k[5 * 64 + 9, 0, 10] = 100.0
    k[8 * 64 + 1, 0, 10] = 50.0
    whole = zx.PagedBatch(torch.tensor([0, 12 * 64], dtype=torch.int32, device="cuda"), s.kv_len, s.table)
    c.append(k, k, whole)
    s.q.zero_()
    s.q[..., 10] = 1.0
    s.q[..., 3] = -1.0
    assert c.select(s.q, b, 2, 0, 0).cpu().tolist() == [[[5, 8]]]


@pytest.mark.parametrize("width", [1, 3000])
def test_many_blocks_without_pages_and_with_nan(width):
    """Blocks that have no page come last with those whose bounds are NaN, the earlier first; err is set."""
    s = Scene(BF16, 1, 2, 64, 16, [1], [16 * 1000], C=16, seed=72, width=width)
    page = s.table[0, 700].item()
    s.bounds[page] = NAN
    s.table[0, 100:400] = -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = s.cache().select(s.q, s.batch(), 900, 0, 0, err=err).cpu()[0, 0].tolist()
    assert int(err.item()) == 4
    last = [j for j in range(1000) if 100 <= j < 400 or j == 700]
    assert got == sorted([j for j in range(1000) if j not in last] + last[:900 - 699])


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("T", [16, 32, 64])
@pytest.mark.parametrize("H,new,total,width", [(2, [1], [700], 1), (2, [7], [700], 1), (2, [170], [700], 1), (8, [170, 200], [700, 931], 1),
                                               (8, [170, 1, 190], [5000, 400, 3333], 900), (8, [300], [20011], 2)])
@pytest.mark.parametrize("window", [17, 50, 129])
def test_pages_behind_the_window_given_away(dtype, T, H, new, total, width, window):
    """Table entries of pages that no new token sees any more may hold anything; one page later is missed."""
    s = Scene(dtype, H, 4, 128, T, new, total, seed=73, width=width)
    c, b = s.cache(), s.batch()
    for causal in (True, False):
        want = c.attend(s.q, b, window=window, causal=causal)
        keep = s.table.clone()
        gone = [max(0, y - n - window + 1) // T for n, y in zip(new, total)]
        for i, n in enumerate(gone):
            s.table[i, :n] = -1
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = c.attend(s.q, b, window=window, causal=causal, err=err)
        assert int(err.item()) == 0 and torch.equal(got, want)
        s.table[0, gone[0]] = -1
        c.attend(s.q, b, window=window, causal=causal, err=err)
        assert int(err.item()) == 4
        s.table.copy_(keep)


@pytest.mark.parametrize("H,new,total", [(2, [1, 3], [700, 90]), (8, [300, 200], [400, 931])])
def test_scales_whose_product_is_below_any_float(H, new, total):
    """Scores of zero, by a scale and a k_scale that are both positive: every seen token weighs the same, masked ones nothing."""
    s = Scene(FP8, H, 4, 128, 64, new, total, seed=74)
    s.ks.fill_(1e-30)
    for causal, window in ((True, 0), (False, 0), (True, 100)):
        out, lse = torch.full_like(s.q, NAN), torch.full(s.q.shape[:2], NAN, device="cuda")
        s.cache().attend(s.q, s.batch(), scale=1e-20, causal=causal, window=window, out=out, lse=lse)
        check_out(s, out, lse, reference(s, lambda b: see_mask(s, b, causal, window), 1e-20))


def test_keys_and_values_that_share_pages_are_refused():
    both = torch.zeros((6, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
    pair = torch.zeros((5, 2, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
    for k, v in ((both[:5], both[:5]), (both[:5], both[1:]), (both[1:], both[:5]), (pair[:4, 0], pair[1:, 0]), (pair[:, 0], pair[:, 0])):
        with pytest.raises(ValueError, match="of their own"):
            zx.PagedKVCache(k.shape[0], 2, 128, 16, k=k, v=v)
    for k, v in ((both[:3], both[3:]), (pair[:, 0], pair[:, 1]), (pair[:, 1], pair[:, 0]), (pair[:3, 1], pair[2:, 0])):
        zx.PagedKVCache(k.shape[0], 2, 128, 16, k=k, v=v)


def test_a_cache_that_autograd_follows_is_refused():
    s = Scene(FP8, 2, 2, 128, 16, [1, 2], [30, 20], C=16, seed=76)
    b = s.batch()
    rows = torch.zeros((3, 2, 128), dtype=torch.bfloat16, device="cuda")
    want = s.cache().attend(s.q, b)
    s.ks.requires_grad_()
    c = s.cache()
    for call in (lambda: c.attend(s.q, b), lambda: c.select(s.q, b, 2), lambda: c.append(rows, rows, b)):
        with pytest.raises(ValueError, match="gradient"):
            call()
    rotary = zx.Rotary(64, inv_freq=torch.ones(32, dtype=torch.float64, device="cuda").requires_grad_())
    with pytest.raises(ValueError, match="gradient"):
        Scene(BF16, 2, 2, 128, 16, [1, 2], [30, 20], seed=76).cache().append(rows, rows, b, rotary=rotary)
    with torch.no_grad():
        assert torch.equal(c.attend(s.q, b), want)


@pytest.mark.parametrize("H,new,total", [(2, [1, 3], [700, 90]), (8, [300, 200], [400, 931])])
def test_a_scale_that_is_nan_shows(H, new, total):
    s = Scene(FP8, H, 4, 128, 64, new, total, seed=77)
    want = s.cache().attend(s.q, s.batch())
    s.ks[1] = NAN
    out = s.cache().attend(s.q, s.batch())
    assert torch.isnan(out[:, 4:8]).all() and torch.equal(out[:, :4], want[:, :4]) and torch.equal(out[:, 8:], want[:, 8:])
