"""Attention over the paged K/V cache at the sizes that serving uses: long prompts, batches of hundreds of
sequences, many heads.  Every row has to be written; sampled rows are compared with the 64-bit form."""
import math
import random
import sys

import pytest
import torch

import lossless_float_compression_amd as zx
from paged_util import Scene

pytestmark = pytest.mark.gpu
BF16, FP8 = zx.BF16, zx.FP8_E4M3FN


@pytest.fixture(autouse=True)
def gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print(request.node.name, file=sys.stderr, flush=True)
    yield
    torch.cuda.synchronize()


def check_rows(s, out, lse, b, rows, causal=True, window=0):
    """Rows `rows` of sequence b, all heads.  The tolerance counts what paged_util.reference counts."""
    H, G, D = s.H, s.G, s.D
    n, y = s.new[b], s.total[b]
    i = torch.tensor(rows, device="cuda")
    r = sum(s.new[:b]) + i
    k, v = (s.tokens(b, x).permute(1, 2, 0).contiguous() if x == "k" else s.tokens(b, x).permute(1, 0, 2).contiguous() for x in "kv")
    q = s.q[r].double().view(len(rows), H, G, D).permute(1, 0, 2, 3).reshape(H, -1, D)
    p = (y - n + i)[:, None]
    t = torch.arange(y, device="cuda")[None, :]
    see = (t <= p) if causal else (t >= 0).expand(len(rows), y)
    if window:
        see = see & (t > p - window)
    see = see[None, :, None, :].expand(H, len(rows), G, y).reshape(H, -1, y)
    sc = (q @ k) * D ** -0.5
    big = ((q.abs() @ k.abs()) * D ** -0.5).masked_fill(~see, 0.0).amax(-1, keepdim=True)
    sc = sc.masked_fill(~see, -math.inf)
    want_lse = torch.logsumexp(sc, -1, keepdim=True)
    w = torch.exp(sc - want_lse)
    o, a = w @ v, w @ v.abs()
    dw = 2 * big * (D + 8) * 2.0 ** -24 + (y + 64) * 2.0 ** -24 + 2.0 ** -21
    tol = 2.0 ** -8 * o.abs() * 1.01 + (2.0 ** -8 * 1.01 + dw) * a + 1e-30
    ltol = dw + want_lse.abs() * 2.0 ** -21
    got = out[r].double().view(len(rows), H, G, D).permute(1, 0, 2, 3).reshape(H, -1, D)
    gl = lse[r].double().view(len(rows), H, G).permute(1, 0, 2).reshape(H, -1, 1)
    bad = ~((got - o).abs() <= tol)
    assert not bad.any(), (b, int(bad.sum()), bad.nonzero()[:4].tolist())
    assert ((gl - want_lse).abs() <= ltol).all(), b


def run(s, sample, causal=True, window=0, **kw):
    out = torch.full_like(s.q, math.nan)
    lse = torch.full(s.q.shape[:2], math.nan, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    s.cache().attend(s.q, s.batch(**kw), causal=causal, window=window, out=out, lse=lse, err=err)
    assert int(err.item()) == 0
    left = ~(torch.isfinite(out).all(-1) & torch.isfinite(lse))[:s.N]
    assert not left.any(), (int(left.sum()), "rows and heads were not written, the first and last of them", left.nonzero()[[0, -1]].tolist())
    assert torch.isnan(out[s.N:]).all() and torch.isnan(lse[s.N:]).all()
    for b, rows in sample:
        check_rows(s, out, lse, b, rows, causal, window)


@pytest.mark.parametrize("dtype,H,G,D,n", [(BF16, 8, 4, 128, 16384), (FP8, 8, 4, 128, 16384), (BF16, 8, 4, 128, 12290), (BF16, 8, 8, 128, 8192),
                                           (FP8, 8, 8, 128, 8192), (BF16, 8, 4, 256, 8192), (FP8, 4, 7, 64, 16384), (BF16, 32, 1, 128, 16384)])
def test_long_prompts(dtype, H, G, D, n):
    s = Scene(dtype, H, G, D, 64, [n], [n], seed=60, pad=1)
    rng = random.Random(n)
    run(s, [(0, [0, 1, 4095, n // 4, n - 1] + [rng.randrange(n) for _ in range(11)])], max_q=n, max_kv=n)


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("b,n,over", [(4, 4096, 8192), (8, 2048, 6000)])
def test_batches_of_pieces(dtype, b, n, over):
    s = Scene(dtype, 8, 4, 128, 512, [n] * b, [over] * b, seed=61)
    run(s, [(i, [0, n // 2, n - 1]) for i in range(b)])
    run(s, [(i, [0, n - 1]) for i in range(b)], window=1000)


@pytest.mark.parametrize("dtype,H,G,D,n", [(BF16, 8, 4, 128, 512), (FP8, 8, 4, 128, 512), (BF16, 8, 4, 128, 385), (BF16, 32, 1, 128, 128),
                                           (FP8, 32, 1, 128, 97), (BF16, 16, 1, 256, 128), (FP8, 16, 1, 256, 65), (BF16, 4, 7, 64, 1000)])
@pytest.mark.parametrize("kind", ["equal", "ragged", "one long"])
def test_many_single_tokens(dtype, H, G, D, n, kind):
    rng = random.Random(n)
    if kind == "equal":
        total = [1000] * n
    elif kind == "ragged":
        total = [max(1, int(2048 * 2.0 ** -rng.uniform(0, 5))) for _ in range(n)]
    else:
        total = [rng.randint(1, 100) for _ in range(n - 1)] + [30000]
    s = Scene(dtype, H, G, D, 64, [1] * n, total, seed=62, pad=1)
    picks = sorted({0, 1, n // 2, n - 2, n - 1} | {rng.randrange(n) for _ in range(20)})
    run(s, [(b, [0]) for b in picks], max_q=1, max_kv=max(total))


def test_long_ones_among_many():
    """One sequence in 16 is long; a few new tokens each; prompts and single tokens of hundreds of users in one call."""
    rng = random.Random(5)
    total = [16384 if i % 16 == 0 else rng.randint(600, 900) for i in range(300)]
    s = Scene(BF16, 8, 4, 128, 16, [1] * 300, total, seed=63)
    run(s, [(b, [0]) for b in (0, 1, 16, 100, 272, 288, 298, 299)])
    new = [rng.choice((1, 1, 1, 2, 5)) for _ in range(700)]
    s = Scene(FP8, 4, 2, 64, 32, new, [x + rng.randint(0, 900) for x in new], seed=64, pad=2)
    run(s, [(b, [0, new[b] - 1]) for b in range(0, 700, 33)] + [(699, [0])])
    new = [rng.choice((1, 1, 1, 400)) for _ in range(150)]
    s = Scene(BF16, 8, 4, 128, 64, new, [x + rng.randint(0, 6000) for x in new], seed=65)
    run(s, [(b, [0, new[b] - 1]) for b in range(0, 150, 7)] + [(149, [0])])
