"""Attention over the paged K/V cache against a plain form in 64 bits."""
import math
import sys

import pytest
import torch

import lossless_float_compression_amd as zx
from paged_util import Scene, check_out, listed_mask, reference, see_mask

pytestmark = pytest.mark.gpu
BF16, FP8 = zx.BF16, zx.FP8_E4M3FN


@pytest.fixture(autouse=True)
def gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print(request.node.name, file=sys.stderr, flush=True)
    yield
    torch.cuda.synchronize()


def run(scene, causal=True, window=0, scale=None, **kw):
    out = torch.full((scene.rows, scene.H * scene.G, scene.D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((scene.rows, scene.H * scene.G), 5.0, dtype=torch.float32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = out.clone()
    got = scene.cache().attend(scene.q, scene.batch(**kw), scale=scale, causal=causal, window=window, out=out, lse=lse, err=err)
    assert got is out
    ref = reference(scene, lambda b: see_mask(scene, b, causal, window), scale)
    check_out(scene, out, lse, ref, before)
    assert torch.equal(lse[scene.N:], torch.full_like(lse[scene.N:], 5.0))
    assert int(err.item()) == 0
    return out


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("H,G,D,T", [(8, 4, 128, 16), (2, 1, 64, 32), (1, 16, 128, 64), (3, 5, 128, 512), (2, 8, 64, 128), (2, 4, 256, 16),
                                     (1, 20, 64, 16), (1, 33, 128, 64)])
def test_single_tokens(dtype, H, G, D, T):
    run(Scene(dtype, H, G, D, T, [1] * 9, [1, 2, 15, 16, 17, 127, 128, 129, 1111], seed=1, pad=2))


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("H,G,D,T", [(2, 4, 128, 16), (2, 7, 64, 64), (1, 3, 256, 32)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 50), (True, 333), (False, 40)])
def test_few_new_tokens(dtype, H, G, D, T, causal, window):
    run(Scene(dtype, H, G, D, T, [4, 1, 2, 3, 4], [4, 300, 129, 3, 777], seed=2, pad=1), causal, window)


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("H,G,D,T", [(2, 4, 128, 16), (2, 1, 64, 32), (1, 3, 256, 16), (1, 5, 128, 256), (3, 2, 64, 64)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 100)])
def test_chunks(dtype, H, G, D, T, causal, window):
    run(Scene(dtype, H, G, D, T, [63, 130, 257, 65], [63, 700, 300, 64 * 9], seed=3, pad=3), causal, window)


@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_mixed_batch(dtype):
    run(Scene(dtype, 4, 4, 128, 32, [1, 200, 1, 0, 7, 90, 8, 9, 1], [999, 200, 1, 50, 40, 1500, 8, 300, 64], seed=4, pad=1))


def test_long_context_split():
    """One chunk over a long context: the tokens of a row tile are split between workgroups."""
    run(Scene(BF16, 2, 4, 128, 64, [100], [9000], seed=5))
    run(Scene(FP8, 1, 8, 128, 512, [33, 5], [20000, 700], seed=6))


@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_empty_rows(dtype):
    """Nothing in the cache, fewer tokens than queries, no new tokens, no sequences."""
    run(Scene(dtype, 2, 4, 128, 16, [1, 3, 0, 5, 2], [0, 1, 0, 2, 9], seed=7))
    run(Scene(dtype, 2, 4, 128, 16, [40, 70, 1], [0, 30, 0], seed=8))
    s = Scene(dtype, 2, 4, 128, 16, [1], [5], seed=9)
    c = s.cache()
    none = zx.PagedBatch(torch.zeros(1, dtype=torch.int32, device="cuda"), s.kv_len[:0].contiguous(), s.table[:0].contiguous())
    out = torch.full_like(s.q, 3.0)
    assert torch.equal(c.attend(s.q, none, out=out), torch.full_like(s.q, 3.0))
    assert c.attend(s.q[:0], s.batch()).shape == (0, 8, 128)


def test_large_scores_and_scale():
    run(Scene(BF16, 2, 4, 128, 16, [1, 40, 2], [500, 600, 9], seed=10, spread=30.0))
    run(Scene(BF16, 2, 4, 64, 16, [1, 40, 2], [500, 600, 9], seed=11), scale=2.5)
    run(Scene(FP8, 2, 4, 64, 16, [1, 40, 2], [500, 600, 9], seed=12, scales=False), scale=1e-6)


@pytest.mark.parametrize("layout", ["tokens", "joint"])
@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_page_layouts(dtype, layout):
    run(Scene(dtype, 3, 2, 128, 32, [1, 100, 3], [400, 333, 70], seed=13, layout=layout))


def test_strided_rows():
    """Queries that are a slice of a joint projection; output with gaps."""
    s = Scene(BF16, 2, 4, 128, 16, [1, 50, 3], [200, 333, 70], seed=14)
    wide = torch.zeros((s.rows, 8 + 4, 136), dtype=torch.bfloat16, device="cuda")
    wide[:, :8, :128] = s.q
    q = wide[:, :8, :128]
    hold = torch.full((s.rows, 16, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    out = hold[:, ::2]
    s.cache().attend(q, s.batch(), out=out)
    check_out(s, out, None, reference(s, lambda b: see_mask(s, b)))
    assert torch.equal(hold[:, 1::2], torch.full_like(hold[:, 1::2], 9.0))
    # one query row for all tokens (stride 0)
    one = s.q[:1].expand(s.rows, 8, 128)
    s.q = one.contiguous()
    assert torch.equal(s.cache().attend(one, s.batch()), s.cache().attend(s.q, s.batch()))


@pytest.mark.parametrize("new", [3, 100])
@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("window", [0, 20])
def test_masked_nan_does_not_leak(dtype, new, window):
    """An infinity or NaN in a token's key or value reaches the rows that see the token, no other."""
    s = Scene(dtype, 2, 4, 128, 16, [new], [150], seed=15)
    clean = s.cache().attend(s.q, s.batch(), window=window).double()
    at = 150 - new + new // 2                              # a new token: the earlier ones do not see it
    page, off = int(s.table[0, at // 16]), at % 16
    nan, inf = (0x7FC0, 0x7F80) if dtype == BF16 else (0x7F, None)
    seen = torch.arange(new, device="cuda") >= new // 2
    if window:
        seen &= torch.arange(new, device="cuda") < new // 2 + window
    for which, bits in (("v", nan), ("k", nan), ("v", inf), ("v", None if inf is None else inf - 0x8000)):
        if bits is None:
            continue
        pages = s.vraw if which == "v" else s.kraw
        old = pages[page, 1, off].clone()
        pages[page, 1, off, 5] = bits
        got = s.cache().attend(s.q, s.batch(), window=window).double()
        pages[page, 1, off] = old
        assert torch.equal(got[:, :4], clean[:, :4])
        assert torch.equal(got[~seen], clean[~seen])
        hit = got[seen][:, 4:]
        if which == "k":
            assert torch.isnan(hit).all()
        else:
            rest = [c for c in range(128) if c != 5]
            assert torch.equal(hit[..., rest], clean[seen][:, 4:][..., rest])
            x = hit[..., 5]
            if bits == nan:
                assert torch.isnan(x).all()
            else:
                assert (torch.isinf(x) & ((x > 0) == (bits > 0))).all()


def test_minus_infinite_scores():
    """Keys that make every score -inf or the lowest value: no NaN from the softmax itself."""
    s = Scene(BF16, 1, 2, 64, 16, [1, 40], [33, 60], seed=16)
    s.q.fill_(1.0)
    low = torch.finfo(torch.bfloat16).min
    s.kraw.view(torch.bfloat16)[s.table[0, 0].long(), :, :8, 0] = low
    s.kraw.view(torch.bfloat16)[s.table[1, 0].long(), :, :8, 0] = -math.inf
    out = s.cache().attend(s.q, s.batch())
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[1 + 20:]).all()


def test_bad_pages_and_lengths():
    """Page ids outside the cache stand for tokens that are not there; sequences whose lengths are out of
    range are left out.  Both are reported."""
    for new in ([1, 2, 1], [1, 70, 2]):
        s = Scene(BF16, 2, 4, 128, 16, new, [100, 90, 50], seed=17)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        good = s.cache().attend(s.q, s.batch(), err=err)
        assert int(err.item()) == 0
        s.table[1, 2] = s.n_pages
        out = s.cache().attend(s.q, s.batch(), err=err)
        assert int(err.item()) == 4

        def see(b):
            m = see_mask(s, b)
            if b == 1:
                m[:, 32:48] = False
            return m
        tab = s.table.clone()
        s.table[1, 2] = s.table[1, 1]     # for the reference only: these tokens are masked
        check_out(s, out, None, reference(s, see))
        s.table.copy_(tab)
        s.table[1, 2] = -5
        assert torch.equal(s.cache().attend(s.q, s.batch()), out)
        for change in (lambda: s.kv_len.__setitem__(1, -3), lambda: s.kv_len.__setitem__(1, 1 << 29),
                       lambda: s.q_start.__setitem__(1, s.rows + 5), lambda: s.q_start.__setitem__(1, -2)):
            keep = s.q_start.clone(), s.kv_len.clone()
            change()
            err.zero_()
            out = torch.full_like(good, 3.0)
            s.cache().attend(s.q, s.batch(), out=out, err=err)
            assert int(err.item()) == 4
            assert torch.equal(out[-new[2]:], good[-new[2]:])
            s.q_start.copy_(keep[0])
            s.kv_len.copy_(keep[1])
        err.zero_()
        out = torch.full_like(good, 3.0)
        s.cache().attend(s.q, s.batch(max_kv=95), out=out, err=err)
        assert int(err.item()) == 4 and torch.equal(out[:1], torch.full_like(out[:1], 3.0))
        err.zero_()
        s.cache().attend(s.q, s.batch(max_q=1), out=out, err=err)
        assert int(err.item()) == 4


def test_overlapping_sequences_stay_in_bounds():
    """Row ranges that overlap are the caller's mistake; nothing outside the arrays is touched."""
    s = Scene(BF16, 2, 4, 128, 16, [8] * 8, [600] * 8, seed=18)
    s.q_start[1::2] = 64
    s.q_start[0::2] = 0
    guard = torch.full((64 + 64, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    s.cache().attend(s.q, s.batch(), out=guard[:64])
    assert torch.equal(guard[64:], torch.full_like(guard[64:], 3.0))


def test_offsets_past_32_bits():
    """Pages more than 4 GiB into the cache."""
    n = 4800
    k = torch.empty((n, 8, 512, 256), dtype=torch.uint8, device="cuda")
    v = torch.empty((n, 8, 512, 256), dtype=torch.uint8, device="cuda")
    s = Scene(FP8, 8, 2, 256, 512, [1, 40], [900, 700], seed=19)
    far = torch.tensor([n - 1 - i for i in range(s.n_pages)], device="cuda")
    k[far], v[far] = s.kraw, s.vraw
    want = s.cache().attend(s.q, s.batch())
    table = torch.where((s.table >= 0) & (s.table < s.n_pages), n - 1 - s.table, s.table)
    c = zx.PagedKVCache(n, 8, 256, 512, FP8, k=k.view(torch.float8_e4m3fn), v=v.view(torch.float8_e4m3fn), k_scale=s.ks, v_scale=s.vs)
    got = c.attend(s.q, zx.PagedBatch(s.q_start, s.kv_len, table))
    assert torch.equal(got, want)


def lists(s, kind, n):
    g = torch.Generator().manual_seed(5)
    b = torch.full((s.rows, s.H, n), -1, dtype=torch.int32)
    for q in range(len(s.new)):
        r0 = sum(s.new[:q])
        for i in range(s.new[q]):
            last = max(0, (s.total[q] - s.new[q] + i) // s.C)
            for h in range(s.H):
                k = {"some": min(n, last + 1), "none": 0, "short": min(n, 1 + (i + h) % 3, last + 1)}[kind if kind in ("some", "none", "short") else "some"]
                pick = torch.randperm(last + 1, generator=g)[:k].to(torch.int32)
                if kind == "twice" and k:
                    pick = torch.cat((pick, pick))[:n]
                if kind == "past":      # blocks behind the sequence's end, and absurd ones
                    pick = torch.cat((torch.tensor([last + 3, 0x7FFFFFFF], dtype=torch.int32), pick))[:n]
                b[r0 + i, h, :pick.numel()] = pick
    return b.cuda()


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("kind", ["some", "none", "short", "twice", "past"])
@pytest.mark.parametrize("H,G,D,T,C,n", [(2, 4, 128, 64, 64, 5), (2, 8, 64, 32, 16, 70), (1, 20, 128, 128, 32, 3), (1, 2, 256, 16, 16, 9)])
def test_block_lists(dtype, kind, H, G, D, T, C, n):
    s = Scene(dtype, H, G, D, T, [1, 6, 0, 1], [900, 333, 20, 7], C=C, seed=20, pad=1)
    b = lists(s, kind, n)
    see, count = listed_mask(s, b)
    out = torch.full_like(s.q, 2.0)
    lse = torch.zeros((s.rows, H * G), device="cuda")
    before = out.clone()
    s.cache().attend(s.q, s.batch(), blocks=b, out=out, lse=lse)
    check_out(s, out, lse, reference(s, see, weight=count), before)


def test_all_blocks_equal_dense():
    s = Scene(BF16, 2, 4, 128, 64, [1, 1], [1000, 64], C=64, seed=21)
    b = torch.arange(16, dtype=torch.int32, device="cuda").expand(2, 2, 16).contiguous()
    ref = reference(s, lambda q: see_mask(s, q))
    check_out(s, s.cache().attend(s.q, s.batch(), blocks=b), None, ref)


def test_same_bits_streams_and_graphs():
    """Equal inputs give equal bits; on another stream after the work that makes the inputs; in a graph that
    is replayed with rewritten lengths, with eager work between; two graphs replayed side by side."""
    s = Scene(BF16, 4, 4, 128, 32, [1, 60, 3], [2000, 1500, 400], C=32, seed=22)
    c, b = s.cache(), s.batch()
    want = c.attend(s.q, b)
    for _ in range(3):
        assert torch.equal(c.attend(s.q, b), want)
    side = torch.cuda.Stream()
    q2 = torch.zeros_like(s.q)
    big = torch.randn(4096, 4096, device="cuda")
    for _ in range(4):
        big = big @ big * 1e-3
    q2.copy_(s.q)                           # late on the current stream
    got = c.attend(q2, b, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    # graphs
    o1, o2 = torch.zeros_like(s.q), torch.zeros_like(s.q)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g1):
        c.attend(s.q, b, out=o1)
    with torch.cuda.graph(g2):
        c.attend(s.q, b, out=o2)
    for total in ([2000, 1500, 400], [64, 1400, 3], [0, 60, 333]):
        s.kv_len.copy_(torch.tensor(total, dtype=torch.int32))
        want = c.attend(s.q, b)
        o1.zero_()
        o2.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            g2.replay()
        g1.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, want) and torch.equal(o2, want)


def test_default_output_and_shapes():
    s = Scene(BF16, 2, 4, 128, 16, [1, 5], [30, 70], seed=23)
    out = s.cache().attend(s.q, s.batch(max_q=5, max_kv=70))
    assert out.shape == s.q.shape and out.dtype == torch.bfloat16
    check_out(s, out, None, reference(s, lambda b: see_mask(s, b)))
