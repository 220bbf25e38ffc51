"""Appending to the paged K/V cache, selecting blocks of it, and a run of all operators together."""
import math
import sys

import pytest
import torch

import lossless_float_compression_amd as zx
from paged_util import RAW, TDT, Scene, blocks_reference, check_out, listed_mask, reference, see_mask

pytestmark = pytest.mark.gpu
BF16, FP8 = zx.BF16, zx.FP8_E4M3FN


@pytest.fixture(autouse=True)
def gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print(request.node.name, file=sys.stderr, flush=True)
    yield
    torch.cuda.synchronize()


def turned(x, pos, rot):
    """(rotated rows, sum of the magnitudes that make each) in 64 bits; x [n, heads, D]."""
    x = x.double()
    if rot is None:
        return x, x.abs()
    a = pos.double()[:, None, None] * rot.inv_freq[None, None, :]
    c, s = torch.cos(a) * rot.magnitude, torch.sin(a) * rot.magnitude
    r = rot.dims
    ia, ib = (slice(0, r, 2), slice(1, r, 2)) if rot.interleaved else (slice(0, r // 2), slice(r // 2, r))
    y, m = x.clone(), x.abs()
    y[..., ia], y[..., ib] = x[..., ia] * c - x[..., ib] * s, x[..., ib] * c + x[..., ia] * s
    m[..., ia] = m[..., ib] = (x[..., ia].abs() + x[..., ib].abs()) * rot.magnitude
    return y, m


def near(got, want, made_of, dtype):
    """One rounding to the stored type, and 32-bit rotation: 2^-20 of what goes into the sum."""
    fuzz = made_of * 2.0 ** -20
    if dtype == FP8:
        want = want.clamp(-448, 448)
        tol = torch.maximum(want.abs() * 2.0 ** -4, torch.full_like(want, 2.0 ** -10)) + fuzz
    else:
        tol = want.abs() * 2.0 ** -8 + fuzz + 1e-38
    d = (got.double() - want).abs()
    assert (d <= tol).all(), float((d / tol).max())


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("D,dims,inter", [(128, 128, False), (128, 64, True), (64, 16, False), (64, 64, True), (256, 256, False), (256, 48, False), (128, 0, False)])
@pytest.mark.parametrize("H,G,T,C", [(8, 4, 16, None), (1, 3, 64, 16), (12, 1, 128, 64), (3, 2, 512, 256)])
def test_append(dtype, D, dims, inter, H, G, T, C):
    s = Scene(dtype, H, G, D, T, [1, 70, 0, 3, 33], [1000, 70, 5, 2, 300], C=C, seed=1, pad=2)
    g = s.gen
    k = torch.randn((s.rows, H, D), generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn((s.rows, H, D), generator=g, device="cuda").to(torch.bfloat16)
    rot = zx.Rotary(dims, base=10000.0, interleaved=inter, scaling="yarn", factor=4.0, original=512) if dims else None
    kb, vb = s.kraw.clone(), s.vraw.clone()
    bb = None if C is None else s.bounds.clone()
    q_out = torch.full_like(s.q, 3.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    s.cache().append(k, v, s.batch(), q=s.q, rotary=rot, q_out=q_out, err=err)
    assert int(err.item()) == 0
    fill = lambda x, sc: x if sc is None else x / sc.double()[:, None]   # noqa: E731
    for b in range(len(s.new)):
        n, y = s.new[b], s.total[b]
        r0 = sum(s.new[:b])
        skip = max(0, n - y)                       # places below zero
        r = torch.arange(r0 + skip, r0 + n, device="cuda")
        p = y - n + (r - r0)
        page, off = s.table[b][p // T].long(), p % T
        want, made = turned(k[r], p, rot)
        got = s.kraw[page, :, off].view(TDT[dtype]).float()
        near(got, fill(want, s.ks), fill(made, s.ks), dtype)
        vv = v[r].float() if s.vs is None else (v[r].float() / s.vs[:, None]).clamp(-448, 448)
        assert torch.equal(s.vraw[page, :, off], vv.to(TDT[dtype]).view(RAW[dtype]))
        want, made = turned(s.q[r], p, rot)
        near(q_out[r].float(), want, made, BF16)
        assert torch.equal(q_out[r0:r0 + skip], torch.full_like(q_out[r0:r0 + skip], 3.0))
        kb[page, :, off], vb[page, :, off] = s.kraw[page, :, off], s.vraw[page, :, off]
        if C:
            for j in sorted(set((p // C).tolist())):
                pg, at = int(s.table[b, j * C // T]), j * C % T
                inside = s.kraw[pg, :, at:at + C].view(TDT[dtype]).float()[:, [i for i in range(C) if j * C + i in set(p.tolist())]]
                lo, hi = inside.amin(1), inside.amax(1)
                if j * C not in set(p.tolist()):    # the block had tokens before
                    old = bb[pg, :, at // C].float()
                    lo, hi = torch.minimum(lo, old[:, 0]), torch.maximum(hi, old[:, 1])
                bb[pg, :, at // C, 0], bb[pg, :, at // C, 1] = lo.to(torch.bfloat16), hi.to(torch.bfloat16)
    # nothing else is touched
    assert torch.equal(s.kraw, kb) and torch.equal(s.vraw, vb)
    if C:
        assert torch.equal(s.bounds.view(torch.int16), bb.view(torch.int16))
    assert torch.equal(q_out[s.N:], torch.full_like(q_out[s.N:], 3.0))


def test_queries_in_place_positions_and_far_angles():
    s = Scene(BF16, 2, 4, 128, 16, [3, 2], [50, 2], seed=2)
    k = torch.randn((5, 2, 128), device="cuda").to(torch.bfloat16)
    pos = torch.tensor([0, 1, 4_000_000, 1_048_575, 2_000_000_011], dtype=torch.int32, device="cuda")
    rot = zx.Rotary(128, base=500000.0)
    q0 = s.q.clone()
    out = s.cache().append(k, k, s.batch(), q=s.q, rotary=rot, positions=pos, q_out=s.q)
    assert out is s.q
    want, made = turned(q0, pos, rot)
    near(s.q.float(), want, made, BF16)
    # without queries, and with rows of a joint projection
    wide = torch.randn((5, 12, 128), device="cuda").to(torch.bfloat16)
    assert s.cache().append(wide[:, 8:10], wide[:, 10:], s.batch(), rotary=rot) is None
    page, off = s.table[0, 3].long(), 1
    assert torch.equal(s.vraw[page, :, off].view(torch.bfloat16), wide[2, 10:])


def test_fp8_edges():
    """Saturation, NaN, infinities, subnormal values: as torch rounds the clamped quotient."""
    s = Scene(FP8, 1, 1, 64, 16, [8], [8], C=16, seed=3)
    x = torch.randn((8, 1, 64), device="cuda")
    x[0, 0, :8] = torch.tensor([1e30, -1e30, math.inf, -math.inf, math.nan, 0.0, -0.0, 1e-30])
    x[1] = torch.linspace(-0.002, 0.002, 64)
    x[2] *= 100
    x = x.to(torch.bfloat16)
    s.cache().append(x, x, s.batch())
    want = (x.float() / s.vs[:, None])
    want = torch.where(torch.isnan(want), want, want.clamp(-448, 448)).to(torch.float8_e4m3fn)
    t = torch.arange(8, device="cuda")
    got = s.vraw[s.table[0, 0].long(), 0, t]
    bits = want.view(torch.uint8)[:, 0]
    same = (got == bits) | (torch.isnan(want.float()[:, 0]) & torch.isnan(got.view(torch.float8_e4m3fn).float()))
    assert same.all()
    b = s.bounds[s.table[0, 0].long(), 0, 0].float()
    assert not torch.isnan(b).any()


def test_append_bad_pages_and_lengths():
    s = Scene(BF16, 2, 2, 128, 16, [20, 20], [40, 60], C=16, seed=4)
    k = torch.randn((40, 2, 128), device="cuda").to(torch.bfloat16)
    for change in (lambda: s.table.__setitem__((0, 2), s.n_pages + 3), lambda: s.table.__setitem__((0, 2), -1)):
        s.kraw.zero_()
        tab = s.table.clone()
        change()
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        s.cache().append(k, k, s.batch(), err=err)
        assert int(err.item()) == 4
        t = torch.arange(20, 32, device="cuda")
        assert torch.equal(s.kraw[s.table[0][t // 16].long(), :, t % 16].view(torch.bfloat16), k[:12])
        t = torch.arange(40, 60, device="cuda")
        assert torch.equal(s.kraw[s.table[1][t // 16].long(), :, t % 16].view(torch.bfloat16), k[20:])
        s.table.copy_(tab)
    for change in (lambda: s.kv_len.__setitem__(0, -1), lambda: s.kv_len.__setitem__(0, 1 << 28), lambda: s.q_start.__setitem__(0, -1)):
        keep = s.q_start.clone(), s.kv_len.clone()
        s.kraw.zero_()
        change()
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        s.cache().append(k, k, s.batch(), err=err)
        assert int(err.item()) == 4
        t = torch.arange(20, 40, device="cuda")
        assert not s.kraw[s.table[0][t // 16].long(), :, t % 16].any()
        s.q_start.copy_(keep[0])
        s.kv_len.copy_(keep[1])


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("H,G,D,T,C", [(2, 4, 128, 64, 64), (1, 8, 64, 32, 16), (3, 1, 256, 512, 32)])
@pytest.mark.parametrize("top_k,first,last", [(1, 0, 0), (2, 1, 1), (7, 0, 1), (12, 2, 3), (64, 1, 1), (5, 5, 0), (4, 0, 4)])
def test_select(dtype, H, G, D, T, C, top_k, first, last):
    s = Scene(dtype, H, G, D, T, [1, 6, 0, 1, 2], [4000, 333, 20, 7, 1500], C=C, seed=5, pad=1)
    blocks = torch.full((s.rows, H, top_k), 77, dtype=torch.int32, device="cuda")
    s.cache().select(s.q, s.batch(), top_k, first, last, blocks=blocks)
    want = blocks_reference(s, top_k, first, last)
    assert torch.equal(blocks[:s.N].cpu(), want[:s.N])
    assert (blocks[s.N:] == 77).all()


def test_select_ties_nan_and_many_blocks():
    """Equal bounds: the earlier block.  NaN bounds last.  More blocks than fit in LDS."""
    s = Scene(BF16, 1, 2, 64, 16, [1], [16 * 6000], C=16, seed=6)
    want = blocks_reference(s, 100, 1, 1)
    assert torch.equal(s.cache().select(s.q, s.batch(), 100).cpu(), want)
    s.bounds.zero_()
    got = s.cache().select(s.q, s.batch(), 100, 0, 1).cpu()[0, 0]
    assert got.tolist() == list(range(99)) + [5999]
    s.bounds[s.table[0, :50].long()] = math.nan
    got = s.cache().select(s.q, s.batch(), 100, 0, 1).cpu()[0, 0]
    assert got.tolist() == list(range(50, 149)) + [5999]
    # the same page under several blocks
    s = Scene(BF16, 2, 2, 128, 16, [3], [16 * 40], C=16, seed=7)
    s.table[0, 10:30] = s.table[0, 5]
    assert torch.equal(s.cache().select(s.q, s.batch(), 9, 0, 0).cpu(), blocks_reference(s, 9, 0, 0))


def test_select_nothing_new():
    s = Scene(BF16, 2, 2, 128, 16, [2, 1], [1, 0], C=16, seed=8)
    assert s.cache().select(s.q, s.batch(), 3).cpu().tolist() == [[[-1] * 3] * 2, [[0, -1, -1]] * 2, [[-1] * 3] * 2]


@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_together(dtype):
    """A prompt in two pieces, then single tokens, with the old pages stowed in a slot pool and brought back
    into other pages: appended, attended densely and over selected blocks at each step, against the plain
    form on the cache's contents."""
    H, G, D, T, C = 8, 2, 128, 512, 64
    s = Scene(dtype, H, G, D, T, [600, 900], [600, 900], C=C, seed=9, width=3)
    cache = s.cache()
    s.n_tab = s.table.shape[1]
    free = [p for p in range(s.n_pages) if p not in set(s.table[:, :2].flatten().tolist())]
    rot = zx.Rotary(128, base=500000.0, scaling="bands", factor=8.0)
    g = s.gen

    def step(new, total):
        s.new, s.total = new, total
        s.N = s.rows = sum(new)
        s.q_start = torch.tensor([0, new[0], sum(new)], dtype=torch.int32, device="cuda")
        s.kv_len = torch.tensor(total, dtype=torch.int32, device="cuda")
        rows = lambda h: torch.randn((s.N, h, D), generator=g, device="cuda").to(torch.bfloat16)   # noqa: E731
        k, v, s.q = rows(H), rows(H), rows(H * G)
        b = s.batch(max_q=max(new), max_kv=max(total))
        cache.append(k, v, b, q=s.q, rotary=rot, q_out=s.q)
        lse = torch.empty((s.N, H * G), device="cuda")
        out = cache.attend(s.q, b, lse=lse)
        check_out(s, out, lse, reference(s, lambda x: see_mask(s, x)))
        if max(new) <= 4:
            blocks = cache.select(s.q, b, 6)
            assert torch.equal(blocks.cpu(), blocks_reference(s, 6, 1, 1))
            sp = cache.attend(s.q, b, blocks=blocks)
            see, _ = listed_mask(s, blocks)
            check_out(s, sp, None, reference(s, see))
            return out, sp
        return out, None

    step([500, 700], [500, 700])
    step([99, 198], [599, 898])
    step([1, 2], [600, 900])
    # page 0 of both sequences goes into the pool and comes back elsewhere
    pool = zx.KVSlotPool(2 * 2 * 8, dtype, cap_words=8192)
    ids = s.table[:, 0].contiguous()
    slots = torch.randperm(32, generator=g, device="cuda").to(torch.int32).view(2, 2, 8)
    status, bounds = cache.stow(ids, pool, slots)
    assert not status.any()
    want = cache.attend(s.q, s.batch()), cache.attend(s.q, s.batch(), blocks=cache.select(s.q, s.batch(), 6))
    cache.k.view(RAW[dtype])[ids.long()] = 1
    cache.v.view(RAW[dtype])[ids.long()] = 1
    cache.bounds[ids.long()] = 0
    others = torch.tensor([int(ids[1]), free[0]], dtype=torch.int32, device="cuda")
    cache.restore(others, pool, slots, bounds)
    s.table[:, 0] = others
    got = cache.attend(s.q, s.batch()), cache.attend(s.q, s.batch(), blocks=cache.select(s.q, s.batch(), 6))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for i in range(3):
        step([1, 1], [601 + i, 901 + i])


def test_step_in_a_graph():
    """A decode step captured once and replayed for growing sequences, against eager steps."""
    H, G, D, T, C = 4, 4, 128, 64, 32
    s = Scene(BF16, H, G, D, T, [1, 1, 1], [200, 64, 1], C=C, seed=10, width=3)
    e = Scene(BF16, H, G, D, T, [1, 1, 1], [200, 64, 1], C=C, seed=10, width=3)
    for x in (s, e):
        x.table[1, 1], x.table[2, 1] = x.n_pages - 1, x.n_pages - 2
        used = set(x.table[:, 0].tolist()) | set(x.table[0, :4].tolist())
        spare = [p for p in range(x.n_pages) if p not in used]
        x.table[1, 1], x.table[2, 1] = spare[0], spare[1]
        x.table[0, 4] = spare[0] if len(spare) < 3 else spare[2]
    rot = zx.Rotary(64, interleaved=True)
    k = torch.zeros((3, H, D), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((3, H * G, D), dtype=torch.bfloat16, device="cuda")
    out, sp = torch.zeros_like(q), torch.zeros_like(q)

    def one(x, q, out, sp):
        c, b = x.cache(), x.batch(max_q=1, max_kv=300)
        qr = c.append(k, k, b, q=q, rotary=rot)
        c.attend(qr, b, out=out)
        c.attend(qr, b, blocks=c.select(qr, b, 3), out=sp)

    one(s, q, out, sp)                       # warm up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one(s, q, out, sp)
    e.kraw.copy_(s.kraw)
    e.vraw.copy_(s.vraw)
    e.bounds.copy_(s.bounds)
    o2, s2 = torch.zeros_like(q), torch.zeros_like(q)
    for i in range(5):
        k.copy_(torch.randn(k.shape, device="cuda"))
        q.copy_(torch.randn(q.shape, device="cuda"))
        for x in (s, e):
            x.kv_len.copy_(torch.tensor([200 + i, 64 + i, 1 + i], dtype=torch.int32))
        one(e, q, o2, s2)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o2) and torch.equal(sp, s2)
        assert torch.equal(s.kraw, e.kraw) and torch.equal(s.bounds.view(torch.int16), e.bounds.view(torch.int16))


def test_append_on_a_side_stream():
    s = Scene(BF16, 2, 2, 128, 16, [3, 2], [50, 40], C=16, seed=11)
    k = torch.zeros((5, 2, 128), dtype=torch.bfloat16, device="cuda")
    big = torch.randn(4096, 4096, device="cuda")
    for _ in range(4):
        big = big @ big * 1e-3
    k.copy_(torch.randn(k.shape, device="cuda"))
    side = torch.cuda.Stream()
    got = s.cache().append(k, k, s.batch(), q=s.q, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, s.q)
    assert torch.equal(s.vraw[s.table[1, 2].long(), :, 6:8].view(torch.bfloat16).transpose(0, 1), k[3:])
