"""Tokens copied between pages, in the caches of all layers: bit for bit, and nothing else is written."""
import pytest
import torch

import lossless_float_compression_amd as zx
from pages_util import i32

pytestmark = pytest.mark.gpu
RAW = {zx.BF16: torch.int16, zx.FP8_E4M3FN: torch.uint8}
TDT = {zx.BF16: torch.bfloat16, zx.FP8_E4M3FN: torch.float8_e4m3fn}


def cache(n, H, D, T, dtype, C, g, layout="heads"):
    """Pages of random bits (NaN patterns too); `layout`: heads ahead of tokens, tokens ahead of heads, or K and V side by side."""
    top = 1 << (16 if dtype == zx.BF16 else 8)

    def bits(*shape):
        return torch.randint(0, top, shape, generator=g, device="cuda").to(RAW[dtype])
    if layout == "heads":
        k, v = bits(n, H, T, D), bits(n, H, T, D)
    elif layout == "tokens":
        k, v = bits(n, T, H, D).transpose(1, 2), bits(n, T, H, D).transpose(1, 2)
    else:
        kv = bits(n, H, T, 2 * D + 16)
        k, v = kv[..., :D], kv[..., D + 16:]
    b = torch.randint(0, 1 << 16, (n, H, T // C, 2, D), generator=g, device="cuda").to(torch.int16).view(torch.bfloat16) if C else None
    return zx.PagedKVCache(n, H, D, T, dtype, block_tokens=C, k=k.view(TDT[dtype]), v=v.view(TDT[dtype]), bounds=b)


def pages(c):
    return [None if t is None else t.view(torch.uint8 if t.dtype == torch.float8_e4m3fn else torch.int16).clone() for t in (c.k, c.v, c.bounds)]


def want(before, moves, C):
    for a, b, n in moves:
        for x, unit in zip(before, (1, 1, C)):
            if x is not None:
                x[b, :, :-(-n // unit)] = x[a, :, :-(-n // unit)]
    return before


def same(c, w):
    for x, y in zip(pages(c), w):
        assert x is None or torch.equal(x, y)


def listed(moves, cap=None):
    cap = len(moves) if cap is None else cap
    t = torch.full((cap, 3), 1 << 30, dtype=torch.int32)
    if moves:
        t[:len(moves)] = torch.tensor(moves, dtype=torch.int32)
    return zx.PageCopies(cap, pairs=t.cuda(), count=i32([len(moves)]))


@pytest.mark.parametrize("layout", ("heads", "tokens", "side"))
@pytest.mark.parametrize("dtype", (zx.BF16, zx.FP8_E4M3FN))
@pytest.mark.parametrize("H,D,T,C", [(1, 64, 16, None), (2, 128, 64, 16), (3, 256, 32, 32), (8, 128, 16, 16), (5, 64, 512, 64), (1, 128, 4096, 256), (40, 64, 16, None)])
def test_copies(H, D, T, C, dtype, layout):
    g = torch.Generator(device="cuda").manual_seed(H * T)
    layers = [cache(12, H, D, T, dtype, C, g, layout) for _ in range(3)]
    moves = [(0, 7, T), (0, 3, 1), (9, 2, T - 1), (4, 8, T // 2 + 1), (5, 5, T), (1, 11, 0), (10, 6, min(T, 16))]
    w = [want(pages(c), moves, C) for c in layers]
    err = i32([0])
    zx.PagedLayers(layers).copy_pages(listed(moves, 20), err=err)
    for c, x in zip(layers, w):
        same(c, x)
    assert int(err) == 0


def test_many_layers():
    """More caches than one launch takes, in one tensor."""
    g = torch.Generator(device="cuda").manual_seed(0)
    k = torch.randint(0, 1 << 16, (2, 95, 6, 2, 16, 64), generator=g, device="cuda").to(torch.int16).view(torch.bfloat16)
    layers = [zx.PagedKVCache(6, 2, 64, 16, k=k[0, i], v=k[1, i]) for i in range(95)]
    moves = [(0, 1, 16), (2, 3, 5)]
    w = [want(pages(c), moves, None) for c in layers]
    zx.PagedLayers(layers).copy_pages(listed(moves))
    for c, x in zip(layers, w):
        same(c, x)


def test_more_pairs_than_workgroups():
    g = torch.Generator(device="cuda").manual_seed(0)
    c = cache(9000, 2, 64, 16, zx.FP8_E4M3FN, 16, g)
    perm = torch.randperm(9000, generator=g, device="cuda").to(torch.int32)
    n = torch.randint(0, 17, (4500,), generator=g, device="cuda", dtype=torch.int32)
    pairs = torch.stack((perm[:4500], perm[4500:], n), 1).contiguous()
    k, v, b = pages(c)
    for x, m in ((k, n), (v, n), (b, (n > 0).int())):
        take = (torch.arange(x.shape[2], device="cuda") < m[:, None]).view(-1, 1, x.shape[2], *[1] * (x.dim() - 3))
        x[perm[4500:].long()] = torch.where(take, x[perm[:4500].long()], x[perm[4500:].long()])
    c.copy_pages(zx.PageCopies(4500, pairs=pairs, count=i32([4500])))
    same(c, (k, v, b))


def test_pages_beyond_32_bits():
    """Pages more than 4 GiB into the cache."""
    k = torch.zeros((2200, 8, 512, 256), dtype=torch.bfloat16, device="cuda")       # 4.6 GB
    v = torch.zeros_like(k)
    k[0], v[0] = 3.0, 5.0
    c = zx.PagedKVCache(2200, 8, 256, 512, k=k, v=v)
    c.copy_pages(listed([(0, 2199, 500)]))
    assert bool((k[2199, :, :500] == 3).all()) and bool((v[2199, :, :500] == 5).all()) and not bool(k[2199, :, 500:].any())
    assert not bool(k[1:2199].any())
    k[2199, :, 0], k[0] = 7.0, 0.0
    c.copy_pages(listed([(2199, 1, 1)]))
    assert bool((k[1, :, 0] == 7).all()) and not bool(k[1, :, 1:].any())


def test_pairs_out_of_range():
    """Left out and reported, the others carried out; counts beyond the list and below nothing."""
    g = torch.Generator(device="cuda").manual_seed(1)
    for bad in [(-1, 3, 16), (3, -1, 16), (12, 3, 16), (3, 12, 5), (3, 4, -1), (3, 4, 17), (2 ** 31 - 1, 1, 1), (1, -2 ** 31, 1), (4, 5, 2 ** 31 - 1)]:
        c = cache(12, 2, 64, 16, zx.BF16, 16, g)
        w = want(pages(c), [(0, 1, 16), (6, 7, 3)], 16)
        err = i32([0])
        c.copy_pages(listed([(0, 1, 16), bad, (6, 7, 3)]), err=err)
        same(c, w)
        assert int(err) == 4
    for count in (5, 2 ** 31 - 1, -1, -2 ** 31):
        c = cache(12, 2, 64, 16, zx.BF16, 16, g)
        w = want(pages(c), [(0, 1, 16), (6, 7, 3)] if count > 0 else [], 16)
        l = listed([(0, 1, 16), (6, 7, 3)])
        l.count.fill_(count)
        err = i32([0])
        c.copy_pages(l, err=err)
        same(c, w)
        assert int(err) == 4


def test_empty_lists():
    g = torch.Generator(device="cuda").manual_seed(1)
    c = cache(3, 1, 64, 16, zx.BF16, None, g)
    w = pages(c)
    c.copy_pages(listed([]))
    c.copy_pages(listed([], 9))
    same(c, w)


def test_streams_and_graph():
    g = torch.Generator(device="cuda").manual_seed(2)
    c = cache(20, 4, 128, 64, zx.BF16, 32, g)
    l = listed([(0, 1, 64)], 8)
    side = torch.cuda.Stream()
    w = torch.randn(4096, 4096, device="cuda")
    for _ in range(3):
        w = (w @ w).mul_(0.01)
    l.pairs[1] = i32([2, 3, 7]) + w[0, 0].clamp(0, 0).to(torch.int32)
    l.count.fill_(2)
    x = want(pages(c), [(0, 1, 64), (2, 3, 7)], 32)
    c.copy_pages(l, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    same(c, x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.copy_pages(l)
    for i in range(4):
        moves = [(i, 10 + i, 64 - i), (4 + i, 15, 3)][:1 + i % 2]
        l.pairs[:len(moves)] = i32(moves)
        l.count.fill_(len(moves))
        x = want(pages(c), moves, 32)
        graph.replay()
        same(c, x)
        c.copy_pages(listed([(0, 19, 64)]))


def test_refusals():
    g = torch.Generator(device="cuda").manual_seed(0)
    a, b = cache(4, 2, 64, 16, zx.BF16, None, g), cache(4, 2, 64, 16, zx.BF16, None, g)
    over = torch.zeros((8, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    share = [zx.PagedKVCache(4, 2, 64, 16, k=over[:4], v=torch.zeros_like(over[:4])), zx.PagedKVCache(4, 2, 64, 16, k=over[3:7], v=torch.zeros_like(over[:4]))]
    bnd = torch.zeros((5, 2, 1, 2, 64), dtype=torch.bfloat16, device="cuda")
    blocks = [zx.PagedKVCache(4, 2, 64, 16, block_tokens=16, bounds=bnd[i:i + 4]) for i in (0, 1)]
    wants = zx.PagedKVCache(4, 2, 64, 16, k=torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda", requires_grad=True), v=over[:4])
    bad = [lambda: zx.PagedLayers([]), lambda: zx.PagedLayers([a, cache(5, 2, 64, 16, zx.BF16, None, g)]), lambda: zx.PagedLayers([a, a]),
           lambda: zx.PagedLayers([a, cache(4, 2, 64, 16, zx.FP8_E4M3FN, None, g)]), lambda: zx.PagedLayers([a, cache(4, 2, 64, 16, zx.BF16, 16, g)]),
           lambda: zx.PagedLayers(share), lambda: zx.PagedLayers(blocks), lambda: a.copy_pages(listed([(0, 1, 2)]), stream=3), lambda: wants.copy_pages(listed([(0, 1, 2)])),
           lambda: a.copy_pages(listed([(0, 1, 2)]), err=torch.zeros(1, device="cuda"))]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    # layers that lie between each other's pages are apart
    mixed = torch.zeros((4, 3, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    zx.PagedLayers([zx.PagedKVCache(4, 2, 64, 16, k=mixed[:, 0], v=mixed[:, 1]), b])


PAST = 16384                             # shares of 16 KB of a list from which on it is carried out past the caches


@pytest.mark.parametrize("layout", ("heads", "tokens", "side"))
@pytest.mark.parametrize("dtype", (zx.BF16, zx.FP8_E4M3FN))
@pytest.mark.parametrize("past", (False, True))
@pytest.mark.parametrize("H,D,T,C,layers", [(1, 64, 16, None, 1), (2, 128, 64, 16, 2), (5, 64, 512, 64, 3), (3, 256, 32, 32, 1)])
def test_long_lists(H, D, T, C, layers, past, dtype, layout):
    """The longest list that goes through the caches and the shortest that goes past them: any number of tokens of each page, nothing else written."""
    ceil = lambda a: -(-a // 16384)                                      # noqa: E731
    per = layers * (2 * ceil(H * T * D * (2 if dtype == zx.BF16 else 1)) + (ceil(H * (T // C) * D * 4) if C else 0))
    n = PAST // per + past
    assert (n * per > PAST) == past
    g = torch.Generator(device="cuda").manual_seed(n)
    caches = [cache(2 * n + 3, H, D, T, dtype, C, g, layout) for _ in range(layers)]
    perm = torch.randperm(2 * n + 3, generator=g, device="cuda").to(torch.int32)
    src, dst = perm[:n], perm[n:2 * n]
    some = torch.randint(0, T + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
    some[:3] = torch.tensor([T, 0, 1], dtype=torch.int32)
    want = [pages(c) for c in caches]
    for w in want:
        for x, unit in zip(w, (1, 1, C)):
            if x is not None:
                m = (some + (unit - 1)) // unit
                take = (torch.arange(x.shape[2], device="cuda") < m[:, None]).view(-1, 1, x.shape[2], *[1] * (x.dim() - 3))
                x[dst.long()] = torch.where(take, x[src.long()], x[dst.long()])
    err = i32([0])
    zx.PagedLayers(caches).copy_pages(zx.PageCopies(n, pairs=torch.stack((src, dst, some), 1).contiguous(), count=i32([n])), err=err)
    for c, w in zip(caches, want):
        same(c, w)
    assert int(err) == 0
