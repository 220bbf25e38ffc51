"""Attention over parts joined, against its definition in 64 bits.

How far a result may be off: a weight's argument l - m is off by 2^-24 of |l - m| (<= 24 here) and its exponential by that, a constant's rounding and two
steps, together less than (3 * 24 + 4) 2^-24 < 2^-17 of the weight; the sums add 2 * 16 * 2^-24; all against the weights' own sum and the
parts' largest value.  The result is rounded to BF16 once, 2^-8 of itself at most."""
import math

import pytest
import torch

import lossless_float_compression_amd as zx

pytestmark = pytest.mark.gpu


def plain(outs, lses):
    x, l = torch.stack([t.double() for t in outs]), torch.stack([t.double() for t in lses])
    lse = torch.logsumexp(l, 0)
    m = l.max(0)[0]                                  # (not by lse: -3e38 + ln 2 is -3e38 in 64 bits too)
    w = torch.exp(l - torch.where(m == -math.inf, 0.0, m))
    w = w / w.sum(0).clamp(min=1e-300)
    x = torch.where((l == -math.inf)[..., None], 0.0, x)
    return (x * w[..., None]).sum(0), lse


def check(out, lse, outs, lses):
    want, want_lse = plain(outs, lses)
    most = torch.stack([torch.where((l == -math.inf)[..., None], 0.0, t.double()).abs() for t, l in zip(outs, lses)]).max(0)[0]
    off = (out.double() - want).abs()
    assert bool((off <= want.abs() * 2.0 ** -8 + most * 2.0 ** -15 + 1e-38).all()), off.max()
    if lse is not None:
        some = want_lse > -math.inf
        assert torch.equal(lse > -math.inf, some)
        off = (lse.double() - want_lse)[some].abs()
        assert bool((off <= 2.0 ** -16 + want_lse[some].abs() * 2.0 ** -23).all()), off.max()


def made(P, N, H, D, seed=0, empty=0.3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    outs = [torch.randn((N, H, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(P)]
    lses = [3.0 * torch.randn((N, H), generator=g, device="cuda") + 5.0 for _ in range(P)]
    for o, l in zip(outs, lses):
        gone = torch.rand((N, H), generator=g, device="cuda") < empty
        l[gone] = -math.inf
        o[gone] = math.nan                           # what a part that has seen nothing holds is not looked at
    return outs, lses


@pytest.mark.parametrize("D", (64, 128, 256))
@pytest.mark.parametrize("P", range(1, 17))
def test_parts(P, D):
    outs, lses = made(P, 37, 5, D, seed=P)
    lse = torch.empty_like(lses[0])
    check(zx.merge_attention(outs, lses, lse=lse), lse, outs, lses)


@pytest.mark.parametrize("N,H,D", [(1, 1, 64), (1, 32, 128), (3, 7, 256), (513, 40, 128), (70000, 1, 64), (0, 8, 128)])
def test_sizes(N, H, D):
    outs, lses = made(3, N, H, D, seed=N)
    check(zx.merge_attention(outs, lses), None, outs, lses)


def test_rows_that_saw_nothing():
    outs, lses = made(2, 9, 4, 128, empty=1.1)
    lse = torch.zeros((9, 4), device="cuda")
    out = zx.merge_attention(outs, lses, lse=lse)
    assert not bool(out.any()) and bool((lse == -math.inf).all())


def test_far_apart():
    """Weights below any float beside one that is all, and lses of any size."""
    outs, lses = made(2, 6, 3, 64, empty=0.0)
    lses[0] += 500.0
    check(zx.merge_attention(outs, lses), None, outs, lses)
    lses = [l * 0 + x for l, x in zip(lses, (-3e38, 3e38))]
    assert torch.equal(zx.merge_attention(outs, lses), outs[1])
    lses = [l * 0 - 3e38 for l in lses]
    check(zx.merge_attention(outs, lses), None, outs, lses)


def test_nan_and_infinite_lses():
    outs, lses = made(3, 5, 2, 128, empty=0.0)
    lses[1][2, 1] = math.nan
    lses[2][4, 0] = math.inf
    out = zx.merge_attention(outs, lses)
    odd = torch.zeros((5, 2), dtype=torch.bool, device="cuda")
    odd[2, 1] = odd[4, 0] = True
    assert bool(out[odd].isnan().all()) and bool(out[~odd].isfinite().all())


def test_strides_and_places():
    g = torch.Generator(device="cuda").manual_seed(3)
    a = torch.randn((4, 30, 3, 128), generator=g, device="cuda").to(torch.bfloat16)
    outs = [a[0].transpose(0, 1), torch.randn((3, 30, 256), generator=g, device="cuda").to(torch.bfloat16)[:, :, 64:192],
            torch.randn((1, 30, 128), generator=g, device="cuda").to(torch.bfloat16).expand(3, 30, 128)]
    lses = [torch.randn((3, 30), generator=g, device="cuda") for _ in outs]
    back = torch.full((3, 31, 160), 7.0, dtype=torch.bfloat16, device="cuda")
    out = back[:, 1:, 16:144]
    zx.merge_attention(outs, lses, out=out)
    check(out, None, outs, lses)
    out.fill_(7.0)
    assert bool((back == 7.0).all())


def test_in_place():
    outs, lses = made(3, 50, 4, 64)
    want_lse = torch.empty_like(lses[0])
    want = zx.merge_attention(outs, lses, lse=want_lse)
    got = zx.merge_attention(outs, lses, out=outs[1], lse=lses[2])
    assert got is outs[1] and torch.equal(got, want) and torch.equal(lses[2], want_lse)


def test_rows_beyond_32_bits():
    far = (1 << 31) + 8
    big = torch.empty(far + 4096, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((2, 3, 128), (far, 128, 1))
    outs, lses = made(2, 2, 3, 128, empty=0.0)
    x.copy_(outs[0])
    assert torch.equal(zx.merge_attention([x, outs[1]], lses), zx.merge_attention(outs, lses))
    zx.merge_attention(outs, lses, out=x)
    check(x, None, outs, lses)


def test_streams_and_graph():
    outs, lses = made(2, 300, 8, 128)
    w = torch.randn(4096, 4096, device="cuda")
    for _ in range(3):
        w = (w @ w).mul_(0.01)
    late = outs[0] + w[0, 0].clamp(0, 0).to(torch.bfloat16)
    side = torch.cuda.Stream()
    got = zx.merge_attention([late, outs[1]], lses, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check(got, None, outs, lses)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = zx.merge_attention(outs, lses)
    for i in range(3):
        more, l = made(2, 300, 8, 128, seed=i)
        for a, b in zip((*outs, *lses), (*more, *l)):
            a.copy_(b)
        g.replay()
        check(out, None, outs, lses)
        zx.merge_attention(outs, lses)


def test_refusals():
    outs, lses = made(2, 4, 3, 128)
    wide = torch.zeros((4, 3, 132), dtype=torch.bfloat16, device="cuda")
    bad = [lambda: zx.merge_attention([], []), lambda: zx.merge_attention(outs, lses[:1]), lambda: zx.merge_attention(outs * 9, lses * 9),
           lambda: zx.merge_attention([t.float() for t in outs], lses), lambda: zx.merge_attention([outs[0], outs[1][:3]], lses),
           lambda: zx.merge_attention([t[:, :, :96].contiguous() for t in outs], lses), lambda: zx.merge_attention(outs, [t.double() for t in lses]),
           lambda: zx.merge_attention(outs, [lses[0], lses[1].t().contiguous().t()]), lambda: zx.merge_attention([t.cpu() for t in outs], lses),
           lambda: zx.merge_attention([outs[0], wide[:, :, :128]], lses), lambda: zx.merge_attention(outs, lses, out=outs[0][:, :1].expand(4, 3, 128)),
           lambda: zx.merge_attention(outs, lses, out=wide[:, :, 4:]), lambda: zx.merge_attention(outs, lses, lse=lses[0][:3]),
           lambda: zx.merge_attention([outs[0].clone().requires_grad_(), outs[1]], lses), lambda: zx.merge_attention(outs, [lses[0].clone().requires_grad_(), lses[1]]),
           lambda: zx.merge_attention(outs, lses, stream=5)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")


def test_parts_larger_than_the_caches():
    """More bytes than 256 MB of parts are read another way: the same values."""
    outs, lses = made(3, 12000, 32, 128)
    whole = zx.merge_attention(outs, lses)
    half = [zx.merge_attention([t[i:i + 4000] for t in outs], [t[i:i + 4000].contiguous() for t in lses]) for i in (0, 4000, 8000)]
    assert torch.equal(whole, torch.cat(half))
    check(whole[::37], None, [t[::37] for t in outs], [t[::37] for t in lses])


@pytest.mark.parametrize("layout", ("parts ahead of heads", "parts behind heads", "parts side by side"))
def test_in_place_among_interleaved_parts(layout):
    """The parts in one tensor, one of them written: the others stay."""
    outs, lses = made(3, 50, 4, 64)
    if layout == "parts ahead of heads":
        big = torch.stack(outs, 1)
        mine = big.unbind(1)
    elif layout == "parts behind heads":
        big = torch.stack(outs, 2)
        mine = big.unbind(2)
    else:
        big = torch.cat(outs, 2)
        mine = big.split(64, 2)
    want = zx.merge_attention(outs, lses)
    check(want, None, outs, lses)
    for i in range(3):
        before = [t.clone() for t in mine]
        assert torch.equal(zx.merge_attention(mine, lses, out=mine[i]), want)
        for j in range(3):
            assert torch.equal(mine[j].view(torch.int16), (want if j == i else before[j]).view(torch.int16))
        mine[i].copy_(before[i])
