"""Refusals of the beam search's entry points before any launch (CPU)."""
import ctypes as C
import math

import pytest
import torch

import lossless_float_compression_amd as zx
from lossless_float_compression_amd import beams, paged, pages

P = C.c_void_p
OK, INVAL, UNSUPPORTED, LIMIT = 0, 1, 2, 7


@pytest.fixture(scope="module")
def lib():
    pages._lib()
    return beams._lib()


def set_(s, kw):
    for k, v in kw.items():
        setattr(s, k, v)
    return C.byref(s)


def select(lib, n_out=8, scores=0x1000, weights=None, finished=None, end=-1, allowed=None, scale=1.0, outs=(0x2000, 0x3000, 0x4000, 0x5000), ws=0x10000,
           ws_bytes=1 << 40, **kw):
    c = beams.zx_beam_logits(0x100000, 4 * 1000, 1000, 0, 2, 4, 1000)
    return lib.zx_beam_select(set_(c, kw), scores, weights, finished, end, allowed, scale, n_out, *outs, ws, ws_bytes, None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(type=3), UNSUPPORTED), (dict(type=-1), UNSUPPORTED), (dict(beams=0), INVAL), (dict(beams=65), INVAL), (dict(vocab=0), INVAL),
    (dict(vocab=(1 << 24) + 1), LIMIT), (dict(n_out=0), INVAL), (dict(n_out=65), INVAL), (dict(logits=None), INVAL), (dict(logits=0x100001), INVAL),
    (dict(logits=0x100002, type=2), INVAL), (dict(scores=None), INVAL), (dict(outs=(None, 0x3000, 0x4000, 0x5000)), INVAL),
    (dict(outs=(0x2000, 0x3000, None, 0x5000)), INVAL), (dict(outs=(0x2000, 0x3000, 0x4000, None)), INVAL), (dict(scale=0.0), INVAL), (dict(scale=-1.0), INVAL),
    (dict(scale=math.nan), INVAL), (dict(scale=math.inf), INVAL), (dict(end=-2), INVAL), (dict(end=1000), INVAL), (dict(finished=0x9000), INVAL),
    (dict(group_stride=1 << 41), INVAL), (dict(beam_stride=1 << 41), INVAL), (dict(ws=None), INVAL), (dict(ws=0x10008), INVAL), (dict(ws_bytes=100), INVAL),
    (dict(n_groups=1 << 30), LIMIT), (dict(n_groups=0), OK), (dict(scores=0x1002), INVAL), (dict(weights=0x1001), INVAL), (dict(allowed=0x1002), INVAL),
    (dict(outs=(0x2001, 0x3000, 0x4000, 0x5000)), INVAL), (dict(outs=(0x2000, 0x3000, 0x4002, 0x5000)), INVAL)])
def test_select(lib, kw, want):
    assert select(lib, **kw) == want


def test_select_workspace(lib):
    f = lib.zx_beam_select_workspace_bytes
    assert f(3, 1, 4, 1000, 8) == 0 and f(0, 1, 65, 1000, 8) == 0 and f(0, 1, 4, 0, 8) == 0 and f(0, 0, 4, 1000, 8) == 0
    for ty in (0, 1, 2):
        for G, K, V, M in [(1, 1, 1, 1), (1, 4, 32000, 8), (64, 8, 128256, 16), (1, 64, 1 << 24, 64)]:
            need = f(ty, G, K, V, M)
            parts = need // (G * K * (64 + 8 * M))
            assert parts * G * K * (64 + 8 * M) == need
            assert any(parts == -(-V // (256 * e)) for e in (4, 8, 16, 32, 64, 128, 256)) or (G, V) == (64, 128256)
            assert select(lib, type=ty, n_groups=0, beams=K, vocab=V, n_out=M, ws_bytes=need) == OK
            assert select(lib, type=ty, n_groups=G, beams=K, vocab=V, n_out=M, ws_bytes=need - 1) == INVAL


def test_merge(lib):
    def call(n=2, tokens=5, heads=4, D=128, part=None, lse=0x8000, out=None, parts=True, lses=True):
        r = (paged.zx_rows * 17)(*[paged.zx_rows(0x10000, 512, 128)] * 17)
        if part is not None:
            r[1] = part
        l = (P * 17)(*[0x8000, lse] + [0x8000] * 15)
        o = paged.zx_rows(0x20000, 512, 128) if out is None else out
        return lib.zx_attention_merge(r if parts else None, l if lses else None, n, tokens, heads, D, C.byref(o), None, None)
    assert call(tokens=0) == OK
    for kw in (dict(n=0), dict(n=17), dict(heads=0), dict(heads=65537), dict(D=96), dict(D=0), dict(parts=False), dict(lses=False), dict(lse=None), dict(lse=0x8002),
               dict(part=paged.zx_rows(0x10008, 512, 128)), dict(part=paged.zx_rows(None, 512, 128)), dict(part=paged.zx_rows(0x10000, 516, 128)),
               dict(out=paged.zx_rows(0x10000, 512, 1 << 41))):
        assert call(**kw) == INVAL, kw
    assert call(tokens=1 << 31, heads=65536, D=256) == LIMIT


def pool(**kw):
    return set_(pages.zx_page_pool(100, 16, 0x1000), kw)


def rows(**kw):
    return set_(pages.zx_page_rows(0x2000, 0x3000, 6, 10), kw)


def copies(**kw):
    return set_(pages.zx_page_copies(0x4000, 0x5000, 60, 0), kw)


def calls(lib, p=None, r=None, c=None):
    p, r, c = p or pool(), r or rows(), c or copies()
    yield "fork", lib.zx_pages_fork(p, r, 3, P(0x6000), None, None)
    yield "trim", lib.zx_pages_trim(p, r, None, None, None)
    yield "extend", lib.zx_pages_extend(p, r, P(0x7000), 9, 99, P(0x8000), c, P(0x10000), 1 << 30, None, None)
    yield "compact", lib.zx_pages_compact(p, r, P(0x9000), c, P(0x10000), 1 << 30, None, None)


@pytest.mark.parametrize("kw,want", [(dict(n_pages=0), INVAL), (dict(n_pages=(1 << 23) + 1), LIMIT), (dict(page_tokens=8), INVAL), (dict(page_tokens=48), INVAL),
                                     (dict(page_tokens=8192), INVAL), (dict(refs=None), INVAL), (dict(refs=0x1002), INVAL)])
def test_pools(lib, kw, want):
    for name, got in calls(lib, p=pool(**kw)):
        assert got == want, name


@pytest.mark.parametrize("kw,want", [(dict(page_table=None), INVAL), (dict(held=None), INVAL), (dict(n_seqs=65537), LIMIT), (dict(table_width=1 << 26), LIMIT),
                                     (dict(page_table=0x2001), INVAL), (dict(held=0x3002), INVAL)])
def test_rows(lib, kw, want):
    for name, got in calls(lib, r=rows(**kw)):
        assert got == want, name


def test_pages(lib):
    no = None
    f = lib.zx_pages_fork
    assert f(no, rows(), 3, P(16), no, no) == INVAL and f(pool(), no, 3, P(16), no, no) == INVAL and f(pool(), rows(), 0, P(16), no, no) == INVAL
    assert f(pool(), rows(), 4, P(16), no, no) == INVAL and f(pool(), rows(), 3, no, no, no) == INVAL and f(pool(), rows(n_seqs=4098), 2049, P(16), no, no) == LIMIT
    assert f(pool(), rows(n_seqs=0), 3, no, no, no) == OK and lib.zx_pages_trim(pool(), rows(n_seqs=0), no, no, no) == OK
    e, ws = lib.zx_pages_extend, lib.zx_pages_extend_workspace_bytes
    need = ws(pool(), 6)
    good = lambda **kw: [kw.get("p") or pool(), kw.get("r") or rows(), P(16), 9, 99, P(32), kw.get("c") or copies(), P(kw.get("ws", 64)), kw.get("b", need), no, no]   # noqa: E731
    assert need > 0 and ws(no, 6) == 0 and ws(pool(), 2049) == 0
    for a in (good(b=need - 1), good(ws=0), good(ws=72), good(c=copies(cap=5)), good(c=copies(pairs=None)), good(c=copies(count=None))):
        assert e(*a) == INVAL
    assert e(*good(r=rows(n_seqs=2049), b=1 << 30)) == LIMIT
    for i in (2, 5, 6):
        a = good()
        a[i] = no
        assert e(*a) == INVAL, i
    for i in (2, 5):
        a = good()
        a[i] = P(0x1002)
        assert e(*a) == INVAL, i
    assert f(pool(), rows(), 3, P(18), no, no) == INVAL and lib.zx_pages_trim(pool(), rows(), P(18), no, no) == INVAL
    assert e(*good(c=copies(pairs=0x4001))) == INVAL and e(*good(c=copies(count=0x5002))) == INVAL
    k, ws = lib.zx_pages_compact, lib.zx_pages_compact_workspace_bytes
    need = ws(pool())
    assert need > 0 and ws(no) == 0
    assert k(pool(), rows(), no, copies(), P(64), need, no, no) == INVAL and k(pool(), rows(), P(16), copies(cap=49), P(64), need, no, no) == INVAL
    assert k(pool(), rows(), P(16), copies(), P(72), need, no, no) == INVAL and k(pool(), rows(), P(16), copies(), P(64), need - 1, no, no) == INVAL


def test_copy(lib):
    def caches(*changes):
        a = (paged.zx_paged_cache * max(1, len(changes)))()
        for i, kw in enumerate(changes):
            a[i] = paged.zx_paged_cache(0, 10, 2, 128, 64, 16, 0x10000, 0x20000, 2 * 64 * 128, 64 * 128, 128, 2 * 64 * 128, 64 * 128, 128, None, None, 0x30000)
            for k, v in kw.items():
                setattr(a[i], k, v)
        return a
    f = lib.zx_paged_copy
    assert f(None, 0, copies(), None, None) == OK and f(caches({}), 1, copies(cap=0, pairs=None), None, None) == OK
    assert f(None, 1, copies(), None, None) == INVAL and f(caches({}), 1, None, None, None) == INVAL and f(caches({}), 1, copies(pairs=None), None, None) == INVAL
    assert f(caches({}), 1, copies(count=None), None, None) == INVAL and f(caches({}), 65537, copies(), None, None) == LIMIT
    for kw in (dict(dtype=1), dict(n_pages=11), dict(kv_heads=3), dict(head_dim=64), dict(page_tokens=128), dict(block_tokens=32), dict(k=None), dict(v=0x20008)):
        assert f(caches({}, kw), 2, copies(), None, None) == INVAL, kw
    assert f(caches(dict(dtype=7)), 1, copies(), None, None) == UNSUPPORTED


@pytest.mark.parametrize("stream", [C.c_void_p(0), 0x1000, "side"])
def test_raw_streams_are_refused(stream):
    with pytest.raises(ValueError, match="torch stream"):
        pages._away(0, stream)


def test_host_tensors_are_refused():
    x, s, i = torch.zeros((1, 2, 8)), torch.zeros((1, 2)), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: zx.beam_select(x, s), lambda: zx.merge_attention([x.bfloat16()], [s]), lambda: zx.PagePool(4, 16, refs=i),
                 lambda: zx.PageCopies(4, pairs=torch.zeros((4, 3), dtype=torch.int32)), lambda: zx.PagedLayers([])):
        with pytest.raises(ValueError):
            call()


def test_what_tensors_reach():
    t = torch.zeros((4, 6))
    p = t.data_ptr()
    assert pages._span(t) == (p, p + 96) and pages._span(t[1:3, 2:4]) == (p + 32, p + 64) and len(set(pages._span(t[:0]))) == 1
    assert pages._meets(t[:2], t[1:]) and not pages._meets(t[:2], t[2:]) and not pages._meets(t[:0], t)


def test_caches_that_autograd_follows_are_not_copied_in():
    """By either mode; without one, as they are."""
    import torch.autograd.forward_ad as forward

    t = torch.zeros((2, 3), dtype=torch.bfloat16)
    list_ = type("Copies", (), dict(device="cpu", pairs=t, count=t))
    of = type("Of", (), dict(_index=0, device="elsewhere", _tensors=(t,), _gradients=False))
    with pytest.MonkeyPatch.context() as m:
        m.setattr(pages, "_device", lambda: 0)
        with pytest.raises(ValueError, match="the copies are on"):
            pages._copy(of, None, 1, list_, None, None)
        of.device = "cpu"
        with forward.dual_level():
            of._tensors = (forward.make_dual(t, torch.ones_like(t)),)
            with pytest.raises(ValueError, match="gradient"):
                pages._copy(of, None, 1, list_, None, None)
        of._tensors, of._gradients = (t.clone().requires_grad_(),), True
        with pytest.raises(ValueError, match="gradient"):
            pages._copy(of, None, 1, list_, None, None)


def test_stretches_that_meet():
    pages._all_apart([(8, 12), (0, 8), (12, 12), (12, 20), (20, 20)])
    for bad in ([(0, 8), (4, 12)], [(0, 20), (4, 8)], [(0, 20), (4, 8), (8, 12)], [(4, 8), (4, 8)]):
        with pytest.raises(ValueError, match="share memory"):
            pages._all_apart(bad)
