"""Refusals of the paged K/V cache, before any launch (CPU), and the frequencies of Rotary."""
import ctypes as C
import math

import pytest
import torch

import lossless_float_compression_amd as zx
from lossless_float_compression_amd import paged

P = C.c_void_p
OK, INVAL, UNSUPPORTED, LIMIT = 0, 1, 2, 7


@pytest.fixture(scope="module")
def lib():
    return paged._lib()


def cache(**kw):
    c = paged.zx_paged_cache(0, 10, 2, 128, 64, 0, 0x10000, 0x20000, 2 * 64 * 128, 64 * 128, 128, 2 * 64 * 128, 64 * 128, 128,
                             None, None, None)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def batch(**kw):
    b = paged.zx_paged_batch(3, 5, 0x7FFFFFFF, 0x7FFFFFFF, 0x1000, 0x2000, 0x3000)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def rows(p=0x40000, t=8 * 128, h=128):
    return paged.zx_rows(p, t, h)


BAD_CACHES = [(dict(dtype=2), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED), (dict(head_dim=96), INVAL), (dict(head_dim=0), INVAL),
              (dict(page_tokens=48), INVAL), (dict(page_tokens=8), INVAL), (dict(page_tokens=8192), INVAL), (dict(n_pages=0), INVAL),
              (dict(kv_heads=0), INVAL), (dict(k=None), INVAL), (dict(v=0x20008), INVAL), (dict(k_token_stride=132), INVAL),
              (dict(k_token_stride=64), INVAL), (dict(v_head_stride=4), INVAL), (dict(k_page_stride=1 << 41), INVAL),
              (dict(k_scale=0x100), INVAL), (dict(block_tokens=64), INVAL), (dict(bounds=0x50000), INVAL),
              (dict(block_tokens=128, bounds=0x50000), INVAL), (dict(block_tokens=24, bounds=0x50000), INVAL),
              (dict(block_tokens=8, bounds=0x50000), INVAL), (dict(block_tokens=32, bounds=0x50004), INVAL)]
BAD_BATCHES = [(dict(q_start=None), INVAL), (dict(kv_len=None), INVAL), (dict(page_table=None), INVAL), (dict(n_seqs=65537), INVAL),
               (dict(table_width=1 << 27), INVAL)]


def calls(lib, c=None, b=None, n=7, **kw):
    """Each entry point with one thing changed."""
    c = cache() if c is None else c
    b = batch() if b is None else b
    r, o = kw.get("r", rows()), kw.get("o", rows(0x80000))
    yield "append", lib.zx_paged_append(C.byref(c), C.byref(b), n, C.byref(r), C.byref(r), None, None, None, 0, None, None, None)
    yield "attend", lib.zx_paged_attend(C.byref(c), C.byref(b), n, C.byref(r), 8, C.byref(o), None, 1.0, 1, 0, None, 0, None, 0, None, None)
    yield "select", lib.zx_paged_select(C.byref(c), C.byref(b), n, C.byref(r), 8, 4, 1, 1, P(0x90000), None, 0, None, None)


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_bad_caches(lib, kw, want):
    for name, st in calls(lib, c=cache(**kw)):
        assert st == want, name


@pytest.mark.parametrize("kw,want", BAD_BATCHES)
def test_bad_batches(lib, kw, want):
    for name, st in calls(lib, b=batch(**kw)):
        assert st == want, name


def test_null_structs_and_rows(lib):
    c, b, r = cache(), batch(), rows()
    assert lib.zx_paged_append(None, C.byref(b), 1, C.byref(r), C.byref(r), None, None, None, 0, None, None, None) == INVAL
    assert lib.zx_paged_append(C.byref(c), None, 1, C.byref(r), C.byref(r), None, None, None, 0, None, None, None) == INVAL
    for bad in (rows(p=None), rows(p=0x40008), rows(t=12), rows(h=4), rows(t=1 << 41)):
        for name, st in calls(lib, c=cache(block_tokens=32, bounds=0x50000), r=bad):
            assert st == INVAL, name
    assert lib.zx_paged_append(C.byref(c), C.byref(b), 1, C.byref(r), None, None, None, None, 0, None, None, None) == INVAL
    # queries without heads or without a place to go
    assert lib.zx_paged_append(C.byref(c), C.byref(b), 1, C.byref(r), C.byref(r), None, None, C.byref(r), 0, C.byref(r), None, None) == INVAL
    assert lib.zx_paged_append(C.byref(c), C.byref(b), 1, C.byref(r), C.byref(r), None, None, C.byref(r), 8, None, None, None) == INVAL


def test_rotary_refusals(lib):
    c, b, r = cache(), batch(), rows()
    for inv, dims in ((None, 64), (0x1004, 64), (0x1000, 0), (0x1000, 24), (0x1000, 256)):
        rot = paged.zx_rotary(inv, dims, 0, 1.0, 0)
        assert lib.zx_paged_append(C.byref(c), C.byref(b), 1, C.byref(r), C.byref(r), C.byref(rot), None, None, 0, None, None, None) == INVAL


def test_attend_refusals(lib):
    c, b, r, o = cache(), batch(), rows(), rows(0x80000)

    def attend(c=c, n=7, heads=8, scale=1.0, causal=1, window=0, blocks=None, nb=0, ws=None, size=0):
        return lib.zx_paged_attend(C.byref(c), C.byref(b), n, C.byref(r), heads, C.byref(o), None, scale, causal, window, blocks, nb, ws, size,
                                   None, None)
    for heads in (0, 3, 65538):
        assert attend(heads=heads) == INVAL
    for scale in (0.0, -1.0, math.nan, math.inf):
        assert attend(scale=scale) == INVAL
    assert attend(window=0x40000000) == INVAL
    assert attend(blocks=P(0x9000)) == INVAL and attend(nb=4) == INVAL
    assert attend(blocks=P(0x9000), nb=4) == INVAL                    # no bounds, no blocks
    cb = cache(block_tokens=32, bounds=0x50000)
    assert attend(c=cb, blocks=P(0x9000), nb=4, causal=0) == INVAL
    assert attend(c=cb, blocks=P(0x9000), nb=4, window=5) == INVAL
    assert attend(c=cb, blocks=P(0x9000), nb=65537) == INVAL
    assert attend(n=1 << 23) == INVAL
    assert lib.zx_paged_attend_workspace_bytes(C.byref(c), C.byref(b), 7, 8, 0, 0) == 0      # at most 320 tokens: nothing is split
    b = batch(table_width=500)
    need = lib.zx_paged_attend_workspace_bytes(C.byref(c), C.byref(b), 7, 8, 0, 0)
    assert need > 0
    assert attend() == INVAL                                          # no workspace
    assert attend(ws=P(0x100000), size=need - 1) == INVAL
    assert attend(ws=P(0x100008), size=need) == INVAL
    assert lib.zx_paged_attend_workspace_bytes(C.byref(c), C.byref(b), 7, 3, 0, 0) == 0
    # more work than 32-bit counts hold, more workgroups than a launch
    one = batch(max_q=1)
    assert lib.zx_paged_attend(C.byref(cb), C.byref(one), 1 << 22, C.byref(rows()), 8, C.byref(rows()), None, 1.0, 1, 0, P(0x9000), 4, None, 0,
                               None, None) == LIMIT
    huge = batch(n_seqs=65536, table_width=1 << 19)
    assert lib.zx_paged_attend(C.byref(cache(page_tokens=512, k_head_stride=512 * 128, v_head_stride=512 * 128)), C.byref(huge), 65536,
                               C.byref(r), 8, C.byref(o), None, 1.0, 1, 0, None, 0, P(0x100000), 1 << 62, None, None) == LIMIT
    # nothing to do
    assert attend(n=0) == OK
    assert lib.zx_paged_attend(C.byref(c), C.byref(batch(n_seqs=0)), 7, C.byref(r), 8, C.byref(o), None, 1.0, 1, 0, None, 0, None, 0, None,
                               None) == OK


def test_select_refusals(lib):
    cb, b, r = cache(block_tokens=32, bounds=0x50000), batch(), rows()

    def select(c=cb, n=7, heads=8, top=4, first=1, last=1, out=P(0x90000), ws=None, size=0):
        return lib.zx_paged_select(C.byref(c), C.byref(b), n, C.byref(r), heads, top, first, last, out, ws, size, None, None)
    assert select(c=cache()) == INVAL
    for kw in (dict(heads=0), dict(heads=3), dict(top=0), dict(top=1025), dict(first=4), dict(last=0xFFFFFFFF), dict(out=None)):
        assert select(**kw) == INVAL, kw
    assert lib.zx_paged_select_workspace_bytes(C.byref(cb), C.byref(b), 7) == 0        # ten blocks: no keys in memory
    b = batch(table_width=5000)
    need = lib.zx_paged_select_workspace_bytes(C.byref(cb), C.byref(b), 7)
    assert need > 0 and select() == INVAL and select(ws=P(0x100000), size=need - 1) == INVAL and select(ws=P(0x100001), size=need) == INVAL
    assert lib.zx_paged_select_workspace_bytes(C.byref(cache()), C.byref(b), 7) == 0
    assert select(n=0) == OK
    b = batch(max_q=1)
    assert select(n=1 << 22) == LIMIT


def test_python_refusals():
    """What the binding refuses by itself, on host tensors."""
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        zx.PagedBatch(i, i[:2], i[:2].view(2, 1))                     # not on a device
    for kw in (dict(head_dim=96), dict(page_tokens=100), dict(page_tokens=8), dict(block_tokens=128, page_tokens=64), dict(block_tokens=8),
               dict(dtype=zx.E8M0), dict(k=torch.zeros(1)), dict(bounds=torch.zeros(1)), dict(n_pages=0), dict(kv_heads=0),
               dict(k=torch.zeros(4, 2, 512, 128), v=torch.zeros(4, 2, 512, 128))):
        with pytest.raises(ValueError):
            zx.PagedKVCache(**{**dict(n_pages=4, kv_heads=2), **kw})
    for kw in (dict(dims=0), dict(dims=24), dict(dims=272), dict(dims=64, scaling="other"), dict(dims=64, base=0.0),
               dict(dims=64, scaling="bands", low=4.0, high=4.0), dict(dims=64, inv_freq=torch.zeros(32)),
               dict(dims=64, inv_freq=torch.zeros(31, dtype=torch.float64)),
               dict(dims=64, inv_freq=torch.zeros(32, dtype=torch.float64), scaling="linear")):
        with pytest.raises(ValueError):
            zx.Rotary(device="cpu", **kw)


def test_rows_apart():
    apart = zx.paged._apart
    assert apart((4, 8), (8 * 128, 128), 128) and apart((4, 8), (128, 4 * 128), 128) and apart((1, 8), (0, 128), 128)
    assert apart((4, 8), (3 * 8 * 128, 136), 128) and apart((0, 8), (5, 128), 128)
    for strides in ((0, 128), (8 * 128, 120), (7 * 128, 128), (128, 128), (8 * 128 - 8, 128)):
        assert not apart((4, 8), strides, 128), strides


def test_frequencies():
    f = zx.Rotary.frequencies(64, 10000.0)
    assert f.dtype == torch.float64 and f[0] == 1.0 and abs(f[1].item() - 10000.0 ** (-2 / 64)) < 1e-15
    assert torch.equal(zx.Rotary.frequencies(64, 10000.0, "linear", 4.0), f / 4.0)
    n = zx.Rotary.frequencies(64, 10000.0, "ntk", 4.0)
    assert n[0] == 1.0 and abs(n[-1].item() * 4.0 / f[-1].item() - 1.0) < 1e-12      # the slowest pair is divided by the factor
    b = zx.Rotary.frequencies(128, 500000.0, "bands", 8.0, 8192, 1.0, 4.0)
    f = zx.Rotary.frequencies(128, 500000.0)
    turns = 8192 * f / (2 * math.pi)
    assert torch.equal(b[turns > 4], f[turns > 4]) and torch.allclose(b[turns < 1], f[turns < 1] / 8, rtol=1e-15)
    mid = (turns >= 1) & (turns <= 4)
    assert mid.any() and (b[mid] <= f[mid]).all() and (b[mid] >= f[mid] / 8).all()
    y = zx.Rotary.frequencies(128, 10000.0, "yarn", 16.0, 4096)
    f = zx.Rotary.frequencies(128, 10000.0)
    assert torch.equal(y[:10], f[:10]) and torch.allclose(y[-5:], f[-5:] / 16, rtol=1e-15)
    assert (y.diff() < 0).all()
    r = zx.Rotary(128, scaling="yarn", factor=16.0, original=4096, device="cpu")
    assert abs(r.magnitude - (0.1 * math.log(16.0) + 1.0)) < 1e-12 and zx.Rotary(64, device="cpu").magnitude == 1.0
