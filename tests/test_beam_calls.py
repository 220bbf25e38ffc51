"""What the beam search's bindings do with their arguments and workspaces (CPU): host tensors that say they are the device's, and
library functions that stand in for the kernels' entry points."""
import weakref

import pytest
import torch

import lossless_float_compression_amd as zx
from lossless_float_compression_amd import beams, pages
from test_beam_launches import select
from test_paged_launches import ask  # noqa: F401


class Here(torch.Tensor):
    """A host tensor that passes for one of the current device (index -1)."""
    is_cuda = True


def here(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Here)


class Spaces:
    """Allocates workspaces, and knows whether the last one is still there."""

    def __init__(self):
        self.last = None

    def new_empty(self, n):
        t = torch.empty(n, dtype=torch.uint8)
        self.last = weakref.ref(t)
        return t

    def holds(self, address):
        t = self.last()
        return t is not None and t.data_ptr() == address


class Library:
    """Entry points that note whether the workspace that they are given is held while they run."""

    def __init__(self, spaces):
        self.spaces, self.ran = spaces, []

    def _size(self, *a):
        return 4096

    zx_beam_select_workspace_bytes = zx_pages_extend_workspace_bytes = zx_pages_compact_workspace_bytes = _size

    def _call(self, name, at):
        def call(*a):
            self.ran.append((name, at is None or self.spaces.holds(a[at])))
            return 0
        return call

    def __getattr__(self, name):
        return self._call(name, {"zx_beam_select": 12, "zx_pages_extend": 7, "zx_pages_compact": 4, "zx_attention_merge": None}[name])


@pytest.fixture
def library(monkeypatch):
    spaces = Spaces()
    lib = Library(spaces)
    for m in (beams, pages):
        monkeypatch.setattr(m, "_bound", lib)
        monkeypatch.setattr(m, "_stream_of", lambda index: None)
    monkeypatch.setattr(beams, "_needs", {})
    monkeypatch.setattr(pages, "_device", lambda: -1)
    of = lambda t: torch.empty(0, dtype=t).new_empty                     # noqa: E731
    monkeypatch.setattr(beams, "_makers", {-1: (of(torch.float32), of(torch.int32), of(torch.bool), spaces.new_empty)})
    return lib


def test_workspaces_are_held_until_the_launches_are_enqueued(library):
    """An entry point runs without the interpreter's lock: memory let go before it returns can be given to another thread on the same stream,
    whose launches then come between these."""
    zx.beam_select(here(2, 4, 100, dtype=torch.bfloat16), here(2, 4, dtype=torch.float32))
    pool = zx.PagePool(64, 16, refs=here(64))
    pool._bytes = library.spaces
    batch = zx.PagedBatch(here(5), here(4), here(4, 8))
    copies = zx.PageCopies(64, pairs=here(64, 3), count=here(1))
    pool.extend(batch, here(4), copies=copies)
    pool.compact(here(4, 8), here(4), copies=copies, remap=here(64))
    pool.compact(copies=copies, remap=here(64))
    assert library.ran == [("zx_beam_select", True), ("zx_pages_extend", True), ("zx_pages_compact", True), ("zx_pages_compact", True)]


SMALLEST = 1e-36


def test_scales_too_small_for_32_bits_are_refused(library):
    """Below about 1e-45 the factor in 32 bits is zero and zero times minus infinity NaN; below 1e-38 differences of logits that pass
    32 bits would still matter."""
    x, s = here(2, 4, 100, dtype=torch.bfloat16), here(2, 4, dtype=torch.float32)
    for scale in (5e-324, 1e-46, 1e-38, SMALLEST * (1 - 1e-6)):
        with pytest.raises(ValueError, match="scale"):
            zx.beam_select(x, s, scale=scale)
    assert library.ran == []
    for scale in (SMALLEST, 1e-30, 1e30):
        zx.beam_select(x, s, scale=scale)
    assert len(library.ran) == 3


def test_the_entry_point_refuses_them_too(ask):  # noqa: F811
    def one(scale):
        c = select(0, 2, 4, 1000, 8)
        c[1][6] = ["c_double", scale]
        return c
    got = ask([one(x) for x in (5e-324, 1e-46, 1e-38, SMALLEST * (1 - 1e-6), SMALLEST, 1e30, 1.1e30)])
    assert [(ret, len(launches)) for ret, launches in got] == [(1, 0)] * 4 + [(0, 2)] * 2 + [(1, 0)]


@pytest.mark.parametrize("shape", [(1, 1, (1 << 24) + 1), (1, 1, (1 << 32) + 5), (1 << 31, 1, 1), ((1 << 32) + 2, 1, 1)])
def test_sizes_past_32_bits_are_refused(library, shape):
    """A count passed on in 32 bits would be taken for what is left of it."""
    x = torch.empty(shape, dtype=torch.bfloat16, device="meta").as_subclass(Here)
    s = torch.empty(shape[:2], device="meta").as_subclass(Here)
    with pytest.raises(ValueError, match="2\\^24 tokens"):
        zx.beam_select(x, s)
    assert library.ran == []


def test_joined_in_place_among_interleaved_parts(library):
    """Parts side by side in one tensor, [token, part, head, channel] and others: one of them may be written. What shares
    memory with another part is refused all the same."""
    bf = dict(dtype=torch.bfloat16)
    lses = [here(5, 4, dtype=torch.float32) for _ in range(3)]
    layouts = (here(5, 3, 4, 64, **bf).unbind(1), here(5, 4, 3, 64, **bf).unbind(2), here(5, 4, 192, **bf).split(64, 2), here(3, 5, 4, 64, **bf).unbind(0),
               [t.transpose(0, 1) for t in here(3, 4, 5, 64, **bf).unbind(0)])
    for outs in layouts:
        for i in range(3):
            assert zx.merge_attention(outs, lses, out=outs[i]) is outs[i]
        spare = here(5, 4, 64, **bf)
        assert zx.merge_attention([outs[0], spare], lses[:2], out=outs[2]) is outs[2]        # beside them
        assert zx.merge_attention([outs[0], outs[1], outs[1]], lses, out=outs[1]) is outs[1]
    assert len(library.ran) == 25
    one = here(8, 4, 64, **bf)
    wide = here(5, 3, 4, 64, **bf)
    flat = here(5 * 4 * 64 + 64, **bf)
    bad = [([one[:5], one[3:]], one[:5]), ([one[1:6], one[:5]], one[:5]), ([wide[:, 0], wide[:, 1, :1].expand(5, 4, 64)], wide[:, 1]),
           ([wide[:, 0], wide[:1, 1].expand(5, 4, 64)], wide[:, 1]), ([flat[:1280].view(5, 4, 64)], flat[8:1288].view(5, 4, 64)),
           ([one[:5]], one[:5].flatten()[:1280].view(4, 5, 64).transpose(0, 1))]
    for i, (outs, out) in enumerate(bad):
        with pytest.raises(ValueError, match="shares memory"):
            zx.merge_attention(outs, lses[:len(outs)], out=out)
            pytest.fail(f"call {i} was taken")
