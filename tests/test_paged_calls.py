"""What the paged K/V cache's binding does with its arguments (CPU)."""
import ctypes as C

import pytest
import torch

import lossless_float_compression_amd as zx


def bare(**kw):
    """A cache without device memory, for what happens before any of it is touched."""
    c = object.__new__(zx.PagedKVCache)
    for k, v in {**dict(_index=-1, device=torch.device("cpu"), head_dim=128, kv_heads=2, block_tokens=16, dtype=zx.BF16, _gradients=False), **kw}.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("stream", [C.c_void_p(0), C.c_void_p(0x1000), 0x1000, "side"])
def test_raw_streams_are_refused(stream):
    """A workspace lies on the stream that uses it, which a raw handle does not allow."""
    c, t = bare(), torch.zeros((1, 2, 128), dtype=torch.bfloat16)
    for call in (lambda: c.append(t, t, None, stream=stream), lambda: c.attend(t, None, stream=stream), lambda: c.select(t, None, 4, stream=stream)):
        with pytest.raises(ValueError, match="torch stream"):
            call()


def test_gradients_are_refused(monkeypatch):
    """Inputs that autograd follows, in either mode, and a cache whose own tensors it follows."""
    import torch.autograd.forward_ad as forward

    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    c, t = bare(), torch.zeros((3, 4, 128), dtype=torch.bfloat16)
    assert c._rows(t, "q", None, None).token_stride == 4 * 128
    wants = t.clone().requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        c._rows(wants, "q", None, None)
    with torch.no_grad():
        c._rows(wants, "q", None, None)
    batch = type("Batch", (), dict(_index=-1, device="cpu"))
    c._tensors = (t,)
    with forward.dual_level():
        dual = forward.make_dual(t, torch.ones_like(t))
        for call in (lambda: c.append(dual, t, batch), lambda: c.append(t, t, batch, q=dual), lambda: c.attend(dual, batch),
                     lambda: c.attend(t, batch, out=dual), lambda: c.select(dual, batch, 4)):
            with pytest.raises(ValueError, match="gradient"):
                call()
            with torch.no_grad(), pytest.raises(ValueError, match="gradient"):   # (tangents are carried without grad mode)
                call()
        c._followed(t, None)
    c._gradients, c._tensors = True, (t, torch.ones(2, requires_grad=True))
    for call in (lambda: c.append(t, t, batch), lambda: c.attend(t, batch), lambda: c.select(t, batch, 4)):
        with pytest.raises(ValueError, match="gradient"):
            call()
    with torch.no_grad():
        c._followed(t, None)


def test_a_batch_remembers_only_so_many_sizes():
    """A long-lived batch that is called with ever other numbers of rows."""
    b = object.__new__(zx.PagedBatch)
    b._needs = {}
    for n in range(2000):
        assert b._ask(("sizes", n), lambda x: 3 * x, n) == 3 * n and b._needs[("sizes", n)] == 3 * n
    assert len(b._needs) <= 256


def rows_of(shape, strides, offset, width):
    """Every element of the rows, as a set."""
    at = [offset]
    for n, st in zip(shape, strides):
        at = [x + i * st for x in at for i in range(n)]
    return {x + c for x in at for c in range(width)}


def test_keys_and_values_that_share_memory():
    """Pages side by side, one inside the other's strides, and any offset between: none that share is taken for apart, and the
    layouts that keep keys and values of a page, a token or a head together are not taken for shared."""
    steps = lambda shape, strides: sorted(((st, n) for st, n in zip(strides, shape) if n > 1), reverse=True)   # noqa: E731
    P, H, T, D = 3, 2, 4, 8
    shape = (P, H, T)
    heads, tokens = (H * T * D, T * D, D), (H * T * D, D, H * D)
    good = [(heads, heads, P * H * T * D), (tokens, tokens, P * H * T * D), (heads, tokens, P * H * T * D),         # two allocations
            ((2 * H * T * D, T * D, D), (2 * H * T * D, T * D, D), H * T * D),                                      # [page, 2, head, token, D]
            ((2 * H * T * D, T * D, D), (2 * H * T * D, D, H * D), H * T * D),                                      # the same, values by token
            ((2 * H * T * D, 2 * T * D, D), (2 * H * T * D, 2 * T * D, D), T * D),                                  # [page, head, 2, token, D]
            ((2 * H * T * D, D, 2 * H * D), (2 * H * T * D, D, 2 * H * D), H * D),                                  # [page, token, 2, head, D]
            ((2 * H * T * D, 2 * D, 2 * H * D), (2 * H * T * D, 2 * D, 2 * H * D), D)]                              # [page, token, head, 2, D]
    for a, b, off in good:
        assert not rows_of(shape, a, 0, D) & rows_of(shape, b, off, D)
        assert not zx.paged._meet(steps(shape, a), steps(shape, b), off, D), (a, b, off)
        assert not zx.paged._meet(steps(shape, b), steps(shape, a), -off, D), (a, b, off)
    layouts = {x for g in good for x in g[:2]}
    for a in layouts:
        mine = rows_of(shape, a, 0, D)
        for b in layouts:
            for off in range(-2 * P * H * T * D, 2 * P * H * T * D, 4):
                shared = bool(mine & rows_of(shape, b, off, D))
                meet = zx.paged._meet(steps(shape, a), steps(shape, b), off, D)
                assert meet or not shared, (a, b, off)
                if a == b:                                      # exact where both step alike
                    assert meet == shared, (a, b, off)
    assert zx.paged._meet([], [], 0, 8) and zx.paged._meet([], [], 7, 8) and not zx.paged._meet([], [], 8, 8)


class Pool:
    """What stow and restore need of a slot pool, noting the device that is current when its launches would run."""

    def __init__(self, current):
        self.dtype, self.signmant, self.current, self.ran = zx.BF16, torch.zeros(1), current, []

    def append(self, blocks, slots, err=None):
        self.ran.append(self.current[0])
        return torch.zeros_like(slots)

    def decode(self, slots, out, err=None):
        self.ran.append(self.current[0])


def test_stow_and_restore_run_on_the_device_of_the_cache(monkeypatch):
    """With another device current, the pool's launches would go to that one's stream; a pool on another device is refused."""
    current = [0]

    class Device:
        def __init__(self, d):
            self.d = 1

        def __enter__(self):
            self.old, current[0] = current[0], self.d

        def __exit__(self, *a):
            current[0] = self.old

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(zx.paged, "_int32", lambda t, *a: t)
    raw = torch.zeros((2, 1, 512, 128), dtype=torch.bfloat16)
    c = bare(_index=1, k=raw, v=raw.clone(), bounds=None, n_pages=2, kv_heads=1, page_tokens=512, torch_dtype=torch.bfloat16)
    pool = Pool(current)
    pages, slots = torch.tensor([1]), torch.tensor([[[0]], [[1]]], dtype=torch.int32)
    c.stow(pages, pool, slots)
    c.restore(pages, pool, slots)
    assert pool.ran == [1, 1] and current == [0]
    pool.signmant = torch.zeros(1, device="meta")
    for call in (lambda: c.stow(pages, pool, slots), lambda: c.restore(pages, pool, slots)):
        with pytest.raises(ValueError, match="the pool is on"):
            call()
