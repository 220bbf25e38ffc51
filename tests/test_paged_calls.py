"""What the paged K/V cache's binding does with its arguments (CPU)."""
import ctypes as C

import pytest
import torch

import lossless_float_compression_amd as zx


def bare(**kw):
    """A cache without device memory, for what happens before any of it is touched."""
    c = object.__new__(zx.PagedKVCache)
    for k, v in {**dict(_index=-1, device=torch.device("cpu"), head_dim=128, kv_heads=2, block_tokens=16, dtype=zx.BF16), **kw}.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("stream", [C.c_void_p(0), C.c_void_p(0x1000), 0x1000, "side"])
def test_raw_streams_are_refused(stream):
    """A workspace lies on the stream that uses it, which a raw handle does not allow."""
    c, t = bare(), torch.zeros((1, 2, 128), dtype=torch.bfloat16)
    for call in (lambda: c.append(t, t, None, stream=stream), lambda: c.attend(t, None, stream=stream), lambda: c.select(t, None, 4, stream=stream)):
        with pytest.raises(ValueError, match="torch stream"):
            call()
