"""Beam search: the choice of the next beams from the logits, and attention over parts of a context joined."""
from __future__ import annotations

import ctypes as C
from typing import NamedTuple, Optional, Sequence

import torch
import torch.autograd.forward_ad as _forward

from . import zx as _zx
from .pages import _away, _elsewhere, _meets, _stream_of
from .paged import _apart, _int32, _meet, _no_gradient, zx_rows

MOST_BEAMS = 64
MOST_VOCAB = 1 << 24
_LOGITS = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class zx_beam_logits(C.Structure):
    _fields_ = [("logits", C.c_void_p), ("group_stride", C.c_uint64), ("beam_stride", C.c_uint64), ("type", C.c_int32),
                ("n_groups", C.c_uint32), ("beams", C.c_uint32), ("vocab", C.c_uint32)]


class Beams(NamedTuple):
    """The next beams of each group, best first: `scores` float32, `parents` and `tokens` int32 and `finished` bool, all [groups, n]."""
    scores: torch.Tensor
    parents: torch.Tensor
    tokens: torch.Tensor
    finished: torch.Tensor


_bound = None
_needs = {}                              # workspace sizes, by the sizes that decide them
_MOST_NEEDS = 256
_makers = {}                             # by device: what allocates floats, words, flags and bytes there


def _like_what(index: int, device: torch.device):
    """Functions of a size that allocate float32, int32, bool and uint8 tensors (an empty tensor's own is the quickest way)."""
    m = _makers.get(index)
    if m is None:
        m = _makers[index] = tuple(torch.empty(0, dtype=t, device=device).new_empty for t in (torch.float32, torch.int32, torch.bool, torch.uint8))
    return m


def _lib():
    global _bound
    if _bound is None:
        L = _zx.lib()
        P, U32, I32, SZ, D = C.c_void_p, C.c_uint32, C.c_int32, C.c_size_t, C.c_double
        L.zx_beam_select_workspace_bytes.argtypes = [I32, U32, U32, U32, U32]
        L.zx_beam_select_workspace_bytes.restype = SZ
        L.zx_beam_select.argtypes = [C.POINTER(zx_beam_logits), P, P, P, I32, P, D, U32, P, P, P, P, P, SZ, P, P]
        L.zx_beam_select.restype = C.c_int
        L.zx_attention_merge.argtypes = [C.POINTER(zx_rows), C.POINTER(P), U32, U32, U32, U32, C.POINTER(zx_rows), P, P]
        L.zx_attention_merge.restype = C.c_int
        _bound = L
    return _bound


def _like(t: torch.Tensor, name: str, dtype: torch.dtype, shape, index: int) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on cuda:{index}")
    return t


def beam_select(logits: torch.Tensor, scores: torch.Tensor, n_out: Optional[int] = None, *, weights: Optional[torch.Tensor] = None,
                finished: Optional[torch.Tensor] = None, end: Optional[int] = None, allowed: Optional[torch.Tensor] = None,
                scale: float = 1.0, out: Optional[Beams] = None, err: Optional[torch.Tensor] = None, stream=None) -> Beams:
    """The n_out (1..64; default: as many as there are) best next beams of each group: beam b that has scored scores[g, b] goes on with token
    t for scores[g, b] + ln softmax(scale * logits[g, b])[t], and the candidates with the largest weights[g, b] times that are
    taken (equal ones: the earlier beam, then the larger logit, which scores in 64 bits may not show, then the earlier token).

    logits    bf16, fp16 or fp32 [groups, beams, vocab] (up to 64 beams, 2^24 tokens), any strides with neighbouring tokens
    scores    float32 [groups, beams]; -inf: the beam is not there (a search begins with all but one of them so)
    weights   float32 [groups, beams], positive, e.g. a length to a negative power; None: 1
    finished  bool [groups, beams]: beams whose only candidate is (end, scores[g, b]); needs `end`
    end       the token that ends a beam; None: none does
    allowed   int32 [groups, beams, ceil(vocab / 32)]: bit t % 32 of word t / 32 says whether token t may be taken; the softmax is over
              those that may.  None: all (logits of -inf are never taken)
    scale     one over a temperature, 1e-36 to 1e30
    out       `Beams` to write into; `out.scores`, `out.finished` may be the `scores` and `finished` given

    Returns `Beams`; `finished` says that a candidate's beam was or its token is `end`.  Behind a group's last candidate: score -inf,
    parent and token -1, which `PagePool.fork` takes for an empty row.  Beams with NaN or +inf logits or scores, or weights that are not positive
    numbers, are left out, with 4 in `err` (device int32 word).  Scores are formed and compared in 64 bits, sums of exponentials begin in 32.  stream: a torch stream to run on
    after the work already enqueued on the current one."""
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda or logits.dtype not in _LOGITS or logits.dim() != 3:
        raise ValueError("logits must be a bfloat16, float16 or float32 device tensor [groups, beams, vocab]")
    index, device = logits.get_device(), logits.device
    if _away(index, stream):
        return _elsewhere(device, stream, (logits, scores, weights, finished, allowed, err, *(out or ())),
                          lambda s: beam_select(logits, scores, n_out, weights=weights, finished=finished, end=end, allowed=allowed,
                                                scale=scale, out=out, err=err, stream=s))
    G, K, V = logits.shape
    M = K if n_out is None else int(n_out)
    if not 0 < K <= MOST_BEAMS or not 0 < M <= MOST_BEAMS or V == 0:
        raise ValueError(f"1 to {MOST_BEAMS} beams, 1 to {MOST_BEAMS} candidates and a vocabulary, please")
    if V > MOST_VOCAB or G > 0x7FFFFFFF // K:                # (counts are passed on in 32 bits)
        raise ValueError("up to 2^24 tokens, and fewer than 2^31 beams in all")
    sg, sk, sv = logits.stride()
    if sv != 1 and V > 1:
        raise ValueError("logits: neighbouring tokens must lie side by side")
    _like(scores, "scores", torch.float32, (G, K), index)
    pw = pf = pa = None
    if weights is not None:
        pw = _like(weights, "weights", torch.float32, (G, K), index).data_ptr()
    if end is None:
        end = -1
        if finished is not None:
            raise ValueError("finished needs end")
    elif not 0 <= end < V:
        raise ValueError("end must be a token")
    if finished is not None:
        pf = _like(finished, "finished", torch.bool, (G, K), index).data_ptr()
    if allowed is not None:
        pa = _like(allowed, "allowed", torch.int32, (G, K, (V + 31) // 32), index).data_ptr()
    if not (1e-36 <= scale <= 1e30):
        raise ValueError("scale must be a number from 1e-36 to 1e30")
    if logits.requires_grad or scores.requires_grad or (weights is not None and weights.requires_grad) or _forward._current_level >= 0:
        for t, name in ((logits, "logits"), (scores, "scores"), (weights, "weights")):
            if t is not None:
                _no_gradient(t, name)
    f32, i32, flags, raw = _like_what(index, device)
    if out is None:
        size = (G, M)
        out = Beams(f32(size), i32(size), i32(size), flags(size))
    else:
        for i, (t, name, dt) in enumerate(zip(out, Beams._fields, (torch.float32, torch.int32, torch.int32, torch.bool))):
            _like(t, "out." + name, dt, (G, M), index)
            # a group's scores and flags are read before its results are written
            own = scores if name == "scores" else finished if name == "finished" else None
            others = [u for u in (logits, weights, allowed, err, scores if own is not scores else None, finished if own is not finished else None,
                                  *out[i + 1:]) if u is not None]
            if any(_meets(t, u) for u in others) or (own is not None and _meets(t, own) and (t.data_ptr() != own.data_ptr() or M != K)):
                raise ValueError(f"out.{name} shares memory with another argument")
    e = None if err is None else _int32(err, "err", index).data_ptr()
    if G == 0:
        return out
    L = _bound or _lib()
    kind = _LOGITS[logits.dtype]
    key = (kind, G, K, V, M)
    need = _needs.get(key)
    if need is None:
        if len(_needs) >= _MOST_NEEDS:
            _needs.clear()
        need = _needs[key] = L.zx_beam_select_workspace_bytes(*key)
    ws = raw(need)                               # (held until the launches are enqueued: the call lets other threads run)
    st = L.zx_beam_select(C.byref(zx_beam_logits(logits.data_ptr(), sg if G > 1 else 0, sk if K > 1 else 0, kind, G, K, V)), scores.data_ptr(),
                          pw, pf, end, pa, scale, M, out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(),
                          ws.data_ptr(), need, e, _stream_of(index))
    if st != 0:
        raise _zx.ZxError("zx_beam_select", st)
    return out


def _part(t: torch.Tensor, name: str, shape, index: int, written: bool = False):
    """The rows, and the first byte that they reach and the one behind the last."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or t.shape != shape or t.get_device() != index:
        raise ValueError(f"{name} must be a bfloat16 tensor {list(shape)} on cuda:{index}")
    if t.requires_grad or _forward._current_level >= 0:
        _no_gradient(t, name)
    n, h, d = shape
    s0, s1, s2 = t.stride()
    p = t.data_ptr()
    if s2 == 1 and s1 == d and s0 == h * d and p % 16 == 0:          # (meets all that is asked for below)
        return zx_rows(p, s0, s1), p, p + 2 * n * s0
    if n < 2:
        s0 = 0
    if h < 2:
        s1 = 0
    if s2 != 1 or s0 % 8 or s1 % 8 or p % 16:
        raise ValueError(f"{name}: channels must be contiguous, and the start and the other strides multiples of 16 bytes")
    if written and not _apart((n, h), (s0, s1), d):
        raise ValueError(f"{name}: rows that are written must not overlap")
    return zx_rows(p, s0, s1), p, p + 2 * ((n - 1) * s0 + (h - 1) * s1 + d) if n else p


def _shared(o: zx_rows, r: zx_rows, shape) -> bool:
    """Whether rows that are written may share memory with a part's whose span they meet (parts may lie between each other's rows)."""
    n, h, d = shape
    steps = lambda x: sorted(((st, k) for st, k in ((x.token_stride, n), (x.head_stride, h)) if k > 1), reverse=True)   # noqa: E731
    return not _apart((n, h), (r.token_stride, r.head_stride), d) or _meet(steps(o), steps(r), (r.p - o.p) // 2, d)


def merge_attention(outs: Sequence[torch.Tensor], lses: Sequence[torch.Tensor], out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention over parts of a context joined: outs[i] (bf16 [tokens, heads, 64, 128 or 256]) and lses[i] (float32 [tokens, heads]) are
    what `PagedKVCache.attend` gives over part i, for up to 16 parts; the result is attention over all of them, and `lse`, where given, is
    filled with its ln of the sum of exp(scores).  So beams read the pages of their prompt once, as the rows of one
    sequence (causal=False), and their own pages each, from a table and lengths that begin behind the prompt.

    A part whose lse is -inf is not looked at; a row where all are is zero.  out and lse may be one of outs and of lses.
    stream: a torch stream to run on after the work already enqueued on the current one."""
    k = len(outs)
    if not 0 < k <= 16 or len(lses) != k:
        raise ValueError("1 to 16 parts, each with its lse")
    f = outs[0]
    shape = f.shape if isinstance(f, torch.Tensor) else ()
    if len(shape) != 3 or shape[2] not in (64, 128, 256) or shape[1] == 0 or not f.is_cuda:
        raise ValueError("outs must be bfloat16 device tensors [tokens, heads, 64, 128 or 256]")
    index, device = f.get_device(), f.device
    if _away(index, stream):
        return _elsewhere(device, stream, (*outs, *lses, out, lse), lambda s: merge_attention(outs, lses, out, lse, s))
    n, heads, d = shape
    rows = shape[:2]
    size = 4 * n * heads
    parts, where, follow = [], [], _forward._current_level >= 0
    for t, l in zip(outs, lses):
        parts.append(_part(t, "a part", shape, index))
        where.append(_like(l, "an lse", torch.float32, rows, index).data_ptr())
        if follow or l.requires_grad:
            _no_gradient(l, "an lse")
    if out is None:
        out = f.new_empty(shape)
        o = zx_rows(out.data_ptr(), heads * d, d)
    else:
        o, p, q = _part(out, "out", shape, index, True)
        if any(p < x + size and x < q for x in where) or any(p < y and x < q and not (
                x == p and r.token_stride == o.token_stride and r.head_stride == o.head_stride) and _shared(o, r, shape) for r, x, y in parts):
            raise ValueError("out shares memory with a part and is not that part")
        if lse is not None and _meets(out, lse):
            raise ValueError("out and lse share memory")
    pl = None
    if lse is not None:
        pl = _like(lse, "lse", torch.float32, rows, index).data_ptr()
        if follow or lse.requires_grad:
            _no_gradient(lse, "lse")
        for (_, x, y), z in zip(parts, where):
            if pl < y and x < pl + size or pl != z and pl < z + size and z < pl + size:
                raise ValueError("lse shares memory with a part and is not that part's")
    if n == 0:
        return out
    st = (_bound or _lib()).zx_attention_merge((zx_rows * k)(*[r for r, _, _ in parts]), (C.c_void_p * k)(*where), k, n, heads, d, C.byref(o), pl,
                                               _stream_of(index))
    if st != 0:
        raise _zx.ZxError("zx_attention_merge", st)
    return out
