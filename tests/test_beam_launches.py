"""What the beam search's entry points launch (CPU): workgroups that cover every logit, row and piece, within the limits of a launch.
The worker and the recorder are those of test_paged_launches.py."""
import ctypes as C
import random
import re

import pytest

from lossless_float_compression_amd import beams, paged, pages
from test_paged_launches import I32, I64, P, U32, ask, ceil  # noqa: F401

WS, WS_SIZE = 1 << 40, 1 << 44
THREADS = (1 << 32) - 1


class BeamArgs(C.Structure):
    _fields_ = [("logits", P), ("group_stride", I64), ("beam_stride", I64), ("scores", P), ("weights", P), ("finished", P), ("allowed", P), ("stat", P),
                ("cand", P), ("out_scores", P), ("parents", P), ("tokens", P), ("out_finished", P), ("err", P), ("scale", C.c_double), ("groups", U32),
                ("beams", U32), ("vocab", U32), ("n_out", U32), ("parts", U32), ("words", U32), ("tiles", U32), ("depth", U32), ("end", I32)]


class ForkArgs(C.Structure):
    _fields_ = [("refs", P), ("n_pages", U32), ("log_page", U32), ("err", P), ("table", P), ("held", P), ("n", U32), ("width", U32), ("cap", I32),
                ("parents", P), ("beams", U32), ("log_strip", U32), ("share", U32)]


def hexed(s):
    return bytes(s).hex()


def select(kind, G, K, V, M, allowed=None):
    c = beams.zx_beam_logits(0x10000000, K * V, V, kind, G, K, V)
    return ["zx_beam_select", [hexed(c), ["c_void_p", 0x1000], None, None, -1, ["c_void_p", allowed], ["c_double", 1.0], M, ["c_void_p", 0x2000],
                               ["c_void_p", 0x3000], ["c_void_p", 0x4000], ["c_void_p", 0x5000], ["c_void_p", WS], ["c_size_t", WS_SIZE], None, None],
            C.sizeof(BeamArgs)]


def test_select(ask):  # noqa: F811
    rng = random.Random(1)
    cases = [(k, G, K, V, M) for k in (0, 1, 2) for G, K, V, M in [(1, 1, 1, 1), (1, 4, 32000, 8), (64, 8, 128256, 16), (1, 64, 1 << 24, 64), (1 << 20, 4, 100, 4),
                                                                  (3 << 20, 5, 9, 5), (16000000, 1, 1, 1), (2000, 1, 32000, 4)]]
    for _ in range(1500):
        V = int(2 ** rng.uniform(0, 24))
        K = rng.randint(1, 64)
        cases.append((rng.randrange(3), max(1, int(2 ** rng.uniform(0, 30) / (K * V))), K, V, rng.randint(1, 64)))
    out = ask([select(*c, allowed=rng.choice((None, 0x6000))) for c in cases])
    for case, (ret, launches) in zip(cases, out):
        kind, G, K, V, M = case
        if ret == 7:                                             # more parts than a launch takes
            assert G * K * ceil(V, 1024) >= 1 << 24 and not launches, case
            continue
        assert ret == 0 and len(launches) == 2, case
        (name, grid, block, arg), (pick, pgrid, pblock, joined) = launches
        a = BeamArgs.from_buffer_copy(bytes.fromhex(arg))
        pieces = int(re.search(r"k_beam_partsILi\dELi(\d)E", name).group(1))
        tile = pieces * 256 * (4 if kind == 2 else 8)
        assert block == 256 and grid == [G * K * a.parts, 1, 1] and grid[0] * block <= THREADS, case
        assert 1 <= a.tiles <= 8 and a.tiles * tile <= 65536, case
        assert (a.parts - 1) * a.tiles * tile < V <= a.parts * a.tiles * tile, case      # all of a row, and no part without any of it
        assert "k_beam_pick" in pick and pgrid == [G, 1, 1] and pblock in (256, 1024) and pgrid[0] * pblock <= THREADS, case
        depth = BeamArgs.from_buffer_copy(bytes.fromhex(joined)).depth
        assert 1 <= depth <= M and (depth == 1 or K * a.parts * depth <= pblock), case


def test_fork(ask):  # noqa: F811
    rng = random.Random(2)
    cases = [(1, 1, 0), (1, 2048, 1), (1, 2048, 100000), (65536, 1, 1), (65536, 1, 9000), (32, 2048, 70), (64, 8, 2068), (1, 4, 70)]
    for _ in range(500):
        K = int(2 ** rng.uniform(0, 11))
        cases.append((max(1, int(2 ** rng.uniform(0, 16)) // K), K, int(2 ** rng.uniform(0, 17))))
    pool = hexed(pages.zx_page_pool(1000, 16, 0x1000))
    calls = [["zx_pages_fork", [pool, hexed(pages.zx_page_rows(0x2000, 0x3000, G * K, W)), K, ["c_void_p", 0x4000], None, None], C.sizeof(ForkArgs)]
             for G, K, W in cases]
    for case, (ret, launches) in zip(cases, ask(calls)):
        G, K, W = case
        assert ret == 0, case
        name, grid, block, arg = launches[0]
        a = ForkArgs.from_buffer_copy(bytes.fromhex(arg))
        assert "k_pages_fork" in name and a.beams == K and a.width == W and a.share >= 1 and a.log_strip >= 2, case
        assert grid == [G * a.share, 1, 1] and grid[0] * block <= THREADS, case
        assert 4 * (3 * K + (K << a.log_strip)) <= 65536 and (K << a.log_strip) <= 8 * block, case      # local memory; entries of a thread
        assert len(launches) == (1 if a.share == 1 else 2), case                         # the lengths are written once
        if a.share > 1:
            assert "fork_held" in launches[1][0] and launches[1][1] == [G, 1, 1] and a.share <= ceil(W, 1 << a.log_strip), case


def test_extend_trim_and_compact(ask):  # noqa: F811
    rng = random.Random(3)
    cases = [(n, s, w) for n in (1, 2, 4096, 4097, 1 << 23) for s in (0, 1, 2048) for w in (0, 1, 9000)]
    cases += [(rng.randint(1, 1 << 23), rng.randint(0, 2048), rng.randint(0, 20000)) for _ in range(200)]
    calls = []
    for n, s, w in cases:
        pool, rows = hexed(pages.zx_page_pool(n, 16, 0x1000)), hexed(pages.zx_page_rows(0x2000, 0x3000, s, w))
        copies = hexed(pages.zx_page_copies(0x4000, 0x5000, max(s, n // 2), 0))
        ws = [["c_void_p", WS], ["c_size_t", WS_SIZE], None, None]
        calls += [["zx_pages_extend", [pool, rows, ["c_void_p", 0x6000], 0x7FFFFFFF, 0x7FFFFFFF, ["c_void_p", 0x7000], copies, *ws], 8],
                  ["zx_pages_trim", [pool, rows, None, None, None], 8], ["zx_pages_compact", [pool, rows, ["c_void_p", 0x8000], copies, *ws], 8]]
    out = ask(calls)
    for i, (n, s, w) in enumerate(cases):
        (r0, extend), (r1, trim), (r2, compact) = out[3 * i:3 * i + 3]
        seg = ceil(n, 4096)
        assert r0 == r1 == r2 == 0
        assert [x[1][0] for x in extend] == ([1] if seg == 1 else [1 + seg, seg])
        assert [x[1][0] for x in trim] == ([s] if s else [])
        if seg == 1 and s * w <= 16384:
            assert [x[1][0] for x in compact] == [1]
        else:
            assert [x[1][0] for x in compact[:2]] == [seg, seg] and len(compact) == 3 and compact[2][1][0] >= 1 + s
        assert all(x[1][0] * x[2] <= THREADS for x in (*extend, *trim, *compact))


def test_copies_and_joins(ask):  # noqa: F811
    rng = random.Random(4)
    calls, want = [], []
    for _ in range(300):
        H, D, T, dtype = rng.randint(1, 70), rng.choice((64, 128, 256)), 16 << rng.randint(0, 8), rng.randrange(2)
        C_ = rng.choice((0, 16))
        n, cap = rng.choice((1, 2, 39, 40, 41, 80, 95)), int(2 ** rng.uniform(0, 22))
        one = paged.zx_paged_cache(dtype, 100, H, D, T, C_, 0x10000000, 0x20000000, H * T * D, T * D, D, H * T * D, T * D, D, None, None, 0x30000000 if C_ else None)
        calls.append(["zx_paged_copy", [hexed((paged.zx_paged_cache * n)(*[one] * n)), n, hexed(pages.zx_page_copies(0x4000, 0x5000, cap, 0)), None, None], 8])
        e = 1 if dtype else 2
        each = 2 * ceil(H * T * D * e, 16384) + (ceil(H * (T // 16) * D * 4, 16384) if C_ else 0)
        want.append([min(8192, cap * m * each) for m in [40] * (n // 40) + ([n % 40] if n % 40 else [])])
    for _ in range(300):
        k, N, H, D = rng.randint(1, 16), int(2 ** rng.uniform(0, 24)), rng.randint(1, 64), rng.choice((64, 128, 256))
        r = paged.zx_rows(0x10000000, H * D, D)
        calls.append(["zx_attention_merge", [hexed((paged.zx_rows * k)(*[r] * k)), hexed((P * k)(*[0x1000] * k)), k, N, H, D, hexed(r), None, None], 8])
        want.append([ceil(N * H * D // 8, 256)] if N * H * D // 8 <= 0xFFFFFF00 else None)
    for w, (ret, launches) in zip(want, ask(calls)):
        if w is None:
            assert ret == 7 and not launches
        else:
            assert ret == 0 and [x[1][0] for x in launches] == w and all(x[1][0] * x[2] <= THREADS for x in launches)
