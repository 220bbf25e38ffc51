"""What the paged K/V cache's entry points launch (CPU): enough workgroups for every row, enough
workspace for every piece, a join for every split row tile.

A worker process binds libzx.so to a recorder in place of the HIP runtime (launch_recorder.c), makes the
calls and hands back grids and kernel arguments.  The items that the kernels would look for are counted
here, by the rules that they follow on the device."""
import ctypes as C
import json
import os
import random
import re
import subprocess
import sys

import numpy as np
import pytest

from lossless_float_compression_amd import paged, zx

HERE = os.path.dirname(os.path.abspath(__file__))
U32, U64, I32, I64, P = C.c_uint32, C.c_uint64, C.c_int32, C.c_int64, C.c_void_p

WORKER = r"""
import ctypes as C, json, sys
job = json.load(sys.stdin)
rec = C.CDLL(job["recorder"], mode=C.RTLD_GLOBAL)
lib = C.CDLL(job["lib"])
class Dim(C.Structure):
    _fields_ = [(x, C.c_uint32) for x in "xyz"]
class Record(C.Structure):
    _fields_ = [("name", C.c_char * 256), ("grid", Dim), ("block", Dim), ("arg", C.c_ubyte * 512)]
records = (Record * 4096).in_dll(rec, "zr_launches")
count, size = C.c_int.in_dll(rec, "zr_count"), C.c_size_t.in_dll(rec, "zr_bytes")
for f in ("zx_paged_attend_workspace_bytes", "zx_paged_select_workspace_bytes"):
    getattr(lib, f).restype = C.c_size_t
def arg(a):
    if isinstance(a, str):
        return C.create_string_buffer(bytes.fromhex(a))
    if isinstance(a, list):
        return getattr(C, a[0])(a[1])
    return a
out = []
for name, args, nbytes in job["calls"]:
    count.value, size.value = 0, nbytes
    ret = getattr(lib, name)(*[arg(a) for a in args])
    out.append([ret, [[r.name.decode(), [r.grid.x, r.grid.y, r.grid.z], r.block.x, bytes(r.arg[:nbytes]).hex()] for r in records[:count.value]]])
json.dump(out, sys.stdout)
"""


class Cache(C.Structure):
    _fields_ = [("k", P), ("v", P), ("strides", I64 * 4), ("tokens", U32 * 2), ("k_scale", P), ("v_scale", P), ("bounds", P),
                ("n_pages", U32), ("heads", U32), ("log_page", U32), ("log_block", U32)]


class Batch(C.Structure):
    _fields_ = [("q_start", P), ("kv_len", P), ("table", P), ("n_seqs", U32), ("width", U32), ("n_tokens", U32), ("max_q", U32), ("cap", I32), ("err", P)]


class Rows(C.Structure):
    _fields_ = [("p", P), ("token", I64), ("head", I64)]


class AttendArgs(C.Structure):
    _fields_ = [("c", Cache), ("b", Batch), ("q", Rows), ("out", Rows), ("lse", P), ("blocks", P), ("part", P), ("stat", P), ("scale", C.c_float),
                ("causal", I32), ("window", I32), ("group", U32), ("q_heads", U32), ("n_blocks", U32), ("lo_rows", U32), ("hi_rows", U32),
                ("slots", U32), ("pieces", U32), ("goal", U32), ("one_round", U32), ("least", U32)]


class SelectArgs(C.Structure):
    _fields_ = [("c", Cache), ("b", Batch), ("q", Rows), ("blocks", P), ("keys", P), ("group", U32), ("top_k", U32), ("keep_first", U32),
                ("keep_last", U32), ("nb", U32), ("slab0", U32), ("slab", U32), ("per", U32), ("head_dim", U32)]


class Turn(C.Structure):
    _fields_ = [("inv_freq", P), ("positions", P), ("half", U32), ("interleaved", I32), ("magnitude", C.c_float)]


class AppendArgs(C.Structure):
    _fields_ = [("c", Cache), ("b", Batch), ("k", Rows), ("v", Rows), ("q", Rows), ("qo", Rows), ("turn", Turn), ("kv_groups", U32), ("kv_log", U32),
                ("q_heads", U32), ("log_seg", U32)]


WS, WS_SIZE = 1 << 40, 1 << 44          # where the workspace lies


class Call:
    """Sequences with `new` new and `kv` total tokens, and the structs that describe them."""

    def __init__(self, H, G, D, new, kv, dtype=0, T=64, block=0, max_q=None, room=None):
        self.H, self.G, self.D, self.T, self.block = H, G, D, T, block
        self.new, self.kv = np.array(new, dtype=np.int64), np.array(kv, dtype=np.int64)
        self.n = int(self.new.sum())
        self.room = int(self.kv.max()) if room is None else room
        self.max_q = int(self.new.max()) if max_q is None else max_q
        self.cache = paged.zx_paged_cache(dtype, 1 << 20, H, D, T, block, 0x10000000, 0x20000000, H * T * D, T * D, D, H * T * D, T * D, D, None, None,
                                          0x30000000 if block else None)
        self.batch = paged.zx_paged_batch(len(new), -(-self.room // T), self.max_q, self.room, 0x1000, 0x2000, 0x3000)
        self.rows = paged.zx_rows(0x40000000, H * G * D, D)
        self.label = f"H {H} G {G} D {D} dtype {dtype} T {T} block {block} n_seqs {len(new)} new {list(new)[:4]} kv {list(kv)[:4]} room {self.room}"

    def attend(self, window=0, blocks=0):
        self.window, self.n_blocks = window, blocks
        s = [bytes(x).hex() for x in (self.cache, self.batch, self.rows)]
        return [["zx_paged_attend_workspace_bytes", [s[0], s[1], self.n, self.H * self.G, window, blocks], 0],
                ["zx_paged_attend", [s[0], s[1], self.n, s[2], self.H * self.G, s[2], None, ["c_float", 0.125], 1, window,
                                     ["c_void_p", 0x50000000 if blocks else None], blocks, ["c_void_p", WS], ["c_size_t", WS_SIZE], None, None],
                 C.sizeof(AttendArgs)]]

    def select(self):
        s = [bytes(x).hex() for x in (self.cache, self.batch, self.rows)]
        return [["zx_paged_select_workspace_bytes", [s[0], s[1], self.n], 0],
                ["zx_paged_select", [s[0], s[1], self.n, s[2], self.H * self.G, 8, 1, 1, ["c_void_p", 0x50000000], ["c_void_p", WS],
                                     ["c_size_t", WS_SIZE], None, None], C.sizeof(SelectArgs)]]

    def append(self):
        s = [bytes(x).hex() for x in (self.cache, self.batch, self.rows)]
        return [["zx_paged_append", [s[0], s[1], self.n, s[2], s[2], None, None, s[2], self.H * self.G, s[2], None, None], C.sizeof(AppendArgs)]]


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("recorder") / "recorder.so")
    subprocess.check_call(["gcc", "-O1", "-shared", "-fPIC", "-o", so, os.path.join(HERE, "launch_recorder.c")])
    zx.lib()                             # (builds it if nothing is built)
    lib = os.path.join(os.path.dirname(paged.__file__), "libzx.so")

    def run(calls):
        r = subprocess.run([sys.executable, "-c", WORKER], input=json.dumps(dict(recorder=so, lib=lib, calls=calls)), capture_output=True, text=True,
                           timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
        return json.loads(r.stdout)
    return run


def ceil(a, b):
    return -(-a // b)


def steps(new, kv, window, unit):
    """Steps of `unit` tokens that cover what a sequence's rows see, one at least."""
    first = kv - new - window + 1
    lo = np.where((window > 0) & (first > 0), first, 0) & ~15
    return np.where(kv > lo, ceil(kv - lo, unit), 1)


def split(call, a, rows, unit):
    """(row tiles, pieces of each) of the sequences that a launch with arguments `a` takes."""
    of = call.new * call.G
    mine = (of > a.lo_rows) & (of <= a.hi_rows)
    tiles, st = ceil(of[mine], rows), steps(call.new[mine], call.kv[mine], call.window, unit)
    if a.slots == 0:
        return mine, tiles, np.ones_like(st)
    c = max(ceil(int((tiles * st).sum()), a.goal), 0)
    if c <= a.least:
        c = a.least
    else:
        for _ in range(3 if a.one_round else 0):
            n = int((tiles * ceil(st, c)).sum())
            if n <= a.goal:
                break
            c = max(ceil(c * n, a.goal), c + 1)
    return mine, tiles, ceil(st, c)


def check_attend(call, need, launches):
    taken = np.zeros(len(call.new), dtype=int)
    joins = []
    work = []
    for name, grid, block, arg in launches:
        a = AttendArgs.from_buffer_copy(bytes.fromhex(arg))
        # the arguments are read as the kernels read them
        assert (a.group, a.q_heads, a.b.n_tokens, a.c.heads) == (call.G, call.H * call.G, call.n, call.H), call.label
        assert grid[0] * block < 1 << 32 and grid[1] == 1 and 1 <= grid[2] <= 65535, call.label
        j = re.search(r"k_joinILi(\d+)ELi(\d+)ELi(\d+)E", name)
        r = re.search(r"k_rowsILi\d+ELi(\d+)ELi(\d+)ELb([01])ELi(\d+)E", name)
        k = re.search(r"k_chunkILi\d+ELi(\d+)ELi(\d+)E", name)
        assert grid[0] % call.H == 0, call.label
        if j:
            joins.append((int(j[2]), int(j[3]), grid[0] // call.H, a))
            continue
        rows, unit = (16 * int(r[2]), 32 * int(r[4])) if r else (32 * int(k[2]), 64)
        if r and r[3] == "1":
            tiles = call.n * ceil(call.G, rows)
            pieces = np.full(tiles, a.pieces)
            assert grid[0] // call.H >= tiles * a.pieces, (call.label, "list items")
            taken += call.new > 0
            work.append((rows, 0, tiles * a.pieces if a.pieces > 1 else 0, tiles if a.pieces > 1 else 0, a))
            continue
        mine, tiles, pieces = split(call, a, rows, unit)
        taken += mine
        items, some = int((tiles * pieces).sum()), pieces > 1
        assert grid[0] // call.H >= items, (call.label, name, "launched", grid[0] // call.H, "needed", items)
        slots, cut = int((tiles * pieces)[some].sum()), int(tiles[some].sum())
        assert slots <= a.slots, (call.label, "slots")
        work.append((rows, unit, slots, cut, a))
    # every sequence with new tokens by one kernel
    assert (taken == (call.new > 0)).all(), call.label
    areas = []
    for rows, unit, slots, cut, a in work:
        if unit and a.slots == 0:
            continue
        if not unit and slots == 0:
            continue
        size = (a.slots if unit else slots) * call.H * rows
        areas += [(a.part, size * call.D * 4), (a.stat, size * 8)]
        mine = [j for j in joins if j[0] == rows and (j[1] == unit or (unit == 32 * 4 and j[1] == 128)) and j[3].part == a.part]
        if cut:
            assert len(mine) == 1 and mine[0][2] >= cut, (call.label, "join", mine, cut)
    end = WS
    for p, size in sorted(areas):
        assert p >= end and p % 16 == 0, (call.label, "workspace areas overlap")
        end = p + size
    assert end <= WS + need, (call.label, "workspace", end - WS, need)


def check_select(call, need, launches):
    heads = call.H
    if "k_pick" in launches[0][0]:
        assert len(launches) == 1 and launches[0][1][0] >= call.n * heads, call.label
        return
    at = 0
    for i in range(0, len(launches), 2):
        (n1, g1, _, arg), (n2, g2, _, _) = launches[i:i + 2]
        tt = int(re.search(r"k_topILi(\d+)E", n2)[1])
        a = SelectArgs.from_buffer_copy(bytes.fromhex(arg))
        assert (a.group, a.c.heads, a.b.n_tokens, a.top_k) == (call.G, heads, call.n, 8), call.label
        assert "k_score" in n1 and a.slab0 == at and g1[0] >= a.slab * heads and g2[0] >= a.slab * tt * heads, call.label
        assert g1[1] * a.per >= a.nb and a.nb * (call.block or 1) >= call.room, call.label
        assert a.slab * tt * heads * a.nb * 8 <= need, call.label
        at += a.slab
    assert at >= int(ceil(call.new, tt).sum()), call.label


def check_append(call, launches):
    (name, grid, block, arg), = launches
    a = AppendArgs.from_buffer_copy(bytes.fromhex(arg))
    assert (a.c.heads, a.b.n_tokens, a.q_heads) == (call.H, call.n, call.H * call.G), call.label
    live = (call.new > 0) & (call.kv > 0)
    first = np.maximum(call.kv - call.new, 0)
    segs = np.where(live, ((call.kv - 1) >> a.log_seg) - (first >> a.log_seg) + 1, 0)
    assert grid[0] >= int(segs.sum()), call.label
    assert a.kv_groups << a.kv_log >= call.H and grid[1] >= 2 * a.kv_groups + ceil(call.H * call.G, 8), call.label


def run_attend(ask, calls):
    """calls: (Call, window, blocks)"""
    asked = [x for c, window, blocks in calls for x in c.attend(window, blocks)]
    got = ask(asked)
    for (c, window, blocks), (need, _), (st, launches) in zip(calls, got[::2], got[1::2]):
        c.window, c.n_blocks = window, blocks
        assert st == 0, c.label
        check_attend(c, need[0] if isinstance(need, list) else need, launches)


def lengths(rng, n, kind, top):
    if kind == "equal":
        return [top] * n
    if kind == "one long":
        return [top] + [rng.randint(1, max(1, top // 20)) for _ in range(n - 1)]
    if kind == "last long":
        return [rng.randint(1, max(1, top // 20)) for _ in range(n - 1)] + [top]
    return [max(1, int(top * 2.0 ** -rng.uniform(0, 5))) for _ in range(n)]


HEADS = [(1, 1), (1, 16), (2, 5), (4, 7), (8, 1), (8, 4), (8, 8), (12, 1), (16, 1), (32, 1), (32, 4)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [0, 1])
def test_single_tokens(ask, D, dtype):
    rng = random.Random(D + dtype)
    calls = []
    for H, G in HEADS:
        for n in (1, 2, 17, 64, 65, 96, 97, 128, 255, 300, 385, 512, 1000, 2000):
            for kind in ("equal", "one long", "last long", "ragged"):
                for top in (100, 2048, 16384, 131072):
                    calls.append((Call(H, G, D, [1] * n, lengths(rng, n, kind, top), dtype), 0, 0))
    run_attend(ask, calls)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prompts(ask, D):
    rng = random.Random(D)
    calls = []
    for H, G in HEADS:
        for n in (1, 300, 1023, 4096, 6145, 8192, 12290, 16384, 32768, 65536):
            calls.append((Call(H, G, D, [n], [n]), 0, 0))
            calls.append((Call(H, G, D, [n], [n + rng.randint(1, 40000)]), rng.choice((0, 128, 4096)), 0))
        for b, n, over in ((4, 4096, 8192), (8, 2048, 6000), (32, 512, 8192), (7, 2048, 32768), (100, 100, 2000), (500, 9, 5000)):
            calls.append((Call(H, G, D, [n] * b, [max(n, over)] * b), 0, 0))
            new = [rng.randint(0, n) for _ in range(b)]
            kv = [max(a, rng.randint(1, over)) for a in new]
            calls.append((Call(H, G, D, new, kv, max_q=n, room=max(kv) + rng.choice((0, 10000))), 0, 0))
    run_attend(ask, calls)


def test_mixed_batches(ask):
    """Single tokens, groups of a few and prompts in one call, with windows, roomy tables and no bound on the new tokens."""
    rng = random.Random(7)
    calls = []
    for _ in range(1500):
        H, G = rng.choice(HEADS)
        n = int(round(2 ** rng.uniform(0, 9.5)))
        top = int(2 ** rng.uniform(0, 13)) if n < 40 else rng.choice((1, 2, 5, 20, 100))
        new = [min(top, rng.choice((0, 1, 1, 1, 2, 7, top))) for _ in range(n)]
        if not any(new):
            new[0] = 1
        kv = [max(1, int(2 ** rng.uniform(0, 16))) for _ in range(n)]
        calls.append((Call(H, G, rng.choice((64, 128, 256)), new, kv, rng.choice((0, 1)), rng.choice((16, 64, 512)),
                           max_q=rng.choice((max(new), 0x7FFFFFFF)), room=rng.choice((max(kv), max(kv) + 50000))), rng.choice((0, 0, 100, 4096)), 0))
    run_attend(ask, calls)


def test_lists(ask):
    rng = random.Random(8)
    calls = []
    for H, G in HEADS:
        for n in (1, 3, 64, 500, 2000):
            for blocks in (1, 16, 64, 1024):
                calls.append((Call(H, G, rng.choice((64, 128, 256)), [1] * n, lengths(rng, n, "ragged", 65536), rng.choice((0, 1)), 64,
                                   rng.choice((16, 64))), 0, blocks))
    run_attend(ask, calls)


def test_select_and_append(ask):
    rng = random.Random(9)
    calls, asked = [], []
    for _ in range(400):
        H, G = rng.choice(HEADS)
        n = int(round(2 ** rng.uniform(0, 10)))
        top = rng.choice((1, 1, 3, 40, 3000 // n + 1))
        new = [rng.randint(0, top) for _ in range(n)]
        new[rng.randrange(n)] = top
        kv = [max(1, int(2 ** rng.uniform(0, 17))) for _ in range(n)]
        block = rng.choice((16, 64))
        c = Call(H, G, rng.choice((64, 128, 256)), new, kv, rng.choice((0, 1)), 64, block, max_q=rng.choice((top, 0x7FFFFFFF)))
        calls.append(c)
        asked += c.select() + c.append()
    got = ask(asked)
    for c, (need, _), (st, launches), (st2, appended) in zip(calls, got[::3], got[1::3], got[2::3]):
        assert st == 0 and st2 == 0, c.label
        check_select(c, need, launches)
        check_append(c, appended)
