"""Cases, inputs and plain forms of the operators of a beam search over the paged K/V cache: the choice of
the next beams from the logits, pages of the cache shared, given out, copied, taken back and moved together,
and the join of attention over parts of a context.

`run` computes a case in plain torch operations (`own` false) or calls the framework (`own` true).
"""
import math
import random

import torch

own = False

LLAMA_V = 128256                         # rows of the Llama-3-8B-shaped lm_head


def _case(name, op, **kw):
    c = dict(name=name, op=op)
    c.update({"select": dict(dtype="bf16", B=1, K=4, V=32000, M=8, pad=0, masked=False, ends=False, weighted=False, scale=1.0),
              "step": dict(dtype="bf16", B=1, K=4, prompt=1000, grown=100, T=16, H=8, D=128, C=0, layers=1, ragged=False, dead=False, q=1),
              "grow": dict(B=1, q=1, kv=1000, T=16, ragged=False, spare=100),
              "compact": dict(dtype="bf16", B=1, kv=1000, T=16, H=8, D=128, C=0, layers=1, ragged=False, spare=100),
              "merge": dict(B=1, HQ=32, D=128, parts=2, empty=False)}[op])
    c.update(kw)
    if name is None:
        del c["name"]
    return c


def listed():
    return [
        # one user's four beams, twice as many candidates as beams: the call after every answered token
        _case("select 1 x 4 of 32000", "select"),
        # a serving batch of beams over a large vocabulary, some beams finished, ranked by length
        _case("select 64 x 8 of 128256", "select", B=64, K=8, V=LLAMA_V, M=16, ends=True, weighted=True),
        # logits in 32 bits of an odd vocabulary, a grammar's mask over the tokens, a temperature
        _case("select 7 x 5 of 50001 masked", "select", dtype="fp32", B=7, K=5, V=50001, M=5, pad=3, masked=True, ends=True,
              scale=1.25),
        # four beams of one user go on from their parents by one token: page tables follow, shared pages
        # that would be written are copied, one layer's cache
        _case("step 1 x 4 over 1000", "step"),
        # a batch of beams in a 32-layer model's 8-bit cache of two heads a card, with block bounds
        _case("step 16 x 6 fp8 32 layers", "step", dtype="fp8", B=16, K=6, prompt=1500, grown=90, T=64, H=2, C=32, layers=32,
              ragged=True, dead=True),
        # many beams over long prompts in small pages: tables are what there is to move
        _case("step 64 x 8 over 32768", "step", B=64, K=8, prompt=32768, grown=300, H=1, D=64, ragged=True),
        # a batch that answers token by token, some of its guessed tokens taken back
        _case("grow 256 x 5", "grow", B=256, q=5, kv=8000, ragged=True, spare=1000),
        # prompts come in
        _case("grow 16 prompts of 20000", "grow", B=16, q=20000, kv=20000, ragged=True, spare=30000),
        # a small pool brought together
        _case("compact 8 of 1000", "compact", B=8, kv=1000, H=2, ragged=True, spare=200),
        # a pool of which half is free, brought together before its end is given to something else
        _case("compact 24 of 8000 bounds", "compact", B=24, kv=8000, T=64, C=64, ragged=True, spare=2000, layers=2),
        # one token's attention over the prompt's pages and over its beams' own
        _case("merge 8 x 2", "merge", B=8),
        # many new tokens over a context read in five parts, some of which a token does not see
        _case("merge 4096 x 5", "merge", B=4096, parts=5, empty=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("select", "select", "step", "grow", "compact", "merge"))
    if op == "select":
        c = dict(dtype=rng.choice(("bf16", "fp16", "fp32")), K=rng.choice((1, 2, 3, 4, 5, 8, 12, 16, 30)))
        c["M"] = min(64, rng.choice((c["K"], 2 * c["K"], 2 * c["K"] + 1)))
        c["V"] = _log(rng, 300, 160000)
        c["B"] = _log(rng, 1, max(1, min(256, (64 * 8 * LLAMA_V // (2 if c["dtype"] == "fp32" else 1)) // (c["K"] * c["V"]))))
        c["pad"] = rng.choice((0, 0, 1, 8, 37))
        c["masked"], c["ends"], c["weighted"] = rng.random() < 0.4, rng.random() < 0.5, rng.random() < 0.5
        c["scale"] = rng.choice((1.0, 1.0, 0.7, 1.6))
    elif op == "step":
        c = dict(dtype=rng.choice(("bf16", "fp8")), K=rng.choice((2, 3, 4, 5, 8, 13)), T=rng.choice((16, 32, 64, 128)),
                 H=rng.choice((1, 2, 4, 8)), D=rng.choice((64, 128, 256)))
        c["C"] = rng.choice((0, 16, min(c["T"], 64)))
        c["layers"] = rng.choice((1, 2, 5, 16))
        c["ragged"], c["dead"], c["q"] = rng.random() < 0.7, rng.random() < 0.3, rng.choice((1, 1, 1, 2, 20))
        c["grown"] = _log(rng, 1, 400)
        token = 2 * c["layers"] * c["H"] * c["D"] * (1 if c["dtype"] == "fp8" else 2)    # bytes of a token
        most = int(1.0e9 / token)
        c["B"] = _log(rng, 1, max(1, min(64, most // (4 * c["K"] * (c["grown"] + c["q"] + c["T"])))))
        c["prompt"] = _log(rng, 1, max(2, min(32768, most // (2 * c["B"]))))
    elif op == "grow":
        c = dict(B=_log(rng, 1, 400), T=rng.choice((16, 32, 64, 256)), ragged=rng.random() < 0.8, spare=_log(rng, 1, 20000))
        c["kv"] = _log(rng, 2, max(3, min(60000, 2000000 // c["B"])))
        c["q"] = _log(rng, 1, c["kv"])
    elif op == "compact":
        c = dict(dtype=rng.choice(("bf16", "fp8")), T=rng.choice((16, 32, 64, 128)), H=rng.choice((1, 2, 4, 8)),
                 D=rng.choice((64, 128, 256)), ragged=rng.random() < 0.8, layers=rng.choice((1, 2, 4)))
        c["C"] = rng.choice((0, 16, min(c["T"], 64)))
        page = 2 * c["layers"] * c["H"] * c["D"] * c["T"] * (1 if c["dtype"] == "fp8" else 2)
        most = int(1.2e9 / page)
        c["B"] = _log(rng, 1, max(1, min(100, most // 8)))
        c["kv"] = _log(rng, 1, max(2, min(40000, most // (2 * c["B"]) * c["T"])))
        c["spare"] = _log(rng, 1, max(2, most // 2))
    else:
        c = dict(HQ=rng.choice((1, 7, 8, 32, 40)), D=rng.choice((64, 128, 256)), parts=rng.randint(2, 8), empty=rng.random() < 0.5)
        c["B"] = _log(rng, 1, int(8.0e7 / (c["HQ"] * c["D"] * c["parts"])))
    return _case(None, op, **c)


# ------------------------------------------------------------------ sizes of a case

def _random_of(c):
    return random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))


def _beams(c):
    """Prompt tokens, tokens in all and parents of each group's beams: from the case alone."""
    r = _random_of(c)
    B, K = c["B"], c["K"]
    some = lambda x: x if not c["ragged"] else max(1, int(x * 2.0 ** -r.uniform(0, 3)))   # noqa: E731
    prompt = [c["prompt"]] + [some(c["prompt"]) for _ in range(B - 1)]
    total = [p + g for p, g in zip(prompt, [c["grown"]] + [some(c["grown"]) for _ in range(B - 1)])]
    parents = [[r.randrange(K) for _ in range(K)] for _ in range(B)]
    if c["dead"]:
        for p in parents:
            if r.random() < 0.5:
                p[r.randrange(K)] = -1
    return prompt, total, parents


def _lengths(c):
    """New tokens and tokens in all of each sequence: from the case alone."""
    r = _random_of(c)
    kv = [c["kv"]] + [c["kv"] if not c["ragged"] else max(1, int(c["kv"] * 2.0 ** -r.uniform(0, 4))) for _ in range(c["B"] - 1)]
    q = c.get("q", 0)
    return [min(y, q if not c["ragged"] else r.randint(0, q)) for y in kv], kv


def _beam_pages(c):
    """The table of a step's beams before it, in page numbers from 0 up, and how many there are: a prompt's whole
    pages are all its beams', later ones of fewer beams the newer they are, the newest each beam's own."""
    prompt, total, _ = _beams(c)
    K, T = c["K"], c["T"]
    table = torch.full((c["B"] * K, max(-(-(x + c["q"]) // T) for x in total) + 1), -1, dtype=torch.int64)
    n, b = 0, torch.arange(K)
    for g, (p, x) in enumerate(zip(prompt, total)):
        rows = table[g * K:(g + 1) * K]
        rows[:, :p // T] = n + torch.arange(p // T)
        n += p // T
        last = -(-x // T) - 1
        for j in range(p // T, last + 1):
            of = b >> min(last - j, 30)
            rows[:, j] = n + of
            n += int(of[-1]) + 1
    return table, n


def _seq_pages(c):
    """The same for sequences with pages of their own."""
    per = [-(-x // c["T"]) for x in _lengths(c)[1]]
    table = torch.full((c["B"], max(per) + 1), -1, dtype=torch.int64)
    n = 0
    for b, m in enumerate(per):
        table[b, :m] = n + torch.arange(m)
        n += m
    return table, n


def _width(c):
    return 1 if c["dtype"] == "fp8" else 2


def _moved_bytes(c, tokens, blocks):
    """Bytes that copying so many tokens, and blocks with bounds, reads and writes in all layers."""
    row = c["H"] * c["D"] * c["layers"]
    return 2 * (tokens * 2 * row * _width(c) + (blocks * row * 4 if c["C"] else 0))


def work(case):
    c = case
    if c["op"] == "select":
        rows, out = c["B"] * c["K"], c["B"] * c["M"]
        e = 4 if c["dtype"] == "fp32" else 2
        b = rows * c["V"] * e + rows * 4 + out * 13
        if c["masked"]:
            b += rows * -(-c["V"] // 32) * 4
        return {"bytes": b + rows * 5, "flops": rows * c["V"] * 4}
    if c["op"] == "merge":
        n = c["B"] * c["HQ"]
        return {"bytes": (c["parts"] + 1) * n * (c["D"] * 2 + 4), "flops": n * c["parts"] * (2 * c["D"] + 4)}
    if c["op"] == "step":
        _, total, parents = _beams(c)
        T, C, K = c["T"], c["C"], c["K"]
        entries = tokens = blocks = 0
        for x, p in zip(total, parents):
            live = [y for y in p if y >= 0]
            entries += (K + len(live)) * -(-x // T)
            if x % T:                    # of the beams that go on from one parent, one keeps the newest page
                copies = len(live) - len(set(live))
                tokens += copies * (x % T)
                blocks += copies * (-(-(x % T) // C) if C else 0)
        n = _beam_pages(c)[1] + _spare(c)
        return {"bytes": entries * 4 + n * 8 + c["B"] * K * 20 + _moved_bytes(c, tokens, blocks), "flops": entries + n}
    _, kv = _lengths(c)
    per = [-(-x // c["T"]) for x in kv]
    n = sum(per) + c["spare"]
    if c["op"] == "grow":
        new = [-(-y // c["T"]) - -(-(y - x) // c["T"]) for x, y in zip(*_lengths(c))]
        return {"bytes": n * 4 + sum(new) * 16 + c["B"] * 24, "flops": n + 2 * sum(new)}
    # pages in use are anywhere: as many of them lie behind as there are holes in front
    moves = sum(per) * c["spare"] / n
    return {"bytes": n * 12 + sum(per) * 8 + _moved_bytes(c, moves * c["T"], moves * (c["T"] // C if (C := c["C"]) else 0)), "flops": 2 * n}


# ------------------------------------------------------------------ inputs

def _spare(c):
    """Free pages before a step: some more than it can take."""
    return c["B"] * c["K"] * (2 + c["q"] // c["T"]) + 9


def _rows(gen, *shape):
    """Keys or values: a normal spread, and four channels of each head far larger than the rest, as caches have."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    x[..., 1::max(1, shape[-1] // 4)] *= 6.0
    return x


def _pages(c, g, n):
    """Keys, values and bounds of all layers' caches of n pages: layers first."""
    L, H, T, D = c["layers"], c["H"], c["T"], c["D"]
    dt = torch.float8_e4m3fn if c["dtype"] == "fp8" else torch.bfloat16

    def filled(dtype, *shape):
        x = torch.empty((L * n, *shape), dtype=dtype, device="cuda")
        step = max(1, (1 << 27) // math.prod(shape))
        for i in range(0, L * n, step):
            x[i:i + step] = _rows(g, min(step, L * n - i), *shape).to(dtype)
        return x.view(L, n, *shape)

    return filled(dt, H, T, D), filled(dt, H, T, D), filled(torch.bfloat16, H, T // c["C"], 2, D) if c["C"] else None


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = {"case": dict(c)}
    i32 = dict(dtype=torch.int32, device=dev)
    if c["op"] == "select":
        B, K, V, M = c["B"], c["K"], c["V"], c["M"]
        dt = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[c["dtype"]]
        x = torch.empty((B, K, V + c["pad"]), dtype=dt, device=dev)
        for b in range(0, B, 16):        # a broad spread, and a few tokens that the model thinks likely
            y = torch.randn((min(16, B - b), K, V + c["pad"]), generator=g, device=dev) * 2.5
            likely = torch.randint(0, V, (y.shape[0], K, 12), generator=g, device=dev)
            y.scatter_add_(2, likely, 6.0 + 4.0 * torch.rand(likely.shape, generator=g, device=dev))
            x[b:b + 16] = y.to(dt)
        x[:, :, V:] = math.nan
        s["logits"] = x[:, :, :V]
        s["scores"] = -20.0 * torch.rand((B, K), generator=g, device=dev)
        s["weights"] = s["finished"] = s["allowed"] = None
        s["end"] = 2 if c["ends"] else None
        if c["weighted"]:                # one over a power of the beams' lengths
            s["weights"] = torch.randint(5, 60, (B, K), generator=g, device=dev).float() ** -0.7
        if c["ends"]:
            s["finished"] = torch.rand((B, K), generator=g, device=dev) < 0.15
        if c["masked"]:
            share = torch.rand((B, K, 1), generator=g, device=dev)
            words = torch.zeros((B, K, -(-V // 32)), **i32)
            for i in range(32):
                words |= (torch.rand(words.shape, generator=g, device=dev) < share).to(torch.int32) << i
            if K > 1:
                words[0, K - 1] = 0      # a beam that its grammar leaves no way on
            s["allowed"] = words
        return s
    if c["op"] == "merge":
        shape = (c["parts"], c["B"], c["HQ"])
        s["outs"] = torch.randn((*shape, c["D"]), generator=g, device=dev).to(torch.bfloat16)
        s["lses"] = 6.0 + 2.0 * torch.randn(shape, generator=g, device=dev)
        if c["empty"]:
            s["lses"][torch.rand(shape, generator=g, device=dev) < 0.2] = -math.inf
        s["outs"], s["lses"] = list(s["outs"].unbind(0)), list(s["lses"].unbind(0))
        return s
    if c["op"] == "step":
        (table, used), spare, n_seqs = _beam_pages(c), _spare(c), c["B"] * c["K"]
        _, total, parents = _beams(c)
        held = [x for x in total for _ in range(c["K"])]
        q = [c["q"]] * n_seqs
        cap = n_seqs
    else:
        (table, used), spare, n_seqs = _seq_pages(c), c["spare"], c["B"]
        q, held = _lengths(c)
        cap = (used + spare) // 2 if c["op"] == "compact" else n_seqs
    n = used + spare
    perm = torch.randperm(n, generator=g, device=dev).to(torch.int32)
    table = table.to(dev)
    table = torch.where(table >= 0, perm[table.clamp(min=0)], -1).to(torch.int32)
    # what a scheduler keeps of its pages, in one buffer: passes begin with it as it was
    sizes = [("refs", (n,)), ("table", tuple(table.shape)), ("held", (n_seqs,)), ("kv_len", (n_seqs,)),
             ("pairs", (max(cap, 1), 3)), ("count", (1,)), ("remap", (n,))]
    s["ints"] = torch.full((sum(math.prod(x) for _, x in sizes),), -1, **i32)
    at = 0
    for name, x in sizes:
        s[name] = s["ints"][at:at + math.prod(x)].view(x)
        at += math.prod(x)
    s["refs"].copy_(torch.bincount(table[table >= 0].long(), minlength=n))
    s["table"].copy_(table)
    s["held"].copy_(torch.tensor(held, **i32))
    s["kept"] = s["ints"].clone()
    s["q_start"] = torch.tensor([0] + [sum(q[:i + 1]) for i in range(n_seqs)], **i32)
    if c["op"] == "step":
        s["parents"] = torch.tensor(parents, **i32)
    if c["op"] == "grow":
        s["keep"] = torch.tensor([y - x for x, y in zip(q, held)], **i32)
    if c["op"] != "grow":
        s["k"], s["v"], s["bounds"] = _pages(c, g, n)
    if own:
        import lossless_float_compression_amd as zx
        s["pool"] = zx.PagePool(n, c["T"], refs=s["refs"])
        s["copies"] = zx.PageCopies(max(cap, 1), pairs=s["pairs"], count=s["count"])
        s["batch"] = zx.PagedBatch(s["q_start"], s["kv_len"], s["table"], max_q=max(q), max_kv=max(held) + max(q))
        if c["op"] != "grow":
            dt = zx.FP8_E4M3FN if c["dtype"] == "fp8" else zx.BF16
            s["caches"] = zx.PagedLayers([
                zx.PagedKVCache(n, c["H"], c["D"], c["T"], dt, block_tokens=c["C"] or None, k=s["k"][i], v=s["v"][i],
                                bounds=s["bounds"][i] if c["C"] else None) for i in range(c["layers"])])
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    c = s["case"]
    if own:
        if c["op"] == "select":
            import lossless_float_compression_amd as zx
            r = zx.beam_select(s["logits"], s["scores"], c["M"], weights=s["weights"], finished=s["finished"], end=s["end"],
                               allowed=s["allowed"], scale=c["scale"])
            return {"scores": r.scores, "parents": r.parents, "tokens": r.tokens, "finished": r.finished}
        if c["op"] == "merge":
            import lossless_float_compression_amd as zx
            lse = torch.empty_like(s["lses"][0])
            return {"out": zx.merge_attention(s["outs"], s["lses"], lse=lse), "lse": lse}
    if c["op"] == "select":
        return _plain_select(s)
    if c["op"] == "merge":
        return _plain_merge(s)
    s["ints"].copy_(s["kept"])
    if c["op"] == "step":
        if own:
            s["pool"].fork(s["table"], s["held"], s["parents"])
            s["pool"].extend(s["batch"], s["held"], copies=s["copies"])
            s["caches"].copy_pages(s["copies"])
        else:
            _plain_fork(s)
            _plain_extend(s)
            _plain_copy(s)
    elif c["op"] == "grow":
        if own:
            s["pool"].trim(s["table"], s["held"], s["keep"])
            s["pool"].extend(s["batch"], s["held"], copies=s["copies"])
        else:
            _plain_trim(s)
            _plain_extend(s)
    else:
        if own:
            s["pool"].compact(s["table"], s["held"], copies=s["copies"], remap=s["remap"])
            s["caches"].copy_pages(s["copies"])
        else:
            _plain_compact(s)
            _plain_copy(s)
    out = {k: s[k] for k in ("refs", "table", "held", "pairs", "count")}
    out["kv_len" if c["op"] != "compact" else "remap"] = s["kv_len" if c["op"] != "compact" else "remap"]
    if c["op"] != "grow":
        out.update(k=s["k"], v=s["v"], bounds=s["bounds"])
    return out


def _plain_select(s):
    c = s["case"]
    B, K, V, M = c["B"], c["K"], c["V"], c["M"]
    # in 64 bits: which candidates are taken, and in which order, must not turn on rounding
    x = s["logits"].double()
    if c["scale"] != 1.0:
        x *= c["scale"]
    if s["allowed"] is not None:
        t = torch.arange(V, device="cuda")
        bit = (s["allowed"][:, :, t >> 5] >> (t & 31).to(torch.int32)) & 1
        x.masked_fill_(bit == 0, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x -= m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))
    score = s["scores"].double()
    x = torch.where(torch.isnan(x), -math.inf, x) + score[:, :, None]
    if s["finished"] is not None:        # a finished beam goes on with its end token, at no cost
        stay = torch.full_like(x, -math.inf)
        stay[:, :, s["end"]] = score
        x = torch.where(s["finished"][:, :, None], stay, x)
        del stay
    rank = (x if s["weights"] is None else x * s["weights"].double()[:, :, None]).view(B, K * V)
    at = torch.sort(rank, dim=-1, descending=True, stable=True)[1][:, :M]
    total = torch.gather(x.view(B, K * V), 1, at)
    some = total > -math.inf
    parents = torch.where(some, torch.div(at, V, rounding_mode="floor"), -1).to(torch.int32)
    tokens = torch.where(some, at % V, -1).to(torch.int32)
    ended = torch.zeros_like(some) if s["end"] is None else some & (tokens == s["end"])
    if s["finished"] is not None:
        ended |= some & torch.gather(s["finished"], 1, parents.clamp(min=0).long())
    return {"scores": total.float(), "parents": parents, "tokens": tokens, "finished": ended}


def _plain_merge(s):
    x, l = torch.stack(s["outs"]).float(), torch.stack(s["lses"])
    m = l.amax(0)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    w = torch.exp(l - m)
    t = w.sum(0)
    o = (x * (w / torch.where(t > 0, t, torch.ones_like(t)))[..., None]).sum(0)
    return {"out": o.to(torch.bfloat16), "lse": m + torch.log(t)}


def _ceil(a, b):
    return torch.div(a + (b - 1), b, rounding_mode="floor")


def _plain_fork(s):
    c = s["case"]
    B, K, T = c["B"], c["K"], c["T"]
    table, held, refs, par = s["table"], s["held"], s["refs"], s["parents"].view(-1).long()
    first = torch.arange(B * K, device="cuda") // K * K
    goes = par >= 0
    of = first + par.clamp(min=0)
    children = torch.zeros_like(held).index_add_(0, of, goes.to(torch.int32))
    j = torch.arange(table.shape[1], device="cuda")
    n = _ceil(held, T)
    used = j < n[:, None]
    # pages that are not used add nothing to page 0
    refs.index_add_(0, torch.where(used, table, 0).view(-1).long(), torch.where(used, (children - 1)[:, None], 0).to(torch.int32).view(-1))
    held.copy_(torch.where(goes, held[of], 0))
    table.copy_(torch.where(j < _ceil(held, T)[:, None], table[of], table))


def _plain_trim(s):
    T, table, held = s["case"]["T"], s["table"], s["held"]
    j = torch.arange(table.shape[1], device="cuda")
    gone = (j < _ceil(held, T)[:, None]) & (j >= _ceil(s["keep"], T)[:, None])
    s["refs"].index_add_(0, torch.where(gone, table, 0).view(-1).long(), -gone.to(torch.int32).view(-1))
    held.copy_(torch.minimum(held, s["keep"]))


def _plain_extend(s):
    T = s["case"]["T"]
    table, held, refs = s["table"], s["held"], s["refs"]
    n_seqs, W = table.shape
    n = refs.numel()
    q = s["q_start"][1:] - s["q_start"][:-1]
    row = torch.arange(n_seqs, device="cuda")
    # sequences that go on in a page that has tokens: how many write each page, and the first that does
    last = torch.div(held, T, rounding_mode="floor").long().clamp(max=W - 1)
    into = (q > 0) & (held % T > 0)
    page = torch.where(into, table[row, last].long(), n)
    writers = torch.zeros(n + 1, dtype=torch.int32, device="cuda").index_add_(0, page, into.to(torch.int32))
    first = torch.full((n + 1,), n_seqs, dtype=torch.int64, device="cuda").scatter_reduce_(0, page, row, "amin")
    holders = torch.nn.functional.pad(refs, (0, 1))
    keeps = (writers[page] >= holders[page]) & (first[page] == row)
    copied = into & ~keeps
    lo = torch.where(copied, last, _ceil(held, T).long())
    hi = _ceil(held + q, T).long()
    need = torch.where(q > 0, hi - lo, 0)
    before = torch.cumsum(need, 0) - need
    free = torch.cumsum((refs <= 0).to(torch.int64), 0)
    enough = free[-1] >= need.sum()
    copied &= enough
    j = torch.arange(W, device="cuda")
    fresh = (j >= lo[:, None]) & (j < hi[:, None]) & (q > 0)[:, None] & enough
    ids = torch.searchsorted(free, torch.where(fresh, before[:, None] + j - lo[:, None] + 1, 1).view(-1)).view(n_seqs, W)
    old = torch.where(copied, page, n)
    where = torch.cumsum(copied.to(torch.int64), 0) - 1
    pairs = torch.cat((s["pairs"], s["pairs"][:1]))
    pairs[torch.where(copied, where, pairs.shape[0] - 1)] = torch.stack((old, ids[row, last], held.long() % T), 1).to(torch.int32)
    s["pairs"].copy_(pairs[:-1])
    s["count"].copy_(copied.sum().to(torch.int32).view(1))
    out = torch.nn.functional.pad(refs, (0, 1))
    out.index_add_(0, old, -copied.to(torch.int32))
    out[torch.where(fresh, ids, n).view(-1)] = 1
    refs.copy_(out[:-1])
    table.copy_(torch.where(fresh, ids.to(torch.int32), table))
    s["kv_len"].copy_(torch.where(enough, held + q, 0))
    held.copy_(torch.where(enough, held + q, held))


def _plain_compact(s):
    T, table, held, refs = s["case"]["T"], s["table"], s["held"], s["refs"]
    n = refs.numel()
    i = torch.arange(n, device="cuda")
    live = refs > 0
    total = live.sum()
    holes = torch.cumsum((~live).to(torch.int64), 0)              # free pages up to and with each
    late = live & (i >= total)
    nth = torch.cumsum(late.to(torch.int64), 0) - 1
    to = torch.where(late, torch.searchsorted(holes, nth.clamp(min=0) + 1), i)
    s["remap"].copy_(torch.where(live, to, -1))
    cap = s["pairs"].shape[0]
    pairs = torch.cat((s["pairs"], s["pairs"][:1]))
    pairs[torch.where(late, nth, cap)] = torch.stack((i, to, torch.full_like(i, T)), 1).to(torch.int32)
    s["pairs"].copy_(pairs[:-1])
    s["count"].copy_(late.sum().to(torch.int32).view(1))
    out = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    out[torch.where(live, to, n)] = refs
    refs.copy_(out[:-1])
    used = torch.arange(table.shape[1], device="cuda") < _ceil(held, T)[:, None]
    table.copy_(torch.where(used, s["remap"][torch.where(used, table, 0).long()], table))


def _plain_copy(s):
    """The first tokens of each pair's source page over those of its destination; pairs behind the count copy a page's tokens
    to where they are."""
    c = s["case"]
    T, C = c["T"], c["C"]
    there = torch.arange(s["pairs"].shape[0], device="cuda") < s["count"]
    # pages are written once: all pairs behind the count do what the first one does, or copy page 0 over itself
    first = torch.where(s["count"] > 0, s["pairs"][0], 0)
    src, dst, n = torch.where(there[:, None], s["pairs"], first).long().unbind(1)
    raw = torch.uint8 if c["dtype"] == "fp8" else torch.int16
    for x, unit in ((s["k"].view(raw), 1), (s["v"].view(raw), 1), (s["bounds"], C)):
        if x is None:
            continue
        i = torch.arange(x.shape[3], device="cuda")
        few = max(1, (1 << 28) // x[:, 0].numel())                # pages at a time
        for a in range(0, src.numel(), few):
            take = (i < _ceil(n[a:a + few], unit)[:, None]).view(-1, 1, x.shape[3], *[1] * (x.dim() - 4))
            x[:, dst[a:a + few]] = torch.where(take, x[:, src[a:a + few]], x[:, dst[a:a + few]])


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "select":
        B, K, V, M = c["B"], c["K"], c["V"], c["M"]
        out = {"scores": torch.full((B, M), -math.inf, dtype=torch.float64), "parents": None, "tokens": None, "finished": None}
        for b in range(B):
            rows, by = [], []
            for k in range(K):
                x = s["logits"][b, k].double() * c["scale"]
                if s["allowed"] is not None:
                    bits = (s["allowed"][b, k].long()[:, None] >> torch.arange(32, device="cuda")) & 1
                    x[bits.view(-1)[:V] == 0] = -math.inf
                lp = x - torch.logsumexp(x, 0) if bool((x > -math.inf).any()) else x
                if s["finished"] is not None and bool(s["finished"][b, k]):
                    lp = torch.full_like(x, -math.inf)
                    lp[s["end"]] = 0.0
                lp = lp + s["scores"][b, k].double()
                rows.append(lp)
                by.append(lp if s["weights"] is None else lp * s["weights"][b, k].double())
            rows, by = torch.cat(rows), torch.cat(by)
            edge = torch.topk(by, min(M, K * V))[0][-1]
            some = torch.nonzero((by >= edge) & (by > -math.inf)).view(-1)
            best = sorted(zip((-by[some]).tolist(), some.tolist()))[:M]
            for i, (_, at) in enumerate(best):
                out["scores"][b, i] = rows[at]
        return out
    if c["op"] == "merge":
        l = torch.stack(s["lses"]).double()
        lse = torch.logsumexp(l, 0)
        w = torch.nan_to_num(torch.exp(l - lse), nan=0.0)
        return {"out": sum(x.double() * y[..., None] for x, y in zip(s["outs"], w)), "lse": lse}
    if c["op"] == "grow":
        return None                      # whole numbers only
    # which page is copied where is found on the host, page by page
    T, C = c["T"], c["C"]
    refs, table, held = s["refs"].tolist(), s["table"].tolist(), s["held"].tolist()
    moves = []
    if c["op"] == "step":
        K = c["K"]
        parents = s["parents"].tolist()
        rows = []
        for r in range(len(held)):
            p = parents[r // K][r % K]
            rows.append((table[r // K * K + p], held[r // K * K + p]) if p >= 0 else ([], 0))
        holders = {}
        for t, x in rows:
            for p in t[:-(-x // T)]:
                holders[p] = holders.get(p, 0) + 1
        free = iter([p for p in range(len(refs)) if p not in holders])
        kept = set()
        for t, x in rows:
            new = -(-(x + c["q"]) // T) - -(-x // T)
            if x % T:
                page = t[x // T]
                if holders[page] > 1 and page in kept:
                    moves.append((page, next(free), x % T))
                kept.add(page)
            for _ in range(new):
                next(free)
    else:
        used = [p for p, x in enumerate(refs) if x > 0]
        holes = [p for p in range(len(used)) if refs[p] <= 0]
        moves = [(p, h, T) for p, h in zip([p for p in used if p >= len(used)], holes)]
    out = {}
    for name, unit in (("k", 1), ("v", 1), ("bounds", C)):
        x = s.pop(name)
        out[name] = x
        if x is not None:
            y = out[name] = x.double()
            for a, b, m in moves:
                y[:, b, :, :-(-m // unit)] = y[:, a, :, :-(-m // unit)]
    return out
