"""Cases, inputs and plain forms of the paged K/V cache operators: appending new keys and values
with the position rotation on the way, attention of new tokens over the cache, and attention over
the blocks of the cache that a cheap score selects.

`run` computes a case in plain torch operations (`own` false) or calls the framework (`own` true).
"""
import math
import random

import torch

own = False

LLAMA_H, LLAMA_G, LLAMA_D = 8, 4, 128   # 8 K/V heads of 128 channels, 32 query heads


def _case(name, op, **kw):
    c = dict(name=name, op=op, dtype="bf16", B=1, q=1, kv=1024, ragged=False, H=LLAMA_H, G=LLAMA_G, D=LLAMA_D,
             T=64, C=0, pad=0, rotary=0, interleaved=False, scaling="none", causal=True, window=0, top_k=0,
             keep_first=1, keep_last=1)
    c.update(kw)
    if name is None:
        del c["name"]
    return c


def listed():
    return [
        # one token of one conversation: the call that every layer makes for every answered token
        _case("append 1 token", "append", B=1, q=1, kv=1000, T=16, rotary=128),
        # a full serving batch, one token each, 8-bit cache with the block bounds kept up, a model
        # stretched to long contexts
        _case("append 256 x 1 fp8 bounds", "append", dtype="fp8", B=256, q=1, kv=32768, ragged=True, T=64, C=64,
              rotary=128, scaling="bands"),
        # prompts of several users packed into one call; half of each head is rotated, pairs interleaved;
        # pages of 512 tokens, the size whose heads are single 65536-element codec blocks
        _case("append 5 ragged prompts", "append", B=5, q=2900, kv=12000, ragged=True, T=512, C=64, rotary=64,
              interleaved=True, pad=3),
        # one conversation, one token: latency
        _case("attend 1 x 1 over 1000", "attend", B=1, q=1, kv=1000, T=16),
        # a serving batch of single tokens over contexts of very different lengths, small pages
        _case("attend 64 x 1 ragged", "attend", B=64, q=1, kv=16384, ragged=True, T=16),
        # four long contexts in an 8-bit cache, pages of 512
        _case("attend 4 x 1 over 131072 fp8", "attend", dtype="fp8", B=4, q=1, kv=131072, T=512),
        # a few guessed tokens checked at once, sliding window, small heads, 8-bit cache
        _case("attend 16 x 5 window fp8", "attend", dtype="fp8", B=16, q=5, kv=9001, H=4, G=8, D=64, T=32, window=4096),
        # a whole prompt at once
        _case("attend 4096 new", "attend", B=1, q=4096, kv=4096, T=64),
        # a further piece of a long prompt (32768 tokens) beside a shorter one
        _case("attend 2 x 777 over 32768", "attend", B=2, q=777, kv=32768, ragged=True, T=512, pad=2),
        # one conversation of 32768 tokens, one token: sixteen blocks of 64 are read
        _case("sparse 1 x 1 over 32768", "sparse", B=1, q=1, kv=32768, T=512, C=64, top_k=16),
        # a batch of long contexts, one token each
        _case("sparse 32 x 1 over 65536", "sparse", B=32, q=1, kv=65536, T=64, C=64, top_k=48, ragged=True),
        # a short chunk of new tokens, each with blocks of its own, 8-bit cache
        _case("sparse 3 x 41 fp8", "sparse", dtype="fp8", B=3, q=41, kv=17000, T=128, C=32, top_k=40, G=8, H=2, pad=1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "sparse"))
    dtype = rng.choice(("bf16", "fp8"))
    H, G, D = rng.choice(((8, 4, 128), (8, 8, 128), (4, 7, 64), (1, 16, 128), (12, 1, 64), (2, 5, 128), (2, 4, 256)))
    T = rng.choice((16, 32, 64, 128, 256, 512))
    ragged = rng.random() < 0.7
    c = dict(dtype=dtype, H=H, G=G, D=D, T=T, ragged=ragged, pad=rng.choice((0, 0, 1, 5)))
    if op == "append":
        c["B"] = _log(rng, 1, 200)
        c["q"] = _log(rng, 1, max(1, 4000 // c["B"]))
        c["kv"] = c["q"] + _log(rng, 1, max(1, 400000 // c["B"]))
        c["C"] = rng.choice((0, 16, min(T, 64)))
        c["rotary"] = rng.choice((D, D // 2, 32, 0))
        c["interleaved"] = rng.random() < 0.5
        c["scaling"] = rng.choice(("none", "linear", "bands"))
    elif op == "attend":
        if rng.random() < 0.5:   # single tokens and small groups of them
            c["B"] = _log(rng, 1, 128)
            c["q"] = rng.choice((1, 1, 1, 2, 4, 7))
            c["kv"] = c["q"] + _log(rng, 1, max(1, 600000 // c["B"] // max(1, H * D // 1024)))
        else:
            c["B"] = rng.randint(1, 6)
            c["q"] = _log(rng, 16, max(17, 4096 // c["B"]))
            most = int(1.5e8 / (H * G * D / 4096) / (c["B"] * c["q"]))
            c["kv"] = c["q"] + _log(rng, 1, max(2, min(most, 40000)))
        c["window"] = rng.choice((0, 0, 0, 128, 1000, 4096))
        c["causal"] = rng.random() < 0.85
    else:
        c["C"] = rng.choice((16, 32, min(T, 64)))
        c["C"] = min(c["C"], T)
        c["B"] = _log(rng, 1, 32)
        c["q"] = rng.choice((1, 1, 1, 2, rng.randint(3, 40)))
        c["q"] = max(1, min(c["q"], 120 // c["B"]))
        c["kv"] = c["q"] + _log(rng, 300, max(301, min(80000, 800000 // c["B"])))
        c["top_k"] = rng.randint(2, 64)
        c["keep_first"], c["keep_last"] = rng.choice(((1, 1), (0, 1), (0, 0), (1, 2) if c["top_k"] > 2 else (1, 1)))
    return _case(None, op, **c)


# ------------------------------------------------------------------ sizes of a case

def _lengths(c):
    """New tokens and total tokens of each sequence: from the case alone."""
    r = random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))
    B, q, kv = c["B"], c["q"], c["kv"]
    if not c["ragged"]:
        return [q] * B, [max(q, kv)] * B
    ql = [q] + [r.randint(max(1, q // 4), q) for _ in range(B - 1)]
    kl = [kv] + [max(1, int(kv * 2.0 ** -r.uniform(0, 4))) for _ in range(B - 1)]
    pairs = [(a, max(a, b)) for a, b in zip(ql, kl)]
    r.shuffle(pairs)
    return [a for a, _ in pairs], [b for _, b in pairs]


def _visible(c):
    """For each sequence, (sum over its new tokens of the tokens each sees, tokens any of them sees)."""
    out = []
    for a, b in zip(*_lengths(c)):
        w = c["window"] if c["window"] else 1 << 60
        s = 0
        for i in range(a):
            p = b - a + i
            hi = p + 1 if c["causal"] else b
            s += hi - max(0, p - w + 1)
        first = max(0, b - a - w + 1)
        out.append((s, b - first))
    return out


def work(case):
    c = case
    ql, kl = _lengths(c)
    N, HQ, e = sum(ql), c["H"] * c["G"], 1 if c["dtype"] == "fp8" else 2
    row = c["H"] * c["D"]
    if c["op"] == "append":
        b = N * (2 * row * 2 + 2 * row * e + 2 * HQ * c["D"] * 2)
        if c["C"]:
            blocks = sum((y - 1) // c["C"] - (y - x) // c["C"] + 1 for x, y in zip(ql, kl))
            b += blocks * row * 2 * 2
        return {"bytes": b, "flops": N * (c["H"] + HQ) * c["rotary"] * 3}
    io = N * HQ * c["D"] * 4 + N * HQ * 4
    if c["op"] == "attend":
        v = _visible(c)
        return {"bytes": io + sum(y for _, y in v) * 2 * row * e, "flops": sum(x for x, _ in v) * 4 * HQ * c["D"]}
    blocks = taken = tokens = 0
    for x, y in zip(ql, kl):
        n = (y - 1) // c["C"] + 1
        blocks += n
        for i in range(x):
            m = min((y - x + i) // c["C"] + 1, c["top_k"])
            taken += m
            tokens += m * c["C"]
    # the blocks of one token at least are read; tokens of one sequence may share theirs
    distinct = sum(min(x * c["top_k"] * c["C"], y) for x, y in zip(ql, kl))
    return {"bytes": io + N * c["H"] * c["top_k"] * 4 + blocks * row * 4 + distinct * 2 * row * e,
            "flops": tokens * 4 * HQ * c["D"] + sum(x * ((y - 1) // c["C"] + 1) for x, y in zip(ql, kl)) * 4 * row}


# ------------------------------------------------------------------ inputs

def _inv_freq(c, device):
    """Angle per position of each rotated pair, in 64 bits; "linear": positions eight times denser;
    "bands": wavelengths beyond 8192 positions eight times slower, those below 2048 unchanged, a
    straight blend between."""
    r = c["rotary"]
    f = 500000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device=device) / r)
    if c["scaling"] == "linear":
        f = f / 8.0
    elif c["scaling"] == "bands":
        wave = 2 * math.pi / f
        s = ((8192.0 / wave - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        f = (1 - s) * f / 8.0 + s * f
    return f


def _rows(gen, *shape):
    """Keys or values: a normal spread, and four channels of each head far larger than the rest, as caches have."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    x[..., 1::max(1, shape[-1] // 4)] *= 6.0
    return x


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    ql, kl = _lengths(c)
    H, G, D, T, C = c["H"], c["G"], c["D"], c["T"], c["C"]
    per = [-(-y // T) for y in kl]
    width = max(per) + 1
    n_pages = sum(per) + 3
    fp8 = c["dtype"] == "fp8"
    cdt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((c["B"], width), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = perm[at:at + n]
        at += n
    s = {"case": dict(c), "table": table,
         "q_start": torch.tensor([0] + [sum(ql[:i + 1]) for i in range(len(ql))], dtype=torch.int32, device=dev),
         "kv_len": torch.tensor(kl, dtype=torch.int32, device=dev), "max_q": max(ql), "max_kv": max(kl)}
    if fp8:
        s["k_scale"] = 0.05 + 0.05 * torch.rand(H, generator=g, device=dev)
        s["v_scale"] = 0.05 + 0.05 * torch.rand(H, generator=g, device=dev)
    else:
        s["k_scale"] = s["v_scale"] = None
    for name in ("k", "v"):
        pages = torch.empty((n_pages, H, T, D), dtype=cdt, device=dev)
        step = max(1, (1 << 27) // (H * T * D))
        for i in range(0, n_pages, step):
            x = _rows(g, min(step, n_pages - i), H, T, D)
            if fp8:
                x = (x / s[name + "_scale"][None, :, None, None]).clamp(-448, 448)
            pages[i:i + step] = x.to(cdt)
        s[name + "_pages"] = pages
    N = sum(ql) + c["pad"]
    HQ = H * G
    s["q"] = torch.randn((N, HQ, D), generator=g, device=dev).to(torch.bfloat16)
    s["out"] = torch.zeros((N, HQ, D), dtype=torch.bfloat16, device=dev)
    s["bounds"] = None
    if C:
        # the bounds of what is in the cache before the call
        before = [y - x for x, y in zip(ql, kl)] if c["op"] == "append" else kl
        full = torch.zeros((n_pages,), dtype=torch.int64, device=dev)
        for b, n in enumerate(before):
            used = -(-n // T)
            if used:
                full[table[b, :used].long()] = T
                full[table[b, used - 1].long()] = n - (used - 1) * T
        s["bounds"] = torch.zeros((n_pages, H, T // C, 2, D), dtype=torch.bfloat16, device=dev)
        step = max(1, (1 << 27) // (H * T * D))
        for i in range(0, n_pages, step):
            x = s["k_pages"][i:i + step].float()
            live = (torch.arange(T, device=dev)[None, :] < full[i:i + step, None])[:, None, :, None]
            some = live.view(-1, 1, T // C, C, 1).any(3)
            for j, (fill, red) in enumerate(((math.inf, "amin"), (-math.inf, "amax"))):
                y = getattr(x.masked_fill(~live, fill).view(-1, H, T // C, C, D), red)(3)
                s["bounds"][i:i + step, :, :, j] = torch.where(some, y, torch.zeros_like(y)).to(torch.bfloat16)
    if c["op"] == "append":
        s["k"] = _rows(g, N, H, D).to(torch.bfloat16)
        s["v"] = _rows(g, N, H, D).to(torch.bfloat16)
        s["inv_freq"] = _inv_freq(c, dev) if c["rotary"] else None
    else:
        s["lse"] = torch.zeros((N, HQ), dtype=torch.float32, device=dev)
    if c["op"] == "sparse":
        s["blocks"] = torch.full((N, H, c["top_k"]), -1, dtype=torch.int32, device=dev)
    if own:
        import lossless_float_compression_amd as zx
        s["cache"] = zx.PagedKVCache(n_pages, H, D, T, zx.FP8_E4M3FN if fp8 else zx.BF16, block_tokens=C or None,
                                     k=s["k_pages"], v=s["v_pages"], bounds=s["bounds"],
                                     k_scale=s["k_scale"], v_scale=s["v_scale"])
        s["batch"] = zx.PagedBatch(s["q_start"], s["kv_len"], table, max_q=s["max_q"], max_kv=s["max_kv"])
        if c["op"] == "append" and c["rotary"]:
            s["rotary"] = zx.Rotary(c["rotary"], interleaved=c["interleaved"], inv_freq=s["inv_freq"])
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    c = s["case"]
    if own:
        cache, batch = s["cache"], s["batch"]
        if c["op"] == "append":
            cache.append(s["k"], s["v"], batch, q=s["q"], rotary=s.get("rotary"), q_out=s["out"])
            return {"k": s["k_pages"], "v": s["v_pages"], "q": s["out"], "bounds": s["bounds"]}
        if c["op"] == "attend":
            cache.attend(s["q"], batch, causal=c["causal"], window=c["window"], out=s["out"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        cache.select(s["q"], batch, c["top_k"], keep_first=c["keep_first"], keep_last=c["keep_last"], blocks=s["blocks"])
        cache.attend(s["q"], batch, blocks=s["blocks"], out=s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"], "blocks": s["blocks"]}
    return {"append": _plain_append, "attend": _plain_attend, "sparse": _plain_sparse}[c["op"]](s)


def _tokens(s):
    """Sequence and position of each packed token; sequence -1 behind the last one."""
    n = s["q"].shape[0]
    t = torch.arange(n, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["q_start"][1:].contiguous(), t, right=True)
    live = b < s["kv_len"].numel()
    b = b.clamp(max=s["kv_len"].numel() - 1)
    p = s["kv_len"][b] - s["q_start"][b + 1] + t
    return b, p.long(), live


def _rotate(x, c, s, interleaved, r):
    x = x.float()
    y = x.clone()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    u, w = a * c - b * s, b * c + a * s
    if interleaved:
        y[..., 0:r:2], y[..., 1:r:2] = u, w
    else:
        y[..., :r // 2], y[..., r // 2:r] = u, w
    return y


def _plain_append(s):
    c = s["case"]
    H, D, T, C = c["H"], c["D"], c["T"], c["C"]
    b, p, live = _tokens(s)
    k, q = s["k"].float(), s["q"].float()
    if c["rotary"]:
        ang = p.double()[:, None] * s["inv_freq"][None, :]
        cs, sn = torch.cos(ang).float()[:, None, :], torch.sin(ang).float()[:, None, :]
        k = _rotate(k, cs, sn, c["interleaved"], c["rotary"])
        q = _rotate(q, cs, sn, c["interleaved"], c["rotary"])
    s["out"].copy_(torch.where(live[:, None, None], q.to(torch.bfloat16), s["out"]))
    v = s["v"].float()
    if c["dtype"] == "fp8":
        k = (k / s["k_scale"][None, :, None]).clamp(-448, 448)
        v = (v / s["v_scale"][None, :, None]).clamp(-448, 448)
    kp, vp = s["k_pages"], s["v_pages"]
    raw = torch.uint8 if c["dtype"] == "fp8" else torch.bfloat16   # 8-bit values move as bytes
    k, v = k.to(kp.dtype).view(raw), v.to(vp.dtype).view(raw)
    # rows behind the last sequence go where the first row goes, with its values
    first = torch.where(live, torch.arange(live.numel(), device="cuda"), torch.zeros_like(b))
    page = s["table"][b[first], torch.div(p[first], T, rounding_mode="floor")].long()
    kp.view(raw)[page, :, p[first] % T] = k[first]
    vp.view(raw)[page, :, p[first] % T] = v[first]
    if C:
        # smallest and largest key of each touched block: the new ones, and what was there unless the block begins here
        nb = T // C
        n_pages = kp.shape[0]
        slot = page * nb + torch.div(p[first] % T, C, rounding_mode="floor")
        begins = torch.zeros(n_pages * nb, dtype=torch.int32, device="cuda")
        begins.index_reduce_(0, slot, (p[first] % C == 0).to(torch.int32), "amax")
        begins = begins.view(n_pages, 1, nb, 1) > 0
        kk = k.view(kp.dtype)[first].float()
        for j, red in ((0, "amin"), (1, "amax")):
            old = s["bounds"][:, :, :, j].float()
            old = torch.where(begins, torch.full_like(old, math.inf if j == 0 else -math.inf), old)
            flat = old.permute(0, 2, 1, 3).reshape(n_pages * nb, H * D)
            flat.index_reduce_(0, slot, kk.reshape(-1, H * D), red)
            s["bounds"][:, :, :, j] = flat.view(n_pages, nb, H, D).permute(0, 2, 1, 3).to(torch.bfloat16)
    return {"k": kp, "v": vp, "q": s["out"], "bounds": s["bounds"]}


def _soften(sc, see):
    """Weights and ln sum exp of scores; a row that sees nothing: zeros and -inf."""
    sc = sc.masked_fill(~see, -math.inf)
    m = sc.amax(-1, keepdim=True)
    e = torch.exp(sc - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = e.sum(-1, keepdim=True)
    return e / torch.where(l > 0, l, torch.ones_like(l)), (m + torch.log(l)).squeeze(-1)


def _plain_attend(s):
    c = s["case"]
    B, H, G, D, T = c["B"], c["H"], c["G"], c["D"], c["T"]
    mq, mk = s["max_q"], s["max_kv"]
    np_ = -(-mk // T)
    pages = s["table"][:, :np_].clamp(min=0).long()
    raw = torch.uint8 if c["dtype"] == "fp8" else torch.bfloat16

    def gathered(x, scale):
        y = x.view(raw)[pages].view(x.dtype).permute(0, 2, 1, 3, 4).float()      # [B, H, pages, T, D]
        if scale is not None:
            y = y * scale[None, :, None, None, None]
        return y.reshape(B * H, np_ * T, D)

    n = s["q"].shape[0]
    i = torch.arange(mq, device="cuda")
    qs, qe = s["q_start"][:-1].long(), s["q_start"][1:].long()
    row = qs[:, None] + i[None, :]
    real = row < qe[:, None]
    q = s["q"][row.clamp(max=n - 1)].float()                                      # [B, mq, HQ, D]
    q = q.view(B, mq, H, G, D).permute(0, 2, 1, 3, 4).reshape(B * H, mq * G, D)
    k = gathered(s["k_pages"], s["k_scale"])
    sc = torch.matmul(q, k.transpose(1, 2)).mul_(1.0 / math.sqrt(D)).view(B, H, mq, G, -1)
    del k
    t = torch.arange(np_ * T, device="cuda")[None, None, :]
    pos = s["kv_len"].long()[:, None] - (qe - qs)[:, None] + i[None, :]           # [B, mq]
    see = t < s["kv_len"].long()[:, None, None]
    if c["causal"]:
        see = see & (t <= pos[:, :, None])
    if c["window"]:
        see = see & (t > pos[:, :, None] - c["window"])
    w, lse = _soften(sc, see.expand(B, mq, -1)[:, None, :, None, :])
    del sc
    o = torch.matmul(w.view(B * H, mq * G, -1), gathered(s["v_pages"], s["v_scale"]))
    o = o.view(B, H, mq, G, D).permute(0, 2, 1, 3, 4).reshape(B * mq, H * G, D)
    lse = lse.permute(0, 2, 1, 3).reshape(B * mq, H * G)
    # each packed row takes its padded one; rows behind the last sequence keep what they hold
    b, p, live = _tokens(s)
    at = b * mq + (torch.arange(n, device="cuda") - qs[b]).clamp(max=mq - 1)
    s["out"].copy_(torch.where(live[:, None, None], o[at].to(torch.bfloat16), s["out"]))
    s["lse"].copy_(torch.where(live[:, None], lse[at], s["lse"]))
    return {"out": s["out"], "lse": s["lse"]}


def _plain_sparse(s):
    c = s["case"]
    H, G, D, T, C, K = c["H"], c["G"], c["D"], c["T"], c["C"], c["top_k"]
    n = s["q"].shape[0]
    nb = T // C
    b, p, live = _tokens(s)
    p = p.clamp(min=0)
    np_ = -(-s["max_kv"] // T)
    pages = s["table"][:, :np_].clamp(min=0).long()
    # bounds in 64 bits: which blocks are taken must not turn on rounding
    bd = s["bounds"][pages].permute(0, 2, 1, 3, 4, 5).reshape(c["B"], H, np_ * nb, 2, D)
    qg = s["q"].double().view(n, H, G, D)
    up, dn = qg.clamp(min=0).sum(2), qg.clamp(max=0).sum(2)                       # [n, H, D]
    mq = s["max_q"]
    qs = s["q_start"][:-1].long()
    row = (qs[:, None] + torch.arange(mq, device="cuda")[None, :]).clamp(max=n - 1)
    pad = lambda x: x[row].permute(0, 2, 1, 3)                                    # noqa: E731  [B, H, mq, D]
    sc = torch.matmul(pad(up), bd[:, :, :, 1].double().transpose(2, 3))
    sc += torch.matmul(pad(dn), bd[:, :, :, 0].double().transpose(2, 3))          # [B, H, mq, blocks]
    at = (torch.arange(n, device="cuda") - qs[b]).clamp(max=mq - 1)
    sc = sc.permute(0, 2, 1, 3)[b, at]                                            # [n, H, blocks]
    j = torch.arange(np_ * nb, device="cuda")[None, :]
    newest = torch.div(p, C, rounding_mode="floor")[:, None]
    seen = j <= newest
    forced = seen & ((j < c["keep_first"]) | (j > newest - c["keep_last"]))
    sc = sc.masked_fill(forced[:, None, :], math.inf).masked_fill(~seen[:, None, :], -math.inf)
    order = torch.sort(sc, dim=-1, descending=True, stable=True)[1][..., :K]      # [n, H, <=K]
    taken = torch.gather(seen[:, None, :].expand(n, H, -1), 2, order)
    idx = torch.where(taken, order, torch.full_like(order, np_ * nb)).sort(-1)[0]
    idx = torch.nn.functional.pad(idx, (0, K - idx.shape[-1]), value=np_ * nb)
    full = torch.where(idx < np_ * nb, idx, torch.full_like(idx, -1))
    s["blocks"].copy_(torch.where(live[:, None, None], full.to(torch.int32), s["blocks"]))
    # the taken blocks' tokens
    real = full >= 0
    f = full.clamp(min=0)
    page = s["table"].clamp(min=0).long()[b[:, None, None], torch.div(f, nb, rounding_mode="floor")]
    h = torch.arange(H, device="cuda")[None, :, None]
    raw = torch.uint8 if c["dtype"] == "fp8" else torch.bfloat16

    def taken_rows(x, scale):
        y = x.view(raw).view(-1, H, nb, C, D)[page, h, f % nb].view(x.dtype).float()   # [n, H, K, C, D]
        if scale is not None:
            y = y * scale[None, :, None, None, None]
        return y.view(n * H, K * C, D)

    t = f[..., None] * C + torch.arange(C, device="cuda")
    see = (real[..., None] & (t <= p[:, None, None, None])).view(n, H, 1, K * C)
    q = s["q"].float().view(n * H, G, D)
    k = taken_rows(s["k_pages"], s["k_scale"])
    w, lse = _soften((torch.matmul(q, k.transpose(1, 2)) * (1.0 / math.sqrt(D))).view(n, H, G, -1), see)
    del k
    o = torch.matmul(w.view(n * H, G, -1), taken_rows(s["v_pages"], s["v_scale"]))
    s["out"].copy_(torch.where(live[:, None, None], o.view(n, H * G, D).to(torch.bfloat16), s["out"]))
    s["lse"].copy_(torch.where(live[:, None], lse.view(n, H * G), s["lse"]))
    return {"out": s["out"], "lse": s["lse"], "blocks": s["blocks"]}


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    c = case
    s = prepare(case, seed)
    H, G, D, T = c["H"], c["G"], c["D"], c["T"]
    start, total = s["q_start"].tolist(), s["kv_len"].tolist()
    table = s["table"].tolist()
    ks = s["k_scale"].double() if s["k_scale"] is not None else torch.ones(H, dtype=torch.float64, device="cuda")
    vs = s["v_scale"].double() if s["v_scale"] is not None else torch.ones(H, dtype=torch.float64, device="cuda")
    if c["op"] == "append":
        r = c["rotary"]

        def turned(x, pos):                                       # [n, heads, D], [n]
            if not r:
                return x
            a = pos.double()[:, None, None] * _inv_freq(c, "cuda")
            z = torch.complex(torch.cos(a), torch.sin(a))
            if c["interleaved"]:
                w = torch.view_as_complex(x[..., :r].reshape(*x.shape[:2], r // 2, 2).contiguous()) * z
                y = torch.view_as_real(w).reshape(*x.shape[:2], r)
            else:
                w = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * z
                y = torch.cat((w.real, w.imag), -1)
            return torch.cat((y, x[..., r:]), -1)

        kp, vp, q = s["k_pages"].double(), s["v_pages"].double(), s["out"].double()
        most = 448.0 if c["dtype"] == "fp8" else math.inf
        for b in range(c["B"]):
            t = torch.arange(start[b], start[b + 1], device="cuda")
            p = total[b] - start[b + 1] + t
            pg = s["table"][b][p // T].long()
            q[t] = turned(s["q"][t].double(), p)
            kp[pg, :, p % T] = (turned(s["k"][t].double(), p) / ks[:, None]).clamp(-most, most)
            vp[pg, :, p % T] = (s["v"][t].double() / vs[:, None]).clamp(-most, most)
        # the bounds are values that were already rounded: they have no value of their own in 64 bits
        return {"k": kp, "v": vp, "q": q, "bounds": None}
    out, lse = s["out"].double(), s["lse"].double()
    blocks = s.get("blocks")
    for b in range(c["B"]):
        n, y = start[b + 1] - start[b], total[b]
        t = torch.arange(y, device="cuda")
        pg = torch.tensor(table[b], device="cuda")[t // T]
        raw = torch.uint8 if c["dtype"] == "fp8" else torch.bfloat16
        if c["op"] == "sparse":
            C, nb = c["C"], T // c["C"]
            m = (y - 1) // C + 1
            jb = torch.arange(m, device="cuda")
            bd = s["bounds"][torch.tensor(table[b], device="cuda")[jb // nb], :, jb % nb].double()   # [m, H, 2, D]
        for h in range(H):
            k = s["k_pages"].view(raw)[pg, h, t % T].view(s["k_pages"].dtype).double() * ks[h]
            v = s["v_pages"].view(raw)[pg, h, t % T].view(s["v_pages"].dtype).double() * vs[h]
            for i0 in range(0, n, 1024):
                i = torch.arange(i0, min(n, i0 + 1024), device="cuda")
                p = y - n + i
                see = torch.ones((i.numel(), y), dtype=torch.bool, device="cuda")
                if c["causal"]:
                    see &= t[None, :] <= p[:, None]
                if c["window"]:
                    see &= t[None, :] >= p[:, None] - (c["window"] - 1)
                qh = s["q"][start[b] + i][:, h * G:(h + 1) * G].double()                              # [i, G, D]
                if c["op"] == "sparse":
                    take = torch.zeros((i.numel(), m), dtype=torch.bool, device="cuda")
                    for e, pe in enumerate(p.tolist()):
                        last = pe // C
                        keep = [x for x in range(last + 1) if x < c["keep_first"] or x > last - c["keep_last"]]
                        z = qh[e][:, None, None, :] * bd[None, :last + 1, h]                          # [G, blocks, 2, D]
                        z = z.amax(2).sum((0, 2))
                        z[keep] = math.inf
                        top = torch.sort(-z, stable=True)[1][:c["top_k"]].sort()[0]
                        take[e, top] = True
                        blocks[start[b] + i0 + e, h, :top.numel()] = top.to(torch.int32)
                    see &= take[:, t // C]
                sc = torch.einsum("igd,td->igt", qh, k) / math.sqrt(D)
                sc.masked_fill_(~see[:, None, :], -math.inf)
                lse[start[b] + i, h * G:(h + 1) * G] = torch.logsumexp(sc, -1)
                w = torch.nan_to_num(torch.softmax(sc, -1), nan=0.0)
                out[start[b] + i, h * G:(h + 1) * G] = torch.einsum("igt,td->igd", w, v)
    res = {"out": out, "lse": lse}
    if c["op"] == "sparse":
        res["blocks"] = blocks
    return res
