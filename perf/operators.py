"""The paged key/value cache and the attention over it, as measurable cases.

Three operators: writing new tokens into a paged cache (quantised to 8 bits as they are
written), reading cached tokens back, and the attention of a chunk of new tokens over the
cache. ``run`` computes them in plain torch (``own`` false) or through the framework's
entry points (``own`` true: ``KvCache.write``, ``.read``, ``.attention``).

A case is a dict: ``op`` ("append": write the new tokens, then read them back; "read":
read whole sequences back; "attend"), ``fmt`` ("int8" or "bf16", what the cache holds),
``heads`` / ``kv_heads`` / ``dim`` (query heads, key/value heads, head dimension),
``page`` (tokens per page), ``seqs`` sequences with ``new_lo..new_hi`` new tokens each
after ``ctx_lo..ctx_hi`` cached ones, ``window`` (0: none), ``fused`` (K, V or Q are slices of
one wider projection output, so that rows are strided).
"""
import math

import torch

own = False

GOLD = 0.6180339887498949
BF16 = torch.bfloat16
TINY = 2.0 ** -126


# ------------------------------------------------------------------ cases

def _case(name, op, fmt, seqs, new, ctx, heads=32, kv_heads=8, dim=128, page=16, window=0, fused=False):
    c = dict(op=op, fmt=fmt, seqs=seqs, new_lo=new[0], new_hi=new[1], ctx_lo=ctx[0], ctx_hi=ctx[1],
             heads=heads, kv_heads=kv_heads, dim=dim, page=page, window=window, fused=fused)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step of 64 requests: each writes its one new token
        _case("append_decode", "append", "int8", 64, (1, 1), (100, 4000)),
        # a prefill step, 8 prompts of 2048 tokens
        _case("append_prefill", "append", "int8", 8, (2048, 2048), (0, 0), page=64),
        # ragged chunks out of a fused projection, an unquantised cache with small heads
        _case("append_ragged", "append", "bf16", 37, (1, 333), (0, 777), heads=12, kv_heads=4, dim=64,
              page=32, fused=True),
        # prefixes taken out of the cache (to move or to re-quantise them): a few short ones
        _case("read_short", "read", "int8", 5, (1, 300), (0, 0)),
        # ... and long ones
        _case("read_long", "read", "int8", 6, (4001, 40000), (0, 0), page=64),
        # one request, one token: the latency of a step
        _case("attend_one", "attend", "int8", 1, (1, 1), (2047, 2047)),
        # a decode step of 64 requests of very different lengths
        _case("attend_decode", "attend", "int8", 64, (1, 1), (17, 8191)),
        # the largest decode batch, unquantised cache
        _case("attend_decode_bf16", "attend", "bf16", 256, (1, 1), (500, 4095), page=32),
        # a few drafted tokens per request checked at once
        _case("attend_draft", "attend", "int8", 32, (3, 6), (300, 6000)),
        # one chunk of a long prompt over what is cached of it
        _case("attend_chunk", "attend", "int8", 1, (512, 512), (32000, 32000), page=64),
        # a prefill step, 8 prompts of 2048 tokens
        _case("attend_prefill", "attend", "bf16", 8, (2048, 2048), (0, 0), page=64),
        # continuous batching: decode steps and chunks in one call, a sliding window, small heads
        _case("attend_mixed", "attend", "int8", 40, (1, 700), (0, 9000), heads=14, kv_heads=2, dim=64,
              page=32, window=4096, fused=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "attend"])
    fmt = rng.choice(["int8", "int8", "bf16"])
    dim = rng.choice([128, 128, 64])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    fused = rng.random() < 0.3
    window = 0
    if op == "append":
        seqs = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, 16384 // seqs)
        new, ctx = (rng.randint(1, hi), hi), (0, rng.randint(0, 4000))
    elif op == "read":
        seqs = _log_int(rng, 1, 16)
        hi = _log_int(rng, 1, 100000 // seqs)
        new, ctx = (rng.randint(1, hi), hi), (0, 0)
    else:
        hi = _log_int(rng, 1, 2048)
        seqs = _log_int(rng, 1, max(1, min(256, 8192 // hi)))
        new = (rng.randint(1, hi), hi)
        ctx_hi = _log_int(rng, 1, min(32000, max(64, 1000000 // seqs)))
        ctx = (rng.randint(0, ctx_hi), ctx_hi)
        window = rng.choice([0, 0, 0, _log_int(rng, 1, 8192)])
    c = _case(None, op, fmt, seqs, new, ctx, heads, kv_heads, dim, page, window, fused)
    # a drawn case costs no more than the largest listed ones
    while work(c)["flops"] > 2.7e11 or work(c)["bytes"] > 2.4e9:
        key = "seqs" if c["seqs"] > 1 else "ctx_hi"
        c[key] = c[key] * 3 // 4
        c["ctx_lo"] = min(c["ctx_lo"], c["ctx_hi"])
    return c


def _spread(lo, hi, n, step):
    """n whole numbers spread over lo..hi, the largest first."""
    if n == 1:
        return [hi]
    return [hi] + [lo + int((hi - lo + 1) * ((i * step) % 1.0)) for i in range(1, n)]


def _lengths(case):
    """New tokens and total tokens of every sequence."""
    n = case["seqs"]
    new = _spread(case["new_lo"], case["new_hi"], n, GOLD)
    if case["op"] == "attend" and case["new_hi"] >= 64 and n >= 16:
        # continuous batching: all but a few sequences decode one token
        new = [x if i % 16 == 0 else case["new_lo"] for i, x in enumerate(new)]
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], n, GOLD * GOLD)
    return new, [a + b for a, b in zip(new, ctx)]


def _pairs(case):
    """Visible (query token, key) pairs, and keys any query of their sequence sees."""
    w = case["window"]
    pairs = keys = 0
    for n, total in zip(*_lengths(case)):
        first = total - n
        if w == 0 or total <= w:
            pairs += n * first + n * (n + 1) // 2
            keys += total
        else:
            full = min(n, max(0, w - first))        # rows whose window is not yet full
            pairs += full * first + full * (full + 1) // 2 + (n - full) * w
            keys += min(total, n + w - 1)
    return pairs, keys


def work(case):
    new, total = _lengths(case)
    T, H, D = sum(new), case["kv_heads"], case["dim"]
    held = D + 2 if case["fmt"] == "int8" else 2 * D     # bytes of a cached row
    table = 4 * sum(-(-t // case["page"]) for t in total)
    if case["op"] == "append":
        # K and V read, the cache written, the same tokens handed back
        return {"bytes": 2 * T * H * (2 * D + held + 2 * D) + table, "flops": 0}
    if case["op"] == "read":
        return {"bytes": 2 * T * H * (held + 2 * D) + table, "flops": 0}
    pairs, keys = _pairs(case)
    Hq = case["heads"]
    return {"bytes": T * Hq * (2 * D + 2 * D + 4) + 2 * keys * H * held + table,
            "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------ inputs

def _quantise(x):
    """Codes (fp32 whole numbers) and scales (fp32 values of bf16) of rows x[..., D]."""
    f = x.float()
    s = (f.abs().amax(-1) / 127.0).to(BF16).float().clamp_min(TINY)
    q = (f / s.unsqueeze(-1)).round().clamp(-127, 127)
    ok = f.isfinite().all(-1)
    q = torch.where(ok.unsqueeze(-1), q, torch.zeros((), device=f.device))
    s = torch.where(ok, s, torch.full((), float("nan"), device=f.device))
    return q, s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(1000003 * seed + 17)
    H, D, Hq, p = case["kv_heads"], case["dim"], case["heads"], case["page"]
    new, total = _lengths(case)
    T = sum(new)
    counts = [-(-t // p) for t in total]
    n_pages = sum(counts) + 3
    # every sequence's pages are scattered over the arena; table entries past its last
    # page are whatever was there before
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    width = max(counts) + 1
    table = torch.full((len(new), width), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = perm[at:at + c]
        at += c
    start = [0]
    for n in new:
        start.append(start[-1] + n)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    # keys have a few loud channels, values do not
    gain = torch.where(torch.rand(H, 1, D, generator=g, device=dev) < 0.05, 4.0, 1.0)
    arenas = []
    for loud in (True, False):
        pages = torch.empty((n_pages, H, p, D), dtype=BF16, device=dev)
        for i in range(0, n_pages, 1024):
            x = normal(min(1024, n_pages - i), H, p, D)
            pages[i:i + 1024] = x * gain if loud else x
        # rows that hold no token: what an earlier request left, here the worst there is
        dead = torch.ones((n_pages, p), dtype=torch.bool, device=dev)
        for b, t in enumerate(total):
            own_rows = torch.arange(counts[b] * p, device=dev).view(counts[b], p) >= t
            dead[table[b, :counts[b]].long()] = own_rows
        pages.masked_fill_(dead[:, None, :, None], float("nan"))
        if case["fmt"] == "int8":
            codes = torch.empty(pages.shape, dtype=torch.int8, device=dev)
            scales = torch.empty(pages.shape[:3], dtype=BF16, device=dev)
            for i in range(0, n_pages, 1024):
                q, s = _quantise(pages[i:i + 1024])
                codes[i:i + 1024], scales[i:i + 1024] = q.to(torch.int8), s.to(BF16)
            arenas += [codes, scales]
        else:
            arenas += [pages, None]
    state = dict(case=case, new=new, total=total, start=start, T=T, table=table,
                 k=arenas[0], ks=arenas[1], v=arenas[2], vs=arenas[3])

    def rows(*heads):
        """Projection outputs [T][h][D], slices of one wider tensor where the case says so."""
        if case["fused"]:
            wide = normal(T, (sum(heads) + 1) * D).to(BF16)
            out, c = [], 0
            for h in heads:
                out.append(wide[:, c * D:(c + h) * D].unflatten(1, (h, D)))
                c += h
            return out
        return [normal(T, h, D).to(BF16) for h in heads]

    if case["op"] == "append":
        state["K"], state["V"] = rows(H, H)
    elif case["op"] == "attend":
        state["Q"] = rows(Hq)[0]
    # the flat (page, row) of every new token, as a program that manages pages has it
    flat_page, flat_row = [], []
    for b in range(len(new)):
        pos = torch.arange(total[b] - new[b], total[b], device=dev)
        flat_page.append(table[b].long()[pos // p])
        flat_row.append(pos % p)
    state["flat_page"], state["flat_row"] = torch.cat(flat_page), torch.cat(flat_row)
    if own:
        import adapter_linear_gb300 as al
        fmt = al.LORA_KV_INT8 if case["fmt"] == "int8" else al.LORA_KV_BF16
        cache = al.KvCache(n_pages, p, H, D, fmt, arenas=(state["k"], state["v"], state["ks"], state["vs"]))
        if case["op"] == "attend":
            cache.reserve(T, Hq, len(new))
        state["cache"] = cache
        state["batch"] = al.KvBatch(table, torch.tensor(start, dtype=torch.int32, device=dev),
                                    torch.tensor(total, dtype=torch.int32, device=dev), T, max(new))
    return state


# ------------------------------------------------------------------ the operators

def _plain_read(st):
    out = []
    for codes, scales in ((st["k"], st["ks"]), (st["v"], st["vs"])):
        x = codes[st["flat_page"], :, st["flat_row"]]
        if scales is not None:
            x = (x.float() * scales[st["flat_page"], :, st["flat_row"]].float().unsqueeze(-1)).to(BF16)
        out.append(x)
    return out


def _plain_write(st):
    for x, codes, scales in ((st["K"], st["k"], st["ks"]), (st["V"], st["v"], st["vs"])):
        if scales is None:
            codes[st["flat_page"], :, st["flat_row"]] = x
        else:
            q, s = _quantise(x)
            codes[st["flat_page"], :, st["flat_row"]] = q.to(torch.int8)
            scales[st["flat_page"], :, st["flat_row"]] = s.to(BF16)


def _sequence(st, b, lo, hi):
    """Keys and values lo..hi of sequence b as fp32 [Hkv][hi - lo][D]."""
    p = st["case"]["page"]
    first = lo // p
    pages = st["table"][b, first:-(-hi // p)].long()
    out = []
    for codes, scales in ((st["k"], st["ks"]), (st["v"], st["vs"])):
        x = codes[pages].float()
        if scales is not None:
            x = x * scales[pages].float().unsqueeze(-1)
        x = x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])
        out.append(x[:, lo - first * p:hi - first * p])
    return out


def _plain_attend(st):
    c = st["case"]
    H, D, Hq, w = c["kv_heads"], c["dim"], c["heads"], c["window"]
    G = Hq // H
    dev = st["Q"].device
    O = torch.empty((st["T"], Hq, D), dtype=BF16, device=dev)
    lse = torch.empty((st["T"], Hq), dtype=torch.float32, device=dev)
    for b, (n, total) in enumerate(zip(st["new"], st["total"])):
        r0 = st["start"][b]
        lo = max(0, total - n - w + 1) if w else 0
        K, V = _sequence(st, b, lo, total)
        q = st["Q"][r0:r0 + n].float().view(n, H, G, D).permute(1, 2, 0, 3).reshape(H, G * n, D)
        z = torch.bmm(q, K.transpose(1, 2)) * (1.0 / math.sqrt(D))
        pos = torch.arange(total - n, total, device=dev)[:, None]
        j = torch.arange(lo, total, device=dev)[None, :]
        seen = j <= pos
        if w:
            seen = seen & (j > pos - w)
        z = z.view(H, G, n, total - lo).masked_fill_(~seen, float("-inf"))
        m = z.amax(-1, keepdim=True)
        z = (z - m).exp_()
        s = z.sum(-1, keepdim=True)
        o = torch.bmm(z.view(H, G * n, total - lo), V).view(H, G, n, D) / s
        O[r0:r0 + n] = o.permute(2, 0, 1, 3).reshape(n, Hq, D).to(BF16)
        lse[r0:r0 + n] = (m + s.log()).squeeze(-1).permute(2, 0, 1).reshape(n, Hq)
    return O, lse


def run(st):
    op = st["case"]["op"]
    if own:
        cache, batch = st["cache"], st["batch"]
        if op == "append":
            cache.write(st["K"], st["V"], batch)
            return cache.read(batch)
        if op == "read":
            return cache.read(batch)
        return cache.attention(st["Q"], batch, window=st["case"]["window"])
    if op == "append":
        _plain_write(st)
        return tuple(_plain_read(st))
    if op == "read":
        return tuple(_plain_read(st))
    return _plain_attend(st)


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """The outputs of ``run`` from the definition, in 64 bits."""
    st = prepare(case, seed)
    c, H, D, p = case, case["kv_heads"], case["dim"], case["page"]
    page, row = st["flat_page"], st["flat_row"]
    if c["op"] == "append":
        outs = []
        for x in (st["K"], st["V"]):
            x = x.double()
            if c["fmt"] == "int8":
                step = (x.abs().amax(-1, keepdim=True) / 127).to(BF16).double().clamp_min(TINY)
                x = torch.clamp(torch.round(x / step), -127, 127) * step
            outs.append(x)
        return tuple(outs)

    def stored(codes, scales, pages, rows):
        x = codes[pages, :, rows].double()                     # [tokens][Hkv][D]
        return x if scales is None else x * scales[pages, :, rows].double()[..., None]

    if c["op"] == "read":
        return tuple(stored(st[a], st[a + "s"], page, row) for a in ("k", "v"))
    if 6 * D * c["heads"] * _pairs(c)[0] > 1.5e13:
        return None
    group = c["heads"] // H
    O = torch.zeros((st["T"], c["heads"], D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((st["T"], c["heads"]), dtype=torch.float64, device="cuda")
    for b, (n, total) in enumerate(zip(st["new"], st["total"])):
        j = torch.arange(total, device="cuda")
        pages, rows = st["table"][b].long()[j // p], j % p
        K, V = (stored(st[a], st[a + "s"], pages, rows) for a in ("k", "v"))
        for i0 in range(0, n, 512):
            i1 = min(n, i0 + 512)
            pos = torch.arange(total - n + i0, total - n + i1, device="cuda")
            hidden = j[None, :] > pos[:, None]
            if c["window"]:
                hidden |= j[None, :] <= pos[:, None] - c["window"]
            at = slice(st["start"][b] + i0, st["start"][b] + i1)
            for h in range(c["heads"]):
                z = st["Q"][at, h].double() @ K[:, h // group].T / math.sqrt(D)
                z[hidden] = float("-inf")
                l = torch.logsumexp(z, 1)
                O[at, h] = torch.exp(z - l[:, None]) @ V[:, h // group]
                lse[at, h] = l
    return O, lse
