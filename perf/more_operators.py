"""Rotary positions, the paged cache's page tables and attention over a shared prefix, as measurable cases.

Five operators of a served layer: rotating queries and keys by their positions (``rotate``); the
cache's write with that rotation on the way (``append``); the page tables' update, which forks,
reorders, trims, frees and extends sequences, with the copies of pages it asks for (``update``); the
compaction of a fragmented arena (``compact``); and the attention of groups of sequences that
share a prefix's pages (``shared``). ``run`` computes them in plain torch (``own`` false) or through
the framework's entry points (``own`` true: ``Rotary.apply``, ``KvCache.write_rotary``,
``KvPages.update``, ``KvPages.compact``, ``KvCache.copy``, ``KvCache.attention_shared``).

What the keys of a case say is written beside the functions that make one.
"""
import math

import torch

own = False

GOLD = 0.6180339887498949
BF16 = torch.bfloat16
TINY = 2.0 ** -126


# ------------------------------------------------------------------ cases

def _rotate(name, tokens, far, heads=32, kv_heads=8, dim=128, rotary=128, layout="half", scaling="none",
            inverse=False, fused=False):
    """``tokens`` tokens at positions up to ``far``, ``heads`` query and ``kv_heads`` key heads of ``dim``
    values, the first ``rotary`` of them rotated; ``inverse`` the other way round; ``fused``: slices of one
    projection's output."""
    return _named(name, dict(op="rotate", tokens=tokens, far=far, heads=heads, kv_heads=kv_heads, dim=dim,
                             rotary=rotary, layout=layout, scaling=scaling, inverse=inverse, fused=fused))


def _append(name, seqs, new, ctx, fmt="int8", heads=32, kv_heads=8, dim=128, rotary=128, layout="half",
            scaling="none", page=16, fused=False):
    """``seqs`` sequences of ``new`` (lowest, highest) new tokens after ``ctx`` cached ones."""
    return _named(name, dict(op="append", seqs=seqs, new_lo=new[0], new_hi=new[1], ctx_lo=ctx[0], ctx_hi=ctx[1],
                             fmt=fmt, heads=heads, kv_heads=kv_heads, dim=dim, rotary=rotary, layout=layout,
                             scaling=scaling, page=page, fused=fused))


def _update(name, slots, prompts, tokens, room, kind, kv_heads=8, dim=128, page=16):
    """``slots`` slots; ``kind`` "step": each keeps its tokens and gets ``room`` more; "fork": each becomes a
    copy of one of the first ``prompts`` slots; "beam": each goes on from a slot of its own group of
    ``slots / prompts``. ``tokens``: lengths, lowest and highest."""
    return _named(name, dict(op="update", slots=slots, prompts=prompts, tok_lo=tokens[0], tok_hi=tokens[1], room=room,
                             kind=kind, kv_heads=kv_heads, dim=dim, page=page))


def _compact(name, pages, slots, fill, kv_heads=8, dim=128, page=16):
    """An arena of ``pages`` pages, ``fill`` percent of them used, by ``slots`` sequences, anywhere."""
    return _named(name, dict(op="compact", pages=pages, slots=slots, fill=fill, kv_heads=kv_heads, dim=dim, page=page))


def _shared(name, groups, members, prefix, own_tokens, new, fmt="int8", heads=32, kv_heads=8, dim=128, page=16):
    """``groups`` groups of ``members`` sequences with a prefix of ``prefix`` (lowest, highest) tokens in common,
    ``own_tokens`` cached ones of their own and ``new`` new ones."""
    return _named(name, dict(op="shared", groups=groups, members=members, pre_lo=prefix[0], pre_hi=prefix[1],
                             ctx_lo=own_tokens[0], ctx_hi=own_tokens[1], new_lo=new[0], new_hi=new[1], fmt=fmt,
                             heads=heads, kv_heads=kv_heads, dim=dim, page=page))


def _named(name, case):
    return dict(case, name=name) if name else case


def listed():
    return [
        # queries and keys of one decode step of 64 requests: latency
        _rotate("rotate_decode", 64, 4000),
        # a long prompt of a model that rotates half of each head, interleaved, with a context stretched
        # far beyond its training length, out of a fused projection
        _rotate("rotate_long", 30011, 1000000, heads=24, kv_heads=8, rotary=64, layout="interleaved",
                scaling="yarn", fused=True),
        # one decode step of 64 requests: its tokens go into an 8-bit cache
        _append("append_decode", 64, (1, 1), (100, 4000)),
        # a prefill step, 8 prompts of 2048 tokens
        _append("append_prefill", 8, (2048, 2048), (0, 0), page=64, scaling="bands"),
        # a step of 64 requests with drafts: what was accepted stays, pages for the next drafts
        _update("update_step", 64, 64, (17, 4000), 5, "step"),
        # four prompts, each answered 63 times more
        _update("update_fork", 256, 4, (1000, 6000), 1, "fork"),
        # a small arena after some requests ended
        _compact("compact_small", 600, 20, 60),
        # a large one
        _compact("compact_large", 24000, 300, 55),
        # one prompt of moderate length with 8 answers under way
        _shared("shared_few", 1, 8, (1000, 1000), (1, 60), (1, 1)),
        # 64 requests with one long system prompt
        _shared("shared_decode", 1, 64, (8192, 8192), (17, 500), (1, 1)),
        # 16 prompts with 16 answers each, an unquantised cache
        _shared("shared_groups", 16, 16, (500, 4000), (1, 400), (1, 1), fmt="bf16", page=32),
        # drafts of 48 requests over a few long documents
        _shared("shared_draft", 3, 16, (9000, 16000), (1, 300), (3, 6)),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "append", "update", "compact", "shared", "shared"])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    dim = rng.choice([128, 128, 64])
    fmt = rng.choice(["int8", "int8", "bf16"])
    layout = rng.choice(["half", "half", "interleaved"])
    scaling = rng.choice(["none", "linear", "ntk", "yarn", "bands"])
    fused = rng.random() < 0.3
    if op == "rotate":
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        rotary = rng.choice([dim, dim, 16 * rng.randint(1, dim // 16)])
        most = min(32768, int(2.4e8 / (2 * dim * (heads + kv_heads))))
        return _rotate(None, _log_int(rng, 1, most), _log_int(rng, 100, 1000000), heads, kv_heads, dim, rotary, layout,
                       scaling, rng.random() < 0.3, fused)
    if op == "append":
        seqs = _log_int(rng, 1, 64)
        most = min(16384, int(1.8e8 / (2 * dim * (heads + 2 * kv_heads))))
        hi = _log_int(rng, 1, most // seqs)
        rotary = rng.choice([dim, dim, 16 * rng.randint(1, dim // 16)])
        return _append(None, seqs, (rng.randint(1, hi), hi), (0, rng.randint(0, 4000)), fmt, heads, kv_heads, dim, rotary,
                       layout, scaling, page, fused)
    if op == "update":
        kind = rng.choice(["step", "fork", "beam"])
        prompts = _log_int(rng, 1, 32)
        slots = prompts * rng.randint(1, 512 // prompts)
        hi = _log_int(rng, 1, max(1, min(16000, 1000000 // (slots if kind != "fork" else prompts))))
        return _update(None, slots, prompts, (rng.randint(1, hi), hi), rng.randint(1, 20), kind, kv_heads, dim, page)
    if op == "compact":
        most = int(1.5e9 / (4 * kv_heads * page * dim))
        pages = _log_int(rng, 20, min(24000, most))
        return _compact(None, pages, _log_int(rng, 1, min(300, pages // 8)), rng.randint(10, 90), kv_heads, dim, page)
    groups = _log_int(rng, 1, 16)
    members = _log_int(rng, 1, 256 // groups)
    hi = rng.choice([1, 1, 1, rng.randint(2, 8)])
    rows = groups * members * hi * heads
    pre = _log_int(rng, 16, max(64, min(16000, int(4.5e10 / (4 * dim * rows)), 100000 // groups)))
    ctx = _log_int(rng, 1, max(2, min(500, 100000 // (groups * members))))
    return _shared(None, groups, members, (rng.randint(1, pre), pre), (rng.randint(0, ctx), ctx),
                   (rng.randint(1, hi), hi), fmt, heads, kv_heads, dim, page)


def _spread(lo, hi, n, step=GOLD):
    """n whole numbers spread over lo..hi, the largest first."""
    return [hi] + [lo + int((hi - lo + 1) * ((i * step) % 1.0)) for i in range(1, n)]


def _lengths(case):
    """New tokens and total tokens of every sequence (append, shared), prefixes of every group."""
    n = case["seqs"] if case["op"] == "append" else case["groups"] * case["members"]
    new = _spread(case["new_lo"], case["new_hi"], n)
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], n, GOLD * GOLD)
    if case["op"] == "append":
        return new, [a + b for a, b in zip(new, ctx)], []
    # what is shared are whole pages
    pre = [x // case["page"] * case["page"] for x in _spread(case["pre_lo"], case["pre_hi"], case["groups"])]
    return new, [pre[b // case["members"]] + a + c for b, (a, c) in enumerate(zip(new, ctx))], pre


def _slots(case):
    """Tokens that the slots hold, parent and tokens kept of every slot (update)."""
    n, held = case["slots"], case["prompts"]
    if case["kind"] != "fork":
        held = n
    tokens = _spread(case["tok_lo"], case["tok_hi"], held) + [0] * (n - held)
    if case["kind"] == "beam":  # the slots of a group are equally far
        tokens = [t for t in tokens[:case["prompts"]] for _ in range(n // case["prompts"])]
    if case["kind"] == "step":
        parent = list(range(n))
    elif case["kind"] == "fork":
        parent = [i if i < held else i % held for i in range(n)]
    else:  # a few slots of each group go on, several times
        size = n // case["prompts"]
        parent = [i // size * size + (i * i // 3) % size // 2 for i in range(n)]
    return tokens, parent, [tokens[p] for p in parent]


def work(case):
    op, D, H = case["op"], case["dim"], case["kv_heads"]
    if op == "rotate":
        T, heads = case["tokens"], case["heads"] + H
        return {"bytes": 4 * T * heads * D + 4 * T, "flops": 3 * T * heads * case["rotary"]}
    if op == "compact":
        used = case["pages"] * case["fill"] // 100
        moved = used * (case["pages"] - used) // case["pages"]   # the expected number
        return {"bytes": 2 * moved * 4 * H * case["page"] * D + 8 * used + 8 * case["pages"], "flops": 0}
    if op == "update":
        tokens, parent, keep = _slots(case)
        p = case["page"]
        ends = sum(1 for i, (a, k) in enumerate(zip(parent, keep)) if a != i and k % p)
        rows = sum(k % p for i, (a, k) in enumerate(zip(parent, keep)) if a != i)
        entries = sum(-(-t // p) for t in tokens), sum(-(-(k + case["room"]) // p) for k in keep)
        return {"bytes": 2 * rows * 4 * H * D + 4 * sum(entries) + 8 * _pages_of(case) + 16 * case["slots"] + 12 * ends,
                "flops": 0}
    new, total, pre = _lengths(case)
    T, Hq = sum(new), case["heads"]
    held = D + 2 if case["fmt"] == "int8" else 2 * D     # bytes of a cached row
    table = 4 * sum(-(-t // case["page"]) for t in total)
    if op == "append":
        # Q, K and V read, Q and the cache written; the cache's tokens come back as bf16
        return {"bytes": T * Hq * 4 * D + 2 * T * H * (2 * D + held + 2 * D) + table, "flops": 3 * T * (Hq + H) * case["rotary"]}
    own_keys = sum(t - pre[b // case["members"]] for b, t in enumerate(total))
    pairs = sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(new, total))
    return {"bytes": T * Hq * (4 * D + 4) + 2 * (sum(pre) + own_keys) * H * held + table, "flops": 4 * D * Hq * pairs}


def _pages_of(case):
    """Pages of an update's arena: what the slots hold before and after, and some more."""
    tokens, _, keep = _slots(case)
    p = case["page"]
    return sum(-(-t // p) for t in tokens) + sum(-(-case["room"] // p) + 1 for _ in keep) + case["slots"] + 7


# ------------------------------------------------------------------ frequencies

SCALE, TRAINED = 8.0, 8192   # of the stretched contexts: eight times 8192 tokens


def _frequencies(case, base=10000.0):
    """The angle a pair turns by from one position to the next, fp64, and the factor of its length."""
    R, kind = case["rotary"], case["scaling"]
    i = torch.arange(R // 2, dtype=torch.float64)
    if kind == "ntk" and R > 2:
        base = base * SCALE ** (R / (R - 2))
    f, factor = base ** (-2.0 * i / R), 1.0
    if kind == "linear":
        f = f / SCALE
    elif kind == "yarn":
        # pairs of fewer than 1 turn over the trained length are stretched, of more than 32 are not
        at = [R * math.log(TRAINED / (2 * math.pi * turns)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), R - 1)
        ramp = ((i - low) / (high - low if high > low else 0.001)).clamp(0, 1)
        f = f / SCALE * ramp + f * (1 - ramp)
        factor = 0.1 * math.log(SCALE) + 1.0
    elif kind == "bands":
        # between 1 and 4 turns over the trained length from stretched to not
        turns = TRAINED * f / (2 * math.pi)
        smooth = ((turns - 1.0) / 3.0).clamp(0, 1)
        f = f / SCALE * (1 - smooth) + f * smooth
    return f, factor


def _turned(x, pos, freq, factor, rotary, layout, inverse=False):
    """x [T, heads, D] in fp32, rotated to positions pos [T]; the angles in fp64."""
    angle = (pos.double().unsqueeze(1) * freq).unsqueeze(1)
    c, s = (angle.cos() * factor).float(), (angle.sin() * factor).float()
    if inverse:
        s = -s
    y = x.float().clone()
    r = y[..., :rotary]
    a, b = (r[..., :rotary // 2], r[..., rotary // 2:]) if layout == "half" else (r[..., 0::2], r[..., 1::2])
    a2, b2 = a * c - b * s, a * s + b * c
    a.copy_(a2)
    b.copy_(b2)
    return y


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 29)
    return g


def _rows(g, T, D, heads, fused):
    """Projection outputs [T][h][D], slices of one wider tensor where the case says so."""
    if fused:
        wide = torch.randn(T, (sum(heads) + 1) * D, generator=g, device="cuda").to(BF16)
        at = [sum(heads[:i]) for i in range(len(heads))]
        return [wide[:, c * D:(c + h) * D].unflatten(1, (h, D)) for c, h in zip(at, heads)]
    return [torch.randn(T, h, D, generator=g, device="cuda").to(BF16) for h in heads]


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _quantise(f):
    """Codes (fp32 whole numbers) and scales (fp32 values of bf16) of fp32 rows f[..., D]."""
    s = (f.abs().amax(-1) / 127.0).to(BF16).float().clamp_min(TINY)
    return (f / s.unsqueeze(-1)).round().clamp(-127, 127), s


def _arena(g, pages, case, fmt):
    """Pages of values [pages][H][p][D], and scales for 8 bits."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    if fmt == "bf16":
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(BF16), None
    codes = torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)
    # (a row's values are near normal ones: codes spread evenly, scales within a factor of two)
    return codes, (torch.rand(shape[:3], generator=g, device="cuda") * 0.01 + 0.01).to(BF16)


def _cached(g, case, pages):
    """A cache's state: arenas, and the framework's handle on them."""
    fmt = case.get("fmt", "bf16")
    st = {}
    st["k"], st["ks"] = _arena(g, pages, case, fmt)
    st["v"], st["vs"] = _arena(g, pages, case, fmt)
    if own:
        import adapter_linear_gb300 as al
        st["cache"] = al.KvCache(pages, case["page"], case["kv_heads"], case["dim"],
                                 al.LORA_KV_INT8 if fmt == "int8" else al.LORA_KV_BF16,
                                 arenas=(st["k"], st["v"], st["ks"], st["vs"]))
    return st


def _table(counts, ids, width):
    """A page table [len(counts)][width] with the next counts[b] of ids in row b, -1 behind them."""
    table = torch.full((len(counts), width), -1, dtype=torch.int32, device="cuda")
    j = torch.arange(width, device="cuda")
    table[j.unsqueeze(0) < _ints(counts).unsqueeze(1)] = ids[:sum(counts)].int()
    return table


def _rotary_state(case, st):
    st["freq"], st["factor"] = _frequencies(case)
    st["freq"] = st["freq"].cuda()
    if own:
        import adapter_linear_gb300 as al
        scaling = None if case["scaling"] == "none" else (case["scaling"], SCALE, TRAINED)
        st["rotary"] = al.Rotary(case["rotary"], layout=case["layout"], scaling=scaling)


def prepare(case, seed):
    g = _generator(seed)
    op, p = case["op"], case.get("page", 16)
    if op == "rotate":
        st = {"case": case}
        _rotary_state(case, st)
        T = case["tokens"]
        st["Q"], st["K"] = _rows(g, T, case["dim"], (case["heads"], case["kv_heads"]), case["fused"])
        # packed chunks: runs of positions
        first = torch.randint(0, max(1, case["far"] - 255), (T // 256 + 1,), generator=g, device="cuda")
        st["pos"] = (first.repeat_interleave(256) + torch.arange(256, device="cuda").repeat(len(first)))[:T].int()
        return st
    if op == "append":
        new, total, _ = _lengths(case)
        counts = [-(-t // p) for t in total]
        pages = sum(counts) + 3
        st = _cached(g, case, pages)
        _rotary_state(case, st)
        T, n = sum(new), _ints(new)
        st["case"], st["len"] = case, _ints(total)
        st["table"] = _table(counts, torch.randperm(pages, generator=g, device="cuda"), max(counts) + 1)
        st["start"] = torch.cat([_ints([0]), n.cumsum(0).int()])
        st["Q"], st["K"], st["V"] = _rows(g, T, case["dim"], (case["heads"], case["kv_heads"], case["kv_heads"]),
                                          case["fused"])
        if own:
            import adapter_linear_gb300 as al
            st["batch"] = al.KvBatch(st["table"], st["start"], st["len"], T, max(new))
        return st
    if op == "update":
        tokens, parent, keep = _slots(case)
        counts = [-(-t // p) for t in tokens]
        pages, width = _pages_of(case), -(-(max(tokens) + case["room"]) // p) + 1
        st = _cached(g, case, pages)
        st["case"], st["len"], st["room"] = case, _ints(tokens), _ints([case["room"]] * len(tokens))
        st["table"] = _table(counts, torch.randperm(pages, generator=g, device="cuda"), width)
        # what a slot goes on from is the seed's choice where slots may be exchanged
        order = torch.arange(len(tokens), device="cuda")
        if case["kind"] == "beam":
            size = case["slots"] // case["prompts"]
            order = (order.view(-1, size).gather(1, torch.rand(case["prompts"], size, generator=g, device="cuda").argsort(1))
                     .flatten())
        st["parent"] = order[_ints(parent).long()].int() if case["kind"] == "beam" else _ints(parent)
        st["keep"] = st["len"][st["parent"].long()].clone()
        st["refs"] = _refs(st["table"], pages)
        if own:
            import adapter_linear_gb300 as al
            st["pages"] = al.KvPages(pages, p, case["slots"], width, tensors=(st["table"], st["len"], st["refs"]))
        return st
    if op == "compact":
        pages, used = case["pages"], max(case["slots"], case["pages"] * case["fill"] // 100)
        st = _cached(g, case, pages)
        st["case"] = case
        each = used // case["slots"]
        counts = [used - each * (case["slots"] - 1)] + [each] * (case["slots"] - 1)
        st["table"] = _table(counts, torch.randperm(pages, generator=g, device="cuda"), max(counts) + 1)
        st["len"] = _ints([c * p - b % p for b, c in enumerate(counts)])
        st["refs"] = _refs(st["table"], pages)
        st["new_table"], st["new_refs"] = torch.empty_like(st["table"]), torch.empty_like(st["refs"])
        if own:
            import adapter_linear_gb300 as al
            st["pages"] = al.KvPages(pages, p, case["slots"], st["table"].shape[1],
                                     tensors=(st["table"], st["len"], st["refs"]))
        return st
    # shared: a group's rows of the table begin with the same pages
    new, total, pre = _lengths(case)
    M, width = case["members"], -(-max(total) // p) + 1
    pre_pages = [x // p for x in pre]
    counts = [-(-t // p) - pre_pages[b // M] for b, t in enumerate(total)]
    pages = sum(pre_pages) + sum(counts) + 3
    st = _cached(g, case, pages)
    ids = torch.randperm(pages, generator=g, device="cuda")
    head = _table(pre_pages, ids, width).repeat_interleave(M, 0)
    tail = _table(counts, ids[sum(pre_pages):], width)
    j = torch.arange(width, device="cuda").unsqueeze(0) - _ints(pre_pages).long().repeat_interleave(M).unsqueeze(1)
    st["table"] = torch.where(j < 0, head, tail.gather(1, j.clamp(0, width - 1))).contiguous()
    st["case"], st["len"], st["pre"] = case, _ints(total), _ints(pre)
    # rows that hold no token: what an earlier request left, here the worst there is
    end = st["len"].long().unsqueeze(1) - 1
    page, dead = st["table"].gather(1, end // p).squeeze(1).long(), torch.arange(p, device="cuda") > end % p
    for x in (st["k"], st["v"]) if st["ks"] is None else (st["ks"], st["vs"]):
        x[page] = x[page].masked_fill(dead.view(len(new), 1, p, *[1] * (x.dim() - 3)), float("nan"))
    st["start"] = torch.cat([_ints([0]), _ints(new).cumsum(0).int()])
    st["new_hi"], st["own_hi"], st["pre_hi"] = max(new), max(t - pre[b // M] for b, t in enumerate(total)), max(pre)
    st["Q"] = torch.randn(sum(new), case["heads"], case["dim"], generator=g, device="cuda").to(BF16)
    if own:
        import adapter_linear_gb300 as al
        members = torch.arange(0, case["groups"] * M + 1, M, dtype=torch.int32, device="cuda")
        st["batch"] = al.KvBatch(st["table"], st["start"], st["len"], sum(new), max(new))
        st["groups"] = al.KvGroups(members, st["pre"], max(sum(new[i * M:(i + 1) * M]) for i in range(case["groups"])))
        st["cache"].reserve_shared(sum(new), case["heads"], len(new))
    return st


def _refs(table, pages):
    """How many entries of the table name each page."""
    refs = torch.zeros(pages + 1, dtype=torch.int32, device=table.device)
    at = torch.where(table < 0, pages, table).long().flatten()
    refs.scatter_add_(0, at, torch.ones_like(at, dtype=torch.int32))
    return refs[:pages].clone()


# ------------------------------------------------------------------ the operators, plain

def _plain_rotate(st):
    c = st["case"]
    return tuple(_turned(x, st["pos"], st["freq"], st["factor"], c["rotary"], c["layout"], c["inverse"]).to(BF16)
                 for x in (st["Q"], st["K"]))


def _plain_append(st):
    c = st["case"]
    T = st["Q"].shape[0]
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(st["start"], t.int(), right=True) - 1
    pos = st["len"][seq] - st["start"][seq + 1] + t
    page, row = st["table"][seq, pos // c["page"]].long(), (pos % c["page"]).long()
    turn = (pos, st["freq"], st["factor"], c["rotary"], c["layout"])
    held = []
    for x, values, scales in ((_turned(st["K"], *turn), st["k"], st["ks"]), (st["V"].float(), st["v"], st["vs"])):
        if scales is None:
            values[page, :, row] = x.to(BF16)
            held.append(values[page, :, row])
        else:
            q, s = _quantise(x)
            values[page, :, row], scales[page, :, row] = q.to(torch.int8), s.to(BF16)
            held.append((values[page, :, row].float() * scales[page, :, row].float().unsqueeze(-1)).to(BF16))
    return (_turned(st["Q"], *turn).to(BF16), *held)


def _plain_update(st):
    p, table, held = st["case"]["page"], st["table"], st["len"].long()
    S, W = table.shape
    P = st["k"].shape[0]
    parent, slot = st["parent"].long(), torch.arange(S, device="cuda")
    src = parent.clamp_min(0)
    kept = torch.where(parent >= 0, torch.minimum(st["keep"].long(), held[src]).clamp_min(0), 0)
    total = kept + st["room"]
    full, ends, used = kept // p, kept % p != 0, (total + p - 1) // p
    j = torch.arange(W, device="cuda").unsqueeze(0)
    above = table[src].long()
    shared = j < full.unsqueeze(1)
    count = torch.zeros(P + 1, dtype=torch.int64, device="cuda")
    count.scatter_add_(0, torch.where(shared, above, P).flatten(), torch.ones_like(above).flatten())
    # a page that a slot ends inside stays with the one that may write it: nobody has all of it, the slot
    # held it before or is the first to ask
    last = torch.where(ends, above.gather(1, full.clamp_max(W - 1).unsqueeze(1)).squeeze(1), P)
    asks = slot + S * (parent != slot)
    first = torch.full((P + 1,), 2 * S, device="cuda").scatter_reduce_(0, last, asks, "amin")
    stays = ends & (first[last] == asks) & (count[last] == 0)
    count.scatter_add_(0, torch.where(stays, last, P), torch.ones_like(last))
    free = (count[:P] == 0).nonzero().squeeze(1)
    old = shared | (stays.unsqueeze(1) & (j == full.unsqueeze(1)))
    fresh = ~old & (j < used.unsqueeze(1))
    rank = (fresh.flatten().cumsum(0) - 1).clamp_min(0).view(S, W)
    new = torch.where(old, above, torch.where(fresh, free[rank.clamp_max(len(free) - 1)], -1))
    copied = (ends & ~stays).nonzero().squeeze(1)
    a, b = last[copied], new[copied, full[copied]]
    rows = torch.arange(p, device="cuda").view(1, 1, p, 1) < (kept[copied] % p).view(-1, 1, 1, 1)
    for x in (st["k"], st["v"]):
        x[b] = torch.where(rows, x[a], x[b])
    table.copy_(new)
    st["len"].copy_(total)
    st["refs"].copy_(_refs(table, P))
    return table, st["len"], st["refs"], st["k"], st["v"]


def _plain_compact(st):
    table, refs = st["table"].long(), st["refs"]
    taken, page = refs > 0, torch.arange(len(refs), device="cuda")
    there = page < taken.sum()
    src, dst = (taken & ~there).nonzero().squeeze(1), (~taken & there).nonzero().squeeze(1)
    page[src] = dst
    st["new_table"].copy_(torch.where(table < 0, -1, page[table.clamp_min(0)]))
    st["new_refs"].copy_(refs)
    st["new_refs"][dst], st["new_refs"][src] = refs[src], 0
    for x in (st["k"], st["v"]):
        x[dst] = x[src]
    return st["new_table"], st["new_refs"], st["k"], st["v"]


def _fetch(st, page, row):
    """Keys and values of the tokens at page, row [n, L], as fp32 [n, H, L, D]."""
    out = []
    for values, scales in ((st["k"], st["ks"]), (st["v"], st["vs"])):
        x = values[page, :, row].float()
        if scales is not None:
            x = x * scales[page, :, row].float().unsqueeze(-1)
        out.append(x.transpose(1, 2))
    return out


def _plain_shared(st):
    c, p, dev = st["case"], st["case"]["page"], "cuda"
    g, M, H, D = c["groups"], c["members"], c["kv_heads"], c["dim"]
    S, G, N, T = g * M, c["heads"] // c["kv_heads"], st["new_hi"], st["Q"].shape[0]
    n, pre = (st["start"][1:] - st["start"][:-1]).long(), st["pre"].long()
    table = st["table"].long().clamp_min(0)
    # queries [S, N], padded
    i = torch.arange(N, device=dev)
    at = (st["start"][:-1].long().unsqueeze(1) + i).clamp_max(T - 1)
    q = st["Q"][at].float().view(S, N, H, G, D).permute(0, 2, 1, 3, 4) * (1.0 / math.sqrt(D))      # [S, H, N, G, D]
    # the prefix, once a group
    j = torch.arange(max(st["pre_hi"], 1), device=dev)
    K, V = _fetch(st, table[::M][:, j // p], (j % p).expand(g, -1))
    beyond = j >= pre.unsqueeze(1)                                                                  # [g, P]
    V = V.masked_fill(beyond.view(g, 1, -1, 1), 0.0)
    q1 = q.reshape(g, M, H, N * G, D).transpose(1, 2).reshape(g, H, M * N * G, D)
    z1 = (q1 @ K.transpose(2, 3)).masked_fill_(beyond.view(g, 1, 1, -1), float("-inf"))
    # every sequence's own tokens
    j = pre.repeat_interleave(M).unsqueeze(1) + torch.arange(st["own_hi"], device=dev)               # [S, L]
    K2, V2 = _fetch(st, table.gather(1, (j // p).clamp_max(table.shape[1] - 1)), j % p)
    pos = st["len"].long().unsqueeze(1) - n.unsqueeze(1) + i                                     # [S, N]
    seen = j.unsqueeze(1) <= torch.minimum(pos, st["len"].long().unsqueeze(1) - 1).unsqueeze(2)      # [S, N, L]
    z2 = (q.reshape(S, H, N * G, D) @ K2.transpose(2, 3)).view(S, H, N, G, -1)
    z2 = z2.masked_fill_(~seen.view(S, 1, N, 1, -1), float("-inf")).view(S, H, N * G, -1)
    V2 = V2.masked_fill((j >= st["len"].unsqueeze(1)).view(S, 1, -1, 1), 0.0)
    # both together
    top1 = z1.amax(-1).view(g, H, M, N * G).transpose(1, 2).reshape(S, H, N * G)
    m = torch.maximum(top1, z2.amax(-1))
    z1 = (z1 - m.view(g, M, H, N * G).transpose(1, 2).reshape(g, H, -1, 1)).exp_()
    z2 = (z2 - m.unsqueeze(-1)).exp_()
    back = lambda x: x.view(g, H, M, N * G, -1).transpose(1, 2).reshape(S, H, N * G, -1)  # noqa: E731
    l = back(z1.sum(-1, keepdim=True)) + z2.sum(-1, keepdim=True)
    o = (back(z1 @ V) + z2 @ V2) / l
    lse = m + l.squeeze(-1).log()
    real = i < n.unsqueeze(1)
    o = o.view(S, H, N, G, D).permute(0, 2, 1, 3, 4).reshape(S, N, H * G, D)
    lse = lse.view(S, H, N, G).permute(0, 2, 1, 3).reshape(S, N, H * G)
    return o[real].to(BF16), lse[real]


# ------------------------------------------------------------------ the framework's

def _own(st):
    c = st["case"]
    if c["op"] == "rotate":
        return st["rotary"].apply((st["Q"], st["K"]), st["pos"], inverse=c["inverse"])
    cache = st["cache"]
    if c["op"] == "append":
        Q = cache.write_rotary(st["rotary"], st["K"], st["V"], st["batch"], Q=st["Q"])
        return (Q, *cache.read(st["batch"]))
    if c["op"] == "update":
        st["pages"].update(st["parent"], st["keep"], st["room"])
        cache.copy(st["pages"])
        return st["table"], st["len"], st["refs"], st["k"], st["v"]
    if c["op"] == "compact":
        st["pages"].compact(out=(st["new_table"], st["new_refs"]))
        cache.copy(st["pages"])
        return st["new_table"], st["new_refs"], st["k"], st["v"]
    return cache.attention_shared(st["Q"], st["batch"], st["groups"])


def run(st):
    if own:
        return _own(st)
    return {"rotate": _plain_rotate, "append": _plain_append, "update": _plain_update, "compact": _plain_compact,
            "shared": _plain_shared}[st["case"]["op"]](st)


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """The outputs of ``run`` from the definition, in 64 bits (the page tables are whole numbers: None)."""
    st = prepare(case, seed)
    op, D = case["op"], case["dim"]
    if op == "rotate":
        return tuple(_complex_turn(case, x.double(), st["pos"].double()) for x in (st["Q"], st["K"]))
    if op == "append":
        new, total, _ = _lengths(case)
        pos = torch.cat([torch.arange(t - n, t, device="cuda", dtype=torch.float64) for n, t in zip(new, total)])
        held = []
        for x in (_complex_turn(case, st["K"].double(), pos), st["V"].double()):
            if case["fmt"] == "int8":
                step = (x.abs().amax(-1, keepdim=True) / 127).to(BF16).double().clamp_min(TINY)
                x = torch.clamp(torch.round(x / step), -127, 127) * step
            held.append(x)
        return (_complex_turn(case, st["Q"].double(), pos), *held)
    if op == "update":
        return (None, None, None, *_exact_update(st))
    if op == "compact":
        taken = [i for i, r in enumerate(st["refs"].tolist()) if r > 0]
        holes = sorted(set(range(len(taken))) - set(taken))
        arenas = [st["k"].double(), st["v"].double()]
        for a, b in zip([i for i in taken if i >= len(taken)], holes):
            for x in arenas:
                x[b] = x[a]
        return (None, None, *arenas)
    new, total, _ = _lengths(case)
    if 6 * D * case["heads"] * sum(n * t for n, t in zip(new, total)) > 1.5e13:
        return None
    p, group = case["page"], case["heads"] // case["kv_heads"]
    O = torch.empty(st["Q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["Q"].shape[:2], dtype=torch.float64, device="cuda")
    row0 = 0
    for b, (n, t) in enumerate(zip(new, total)):
        j = torch.arange(t, device="cuda")
        pages, rows = st["table"][b].long()[j // p], j % p
        K, V = (st[a][pages, :, rows].double() * (st[s][pages, :, rows].double()[..., None] if st[s] is not None else 1)
                for a, s in (("k", "ks"), ("v", "vs")))
        q = st["Q"][row0:row0 + n].double()
        hidden = j[None, :] > torch.arange(t - n, t, device="cuda")[:, None]
        z = torch.einsum("nhd,jhd->hnj", q, K.repeat_interleave(group, 1)) / math.sqrt(D)
        z = z.masked_fill(hidden, float("-inf"))
        l = torch.logsumexp(z, 2)
        O[row0:row0 + n] = torch.einsum("hnj,jhd->nhd", torch.exp(z - l[..., None]), V.repeat_interleave(group, 1))
        lse[row0:row0 + n] = l.T
        row0 += n
    return O, lse


def _complex_turn(case, x, pos):
    """Rotation as the product with exp(i angle)."""
    R, kind = case["rotary"], case["scaling"]
    f, length = [], 1.0
    for i in range(R // 2):
        w = math.exp(-2 * i / R * math.log(10000.0 * (SCALE ** (R / (R - 2)) if kind == "ntk" and R > 2 else 1.0)))
        turns = TRAINED * w / (2 * math.pi)
        if kind == "linear":
            w /= SCALE
        elif kind == "bands":
            part = min(1.0, max(0.0, (turns - 1) / 3))
            w = (1 - part) * w / SCALE + part * w
        elif kind == "yarn":
            ln = 2 * math.log(10000.0) / R
            lo = max(0, math.floor(math.log(TRAINED / (64 * math.pi)) / ln))
            hi = min(R - 1, math.ceil(math.log(TRAINED / (2 * math.pi)) / ln))
            part = min(1.0, max(0.0, (i - lo) / (hi - lo if hi > lo else 0.001)))
            w = part * w / SCALE + (1 - part) * w
            length = 1 + math.log(SCALE) / 10
        f.append(w)
    angle = pos[:, None] * torch.tensor(f, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full_like(angle, length), -angle if case.get("inverse") else angle)[:, None, :]
    r = x[..., :R].unflatten(-1, (2, R // 2) if case["layout"] == "half" else (R // 2, 2))
    pair = r.transpose(-1, -2) if case["layout"] == "half" else r
    pair = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
    out = x.clone()
    out[..., :R] = (pair.transpose(-1, -2) if case["layout"] == "half" else pair).flatten(-2)
    return out


def _exact_update(st):
    """The arenas after an update, slot by slot."""
    p, S = st["case"]["page"], st["case"]["slots"]
    table, held = st["table"].tolist(), st["len"].tolist()
    parent, keep, room = st["parent"].tolist(), st["keep"].tolist(), st["room"].tolist()
    kept = [min(keep[i], held[a]) if a >= 0 else 0 for i, a in enumerate(parent)]
    whole, asks = set(), {}
    for i, a in enumerate(parent):
        whole.update(table[a][:kept[i] // p] if a >= 0 else [])
        if kept[i] % p:
            asks.setdefault(table[a][kept[i] // p], []).append((a != i, i))
    owner = {x: min(who)[1] for x, who in asks.items() if x not in whole}
    free = (x for x in range(st["k"].shape[0]) if x not in whole and x not in owner)
    arenas = [st["k"].double(), st["v"].double()]
    moves = []
    for i in range(S):
        for q in range(kept[i] // p, -(-(kept[i] + room[i]) // p)):
            x = table[parent[i]][q] if q * p < kept[i] else -1
            if x < 0 or owner.get(x) != i:
                y = next(free)
                if x >= 0:
                    moves.append((x, y, kept[i] % p))
    for x, y, rows in moves:
        for t in arenas:
            t[y, :, :rows] = t[x, :, :rows]
    return arenas
