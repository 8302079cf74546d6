"""GPU tests of the paged key/value cache (write, read) and the attention over it against plain
64-bit forms (tests/_kv_reference.py): lengths of zero and one, odd sizes, strides, windows, rows
that see nothing, rows of the cache that hold garbage, long arenas, streams, graphs."""
import math

import pytest

import _kv_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
al = pytest.importorskip("adapter_linear_gb300")

INT8, BF16 = 1, 0


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    al.load_library()
    torch.cuda.set_device(0)


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def hard_rows(n, H, D, seed):
    """bf16 rows with what rounding and scaling can get wrong: ties, zeros, one loud value,
    subnormal and huge magnitudes, infinities and NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, H, D, generator=g, device="cuda")
    kind = torch.arange(n * H, device="cuda").view(n, H) % 11
    x = torch.where((kind == 1)[..., None], torch.zeros_like(x), x)
    x[..., 0] = torch.where(kind == 2, 300.0, x[..., 0])                      # one loud value
    half = torch.randint(-128, 129, x.shape, generator=g, device="cuda") / 128.0
    x = torch.where((kind == 3)[..., None], half, x)                          # amax 1: ties at x / s
    x[..., 1] = torch.where(kind == 3, 1.0, x[..., 1])
    m254 = torch.randint(-254, 255, x.shape, generator=g, device="cuda") / 128.0
    x = torch.where((kind == 4)[..., None], m254, x)                          # s a power of two
    x[..., 2] = torch.where(kind == 4, 254.0 / 128.0, x[..., 2])
    x = torch.where((kind == 5)[..., None], x * 2.0 ** -128, x)               # subnormal
    x = torch.where((kind == 6)[..., None], x.clamp(-3, 3) * 2.0 ** 126, x)   # near the largest
    x = torch.where((kind == 7)[..., None], x * 1e-3, x)
    x[..., D - 1] = torch.where(kind == 8, float("inf"), x[..., D - 1])
    x[..., 3] = torch.where(kind == 9, float("nan"), x[..., 3])
    x[..., D // 2] = torch.where(kind == 10, float("-inf"), x[..., D // 2])
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("fmt,H,D,page,lens,new", [
    (INT8, 8, 128, 16, [1, 17, 16, 400], [1, 5, 0, 203]),
    (INT8, 1, 64, 32, [33, 1, 90], [33, 1, 7]),
    (INT8, 3, 64, 256, [300, 2], [299, 2]),
    (BF16, 2, 128, 64, [64, 65, 0, 7], [64, 1, 0, 3]),
    (BF16, 5, 64, 128, [1000], [77]),
    (INT8, 8, 128, 16, [40 + i for i in range(67)], [1] * 67),
    (INT8, 2, 128, 16, [5, 0, 3], [9, 2, 3]),          # more rows than tokens: positions below zero
])
def test_write_and_read(fmt, H, D, page, lens, new):
    p = R.Paged(al, fmt, lens, new, H, D, page, seed=3)
    K, V = hard_rows(p.T, H, D, 5), hard_rows(p.T, H, D, 6)
    before = [t.clone() for t in (p.cache.k, p.cache.v, p.cache.k_scales, p.cache.v_scales) if t is not None]
    p.cache.write(K, V, p.batch)
    Kr, Vr = p.cache.read(p.batch)
    assert p.cache.check_errors() == al.LORA_OK
    want = [t.clone() for t in before]
    for i, x in enumerate((K, V)):
        got = (Kr, Vr)[i]
        for b, (n, L) in enumerate(zip(new, lens)):
            skip = max(0, n - L)                       # rows of positions below zero
            r0 = p.start[b]
            assert not got[r0:r0 + skip].any()
            rows = x[r0 + skip:r0 + n]
            pages, offs = p.where(b, torch.arange(L - n + skip, L, device="cuda"))
            if fmt == INT8:
                q, s = R.quantise(rows)
                want[i][pages, :, offs] = q.to(torch.int8)
                want[2 + i][pages, :, offs] = s.to(torch.bfloat16)
                back = R.bf16_of_f64(q * s[..., None])
            else:
                want[i][pages, :, offs] = rows
                back = rows
            nan = torch.isnan(back)
            assert torch.equal(torch.isnan(got[r0 + skip:r0 + n]), nan)
            assert torch.equal(got[r0 + skip:r0 + n][~nan], back[~nan])
    after = [t for t in (p.cache.k, p.cache.v, p.cache.k_scales, p.cache.v_scales) if t is not None]
    for a, w in zip(after, want):                      # codes and scales, and nothing else touched
        if a.dtype == torch.bfloat16:
            nan = torch.isnan(w)
            assert torch.equal(torch.isnan(a), nan) and torch.equal(a[~nan], w[~nan])
        else:
            assert torch.equal(a, w)


def test_strided_rows_and_padding():
    """K and V as slices of a fused projection's output; rows after the last sequence stay."""
    p = R.Paged(al, INT8, [20, 7], [13, 2], 2, 64, 16, seed=9)
    T = p.T + 5
    wide = torch.randn(T, 7 * 64, device="cuda").to(torch.bfloat16)
    K, V = wide[:, 64:192].unflatten(1, (2, 64)), wide[:, 256:384].unflatten(1, (2, 64))
    batch = al.KvBatch(p.table, p.batch.start, p.batch.kv_len, T, 13)
    p.cache.write(K, V, batch)
    out = torch.full((T, 5, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    p.cache.read(batch, K=out[:, 0:2], V=out[:, 3:5])
    for x, got in ((K, out[:, 0:2]), (V, out[:, 3:5])):
        q, s = R.quantise(x[:p.T])
        assert torch.equal(got[:p.T], R.bf16_of_f64(q * s[..., None]))
    assert (out[p.T:] == 3.0).all() and (out[:, 2] == 3.0).all()
    assert p.cache.check_errors() == al.LORA_OK


ATTENTION = [
    # fmt, Hq, H, D, page, lens, new, window
    (INT8, 32, 8, 128, 16, [1], [1], 0),
    (INT8, 32, 8, 128, 16, [2048], [1], 0),
    (BF16, 32, 8, 128, 32, [1, 2, 63, 64, 65, 127, 128, 129, 1000, 4097], [1] * 10, 0),
    (INT8, 8, 8, 64, 16, [5, 16, 17, 300], [1, 1, 1, 1], 0),
    (INT8, 14, 2, 64, 32, [700, 1, 350], [1, 1, 2], 0),
    (BF16, 16, 1, 128, 16, [333, 40], [1, 1], 0),
    (INT8, 24, 1, 64, 64, [100, 515], [1, 3], 0),           # 24 query heads on one kv head
    (INT8, 32, 8, 128, 16, [300, 1024, 77], [4, 5, 3], 0),
    (BF16, 12, 4, 64, 32, [500, 128, 33], [17, 128, 33], 0),
    (INT8, 8, 2, 128, 64, [600], [257], 0),
    (BF16, 8, 2, 128, 128, [1024], [1024], 0),
    (BF16, 2, 1, 64, 256, [900], [400], 0),
    (INT8, 4, 4, 128, 16, [2500, 10], [90, 10], 0),
    (INT8, 14, 2, 64, 32, [900, 40, 3, 0, 260], [300, 1, 3, 0, 1], 128),
    (BF16, 8, 8, 128, 16, [700, 300], [200, 1], 1),         # a window of one token
    (INT8, 8, 2, 128, 16, [700, 300], [65, 1], 50),
    (BF16, 8, 2, 64, 16, [3, 0, 20], [9, 4, 20], 0),        # rows that see nothing
    (INT8, 8, 2, 128, 16, [3, 0, 130], [200, 1, 130], 16),
    (INT8, 32, 8, 128, 16, [9 * i + 1 for i in range(70)], [1] * 70, 0),
    (INT8, 256, 1, 128, 32, [200, 64], [2, 1], 0),          # many heads on one kv head
]


@pytest.mark.parametrize("case", range(len(ATTENTION)))
def test_attention(case):
    fmt, Hq, H, D, page, lens, new, window = ATTENTION[case]
    p = R.Paged(al, fmt, lens, new, H, D, page, seed=case)
    g = torch.Generator(device="cuda").manual_seed(case)
    Q = torch.randn(p.T, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
    scale = 1.0 / math.sqrt(D)
    O, lse = p.cache.attention(Q, p.batch, window=window)
    assert p.cache.check_errors() == al.LORA_OK
    R.check_attention(O, lse, R.attention(Q, p, scale, window), str(ATTENTION[case]))
    O2, lse2 = p.cache.attention(Q, p.batch, window=window)
    assert same_bits(O, O2) and torch.equal(lse, lse2)      # the same call gives the same bits


@pytest.mark.parametrize("fmt", [INT8, BF16])
@pytest.mark.parametrize("max_new", [0, 1, 100000])
def test_a_wrong_bound_on_the_rows_changes_only_the_time(fmt, max_new):
    lens, new = [400, 200, 90, 1], [150, 1, 90, 1]
    p = R.Paged(al, fmt, lens, new, 2, 128, 16, seed=21)
    Q = torch.randn(p.T, 8, 128, device="cuda").to(torch.bfloat16)
    batch = al.KvBatch(p.table, p.batch.start, p.batch.kv_len, p.T, max_new)
    O, lse = p.cache.attention(Q, batch)
    assert p.cache.check_errors() == al.LORA_OK
    R.check_attention(O, lse, R.attention(Q, p, 1.0 / math.sqrt(128)), f"max_new {max_new}")


@pytest.mark.parametrize("new", [[1, 1, 1], [70, 1, 40]])
@pytest.mark.parametrize("std,scale", [(8.0, 0.5), (1e-3, 1.0), (1.0, -0.25), (1.0, 0.0), (30.0, 1.0)])
def test_scores_large_small_and_negative(new, std, scale):
    """Scores in the hundreds and thousands (one key takes all), tiny values, a negative and a
    zero scale."""
    p = R.Paged(al, INT8, [513, 40, 300], new, 2, 128, 16, seed=31, std=std)
    Q = torch.randn(p.T, 8, 128, device="cuda").to(torch.bfloat16)
    O, lse = p.cache.attention(Q, p.batch, scale=scale)
    R.check_attention(O, lse, R.attention(Q, p, scale), f"std {std} scale {scale}")


@pytest.mark.parametrize("new", [[1, 1], [60, 33]])
def test_a_non_finite_token_stays_with_the_rows_that_see_it(new):
    """int8: a token stored as NaN makes exactly the rows NaN that see it."""
    lens = [200, 150]
    p = R.Paged(al, INT8, lens, new, 2, 64, 16, seed=41)
    bad = [199, 140]                                    # the last token of 0; one inside 1's chunk
    for b in range(2):
        pg, r = p.where(b, torch.tensor([bad[b]], device="cuda"))
        p.cache.v_scales[pg, :, r] = float("nan")
        p.cache.k_scales[pg, :, r] = float("nan")
    Q = torch.randn(p.T, 4, 64, device="cuda").to(torch.bfloat16)
    O, lse = p.cache.attention(Q, p.batch)
    ref = R.attention(Q, p, 1.0 / 8.0)
    for b in range(2):
        for i in range(new[b]):
            t = p.start[b] + i
            sees = lens[b] - new[b] + i >= bad[b]
            assert bool(torch.isnan(O[t].float()).all()) == sees and bool(torch.isnan(lse[t]).all()) == sees
    ok = ~torch.isnan(lse[:, 0])
    R.check_attention(O[ok], lse[ok], tuple(x[ok] for x in ref), "rows before the bad token")


def test_attention_on_strided_tensors():
    p = R.Paged(al, BF16, [90, 300], [33, 1], 2, 64, 16, seed=51)
    wide = torch.randn(p.T, 12 * 64, device="cuda").to(torch.bfloat16)
    Q = wide[:, 64:64 * 7].unflatten(1, (6, 64))
    out = torch.full((p.T, 8, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    O, lse = p.cache.attention(Q, p.batch, O=out[:, 1:7])
    R.check_attention(O, lse, R.attention(Q, p, 1.0 / 8.0), "strided")
    assert (out[:, 0] == 5.0).all() and (out[:, 7] == 5.0).all()


@pytest.mark.parametrize("new", [1, 50])
def test_sequences_share_prefix_pages(new):
    """Two sequences whose tables name the same pages for their first 64 tokens."""
    p = R.Paged(al, INT8, [100, 64 + 30 + new], [new, new], 2, 128, 16, seed=61)
    p.table[1, :4] = p.table[0, :4]
    for i in range(2):
        p.values[1][i][:64] = p.values[0][i][:64]
    Q = torch.randn(p.T, 8, 128, device="cuda").to(torch.bfloat16)
    O, lse = p.cache.attention(Q, p.batch)
    R.check_attention(O, lse, R.attention(Q, p, 1.0 / math.sqrt(128)), "shared prefix")


@pytest.mark.parametrize("fmt,new", [(INT8, 1), (INT8, 40), (BF16, 1), (BF16, 40)])
def test_arenas_past_32_bit_offsets(fmt, new):
    """Pages whose byte and element offsets pass 2^32 (the last pages of a 5 G element arena)."""
    H, D, page = 8, 128, 64
    P = (5 << 30) // (H * D * page)
    k, v = (torch.empty((P, H, page, D), dtype=torch.int8 if fmt else torch.bfloat16, device="cuda")
            for _ in range(2))
    ks, vs = ((torch.empty((P, H, page), dtype=torch.bfloat16, device="cuda") for _ in range(2))
              if fmt else (None, None))
    lens = [100, 150]
    small = R.Paged(al, fmt, lens, [new, new], H, D, page, seed=71)
    table = small.table.clone()
    with al.KvCache(P, page, H, D, fmt, arenas=(k, v, ks, vs)) as cache:
        for b, L in enumerate(lens):
            for i in range(-(-L // page)):
                far = P - 1 - 5 * b - i
                src = int(small.table[b, i])
                k[far], v[far] = small.cache.k[src], small.cache.v[src]
                if fmt:
                    ks[far], vs[far] = small.cache.k_scales[src], small.cache.v_scales[src]
                table[b, i] = far
        Q = torch.randn(small.T, 32, D, device="cuda").to(torch.bfloat16)
        K, V = (torch.randn(small.T, H, D, device="cuda").to(torch.bfloat16) for _ in range(2))
        batch = al.KvBatch(table, small.batch.start, small.batch.kv_len, small.T, new)
        outs = []
        for c, bt in ((cache, batch), (small.cache, small.batch)):
            c.write(K, V, bt)
            outs.append((*c.read(bt), *c.attention(Q, bt)))
            assert c.check_errors() == al.LORA_OK
        for a, b in zip(*outs):
            assert torch.equal(a, b)


def test_streams_and_graph_replay():
    """Calls on a side stream; a captured step replayed with other lengths and inputs."""
    H, D, page, n = 2, 128, 16, 5
    P = 64
    cache = al.KvCache(P, page, H, D, INT8)
    table = torch.randperm(P, device="cuda").int()[:n * 12].view(n, 12).contiguous()
    start = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    kv_len = torch.zeros(n, dtype=torch.int32, device="cuda")
    K, V = (torch.zeros(n, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    Q = torch.zeros(n, 8, D, dtype=torch.bfloat16, device="cuda")
    batch = al.KvBatch(table, start, kv_len, n, 1)
    cache.reserve(n, 8, n)
    O = torch.empty_like(Q)
    lse = torch.empty(n, 8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kv_len += 1
        cache.write(K, V, batch)
        cache.attention(Q, batch, O=O, lse=lse)
        kv_len -= 1
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv_len += 1
        cache.write(K, V, batch)
        cache.attention(Q, batch, O=O, lse=lse)
    g = torch.Generator(device="cuda").manual_seed(81)
    hist = [[], []]
    for step in range(40):
        for x in (K, V, Q):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        graph.replay()
        for h, x in zip(hist, (K, V)):
            q, s = R.quantise(x)
            h.append(q * s[..., None])
    torch.cuda.synchronize()
    ref = R.Paged.__new__(R.Paged)
    ref.H, ref.new, ref.lens, ref.start = H, [1] * n, [40] * n, list(range(n + 1))
    ref.values = [[torch.stack([x[b] for x in h]) for h in hist] for b in range(n)]
    R.check_attention(O, lse, R.attention(Q, ref, 1.0 / math.sqrt(D)), "graph")
    assert cache.check_errors() == al.LORA_OK
    cache.close()


def test_two_streams_share_a_cache():
    """Attention calls on two streams at once (they share scratch) give what each gives alone."""
    p = R.Paged(al, INT8, [3000, 2500], [1, 1], 2, 128, 16, seed=91)
    q = R.Paged(al, INT8, [3000, 2500], [1, 1], 2, 128, 16, seed=91)
    Qs = [torch.randn(2, 8, 128, device="cuda").to(torch.bfloat16) for _ in range(2)]
    alone = [q.cache.attention(x, q.batch) for x in Qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(p.cache.attention(Qs[i], p.batch))
    torch.cuda.synchronize()
    for i in range(2):
        for O, lse in got[i]:
            assert same_bits(O, alone[i][0]) and torch.equal(lse, alone[i][1])


@pytest.mark.parametrize("new", [[1, 1, 1], [40, 3, 1]])
@pytest.mark.parametrize("bad", ["page_high", "page_negative", "kv_len"])
def test_bad_tables_are_reported_and_not_followed(new, bad):
    lens = [100, 90, 80]
    p = R.Paged(al, INT8, lens, new, 2, 128, 16, seed=101)
    table, kv_len = p.table.clone(), p.batch.kv_len.clone()
    if bad == "kv_len":
        kv_len[1] = table.shape[1] * 16 + 1
    else:
        table[1, 5] = 1 << 30 if bad == "page_high" else -1
    batch = al.KvBatch(table, p.batch.start, kv_len, p.T, max(new))
    Q = torch.randn(p.T, 8, 128, device="cuda").to(torch.bfloat16)
    K = torch.randn(p.T, 2, 128, device="cuda").to(torch.bfloat16)
    ref = R.attention(Q, p, 1.0 / math.sqrt(128))
    O, lse = p.cache.attention(Q, batch)
    assert p.cache.check_errors() == al.LORA_ERR_RANGE
    assert p.cache.check_errors() == al.LORA_OK                 # read and cleared
    keep = torch.tensor([b != 1 for b, n in enumerate(new) for _ in range(n)], device="cuda")
    R.check_attention(O[keep], lse[keep], tuple(x[keep] for x in ref), bad)
    p.cache.read(batch)
    assert p.cache.check_errors() == al.LORA_ERR_RANGE
    p.cache.write(K, K, batch)
    assert p.cache.check_errors() == al.LORA_ERR_RANGE


def test_bad_starts_are_reported():
    p = R.Paged(al, INT8, [100, 90], [3, 4], 2, 128, 16, seed=111)
    start = torch.tensor([0, 3, 8], dtype=torch.int32, device="cuda")     # one past T = 7
    batch = al.KvBatch(p.table, start, p.batch.kv_len, p.T, 5)
    Q = torch.randn(p.T, 8, 128, device="cuda").to(torch.bfloat16)
    ref = R.attention(Q, p, 1.0 / math.sqrt(128))
    O, lse = p.cache.attention(Q, batch)
    assert p.cache.check_errors() == al.LORA_ERR_RANGE
    R.check_attention(O[:3], lse[:3], tuple(x[:3] for x in ref), "start")


def test_refusals():
    p = R.Paged(al, INT8, [20], [2], 2, 64, 16, seed=121)
    bf = torch.bfloat16
    Q = torch.zeros(2, 4, 64, dtype=bf, device="cuda")

    def refused(status, call):
        with pytest.raises(al.LoraError) as e:
            call()
        assert e.value.status == status

    refused(al.LORA_ERR_SHAPE, lambda: p.cache.attention(Q[:, :3], p.batch))          # 3 heads over 2
    refused(al.LORA_ERR_SHAPE, lambda: p.cache.attention(Q[:1], p.batch))             # rows
    refused(al.LORA_ERR_SHAPE, lambda: p.cache.attention(Q.float(), p.batch))
    refused(al.LORA_ERR_ARG, lambda: p.cache.attention(Q, p.batch, window=-1))
    refused(al.LORA_ERR_ARG, lambda: p.cache.attention(Q.transpose(0, 1).contiguous().transpose(0, 1), p.batch))
    wide = torch.zeros(2, 4 * 64 + 4, dtype=bf, device="cuda")
    refused(al.LORA_ERR_ARG, lambda: p.cache.attention(wide[:, :256].unflatten(1, (4, 64)), p.batch))  # stride
    wide = torch.zeros(2, 5 * 64, dtype=bf, device="cuda")
    refused(al.LORA_ERR_ARG, lambda: p.cache.attention(wide[:, 4:260].unflatten(1, (4, 64)), p.batch))  # alignment
    K = torch.zeros(2, 2, 64, dtype=bf, device="cuda")
    refused(al.LORA_ERR_SHAPE, lambda: p.cache.write(K, K[:, :1], p.batch))
    refused(al.LORA_ERR_SHAPE, lambda: p.cache.reserve(4, 3, 1))
    refused(al.LORA_ERR_SHAPE, lambda: al.KvCache(4, 48, 2, 64))
    refused(al.LORA_ERR_SHAPE, lambda: al.KvCache(4, 16, 2, 96))
    refused(al.LORA_ERR_SHAPE, lambda: al.KvBatch(p.table, p.batch.start[:1], p.batch.kv_len, 2, 1))
    refused(al.LORA_ERR_ARG, lambda: al.KvBatch(p.table.long(), p.batch.start, p.batch.kv_len, 2, 1))
    empty = al.KvBatch(p.table[:0], p.batch.start[:1], p.batch.kv_len[:0], 0, 0)      # nothing to do
    O, lse = p.cache.attention(Q[:0], empty)
    assert O.shape[0] == 0 and p.cache.check_errors() == al.LORA_OK
