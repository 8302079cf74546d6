"""GPU tests of the attention of groups that share a prefix's pages, against the plain 64-bit form
(tests/_kv_reference.py) and against the attention of every sequence by itself."""
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


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Shared(R.Paged):
    """groups: (prefix, [(tokens behind it, new ones of them), ...]); the members' whole pages of the prefix are
    the first member's, what they had in their place is made NaN. alone: sequences behind the groups."""

    def __init__(self, fmt, H, D, page, groups, alone=(), seed=0, std=1.0):
        lens = [pre + own for pre, members in groups for own, _ in members] + [own for own, _ in alone]
        new = [n for _, members in groups for _, n in members] + [n for _, n in alone]
        super().__init__(al, fmt, lens, new, H, D, page, seed=seed, std=std)
        first = 0
        self.seq_start, self.prefix = [0], []
        for pre, members in groups:
            whole = pre // page
            for b in range(first + 1, first + len(members)):
                dead = self.table[b, :whole].long()
                for x in (self.cache.k_scales, self.cache.v_scales) if fmt == INT8 else (self.cache.k, self.cache.v):
                    x[dead] = float("nan")
                self.table[b, :whole] = self.table[first, :whole]
                for mine, theirs in zip(self.values[b], self.values[first]):
                    mine[:whole * page] = theirs[:whole * page]
            first += len(members)
            self.seq_start.append(first)
            self.prefix.append(pre)
        self.groups = al.KvGroups(ints(self.seq_start), ints(self.prefix),
                                  max(self.start[b] - self.start[a] for a, b in zip(self.seq_start, self.seq_start[1:])))

    def queries(self, Hq, seed=11):
        g = torch.Generator(device="cuda").manual_seed(seed)
        return torch.randn(self.T, Hq, self.D, generator=g, device="cuda").to(torch.bfloat16)


CASES = [
    # fmt, Hq, H, D, page, groups, alone
    (INT8, 8, 2, 128, 16, [(64, [(1, 1), (5, 1)])], []),                                 # 8 rows: the short-chunk kernel
    (INT8, 32, 8, 128, 16, [(1000, [(1 + 7 * i, 1) for i in range(8)])], []),
    (BF16, 4, 4, 64, 32, [(333, [(3, 1), (40, 1), (1, 1)])], [(70, 1)]),
    (BF16, 32, 8, 128, 32, [(500, [(i + 1, 1) for i in range(16)]), (130, [(1, 1), (200, 1)])], [(5, 1), (90, 1)]),
    (INT8, 14, 2, 64, 16, [(4000, [(17 * i + 1, 1) for i in range(40)])], []),
    (INT8, 16, 1, 128, 64, [(2000, [(30, 3), (9, 9), (100, 5)]), (64, [(2, 2), (2, 1)])], [(33, 20)]),
    (BF16, 8, 2, 128, 16, [(700, [(300, 200), (65, 65), (1, 1)])], []),                  # long chunks
    (INT8, 8, 2, 64, 128, [(260, [(500, 257), (3, 3)]), (128, [(1, 1)] * 5)], [(400, 300)]),
    (BF16, 6, 2, 64, 16, [(0, [(30, 1), (20, 1)]), (15, [(30, 1), (20, 1)]), (16, [(1, 1), (1, 1)])], []),
    (INT8, 4, 1, 128, 16, [(100, [(50, 1)]), (48, [(9, 1), (9, 0), (9, 2)])], [(12, 0), (20, 1)]),  # one sequence; no rows
    (INT8, 4, 1, 128, 16, [(160, [(9, 0), (9, 1), (20, 1)])], []),                       # the first one has no rows
    (BF16, 24, 3, 128, 256, [(5000, [(1, 1)] * 30)], []),
    (INT8, 256, 1, 128, 32, [(300, [(2, 2), (1, 1)])], []),                              # many heads on one kv head
    (BF16, 8, 8, 64, 16, [(16 * i + 5, [(3, 1)] * (i % 4 + 1)) for i in range(70)], []),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("scale", [None, -0.31])
def test_against_the_definition(case, scale):
    fmt, Hq, H, D, page, groups, alone = CASES[case]
    p = Shared(fmt, H, D, page, groups, alone, seed=case)
    Q = p.queries(Hq)
    O, lse = p.cache.attention_shared(Q, p.batch, p.groups, scale=scale)
    assert p.cache.check_errors() == al.LORA_OK
    R.check_attention(O, lse, R.attention(Q, p, scale or D ** -0.5), f"case {case}")
    again, lse2 = p.cache.attention_shared(Q, p.batch, p.groups, scale=scale)
    assert torch.equal(O, again) and torch.equal(lse, lse2)


def test_prefixes_that_are_cut():
    """A prefix that reaches into a sequence's new tokens is shared as far as they begin; one below zero and one
    beyond everything are not taken at their word; more rows than tokens: nothing is shared."""
    p = Shared(INT8, 2, 128, 16, [(200, [(40, 1), (3, 3), (17, 10)])], [(2, 5)], seed=4)
    Q = p.queries(8)
    want = R.attention(Q, p, 0.1)
    for prefix, starts in ((200, [0, 3]), (203, [0, 3]), (2 ** 31 - 1, [0, 3]), (-5, [0, 3]), (150, [1, 3]), (0, [0, 4])):
        if prefix > 200:
            # all of their tokens may be named: what is shared ends where the first new token is, 200
            assert min(L - n for L, n in zip(p.lens[:3], p.new[:3])) == 200
        got = p.cache.attention_shared(Q, p.batch, al.KvGroups(ints(starts), ints([prefix]), p.T), scale=0.1)
        assert p.cache.check_errors() == al.LORA_OK
        R.check_attention(*got, want, f"prefix {prefix}")
    # the group ends at the sequence of 2 tokens and 5 rows
    got = p.cache.attention_shared(Q, p.batch, al.KvGroups(ints([0, 4]), ints([100]), p.T), scale=0.1)
    R.check_attention(*got, want, "a sequence of more rows than tokens")


@pytest.mark.parametrize("fmt", [INT8, BF16])
@pytest.mark.parametrize("members", [2, 30])
@pytest.mark.parametrize("loud", ["prefix", "own"])
def test_one_part_holds_all_the_weight(fmt, members, loud):
    """Scores that differ by hundreds: the other part's weight is 0 or next to it."""
    p = Shared(fmt, 1, 128, 16, [(96, [(20 + i, 1) for i in range(members)])], seed=2)
    for b, L in enumerate(p.lens):
        lo, hi = (0, 96) if loud == "prefix" else (96, L)
        pages, rows = p.where(b, torch.arange(lo, hi, device="cuda"))
        if fmt == INT8:
            p.cache.k_scales[pages, :, rows] = (p.cache.k_scales[pages, :, rows] * (16 if b == 0 or loud == "own" else 1))
        elif b == 0 or loud == "own":
            p.cache.k[pages, :, rows] = p.cache.k[pages, :, rows] * 16
        p.values[b][0][lo:hi] *= 16
    Q = p.queries(4)
    O, lse = p.cache.attention_shared(Q, p.batch, p.groups, scale=1.0)
    R.check_attention(O, lse, R.attention(Q, p, 1.0), loud)


@pytest.mark.parametrize("members,n", [(2, 1), (12, 1), (3, 40)])
@pytest.mark.parametrize("bad", [(float("inf"),), (float("nan"),), (float("inf"), float("-inf"))])
def test_infinities_of_the_prefix(members, n, bad):
    """V of a prefix's token reaches every row of the group, and no other group's, as in the attention of every
    sequence by itself; so does one of the own tokens, which earlier rows do not see."""
    p = Shared(BF16, 2, 64, 16, [(80, [(n + i, n) for i in range(members)]), (64, [(n, n)] * members)], seed=6)
    for i, x in enumerate(bad):
        pages, rows = p.where(0, torch.tensor([7 + 30 * i], device="cuda"))
        p.cache.v[pages, 1, rows, 5] = x
        p.cache.v[pages, 0, rows, 63 - i] = x
    pages, rows = p.where(members - 1, torch.tensor([p.lens[members - 1] - 1], device="cuda"))
    p.cache.v[pages, 0, rows, 20] = bad[0]
    Q = p.queries(4)
    O, lse = p.cache.attention_shared(Q, p.batch, p.groups)
    want, lse2 = p.cache.attention(Q, p.batch)
    assert not torch.isfinite(want).all() and torch.isfinite(want[p.start[members]:]).all()
    for f in (torch.isnan, torch.isposinf, torch.isneginf):
        assert torch.equal(f(O), f(want))
    good = torch.isfinite(want)
    # the same sums in another order: each output rounded once, its weights to 2^-8 at most
    assert ((O[good].float() - want[good].float()).abs() <= 2.0 ** -6).all()
    assert ((lse - lse2).abs() <= 1e-4).all()


@pytest.mark.parametrize("bad", [(float("inf"),), (float("nan"),), (float("inf"), float("-inf"))])
@pytest.mark.parametrize("spread", [1.0, 30.0])
def test_infinities_of_a_prefix_that_many_short_chunks_share(bad, spread):
    """There every weight has two parts, the second zero or negative as often as not; with scores far apart most
    weights are 0."""
    p = Shared(BF16, 2, 64, 16, [(400, [(1 + i, 1) for i in range(40)]), (64, [(1, 1)] * 30)], seed=6)
    for i, x in enumerate(bad):
        pages, rows = p.where(0, torch.tensor([7 + 300 * i], device="cuda"))
        p.cache.v[pages, 1, rows, 5] = x
        p.cache.v[pages, 0, rows, 63 - i] = x
    Q = p.queries(4)
    O, lse = p.cache.attention_shared(Q, p.batch, p.groups, scale=0.125 * spread)
    want, _ = p.cache.attention(Q, p.batch, scale=0.125 * spread)
    assert not torch.isfinite(want[:40]).all() and torch.isfinite(want[40:]).all()
    for f in (torch.isnan, torch.isposinf, torch.isneginf):
        assert torch.equal(f(O), f(want))
    # the values beside them (whose V the reference has): a rounding of the output, 2^-8 of it, of each weight, 2^-16, and
    # scores off by dz, as in check_attention
    ref, lse64, A, S = R.attention(Q, p, 0.125 * spread)
    dz = 2.0 ** -17 * S + 2.0 ** -20
    bound = A * (2.0 ** -8 + 2.0 ** -16 + 2 * dz[..., None]) + 2.0 ** -100
    good = torch.isfinite(want)
    assert ((O.double() - ref).abs()[good] <= bound[good]).all()
    assert ((lse.double() - lse64).abs() <= dz + 2.0 ** -20 * (1 + lse64.abs())).all()


def test_queries_that_are_not_finite_reach_their_rows_only():
    p = Shared(INT8, 2, 128, 16, [(160, [(9, 1)] * 9)], seed=6)
    Q = p.queries(4)
    clean, _ = p.cache.attention_shared(Q, p.batch, p.groups)
    Q[4, 1, 3] = float("nan")
    O, lse = p.cache.attention_shared(Q, p.batch, p.groups)
    hit = torch.zeros(9, 4, dtype=torch.bool, device="cuda")
    hit[4, 1] = True
    assert torch.isnan(O[hit]).all() and torch.isnan(lse[hit]).all() and torch.equal(O[~hit], clean[~hit])


def test_rows_behind_the_last_sequence_and_strides():
    p = Shared(BF16, 2, 64, 16, [(100, [(9, 2), (30, 1)])], [(40, 1)], seed=3)
    T = p.T + 3
    wide = torch.randn(T, 9, 64, device="cuda").to(torch.bfloat16)
    Q, out = wide[:, 2:8], torch.full((T, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, 6), 7.0, device="cuda")
    batch = al.KvBatch(p.table, p.batch.start, p.batch.kv_len, T, 2)
    p.cache.attention_shared(Q, batch, p.groups, O=out[:, 1:7], lse=lse)
    R.check_attention(out[:p.T, 1:7], lse[:p.T], R.attention(Q[:p.T], p, 64 ** -0.5))
    assert (out[p.T:] == 7).all() and (out[:, 0] == 7).all() and (out[:, 7] == 7).all() and (lse[p.T:] == 7).all()


def test_a_captured_step_serves_later_lengths_and_prefixes():
    p = Shared(INT8, 2, 64, 16, [(160, [(40, 1)] * 8), (320, [(40, 1)] * 4)], seed=8)
    Q = p.queries(8)
    p.cache.reserve_shared(p.T, 8, 12)
    lens, prefix = ints(p.lens), ints(p.prefix)
    batch = al.KvBatch(p.table, p.batch.start, lens, p.T, 1)
    groups = al.KvGroups(ints(p.seq_start), prefix, 8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O, lse = p.cache.attention_shared(Q, batch, groups)
    for drop, pre in ((0, [160, 320]), (25, [96, 0]), (39, [160, 17])):
        lens.copy_(ints([x - drop for x in p.lens]))
        prefix.copy_(ints(pre))
        graph.replay()
        torch.cuda.synchronize()
        want, lse2 = p.cache.attention(Q, batch)
        assert ((O.float() - want.float()).abs() <= 2.0 ** -6).all() and ((lse - lse2).abs() <= 1e-4).all()
    assert p.cache.check_errors() == al.LORA_OK


def test_scratch_that_grows_leaves_captured_calls_theirs():
    p = Shared(BF16, 1, 64, 16, [(64, [(9, 1)] * 8)], seed=8)
    Q = p.queries(4)
    want, _ = p.cache.attention_shared(Q, p.batch, p.groups)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O, _ = p.cache.attention_shared(Q, p.batch, p.groups)
    p.cache.reserve_shared(50000, 4, 400)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(O, want)


def test_a_reservation_takes_what_its_size_needs():
    """And not twice what an earlier one took; a call of that size then takes nothing."""
    p = Shared(BF16, 1, 64, 16, [(64, [(9, 1)] * 8)], seed=8)

    def taken(call):
        torch.cuda.synchronize()
        before = torch.cuda.mem_get_info()[0]
        call()
        torch.cuda.synchronize()
        return before - torch.cuda.mem_get_info()[0]

    Q = p.queries(4)
    p.cache.attention_shared(Q, p.batch, p.groups)                 # (its kernels are loaded)
    taken(lambda: p.cache.reserve_shared(10, 4, 8))                # (and lora_kv_reserve's 20 MB)
    for tokens in (200000, 230000, 240000):
        # O, lse and a place of 8 bytes a row and head; pieces of 256 and 48 rows an SM twice; whole 2 MB from the driver
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        need = tokens * 4 * (64 + 3) * 4 + 2 * sms * (256 + 48) * (64 + 2) * 4
        assert need <= taken(lambda: p.cache.reserve_shared(tokens, 4, 8)) <= need + 8e6
    assert taken(lambda: p.cache.reserve_shared(240000, 4, 8)) == 0
    O, lse = torch.empty_like(Q), torch.empty(p.T, 4, device="cuda")
    assert taken(lambda: p.cache.attention_shared(Q, p.batch, p.groups, O=O, lse=lse)) == 0
    R.check_attention(O, lse, R.attention(Q, p, 0.125))


def test_short_chunks_behind_a_wide_prefix_take_no_other_scratch():
    """The tcgen05 kernel leaves a prefix's pieces in the shared scratch, not in the 40 MB of its own."""
    taken = []
    for cache in range(2):                                         # (the first call's kernels are loaded)
        p = Shared(INT8, 1, 128, 16, [(2000, [(9, 1)] * 40)], seed=8)
        Q = p.queries(4)
        O, lse = torch.empty_like(Q), torch.empty(p.T, 4, device="cuda")
        want = R.attention(Q, p, 128 ** -0.5)
        torch.cuda.synchronize()
        before = torch.cuda.mem_get_info()[0]
        p.cache.attention_shared(Q, p.batch, p.groups, O=O, lse=lse)
        torch.cuda.synchronize()
        taken.append(before - torch.cuda.mem_get_info()[0])
        R.check_attention(O, lse, want)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert taken[1] <= 2 * sms * (256 + 48) * (128 + 2) * 4 + 8e6


@pytest.mark.parametrize("fmt", [INT8, BF16])
@pytest.mark.parametrize("groups", [
    [(3000, [(9, 1), (2000, 1)])],                                 # the short-chunk kernel, twice
    [(3000, [(40 + i, 1) for i in range(30)]), (500, [(9, 2)] * 9)],  # the tcgen05 kernel, its pieces read behind it
    [(3000, [(90, 70), (300, 200), (5, 1)])],                      # its pieces joined, long chunks
])
def test_the_cache_works_again_after_a_timeout(groups, fmt):
    """Which a hook stands in for: it leaves arrivals of pieces that no call waits for any more, and numbers in the
    scratch that name no CTA and no row."""
    p = Shared(fmt, 2, 128, 16, groups, seed=8)
    Q = p.queries(8)
    want = R.attention(Q, p, 128 ** -0.5)
    first = p.cache.attention_shared(Q, p.batch, p.groups)
    R.check_attention(*first, want)
    p.cache.selftest_timeout()
    assert p.cache.check_errors() == al.LORA_ERR_TIMEOUT and p.cache.check_errors() == al.LORA_OK
    for _ in range(3):
        O, lse = torch.full_like(Q, float("nan")), torch.full((p.T, 8), float("nan"), device="cuda")
        p.cache.attention_shared(Q, p.batch, p.groups, O=O, lse=lse)
        assert torch.equal(O, first[0]) and torch.equal(lse, first[1])
    assert p.cache.check_errors() == al.LORA_OK


def test_calls_on_two_streams():
    p = Shared(INT8, 8, 128, 16, [(3000, [(40 + i, 1) for i in range(64)])], seed=8)
    a, b = p.queries(32, 1), p.queries(32, 2)
    want = [p.cache.attention_shared(q, p.batch, p.groups)[0] for q in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [p.cache.attention_shared((a, b)[i % 2], p.batch, p.groups, stream=streams[i % 2])[0] for i in range(8)]
    torch.cuda.synchronize()
    for i, x in enumerate(got):
        assert torch.equal(x, want[i % 2])


def test_bad_groups_share_nothing_and_are_reported():
    p = Shared(INT8, 2, 64, 16, [(64, [(9, 1), (20, 1)]), (32, [(5, 1), (6, 1), (7, 1)])], seed=1)
    Q = p.queries(4)
    want = R.attention(Q, p, 0.125)
    for starts in ([0, 2, 6], [-1, 2, 5], [2, 0, 5], [0, 6, 5], [0, 2 ** 31 - 1, 5]):
        got = p.cache.attention_shared(Q, p.batch, al.KvGroups(ints(starts), ints([64, 32]), 3), scale=0.125)
        assert p.cache.check_errors() == al.LORA_ERR_RANGE
        R.check_attention(*got, want, str(starts))
    assert p.cache.check_errors() == al.LORA_OK
    # a bad length: its group is not shared, the other one is as it was
    lens = ints(p.lens)
    lens[1] = 10 ** 6
    batch = al.KvBatch(p.table, p.batch.start, lens, p.T, 1)
    O, lse = p.cache.attention_shared(Q, batch, p.groups, scale=0.125)
    assert p.cache.check_errors() == al.LORA_ERR_RANGE
    keep = [0, 2, 3, 4]
    R.check_attention(O[keep], lse[keep], [x[keep] for x in want])
    # a bad page of the prefix
    table = p.table.clone()
    table[2, 1] = -4
    batch = al.KvBatch(table, p.batch.start, p.batch.kv_len, p.T, 1)
    O, lse = p.cache.attention_shared(Q, batch, p.groups, scale=0.125)
    assert p.cache.check_errors() == al.LORA_ERR_RANGE
    R.check_attention(O[:2], lse[:2], [x[:2] for x in want])


@pytest.mark.parametrize("start", [-1, 0, 4, 10 ** 9])
def test_bad_starts_are_reported_and_not_followed(start):
    p = Shared(INT8, 2, 64, 16, [(64, [(9, 1), (20, 1)]), (32, [(5, 1), (6, 1), (7, 1)])], seed=1)
    Q = p.queries(4)
    want = R.attention(Q, p, 0.125)
    starts = p.batch.start.clone()
    starts[2] = start   # of sequences 1 and 2: one of them, or both, have none of the rows
    batch = al.KvBatch(p.table, starts, p.batch.kv_len, p.T, 1)
    O, lse = p.cache.attention_shared(Q, batch, p.groups, scale=0.125)
    assert p.cache.check_errors() == al.LORA_ERR_RANGE
    keep = {0: [3, 4], 4: [0, 4]}.get(start, [0, 3, 4])   # (rows that no other sequence has, too)
    R.check_attention(O[keep], lse[keep], [x[keep] for x in want])


@pytest.mark.parametrize("heads", [4, 8])   # the last group's rows: a short chunk's, or the tcgen05 kernel's
def test_more_groups_and_sequences_than_a_block_has_threads(heads):
    groups = [(16 * (1 + i % 3), [(1 + i % 5, 1), (2, 1)]) for i in range(1100)] + [(400, [(3 + i, 1) for i in range(5)])]
    p = Shared(BF16, 1, 64, 16, groups, [(20, 1)], seed=2)
    Q = p.queries(heads)
    O, lse = p.cache.attention_shared(Q, p.batch, p.groups)
    assert p.cache.check_errors() == al.LORA_OK
    R.check_attention(O, lse, R.attention(Q, p, 0.125))


def test_no_groups_is_the_plain_attention():
    p = Shared(INT8, 2, 64, 16, [(64, [(9, 1), (20, 1)])], seed=1)
    Q = p.queries(4)
    for none in (al.KvGroups(ints([0]), ints([]), 0), None):
        for a, b in zip(p.cache.attention_shared(Q, p.batch, none), p.cache.attention(Q, p.batch)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("bound", [0, 1, 10 ** 9])
def test_a_wrong_bound_on_a_groups_rows_costs_time_only(bound):
    p = Shared(INT8, 2, 64, 16, [(64, [(9, 1)] * 20), (32, [(40, 30), (6, 1)])], [(90, 3)], seed=1)
    Q = p.queries(8)
    groups = al.KvGroups(ints(p.seq_start), ints(p.prefix), bound)
    for max_new in (0, 1, 30, 10 ** 6):
        batch = al.KvBatch(p.table, p.batch.start, p.batch.kv_len, p.T, max_new)
        R.check_attention(*p.cache.attention_shared(Q, batch, groups), R.attention(Q, p, 0.125), f"{bound} {max_new}")


def test_refusals():
    p = Shared(INT8, 2, 64, 16, [(64, [(9, 1), (20, 1)])], seed=1)
    Q = p.queries(4)

    def refused(status, call):
        with pytest.raises(al.LoraError) as e:
            call()
        assert e.value.status == status

    refused(al.LORA_ERR_SHAPE, lambda: al.KvGroups(ints([0, 1]), ints([1, 2]), 1))
    refused(al.LORA_ERR_ARG, lambda: al.KvGroups(ints([0, 1]).long(), ints([1]), 1))
    refused(al.LORA_ERR_ARG, lambda: al.KvGroups(torch.zeros(2, dtype=torch.int32), ints([1]), 1))
    refused(al.LORA_ERR_ARG, lambda: p.cache.attention_shared(Q, p.batch, al.KvGroups(ints([0, 1, 1, 2]), ints([1] * 3), 1)))
    refused(al.LORA_ERR_ARG, lambda: p.cache.attention_shared(Q, p.batch, al.KvGroups(ints([0, 1]), ints([1]), -1)))
    refused(al.LORA_ERR_SHAPE, lambda: p.cache.attention_shared(p.queries(3), p.batch, p.groups))
    refused(al.LORA_ERR_SHAPE, lambda: p.cache.attention_shared(Q[:1], p.batch, p.groups))
    refused(al.LORA_ERR_SHAPE, lambda: p.cache.reserve_shared(5, 3, 1))
    refused(al.LORA_ERR_ARG, lambda: p.cache.reserve_shared(-1, 4, 1))
    refused(al.LORA_ERR_ARG, lambda: p.cache.reserve_shared(2 ** 30, 1024, 1))
