"""GPU tests of the page tables (update, compaction, copies of pages) against a plain model of lists."""
import random

import pytest

from _kv_pages_reference import Tables, apply_moves

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
    return None if values is None else torch.tensor(values, dtype=torch.int32, device="cuda")


class Pair:
    """The library's tables and caches beside the model and copies of the arenas."""

    def __init__(self, P, page, S, W, caches=((INT8, 2, 64),), seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.model, self.pages = Tables(P, page, S, W), al.KvPages(P, page, S, W)
        self.caches, self.want = [], []
        for fmt, H, D in caches:
            shape = (P, H, page, D)
            if fmt == INT8:
                arenas = [torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8) for _ in "kv"]
                arenas += [torch.randn(shape[:3], generator=g, device="cuda").to(torch.bfloat16) for _ in "kv"]
            else:
                arenas = [torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv"] + [None] * 2
            self.caches.append(al.KvCache(P, page, H, D, fmt, arenas=tuple(arenas)))
            self.want.append([a.clone() for a in arenas if a is not None])

    def arenas(self, c):
        return [t for t in (c.k, c.v, c.k_scales, c.v_scales) if t is not None]

    def copied(self, moves):
        for c, want in zip(self.caches, self.want):
            c.copy(self.pages)
            apply_moves(want, moves if isinstance(moves, list) else [])

    def update(self, parent=None, keep=None, room=None):
        moves = self.model.update(parent, keep, room)
        self.pages.update(ints(parent), ints(keep), ints(room))
        self.copied(moves)
        want = {"oom": al.LORA_ERR_OOM, "range": al.LORA_ERR_RANGE}.get(moves if isinstance(moves, str) else "", al.LORA_OK)
        assert self.pages.check_errors() == want
        self.check()
        return moves

    def compact(self):
        moves = self.model.compact()
        self.pages.compact()
        self.copied(moves)
        assert self.pages.check_errors() == al.LORA_OK
        self.check()
        return moves

    def check(self):
        assert torch.equal(self.pages.table.cpu(), torch.tensor(self.model.table, dtype=torch.int32))
        assert self.pages.kv_len.tolist() == self.model.len
        refs = self.model.refs()
        assert self.pages.refs.tolist() == refs
        assert self.pages.used() == sum(r > 0 for r in refs)
        for c, want in zip(self.caches, self.want):
            assert c.check_errors() == al.LORA_OK
            for a, w in zip(self.arenas(c), want):
                assert torch.equal(a.view(torch.uint8), w.view(torch.uint8))


def test_one_of_everything():
    t = Pair(40, 16, 6, 10, caches=((INT8, 2, 64), (BF16, 3, 128)))
    assert t.update() == []                                        # nothing from nothing
    t.update(room=[40, 0, 16, 1, 0, 0])
    t.update(parent=[0, 0, 2, 3, 2, 0], room=[1, 2, 0, 0, 1, 17])  # forks: 0 -> 1, 5 (inside a page), 2 -> 4 (at its end)
    assert max(t.pages.refs.tolist()) == 3
    t.update(parent=[5, 4, 3, 2, 1, 0])                            # all change places, nothing is copied
    t.update(keep=[0, 5, 100, 3, 20, 33])                          # trimmed
    t.update(parent=[-1, 1, -1, 4, 4, 5], keep=[9, 3, 9, 30, 16, 1], room=[20, 0, 0, 5, 5, 5])
    t.compact()
    t.update(parent=[-1] * 6)
    assert t.pages.used() == 0
    assert t.compact() == []


def test_a_page_that_others_have_whole_is_copied():
    """Slot 1 shares slot 0's three pages; then it ends inside the second: it may not write that one."""
    t = Pair(12, 16, 3, 6)
    t.update(room=[48, 0, 0])
    t.update(parent=[0, 0, -1])
    moves = t.update(keep=[48, 20, 0], room=[0, 1, 0])
    assert len(moves) == 1 and moves[0][2] == 4
    # ... and where nobody has it whole, the lowest of the slots that go on from elsewhere keeps it
    moves = t.update(parent=[-1, 0, 0], keep=[0, 20, 20])
    assert [m[2] for m in moves] == [4] and t.model.table[1][1] != t.model.table[2][1]
    moves = t.update(parent=[2, 1, 2], keep=[7, 20, 9])             # slot 1 has that page whole: two copies
    assert [m[2] for m in moves] == [7, 9]
    own = t.model.table[2][0]
    moves = t.update(parent=[2, 1, 2], keep=[5, 20, 8])             # slot 2 stays itself: it keeps the page
    assert [m[2] for m in moves] == [5] and t.model.table[2][0] == own


@pytest.mark.parametrize("P,page,S,W,caches", [
    (7, 16, 1, 7, ((BF16, 1, 64),)),
    (61, 16, 9, 12, ((INT8, 2, 64), (BF16, 1, 128))),
    (200, 32, 33, 9, ((BF16, 2, 64),)),
    (150, 256, 5, 40, ((INT8, 1, 128),)),
    (5000, 16, 1500, 5, ((INT8, 1, 64),)),          # more slots than a block has threads
    (3001, 16, 12, 400, ((INT8, 1, 64),)),          # rows longer than a warp's piece of them
    (20000, 16, 300, 130, ((BF16, 1, 64),)),
])
def test_random_calls(P, page, S, W, caches):
    rng = random.Random(P)
    t = Pair(P, page, S, W, caches, seed=P)
    for step in range(14):
        held = [max(1, x) for x in t.model.len]
        most = max(1, P * page // (2 * S))
        kind = rng.choice(["grow", "grow", "fork", "beam", "trim", "mix", "compact"])
        if step == 0 or kind == "grow":
            t.update(room=[rng.choice([0, 1, 5, rng.randint(0, most)]) for _ in range(S)])
        elif kind == "fork":
            some = [rng.randrange(S) for _ in range(3)]
            t.update(parent=[i if rng.random() < 0.5 else rng.choice(some) for i in range(S)],
                     room=[rng.randint(0, 3) for _ in range(S)])
        elif kind == "beam":
            t.update(parent=[rng.randrange(S) for _ in range(S)], room=[1] * S)
        elif kind == "trim":
            t.update(keep=[rng.randint(-2, x + 3) for x in held])
        elif kind == "mix":
            t.update(parent=[rng.randrange(-1, S) for _ in range(S)],
                     keep=[rng.choice([page * rng.randint(0, 4), rng.randint(0, 200)]) for _ in range(S)],
                     room=[rng.randint(0, 2 * page) if rng.random() < 0.3 else 0 for _ in range(S)])
        else:
            t.compact()
    t.update(parent=[i if i % 3 else -1 for i in range(S)])
    t.compact()


def test_what_cannot_be_done_changes_nothing():
    t = Pair(10, 16, 3, 8)
    t.update(room=[50, 20, 0])                                     # 4 + 2 pages
    assert t.update(room=[0, 0, 65]) == "oom"                      # 5 of 4
    assert t.update(parent=[0, 0, 0], room=[100, 100, 0]) == "range"
    t.update(room=[0, 0, 64])                                      # all of them
    assert t.pages.used() == 10
    assert t.update(room=[14, 12, 1]) == "oom"
    t.update(parent=[2, 1, 0], room=[0, 12, 0])                    # rows that are left need no page
    assert t.update(parent=[0, 0, 0]) == []                        # pages given back by the call itself serve it
    assert t.update(parent=[0, 1, 3]) == "range" and t.update(parent=[0, -2, 1]) == "range"
    assert t.update(room=[0, -1, 0]) == "range"


def test_bad_tables_are_reported_and_left():
    t = Pair(20, 16, 3, 8)
    t.update(room=[40, 20, 0])
    keep = t.pages.table.clone()
    for bad in (20, -1, 10 ** 9):
        t.pages.table[0, 1] = bad
        before = [x.clone() for x in (t.pages.table, t.pages.kv_len, t.pages.refs)]
        t.pages.update(room=ints([1, 1, 1]))
        t.caches[0].copy(t.pages)
        assert t.pages.check_errors() == al.LORA_ERR_RANGE
        t.pages.compact()
        t.caches[0].copy(t.pages)
        assert t.pages.check_errors() == al.LORA_ERR_RANGE
        for a, b in zip((t.pages.table, t.pages.kv_len, t.pages.refs), before):
            assert torch.equal(a, b)
    t.pages.table.copy_(keep)
    for bad in (-1, 129, 2 ** 31 - 1):
        t.pages.kv_len[2] = bad
        t.pages.update(room=ints([1, 1, 1]))
        assert t.pages.check_errors() == al.LORA_ERR_RANGE
    t.pages.kv_len[2] = 0
    t.check()


def test_what_cannot_be_done_with_many_slots():
    t = Pair(3000, 16, 1500, 4, ((BF16, 1, 64),))
    t.update(room=[17 + i % 3 for i in range(1500)])
    bad = list(range(1500))
    bad[1400] = 1500
    assert t.update(parent=bad) == "range"
    assert t.update(room=[0] * 1499 + [64]) == "range"
    assert t.update(parent=[i // 2 for i in range(1500)], room=[32] * 1500) == "oom"
    t.update(parent=[i // 2 for i in range(1500)])


@pytest.mark.parametrize("S", [256, 1024, 1030])
def test_one_bad_slot_is_always_reported(S):
    """Whichever of them it is, and so whichever thread of whichever CTA finds it, call after call: a CTA's error word
    is cleared by other threads than those that set it."""
    t = Pair(2 * S, 16, S, 2, ((BF16, 1, 64),))
    t.update(room=[17] * S)
    parent, room = ints(list(range(S))), ints([0] * S)
    for i in sorted({0, 1, 2, 7, 8, 9, 63, 64, 255, S // 2, S - 9, S - 8, S - 2, S - 1} & set(range(S))):
        for _ in range(8):
            room[i] = 16                                           # one token more than its row of the table holds
            t.pages.update(room=room)
            assert t.pages.check_errors() == al.LORA_ERR_RANGE, i
            room[i] = 0
            parent[i] = S
            t.pages.update(parent, None, room)
            assert t.pages.check_errors() == al.LORA_ERR_RANGE, i
            parent[i] = i
    t.pages.update(parent, None, room)
    assert t.pages.check_errors() == al.LORA_OK
    t.check()


def test_a_shared_page_that_slots_end_inside():
    """Tables of the caller's own making: with room alone the call says so, with a parent it mends them."""
    t = Pair(20, 16, 3, 8)
    t.update(room=[20, 0, 0])
    t.pages.table[1] = t.pages.table[0]
    t.pages.kv_len[1] = 20
    t.pages.refs[:2] = 2
    t.model.table[1], t.model.len[1] = t.model.table[0][:], 20
    assert t.model.refs() == t.pages.refs.tolist()
    t.pages.update(room=ints([1, 1, 0]))
    assert t.pages.check_errors() == al.LORA_ERR_RANGE
    t.check()
    assert [m[2] for m in t.update(parent=[0, 1, 2], room=[1, 1, 0])] == [4]
    t.update(room=[1, 1, 1])


def test_the_tables_own_arrays_as_arguments():
    t = Pair(60, 16, 3, 8)
    t.update(room=[20, 5, 33])
    t.pages.update(keep=t.pages.kv_len, room=t.pages.kv_len)
    t.caches[0].copy(t.pages)
    assert t.model.update(keep=[20, 5, 33], room=[20, 5, 33]) == []
    t.check()


def test_compaction_into_other_tables():
    t = Pair(30, 16, 5, 6)
    t.update(room=[60, 33, 16, 80, 1])
    t.update(parent=[0, -1, 2, -1, 0])
    table, refs = torch.full_like(t.pages.table, 77), torch.full_like(t.pages.refs, 77)
    t.pages.compact(out=(table, refs))
    t.caches[0].copy(t.pages)
    t.model.refs()
    old = t.model.copy()
    moves = t.model.compact()
    assert moves
    apply_moves(t.want[0], moves)
    assert table.tolist() == t.model.table and refs.tolist() == t.model.refs()
    t.model = old
    t.check()                                                      # the handle's own are as they were
    t.pages.compact()
    t.model.compact()
    t.check()


def test_copies_of_lists():
    for fmt, H, D, page in ((INT8, 3, 64, 16), (BF16, 1, 128, 256), (INT8, 2, 128, 32)):
        t = Pair(25, page, 1, 1, ((fmt, H, D),))
        src, dst = [3, 7, -1, 7, 9, 4, 12], [11, 0, 5, 1, 9, -3, 24]
        rows = [1, page, 3, page - 1, 2, 5, 0]
        t.caches[0].copy_pages(ints(src), ints(dst), ints(rows))
        apply_moves(t.want[0], [(a, b, r) for a, b, r in zip(src, dst, rows) if min(a, b) >= 0])
        t.caches[0].copy_pages(ints([2, 6]), ints([20, 21]))
        apply_moves(t.want[0], [(2, 20, page), (6, 21, page)])
        t.check()
        for a, b, r in ((25, 0, 1), (0, 25, 1), (0, 1, page + 1), (0, 1, -1), (2 ** 31 - 1, 1, 1)):
            t.caches[0].copy_pages(ints([a]), ints([b]), ints([r]))
            assert t.caches[0].check_errors() == al.LORA_ERR_RANGE
        t.check()
        t.caches[0].copy_pages(ints([]), ints([]))


def test_pages_past_four_gigabytes():
    P = 70000                                                      # 2 x 4.6 GB
    c = al.KvCache(P, 64, 4, 128, BF16)
    c.k[5], c.v[5] = 1.0, 2.0
    c.copy_pages(ints([5]), ints([P - 1]))
    c.k[5] = 0.0
    c.copy_pages(ints([P - 1]), ints([4]), ints([3]))
    assert (c.k[4, :, :3] == 1).all() and not c.k[4, :, 3:].any() and (c.v[4, :, :3] == 2).all()
    assert not c.k[P - 2].any() and c.check_errors() == al.LORA_OK


def test_streams_and_graphs():
    """A captured step (update and copy) replayed, and calls on several streams in the order they are made."""
    t = Pair(400, 16, 8, 30)
    t.update(room=[20 + i for i in range(8)])
    parent, room = ints(list(range(8))), ints([3] * 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.pages.update(parent, None, room)
        t.caches[0].copy(t.pages)
    for p in ([1, 1, 2, 2, 4, 4, 4, 7], [7, 6, 5, 4, 3, 2, 1, 0], list(range(8))):
        parent.copy_(ints(p))
        graph.replay()
        torch.cuda.synchronize()
        apply_moves(t.want[0], t.model.update(p, None, [3] * 8))
        t.check()
    a, b = ints([0, 0, 2, 3, 4, 5, 6, 7]), ints([7, 1, 2, 3, 4, 5, 6, 0])
    torch.cuda.synchronize()
    for p, s in ((a, side), (b, torch.cuda.current_stream()), (a, side)):
        t.pages.update(p, stream=s)                                # no waits of ours in between
        t.caches[0].copy(t.pages, stream=torch.cuda.current_stream())
        apply_moves(t.want[0], t.model.update(p.tolist()))
    t.check()


def test_refusals():
    t = Pair(20, 16, 3, 8)

    def refused(status, call):
        with pytest.raises(al.LoraError) as e:
            call()
        assert e.value.status == status

    refused(al.LORA_ERR_SHAPE, lambda: t.pages.update(room=ints([1, 2])))
    refused(al.LORA_ERR_SHAPE, lambda: t.pages.update(parent=ints([0, 1, 2]).long()))
    refused(al.LORA_ERR_ARG, lambda: t.pages.update(keep=torch.zeros(3, dtype=torch.int32)))
    refused(al.LORA_ERR_SHAPE, lambda: t.pages.compact(out=(t.pages.table.clone(), t.pages.refs[:5].clone())))
    other = al.KvPages(20, 32, 3, 8)
    refused(al.LORA_ERR_ARG, lambda: t.caches[0].copy(other))
    refused(al.LORA_ERR_ARG, lambda: t.caches[0].copy(al.KvPages(21, 16, 3, 8)))
    refused(al.LORA_ERR_SHAPE, lambda: t.caches[0].copy_pages(ints([1]), ints([1, 2])))
    refused(al.LORA_ERR_ARG, lambda: t.caches[0].copy_pages(torch.zeros(1, dtype=torch.int32), ints([1])))
    t.check()
