"""GPU tests of rotary positions against the definition in 64 bits: layouts, part of the head, far and
negative positions, strides, in place, inverse, and the cache's write with the rotation on the way."""
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


def turned(x, pos, rot, inverse=False):
    """x [T, heads, D] rotated in float64, and the length of each value's pair times the factor."""
    f = torch.tensor(rot.freq, dtype=torch.float64, device=x.device)
    # |p| f may be large: reduced by the exact remainder of fp64
    a = torch.remainder(pos.double()[:, None] * f, 2 * math.pi)[:, None, :]
    c, s = a.cos() * rot.factor, a.sin() * rot.factor * (-1 if inverse else 1)
    y, size = x.double().clone(), x.double().abs()
    n = rot.rotary_dim
    lo, hi = (slice(0, n // 2), slice(n // 2, n)) if rot.layout == "half" else (slice(0, n, 2), slice(1, n, 2))
    u, v = x[..., lo].double(), x[..., hi].double()
    y[..., lo], y[..., hi] = u * c - v * s, u * s + v * c
    size[..., lo] = size[..., hi] = torch.sqrt(u * u + v * v) * abs(rot.factor)
    return y, size


def check(got, want, size, far, freq=1.0):
    """Bounds: one rounding to bf16 (half a step, 2^-8 of what is rounded); sine and cosine off by 2^-22 (the
    angle) and 2^-23 (their own), two products and a sum in fp32, 2^-23 together: 2^-20 of the pair's length;
    the angle in the reference and the frequency in turns off by 2^-51 of |p| freq."""
    dx = size * (2.0 ** -20 + 2.0 ** -50 * far * freq)
    bound = (want.abs() + dx) * 2.0 ** -8 + dx + 2.0 ** -134
    err = (got.double() - want).abs()
    assert (err <= bound).all(), f"worst {float((err - bound).max()):.3g}"


def rows(T, heads, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(T, heads, D, generator=g, device="cuda").to(torch.bfloat16)


CASES = [  # T, heads of the tensors, D, rotary_dim, layout, scaling
    (1, (1,), 16, 16, "half", None),
    (1, (32, 8), 128, 128, "half", None),
    (7, (3, 1), 64, 32, "interleaved", ("linear", 4.0, 2048)),
    (33, (5, 2, 7), 80, 80, "half", ("yarn", 8.0, 4096)),
    (129, (6,), 96, 64, "half", ("bands", 8.0, 8192)),
    (50, (4, 4, 1, 2), 192, 96, "interleaved", ("ntk", 4.0, 2048)),
    (300, (24, 8), 256, 256, "interleaved", None),
    (2000, (14, 2), 64, 64, "half", ("yarn", 40.0, 4096)),
    (1111, (1,), 112, 48, "half", None),
    (65, (200,), 128, 16, "interleaved", None),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("inverse", [False, True])
def test_apply(case, inverse):
    T, heads, D, n, layout, scaling = CASES[case]
    rot = al.Rotary(n, layout=layout, scaling=scaling)
    g = torch.Generator(device="cuda").manual_seed(case)
    for far in (100, 1 << 20, (1 << 31) - 1):
        pos = torch.randint(-far - 1, far, (T,), generator=g, device="cuda").int()
        pos[0] = far
        xs = [rows(T, h, D, 7 * case + i) for i, h in enumerate(heads)]
        before = [x.clone() for x in xs]
        got = rot.apply(xs, pos, inverse=inverse)
        for x, b, y in zip(xs, before, got):
            assert torch.equal(x, b)
            assert torch.equal(y[..., n:], x[..., n:])
            check(y, *turned(x, pos, rot, inverse), far)


def test_position_zero_changes_nothing():
    for layout in ("half", "interleaved"):
        x = rows(9, 3, 128, 3)
        x[2, 1, 5], x[3, 0, 100] = 3.0e38, -3.0e38
        (y,) = al.Rotary(64, layout=layout).apply((x,), torch.zeros(9, dtype=torch.int32, device="cuda"))
        assert torch.equal(x, y)


def test_strided_in_place_and_into_given_tensors():
    rot = al.Rotary(64)
    wide = rows(37, 11, 128, 5).flatten(1)
    want = [turned(x, torch.arange(37, device="cuda"), rot) for x in (wide[:, 128:640].unflatten(1, (4, 128)),
                                                                   wide[:, 1024:1280].unflatten(1, (2, 128)))]
    pos = torch.arange(37, device="cuda").int()
    out = torch.full((37, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    q, k = wide[:, 128:640].unflatten(1, (4, 128)), wide[:, 1024:1280].unflatten(1, (2, 128))
    got = rot.apply((q, k), pos, out=(out[:, 1:5], out[:, 6:8]))
    assert got[0].data_ptr() == out[:, 1:5].data_ptr()
    for y, w in zip(got, want):
        check(y, *w, 37)
    assert (out[:, 0] == 5).all() and (out[:, 5] == 5).all()
    keep = wide.clone()
    rot.apply((q, k), pos, out=(q, k))
    assert torch.equal(q, out[:, 1:5]) and torch.equal(k, out[:, 6:8])
    for a, b in ((0, 128), (640, 1024), (1280, 1408)):
        assert torch.equal(wide[:, a:b], keep[:, a:b])


def test_rows_that_are_not_finite_reach_their_pair_only():
    rot = al.Rotary(32)
    x = rows(4, 2, 64, 1)
    x[1, 0, 3], x[2, 1, 40], x[3, 1, 17] = float("nan"), float("inf"), float("-inf")
    (y,) = rot.apply((x,), torch.arange(4, device="cuda").int() + 1)
    bad = torch.zeros_like(x, dtype=torch.bool)
    bad[1, 0, 3] = bad[1, 0, 19] = bad[2, 1, 40] = bad[3, 1, 17] = bad[3, 1, 1] = True
    assert torch.equal(~torch.isfinite(y), bad) and y[2, 1, 40] == float("inf")


def test_gradient_against_differences():
    """<g, f(x + d) - f(x - d)> = <inverse(g), (x + d) - (x - d)> for the linear map f. Every result is rounded
    to bf16 once, 2^-8 of it at most; the fp32 arithmetic below that is 2^-20 of a pair's length."""
    rot = al.Rotary(64, scaling=("yarn", 8.0, 4096))
    pos = torch.randint(0, 100000, (6,), device="cuda").int()
    x, d, g = rows(6, 2, 64, 1), rows(6, 2, 64, 2), rows(6, 2, 64, 3)
    plus, minus = x + d, x - d
    up, down = (y.double() for y in rot.apply((plus, minus), pos))
    back = rot.apply((g,), pos, inverse=True)[0].double()
    step = plus.double() - minus.double()
    left, right = (g.double() * (up - down)).sum(), (back * step).sum()
    size = (g.double().abs() * (up.abs() + down.abs()) + back.abs() * step.abs()).sum()
    assert size > 100 and abs(left - right) <= size * (2.0 ** -8 + 2.0 ** -9)


def test_streams_and_graph():
    rot = al.Rotary(128)
    x, pos = rows(64, 40, 128, 1), torch.arange(64, device="cuda").int()
    (want,) = rot.apply((x,), pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    (got,) = rot.apply((x,), pos, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rot.apply((x,), pos, out=(out,))
    pos += 5
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, rot.apply((x,), pos)[0])


@pytest.mark.parametrize("T", [64, 20000])
def test_positions_that_the_kernel_ahead_writes(T):
    """A call's kernel may start while the one ahead of it still runs: it turns by the positions that one leaves. Page
    tables' updates let it start at once, call after call, and so from a graph; lengths are the positions."""
    rot, S = al.Rotary(64), T
    pages = al.KvPages(S, 16, S, 1)
    x, room = rows(T, 2, 64, 1), torch.ones(S, dtype=torch.int32, device="cuda")

    def three():
        got = []
        for _ in range(3):
            pages.update(room=room)
            got.append(rot.apply((x,), pages.kv_len)[0])
        return got

    first = three()
    want = [rot.apply((x,), torch.full((T,), n, dtype=torch.int32, device="cuda"))[0] for n in range(1, 10)]
    for n, y in enumerate(first):
        assert torch.equal(y, want[n])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = three()
    for n in (3, 6):
        graph.replay()
        torch.cuda.synchronize()
        for i, y in enumerate(got):
            assert torch.equal(y, want[n + i])
    assert pages.check_errors() == al.LORA_OK


@pytest.mark.parametrize("fmt,Hq,H,D,page,lens,new,n,layout", [
    (INT8, 32, 8, 128, 16, [1, 17, 16, 400], [1, 5, 0, 203], 128, "half"),
    (INT8, 3, 1, 64, 32, [33, 1, 90], [33, 1, 7], 32, "interleaved"),
    (INT8, 7, 3, 64, 256, [300, 2], [299, 2], 64, "half"),
    (BF16, 4, 2, 128, 64, [64, 65, 0, 7], [64, 1, 0, 3], 64, "interleaved"),
    (BF16, 5, 5, 64, 128, [1000], [77], 64, "half"),
    (INT8, 32, 8, 128, 16, [40 + i for i in range(67)], [1] * 67, 96, "half"),
    (BF16, 6, 2, 128, 16, [5, 0, 3], [9, 2, 3], 128, "half"),        # positions below zero
    (INT8, 0, 2, 128, 16, [5, 60], [5, 9], 128, "half"),             # no queries
    (INT8, 14, 2, 128, 16, [2500], [2500], 128, "interleaved"),
])
def test_write_rotary(fmt, Hq, H, D, page, lens, new, n, layout):
    p = R.Paged(al, fmt, lens, new, H, D, page, seed=3)
    rot = al.Rotary(n, layout=layout, scaling=("yarn", 8.0, 4096))
    K, V, Q = rows(p.T, H, D, 5), rows(p.T, H, D, 6), rows(p.T, max(Hq, 1), D, 7)
    got_q = p.cache.write_rotary(rot, K, V, p.batch, Q=Q if Hq else None)
    Kr, Vr = p.cache.read(p.batch)
    assert p.cache.check_errors() == al.LORA_OK
    twin = R.Paged(al, fmt, lens, new, H, D, page, seed=3)
    twin.cache.write(K, V, twin.batch)
    assert torch.equal(twin.cache.read(twin.batch)[1], Vr)            # V as the plain write has it
    for b, (m, L) in enumerate(zip(new, lens)):
        r0, skip = p.start[b], max(0, m - L)
        sl = slice(r0 + skip, r0 + m)
        pos = torch.arange(L - m + skip, L, device="cuda")
        if Hq:
            check(got_q[sl], *turned(Q[sl], pos, rot), max(lens))
            assert not got_q[r0:r0 + skip].any()
        want, size = turned(K[sl], pos, rot)
        if fmt == BF16:
            check(Kr[sl], want, size, max(lens))
            continue
        # the stored scale is bf16(amax / 127) of values that are off by 2^-20; a code is within
        # 1/2 + 2^-10 of a step
        pages, offs = p.where(b, pos)
        s = p.cache.k_scales[pages, :, offs].double()
        amax = want.abs().amax(-1)
        assert ((s - amax / 127).abs() <= amax / 127 * (2.0 ** -8 + 2.0 ** -18)).all()
        code = p.cache.k[pages, :, offs].double()
        assert ((code * s[..., None] - want).abs() <= s[..., None] * (0.5 + 2.0 ** -10)).all()
    # nothing but the batch's rows was touched
    untouched = torch.ones(p.cache.k.shape[0], page, dtype=torch.bool, device="cuda")
    for b, (m, L) in enumerate(zip(new, lens)):
        if min(m, L) > 0:
            pages, offs = p.where(b, torch.arange(max(0, L - m), L, device="cuda"))
            untouched[pages, offs] = False
    fresh = R.Paged(al, fmt, lens, new, H, D, page, seed=3)
    for a, b in ((p.cache.k, fresh.cache.k), (p.cache.v, fresh.cache.v)):
        a, b = a.transpose(1, 2)[untouched], b.transpose(1, 2)[untouched]
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("D,n", [(128, 128), (64, 64), (128, 32)])
def test_codes_of_fp32_keys_are_rounded_once(D, n):
    """Without an angle a key is fp32(x factor), what its code comes from is known: rint(that / scale), to even at a tie,
    but for 2^-17 of a step beside a tie (the quotient in fp32: half of its 2^-17 below 128, twice that allowed). Keys
    that are not rotated are bf16: exactly rint."""
    H, L = 8, 3000
    p = R.Paged(al, INT8, [L], [L], H, D, 16, seed=3)
    K, V = rows(L, H, D, 5), rows(L, H, D, 6)
    factor = torch.tensor(1.0123457, dtype=torch.float32)
    p.cache.write_rotary(al.Rotary(n, freq=[0.0] * (n // 2), factor=float(factor)), K, V, p.batch)
    assert p.cache.check_errors() == al.LORA_OK
    pages, offs = p.where(0, torch.arange(L, device="cuda"))
    x = K.float()
    x[..., :n] *= factor.cuda()
    s, code = p.cache.k_scales[pages, :, offs].double(), p.cache.k[pages, :, offs].double()
    assert torch.equal(s.to(torch.bfloat16), R.bf16_of_f64((x.abs().amax(-1) / torch.full_like(x[..., 0], 127)).double()))
    y = x.double() / s[..., None]
    beside = (y - torch.floor(y) - 0.5).abs()
    sure = (beside > 2.0 ** -17) | (torch.arange(D, device="cuda") >= n)
    assert torch.equal(code[sure], torch.round(y)[sure])
    # what a rounding to a multiple of 2^-11 ahead would have moved is among them
    assert int((sure & (beside < 2.0 ** -12)).sum()) > 300
    want, _ = R.quantise(V)
    assert torch.equal(p.cache.v[pages, :, offs].double(), want)


def test_write_rotary_strided_in_place_padded():
    p = R.Paged(al, INT8, [20, 7], [13, 2], 2, 64, 16, seed=9)
    rot = al.Rotary(64)
    T = p.T + 5
    wide = rows(T, 9, 64, 2).flatten(1)
    Q, K, V = (wide[:, a * 64:b * 64].unflatten(1, (b - a, 64)) for a, b in ((0, 4), (5, 7), (7, 9)))
    keep = wide.clone()
    batch = al.KvBatch(p.table, p.batch.start, p.batch.kv_len, T, 13)
    want = p.cache.write_rotary(rot, K, V, batch, Q=Q)[:p.T].clone()
    k0 = p.cache.k.clone()
    got = p.cache.write_rotary(rot, K, V, batch, Q=Q, Q_out=Q)
    assert got.data_ptr() == wide.data_ptr() and torch.equal(got[:p.T], want) and torch.equal(p.cache.k, k0)
    assert torch.equal(wide[p.T:], keep[p.T:]) and torch.equal(wide[:, 4 * 64:], keep[:, 4 * 64:])
    assert p.cache.check_errors() == al.LORA_OK


def test_write_rotary_not_finite():
    """A row of K with a bad value reads back as NaN; the rows beside it and V are what they were."""
    p = R.Paged(al, INT8, [6], [6], 2, 64, 16, seed=9)
    K, V = rows(6, 2, 64, 1), rows(6, 2, 64, 2)
    K[1, 0, 3], K[2, 1, 63], V[4, 1, 7] = float("nan"), float("inf"), float("-inf")
    K[5] = 3.3e38                                       # pairs longer than the largest value
    p.cache.write_rotary(al.Rotary(32), K, V, p.batch)
    Kr, Vr = p.cache.read(p.batch)
    bad = torch.isnan(Kr).all(-1)
    want = torch.zeros(6, 2, dtype=torch.bool, device="cuda")
    want[1, 0] = want[2, 1] = True
    y, _ = turned(K, torch.arange(6, device="cuda"), al.Rotary(32))
    want |= y.abs().amax(-1) > 3.402823e38
    assert torch.equal(bad, want) and want[5].all()
    assert torch.equal(torch.isnan(Vr).all(-1), (torch.arange(12, device="cuda") == 9).view(6, 2))


def test_write_rotary_refusals_and_bad_tables():
    p = R.Paged(al, INT8, [20, 7], [3, 2], 2, 64, 16, seed=9)
    K, V, Q = rows(5, 2, 64, 1), rows(5, 2, 64, 2), rows(5, 4, 64, 3)
    rot = al.Rotary(64)

    def refused(status, **kw):
        a = dict(rotary=rot, K=K, V=V, batch=p.batch, Q=Q, Q_out=None) | kw
        with pytest.raises(al.LoraError) as e:
            p.cache.write_rotary(a["rotary"], a["K"], a["V"], a["batch"], Q=a["Q"], Q_out=a["Q_out"])
        assert e.value.status == status

    before = p.cache.k.clone()
    refused(al.LORA_ERR_SHAPE, rotary=al.Rotary(128))
    refused(al.LORA_ERR_SHAPE, K=K[:4])
    refused(al.LORA_ERR_SHAPE, Q=Q.float())
    refused(al.LORA_ERR_ARG, Q=None, Q_out=Q)
    refused(al.LORA_ERR_ARG, Q=rows(5, 4, 65, 3)[..., 1:])
    torch.cuda.synchronize()
    assert torch.equal(p.cache.k, before)
    table = p.table.clone()
    table[0, 1] = 10 ** 6                                # page of tokens 16..19: rows 0..2 of the batch
    bad = al.KvBatch(table, p.batch.start, p.batch.kv_len, 5, 3)
    got = p.cache.write_rotary(rot, K, V, bad, Q=Q)
    assert p.cache.check_errors() == al.LORA_ERR_RANGE and p.cache.check_errors() == al.LORA_OK
    check(got[3:], *turned(Q[3:], torch.arange(5, 7, device="cuda"), rot), 7)
    pages, offs = p.where(1, torch.arange(5, 7, device="cuda"))
    want, _ = turned(K[3:], torch.arange(5, 7, device="cuda"), rot)
    s = p.cache.k_scales[pages, :, offs].double()[..., None]
    assert ((p.cache.k[pages, :, offs].double() * s - want).abs() <= s * (0.5 + 2.0 ** -10)).all()
