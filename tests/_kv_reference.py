"""Plain 64-bit forms of the paged cache's operators (numpy / torch float64), and a builder of
paged caches with scattered pages for their tests."""
from __future__ import annotations

import numpy as np
import torch

TINY = 2.0 ** -126


def bf16_of_f64(x: torch.Tensor) -> torch.Tensor:
    """float64 -> bf16 rounded once (to nearest, ties to even), by integer arithmetic on the
    float64 bits for finite normal results; smaller ones go through the exact multiple of the
    smallest subnormal."""
    step = torch.full_like(x, 2.0 ** -133)          # bf16's smallest subnormal
    m, e = torch.frexp(x)
    # 8 significant bits; the power of two from its bits (torch.ldexp on a GPU goes through an
    # inexact fp32 power)
    ulp = ((e.long() - 8 + 1023) << 52).view(torch.float64)
    ulp = torch.maximum(ulp, step)
    return torch.where(torch.isfinite(x), torch.round(x / ulp) * ulp, x).to(torch.bfloat16)


def quantise(x: torch.Tensor):
    """(codes, scales) float64 of rows x[..., D] (bf16), from the definition."""
    f = x.double()
    s = bf16_of_f64(f.abs().amax(-1) / 127.0).double().clamp_min(TINY)
    q = torch.clamp(torch.round(f / s[..., None]), -127, 127)
    ok = torch.isfinite(f).all(-1)
    q = torch.where(ok[..., None], q, torch.zeros_like(q))
    s = torch.where(ok, s, torch.full_like(s, float("nan")))
    return q, s


class Paged:
    """Sequences of given lengths in a paged cache with scattered pages. Rows that hold no
    token are NaN (bf16) or code 77 with a NaN scale (int8)."""

    def __init__(self, al, fmt, lens, new, H, D, page, seed=0, spare=3, std=1.0, device="cuda"):
        g = torch.Generator(device="cpu").manual_seed(seed)
        self.al, self.fmt, self.H, self.D, self.page = al, fmt, H, D, page
        self.lens, self.new = list(lens), list(new)
        int8 = fmt == al.LORA_KV_INT8
        counts = [-(-n // page) for n in self.lens]
        P = sum(counts) + spare
        perm = torch.randperm(P, generator=g).int()
        table = torch.full((len(self.lens), max(counts + [1]) + 1), -7, dtype=torch.int32)
        at = 0
        for b, c in enumerate(counts):
            table[b, :c] = perm[at:at + c]
            at += c
        self.table = table.to(device)
        self.start = [0]
        for n in self.new:
            self.start.append(self.start[-1] + n)
        self.T = self.start[-1]
        self.values = []          # per sequence (K, V) float64 [L][H][D], what the cache stands for
        dtype = torch.int8 if int8 else torch.bfloat16
        fill = 77 if int8 else float("nan")
        arenas, scales = [], []
        for _ in range(2):
            arenas.append(torch.full((P, H, page, D), fill, dtype=dtype, device=device))
            scales.append(torch.full((P, H, page), float("nan"), dtype=torch.bfloat16, device=device)
                          if int8 else None)
        gd = torch.Generator(device=device).manual_seed(seed + 1)
        for b, L in enumerate(self.lens):
            pair = []
            for a, s in zip(arenas, scales):
                x = (torch.randn(L, H, D, generator=gd, device=device) * std).to(torch.bfloat16)
                pages, rows = self.where(b, torch.arange(L, device=device))
                if int8:
                    q, sc = quantise(x)
                    a[pages, :, rows] = q.to(torch.int8)
                    s[pages, :, rows] = sc.to(torch.bfloat16)
                    pair.append(q * sc[..., None])
                else:
                    a[pages, :, rows] = x
                    pair.append(x.double())
            self.values.append(pair)
        self.cache = al.KvCache(P, page, H, D, fmt, arenas=(arenas[0], arenas[1], scales[0], scales[1]))
        self.batch = al.KvBatch(self.table, torch.tensor(self.start, dtype=torch.int32, device=device),
                                torch.tensor(self.lens, dtype=torch.int32, device=device), self.T,
                                max(self.new + [0]))

    def where(self, b, pos):
        return self.table[b].long()[pos // self.page], pos % self.page


def attention(Q, paged: Paged, scale, window=0):
    """(O, lse, A, S) in float64: the outputs, sum_j p_j |V_j| (what an error in p is multiplied
    by) and max_j sum_d |q_d K_jd| scale (what an error in a product is relative to)."""
    T, Hq, D = Q.shape
    G = Hq // paged.H
    O = torch.zeros((T, Hq, D), dtype=torch.float64, device=Q.device)
    A = torch.zeros_like(O)
    lse = torch.full((T, Hq), float("-inf"), dtype=torch.float64, device=Q.device)
    S = torch.zeros_like(lse)
    for b, (n, L) in enumerate(zip(paged.new, paged.lens)):
        if n == 0 or L == 0:
            continue
        K, V = paged.values[b]
        pos = torch.arange(L - n, L, device=Q.device)
        j = torch.arange(L, device=Q.device)
        seen = j[None, :] <= pos[:, None]
        if window > 0:
            seen &= j[None, :] > pos[:, None] - window
        rows = slice(paged.start[b], paged.start[b] + n)
        some = seen.any(1)
        for h in range(Hq):
            q = Q[rows, h].double()
            z = (q @ K[:, h // G].T) * scale
            z = z.masked_fill(~seen, float("-inf"))
            l = torch.logsumexp(z, 1)
            p = torch.exp(z - torch.where(some, l, torch.zeros_like(l))[:, None])
            O[rows, h] = p @ V[:, h // G]
            A[rows, h] = p @ V[:, h // G].abs()
            lse[rows, h] = l
            S[rows, h] = ((q.abs() @ K[:, h // G].abs().T) * abs(scale)).masked_fill(~seen, 0).amax(1)
    return O, lse, A, S


def check_attention(got_O, got_lse, ref, what=""):
    """Bounds, derived: each softmax weight may be rounded to bf16 (2^-9 of it, so 2^-9 A in all),
    the output is (2^-9 |O| <= 2^-9 A); a score is a sum of D products in fp32, with at most 16
    steps that each lose 2^-22 of the largest partial sum: 2^-18 S, allowed twice, and moves
    O by at most twice that times A."""
    O, lse, A, S = ref
    dz = 2.0 ** -17 * S + 2.0 ** -20
    err = (got_O.double() - O).abs()
    bound = A * (2.0 ** -8 + 2 * dz[..., None]) + 2.0 ** -100
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outputs off, worst {float(err.max()):.3g}"
    if got_lse is not None:
        empty = torch.isinf(lse)
        assert torch.equal(torch.isneginf(got_lse), empty), f"{what}: rows that see nothing"
        e = (got_lse.double() - lse).abs()[~empty]
        assert (e <= (dz + 2.0 ** -20 * (1 + lse.abs()))[~empty]).all(), \
            f"{what}: lse off by {float(e.max()) if e.numel() else 0:.3g}"
