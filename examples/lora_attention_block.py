"""One attention block of a served decoder layer, all on this library's kernels: multi-LoRA q, k
and v projections, the paged key/value cache, attention over it, the multi-LoRA o_proj.

    python examples/lora_attention_block.py [int8|bf16]

A ragged prefill of a few prompts, one more chunk of each, then decode steps replayed from one CUDA
graph: sequence lengths and page tables are device arrays, so the graph is captured once. Every
token's output is compared with the same block computed by plain PyTorch in one go.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import adapter_linear_gb300 as al  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, RANK, ADAPTERS, PAGE = 1024, 8, 2, 128, 16, 4, 16
WIDTHS = {"q": HEADS * DIM, "k": KV_HEADS * DIM, "v": KV_HEADS * DIM, "o": HIDDEN}


class Block:
    """The block's weights, its four adapter pools and its cache."""

    def __init__(self, fmt, max_seqs, max_tokens, seed=0):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        d_in = {"q": HIDDEN, "k": HIDDEN, "v": HIDDEN, "o": HEADS * DIM}
        self.weights = {m: self.normal(n, d_in[m], std=d_in[m] ** -0.5) for m, n in WIDTHS.items()}
        self.pools, self.adapters = {}, {}
        for m, n in WIDTHS.items():
            self.pools[m] = al.LoraPool(ADAPTERS, RANK, d_in[m], n)
            for slot in range(ADAPTERS):
                A, B = self.normal(d_in[m], RANK, std=d_in[m] ** -0.5), self.normal(RANK, n, std=0.3)
                self.pools[m].load_adapter(slot, A, B, RANK, float(RANK))
                self.adapters[m, slot] = (A, B)
        pages = -(-max_tokens // PAGE)
        self.cache = al.KvCache(max_seqs * pages, PAGE, KV_HEADS, DIM, fmt)
        order = torch.randperm(max_seqs * pages, generator=self.gen, device="cuda")
        self.table = order.view(max_seqs, pages).int()  # scattered, as a serving pool's pages are

    def normal(self, *shape, std=1.0):
        return (torch.randn(*shape, generator=self.gen, device="cuda") * std).to(torch.bfloat16)

    def reserve(self, tokens, seqs):
        """Scratch for calls of this size, so that they can be captured in a graph."""
        for p in self.pools.values():
            p.reserve(tokens)
        self.cache.reserve(tokens, HEADS, seqs)

    def forward(self, x, ids, batch):
        """x bf16 [T, HIDDEN], ids int32 [T] (an adapter each, or -1), batch: where the tokens belong."""
        q, k, v = al.LoraPool.linear_grouped([self.pools[m] for m in "qkv"], [x] * 3,
                                             [self.weights[m] for m in "qkv"], ids)
        self.cache.write(k.unflatten(1, (KV_HEADS, DIM)), v.unflatten(1, (KV_HEADS, DIM)), batch)
        out, _ = self.cache.attention(q.unflatten(1, (HEADS, DIM)), batch)
        return self.pools["o"].linear(out.flatten(1), self.weights["o"], ids)

    def errors(self):
        torch.cuda.synchronize()
        return [p.check_errors() for p in self.pools.values()] + [self.cache.check_errors()]

    def plain(self, x, adapter):
        """A whole sequence of one adapter by PyTorch in fp32, without a cache."""
        def linear(m, t):
            y = t @ self.weights[m].float().T
            if adapter >= 0:
                A, B = self.adapters[m, adapter]
                y += t @ A.float() @ B.float()
            return y
        q, k, v = (linear(m, x.float()).unflatten(1, (-1, DIM)).transpose(0, 1) for m in "qkv")
        k, v = (t.repeat_interleave(HEADS // KV_HEADS, 0) for t in (k, v))
        z = q @ k.transpose(1, 2) / math.sqrt(DIM)
        z = z.masked_fill(torch.ones_like(z[0], dtype=torch.bool).triu(1), float("-inf"))
        return linear("o", (torch.softmax(z, -1) @ v).transpose(0, 1).flatten(1))

    def close(self):
        self.cache.close()
        for p in self.pools.values():
            p.close()


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def run(fmt=al.LORA_KV_INT8, prompts=(70, 1, 129, 16), chunk=5, steps=8):
    """Returns the largest relative error (of a token's output, in its norm) against the plain block."""
    n = len(prompts)
    block = Block(fmt, n, max(prompts) + chunk + steps)
    adapters = [i % (ADAPTERS + 1) - 1 for i in range(n)]  # -1: the base model
    x = [block.normal(p + chunk + steps, HIDDEN) for p in prompts]
    got = [[] for _ in prompts]
    lens = [0] * n

    def chunk_of(new):  # the next new[i] tokens of every sequence
        start = [0]
        for i, m in enumerate(new):
            lens[i] += m
            start.append(start[-1] + m)
        rows = torch.cat([x[i][lens[i] - m:lens[i]] for i, m in enumerate(new)])
        ids = ints(sum(([adapters[i]] * m for i, m in enumerate(new)), []))
        batch = al.KvBatch(block.table, ints(start), ints(lens), start[-1], max(new))
        y = block.forward(rows, ids, batch)
        for i in range(n):
            got[i].append(y[start[i]:start[i + 1]])

    chunk_of(list(prompts))  # the prompts, all in one call
    chunk_of([chunk] * n)    # a few tokens more of each

    # decode: one token a sequence, the step captured once
    rows, kv_len = torch.empty(n, HIDDEN, dtype=torch.bfloat16, device="cuda"), ints(lens)
    batch = al.KvBatch(block.table, ints(list(range(n + 1))), kv_len, n, 1)
    ids = ints(adapters)
    block.reserve(max(sum(prompts), n), n)
    graph, y = torch.cuda.CUDAGraph(), None
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kv_len += 1
        y = block.forward(rows, ids, batch)
    kv_len.copy_(ints(lens))
    for s in range(steps):
        rows.copy_(torch.stack([x[i][lens[i] + s] for i in range(n)]))
        graph.replay()
        for i in range(n):
            got[i].append(y[i:i + 1].clone())

    assert block.errors() == [al.LORA_OK] * 5, block.errors()
    worst = 0.0
    for i in range(n):
        want = block.plain(x[i], adapters[i])
        err = (torch.cat(got[i]).float() - want).norm(dim=1) / want.norm(dim=1)
        worst = max(worst, float(err.max()))
    block.close()
    return worst


if __name__ == "__main__":
    name = sys.argv[1] if len(sys.argv) > 1 else "int8"
    err = run(al.LORA_KV_INT8 if name == "int8" else al.LORA_KV_BF16)
    print(f"{name} cache: prefill, chunk and decode agree with the plain block, "
          f"largest relative error of a token {err:.2e}")
