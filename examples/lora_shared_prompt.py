"""Several answers to each of a few prompts, all on this library's kernels: multi-LoRA projections with rotary
positions, page tables that fork, grow and shrink on the GPU, and attention that reads a prompt's pages
once for all its answers.

    python examples/lora_shared_prompt.py [int8|bf16]

Each prompt is prefilled once and forked into its answers, which share the prompt's whole pages. The answers
then decode from one captured graph: page tables, lengths and rows are device arrays that the graph's own calls
advance. When some answers end, their pages are freed, the arena is compacted, and the same graph goes
on with the rest. Every token's output is compared with the same block computed by plain PyTorch in one go.
"""
import math
import sys

import torch

from lora_attention_block import DIM, HEADS, HIDDEN, KV_HEADS, PAGE, Block, al, ints


class SharedBlock(Block):
    """The attention block with rotary positions and page tables of its own."""

    def __init__(self, fmt, slots, max_tokens, seed=0):
        super().__init__(fmt, slots, max_tokens, seed)
        self.rotary = al.Rotary(DIM, scaling=("yarn", 4.0, 64))
        self.pages = al.KvPages(self.cache.num_pages, PAGE, slots, -(-max_tokens // PAGE))
        self.start = ints([0] * (slots + 1))
        self.slots = slots

    def batch(self, T, max_new):
        """The step's rows: slot s has rows start[s] .. start[s + 1], the last of its kv_len[s] tokens."""
        return al.KvBatch(self.pages.table, self.start, self.pages.kv_len, T, max_new)

    def rows_of(self, new):
        self.start.copy_(ints([sum(new[:i]) for i in range(len(new) + 1)]))

    def forward(self, x, ids, batch, groups=None):
        q, k, v = al.LoraPool.linear_grouped([self.pools[m] for m in "qkv"], [x] * 3, [self.weights[m] for m in "qkv"], ids)
        q = q.unflatten(1, (HEADS, DIM))
        self.cache.write_rotary(self.rotary, k.unflatten(1, (KV_HEADS, DIM)), v.unflatten(1, (KV_HEADS, DIM)), batch,
                                Q=q, Q_out=q)
        out, _ = self.cache.attention_shared(q, batch, groups) if groups else self.cache.attention(q, batch)
        return self.pools["o"].linear(out.flatten(1), self.weights["o"], ids)

    def turned(self, x):
        """x [heads, L, DIM] in fp32, rotated by the position of its row."""
        angle = torch.arange(x.shape[1], device="cuda", dtype=torch.float64)[:, None] * torch.tensor(
            self.rotary.freq, dtype=torch.float64, device="cuda")
        c, s = ((f * self.rotary.factor).float() for f in (angle.cos(), angle.sin()))
        a, b = x.chunk(2, -1)
        return torch.cat([a * c - b * s, a * s + b * c], -1)

    def plain(self, x, adapter):
        def linear(m, t):
            y = t @ self.weights[m].float().T
            if adapter >= 0:
                A, B = self.adapters[m, adapter]
                y += t @ A.float() @ B.float()
            return y
        q, k, v = (linear(m, x.float()).unflatten(1, (-1, DIM)).transpose(0, 1) for m in "qkv")
        q, k = self.turned(q), self.turned(k)
        k, v = (t.repeat_interleave(HEADS // KV_HEADS, 0) for t in (k, v))
        z = q @ k.transpose(1, 2) / math.sqrt(DIM)
        z = z.masked_fill(torch.ones_like(z[0], dtype=torch.bool).triu(1), float("-inf"))
        return linear("o", (torch.softmax(z, -1) @ v).transpose(0, 1).flatten(1))

    def errors(self):
        return super().errors() + [self.pages.check_errors()]

    def close(self):
        self.pages.close()
        super().close()


def run(fmt=al.LORA_KV_INT8, prompts=(70, 129), answers=4, steps=(6, 9)):
    """Returns the largest relative error (of a token's output, in its norm) against the plain block."""
    n, slots = len(prompts), len(prompts) * answers
    first = [p * answers for p in range(n)]                # the slot of a prompt, the first of its answers
    block = SharedBlock(fmt, slots, max(prompts) + sum(steps))
    block.reserve(max(sum(prompts), slots), slots)
    block.cache.reserve_shared(slots, HEADS, slots)
    adapters = [p % 2 * 2 - 1 for p in range(n)]            # the base model, adapter 1, ...
    prompt_x = [block.normal(L, HIDDEN) for L in prompts]
    answer_x = [block.normal(sum(steps), HIDDEN) for _ in range(slots)]
    got = [[] for _ in range(slots)]

    # the prompts, in one call
    new = [prompts[s // answers] if s in first else 0 for s in range(slots)]
    block.rows_of(new)
    block.pages.update(room=ints(new))
    ids = ints(sum(([adapters[p]] * L for p, L in enumerate(prompts)), []))
    y = block.forward(torch.cat(prompt_x), ids, block.batch(sum(prompts), max(prompts)))
    prompt_y = y.split(list(prompts))

    # each prompt's answers: what its whole pages hold is shared, the rest copied
    block.pages.update(parent=ints([s // answers * answers for s in range(slots)]))
    block.cache.copy(block.pages)
    groups = al.KvGroups(ints([p * answers for p in range(n + 1)]), ints(list(prompts)), answers)

    # one token of each answer, the step captured once
    rows = torch.zeros(slots, HIDDEN, dtype=torch.bfloat16, device="cuda")
    ids, room = ints([0] * slots), ints([0] * slots)
    batch, graph = block.batch(slots, 1), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        block.pages.update(room=room)
        out = block.forward(rows, ids, batch, groups)

    done = 0
    alive = list(range(slots))
    for phase in steps:
        room.copy_(ints([int(s in alive) for s in range(slots)]))
        block.rows_of([int(s in alive) for s in range(slots)])
        ids[:len(alive)] = ints([adapters[s // answers] for s in alive])
        for i in range(done, done + phase):
            rows[:len(alive)] = torch.stack([answer_x[s][i] for s in alive])
            graph.replay()
            for r, s in enumerate(alive):
                got[s].append(out[r].clone())
        done += phase
        if len(alive) == slots:                             # every other answer ends here
            alive = [s for s in alive if s % 2 == 0]
            block.pages.update(parent=ints([s if s in alive else -1 for s in range(slots)]))
            block.pages.compact()
            block.cache.copy(block.pages)
            used = block.pages.used()
            assert int(block.pages.table.max()) < used < block.cache.num_pages
    assert block.errors() == [al.LORA_OK] * 6, block.errors()

    worst = 0.0
    for s in range(slots):
        p = s // answers
        want = block.plain(torch.cat([prompt_x[p], answer_x[s][:len(got[s])]]), adapters[p])
        have = torch.cat([prompt_y[p], torch.stack(got[s])]).float()
        worst = max(worst, float(((have - want).norm(dim=1) / want.norm(dim=1)).max()))
    block.close()
    return worst


if __name__ == "__main__":
    name = sys.argv[1] if len(sys.argv) > 1 else "int8"
    err = run(al.LORA_KV_INT8 if name == "int8" else al.LORA_KV_BF16)
    print(f"{name} cache: prompts, forked answers and the compacted rest agree with the plain block, "
          f"largest relative error of a token {err:.2e}")
