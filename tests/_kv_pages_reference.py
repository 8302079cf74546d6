"""A plain model of the page tables: lists, one slot after the other."""
from __future__ import annotations


class Tables:
    def __init__(self, num_pages, page, slots, width):
        self.P, self.page, self.S, self.W = num_pages, page, slots, width
        self.table = [[-1] * width for _ in range(slots)]
        self.len = [0] * slots

    def copy(self):
        t = Tables(self.P, self.page, self.S, self.W)
        t.table, t.len = [r[:] for r in self.table], self.len[:]
        return t

    def entries(self, n):
        return -(-n // self.page)

    def refs(self):
        r = [0] * self.P
        for row, n in zip(self.table, self.len):
            for x in row[:self.entries(n)]:
                r[x] += 1
        return r

    def update(self, parent=None, keep=None, room=None):
        """Returns the copies (page, page, rows), or "oom" / "range" (nothing changed)."""
        S, p = self.S, self.page
        parent = list(range(S)) if parent is None else parent
        room = [0] * S if room is None else room
        n = []
        for i in range(S):
            if not -1 <= parent[i] < S or room[i] < 0:
                return "range"
            have = self.len[parent[i]] if parent[i] >= 0 else 0
            n.append(have if keep is None else min(have, max(0, keep[i])))
            if n[i] + room[i] > self.W * p:
                return "range"
        whole, ends = set(), {}
        for i in range(S):
            whole.update(self.table[parent[i]][:n[i] // p] if parent[i] >= 0 else [])
            if n[i] % p:
                ends.setdefault(self.table[parent[i]][n[i] // p], []).append((parent[i] != i, i))
        stays = {min(who)[1]: x for x, who in ends.items() if x not in whole}
        free = [x for x in range(self.P) if x not in whole and x not in stays.values()]
        table, moves = [], []
        for i in range(S):
            row = self.table[parent[i]][:n[i] // p] if parent[i] >= 0 else []
            if i in stays:
                row = row + [stays[i]]
            while len(row) < self.entries(n[i] + room[i]):
                if not free:
                    return "oom"
                if len(row) == n[i] // p and n[i] % p:
                    moves.append((self.table[parent[i]][len(row)], free[0], n[i] % p))
                row = row + [free.pop(0)]
            table.append(row + [-1] * (self.W - len(row)))
        self.table, self.len = table, [a + b for a, b in zip(n, room)]
        return moves

    def compact(self):
        refs = self.refs()
        used = [x for x in range(self.P) if refs[x]]
        n = len(used)
        moves = list(zip([x for x in used if x >= n], [x for x in range(n) if not refs[x]]))
        to = dict(moves)
        self.table = [[to.get(x, x) for x in row] for row in self.table]
        return [(a, b, self.page) for a, b in moves]


def apply_moves(arenas, moves):
    """Copies of rows in [P][H][p][...] tensors, all sources read first."""
    for t in arenas:
        rows = [t[a, :, :r].clone() for a, _, r in moves]
        for (_, b, r), x in zip(moves, rows):
            t[b, :, :r] = x
