"""The page steps on the host, one sequence after another: what the library's calls must give."""
import numpy as np

PAGE = 64


def n_pages(t):
    return (t + PAGE - 1) // PAGE


class Pool:
    """Numpy state: table [B, max_blocks], lens [B], refs [n_blocks]; codes / scales optional."""

    def __init__(self, B, max_blocks, n_blocks):
        self.table = np.full((B, max_blocks), -1, np.int32)
        self.lens = np.zeros(B, np.int32)
        self.refs = np.zeros(n_blocks, np.int32)

    def copy(self):
        p = Pool(*self.table.shape, len(self.refs))
        p.table, p.lens, p.refs = self.table.copy(), self.lens.copy(), self.refs.copy()
        return p

    def free_pages(self):
        return [int(p) for p in np.flatnonzero(self.refs == 0)]

    def append(self, n_new, cap):
        """(q_start, dst_slot, err)"""
        B, mb = self.table.shape
        q_start, slots = np.zeros(B + 1, np.int32), np.full(cap, -1, np.int64)
        err, need = 0, 0
        for b in range(B):
            t, n = int(self.lens[b]), int(n_new[b])
            if t < 0 or n < 0 or t > mb * PAGE:
                err |= 1
                continue
            if n and t + n > mb * PAGE:
                err |= 2
            elif n and t % PAGE:
                p = int(self.table[b, n_pages(t) - 1])
                if not (0 <= p < len(self.refs)) or self.refs[p] != 1:
                    err |= 1
            need += n_pages(t + n) - n_pages(t)
        if not err and (int(np.sum(n_new)) > cap or need > len(self.free_pages())):
            err = 2
        if err:
            return q_start, slots, err
        free = self.free_pages()
        i = 0
        for b in range(B):
            q_start[b] = i
            for _ in range(int(n_new[b])):
                t = int(self.lens[b])
                if t % PAGE == 0:
                    p = free.pop(0)
                    self.table[b, t // PAGE] = p
                    self.refs[p] = 1
                slots[i] = int(self.table[b, t // PAGE]) * PAGE + t % PAGE
                self.lens[b] += 1
                i += 1
        q_start[B] = i
        return q_start, slots, 0

    def fork(self, src, dst, fork_len=None):
        """(moves, err)"""
        B = len(self.lens)
        ok = len(set(dst)) == len(dst) and not set(src) & set(dst)
        for k, (a, d) in enumerate(zip(src, dst)):
            ok = ok and 0 <= a < B and 0 <= d < B and self.lens[d] == 0
            if ok and fork_len is not None:
                ok = 0 <= fork_len[k] <= self.lens[a]
        if not ok:
            return [], 1
        take = [int(self.lens[a]) if fork_len is None else int(fork_len[k]) for k, a in enumerate(src)]
        if sum(t % PAGE != 0 for t in take) > len(self.free_pages()):
            return [], 2
        free, moves = self.free_pages(), []
        for a, d, t in zip(src, dst, take):
            for c in range(t // PAGE):
                self.table[d, c] = self.table[a, c]
                self.refs[self.table[a, c]] += 1
            if t % PAGE:
                p = free.pop(0)
                moves.append((int(self.table[a, t // PAGE]), p))
                self.table[d, t // PAGE] = p
                self.refs[p] = 1
            self.lens[d] = t
        return moves, 0

    def free(self, seq):
        if len(set(seq)) != len(seq) or any(not 0 <= b < len(self.lens) for b in seq):
            return 1
        for b in seq:
            for c in range(n_pages(int(self.lens[b]))):
                self.refs[self.table[b, c]] -= 1
                self.table[b, c] = -1
            self.lens[b] = 0
        return 0

    def compact(self):
        """(moves, live)"""
        used = [int(p) for p in np.flatnonzero(self.refs > 0)]
        L = len(used)
        holes = [p for p in range(L) if self.refs[p] == 0]
        movers = [p for p in used if p >= L]
        to = dict(zip(movers, holes))
        for b in range(len(self.lens)):
            for c in range(n_pages(int(self.lens[b]))):
                p = int(self.table[b, c])
                self.table[b, c] = to.get(p, p)
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        return list(to.items()), L

    def consistent(self):
        """The counts are those of the held entries."""
        want = np.zeros_like(self.refs)
        for b in range(len(self.lens)):
            for c in range(n_pages(int(self.lens[b]))):
                want[self.table[b, c]] += 1
        return np.array_equal(want, self.refs)
