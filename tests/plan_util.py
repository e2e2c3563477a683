"""The plan of a step as lists on the host (not a test module): what pa_plan_step
has to do, page by page."""
import numpy as np
import torch


class Model:
    def __init__(self, num_seqs, width, num_blocks, bs, order=None, first=0):
        self.S, self.width, self.NB, self.bs = num_seqs, width, num_blocks, bs
        self.pages = {s: [] for s in range(num_seqs)}
        self.lens = [0] * num_seqs
        self.free = list(range(num_blocks) if order is None else order)  # front first
        self.first, self.refused = first, 0

    def state(self, device="cuda"):
        """The same as tensors: rows and ring entries that mean nothing hold -7."""
        from paged_kv_cache_192_gb300 import ops
        pages = np.full((self.S, self.width), -7, np.int32)
        for s, p in self.pages.items():
            pages[s, :len(p)] = p
        ring = np.full(self.NB, -7, np.int32)
        for i, p in enumerate(self.free):
            ring[(self.first + i) % self.NB] = p
        t = [torch.from_numpy(x).to(device) for x in
             (pages, np.array(self.lens, np.int32), ring,
              np.array([self.first, len(self.free), 0, self.refused], np.int32))]
        return ops.PageState(*t)

    def blocks(self, n):
        return -(-n // self.bs)

    def fits(self, ids, change, max_tokens, table_blocks):
        live = [s for s in ids if s >= 0]
        if any(s >= self.S for s in live) or len(set(live)) < len(live):
            return "request"
        need = 0
        for s, c in zip(ids, change):
            if s < 0:
                continue
            b = self.blocks(max(0, self.lens[s] + c))
            if b > min(self.width, table_blocks):
                return "blocks"
            need += max(0, b - len(self.pages[s]))
        if need > len(self.free) or sum(c for s, c in zip(ids, change) if s >= 0 and c > 0) > max_tokens:
            return "blocks"
        return None

    def step(self, ids, change, max_tokens, table_blocks=None):
        """(table, context_lens, query_start, slots, positions) as arrays, and why the
        step was refused."""
        W = self.width if table_blocks is None else table_blocks
        why = self.fits(ids, change, max_tokens, W)
        table = np.zeros((len(ids), W), np.int32)
        lens, start, slots, pos = [], [0], [], []
        given = []
        for r, (s, c) in enumerate(zip(ids, change)):
            c = 0 if why else c
            if s < 0 or s >= self.S:
                lens.append(0)
                start.append(start[-1])
                continue
            old = self.lens[s]
            new = max(0, old + c)
            own = self.pages[s]
            if not why:
                self.lens[s] = new
                while len(own) < self.blocks(new):
                    own.append(self.free.pop(0))
                    self.first = (self.first + 1) % self.NB
                while len(own) > self.blocks(new):
                    given.append((r, len(own) - 1, own.pop()))
            if len(own) > W:  # (refused: the table cannot show the row)
                lens.append(0)
                start.append(start[-1])
                continue
            table[r, :len(own)] = own
            lens.append(new)
            start.append(start[-1] + max(0, new - old))
            for p in range(old, new):
                slots.append(own[p // self.bs] * self.bs + p % self.bs)
                pos.append(p)
        self.free += [p for _, _, p in sorted(given)]
        self.refused += bool(why)
        slots += [-1] * (max_tokens - len(slots))
        pos += [0] * (max_tokens - len(pos))
        return (table, np.array(lens, np.int32), np.array(start, np.int32), np.array(slots, np.int64),
                np.array(pos, np.int64)), why

    def check(self, state):
        """The tensors hold what this model holds."""
        lens, ring, fs = (x.cpu().numpy() for x in state[1:])
        assert lens.tolist() == self.lens
        assert fs.tolist() == [self.first, len(self.free), 0, self.refused]
        assert [int(ring[(self.first + i) % self.NB]) for i in range(len(self.free))] == self.free
        pages = state[0].cpu().numpy()
        for s, p in self.pages.items():
            assert pages[s, :len(p)].tolist() == p


def same(plan, want):
    for got, ref in zip(plan, want):
        got = got.cpu().numpy()
        assert got.dtype == ref.dtype and got.shape == ref.shape
        assert np.array_equal(got, ref)
