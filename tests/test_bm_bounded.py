"""Block manager of a bounded cache: blocks that a window has left are freed
(trim) and sequences take shorter block lists for the tokens they keep
(compact), against a plain model, with forks, copy-on-write, shortage and host
allocation failures."""
import numpy as np
import pytest

from oracle.bm_model import BlockManagerModel, OutOfBlocks


class Model(BlockManagerModel):
    def _release(self, b):
        if b >= 0:
            super()._release(b)

    def fork(self, parent, child):
        self.blocks[child] = list(self.blocks[parent])
        self.length[child] = self.length[parent]
        for b in self.blocks[child]:
            if b >= 0:
                self.ref[b] += 1

    def trim(self, seq, window, sinks):
        n, L = 0, self.length[seq]
        for i, b in enumerate(self.blocks[seq]):
            tokens = range(i * self.bs, min((i + 1) * self.bs, L))
            if b >= 0 and not any(t < sinks or t >= L - window for t in tokens):
                self._release(b)
                self.blocks[seq][i] = -1
                n += 1
        return n

    def compact(self, seqs, n_tokens):
        lists = []
        for s, n in zip(seqs, n_tokens):
            if s not in self.blocks or not 0 <= n <= self.length[s] or list(seqs).count(s) > 1:
                raise ValueError
            lists.append([b if b >= 0 and self.ref[b] == 1 else -1
                          for b in self.blocks[s][:-(-n // self.bs)]])
        if sum(b < 0 for x in lists for b in x) > len(self.free):
            raise OutOfBlocks()
        lists = [[b if b >= 0 else self._take() for b in x] for x in lists]
        for s, n, x in zip(seqs, n_tokens, lists):
            for i, b in enumerate(self.blocks[s]):
                if i >= len(x) or x[i] != b:
                    self._release(b)
            self.blocks[s], self.length[s] = x, n


@pytest.fixture(scope="module")
def BM():
    from paged_kv_cache_192_gb300 import build
    build.build()
    from paged_kv_cache_192_gb300.block_manager import BlockManager
    return BlockManager


def same(bm, model):
    assert bm.num_free() == len(model.free)
    for s in model.blocks:
        assert bm.seq_len(s) == model.length[s] and bm.seq_blocks(s) == model.blocks[s]
    assert [bm.refcount(b) for b in range(model.nb)] == model.ref


@pytest.mark.parametrize("seed", [0, 3, 77])
def test_random_operations_match_model(BM, seed):
    from paged_kv_cache_192_gb300._lib import OutOfBlocks as NativeOOB
    rng = np.random.default_rng(seed)
    nb, bs = 64, 4
    bm, model, next_id = BM(nb, bs, seed=seed), Model(nb, bs, seed=seed), 0
    for _ in range(700):
        live = list(model.blocks)
        pick = lambda: live[int(rng.integers(0, len(live)))]  # noqa: E731
        op = rng.integers(0, 9) if live else 0
        if op == 0:
            args, what = (next_id, int(rng.integers(0, 40))), "add_seq"
            next_id += 1
        elif op == 1:
            args, what = (pick(), next_id), "fork"
            next_id += 1
        elif op == 2 and len(live) > 3:
            args, what = (pick(),), "free_seq"
        elif op <= 4:
            args, what = (pick(), int(rng.integers(1, 14))), "append_n"
        elif op <= 6:
            args, what = (pick(), int(rng.integers(1, 30)), int(rng.integers(0, 9))), "trim"
        else:
            k = int(rng.integers(1, min(4, len(live)) + 1))
            seqs = [int(x) for x in rng.permutation(live)[:k]]
            args, what = (seqs, [int(rng.integers(0, model.length[s] + 1)) for s in seqs]), "compact"
        try:
            ref = getattr(model, what)(*args)
        except OutOfBlocks:
            with pytest.raises(NativeOOB):
                getattr(bm, what)(*args)
            same(bm, model)
            continue
        got = getattr(bm, what)(*args)
        if what == "trim":
            assert got == ref
        elif what == "append_n":
            assert list(got[0]) == ref[0] and got[1] == ref[1]
        same(bm, model)
    live = list(model.blocks)
    mb = max(len(model.blocks[s]) for s in live) + 1
    table = bm.block_table(live, mb)
    for row, s in zip(table.tolist(), live):
        assert row == model.blocks[s] + [0] * (mb - len(model.blocks[s]))


def test_trim_keeps_what_the_newest_token_sees(BM):
    bm = BM(64, 8)
    bm.add_seq(0, 100)  # 13 blocks, the last with 4 tokens
    assert bm.trim(0, window=100) == 0 and bm.trim(0, window=2 ** 62, num_sinks=2 ** 62) == 0
    # window 30: tokens 70.. ; sinks 9: blocks 0 and 1 stay
    assert bm.trim(0, window=30, num_sinks=9) == 6  # blocks 2 .. 7
    assert [i for i, b in enumerate(bm.seq_blocks(0)) if b < 0] == [2, 3, 4, 5, 6, 7]
    assert bm.trim(0, window=30, num_sinks=9) == 0
    bm.append_n(0, 2)
    assert bm.trim(0, window=30, num_sinks=9) == 1  # tokens 72..: block 8 is 64..71
    assert bm.trim(0, window=1) == 5                # sinks given up; the newest token's block stays
    assert bm.seq_blocks(0)[-1] >= 0 and sum(b >= 0 for b in bm.seq_blocks(0)) == 1
    bm.free_seq(0)
    assert bm.num_free() == 64


def test_trimmed_blocks_of_a_fork_stay_with_the_other_branch(BM):
    bm = BM(32, 8)
    bm.add_seq(0, 64)
    bm.fork(0, 1)
    free = bm.num_free()
    assert bm.trim(0, 8) == 7 and bm.num_free() == free
    assert all(bm.refcount(b) == 1 for b in bm.seq_blocks(1)[:-1])
    bm.fork(0, 2)  # a fork of a trimmed sequence has the same places
    assert bm.seq_blocks(2) == bm.seq_blocks(0)
    for s in (0, 1, 2):
        bm.free_seq(s)
    assert bm.num_free() == 32


def test_compact_in_place_and_with_shared_blocks(BM):
    bm = BM(32, 8)
    bm.add_seq(0, 64)
    before = bm.seq_blocks(0)
    bm.compact([0], [20])
    assert bm.seq_blocks(0) == before[:3] and bm.seq_len(0) == 20 and bm.num_free() == 29
    bm.fork(0, 1)
    shared = bm.seq_blocks(0)
    bm.compact([0, 1], [16, 9])  # both lists are new; the old blocks are free afterwards
    a, b = bm.seq_blocks(0), bm.seq_blocks(1)
    assert len(set(a + b + shared)) == 7 and len(a) == len(b) == 2 and bm.num_free() == 28


def test_refusals(BM):
    from paged_kv_cache_192_gb300._lib import OutOfBlocks as NativeOOB, PAError
    bm = BM(8, 8)
    bm.add_seq(0, 60)
    with pytest.raises(PAError):
        bm.trim(0, 0)
    with pytest.raises(PAError):
        bm.trim(0, 5, -1)
    with pytest.raises(PAError):
        bm.trim(7, 5)
    for seqs, n in (([0, 0], [5, 5]), ([7], [1]), ([0], [61]), ([0], [-1])):
        with pytest.raises(PAError):
            bm.compact(seqs, n)
    with pytest.raises(ValueError):
        bm.compact([0], [1, 2])
    bm.fork(0, 1)
    before = bm.seq_blocks(0), bm.seq_blocks(1)
    with pytest.raises(NativeOOB):
        bm.compact([0], [10])  # two fresh blocks, none free
    assert (bm.seq_blocks(0), bm.seq_blocks(1)) == before
    bm.compact([], [])


def test_host_allocation_failures_leave_state_unchanged(BM):
    from paged_kv_cache_192_gb300._lib import OutOfBlocks as NativeOOB
    from paged_kv_cache_192_gb300.block_manager import inject_alloc_failure
    bm, model = BM(64, 8, seed=4), Model(64, 8, seed=4)
    for m in (bm, model):
        m.add_seq(0, 100)
        m.fork(0, 1)
        m.add_seq(2, 30)
        m.trim(2, 9, 1)
    failures = 0
    while True:
        inject_alloc_failure(failures)
        try:
            bm.compact([0, 2, 1], [50, 20, 70])
        except NativeOOB as e:
            assert "host allocation failed" in str(e)
            same(bm, model)
            failures += 1
            continue
        finally:
            inject_alloc_failure(-1)
        break
    assert failures >= 5
    model.compact([0, 2, 1], [50, 20, 70])
    same(bm, model)
