"""The bounded-cache operators together, as a serving loop uses them: rotary
store, windowed prefill of a prompt in chunks, windowed decode steps, pages
freed behind the window and given to other sequences, a fork with
copy-on-write, and a compaction after which plain decode reads the cache."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV, bf16 = "cuda", torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_192_gb300 import build
    build.build()


class Loop:
    W, S, Hq, Hkv, d, bs = 48, 5, 8, 2, 64, 8

    def __init__(self, num_blocks, dtype=bf16):
        from paged_kv_cache_192_gb300 import layout
        from paged_kv_cache_192_gb300.block_manager import BlockManager
        self.bm = BlockManager(num_blocks, self.bs, seed=5)
        self.k, self.v = layout.alloc_pools(num_blocks, self.Hkv, self.bs, self.d, dtype, DEV)
        self.hist = {}  # sequence -> rows stored so far (K as stored, V)
        self.g = torch.Generator().manual_seed(11)
        self.inv = (10000.0 ** (-torch.arange(self.d // 2).double() / (self.d // 2))).float().to(DEV)
        self.dtype = dtype

    def rand(self, *shape):
        return torch.randn(*shape, generator=self.g).to(self.dtype).to(DEV)

    def store(self, tokens):
        """tokens: {seq: n} appended and stored; returns the rotated queries."""
        from paged_kv_cache_192_gb300 import ops
        slots, pos, pairs = [], [], []
        for s, n in tokens.items():
            L = self.bm.seq_len(s)
            sl, cow = self.bm.append_n(s, n)
            slots += list(sl)
            pos += list(range(L, L + n))
            pairs += cow
        if pairs:
            ops.copy_blocks(self.k, self.v, torch.tensor(pairs, dtype=torch.int64, device=DEV))
        T = len(slots)
        q, k, v = self.rand(T, self.Hq, self.d), self.rand(T, self.Hkv, self.d), self.rand(T, self.Hkv, self.d)
        slots = torch.tensor(slots, dtype=torch.int64, device=DEV)
        q = ops.rope_reshape_and_cache(q, k, v, self.k, self.v, slots,
                                       torch.tensor(pos, dtype=torch.int64, device=DEV), self.inv)
        kr = self.k[slots // self.bs, :, slots % self.bs].double().cpu()
        at = 0
        for s, n in tokens.items():
            old = self.hist.get(s, (kr[:0], kr[:0]))
            self.hist[s] = (torch.cat([old[0], kr[at:at + n]]),
                            torch.cat([old[1], v[at:at + n].double().cpu()]))
            at += n
        return q

    def tables(self, seqs):
        mb = max(len(self.bm.seq_blocks(s)) for s in seqs)
        return (torch.from_numpy(self.bm.block_table(seqs, mb)).to(DEV),
                torch.tensor([self.bm.seq_len(s) for s in seqs], dtype=torch.int32, device=DEV))

    def check(self, out, q, tokens):
        """Half a step of the output plus 2^-13 of the largest value (the bound
        of the windowed tests)."""
        gq, at = self.Hq // self.Hkv, 0
        for s, n in tokens.items():
            k, v = (x.repeat_interleave(gq, 1) for x in self.hist[s])
            L = k.shape[0]
            j, p = torch.arange(L), torch.arange(L - n, L)[:, None]
            sees = (j <= p) & ((j < self.S) | (j > p - self.W))
            w = torch.einsum("nhd,jhd->hnj", q[at:at + n].double().cpu(), k) * self.d ** -0.5
            ref = torch.einsum("hnj,jhd->nhd", w.masked_fill(~sees, -float("inf")).softmax(-1), v)
            err = (out[at:at + n].double().cpu() - ref).abs()
            assert bool((err <= 2.0 ** -8 * ref.abs() + 2.0 ** -13 * v.abs().max()).all()), float(err.max())
            at += n

    def prefill(self, tokens):
        from paged_kv_cache_192_gb300 import ops
        q = self.store(tokens)
        table, lens = self.tables(list(tokens))
        start = torch.tensor([0] + list(np.cumsum(list(tokens.values()))), dtype=torch.int32, device=DEV)
        out = ops.prefill_window(q, self.k, self.v, table, start, lens, max(tokens.values()), self.W, self.S)
        self.check(out, q, tokens)
        self.trim(tokens)

    def decode(self, seqs):
        from paged_kv_cache_192_gb300 import ops
        q = self.store({s: 1 for s in seqs})
        table, lens = self.tables(seqs)
        out = ops.decode_window(q, self.k, self.v, table, lens, self.W, self.S)
        self.check(out, q, {s: 1 for s in seqs})
        self.trim(seqs)
        return q, out

    def trim(self, seqs):
        for s in seqs:
            self.bm.trim(s, self.W, self.S)


def test_serving_loop_in_a_pool_that_only_holds_the_windows():
    from paged_kv_cache_192_gb300 import ops
    # three sequences of about 200 tokens need 75 pages whole; sinks, window and
    # a chunk of up to 41 tokens fit in 14 each
    lp = Loop(num_blocks=42)
    lens = {0: 200, 1: 173, 2: 90}
    for s in lens:
        lp.bm.add_seq(s, 0)
    done = {s: 0 for s in lens}
    while any(done[s] < n for s, n in lens.items()):
        chunk = {s: min(n - done[s], 41 - 7 * s) for s, n in lens.items() if done[s] < n}
        lp.prefill(chunk)
        for s, n in chunk.items():
            done[s] += n
    for _ in range(20):
        lp.decode([0, 1, 2])
    # a branch of sequence 1 shares its pages and writes its own copy of the last
    lp.bm.fork(1, 7)
    lp.hist[7] = lp.hist[1]
    for _ in range(11):
        lp.decode([0, 7, 1, 2])
    assert ops.device_error() == 0
    # every sequence keeps its sinks and window: plain decode then sees the same
    seqs = [0, 1, 2, 7]
    table, L = lp.tables(seqs)
    q = lp.rand(4, lp.Hq, lp.d)
    want = ops.decode_window(q, lp.k, lp.v, table, L, lp.W, lp.S)
    n = lp.S + lp.W
    keep = np.stack([np.concatenate([np.arange(lp.S), np.arange(int(x) - lp.W, int(x))]) for x in L.cpu()])
    keep = torch.from_numpy(np.repeat(keep[:, None], lp.Hkv, 1).astype(np.int32)).to(DEV)
    ops.set_validate(True)
    try:
        for i, s in enumerate(seqs):  # one at a time: the pool has no room for all the fresh pages
            src = table[i:i + 1].contiguous()
            lp.bm.compact([s], [n])
            ops.compact_cache(lp.k, lp.v, src, lp.tables([s])[0], keep[i:i + 1].contiguous(),
                              torch.tensor([n], dtype=torch.int32, device=DEV))
    finally:
        ops.set_validate(False)
    dst, new_lens = lp.tables(seqs)
    assert new_lens.tolist() == [n] * 4 and (dst >= 0).all()
    got = ops.decode(q, lp.k, lp.v, dst, new_lens)
    # both are within the bound of the exact result: twice it from each other
    vmax = max(float(v.abs().max()) for _, v in lp.hist.values())
    assert bool(((got.double() - want.double()).abs() <= 2.0 ** -7 * want.double().abs() + 2.0 ** -12 * vmax).all())
    assert lp.bm.num_free() == 42 - 4 * 7 and ops.device_error() == 0
    # and the sequences go on from there, through the plain calls
    slots = torch.tensor([lp.bm.append(s)[0] for s in seqs], dtype=torch.int64, device=DEV)
    kn, vn = lp.rand(4, lp.Hkv, lp.d), lp.rand(4, lp.Hkv, lp.d)
    ops.reshape_and_cache(kn, vn, lp.k, lp.v, slots)
    table, L = lp.tables(seqs)
    a = ops.decode(q, lp.k, lp.v, table, L)
    b = ops.decode_window(q, lp.k, lp.v, table, L, n + 1)
    assert bool(((a.double() - b.double()).abs() <= 2.0 ** -7 * b.double().abs() + 2.0 ** -12 * max(vmax, float(vn.abs().max()))).all())
    assert ops.device_error() == 0


def test_decode_step_captured_as_one_graph():
    """Store and windowed decode of a batch with two padding rows, captured
    once and replayed with new tokens in the same buffers."""
    from paged_kv_cache_192_gb300 import ops
    lp = Loop(num_blocks=64)
    for s in (0, 1, 2):
        lp.bm.add_seq(s, 0)
    lp.prefill({0: 90, 1: 33, 2: 61})
    B = 5
    MB = 24
    q, k, v = (torch.zeros(B, h, lp.d, dtype=bf16, device=DEV) for h in (lp.Hq, lp.Hkv, lp.Hkv))
    slots = torch.full((B,), -1, dtype=torch.int64, device=DEV)
    pos = torch.zeros(B, dtype=torch.int64, device=DEV)
    table = torch.zeros(B, MB, dtype=torch.int32, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)

    def step():
        r = ops.rope_reshape_and_cache(q, k, v, lp.k, lp.v, slots, pos, lp.inv)
        return r, ops.decode_window(r, lp.k, lp.v, table, lens, lp.W, lp.S)

    step()  # with padding only
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rot, out = step()
    for _ in range(12):
        rows = [0, 2, 4]  # rows 1 and 3 are padding
        for r, s in zip(rows, (0, 1, 2)):
            slot, _, _ = lp.bm.append(s)
            slots[r], pos[r] = slot, lp.bm.seq_len(s) - 1
            lens[r] = lp.bm.seq_len(s)
            row = lp.bm.block_table([s], MB)
            table[r] = torch.from_numpy(row[0]).to(DEV)
        for t in (q, k, v):
            t.copy_(lp.rand(*t.shape))
        g.replay()
        torch.cuda.synchronize()
        for r, s in zip(rows, (0, 1, 2)):
            kr = lp.k[slots[r] // lp.bs, :, slots[r] % lp.bs].double().cpu()[None]
            lp.hist[s] = (torch.cat([lp.hist[s][0], kr]), torch.cat([lp.hist[s][1], v[r:r + 1].double().cpu()]))
            lp.check(out[r:r + 1], rot[r:r + 1], {s: 1})
        assert not out[[1, 3]].any()
        lp.trim([0, 1, 2])
    assert ops.device_error() == 0


FIRST_CALLS = """
import sys, torch
sys.path.insert(0, {root!r})
from paged_kv_cache_192_gb300 import ops
dev, bf16 = "cuda", torch.bfloat16
g = torch.Generator().manual_seed(1)
R = lambda *s: torch.randn(*s, generator=g).to(bf16).to(dev)
k, v = R(64, 2, 16, 128), R(64, 2, 16, 128)
table = torch.arange(60, dtype=torch.int32, device=dev).view(2, 30)
lens = torch.tensor([470, 33], dtype=torch.int32, device=dev)
start = torch.tensor([0, 40, 73], dtype=torch.int32, device=dev)
q, qp = R(2, 8, 128), R(73, 8, 128)
kn, vn = R(2, 2, 128), R(2, 2, 128)
slots = torch.tensor([1000, 1001], device=dev)
pos = torch.tensor([5, 6], device=dev)
inv = torch.ones(64, device=dev)
keep = torch.arange(0, 40, 2, dtype=torch.int32, device=dev).expand(2, 2, -1).contiguous()
kl = torch.tensor([20, 10], dtype=torch.int32, device=dev)
dst = torch.arange(60, 64, dtype=torch.int32, device=dev).view(2, 2)
def calls():
    a = ops.rope_reshape_and_cache(q, kn, vn, k, v, slots, pos, inv)
    ops.compact_cache(k, v, table, dst, keep, kl)
    return a, ops.decode_window(q, k, v, table, lens, 200, 4), ops.prefill_window(
        qp, k, v, table, start, lens, 40, 200, 4)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = calls()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(captured, calls()))
assert ops.device_error() == 0
# two threads, a stream each
import threading
bad = []
def work():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.default_stream())
    with torch.cuda.stream(s):
        for _ in range(50):
            o = ops.decode_window(q, k, v, table, lens, 200, 4), ops.prefill_window(
                qp, k, v, table, start, lens, 40, 200, 4)
            s.synchronize()
            if not (torch.equal(o[0], captured[1]) and torch.equal(o[1], captured[2])):
                bad.append(1)
threads = [threading.Thread(target=work) for _ in range(3)]
for t in threads: t.start()
for t in threads: t.join()
assert not bad and ops.device_error() == 0
print("ok")
"""


def test_first_calls_of_a_process_may_be_captured():
    """Nothing has to be called before a capture; and threads may call at once."""
    import subprocess
    import sys

    from conftest import ROOT
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(root=ROOT)], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr


def test_positions_go_on_behind_a_compaction():
    """A compaction shortens a sequence's rows, not its positions: the next
    tokens are rotated by how many tokens the sequence has had, which the caller
    counts, and the plain call then equals attention over the kept tokens at
    their own positions.  (seq_len, the row count, as the position does not.)

    fp32.  Bound: the library's 1e-5 + 1e-5 |o|, and the rotations': an element
    is off by at most 6 steps of 2^-24 of its pair (two products, a sum, sine and
    cosine to 2^-22), a score by 2 * 6 * 2^-24 * sum |q| |k| * scale < 2.3e-5
    (sum below 256 here), twice that relative in a weight with its sum, times
    max |v| (below 6): 2.8e-4."""
    from paged_kv_cache_192_gb300 import ops
    lp = Loop(num_blocks=64, dtype=torch.float32)
    lens, n, more = {0: 90, 1: 61}, {0: 40, 1: 17}, 3
    raw = {s: [] for s in lens}  # (k, v) of each token before its rotation

    def put(s, count, first):
        sl, _ = lp.bm.append_n(s, count)
        q, k, v = lp.rand(count, lp.Hq, lp.d), lp.rand(count, lp.Hkv, lp.d), lp.rand(count, lp.Hkv, lp.d)
        raw[s] += list(zip(k.double().cpu(), v.double().cpu()))
        pos = torch.arange(first, first + count, device=DEV)
        r = ops.rope_reshape_and_cache(q, k, v, lp.k, lp.v, torch.from_numpy(sl).to(DEV), pos, lp.inv)
        return q.double().cpu(), r

    def turned(x, p):
        a = p * lp.inv.double().cpu()
        x0, x1 = x[..., :lp.d // 2], x[..., lp.d // 2:]
        return torch.cat([x0 * a.cos() - x1 * a.sin(), x0 * a.sin() + x1 * a.cos()], -1)

    for s, L in lens.items():
        lp.bm.add_seq(s, 0)
        put(s, L, 0)
    seqs, rng = list(lens), np.random.default_rng(3)
    keep = np.zeros((2, lp.Hkv, max(n.values())), dtype=np.int32)
    for s in seqs:
        for h in range(lp.Hkv):
            keep[s, h, :n[s]] = np.sort(rng.permutation(lens[s])[:n[s]])
    src, _ = lp.tables(seqs)
    lp.bm.compact(seqs, [n[s] for s in seqs])
    dst, rows = lp.tables(seqs)
    assert rows.tolist() == [40, 17]
    ops.compact_cache(lp.k, lp.v, src, dst, torch.from_numpy(keep).to(DEV), rows)

    def formula(s, q, p, shift):
        """The query at position p over the kept tokens and the new ones up to
        itself; shift: how far the new tokens' positions are off."""
        out = torch.zeros(lp.Hq, lp.d, dtype=torch.float64)
        for h in range(lp.Hkv):
            at = [int(j) for j in keep[s, h, :n[s]]] + list(range(lens[s], p + 1))
            k = torch.stack([turned(raw[s][j][0][h], j - (shift if j >= lens[s] else 0)) for j in at])
            v = torch.stack([raw[s][j][1][h] for j in at])
            for x in range(h * lp.Hq // lp.Hkv, (h + 1) * lp.Hq // lp.Hkv):
                out[x] = torch.softmax(k @ turned(q[x], p - shift) * lp.d ** -0.5, 0) @ v
        return out

    for step in range(more):
        for s in seqs:
            p = lens[s] + step
            q, r = put(s, 1, p)
            table, L = lp.tables([s])
            assert int(L) == n[s] + step + 1
            got = ops.decode(r, lp.k, lp.v, table, L)[0].double().cpu()
            windowed = ops.decode_window(r, lp.k, lp.v, table, L, int(L))[0].double().cpu()
            ref = formula(s, q[0], p, 0)
            tol = 1e-5 + 1e-5 * ref.abs() + 2.8e-4
            assert bool(((got - ref).abs() <= tol).all()) and bool(((windowed - ref).abs() <= tol).all())
            assert float((formula(s, q[0], p, lens[s] - n[s]) - ref).abs().max()) > 0.01
    assert ops.device_error() == 0


def test_captured_branches_that_join():
    """A graph whose two branches (streams) run the calls side by side, fork
    from a call and join into one: every node has more than one neighbour."""
    from paged_kv_cache_192_gb300 import ops
    lp = Loop(num_blocks=64)
    for s in (0, 1):
        lp.bm.add_seq(s, 0)
    lp.store({0: 150, 1: 77})
    table, lens = lp.tables([0, 1])
    q, kn, vn = lp.rand(2, lp.Hq, lp.d), lp.rand(2, lp.Hkv, lp.d), lp.rand(2, lp.Hkv, lp.d)
    qp = lp.rand(40, lp.Hq, lp.d)
    start = torch.tensor([0, 30, 40], dtype=torch.int32, device=DEV)
    unused = [b for b in range(64) if b not in lp.bm.seq_blocks(0) + lp.bm.seq_blocks(1)]
    slots = torch.tensor([0, 1], dtype=torch.int64, device=DEV) + unused[4] * lp.bs
    pos = torch.tensor([150, 77], dtype=torch.int64, device=DEV)
    free = unused[:4]
    dst = torch.tensor(free, dtype=torch.int32, device=DEV).view(2, 2)
    keep = torch.arange(0, 32, 2, dtype=torch.int32, device=DEV).expand(2, lp.Hkv, -1).contiguous()
    n = torch.tensor([16, 9], dtype=torch.int32, device=DEV)

    def branches(side):
        main = torch.cuda.current_stream()
        r = ops.rope_reshape_and_cache(q, kn, vn, lp.k, lp.v, slots, pos, lp.inv)
        side.wait_stream(main)
        a = ops.decode_window(r, lp.k, lp.v, table, lens, lp.W, lp.S)
        with torch.cuda.stream(side):
            b = ops.prefill_window(qp, lp.k, lp.v, table, start, lens, 30, lp.W, lp.S)
            ops.compact_cache(lp.k, lp.v, table, dst, keep, n)
        main.wait_stream(side)
        return r, a, b, ops.decode_window(r, lp.k, lp.v, dst, n, lp.W, lp.S)

    side = torch.cuda.Stream()
    eager = branches(side)
    torch.cuda.synchronize()
    for b in free:
        lp.k[b], lp.v[b] = 0, 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = branches(side)
    for _ in range(3):
        for o in captured:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(captured, eager))
    assert ops.device_error() == 0


@pytest.mark.parametrize("R", [3, 300])
def test_requests_without_new_tokens_leave_the_output(R):
    from paged_kv_cache_192_gb300 import ops
    lp = Loop(num_blocks=8)
    out = torch.full((10, lp.Hq, lp.d), 3.0, dtype=bf16, device=DEV)
    table = torch.full((R, 2), -1, dtype=torch.int32, device=DEV)
    zero = torch.zeros(R + 1, dtype=torch.int32, device=DEV)
    assert ops.prefill_window_kernel_for(R, 10, 16, lp.Hq, lp.Hkv) == ("split" if R == 3 else "persistent")
    ops.prefill_window(torch.zeros_like(out), lp.k, lp.v, table, zero, zero[:R] + 7, 16, lp.W, lp.S, out=out)
    torch.cuda.synchronize()
    assert (out == 3.0).all() and ops.device_error() == 0


def test_stores_and_compactions_from_several_threads():
    """Each thread its stream, pools and tokens; the same bits as alone."""
    import threading

    from paged_kv_cache_192_gb300 import ops
    g = torch.Generator().manual_seed(2)
    R = lambda *s: torch.randn(*s, generator=g).to(bf16).to(DEV)  # noqa: E731
    q, kn, vn = R(200, 8, 128), R(200, 2, 128), R(200, 2, 128)
    inv = torch.rand(64, generator=g).to(DEV)
    slots = torch.randperm(256, generator=g)[:200].to(DEV)
    pos = torch.arange(200, device=DEV)
    table = torch.arange(16, dtype=torch.int32, device=DEV).view(1, 16)
    keep = torch.arange(1, 256, 3, dtype=torch.int32, device=DEV).expand(1, 2, -1).contiguous()
    n = torch.tensor([keep.shape[2]], dtype=torch.int32, device=DEV)
    base = R(16, 2, 16, 128)

    def work():
        k, v = base.clone(), base.clone()
        r = ops.rope_reshape_and_cache(q, kn, vn, k, v, slots, pos, inv)
        ops.compact_cache(k, v, table, table, keep, n)
        return r, k, v
    want = work()
    torch.cuda.synchronize()
    bad = []

    def run():
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.default_stream())
        with torch.cuda.stream(s):
            for _ in range(40):
                got = work()
                s.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want)):
                    bad.append(1)
    threads = [threading.Thread(target=run) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and ops.device_error() == 0
