"""The calls of a serving step together: a plan on the device, the rotary store into
its slots, windowed attention over its tables, attention to an encoder's states whose
pages were planned the same way, linear attention whose states follow the sequences;
prompts, single tokens from a captured graph, dropped drafts, ended sequences."""
import pytest
import torch

from linear_util import Linear

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16
S, HQ, HKV, D, BS, W = 6, 8, 2, 64, 16, 48  # sequences; heads; window


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_192_gb300 import build
    build.build()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def near(got, ref, rest):
    """Half a step of the output and `rest` (the bounds of the operators' own tests)."""
    worst = float(((got.double() - ref).abs() / (2.0 ** -8 * ref.abs() + rest + 1e-30)).max())
    assert worst <= 1, f"{worst:.3f} of the bound"


class Serving:
    def __init__(self, seed=0):
        from paged_kv_cache_192_gb300 import layout
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.NB = 60
        self.pages = layout.page_state(S, 20, self.NB)
        self.k_cache, self.v_cache = layout.alloc_pools(self.NB, HKV, BS, D, bf16)
        self.enc_pages = layout.page_state(S, 10, 40)
        self.ek, self.ev = layout.alloc_pools(40, HKV, BS, D, bf16)
        self.states = torch.full((S, 4, D, D), float("nan"), device="cuda")
        self.decay = torch.tensor([0.0, -0.01, -0.3, -2.0], device="cuda")
        self.freq = torch.zeros(D // 2, device="cuda")  # (rotations have tests of their own)
        self.K, self.V = {s: [] for s in range(S)}, {s: [] for s in range(S)}   # what each sequence holds
        self.E, self.L = {}, {s: [] for s in range(S)}                           # encoder states, linear inputs

    def rand(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda", dtype=torch.float32).to(bf16)

    def encode(self, lens):
        """Encoder states of every sequence (0: none) into planned pages; -: ended."""
        from paged_kv_cache_192_gb300 import ops
        n = sum(max(0, x) for x in lens)
        plan = ops.plan_step(self.enc_pages, ints(range(S)), ints(lens), BS, n)
        k, v = self.rand(n, HKV, D), self.rand(n, HKV, D)
        ops.reshape_and_cache(k, v, self.ek, self.ev, plan.slots)
        at = 0
        for s, x in enumerate(lens):
            if x > 0:
                self.E[s] = (k[at:at + x], v[at:at + x])
                at += x
        return plan

    def inputs(self, T):
        return dict(q=self.rand(T, HQ, D), k=self.rand(T, HKV, D), v=self.rand(T, HKV, D), lin=self.rand(T, 3, 4, D))

    def step(self, ids, change, T, x, most, enc, out=None):
        """One step's calls; rows of padding and slots behind the last token included."""
        from paged_kv_cache_192_gb300 import ops
        plan = ops.plan_step(self.pages, ids, change, BS, T, out=out)
        q = ops.rope_reshape_and_cache(x["q"], x["k"], x["v"], self.k_cache, self.v_cache, plan.slots,
                                       plan.positions, self.freq)
        o = ops.prefill_window(q, self.k_cache, self.v_cache, plan.block_table, plan.query_start,
                               plan.context_lens, most, W)
        # the encoder tables of the step's rows
        c = ops.cross_attention(o, self.ek, self.ev, enc[0], plan.query_start, enc[1], most)
        lq, lk, lv = x["lin"].unbind(1)
        z = ops.linear_prefill(lq, lk, lv, self.states, ids, plan.query_start, plan.context_lens, most, self.decay)
        return plan, o, c, z

    def attend(self, q, k, v):
        """q [n][HQ][D] at the ends of prefixes of k, v [L][HKV][D], through the window."""
        L, n = len(k), len(q)
        pos, j = torch.arange(L - n, L, device="cuda")[:, None], torch.arange(L, device="cuda")
        s = torch.einsum("nhd,jhd->hnj", q.double(), k.double().repeat_interleave(HQ // HKV, 1)) * D ** -0.5
        s = s.masked_fill((j > pos) | (j <= pos - W), -float("inf"))
        return torch.einsum("hnj,jhd->nhd", s.softmax(-1), v.double().repeat_interleave(HQ // HKV, 1))

    def check(self, ids, change, x, plan, o, c, z):
        at = 0
        for s, n in zip(ids, change):
            if s < 0:
                continue
            if n <= 0:
                keep = max(0, len(self.K[s]) + n)
                for held in (self.K, self.V, self.L):
                    held[s] = held[s][:keep]
                continue
            r = slice(at, at + n)
            at += n
            # (copies: the buffers of a captured step take the next inputs)
            self.K[s] += list(x["k"][r].clone())
            self.V[s] += list(x["v"][r].clone())
            self.L[s] += list(x["lin"][r].clone())
            k, v = torch.stack(self.K[s]), torch.stack(self.V[s])
            ref = self.attend(x["q"][r], k, v)
            near(o[r], ref, 2.0 ** -13 * v.abs().max())
            if s in self.E:
                ek, ev = self.E[s]
                w = torch.einsum("nhd,jhd->hnj", o[r].double(), ek.double().repeat_interleave(HQ // HKV, 1)) * D ** -0.5
                ref = torch.einsum("hnj,jhd->nhd", w.softmax(-1), ev.double().repeat_interleave(HQ // HKV, 1))
                near(c[r], ref, 2.0 ** -13 * ev.abs().max())
            else:
                assert bool((c[r] == 0).all())
            lin = torch.stack(self.L[s]).double()
            i = torch.arange(len(lin), device="cuda")
            dec = torch.where(i[:, None] >= i, ((i[:, None] - i).clamp(min=0) * self.decay.double()[:, None, None]).exp(), 0.0)
            a = torch.einsum("ihd,jhd->hij", lin[:, 0], lin[:, 1]) * dec * D ** -0.5
            ref = torch.einsum("hij,jhd->ihd", a, lin[:, 2])[-n:]
            amount = torch.einsum("hij,jhd->ihd", torch.einsum("ihd,jhd->hij", lin[:, 0].abs(), lin[:, 1].abs()) * dec,
                                  lin[:, 2].abs())[-n:] * D ** -0.5
            near(z[r], ref, 2.0 ** -14 * amount)
        assert plan.query_start[-1] == at


def run(sv, ids, change, enc_lens, most=None):
    """A step without a graph, checked."""
    T = sum(max(0, c) for s, c in zip(ids, change) if s >= 0)
    x = sv.inputs(T + 2)
    table = torch.zeros(len(ids), 10, dtype=torch.int32, device="cuda")
    lens = [0] * len(ids)
    for i, s in enumerate(ids):
        if s >= 0:
            table[i] = sv.enc_pages.seq_pages[s]
            lens[i] = enc_lens[s]
    got = sv.step(ints(ids), ints(change), T + 2, x, most or max(1, max(change)), (table, ints(lens)))
    torch.cuda.synchronize()
    sv.check(ids, change, x, *got)


def test_sequences_come_grow_shrink_and_go():
    from paged_kv_cache_192_gb300 import ops
    sv = Serving()
    enc = [33, 0, 100, 1, 16, 64]
    sv.encode(enc)
    # prompts, one of them long; then decodes, drafts, rejected drafts, ends, new sequences
    for ids, change in (([0, 1, 2], [5, 130, 17]), ([0, -1, 2, 1], [1, 1, 1, 1]), ([3, 0, 4], [64, 8, 65]),
                        ([0, 3, 4, 1, 2], [-5, 1, 1, 1, 1]), ([1, 0], [-10 ** 6, 1]), ([1, 5, 2], [3, 80, -200]),
                        ([2, 1, 5, 4, 3, 0], [1] * 6), ([2, 1, 5, 4, 3, 0], [9, 1, 2, 1, 10, 1])):
        run(sv, ids, change, enc)
        # a sequence that gave up tokens starts its linear state anew: the state has seen
        # the dropped ones (a user keeps copies, or drops whole sequences)
        for s, c in zip(ids, change):
            if s >= 0 and c < 0 and len(sv.L[s]):
                lin = torch.stack(sv.L[s])
                one = torch.tensor([s], dtype=torch.int32, device="cuda")
                start, n = ints([0, len(lin)]), ints([len(lin)])
                ops.linear_prefill(*lin.unbind(1), sv.states, one, start, n, len(lin), sv.decay)
    sv.encode([-x for x in enc])
    assert sv.enc_pages.free_state.tolist()[1:] == [40, 0, 0]
    assert ops.device_error() == 0


def test_captured_decode_loop():
    """Forty replays of one step, rows of padding among them, each checked; no host work
    but new inputs."""
    from paged_kv_cache_192_gb300 import ops
    sv = Serving(1)
    enc = [20, 47, 0, 160, 5, 1]
    sv.encode(enc)
    run(sv, [0, 1, 2, 3], [7, 50, 16, 90], enc)
    ids, change = [3, -1, 0, 2, 1], [1, 1, 1, 1, 1]
    ids_t, change_t = ints(ids), ints(change)
    table = torch.stack([sv.enc_pages.seq_pages[max(s, 0)] for s in ids]).contiguous()
    lens = ints([enc[s] if s >= 0 else 0 for s in ids])
    x = sv.inputs(6)
    keep = [t.clone() for t in sv.pages], sv.states.clone(), sv.k_cache.clone(), sv.v_cache.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sv.step(ids_t, change_t, 6, x, 1, (table, lens))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = sv.step(ids_t, change_t, 6, x, 1, (table, lens))
    for t, old in zip(list(sv.pages) + [sv.states, sv.k_cache, sv.v_cache], list(keep[0]) + list(keep[1:])):
        t.copy_(old)
    for i in range(40):
        for name, t in sv.inputs(6).items():
            x[name].copy_(t)
        g.replay()
        torch.cuda.synchronize()
        sv.check(ids, change, x, *got)
    assert sv.pages.seq_lens.tolist() == [47, 90, 56, 130, 0, 0]
    assert ops.device_error() == 0


def test_a_refused_step_leaves_everything():
    """Too few pages: no token is stored, nothing advances, the calls behind run on what
    there was."""
    from paged_kv_cache_192_gb300 import ops
    sv = Serving(2)
    enc = [0] * S
    run(sv, [0, 1], [100, 40], enc)
    before = [t.clone() for t in (sv.k_cache, sv.v_cache, sv.states)] + [t.clone() for t in sv.pages[:3]]
    x = sv.inputs(1003)
    table, lens = torch.zeros(3, 10, dtype=torch.int32, device="cuda"), ints([0, 0, 0])
    plan, o, c, z = sv.step(ints([0, 2, 1]), ints([1, 1000, 1]), 1003, x, 1000, (table, lens))
    torch.cuda.synchronize()
    assert ops.device_error() == 8
    assert plan.query_start.tolist() == [0] * 4 and plan.context_lens.tolist() == [100, 0, 40]
    assert set(plan.slots.tolist()) == {-1}
    after = [sv.k_cache, sv.v_cache, sv.states] + list(sv.pages[:3])
    for a, b in zip(after, before):
        assert torch.equal(a.view(torch.int16) if a.dtype == bf16 else a.view(torch.int32),
                           b.view(torch.int16) if b.dtype == bf16 else b.view(torch.int32))
    run(sv, [0, 2, 1], [1, 60, 1], enc)
    assert ops.device_error() == 0


def test_linear_prompts_and_tokens_through_a_plan():
    """Long prompts, then single tokens by pa_linear_decode with the plan's lengths."""
    from paged_kv_cache_192_gb300 import layout, ops
    pages = layout.page_state(4, 300, 600)
    x = Linear([700, 90], [0, 0], H=3, d=128, ids=[2, 0], num_states=4)
    plan = ops.plan_step(pages, x.ids_t, ints([700, 90]), BS, 790)
    out = ops.linear_prefill(x.q, x.k, x.v, x.states, x.ids_t, plan.query_start, plan.context_lens, 700, x.decay_t)
    x.check(out, terms=(2.0 ** -15, 2.0 ** -18))
    y = Linear([1, 1], [700, 90], H=3, d=128, ids=[2, 0], num_states=4, seed=5)
    y.states, y.states0 = x.states, x.states.cpu()
    plan = ops.plan_step(pages, y.ids_t, ints([1, 1]), BS, 2)
    y.check(ops.linear_decode(y.q, y.k, y.v, y.states, y.ids_t, plan.context_lens, y.decay_t))
    assert ops.device_error() == 0


FIRST_CALLS = """
import sys, torch
sys.path.insert(0, {root!r})
from paged_kv_cache_192_gb300 import layout, ops
dev, bf16 = "cuda", torch.bfloat16
g = torch.Generator().manual_seed(1)
R = lambda *s: torch.randn(*s, generator=g).to(bf16).to(dev)
ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
k, v = R(64, 2, 16, 128), R(64, 2, 16, 128)
table = torch.arange(60, dtype=torch.int32, device=dev).view(2, 30)
enc, one, many = ints([470, 33]), ints([0, 1, 3]), ints([0, 40, 140])
q1, q2 = R(3, 8, 128), R(140, 8, 128)
x1, x2 = R(2, 3, 2, 128), R(3000, 3, 2, 128)
ids, lens1, start, lens2, decay = ints([1, 0]), ints([5, 1]), ints([0, 2500, 3000]), ints([2500, 600]), torch.tensor([-0.1, 0.0], device=dev)
first = torch.randn(2, 2, 128, 128, generator=g).to(dev)
seqs, grow, shrink = ints([2, -1, 0]), ints([20, 7, 3]), ints([-20, 0, -3])
base = layout.page_state(3, 8, 30)
def calls():
    pages = ops.PageState(*(t.clone() for t in base))
    state = [first.clone(), first.clone()]
    p = ops.plan_step(pages, seqs, grow, 16, 25), ops.plan_step(pages, seqs, shrink, 16, 1)
    c = ops.cross_attention(q1, k, v, table, one, enc, 2), ops.cross_attention(q2, k, v, table, many, enc, 100)
    o = ops.linear_decode(*x1.unbind(1), state[0], ids, lens1, decay)
    z = ops.linear_prefill(*x2.unbind(1), state[1], ids, start, lens2, 2500, decay)
    return list(p[0]) + list(p[1]) + list(c) + [o, z] + state + list(pages)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = calls()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(captured, calls()))
assert ops.device_error() == 0
# threads, a stream each
import threading
bad = []
def work():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.default_stream())
    with torch.cuda.stream(s):
        for _ in range(40):
            got = calls()
            s.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(captured, got)):
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
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(root=ROOT)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr


def test_captured_branches_that_join():
    """Two branches side by side, forked behind a plan and joined into a call: every node
    has more than one neighbour."""
    from paged_kv_cache_192_gb300 import layout, ops
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(40, 2, 16, 64, generator=g).to(bf16).cuda() for _ in range(2))
    q, qs = torch.randn(140, 8, 64, generator=g).to(bf16).cuda(), torch.randn(2, 8, 64, generator=g).to(bf16).cuda()
    x = torch.randn(1602, 3, 2, 64, generator=g).to(bf16).cuda()
    enc, ids, decay = ints([300, 77]), ints([1, 0]), torch.tensor([-0.2, -0.001], device="cuda")
    first = torch.randn(2, 2, 64, 64, generator=g).cuda()
    pages, states = layout.page_state(2, 120, 240), first.clone()

    def branches(side):
        main = torch.cuda.current_stream()
        a = ops.plan_step(pages, ids, ints_grow, 16, 1602)
        side.wait_stream(main)
        b = ops.linear_prefill(*x.unbind(1), states, ids, a.query_start, a.context_lens, 1500, decay)
        with torch.cuda.stream(side):
            c = ops.cross_attention(q, k, v, tables, starts, enc, 100)
            d = ops.cross_attention(qs, k, v, tables, ones, enc, 1)
        main.wait_stream(side)
        e = ops.plan_step(pages, ids, ints_drop, 16, 1)
        f = ops.linear_decode(*x[:2].unbind(1), states, ids, e.context_lens, decay)
        return list(a) + [b, c, d] + list(e) + [f]

    ints_grow, ints_drop = ints([1500, 102]), ints([-1500, -100])
    tables, starts, ones = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20), ints([0, 100, 140]), ints([0, 1, 2])
    keep = [t.clone() for t in pages]
    side = torch.cuda.Stream()
    eager, after = branches(side), states.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = branches(side)
    for _ in range(3):
        for t, old in zip(pages, keep):
            t.copy_(old)
        states.copy_(first)
        for o in captured:
            o.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager)) and torch.equal(states, after)
    assert ops.device_error() == 0
