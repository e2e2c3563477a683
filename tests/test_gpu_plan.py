"""pa_plan_step against a page-by-page model on the host: growth, dropped tokens,
padding, ring wraps, refusals that change nothing, tables of other widths, graphs,
streams; then the calls that read a plan."""
import random

import numpy as np
import pytest
import torch

from plan_util import Model, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_192_gb300 import build
    build.build()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def call(state, ids, change, bs, max_tokens, **kw):
    from paged_kv_cache_192_gb300 import ops
    return ops.plan_step(state, ints(ids), ints(change), bs, max_tokens, **kw)


def errors():
    from paged_kv_cache_192_gb300 import ops
    return ops.device_error()


@pytest.mark.parametrize("S,width,NB,bs,most", [
    (1, 4, 5, 16, 40), (7, 12, 60, 8, 60), (40, 33, 500, 16, 300), (40, 36, 900, 32, 300),
    (300, 20, 4000, 8, 100), (1500, 9, 6000, 16, 50), (5, 1024, 3000, 16, 9000), (3, 261, 600, 128, 9000)])
@pytest.mark.parametrize("seed", [0, 1])
def test_steps(S, width, NB, bs, most, seed):
    """Random steps: sequences grow, shrink, end; some steps do not fit."""
    rng = random.Random(seed * 1000 + S)
    order = list(range(NB))
    rng.shuffle(order)
    m = Model(S, width, NB, bs, order, first=rng.randrange(NB))
    state = m.state()
    refused = 0
    for _ in range(25):
        ids = rng.sample(range(S), rng.randint(1, S))
        for i in range(len(ids)):
            if rng.random() < 0.1:
                ids[i] = -rng.randint(1, 5)
        change = [rng.choice([1, 1, 0, rng.randint(1, most), -rng.randint(1, most), -2 ** 31]) for _ in ids]
        tokens = sum(max(0, c) for s, c in zip(ids, change) if s >= 0) + rng.choice([0, 0, 3, -1])
        tokens = max(0, tokens)
        plan = call(state, ids, change, bs, tokens)
        want, why = m.step(ids, change, tokens)
        same(plan, want)
        m.check(state)
        assert errors() == {None: 0, "request": 4, "blocks": 8}[why]
        refused += bool(why)
    assert refused < 25


@pytest.mark.parametrize("ids,change,max_tokens,W,bits", [
    ([0, 1, 0], [1, 1, 1], 3, 8, 4),          # a sequence twice
    ([0, 6], [1, 1], 2, 8, 4),                # no such sequence
    ([0, 2 ** 31 - 1], [1, 1], 2, 8, 4),
    ([0, 1], [1, 1], 1, 8, 8),                # more tokens than slots
    ([0, 1], [1, 200], 201, 8, 8),            # more than a table holds
    ([0, 1], [1, 2 ** 31 - 1], 2 ** 12, 8, 8),
    ([2, 3, 4, 5], [128] * 4, 512, 8, 8),     # more pages than are free
    ([0, 1], [1, 1], 2, 2, 8),                # a table too narrow for what is held
])
def test_refused_steps_change_nothing(ids, change, max_tokens, W, bits):
    m = Model(6, 8, 20, 16)
    m.step([0, 1], [33, 16], 49)
    state = m.state()
    before = [x.clone() for x in state]
    plan = call(state, ids, change, 16, max_tokens, table_blocks=W)
    want, why = m.step(ids, change, max_tokens, W)
    assert why == {4: "request", 8: "blocks"}[bits]
    same(plan, want)
    assert errors() == bits
    for a, b in zip(state[:3], before[:3]):
        assert torch.equal(a, b)
    assert state[3].tolist() == before[3].tolist()[:3] + [1]
    # and the next step that fits runs
    plan = call(state, [1, 0], [1, 2], 16, 3)
    same(plan, m.step([1, 0], [1, 2], 3)[0])
    m.check(state)
    assert errors() == 0


def test_two_rows_of_a_sequence_far_apart():
    """Rows of different warps, and CTAs that see them in any order: refused, every row
    shows what its sequence holds."""
    m = Model(600, 8, 6000, 8)
    m.step(list(range(600)), [1 + i % 60 for i in range(600)], 600 * 61)
    state = m.state()
    for _ in range(20):
        ids = list(range(600)) + [5, 17, 599, 3]
        plan = call(state, ids, [1] * 604, 8, 604)
        want, why = m.step(ids, [1] * 604, 604)
        assert why == "request"
        same(plan, want)
    m.check(state)
    assert errors() == 4


@pytest.mark.parametrize("word,value", [(0, -1), (0, 20), (1, -1), (1, 21)])
def test_a_ring_that_cannot_be(word, value):
    m = Model(6, 8, 20, 16)
    state = m.state()
    state[3][word] = value
    plan = call(state, [0, 1], [5, 40], 16, 45)
    assert errors() == 4
    assert plan.query_start.tolist() == [0, 0, 0] and set(plan.slots.tolist()) == {-1}
    assert state[3][word] == value and state[1].tolist() == [0] * 6


def test_more_given_back_than_the_pool_has_room_for():
    m = Model(2, 8, 20, 16)
    m.step([0], [100], 100)
    state = m.state()
    state[3][1] = 20  # says that all pages are free
    call(state, [0], [-100], 16, 0)
    assert errors() == 4 and state[1].tolist() == [100, 0]


def test_lengths_that_cannot_be():
    for L in (-1, 8 * 16 + 1, 2 ** 31 - 1):
        m = Model(2, 8, 20, 16)
        state = m.state()
        state[1][0] = L
        plan = call(state, [0, 1], [1, 1], 16, 2)
        assert errors() == 4
        assert plan.context_lens.tolist() == [0, 0] and plan.slots.tolist() == [-1, -1]


def test_pages_outside_the_pool_get_no_slot():
    m = Model(2, 8, 20, 16)
    state = m.state()
    state[2][0], state[2][1] = 20, -1
    plan = call(state, [0, 1], [3, 2], 16, 5)
    assert errors() == 1
    assert plan.slots.tolist() == [-1] * 5 and plan.positions.tolist() == [0, 1, 2, 0, 1]


@pytest.mark.parametrize("W", [3, 4, 8, 13])
def test_other_table_widths_and_given_outputs(W):
    """Narrower and wider tables than the sequences', outputs that hold something."""
    from paged_kv_cache_192_gb300 import ops
    m = Model(6, 8, 40, 16)
    m.step([0, 1, 2], [33, 16, 1], 50)
    state = m.state()
    out = ops.StepPlan(torch.full((4, W), -9, dtype=torch.int32, device="cuda"), ints([9] * 4), ints([9] * 5),
                       torch.full((20,), 9, dtype=torch.int64, device="cuda"),
                       torch.full((20,), 9, dtype=torch.int64, device="cuda"))
    plan = call(state, [2, -1, 0, 1], [16, 5, -2, 1], 16, 20, out=out)
    want, why = m.step([2, -1, 0, 1], [16, 5, -2, 1], 20, W)
    assert why is None and all(a.data_ptr() == b.data_ptr() for a, b in zip(plan, out))
    same(out, want)
    m.check(state)
    assert errors() == 0


def test_unaligned_tensors():
    """Views that do not start on 16 bytes take the narrow accesses."""
    from paged_kv_cache_192_gb300 import ops
    m = Model(5, 8, 40, 16)
    m.step([0, 1, 2], [33, 16, 1], 50)
    s = m.state()
    flat = torch.full((5 * 8 + 1,), -7, dtype=torch.int32, device="cuda")
    flat[1:] = s[0].view(-1)
    state = ops.PageState(flat[1:].view(5, 8), s[1], s[2], s[3])
    for ids, change in (([0, 1, 4], [1, 17, 100]), ([4, 0], [-60, 3])):
        n = sum(max(0, c) for c in change)
        same(call(state, ids, change, 16, n), m.step(ids, change, n)[0])
        m.check(state)


def test_empty_steps():
    m = Model(3, 4, 9, 16)
    state = m.state()
    plan = call(state, [], [], 16, 4)
    same(plan, m.step([], [], 4)[0])
    same(call(state, [-1], [7], 16, 0), m.step([-1], [7], 0)[0])
    m.check(state)
    assert errors() == 0


def test_the_largest_step():
    """4096 rows, and sequence ids past 2^18."""
    rng = random.Random(3)
    m = Model(2 ** 19, 4, 30000, 8)
    ids = rng.sample(range(2 ** 19), 4095) + [2 ** 19 - 1]
    if len(set(ids)) < 4096:
        ids[ids.index(2 ** 19 - 1)] = 0
    change = [rng.randint(0, 32) for _ in ids]
    state = m.state()
    n = sum(change)
    same(call(state, ids, change, 8, n), m.step(ids, change, n)[0])
    change = [rng.randint(-32, 0) for _ in ids]
    same(call(state, ids, change, 8, 0), m.step(ids, change, 0)[0])
    m.check(state)


def test_refusals_before_anything_runs():
    from paged_kv_cache_192_gb300 import _lib, ops
    m = Model(3, 4, 9, 16)
    state = m.state()
    with pytest.raises(_lib.PAError, match="at most 4096"):
        call(state, [-1] * 4097, [0] * 4097, 16, 0)
    with pytest.raises(_lib.PAError, match="block_size"):
        call(state, [0], [1], 24, 1)
    with pytest.raises(TypeError, match="seq_ids"):
        ops.plan_step(state, ints([0]).long(), ints([1]), 16, 1)
    with pytest.raises(ValueError, match="contiguous"):
        ops.plan_step(state, ints([0, 1, 2, 0])[::2], ints([1, 1]), 16, 1)
    with pytest.raises(ValueError, match="out must be"):
        call(state, [0], [1], 16, 1, out=call(state, [-1], [1], 16, 2))
    assert state[1].tolist() == [0, 0, 0]


@pytest.mark.parametrize("spoil,msg", [
    (lambda s, ids: ids.__setitem__(1, 0), "named twice"),
    (lambda s, ids: ids.__setitem__(1, 7), "outside"),
    (lambda s, ids: s[2].__setitem__(5, 6), "there twice"),
    (lambda s, ids: s[0].__setitem__((0, 0), 19), "used twice"),
    (lambda s, ids: s[0].__setitem__((0, 0), 20), "used twice"),
    (lambda s, ids: s[3].__setitem__(2, 1), "no state"),
    (lambda s, ids: s[1].__setitem__(2, -4), "length"),
])
def test_validate_mode(spoil, msg):
    from paged_kv_cache_192_gb300 import _lib, ops
    m = Model(6, 8, 20, 16)
    m.step([0, 1], [33, 16], 49)
    state, ids = m.state(), ints([0, 1])
    ops.set_validate(True)
    try:
        plan = ops.plan_step(state, ids, ints([1, 1]), 16, 2)
        same(plan, m.step([0, 1], [1, 1], 2)[0])
        spoil(state, ids)
        with pytest.raises(_lib.PAError, match=msg):
            ops.plan_step(state, ids, ints([1, 1]), 16, 2)
    finally:
        ops.set_validate(False)


def test_back_to_back_steps_and_other_streams():
    """A hundred steps that nothing waits between, half of them on another stream."""
    m = Model(64, 40, 2000, 16)
    state = m.state()
    ids, change = ints(range(64)), ints([1 + i % 7 for i in range(64)])
    n = int(change.sum())
    side = torch.cuda.Stream()
    from paged_kv_cache_192_gb300 import ops
    torch.cuda.synchronize()
    plans = []
    for i in range(50):
        plans.append(ops.plan_step(state, ids, change, 16, n))
    side.wait_stream(torch.cuda.current_stream())
    for i in range(25):
        plans.append(ops.plan_step(state, ids, change, 16, n, stream=side))
    with torch.cuda.stream(side):
        for i in range(25):
            plans.append(ops.plan_step(state, ids, -change, 16, 0))
    torch.cuda.synchronize()
    for i, p in enumerate(plans):
        c = change.tolist() if i < 75 else (-change).tolist()
        same(p, m.step(list(range(64)), c, n if i < 75 else 0)[0])
    m.check(state)
    assert errors() == 0


def test_captured_steps():
    from paged_kv_cache_192_gb300 import ops
    m = Model(8, 16, 200, 16)
    state = m.state()
    ids, change = ints([3, 1, -1, 7]), ints([1, 1, 1, 1])
    out = ops.plan_step(state, ids, change, 16, 4)
    m.step([3, 1, -1, 7], [1, 1, 1, 1], 4)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.plan_step(state, ids, change, 16, 4, out=out)
        ops.plan_step(state, ids, change, 16, 4, out=out)
    for _ in range(20):
        g.replay()
        torch.cuda.synchronize()
        m.step([3, 1, -1, 7], [1, 1, 1, 1], 4)
        same(out, m.step([3, 1, -1, 7], [1, 1, 1, 1], 4)[0])
    ids.copy_(ints([0, 3, 1, 2]))
    change.copy_(ints([17, -40, -3, 0]))
    g.replay()
    m.step([0, 3, 1, 2], [17, -40, -3, 0], 4)
    want, why = m.step([0, 3, 1, 2], [17, -40, -3, 0], 4)
    assert why == "blocks"  # 17 tokens, 4 slots
    same(out, want)
    m.check(state)
    assert errors() == 8
