"""Single tokens of linear attention behind a plan: rows that gained no token (of refused
steps, padding, dropped drafts, sequences that wait) leave their states as they are."""
import pytest
import torch

from linear_util import Linear

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_192_gb300 import build
    build.build()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def decode(x, plan, ids=None, **kw):
    from paged_kv_cache_192_gb300 import ops
    return ops.linear_decode(x.q, x.k, x.v, x.states, x.ids_t if ids is None else ids, plan.context_lens, x.decay_t,
                             query_start=plan.query_start, **kw)


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int32), b.contiguous().view(torch.int32))


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("d", [64, 128])
def test_a_refused_step_leaves_the_states(dtype, d):
    """Also that of a sequence of one token, which must not start anew, and of one of none."""
    from paged_kv_cache_192_gb300 import layout, ops
    pages = layout.page_state(4, 4, 6)
    ops.plan_step(pages, ints([0, 1]), ints([1, 40]), 16, 41)
    x = Linear([1] * 3, [1, 40, 0], d=d, dtype=dtype, ids=[0, 1, 2], num_states=4)
    before = x.states.clone()
    plan = ops.plan_step(pages, ints([0, 1, 2]), ints([1, 1, 65]), 16, 70)  # five pages where two are free
    out = decode(x, plan)
    assert plan.context_lens.tolist() == [1, 40, 0] and ops.device_error() == 8
    assert bool((out == 0).all()) and same_bits(x.states, before)
    # the same tokens again, as a step that fits
    plan = ops.plan_step(pages, ints([0, 1, 2]), ints([1, 1, 1]), 16, 3)
    x.check(decode(x, plan))
    assert ops.device_error() == 0


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_rows_without_a_new_token(dtype):
    """Dropped drafts, a sequence that waits, padding: zeros and the old state; the token of
    another row is that row's."""
    from paged_kv_cache_192_gb300 import layout, ops
    pages = layout.page_state(6, 8, 40)
    ops.plan_step(pages, ints([0, 1, 2, 3]), ints([10, 20, 1, 30]), 16, 61)
    x = Linear([1, 0, 1, 0, 0, 1], [10, 0, 1, 0, 0, 0], dtype=dtype, ids=[0, 1, 2, -1, 3, 5], num_states=6)
    x.qkv = torch.randn(6, 3, 3, 64, device="cuda").to(dtype)
    x.q, x.k, x.v = x.qkv.unbind(1)
    plan = ops.plan_step(pages, ints([0, 1, 2, -1, 3, 5]), ints([1, -4, 1, 1, 0, 1]), 16, 6)
    assert plan.query_start.tolist() == [0, 1, 1, 2, 2, 2, 3]
    out = decode(x, plan)
    rows, idle = [0, 2, 5], [1, 3, 4]
    assert bool((out[idle] == 0).all())
    x.qkv, x.T, x.n, x.prior, x.ids = x.qkv[rows], 3, [1, 1, 1], [10, 1, 0], [0, 2, 5]
    x.check(out[rows])
    assert ops.device_error() == 0


def test_a_row_that_gained_more_than_one_token():
    """Recorded; zeros, its state as it was; the others are right."""
    from paged_kv_cache_192_gb300 import layout, ops
    pages = layout.page_state(3, 8, 20)
    x = Linear([1] * 3, [0, 0, 0], ids=[0, 1, 2], num_states=3)
    keep = x.states0[1] = torch.randn(3, 64, 64)
    x.states[1] = keep.cuda()
    plan = ops.plan_step(pages, x.ids_t, ints([1, 2, 1]), 16, 4)
    out = decode(x, plan)
    assert ops.device_error() == 4 and bool((out[1] == 0).all())
    x.ids[1] = -1
    x.check(out)


@pytest.mark.parametrize("start", [[0, 1, 0, 1], [0, 2 ** 31 - 1, 2 ** 31 - 1, 0], [5, 6, 9, 10]])
def test_prefix_sums_that_no_plan_writes(start):
    """A difference of one is a token, of none is none; others do not fit."""
    from paged_kv_cache_192_gb300 import ops
    x = Linear([1] * 3, [4, 4, 4], ids=[2, 0, 1], num_states=3)
    out = ops.linear_decode(x.q, x.k, x.v, x.states, x.ids_t, x.lens, x.decay_t, query_start=ints(start))
    ok = [b - a == 1 for a, b in zip(start, start[1:])]
    assert ops.device_error() == 4
    for r in range(3):
        if not ok[r]:
            assert bool((out[r] == 0).all())
            x.ids[r] = -1
    x.check(out)


def test_validate_mode():
    from paged_kv_cache_192_gb300 import _lib, layout, ops
    pages = layout.page_state(3, 8, 20)
    x = Linear([1] * 3, [0, 0, 0], ids=[0, 1, 2], num_states=3)
    ops.set_validate(True)
    try:
        plan = ops.plan_step(pages, x.ids_t, ints([1, 1, 1]), 16, 3)
        x.check(decode(x, plan))
        with pytest.raises(_lib.PAError, match="2 new tokens"):
            decode(x, plan._replace(query_start=ints([0, 1, 3, 4])))
        with pytest.raises(_lib.PAError, match="new tokens"):
            decode(x, plan._replace(query_start=ints([0, 1, 0, 1])))
    finally:
        ops.set_validate(False)


@pytest.mark.parametrize("B,H", [(1, 16), (64, 4), (300, 1)])
def test_rows_that_all_gained_one_have_the_same_bits(B, H):
    from paged_kv_cache_192_gb300 import ops
    x = Linear([1] * B, [i % 4 for i in range(B)], H=H, d=128)
    out = ops.linear_decode(x.q, x.k, x.v, x.states, x.ids_t, x.lens, x.decay_t, query_start=x.start)
    states = x.states.clone()
    x.check(out)
    x.states.copy_(x.states0)
    assert torch.equal(out, ops.linear_decode(x.q, x.k, x.v, x.states, x.ids_t, x.lens, x.decay_t))
    assert same_bits(states, x.states)


def test_a_captured_loop_that_runs_out_of_pages():
    """Plan, rotary store, windowed decode and linear decode in one graph.  Replays that do
    not fit leave pages, caches and states; when pages come back the loop goes on, and the
    states are those of the accepted tokens alone."""
    from paged_kv_cache_192_gb300 import layout, ops
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(bf16)
    pages = layout.page_state(4, 4, 5)
    kc, vc = layout.alloc_pools(5, 2, 16, 64, bf16)
    decay, freq = torch.tensor([-0.01, -0.7], device="cuda"), torch.zeros(32, device="cuda")
    states = torch.full((4, 2, 64, 64), float("nan"), device="cuda")
    ids, change = ints([2, 0, -1]), ints([1, 1, 1])
    x = dict(q=rand(3, 4, 64), k=rand(3, 2, 64), v=rand(3, 2, 64), lin=rand(3, 3, 2, 64))

    def step():
        plan = ops.plan_step(pages, ids, change, 16, 3)
        q = ops.rope_reshape_and_cache(x["q"], x["k"], x["v"], kc, vc, plan.slots, plan.positions, freq)
        o = ops.decode_window(q, kc, vc, plan.block_table, plan.context_lens, 64)
        z = ops.linear_decode(*x["lin"].unbind(1), states, ids, plan.context_lens, decay, query_start=plan.query_start)
        return plan, o, z

    first = [t.clone() for t in pages]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan, o, z = step()
    for t, old in zip(pages, first):
        t.copy_(old)
    ops.plan_step(pages, ints([1]), ints([40]), 16, 40)  # three of five pages: 16 tokens fit each row
    taken, refused = [], 0
    for i in range(30):
        for t in x.values():
            t.copy_(rand(*t.shape))
        if i == 22:
            ops.plan_step(pages, ints([1]), ints([-40]), 16, 0)
        before = [t.clone() for t in (kc, vc, states, *pages[:3])]
        graph.replay()
        torch.cuda.synchronize()
        if plan.query_start.tolist()[-1] == 0:
            refused += 1
            for a, b in zip((kc, vc, states, *pages[:3]), before):
                assert torch.equal(a.view(torch.int16) if a.dtype == bf16 else a.view(torch.int32),
                                   b.view(torch.int16) if b.dtype == bf16 else b.view(torch.int32))
            assert bool((z == 0).all())
            continue
        taken.append(x["lin"].clone())
        lin = torch.stack(taken).double()[:, :2]  # [n][row][3][H][d]
        n = len(lin)
        dec = (torch.arange(n - 1, -1, -1, device="cuda")[:, None].double() * decay.double()).exp()
        S = torch.einsum("nh,nrhi,nrhj->rhij", dec, lin[:, :, 1], lin[:, :, 2])
        A = torch.einsum("nh,nrhi,nrhj->rhij", dec, lin[:, :, 1].abs(), lin[:, :, 2].abs())
        assert bool(((states[[2, 0]] - S).abs() <= 2.0 ** -16 * A).all())  # (24 roundings and factors at most: 24 x 2^-21.6)
        ref = torch.einsum("rhi,rhij->rhj", lin[-1, :, 0], S) / 8
        tol = 2.0 ** -8 * ref.abs() + 2.0 ** -16 * torch.einsum("rhi,rhij->rhj", lin[-1, :, 0].abs(), A) / 8
        assert bool(((z[:2] - ref).abs() <= tol).all()) and bool((z[2] == 0).all())
    assert refused == 6 and len(taken) == 24 and pages.free_state[3] == 6
    assert ops.device_error() == 8
