"""Kernels whose warps hand tiles on to one another, under loads whose tiles land late and
out of order: many CTAs, each with more tiles than its ring has stages, call after call.
The split kernel of windowed prefills and cross attention has two groups that take every
other tile."""
import pytest
import torch

from window_util import Batch

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_192_gb300 import build
    build.build()


def repeat(call, times=4000):
    """Every call gives the first one's bits, and no wait runs out."""
    from paged_kv_cache_192_gb300 import ops
    first = call(None).clone()
    assert ops.device_error() == 0
    out, changed = torch.empty_like(first), torch.zeros((), dtype=torch.bool, device="cuda")
    for i in range(times):
        call(out)
        if i % 8 == 0:
            changed |= (out.view(torch.int16) != first.view(torch.int16)).any()
        if i % 500 == 499:
            assert ops.device_error() == 0
    assert not bool(changed)
    return first


@pytest.mark.parametrize("d", [64, 128])
def test_cross_attention(d):
    from paged_kv_cache_192_gb300 import ops
    from test_gpu_cross import Cross
    x = Cross([40] + [1] * 39, [3200, 0, 1, 63] * 10, Hq=4, Hkv=4, d=d, bs=64, seed=d)
    x.check(repeat(lambda out: ops.cross_attention(x.q_t, x.k_cache, x.v_cache, x.table_t, x.start_t, x.lens_t,
                                                   40, out=out)))


@pytest.mark.parametrize("d", [64, 128])
def test_windowed_prefill(d):
    from paged_kv_cache_192_gb300 import ops
    bt = Batch([3000, 2000, 2500, 2990] * 4, [20, 1, 16, 3] * 4, 2500, 4, 8, 8, d, 16, bf16, seed=d)
    kw = dict(num_sinks=bt.S)
    bt.check(repeat(lambda out: ops.prefill_window(bt.q_t, bt.k_cache, bt.v_cache, bt.table_t, bt.start_t, bt.lens_t,
                                                   20, bt.W, out=out, **kw)))


@pytest.mark.parametrize("most", [1, 5, 300])
def test_cross_attention_of_other_kernels(most):
    from paged_kv_cache_192_gb300 import ops
    from test_gpu_cross import Cross
    x = Cross([most] * 8, [900, 31, 1500, 64, 1, 0, 700, 1000], Hq=32, Hkv=16, d=128, bs=16, seed=most)
    x.check(repeat(lambda out: ops.cross_attention(x.q_t, x.k_cache, x.v_cache, x.table_t, x.start_t, x.lens_t,
                                                   most, out=out), 2000))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,H", [([100, 700, 5, 64, 330] * 4, 16), ([3000, 40], 8), ([65] * 40, 32), ([9] * 30, 8)])
def test_linear_prompts(n, H, d):
    """Requests at their first token: a call's states do not enter the next."""
    from linear_util import Linear
    from paged_kv_cache_192_gb300 import ops
    x = Linear(n, [0] * len(n), H=H, d=d, seed=d)

    def call(out):
        return ops.linear_prefill(x.q, x.k, x.v, x.states, x.ids_t, x.start, x.lens, max(n), x.decay_t, out=out)

    call(None)
    states = x.states.clone()
    repeat(call, 1500)
    assert torch.equal(states[x.ids].view(torch.int32), x.states[x.ids].view(torch.int32))


def test_plans():
    """No call between two waits for the one before: rings and lengths as the model's."""
    import random
    from plan_util import Model
    from paged_kv_cache_192_gb300 import ops
    rng = random.Random(0)
    m = Model(300, 40, 5000, 16, list(range(5000)))
    state, steps = m.state(), []
    for i in range(400):
        ids = rng.sample(range(300), rng.randint(1, 300))
        change = [rng.choice([1, 20, -3, -9, rng.randint(1, 90)]) for _ in ids]
        tokens = sum(max(0, c) for c in change)
        m.step(ids, change, tokens)
        steps.append([torch.tensor(x, dtype=torch.int32, device="cuda") for x in (ids, change)] + [tokens])
    for ids, change, tokens in steps:
        ops.plan_step(state, ids, change, 16, tokens)
    m.check(state)
    ops.device_error()
