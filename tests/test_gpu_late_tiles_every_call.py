"""The loads of test_gpu_late_tiles, with every call's output compared: a fault of one call
in 1,000 shows in nearly every run."""
import pytest
import torch

from window_util import Batch

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_192_gb300 import build
    build.build()


def repeat(call, check, times=4000, ring=8):
    """`ring` calls after one another into outputs of their own, then all of them against
    the first call's bits (which `check` has looked at)."""
    from paged_kv_cache_192_gb300 import ops
    first = call(None).clone()
    check(first)
    assert ops.device_error() == 0
    outs = torch.empty(ring, *first.shape, dtype=first.dtype, device="cuda")
    changed = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(times // ring):
        outs.fill_(float("nan"))
        for out in outs:
            call(out)
        changed += (outs.view(torch.int16) != first.view(torch.int16)).flatten(1).any(1).sum()
        if i % 64 == 63:
            assert ops.device_error() == 0
    assert ops.device_error() == 0
    assert int(changed) == 0, f"{int(changed)} of {times} calls"


@pytest.mark.parametrize("d", [64, 128])
def test_cross_attention(d):
    from paged_kv_cache_192_gb300 import ops
    from test_gpu_cross import Cross
    x = Cross([40] + [1] * 39, [3200, 0, 1, 63] * 10, Hq=4, Hkv=4, d=d, bs=64, seed=d)
    repeat(lambda out: ops.cross_attention(x.q_t, x.k_cache, x.v_cache, x.table_t, x.start_t, x.lens_t, 40, out=out),
           x.check)


@pytest.mark.parametrize("d", [64, 128])
def test_windowed_prefill(d):
    from paged_kv_cache_192_gb300 import ops
    bt = Batch([3000, 2000, 2500, 2990] * 4, [20, 1, 16, 3] * 4, 2500, 4, 8, 8, d, 16, bf16, seed=d)
    kw = dict(num_sinks=bt.S)
    repeat(lambda out: ops.prefill_window(bt.q_t, bt.k_cache, bt.v_cache, bt.table_t, bt.start_t, bt.lens_t, 20, bt.W,
                                          out=out, **kw), bt.check)


@pytest.mark.parametrize("most", [1, 5, 300])
def test_cross_attention_of_other_kernels(most):
    from paged_kv_cache_192_gb300 import ops
    from test_gpu_cross import Cross
    x = Cross([most] * 8, [900, 31, 1500, 64, 1, 0, 700, 1000], Hq=32, Hkv=16, d=128, bs=16, seed=most)
    repeat(lambda out: ops.cross_attention(x.q_t, x.k_cache, x.v_cache, x.table_t, x.start_t, x.lens_t, most, out=out),
           x.check, 2000)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,H", [([100, 700, 5, 64, 330] * 4, 16), ([3000, 40], 8), ([65] * 40, 32), ([9] * 30, 8)])
def test_linear_prompts(n, H, d):
    from linear_util import Linear
    from test_gpu_linear import TERMS
    from paged_kv_cache_192_gb300 import ops
    x = Linear(n, [0] * len(n), H=H, d=d, seed=d)
    # (the bounds themselves have tests of their own at these lengths)
    repeat(lambda out: ops.linear_prefill(x.q, x.k, x.v, x.states, x.ids_t, x.start, x.lens, max(n), x.decay_t, out=out),
           lambda out: x.check(out, terms=TERMS) if sum(n) * H <= 40000 else None, 1600)
