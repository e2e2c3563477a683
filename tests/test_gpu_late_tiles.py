"""The split kernel of windowed prefills and cross attention, whose two groups take every
other tile, under loads whose tiles land late and out of order: many CTAs, each with
more tiles than the ring has stages, call after call."""
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
