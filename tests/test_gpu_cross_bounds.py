"""Cross attention with a bound above the call's rows."""
import pytest
import torch

from test_gpu_cross import Cross, _built  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,gq", [([1], 1), ([1], 8), ([2, 0, 3], 4), ([1, 1, 30], 1)])
def test_a_bound_above_the_calls_rows(n, gq, d):
    """The kernel and the bits of the exact bound."""
    x = Cross(n, [700, 33, 64][:len(n)], Hq=2 * gq, Hkv=2, d=d, seed=gq)
    want = x.run(max_query_len=sum(n))
    x.check(want)
    for bound in (sum(n) + 1, 2048, 2 ** 31 - 1):
        assert torch.equal(x.run(max_query_len=bound), want)


@pytest.mark.parametrize("bound", [33, 128, 129, 5000, 2 ** 31 - 1])
def test_any_bound_at_or_above_the_rows(bound):
    x = Cross([33, 1, 0, 7], [700, 33, 64, 129], Hq=8, Hkv=2, d=128, seed=bound % 97)
    x.check(x.run(max_query_len=bound))
