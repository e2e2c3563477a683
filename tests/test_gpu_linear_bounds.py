"""Which kernel a prompt of linear attention takes: bounds above its tokens."""
import pytest
import torch

from linear_util import Linear
from test_gpu_linear import TERMS, _built, errors, prefill  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [[1], [2, 1, 4], [8]])
def test_a_bound_above_the_calls_tokens(n, d):
    """As with the exact one: token by token, where what is not finite in v reaches no
    earlier token."""
    x = Linear(n, [3] * len(n), d=d, seed=len(n))
    want = prefill(x)
    states = x.states.clone()
    x.states.copy_(x.states0)
    assert torch.equal(prefill(x, max_query_len=2048), want)
    assert torch.equal(x.states.view(torch.int32), states.view(torch.int32))
    x.check(want, terms=TERMS)
    x.states.copy_(x.states0)
    last = n[0] - 1
    x.qkv[last, 2] = float("nan")
    got = prefill(x, max_query_len=2 ** 31 - 1)
    assert torch.equal(got[:last], want[:last]) and bool(torch.isnan(got[last]).all())
    assert errors() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bound", [9, 64, 65, 500, 2 ** 31 - 1])
def test_any_bound_at_or_above_the_lengths(bound, d):
    """Also where a bound alone turns to other kernels, or to segments."""
    x = Linear([9, 1, 3, 0, 5] * 4, [0, 3, 2, 1, 0] * 4, H=3, d=d, seed=d)
    x.check(prefill(x, max_query_len=bound), terms=TERMS)
    x = Linear([9, 1, 1, 300], [0, 3, 2, 1], H=2, d=d, seed=d)
    x.check(prefill(x, max_query_len=max(bound, 300)), terms=TERMS)
    assert errors() == 0
