"""Linear attention where the old state is what counts: large states from before, tokens
whose keys are 0, decays of every strength.  A factor l^n has to be right relative to
itself; what it multiplies may be all that is left."""
import pytest
import torch

from linear_util import Linear
from test_gpu_linear import TERMS, _built, decode, errors, prefill  # noqa: F401

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32


def large(n, prior, log_decay, keys=0, **kw):
    """Requests whose states hold about 3e6 and whose tokens from the `keys`-th on add
    nothing."""
    x = Linear(n, prior, H=len(log_decay), log_decay=log_decay, **kw)
    at = 0
    for m in n:
        x.qkv[at + keys:at + m, 1] = 0
        at += m
    if not kw.get("fused", True):
        x.q, x.k, x.v = (t.contiguous() for t in x.qkv.unbind(1))
    x.states0 *= 1e6
    x.states = x.states0.cuda()
    return x


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B", [2, 40])
def test_decode(dtype, d, B):
    """One token: l S is all that the state is."""
    x = large([1] * B, [5] * B, [-1e-6, -0.3, -0.69, -0.7, -2.0, -4.0, -5.5, -8.0, -10.0, -12.0, -15.0, -17.0, -24.0, -60.0],
              d=d, dtype=dtype, seed=B)
    x.check(decode(x))
    assert errors() == 0


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_decode_beside_small_products(dtype):
    """The products are there, and far smaller than what the state was."""
    x = large([1] * 3, [5] * 3, [-4.0, -8.0, -12.0, -17.0], keys=1, d=128, dtype=dtype)
    x.check(decode(x))


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("n", [2, 5, 8])
def test_few_tokens(dtype, n):
    """Token by token, l^n in n steps."""
    x = large([n, 1], [5, 1], [-0.05, -0.693, -0.694, -2.0, -4.0, -7.0], d=128, dtype=dtype, seed=n)
    x.check(prefill(x), terms=TERMS)


@pytest.mark.parametrize("keys", [0, 1])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,log_decay", [
    (63, [-0.01, -0.1, -0.2, -0.231, -0.3, -0.4, -0.9]), (64, [-0.0107, -0.0109, -0.2, -0.231, -0.3, -0.4, -0.9]),
    (65, [-0.1, -0.2, -0.231, -0.3, -0.4, -0.8]), (66, [-0.25, -0.3, -0.5, -0.9]),
    (130, [-0.05, -0.1, -0.2, -0.231, -0.3, -0.4]), (200, [-0.05, -0.1, -0.2, -0.231, -0.28])])
def test_chunks(n, log_decay, d, keys):
    """l^64 and l^(tokens of the last chunk) of a state whose chunks add nothing, or the
    first token's product alone."""
    x = large([n, 30], [5, 0], log_decay, keys=keys, d=d, seed=n)
    x.check(prefill(x), terms=TERMS)
    assert errors() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1100, 2500])
def test_segments(n, d):
    """l^(tokens of a segment) where a request is cut: the state from before, and the
    first token's product, through all segments."""
    from paged_kv_cache_192_gb300 import ops
    decay = [-1e-4, -0.004, -20.0 / n, -70.0 / n]
    assert ops.linear_prefill_workspace_size(1, n, n, len(decay), d) > 0
    for keys, prior in ((0, 5), (1, 5), (1, 0)):
        x = large([n], [prior], decay, keys=keys, d=d, seed=n)
        x.check(prefill(x), terms=TERMS)
    assert errors() == 0


def check_with_infinities(x, out, terms=(0.0, 0.0)):
    """x.check's bounds where the result is finite, the same infinities elsewhere."""
    ref, rs, oa, ob, sa, sb = x.reference()
    for got, want, tol in (
            (x.states.double(), rs, (2.0 ** -22 + 2.0 ** -20 + terms[1]) * sa + (2.0 ** -22 + 2.0 ** -24) * sb),
            (out.double(), ref, torch.finfo(x.dtype).eps / 2 * ref.abs() + ((x.d + 20) * 2.0 ** -24 + terms[0]) * oa +
             (2.0 ** -22 + 2.0 ** -24) * ob)):
        inf = torch.isinf(want)
        assert bool(inf.any()) and torch.equal(got[inf], want[inf])
        fin = torch.isfinite(want)
        assert bool((got[fin] - want[fin]).abs().le(tol[fin]).all())
        assert bool(torch.isnan(got[torch.isnan(want)]).all())


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("n", [1, 3])
def test_an_infinite_state_stays_infinite(dtype, n):
    """Decays of both kinds and none; an output sees it with the sign of its query."""
    x = Linear([n, n], [5, 3], H=5, d=64, dtype=dtype, log_decay=[0.0, -0.01, -0.69, -3.0, -30.0])
    x.states0[x.ids[0], :, 7, 11] = float("inf")
    x.states0[x.ids[1], :, 60, 3] = -float("inf")
    x.states = x.states0.cuda()
    check_with_infinities(x, decode(x) if n == 1 else prefill(x))


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("n", [1, 4, 100, 1500])
def test_a_decay_that_is_nan_shows(n, dtype):
    """In every output and state of its head, and in no other's."""
    if dtype == f32 and n > 100:
        n = 130
    x = Linear([n, n], [5, 0], H=3, d=64, dtype=dtype, log_decay=[-0.1, float("nan"), -2.0])
    y = Linear([n, n], [5, 0], H=3, d=64, dtype=dtype, log_decay=[-0.1, -0.5, -2.0])
    got, want = prefill(x), prefill(y)
    assert bool(torch.isnan(got[:, 1]).all()) and torch.equal(got[:, ::2], want[:, ::2])
    assert bool(torch.isnan(x.states[x.ids, 1]).all()) and torch.equal(x.states[x.ids][:, ::2], y.states[y.ids][:, ::2])
    if n == 1:
        x.states.copy_(x.states0)
        got = decode(x)
        assert bool(torch.isnan(got[:, 1]).all()) and torch.equal(got[:, ::2], want[:, ::2])
        assert bool(torch.isnan(x.states[x.ids, 1]).all())
    assert errors() == 0


@pytest.mark.parametrize("n", [30, 100, 1500])
@pytest.mark.parametrize("d", [64, 128])
def test_prompts_keep_an_infinite_state(n, d):
    """One that was there before, through chunks and segments, and its outputs."""
    x = Linear([n, n], [5, 3], H=3, d=d, log_decay=[0.0, -0.001, -20.0 / n])
    x.states0[x.ids[0], :, 7, 11] = float("inf")
    x.states0[x.ids[1], :, d - 4, 3] = -float("inf")
    x.qkv[..., [7, d - 4]] += (x.qkv[..., [7, d - 4]] == 0).to(bf16)  # (0 x inf is NaN in the formula too)
    x.states = x.states0.cuda()
    check_with_infinities(x, prefill(x), terms=TERMS)


@pytest.mark.parametrize("n,at", [(30, 3), (100, 99), (100, 70), (1500, 20), (1500, 800), (1500, 1499)])
def test_prompts_with_an_infinite_value(n, at):
    """It reaches the state with the sign of k v, and no other dimension of v."""
    x = Linear([n, 40], [5, 0], H=2, d=64, log_decay=[0.0, -0.01], seed=at)
    x.qkv[at, 1] += (x.qkv[at, 1] == 0).to(bf16)
    x.qkv[at, 2, :, 9] = float("inf")
    x.qkv[at, 2, :, 50] = -float("inf")
    out = prefill(x)
    ref, rs, oa, ob, sa, sb = x.reference()
    got, want = x.states[x.ids].double(), rs[x.ids]
    assert bool(torch.isinf(want[0, :, :, [9, 50]]).all()) and torch.equal(got[0, :, :, [9, 50]], want[0, :, :, [9, 50]])
    keep = torch.ones(64, dtype=torch.bool)
    keep[[9, 50]] = False
    tol = (2.0 ** -22 + 2.0 ** -20 + TERMS[1]) * sa + (2.0 ** -22 + 2.0 ** -24) * sb
    assert bool(((got - want).abs() <= tol[x.ids])[..., keep].all()) and bool(torch.isfinite(got[1]).all())
    tol = 2.0 ** -8 * ref.abs() + ((64 + 20) * 2.0 ** -24 + TERMS[0]) * oa + (2.0 ** -22 + 2.0 ** -24) * ob
    assert bool(((out.double() - ref).abs() <= tol)[..., keep].all())
    # behind it the state's part is not finite; 64 tokens and more before it all is
    assert not bool(torch.isfinite(out[at:n, :, [9, 50]]).any())
    early = out[:max(0, at - 63), :, [9, 50]].double() - ref[:max(0, at - 63), :, [9, 50]]
    assert bool((early.abs() <= tol[:max(0, at - 63), :, [9, 50]]).all())


@pytest.mark.parametrize("sign", [1, -1])
def test_prompts_of_states_past_the_range_of_bf16(sign):
    """Between bf16's largest number and fp32's."""
    x = Linear([70], [5], H=1, d=64, log_decay=[-0.5])
    x.qkv[:, 0, :, 4] *= 2.0 ** -10
    x.qkv[:, 1] = 0
    x.states0[x.ids[0], 0, 4, 4] = sign * 3.4e38
    x.states = x.states0.cuda()
    x.check(prefill(x), terms=TERMS)
