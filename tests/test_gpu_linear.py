"""Linear attention with a decay for each head, single tokens and prompts, against
the recurrence in 64 bits."""
import pytest
import torch

from linear_util import Linear

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32
# The kernel of long prompts gives the tensor core its weights (scores times decays,
# states, decayed values) in two bf16 terms or more: each off by at most half a step
# of the second, 2^-17 of itself, and two of them meet in an output's earlier part.
TERMS = 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_192_gb300 import build
    build.build()


def decode(x, **kw):
    from paged_kv_cache_192_gb300 import ops
    return ops.linear_decode(x.q, x.k, x.v, x.states, x.ids_t, x.lens, x.decay_t, **kw)


def errors():
    from paged_kv_cache_192_gb300 import ops
    return ops.device_error()


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H", [(1, 1), (1, 16), (3, 5), (70, 4), (1, 200)])
def test_decode(dtype, d, B, H):
    """Few states (cut into slices) and many; some sequences at their first token."""
    prior = [0 if i % 3 == 2 else 1 + 977 * i for i in range(B)]
    x = Linear([1] * B, prior, H=H, d=d, dtype=dtype, seed=B + H, fused=H % 2 == 0)
    x.check(decode(x))
    assert errors() == 0


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_decode_steps_follow_one_another(dtype):
    """Eight steps on one state, back to back, as one request of eight tokens."""
    x = Linear([8], [5], H=4, d=128, dtype=dtype)
    outs = []
    from paged_kv_cache_192_gb300 import ops
    for t in range(8):
        outs.append(ops.linear_decode(x.q[t:t + 1], x.k[t:t + 1], x.v[t:t + 1], x.states, x.ids_t,
                                      x.lens - 7 + t, x.decay_t))
    x.check(torch.cat(outs))


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_decode_padding(dtype):
    """Rows without a state or without a length: zeros, no state touched."""
    x = Linear([1] * 5, [4, 0, 7, 9, 0], dtype=dtype, ids=[2, -1, 0, 1, 4], num_states=6)
    x.lens[3] = 0
    x.n = [1, 1, 1, 0, 1]
    x.states0[1] = 7.5
    x.states[1] = 7.5
    got = decode(x)
    assert bool((got[1] == 0).all()) and bool((got[3] == 0).all())
    x.n = [1, 1, 1, 1, 1]
    x.ids[3] = -1
    ref = x.reference()[0]
    ref[[1, 3]] = float("nan")
    x.check(got)
    assert errors() == 0


@pytest.mark.parametrize("what,value", [("ids", 6), ("ids", 2 ** 31 - 1), ("lens", -1), ("lens", -2 ** 31)])
def test_decode_rows_that_do_not_fit(what, value):
    x = Linear([1] * 3, [4, 2, 7], ids=[2, 3, 0], num_states=6)
    {"ids": x.ids_t, "lens": x.lens}[what][1] = value
    x.ids[1] = -1
    x.states0[3] = float("nan")
    x.states[3] = float("nan")
    got = decode(x)
    assert errors() == 4 and bool((got[1] == 0).all())
    x.check(got)


@pytest.mark.parametrize("log_decay", [[0.0, -1e-7, -30.0], [-200.0, -1e5, float("-inf")]])
@pytest.mark.parametrize("dtype", [bf16, f32])
def test_decode_extreme_decays(log_decay, dtype):
    x = Linear([1] * 4, [3, 0, 5, 9], d=128, dtype=dtype, log_decay=log_decay)
    x.check(decode(x))


def test_decode_scale_out_stream_and_graph():
    x = Linear([1] * 6, [3] * 6, H=8, d=128)
    out = torch.full_like(x.q, float("nan"), memory_format=torch.contiguous_format)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert decode(x, scale=0.3, out=out, stream=side).data_ptr() == out.data_ptr()
    torch.cuda.synchronize()
    x.check(out, scale=0.3)
    x.states.copy_(x.states0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        decode(x, scale=0.3, out=out)
    x.states.copy_(x.states0)
    out.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    x.check(out, scale=0.3)


def test_decode_state_past_4_gib():
    """States behind byte 2^32 of the pool."""
    x = Linear([1] * 2, [3, 4], H=32, d=128, ids=[0, 1])
    NS = 2 ** 32 // (32 * 128 * 128 * 4) + 3
    big = torch.empty(NS, 32, 128, 128, device="cuda")
    big[NS - 2:] = x.states[:2]
    x.ids_t += NS - 2
    from paged_kv_cache_192_gb300 import ops
    got = ops.linear_decode(x.q, x.k, x.v, big, x.ids_t, x.lens, x.decay_t)
    x.states[:2] = big[NS - 2:]
    x.check(got)


def test_validate_mode():
    from paged_kv_cache_192_gb300 import _lib, ops
    x = Linear([1] * 3, [4, 2, 7])
    ops.set_validate(True)
    try:
        x.check(decode(x))
        for t, i, v, msg in ((x.ids_t, 1, int(x.ids_t[0]), "named twice"), (x.ids_t, 1, 99, "outside"),
                             (x.lens, 1, -3, "new tokens"), (x.decay_t, 0, 0.5, "positive"),
                             (x.decay_t, 0, float("nan"), "positive")):
            keep = t[i].clone()
            t[i] = v
            with pytest.raises(_lib.PAError, match=msg):
                decode(x)
            t[i] = keep
    finally:
        ops.set_validate(False)


# ---- prompts ---------------------------------------------------------------------
def prefill(x, max_query_len=None, **kw):
    from paged_kv_cache_192_gb300 import ops
    return ops.linear_prefill(x.q, x.k, x.v, x.states, x.ids_t, x.start, x.lens,
                              max(x.n) if max_query_len is None else max_query_len, x.decay_t, **kw)


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("n,prior", [
    ([1], [0]), ([1], [9]), ([2, 1, 7], [0, 3, 0]), ([5, 0, 3], [1, 4, 0]), ([4] * 40, list(range(40)))])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_few_tokens(dtype, n, prior, d):
    x = Linear(n, prior, H=3, d=d, dtype=dtype, seed=len(n))
    x.check(prefill(x), terms=TERMS)
    assert errors() == 0
