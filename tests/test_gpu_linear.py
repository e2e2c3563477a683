"""Linear attention with a decay for each head, single tokens and prompts, against
the recurrence in 64 bits."""
import pytest
import torch

from linear_util import Linear

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32
# The kernels of long prompts give the tensor core scores times decays, and states, in
# two bf16 terms (each off by at most half a step, 2^-8, of what is left: 2^-16 in
# all), of which a term of an output passes one; decayed values in three (2^-24).  The
# tensor core adds 16 products at a time to a sum in 32 bits, which may cut up to 2^-22
# of the amounts: 12 times in a chunk's part of a state (2^-18.4), up to 24 times and 8
# in an output and its scores (2^-17).
TERMS = 2.0 ** -15, 2.0 ** -18


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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,prior", [
    ([9], [0]), ([63], [5]), ([64], [0]), ([65], [1]), ([128], [3]), ([129], [0]), ([191, 192, 193], [0, 7, 1]),
    ([320, 1, 0, 64, 17], [3, 5, 2, 0, 1]), ([450], [9])])
def test_prefill_chunks(n, prior, d):
    """Chunks of 64 tokens that end anywhere; the rings go round."""
    x = Linear(n, prior, H=3, d=d, seed=len(n))
    x.check(prefill(x), terms=TERMS)
    assert errors() == 0


@pytest.mark.parametrize("d,H", [(64, 1), (128, 2)])
@pytest.mark.parametrize("n,prior", [([3000], [0]), ([1024, 1500], [4, 0]), ([2049, 5, 0, 1023], [1, 1, 1, 1]),
                                     ([1025], [0])])
def test_prefill_segments(n, prior, d, H):
    """Few (request, head) pairs and many tokens: requests are cut into segments."""
    from paged_kv_cache_192_gb300 import ops
    x = Linear(n, prior, H=H, d=d, seed=len(n))
    assert ops.linear_prefill_workspace_size(len(n), sum(n), max(n), H, d) > 0
    x.check(prefill(x), terms=TERMS)
    assert errors() == 0


@pytest.mark.parametrize("log_decay", [[0.0, -1e-7, -1e-3], [-1.0, -30.0, -88.0], [-200.0, -1e5, float("-inf")]])
@pytest.mark.parametrize("n", [200, 2500])
def test_prefill_extreme_decays(log_decay, n):
    x = Linear([n, 70], [3, 0], d=128, log_decay=log_decay)
    x.check(prefill(x), terms=TERMS)


@pytest.mark.parametrize("R,H", [(2, 100), (33, 8), (63, 3), (64, 4), (65, 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_requests_of_all_lengths(R, H, d):
    """More (request, head) pairs than SMs, in any order of lengths, equal ones too; some
    requests without new tokens or without a state."""
    n = [i * 37 % 131 if i % 5 else 70 for i in range(R)]
    n[R // 2] = 200
    ids = [-1 if i % 9 == 4 else R - i for i in range(R)]
    x = Linear(n, [i % 3 for i in range(R)], H=H, d=d, seed=R, ids=ids)
    got = prefill(x)
    start = x.start.tolist()
    for i, s in enumerate(ids):  # the rows of requests that were left out hold anything
        if s < 0:
            got[start[i]:start[i + 1]] = 0
    x.check(got, terms=TERMS)
    assert errors() == 0


@pytest.mark.parametrize("n", [100, 2500])
def test_prefill_many_requests_and_heads(n):
    x = Linear([n] + [10 + 7 * i for i in range(12)], [0, 3] * 6 + [1], H=16, d=64 if n == 100 else 128)
    x.check(prefill(x), terms=TERMS)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [5, 40, 70, 1100])
def test_prefill_what_no_request_owns(n, d):
    """Rows before, between (requests left out) and behind the requests hold NaN or
    infinities: they reach nothing, and the output's rows stay."""
    x = Linear([3, n, 6, n, 2], [1, 0, 4, 2, 1], H=2, d=d, ids=[-1, 3, -1, 0, -5], num_states=5, gap=9)
    at, bad = 0, torch.ones(x.T, dtype=torch.bool)
    for m, i in zip(x.n, x.ids):
        if i >= 0:
            bad[at:at + m] = False
        at += m
    poison = torch.tensor([float("nan"), float("inf"), -float("inf")])
    rows = bad.nonzero()[:, 0].cuda()
    x.qkv[rows] = poison[torch.randint(0, 3, (len(rows), 3, 2, d))].cuda().to(bf16)
    out = torch.full((x.T, 2, d), 7.0, dtype=bf16, device="cuda")
    x.check(prefill(x, out=out), terms=TERMS)
    assert bool((out[rows] == 7).all())
    assert errors() == 0


@pytest.mark.parametrize("n", [4, 100, 1500])
@pytest.mark.parametrize("what,i,value", [("ids_t", 1, 9), ("lens", 1, 2), ("lens", 1, -1), ("start", 2, -1),
                                          ("start", 2, 10 ** 6), ("start", 2, 2 ** 31 - 1)])
def test_prefill_requests_that_do_not_fit(n, what, i, value):
    """Recorded and left out; request 0 is right."""
    x = Linear([n, n, n], [3, 0, 2], H=2, d=128, ids=[2, 0, 4], num_states=6)
    getattr(x, what)[i] = value
    out = torch.full_like(x.q, 7.0, memory_format=torch.contiguous_format)
    prefill(x, out=out)
    assert errors() == 4
    # request 2 runs where its own rows fit
    left = [1, 2] if what == "start" else [1]
    for r in left:
        x.ids[r] = -1
    x.states0[0] = float("nan")
    x.check(out, terms=TERMS)


@pytest.mark.parametrize("n", [6, 200, 3000])
def test_prefill_scale_stream_workspace_and_graph(n):
    from paged_kv_cache_192_gb300 import ops
    x = Linear([n, 3], [3, 0], H=2, d=128)
    out = torch.full_like(x.q, float("nan"), memory_format=torch.contiguous_format)
    ws = torch.full((max(4, ops.linear_prefill_workspace_size(2, n + 3, n, 2, 128) // 4),), float("nan"), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert prefill(x, scale=0.3, out=out, workspace=ws, stream=side).data_ptr() == out.data_ptr()
    torch.cuda.synchronize()
    x.check(out, scale=0.3, terms=TERMS)
    g = torch.cuda.CUDAGraph()
    x.states.copy_(x.states0)
    with torch.cuda.graph(g):
        got = prefill(x, scale=0.3)
    for _ in range(2):
        x.states.copy_(x.states0)
        got.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        x.check(got, scale=0.3, terms=TERMS)


@pytest.mark.parametrize("n", [70, 2500])
def test_prefill_calls_back_to_back_agree(n):
    """Twenty calls that nothing waits between: the same bits each time."""
    x = Linear([n, 30], [3, 0], H=4, d=128)
    first = prefill(x)
    torch.cuda.synchronize()
    after = x.states.clone()
    outs, states = [], [x.states0.cuda() for _ in range(20)]
    torch.cuda.synchronize()
    for s in states:
        x.states = s
        outs.append(prefill(x))
    torch.cuda.synchronize()
    for o, s in zip(outs, states):
        assert torch.equal(o, first) and torch.equal(s.view(torch.int32), after.view(torch.int32))


def test_prefill_then_decode_is_one_sequence():
    """A prompt, a chunk, single tokens: as one request of all of them."""
    from paged_kv_cache_192_gb300 import ops
    x = Linear([300], [0], H=4, d=128)
    outs, at = [], 0
    for n in (200, 90, 7, 1, 1, 1):
        q, k, v = (t[at:at + n] for t in (x.q, x.k, x.v))
        at += n
        lens = torch.tensor([at], dtype=torch.int32, device="cuda")
        if n == 1:
            outs.append(ops.linear_decode(q, k, v, x.states, x.ids_t, lens, x.decay_t))
        else:
            start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
            outs.append(ops.linear_prefill(q, k, v, x.states, x.ids_t, start, lens, n, x.decay_t))
    x.check(torch.cat(outs), terms=TERMS)


def test_prefill_validate_mode_and_workspace():
    from paged_kv_cache_192_gb300 import _lib, ops
    x = Linear([300, 2], [4, 0])
    ops.set_validate(True)
    try:
        x.check(prefill(x), terms=TERMS)
        for t, i, v, msg in ((x.ids_t, 1, int(x.ids_t[0]), "named twice"), (x.start, 2, 400, "new tokens"),
                             (x.lens, 0, 299, "new tokens")):
            keep = t[i].clone()
            t[i] = v
            with pytest.raises(_lib.PAError, match=msg):
                prefill(x)
            t[i] = keep
        with pytest.raises(_lib.PAError, match="max_query_len 299"):
            prefill(x, max_query_len=299)
    finally:
        ops.set_validate(False)
    x = Linear([3000], [0], H=1)
    with pytest.raises(_lib.PAError, match="needed"):
        prefill(x, workspace=torch.zeros(16, device="cuda"))
