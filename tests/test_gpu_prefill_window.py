"""pa_prefill_window against the formula in 64 bits: windows and sinks against
chunk and context, page sizes, head groups, ragged and empty requests, many
requests, freed pages and poisoned slots, streams and graphs."""
import numpy as np
import pytest
import torch

from window_util import DEV, Batch

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_192_gb300 import build
    build.build()


def call(bt, **kw):
    from paged_kv_cache_192_gb300 import ops
    kw.setdefault("num_sinks", bt.S)
    return ops.prefill_window(bt.q_t, bt.k_cache, bt.v_cache, bt.table_t, bt.start_t, bt.lens_t,
                              max(bt.n_new), bt.W, **kw)


def run(bt, **kw):
    from paged_kv_cache_192_gb300 import ops
    out = call(bt, **kw)
    torch.cuda.synchronize()
    assert ops.device_error() == 0
    return out


def batch(lens, n_new, W, S, Hq=8, Hkv=2, d=128, bs=16, **kw):
    return Batch(lens, n_new, W, S, Hq, Hkv, d, bs, bf16, **kw)


LENS = [1, 40, 64, 65, 130, 300, 517, 200, 90]
NEW = [1, 40, 1, 64, 65, 129, 200, 0, 7]


@pytest.mark.parametrize("W,S", [(1, 0), (1, 3), (7, 1), (64, 64), (63, 4), (65, 0), (100, 37),
                                 (128, 200), (300, 8), (2 ** 31 - 1, 0), (5, 2 ** 31 - 1)])
def test_windows_and_sinks(W, S):
    bt = batch(LENS, NEW, W, S, seed=W % 97)
    bt.check(run(bt))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gq", [1, 2, 4, 8])
@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128])
def test_shapes(d, gq, bs):
    bt = batch([70, 300, 20, 500], [70, 90, 1, 270], 77, 5, Hq=3 * gq, Hkv=3, d=d, bs=bs,
               seed=bs + gq)
    bt.check(run(bt))


@pytest.mark.parametrize("L,n,W,S", [(2000, 700, 512, 4), (1500, 1500, 1000, 64), (3000, 33, 2049, 0),
                                     (2600, 300, 256, 300)])
def test_long(L, n, W, S):
    bt = batch([L], [n], W, S, Hq=8, Hkv=2)
    bt.check(run(bt))


@pytest.mark.parametrize("L,n,W,S", [(2500, 1, 2200, 4), (2500, 20, 2200, 0), (1100, 40, 1000, 70),
                                     (600, 30, 500, 3), (300, 70, 100, 64), (70, 70, 20, 2), (3, 3, 9, 0)])
@pytest.mark.parametrize("d,gq,bs", [(128, 4, 16), (64, 1, 128), (64, 8, 8), (128, 2, 64)])
def test_few_query_tiles(L, n, W, S, d, gq, bs):
    """Batches so small that a cluster divides the keys of one query tile, from
    one CTA to the largest cluster, down to fewer K/V tiles than CTAs."""
    bt = batch([L, L // 2 + n], [n, n // 2], W, S, Hq=2 * gq, Hkv=2, d=d, bs=bs, seed=L + d)
    bt.check(run(bt))


def test_overlapping_requests_do_not_pass_the_grid():
    """Row ranges that overlap (no prefix sum) make more query tiles than the
    rows bound: recorded, and nothing is read or written out of range."""
    from paged_kv_cache_192_gb300 import ops
    bt = batch([200, 200, 200, 200], [50, 50, 50, 50], 64, 0)
    start = torch.tensor([0, 200, 0, 200, 0], dtype=torch.int32, device=DEV)
    ops.prefill_window(bt.q_t, bt.k_cache, bt.v_cache, bt.table_t, start, bt.lens_t, 50, 64)
    assert ops.device_error() == 1


@pytest.mark.parametrize("R", [300, 1300])
def test_many_requests(R):
    """More items than CTAs, and more requests than one launch holds."""
    rng = np.random.default_rng(R)
    n = [int(x) for x in rng.integers(0, 6, size=R)]
    lens = [int(x + y) for x, y in zip(n, rng.integers(0, 40, size=R))]
    bt = batch(lens, n, 9, 2, Hq=4, Hkv=1, d=64, bs=8, seed=R)
    bt.check(run(bt))


def test_long_table():
    """A table longer than any kernel's slice of it, deep positions."""
    bt = batch([20000, 60], [30, 60], 200, 5, bs=8, extra_blocks=300)
    bt.check(run(bt))


def test_window_beyond_the_context_matches_prefill_chunk():
    from paged_kv_cache_192_gb300 import ops
    bt = batch([100, 333, 400], [100, 50, 400], 1000, 0)
    ref = ops.prefill_chunk(bt.q_t, bt.k_cache, bt.v_cache, bt.table_t, bt.start_t, bt.lens_t, 400)
    bt.check(ref)
    bt.check(run(bt))


def test_scale_and_rows_outside_the_requests():
    """Rows before the first request and behind the last stay as they were."""
    from paged_kv_cache_192_gb300 import ops
    bt = batch([90, 300], [30, 70], 50, 3)
    pad = torch.full((13, 8, 128), float("nan"), dtype=bf16, device=DEV)
    q = torch.cat([pad[:5], bt.q_t, pad])
    out = torch.full_like(q, 7.0)
    r = ops.prefill_window(q, bt.k_cache, bt.v_cache, bt.table_t, bt.start_t + 5, bt.lens_t, 70, 50, 3,
                           scale=0.3, out=out)
    torch.cuda.synchronize()
    assert r.data_ptr() == out.data_ptr() and ops.device_error() == 0
    assert (out[:5] == 7.0).all() and (out[105:] == 7.0).all()
    bt.check(out[5:105], scale=0.3)


def test_chunks_equal_one_call():
    """A prompt in chunks over its own cache, within the bound of one call."""
    from paged_kv_cache_192_gb300 import ops
    bt = batch([700], [700], 150, 10)
    whole = run(bt)
    bt.check(whole)
    parts = []
    for a in range(0, 700, 233):
        b = min(700, a + 233)
        parts.append(ops.prefill_window(bt.q_t[a:b], bt.k_cache, bt.v_cache, bt.table_t,
                                        torch.tensor([0, b - a], dtype=torch.int32, device=DEV),
                                        torch.tensor([b], dtype=torch.int32, device=DEV), b - a, 150, 10))
    bt.check(torch.cat(parts))


def test_placement_does_not_change_a_bit():
    from paged_kv_cache_192_gb300 import ops
    bt = batch(LENS, NEW, 100, 20, seed=3)
    a = run(bt)
    perm = torch.randperm(bt.k_cache.shape[0], generator=torch.Generator().manual_seed(1)).to(DEV)
    k2, v2 = torch.empty_like(bt.k_cache), torch.empty_like(bt.v_cache)
    k2[perm], v2[perm] = bt.k_cache, bt.v_cache
    t2 = torch.where(bt.table_t >= 0, perm[bt.table_t.clamp(min=0).long()].int(), bt.table_t)
    b = ops.prefill_window(bt.q_t, k2, v2, t2, bt.start_t, bt.lens_t, max(NEW), 100, 20)
    assert torch.equal(a, b)


def test_pool_past_4_gib():
    NB = 2 ** 32 // (2 * 16 * 128 * 2) + 200
    bt = batch([700, 33, 900], [100, 33, 300], 300, 10, num_blocks=NB)
    bt.check(run(bt))


def test_bad_pages_and_lengths_are_recorded():
    from paged_kv_cache_192_gb300 import ops
    bt = batch([90, 300], [30, 70], 50, 3)
    good = run(bt)
    t = bt.table_t.clone()
    t[bt.table_t < 0] = 2 ** 31 - 1  # freed pages: anything
    assert torch.equal(run(bt), good)
    t[0, 89 // 16] = bt.k_cache.shape[0]
    out = ops.prefill_window(bt.q_t, bt.k_cache, bt.v_cache, t, bt.start_t, bt.lens_t, 70, 50, 3)
    assert ops.device_error() == 1
    assert torch.equal(out[30:], good[30:])
    for lens, start in (([29, 300], [0, 30, 100]), ([10 ** 6, 300], [0, 30, 100]),
                        ([90, 300], [-70, 30, 100])):
        out = torch.full_like(bt.q_t, 7.0)
        ops.prefill_window(bt.q_t, bt.k_cache, bt.v_cache, bt.table_t,
                           torch.tensor(start, dtype=torch.int32, device=DEV),
                           torch.tensor(lens, dtype=torch.int32, device=DEV), 70, 50, 3, out=out)
        assert ops.device_error() == 1
        assert (out[:30] == 7.0).all() and torch.equal(out[30:], good[30:])
    out = torch.full_like(bt.q_t, 7.0)
    ops.prefill_window(bt.q_t, bt.k_cache, bt.v_cache, bt.table_t,
                       torch.tensor([0, 30, 101], dtype=torch.int32, device=DEV), bt.lens_t, 70, 50, 3,
                       out=out)
    assert ops.device_error() == 1
    assert (out[30:] == 7.0).all() and torch.equal(out[:30], good[:30])


def test_validate_mode():
    from paged_kv_cache_192_gb300 import ops
    from paged_kv_cache_192_gb300._lib import PAError
    bt = batch([900, 400], [100, 0], 100, 20)
    ops.set_validate(True)
    try:
        bt.check(run(bt))
        t = bt.table_t.clone()
        t[0, 0] = -1
        with pytest.raises(PAError, match="block_table"):
            ops.prefill_window(bt.q_t, bt.k_cache, bt.v_cache, t, bt.start_t, bt.lens_t, 100, 100, 20)
        with pytest.raises(PAError, match="new tokens"):
            ops.prefill_window(bt.q_t, bt.k_cache, bt.v_cache, bt.table_t, bt.start_t,
                               bt.lens_t - 850, 100, 100, 20)
    finally:
        ops.set_validate(False)


def test_streams_graphs_and_back_to_back():
    from paged_kv_cache_192_gb300 import ops
    a, c = batch([900, 400, 77], [300, 50, 77], 300, 20, seed=1), batch([300] * 9, [40] * 9, 128, 4, seed=2)
    ra, rc = run(a), run(c)
    outs = [call(a) for _ in range(12)]  # each overlaps the tail of the one before
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    s1.wait_stream(torch.cuda.current_stream())
    s2.wait_stream(torch.cuda.current_stream())
    other = []
    for _ in range(6):
        outs.append(call(a, stream=s1))
        other.append(call(c, stream=s2))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ra) for o in outs) and all(torch.equal(o, rc) for o in other)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = call(a)
    for _ in range(3):
        o.zero_()
        g.replay()
        e = call(c)
    torch.cuda.synchronize()
    assert torch.equal(o, ra) and torch.equal(e, rc) and ops.device_error() == 0


def test_validate_mode_checks_rows_and_the_longest_request():
    from paged_kv_cache_192_gb300 import ops
    from paged_kv_cache_192_gb300._lib import PAError
    bt = batch([90, 300], [30, 70], 50, 3)

    def call_with(start, max_query_len):
        return ops.prefill_window(bt.q_t, bt.k_cache, bt.v_cache, bt.table_t,
                                  torch.tensor(start, dtype=torch.int32, device=DEV), bt.lens_t,
                                  max_query_len, 50, 3)
    ops.set_validate(True)
    try:
        bt.check(call_with([0, 30, 100], 70))
        call_with([30, 30, 100], 70)  # a request without new tokens
        with pytest.raises(PAError, match="max_query_len 69"):
            call_with([0, 30, 100], 69)
        for start in ([-1, 29, 99], [1, 31, 101]):
            with pytest.raises(PAError, match="rows"):
                call_with(start, 70)
    finally:
        ops.set_validate(False)
    assert ops.device_error() == 0
