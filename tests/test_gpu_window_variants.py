"""The windowed calls' kernel variants over long windows: the persistent prefill
kernel (several tiles per item, ring and block-table batches wrapping, items one
after another), windowed decode on clusters of one CTA with many tiles per warp
and with the deeper ring; scores that force the running maximum to move; freed
pages; and how far a NaN or infinity in a visible token spreads."""
import numpy as np
import pytest
import torch

from window_util import DEV, Batch

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_192_gb300 import build
    build.build()


def check_peaked(bt, got, scale):
    """Batch.check for a scale at which a score's own error counts: with A the
    largest sum |q| |k| of a score, d additions of at most 2^-23 of it (the tensor
    core may truncate) are e = d 2^-23 A scale, twice that relative in a weight
    with its sum; the weights enter the product with 16 bits.  Half a step of the
    output, and (2 e + 2^-15) max |v|."""
    gq, at, A = bt.Hq // bt.Hkv, 0, 0.0
    for L, n, k in zip(bt.lens, bt.n_new, bt.k):
        if L and n:
            q = bt.q[at:at + n].float().abs()
            A = max(A, float(torch.einsum("nhd,jhd->hnj", q, k.float().abs().repeat_interleave(gq, 1)).max()))
        at += n
    ref = bt.reference(scale)
    vmax = max(float(v.abs().max()) for v in bt.v if v.numel())
    tol = 2.0 ** -8 * ref.abs() + (2 * bt.d * 2.0 ** -23 * A * scale + 2.0 ** -15) * vmax
    err = (got.double().cpu() - ref).abs()
    assert bool((err <= tol).all()), f"max excess {float((err - tol).max()):.3e}"


# ---- prefill ----------------------------------------------------------------------
def prefill(bt, table=None, **kw):
    from paged_kv_cache_192_gb300 import ops
    return ops.prefill_window(bt.q_t, bt.k_cache, bt.v_cache, bt.table_t if table is None else table,
                              bt.start_t, bt.lens_t, max(bt.n_new), bt.W, bt.S, **kw)


def kernel_of(bt):
    from paged_kv_cache_192_gb300 import ops
    return ops.prefill_window_kernel_for(len(bt.lens), sum(bt.n_new), max(bt.n_new), bt.Hq, bt.Hkv)


def run(bt, **kw):
    from paged_kv_cache_192_gb300 import ops
    out = prefill(bt, **kw)
    torch.cuda.synchronize()
    assert ops.device_error() == 0
    return out


def serving(gq, d, bs, W=350, S=40, Hkv=8, seed=0, far=(500, 640), deep=()):
    """24 requests of 0 to 5 query tiles behind contexts of `far` tokens, more
    items than SMs; deep: prior contexts of the first requests."""
    rng = np.random.default_rng(seed)
    qt = 128 // gq
    n = [5 * qt + 3, qt, 1, 2 * qt, qt // 2 + 3, 0, 2 * qt - 1, qt + 1] + \
        [int(x) for x in rng.integers(1, qt + 1, size=16)]
    prior = [int(x) for x in rng.integers(*far, size=24)]
    prior[1], prior[4], prior[9] = 0, 3, 70
    for i, p in enumerate(deep):
        n[i], prior[i] = qt + 5, p
    bt = Batch([a + b for a, b in zip(n, prior)], n, W, S, Hkv * gq, Hkv, d, bs, bf16, seed=seed)
    assert kernel_of(bt) == "persistent"
    return bt


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gq", [1, 2, 4, 8])
@pytest.mark.parametrize("bs", [8, 16, 64, 128])
def test_persistent_prefill(d, gq, bs):
    """Windows of 6 to 8 tiles apart from the sinks' (the ring has 4 stages)."""
    bt = serving(gq, d, bs, S=40 if bs <= 16 else 70, seed=bs + gq)
    bt.check(run(bt))


@pytest.mark.parametrize("d,gq,bs", [(128, 4, 64), (64, 8, 128), (128, 1, 16), (64, 2, 8)])
def test_persistent_prefill_of_long_windows(d, gq, bs):
    """More (tile, block) slots per item than a batch of table entries holds,
    for every page size."""
    bt = serving(gq, d, bs, W=2300, S=70, Hkv=8, far=(20, 90), deep=(2700, 2650), seed=bs)
    bt.check(run(bt))


@pytest.mark.parametrize("d,gq,bs", [(128, 4, 16), (64, 1, 32), (64, 8, 64)])
def test_persistent_prefill_rescales(d, gq, bs):
    """Scores of up to about 60: the maximum moves past its headroom in later tiles."""
    bt = serving(gq, d, bs, seed=7)
    check_peaked(bt, run(bt, scale=1.0), 1.0)


@pytest.mark.parametrize("d,gq,bs", [(128, 4, 16), (64, 1, 32)])
def test_split_prefill_rescales(d, gq, bs):
    bt = Batch([1500, 700], [40, 30], 1200, 70, 2 * gq, 2, d, bs, bf16, seed=8)
    assert kernel_of(bt) == "split"
    check_peaked(bt, run(bt, scale=1.0), 1.0)


def test_persistent_prefill_of_more_requests_than_a_launch():
    """300 requests with several tiles each: a second launch behind the first."""
    rng = np.random.default_rng(4)
    n = [int(x) for x in rng.integers(0, 9, size=300)]
    lens = [int(x + y) for x, y in zip(n, rng.integers(0, 500, size=300))]
    bt = Batch(lens, n, 200, 5, 8, 2, 64, 8, bf16, seed=4)
    assert kernel_of(bt) == "persistent"
    bt.check(run(bt))


def test_persistent_prefill_placement_streams_and_graphs():
    """The same bits under another placement, back to back, on two streams and
    replayed from a graph beside eager calls."""
    from paged_kv_cache_192_gb300 import ops
    a, c = serving(4, 128, 16, seed=1), serving(8, 64, 8, seed=2)
    ra, rc = run(a), run(c)
    perm = torch.randperm(a.k_cache.shape[0], generator=torch.Generator().manual_seed(1)).to(DEV)
    k2, v2 = torch.empty_like(a.k_cache), torch.empty_like(a.v_cache)
    k2[perm], v2[perm] = a.k_cache, a.v_cache
    t2 = torch.where(a.table_t >= 0, perm[a.table_t.clamp(min=0).long()].int(), a.table_t)
    assert torch.equal(ra, ops.prefill_window(a.q_t, k2, v2, t2, a.start_t, a.lens_t, max(a.n_new), a.W, a.S))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    s1.wait_stream(torch.cuda.current_stream())
    s2.wait_stream(torch.cuda.current_stream())
    outs = [prefill(a) for _ in range(6)]
    other = []
    for _ in range(4):
        outs.append(prefill(a, stream=s1))
        other.append(prefill(c, stream=s2))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ra) for o in outs) and all(torch.equal(o, rc) for o in other)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = prefill(a)
    for _ in range(3):
        o.zero_()
        g.replay()
        e = prefill(c)
    torch.cuda.synchronize()
    assert torch.equal(o, ra) and torch.equal(e, rc) and ops.device_error() == 0


def test_persistent_prefill_leaves_rows_outside_the_requests():
    from paged_kv_cache_192_gb300 import ops
    bt = serving(4, 128, 16, seed=3)
    T = sum(bt.n_new)
    pad = torch.full((40, bt.Hq, bt.d), float("nan"), dtype=bf16, device=DEV)
    q = torch.cat([pad[:5], bt.q_t, pad])
    out = torch.full_like(q, 7.0)
    ops.prefill_window(q, bt.k_cache, bt.v_cache, bt.table_t, bt.start_t + 5, bt.lens_t, max(bt.n_new),
                       bt.W, bt.S, out=out)
    torch.cuda.synchronize()
    assert ops.device_error() == 0
    assert (out[:5] == 7.0).all() and (out[5 + T:] == 7.0).all()
    bt.check(out[5:5 + T])


def small():
    bt = Batch([90, 600], [30, 70], 50, 3, 8, 2, 128, 16, bf16)
    assert kernel_of(bt) == "split"
    return bt


@pytest.mark.parametrize("make", [small, lambda: serving(4, 128, 16, seed=5)], ids=["split", "persistent"])
def test_freed_entries_of_a_prefill_are_not_read(make):
    """Table entries of freed pages may be anything; a bad entry of a visible
    page is recorded and leaves the other requests whole."""
    from paged_kv_cache_192_gb300 import ops
    bt = make()
    good = run(bt)
    t = bt.table_t.clone()
    assert (t < 0).any()
    t[t < 0] = 2 ** 31 - 1
    assert torch.equal(prefill(bt, table=t), good)
    torch.cuda.synchronize()
    assert ops.device_error() == 0
    t[0, (bt.lens[0] - 1) // bt.bs] = bt.k_cache.shape[0]
    got = prefill(bt, table=t)
    torch.cuda.synchronize()
    assert ops.device_error() == 1
    assert torch.equal(got[bt.n_new[0]:], good[bt.n_new[0]:])


@pytest.mark.parametrize("make", [small, lambda: serving(4, 128, 16, seed=6)], ids=["split", "persistent"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_value_stays_with_its_request_and_head(make, bad):
    """A NaN or infinity in one head's K reaches the queries that see the token
    and no other.  In V it reaches those, and may reach others of the same
    request and KV head (their weight is 0, and 0 x NaN is NaN), but not another
    request or head."""
    bt = make()
    good = run(bt)
    r, h = 0, 1
    n, L, gq = bt.n_new[r], bt.lens[r], bt.Hq // bt.Hkv
    j = L - n + 5  # seen by new tokens 5, 6, ... (all within the window here)
    blk, off = int(bt.table[r, j // bt.bs]), j % bt.bs
    rows = torch.zeros(good.shape[:2], dtype=torch.bool, device=DEV)
    rows[5:min(n, 5 + bt.W), h * gq:(h + 1) * gq] = True
    for pool, spread in ((bt.k_cache, False), (bt.v_cache, True)):
        old = pool[blk, h, off].clone()
        pool[blk, h, off] = bad
        got = run(bt)
        pool[blk, h, off] = old
        broken = ~torch.isfinite(got.float()).all(-1)
        if spread:
            assert bool(broken[rows].all())
            rows[:n, h * gq:(h + 1) * gq] = True  # may be broken
        elif bad != bad:
            assert bool(broken[rows].all())
        assert torch.equal(got[~rows], good[~rows])


# ---- decode -----------------------------------------------------------------------
def decode(bt, **kw):
    from paged_kv_cache_192_gb300 import ops
    out = ops.decode_window(bt.q_t, bt.k_cache, bt.v_cache, bt.table_t, bt.lens_t, bt.W, bt.S, **kw)
    torch.cuda.synchronize()
    assert ops.device_error() == 0
    return out


def ragged(B, W, S, gq, d, bs, dtype, seed=0):
    """B sequences, three of them longer than the window and apart from the
    sinks, the rest short; 8 KV heads."""
    rng = np.random.default_rng(seed)
    lens = [int(x) for x in rng.integers(0, 60, size=B)]
    lens[1], lens[B // 2], lens[-1] = W + 333, 2 * W + 71, W + S + 1
    return Batch(lens, [1] * B, W, S, 8 * gq, 8, d, bs, dtype, seed=seed)


@pytest.mark.parametrize("dtype,d,gq", [(bf16, 128, 4), (bf16, 64, 1), (bf16, 64, 8), (f32, 64, 1),
                                        (f32, 128, 4), (f32, 128, 8)])
@pytest.mark.parametrize("W,bs", [(2133, 8), (4260, 16)])
def test_decode_of_many_tiles_per_warp(dtype, d, gq, W, bs):
    """Too many (sequence, KV head) items for clusters (every SM has at most 3
    CTAs of 64 KB, 456 on 152): a warp walks a quarter of a window, 33 tiles or
    more of the tensor-core tile, past the 32 or 16 whose table entries it holds
    at first."""
    B = 1 + 4 * torch.cuda.get_device_properties(0).multi_processor_count // 8
    bt = ragged(B, W, 40, gq, d, bs, dtype, seed=bs)
    bt.check(decode(bt))


@pytest.mark.parametrize("B", [40, 50, 57, 60, 64, 70, 76, 80, 100, 120])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_batches_around_a_full_wave(B, d):
    """Item counts around and past what runs at once, of long windows: the
    ordinary ring, and the deeper one where the last wave would be short (320
    to 960 items; 512 of d 128 take it on 152 SMs), which then wraps."""
    bt = ragged(B, 2133, 40, 4, d, 16, bf16, seed=B)
    bt.check(decode(bt))


@pytest.mark.parametrize("B", [1, 64])
@pytest.mark.parametrize("d,gq,bs", [(128, 4, 16), (64, 1, 8)])
def test_decode_rescales(B, d, gq, bs):
    """Clusters and none, with scores of up to about 60."""
    bt = ragged(max(B, 3), 1100, 20, gq, d, bs, bf16, seed=9) if B > 1 else \
        Batch([3000], [1], 1100, 20, 8 * gq, 8, d, bs, bf16, seed=9)
    check_peaked(bt, decode(bt, scale=1.0), 1.0)


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_value_of_a_decode_stays_with_its_sequence_and_head(dtype, bad):
    bt = Batch([700, 700, 33], [1, 1, 1], 300, 20, 8, 2, 128, 16, dtype, seed=2)
    good = decode(bt)
    for pool in (bt.k_cache, bt.v_cache):
        blk, off = int(bt.table[0, 650 // 16]), 650 % 16
        old = pool[blk, 1, off].clone()
        pool[blk, 1, off] = bad
        got = decode(bt)
        pool[blk, 1, off] = old
        assert torch.equal(got[1:], good[1:]) and torch.equal(got[0, :4], good[0, :4])
        if pool is bt.v_cache or bad != bad:
            assert not torch.isfinite(got[0, 4:].float()).any()
