"""pa_decode_window against the formula in 64 bits: windows and sinks of every
relation to the context (inside, touching, beyond it), page sizes, head groups
and both types; freed pages, poisoned invisible slots, empty rows, placement,
streams, graphs and pools past 2^32 bytes."""
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


def run(bt, **kw):
    from paged_kv_cache_192_gb300 import ops
    out = ops.decode_window(bt.q_t, bt.k_cache, bt.v_cache, bt.table_t, bt.lens_t, bt.W,
                            num_sinks=bt.S, **kw)
    torch.cuda.synchronize()
    assert ops.device_error() == 0
    return out


RAGGED = [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 64, 100, 129, 257, 300, 0, 511, 40, 0, 5]


def batch(lens, W, S, Hq=8, Hkv=2, d=128, bs=16, dtype=bf16, **kw):
    return Batch(lens, [1] * len(lens), W, S, Hq, Hkv, d, bs, dtype, **kw)


@pytest.mark.parametrize("W,S", [(1, 0), (1, 3), (7, 0), (7, 1), (16, 16), (33, 4), (100, 37),
                                 (64, 64), (250, 8), (2 ** 31 - 1, 0), (5, 2 ** 31 - 1)])
@pytest.mark.parametrize("dtype", [bf16, f32])
def test_windows_and_sinks(W, S, dtype):
    bt = batch(RAGGED, W, S, dtype=dtype, seed=W % 97)
    bt.check(run(bt))


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gq", [1, 2, 4, 8])
@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128])
def test_shapes(dtype, d, gq, bs):
    bt = batch([1, 30, 257, 0, 500], 77, 5, Hq=3 * gq, Hkv=3, d=d, bs=bs, dtype=dtype, seed=bs + gq)
    bt.check(run(bt))


@pytest.mark.parametrize("B,L,W", [(1, 5000, 4100), (1, 1300, 1024), (2, 3000, 700), (40, 300, 200),
                                   (330, 60, 33), (700, 20, 64)])
@pytest.mark.parametrize("dtype,gq", [(bf16, 4), (bf16, 1), (f32, 8)])
def test_cluster_sizes(B, L, W, dtype, gq):
    """Few sequences with long windows (large clusters) to many short ones."""
    rng = np.random.default_rng(B)
    lens = [L] + [int(x) for x in rng.integers(1, L + 1, size=B - 1)]
    bt = batch(lens, W, 4, Hq=2 * gq, Hkv=2, dtype=dtype, seed=B)
    bt.check(run(bt))


@pytest.mark.parametrize("d,B", [(128, 230), (64, 310)])
@pytest.mark.parametrize("gq", [1, 8])
def test_batches_that_end_in_a_short_wave(d, B, gq):
    """A few more items than run at once: the kernel with the deeper ring."""
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(1, 150, size=B)]
    bt = batch(lens, 70, 3, Hq=2 * gq, Hkv=2, d=d, bs=8, seed=B)
    bt.check(run(bt))


def test_window_beyond_the_context_matches_decode():
    from paged_kv_cache_192_gb300 import ops
    bt = batch([5, 100, 333, 1000], 1000, 0)
    got = run(bt)
    ref = ops.decode(bt.q_t, bt.k_cache, bt.v_cache, bt.table_t, bt.lens_t)
    bt.check(got)
    bt.check(ref)


def test_scale_and_out():
    from paged_kv_cache_192_gb300 import ops
    bt = batch([5, 100, 333], 50, 3)
    out = torch.full_like(bt.q_t, float("nan"))
    r = ops.decode_window(bt.q_t, bt.k_cache, bt.v_cache, bt.table_t, bt.lens_t, 50, 3, scale=0.3,
                          out=out)
    assert r.data_ptr() == out.data_ptr()
    bt.check(out, scale=0.3)


def test_placement_does_not_change_a_bit():
    from paged_kv_cache_192_gb300 import ops
    bt = batch(RAGGED, 100, 20, seed=3)
    a = run(bt)
    perm = torch.randperm(bt.k_cache.shape[0], generator=torch.Generator().manual_seed(1)).to(DEV)
    k2, v2 = torch.empty_like(bt.k_cache), torch.empty_like(bt.v_cache)
    k2[perm], v2[perm] = bt.k_cache, bt.v_cache
    t2 = torch.where(bt.table_t >= 0, perm[bt.table_t.clamp(min=0).long()].int(), bt.table_t)
    b = ops.decode_window(bt.q_t, k2, v2, t2, bt.lens_t, 100, 20)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_pool_past_4_gib(dtype):
    """Pages at the end of a pool whose byte offsets pass 2^32."""
    d, Hkv, bs = 128, 2, 16
    NB = (2 ** 32 // (Hkv * bs * d * (2 if dtype == bf16 else 4))) + 200
    bt = batch([700, 33, 1000], 300, 10, Hq=8, Hkv=Hkv, d=d, bs=bs, dtype=dtype, num_blocks=NB)
    bt.check(run(bt))


def test_freed_entries_may_hold_anything_and_bad_ones_are_recorded():
    from paged_kv_cache_192_gb300 import ops
    bt = batch([900, 400], 100, 20)
    t = bt.table_t.clone()
    t[bt.table_t < 0] = 2 ** 31 - 1
    got = ops.decode_window(bt.q_t, bt.k_cache, bt.v_cache, t, bt.lens_t, 100, 20)
    bt.check(got)
    assert ops.device_error() == 0
    t[1, 399 // 16] = bt.k_cache.shape[0]  # the newest token's page: outside the pool
    got = ops.decode_window(bt.q_t, bt.k_cache, bt.v_cache, t, bt.lens_t, 100, 20)
    torch.cuda.synchronize()
    assert ops.device_error() == 1
    assert torch.equal(got[0].cpu(), run(bt)[0].cpu())  # the other sequence is whole


def test_length_past_the_table_is_recorded():
    from paged_kv_cache_192_gb300 import ops
    bt = batch([64, 64], 64, 0)
    lens = torch.tensor([64, 65], dtype=torch.int32, device=DEV)
    ops.decode_window(bt.q_t, bt.k_cache, bt.v_cache, bt.table_t, lens, 64)
    assert ops.device_error() == 1
    lens = torch.tensor([64, -1], dtype=torch.int32, device=DEV)
    out = ops.decode_window(bt.q_t, bt.k_cache, bt.v_cache, bt.table_t, lens, 64)
    assert ops.device_error() == 1
    assert not out[1].any()


def test_validate_mode():
    from paged_kv_cache_192_gb300 import ops
    from paged_kv_cache_192_gb300._lib import PAError
    bt = batch([900, 400, 0], 100, 20)
    ops.set_validate(True)
    try:
        bt.check(run(bt))  # freed entries (-1) pass
        t = bt.table_t.clone()
        t[0, 0] = -1  # a sink's page
        with pytest.raises(PAError, match="block_table"):
            ops.decode_window(bt.q_t, bt.k_cache, bt.v_cache, t, bt.lens_t, 100, 20)
        with pytest.raises(PAError, match="context_lens"):
            ops.decode_window(bt.q_t, bt.k_cache, bt.v_cache, bt.table_t, bt.lens_t + 4096, 100, 20)
    finally:
        ops.set_validate(False)


def test_streams_and_graphs():
    """Two streams at once, and a captured call replayed on new inputs while
    eager calls run beside it: every result is the plain call's."""
    from paged_kv_cache_192_gb300 import ops
    a, c = batch([900, 400, 77], 300, 20, seed=1), batch([300] * 9, 128, 4, seed=2)
    ra, rc = run(a), run(c)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    s1.wait_stream(torch.cuda.current_stream())
    s2.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(8):
        outs.append(ops.decode_window(a.q_t, a.k_cache, a.v_cache, a.table_t, a.lens_t, a.W, a.S,
                                      stream=s1))
        outs.append(ops.decode_window(c.q_t, c.k_cache, c.v_cache, c.table_t, c.lens_t, c.W, c.S,
                                      stream=s2))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ra) for o in outs[::2])
    assert all(torch.equal(o, rc) for o in outs[1::2])
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    q = a.q_t.clone()
    with torch.cuda.graph(g1):
        o1 = ops.decode_window(q, a.k_cache, a.v_cache, a.table_t, a.lens_t, a.W, a.S)
    with torch.cuda.graph(g2):
        o2 = ops.decode_window(c.q_t, c.k_cache, c.v_cache, c.table_t, c.lens_t, c.W, c.S)
    for _ in range(3):
        g1.replay()
        g2.replay()
        e = ops.decode_window(c.q_t, c.k_cache, c.v_cache, c.table_t, c.lens_t, c.W, c.S)
    torch.cuda.synchronize()
    assert torch.equal(o1, ra) and torch.equal(o2, rc) and torch.equal(e, rc)
    q.mul_(0.5)
    g1.replay()
    torch.cuda.synchronize()
    half = ops.decode_window(q, a.k_cache, a.v_cache, a.table_t, a.lens_t, a.W, a.S)
    assert torch.equal(o1, half) and not torch.equal(o1, ra)


def test_tensors_elsewhere_and_of_other_types_are_refused():
    from paged_kv_cache_192_gb300 import ops
    bt = batch([30], 16, 0)
    args = dict(q=bt.q_t, k_cache=bt.k_cache, v_cache=bt.v_cache, block_table=bt.table_t,
                context_lens=bt.lens_t, window=16)
    for name in ("k_cache", "v_cache", "block_table", "context_lens"):
        with pytest.raises(ValueError, match=f"{name} must be a CUDA tensor on cuda:0"):
            ops.decode_window(**{**args, name: args[name].cpu()})
    for name, other in (("q", f32), ("v_cache", f32), ("block_table", torch.int64),
                        ("context_lens", torch.int64)):
        with pytest.raises(TypeError, match=f"{name} must be"):
            ops.decode_window(**{**args, name: args[name].to(other)})
    with pytest.raises(TypeError, match="unsupported dtype"):
        ops.decode_window(**{**args, **{n: args[n].half() for n in ("q", "k_cache", "v_cache")}})
    wide = torch.zeros(1, 8, 256, dtype=bf16, device=DEV)
    with pytest.raises(ValueError, match="q must be contiguous"):
        ops.decode_window(**{**args, "q": wide[..., ::2]})
    with pytest.raises(ValueError, match="out must be contiguous"):
        ops.decode_window(**{**args, "out": wide[..., ::2]})
    with pytest.raises(TypeError, match="out must be"):
        ops.decode_window(**{**args, "out": torch.zeros(1, 8, 128, device=DEV)})
    with pytest.raises(AttributeError):
        ops.decode_window(**args, stream=7)


def test_empty_batch():
    from paged_kv_cache_192_gb300 import ops
    bt = batch([30], 16, 0)
    out = ops.decode_window(bt.q_t[:0], bt.k_cache, bt.v_cache, bt.table_t[:0], bt.lens_t[:0], 16)
    assert out.shape == (0, 8, 128)
