"""pa_cross_attention against the formula in 64 bits: query rows of every number
(the streaming kernel's sets of columns, the tensor-core kernels), encoder lengths
that end anywhere in a page, none at all, freed pages, poisoned slots."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_192_gb300 import build
    build.build()


class Cross:
    """Requests of n[r] query rows over e[r] states; slots behind the states hold NaN or
    infinities, table entries behind them -1, `gap` rows of q belong to no request."""

    def __init__(self, n, e, Hq=4, Hkv=2, d=64, bs=16, seed=0, extra_blocks=0, gap=0, num_blocks=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.n, self.e, self.Hq, self.Hkv, self.d = n, e, Hq, Hkv, d
        blocks = [-(-x // bs) for x in e]
        need = sum(blocks)
        NB = num_blocks or need + 3
        ids = (rng.permutation(NB) if num_blocks is None else np.arange(NB - need, NB))[:need]
        self.table = np.full((len(n), max(1, max(blocks)) + extra_blocks), -1, np.int32)
        poison = torch.tensor([float("nan"), float("inf"), -float("inf")])
        pools = [poison[torch.randint(0, 3, (need, Hkv, bs, d), generator=g)].to(bf16) for _ in range(2)]
        self.k, self.v, at = [], [], 0
        for r, (m, x) in enumerate(zip(blocks, e)):
            self.table[r, :m] = ids[at:at + m]
            for pool, to in zip(pools, (self.k, self.v)):
                rows = torch.randn(x, Hkv, d, generator=g).to(bf16)
                to.append(rows)
                for j in range(m):
                    part = rows[j * bs:(j + 1) * bs]
                    pool[at + j, :, :len(part)] = part.transpose(0, 1)
            at += m
        full = []
        for pool in pools:
            t = torch.full((NB, Hkv, bs, d), float("nan"), dtype=bf16, device="cuda") if num_blocks is None \
                else torch.empty(NB, Hkv, bs, d, dtype=bf16, device="cuda")
            if need:
                t[torch.from_numpy(ids).long().cuda()] = pool.cuda()
            full.append(t)
        self.k_cache, self.v_cache = full
        self.q = torch.randn(sum(n) + gap, Hq, d, generator=g).to(bf16)
        self.q_t, self.table_t = self.q.cuda(), torch.from_numpy(self.table).cuda()
        i32 = dict(dtype=torch.int32, device="cuda")
        self.start_t = torch.tensor([0] + list(np.cumsum(n)), **i32)
        self.lens_t = torch.tensor(e, **i32)

    def run(self, max_query_len=None, **kw):
        from paged_kv_cache_192_gb300 import ops
        out = ops.cross_attention(self.q_t, self.k_cache, self.v_cache, self.table_t, self.start_t, self.lens_t,
                                  max(self.n) if max_query_len is None else max_query_len, **kw)
        torch.cuda.synchronize()
        return out

    def reference(self, scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        out, at, gq = [], 0, self.Hq // self.Hkv
        for r, (n, e) in enumerate(zip(self.n, self.e)):
            q = self.q_t[at:at + n].double()
            at += n
            if e == 0:
                out.append(torch.zeros_like(q))
                continue
            k, v = (x[r].cuda().double().repeat_interleave(gq, 1) for x in (self.k, self.v))
            w = torch.softmax(torch.einsum("nhd,jhd->hnj", q, k) * scale, -1)
            out.append(torch.einsum("hnj,jhd->nhd", w, v))
        return torch.cat(out)

    def check(self, got, scale=None):
        """As of the windowed calls: half a step of the output, and 2^-13 of the largest
        value for the weights (scores in fp32, weights of 16 bits)."""
        from paged_kv_cache_192_gb300 import ops
        assert ops.device_error() == 0
        ref = self.reference(scale)
        got = got[:len(ref)].double()
        assert torch.isfinite(got).all(), "a slot behind the states entered the result"
        vmax = max([float(v.abs().max()) for v in self.v if v.numel()], default=1.0)
        err, tol = (got - ref).abs(), 2.0 ** -8 * ref.abs() + 2.0 ** -13 * vmax
        assert bool((err <= tol).all()), f"max excess {(err - tol).max():.3e}, max err {err.max():.3e}"


LENS = [1, 0, 2, 15, 16, 17, 31, 33, 63, 64, 65, 100, 129, 257, 300, 0, 511, 40]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gq", [1, 2, 4, 8])
@pytest.mark.parametrize("most", [1, 3, 8, 20, 70])
def test_rows_and_groups(d, gq, most):
    """Every set count of the streaming kernel and the tensor-core kernels, ragged."""
    rng = np.random.default_rng(most + gq)
    n = [most] + [int(x) for x in rng.integers(0, most + 1, size=len(LENS) - 1)]
    x = Cross(n, LENS, Hq=3 * gq, Hkv=3, d=d, seed=most)
    x.check(x.run())


@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("most,gq", [(1, 1), (5, 4), (40, 4), (300, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_page_sizes(bs, most, gq, d):
    x = Cross([most, 1, most // 2], [700, 129, 40], Hq=2 * gq, Hkv=2, bs=bs, d=d, seed=bs, extra_blocks=3)
    x.check(x.run())


@pytest.mark.parametrize("R,n,e", [(1, 1, 5000), (2, 4, 3001), (40, 1, 300), (330, 2, 60), (700, 1, 20),
                                   (1, 130, 4000), (3, 200, 900), (300, 40, 30), (600, 9, 33)])
@pytest.mark.parametrize("gq", [1, 8])
def test_clusters_and_waves(R, n, e, gq):
    """Few requests with many states to many with few; more than 256 requests."""
    rng = np.random.default_rng(R)
    x = Cross([n] + [int(v) for v in rng.integers(0, n + 1, size=R - 1)],
              [e] + [int(v) for v in rng.integers(0, e + 1, size=R - 1)], Hq=2 * gq, Hkv=2, d=128, seed=R)
    x.check(x.run())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,e,gq,Hkv", [
    ([650, 641], [8000, 1], 8, 2),                    # long states: two CTAs per query tile
    ([40] + [1] * 39, [6400, 0, 1, 63] * 10, 1, 4),   # most query tiles partly filled: four
    ([100, 33, 64] * 5, [500, 40, 0] * 5, 1, 16)])    # short states: one
def test_query_tiles_in_several_waves(n, e, gq, Hkv, d):
    x = Cross(n, e, Hq=gq * Hkv, Hkv=Hkv, d=d, seed=len(n))
    x.check(x.run())


@pytest.mark.parametrize("most", [1, 30, 100])
def test_no_states_at_all(most):
    x = Cross([most, 1, 0], [0, 0, 0])
    out = torch.full_like(x.q_t, float("nan"))
    x.run(out=out)
    assert bool((out == 0).all())


@pytest.mark.parametrize("most", [2, 30, 100])
def test_rows_outside_every_request_stay(most):
    x = Cross([most, 0, 1], [50, 20, 0], gap=9)
    out = torch.full_like(x.q_t, 7.0)
    x.check(x.run(out=out))
    assert bool((out[-9:] == 7).all())
    x.start_t += 4  # and rows before the first
    x.q_t[4:] = x.q_t[:-4].clone()
    out.fill_(7.0)
    x.run(out=out)
    assert bool((out[:4] == 7).all()) and bool((out[-5:] == 7).all())
    x.q_t = x.q_t[4:]
    x.check(out[4:])


@pytest.mark.parametrize("most", [2, 30, 100])
@pytest.mark.parametrize("what,i,value", [("lens_t", 1, -1), ("lens_t", 1, 10 ** 6), ("start_t", 3, 10 ** 6),
                                          ("start_t", 2, -1), ("start_t", 2, 2 ** 31 - 1)])
def test_requests_that_do_not_fit(most, what, i, value):
    """Recorded, nothing out of range read; request 0 is right."""
    from paged_kv_cache_192_gb300 import ops
    x = Cross([most, most, most], [50, 20, 33])
    getattr(x, what)[i] = value
    out = torch.full_like(x.q_t, 7.0)
    x.run(out=out)
    assert ops.device_error() == 4
    x.n, x.e = [most], [50]
    x.check(out)


@pytest.mark.parametrize("most", [2, 30, 100])
def test_pages_outside_the_pool_are_recorded(most):
    from paged_kv_cache_192_gb300 import ops
    x = Cross([most, most], [50, 40])
    x.table_t[1, 1] = x.k_cache.shape[0]
    out = x.run()
    assert ops.device_error() == 1
    x.n, x.e = [most], [50]
    x.check(out)


def test_max_query_len_too_small_for_the_streaming_kernel():
    from paged_kv_cache_192_gb300 import ops
    x = Cross([8, 9], [50, 40], Hq=2, Hkv=2)
    out = torch.full_like(x.q_t, 7.0)
    x.run(max_query_len=8, out=out)
    assert ops.device_error() == 4 and bool((out[8:] == 7).all())
    x.n, x.e = [8], [50]
    x.check(out)


@pytest.mark.parametrize("most", [1, 100])
def test_pool_past_4_gib(most):
    d, Hkv, bs = 128, 2, 16
    x = Cross([most, 2], [700, 33], Hq=8, Hkv=Hkv, d=d, bs=bs, num_blocks=2 ** 32 // (Hkv * bs * d * 2) + 200)
    x.check(x.run())


@pytest.mark.parametrize("most", [1, 12, 100])
def test_placement_does_not_change_a_bit(most):
    x = Cross([most] * 4, [100, 33, 600, 0], Hq=8, d=128)
    a = x.run()
    perm = torch.randperm(x.k_cache.shape[0], generator=torch.Generator().manual_seed(1)).cuda()
    k2, v2 = torch.empty_like(x.k_cache), torch.empty_like(x.v_cache)
    k2[perm], v2[perm] = x.k_cache, x.v_cache
    x.table_t = torch.where(x.table_t >= 0, perm[x.table_t.clamp(min=0).long()].int(), x.table_t)
    x.k_cache, x.v_cache = k2, v2
    assert torch.equal(a, x.run())


@pytest.mark.parametrize("most", [1, 100])
def test_scale_stream_and_graph(most):
    x = Cross([most, 3], [100, 333], Hq=8, d=128)
    out = torch.full_like(x.q_t, float("nan"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert x.run(scale=0.3, out=out, stream=side).data_ptr() == out.data_ptr()
    x.check(out, scale=0.3)
    g = torch.cuda.CUDAGraph()
    from paged_kv_cache_192_gb300 import ops
    with torch.cuda.graph(g):
        got = ops.cross_attention(x.q_t, x.k_cache, x.v_cache, x.table_t, x.start_t, x.lens_t, max(x.n))
    keep_k, keep_v = x.k, x.v
    for e in ([100, 333], [64, 0], [0, 1]):
        x.e = e
        x.lens_t.copy_(torch.tensor(e))
        x.k, x.v = ([a[:m] for a, m in zip(p, e)] for p in (keep_k, keep_v))
        g.replay()
        torch.cuda.synchronize()
        x.check(got)


def test_a_decode_of_the_whole_context_agrees():
    """One row per request, as pa_decode over the same pages."""
    from paged_kv_cache_192_gb300 import ops
    x = Cross([1] * 5, [5, 100, 333, 1000, 64], Hq=8, d=128)
    x.check(x.run())
    x.check(ops.decode(x.q_t, x.k_cache, x.v_cache, x.table_t.clamp(min=0), x.lens_t))


def test_validate_mode():
    from paged_kv_cache_192_gb300 import _lib, ops
    x = Cross([2, 3], [50, 40])
    ops.set_validate(True)
    try:
        x.check(x.run())
        for t, i, v, msg in ((x.lens_t, 1, -1, "encoder_lens"), (x.lens_t, 1, 10 ** 5, "encoder_lens"),
                             (x.start_t, 2, 6, "rows"), (x.table_t, (0, 1), -1, "outside pool")):
            keep = t[i].clone()
            t[i] = v
            with pytest.raises(_lib.PAError, match=msg):
                x.run()
            t[i] = keep
        with pytest.raises(_lib.PAError, match="max_query_len 2"):
            x.run(max_query_len=2)
    finally:
        ops.set_validate(False)
