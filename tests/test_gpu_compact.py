"""pa_compact_cache: bit exact against row copies on the host, in place and
into other pages."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
bf16, f32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_192_gb300 import build
    build.build()


def bits(t):
    t = t.cpu()
    return (t.view(torch.int16) if t.dtype == bf16 else t.view(torch.int32)).numpy()


class Case:
    """mode: "in_place" (the same pages), "fresh" (other pages), "mixed" (every
    other page replaced)."""

    def __init__(self, lens, n_keep, Hkv, d, bs, dtype, mode, seed=0, kind="random", base=0, NB=None):
        rng = np.random.default_rng(seed)
        self.lens, self.n, self.Hkv, self.bs = lens, n_keep, Hkv, bs
        B = len(lens)
        MBs = max(-(-L // bs) for L in lens) + 1
        MBd = max(1, max(-(-n // bs) for n in n_keep))
        total = sum(-(-L // bs) for L in lens) + sum(-(-n // bs) for n in n_keep)
        self.NB = NB or total + 2
        ids = iter(base + rng.permutation(total + 2))
        self.src = np.full((B, MBs), -1, dtype=np.int32)
        self.dst = np.full((B, MBd), -1, dtype=np.int32)
        self.keep = np.full((B, Hkv, max(1, max(n_keep))), -7, dtype=np.int32)
        for b, (L, n) in enumerate(zip(lens, n_keep)):
            for j in range(-(-L // bs)):
                self.src[b, j] = next(ids)
            for j in range(-(-n // bs)):
                fresh = mode == "fresh" or (mode == "mixed" and j % 2)
                self.dst[b, j] = next(ids) if fresh else self.src[b, j]
            for h in range(Hkv):
                if kind == "random":
                    p = np.sort(rng.permutation(L)[:n])
                elif kind == "window":  # sinks and the last tokens
                    p = np.array([i if i < min(n, 4) else L - n + i for i in range(n)])
                else:  # everything up to n
                    p = np.arange(n)
                self.keep[b, h, :n] = p
        shape = (self.NB, Hkv, bs, d)
        self.k = torch.randn(total + 2, *shape[1:], generator=torch.Generator().manual_seed(seed)).to(dtype)
        self.v = torch.randn(total + 2, *shape[1:], generator=torch.Generator().manual_seed(seed + 1)).to(dtype)
        self.base = base
        if NB:
            self.kd = torch.empty(shape, dtype=dtype, device=DEV)
            self.vd = torch.empty_like(self.kd)
            self.kd[base:base + total + 2], self.vd[base:base + total + 2] = self.k.to(DEV), self.v.to(DEV)
        else:
            self.kd, self.vd = self.k.to(DEV), self.v.to(DEV)

    def args(self):
        t = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
        return (self.kd, self.vd, t(self.src), t(self.dst), t(self.keep),
                torch.tensor(self.n, dtype=torch.int32, device=DEV))

    def reference(self):
        out = []
        for pool in (self.k, self.v):
            old = bits(pool)
            new = old.copy()
            for b, n in enumerate(self.n):
                for h in range(self.Hkv):
                    for i in range(n):
                        j = self.keep[b, h, i]
                        new[self.dst[b, i // self.bs] - self.base, h, i % self.bs] = \
                            old[self.src[b, j // self.bs] - self.base, h, j % self.bs]
            out.append(new)
        return out

    def check(self):
        from paged_kv_cache_192_gb300 import ops
        torch.cuda.synchronize()
        assert ops.device_error() == 0
        rk, rv = self.reference()
        sl = slice(self.base, self.base + rk.shape[0])
        assert np.array_equal(bits(self.kd[sl]), rk) and np.array_equal(bits(self.vd[sl]), rv)


def run(c, **kw):
    from paged_kv_cache_192_gb300 import ops
    ops.compact_cache(*c.args(), **kw)


@pytest.mark.parametrize("mode", ["in_place", "fresh", "mixed"])
@pytest.mark.parametrize("kind", ["random", "window", "all"])
@pytest.mark.parametrize("Hkv,d,bs,dtype", [(2, 128, 16, bf16), (3, 64, 8, bf16), (1, 128, 128, f32),
                                            (8, 64, 32, f32), (2, 96, 16, bf16), (1, 8, 1, bf16)])
def test_batches(mode, kind, Hkv, d, bs, dtype):
    c = Case([1, 40, 333, 700, 5], [1, 17, 100, 699, 0], Hkv, d, bs, dtype, mode, kind=kind, seed=bs)
    run(c)
    c.check()


@pytest.mark.parametrize("mode", ["in_place", "fresh", "mixed"])
@pytest.mark.parametrize("B,L,n", [(1, 9000, 3000), (1, 9000, 8999), (3, 5000, 2501), (40, 700, 400)])
def test_long_in_place(mode, B, L, n):
    """Many chunks per head: rows that are read lie where others are written."""
    c = Case([L] * B, [n] * B, 2, 128, 16, bf16, mode, seed=B + n)
    run(c)
    c.check()


def test_padding_of_the_lists_is_not_read():
    c = Case([50, 60], [3, 30], 2, 64, 16, bf16, "in_place")
    assert (c.keep[0, :, 3:] < 0).all()
    run(c)
    c.check()


def test_pool_past_4_gib():
    NB = 2 ** 32 // (2 * 16 * 128 * 2) + 100
    c = Case([200, 300], [90, 100], 2, 128, 16, bf16, "mixed", base=NB - 60, NB=NB)
    run(c)
    c.check()


def test_bad_entries_are_skipped_and_recorded():
    from paged_kv_cache_192_gb300 import ops
    c = Case([100, 100], [20, 20], 2, 64, 16, bf16, "fresh")
    c.keep[0, 0, 3] = 10 ** 9
    c.keep[0, 1, 4] = -5
    c.src[1, 0] = c.NB
    c.dst[1, 1] = -1
    run(c)
    torch.cuda.synchronize()
    assert ops.device_error() == 1
    c.n[0], c.n[1] = 20, 16
    rk = bits(c.k).copy()
    old = bits(c.k)
    for b in range(2):
        for h in range(2):
            for i in range(c.n[b]):
                j = c.keep[b, h, i]
                if 0 <= j < c.src.shape[1] * 16 and 0 <= c.src[b, j // 16] < c.NB:
                    rk[c.dst[b, i // 16], h, i % 16] = old[c.src[b, j // 16], h, j % 16]
    assert np.array_equal(bits(c.kd), rk)


def test_stream_and_graph():
    from paged_kv_cache_192_gb300 import ops
    c = Case([400, 300], [90, 100], 2, 128, 16, bf16, "fresh")
    args = c.args()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ops.compact_cache(*args, stream=s)
    torch.cuda.synchronize()
    c.check()
    c.kd.copy_(c.k), c.vd.copy_(c.v)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.compact_cache(*args)
    c.kd.copy_(c.k), c.vd.copy_(c.v)
    g.replay()
    c.check()


@pytest.mark.parametrize("plant,msg", [("descending", "ascending"), ("twice", "written twice"),
                                       ("other", "written elsewhere"), ("outside", "outside pool"),
                                       ("many", "keep_lens")])
def test_validate_mode(plant, msg):
    from paged_kv_cache_192_gb300 import ops
    from paged_kv_cache_192_gb300._lib import PAError
    ops.set_validate(True)
    try:
        c = Case([100, 100], [40, 40], 2, 64, 16, bf16, "mixed")
        run(c)
        c.check()
        c = Case([100, 100], [40, 40], 2, 64, 16, bf16, "mixed")
        if plant == "descending":
            c.keep[1, 1, 7] = c.keep[1, 1, 8]
        elif plant == "twice":
            c.dst[1, 0] = c.dst[0, 0]
        elif plant == "other":
            c.keep[0, 0, :40] = np.arange(40)
            c.dst[1, 0] = c.src[0, 1]
            c.dst[0, 1] = c.src[1, 0]
        elif plant == "outside":
            c.dst[1, 0] = c.NB
        else:
            c.n[1] = 41
        with pytest.raises(PAError, match=msg):
            run(c)
    finally:
        ops.set_validate(False)


@pytest.mark.parametrize("mode", ["in_place", "fresh", "mixed"])
@pytest.mark.parametrize("d,bs,dtype", [(64, 16, bf16), (128, 16, bf16), (128, 8, f32), (256, 32, bf16)])
def test_several_batches_of_looked_up_rows(mode, d, bs, dtype):
    """Too many lists for clusters: one CTA per list, rows looked up 512 at a
    time; lists around and past one such batch.  Rows of 8 lanes (d 64) make a
    batch exactly as many chunks as there are stages."""
    B, Hkv = 40, 2
    assert B * Hkv * 8 >= 3 * torch.cuda.get_device_properties(0).multi_processor_count
    n = ([511, 512, 513, 1023, 1025, 2500, 1537, 3, 0, 2048] * 4)[:B]
    lens = [3000 if x > 1000 else 1400 + x for x in n]
    c = Case(lens, n, Hkv, d, bs, dtype, mode, seed=d + bs)
    run(c)
    c.check()


@pytest.mark.parametrize("mode", ["in_place", "mixed"])
@pytest.mark.parametrize("d,dtype", [(64, bf16), (128, f32)])
def test_several_batches_of_a_cluster(mode, d, dtype):
    """Few lists: a cluster's batch is 512 rows of each of its CTAs."""
    c = Case([20000], [17001], 2, d, 16, dtype, mode, seed=d)
    run(c)
    c.check()
