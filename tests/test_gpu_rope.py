"""pa_rope_reshape_and_cache against the rotation in 64 bits and the slot rule."""
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


class Case:
    def __init__(self, T, Hq, Hkv, d, bs, dtype, axes=1, rot=None, inter=False, far=5000, NB=None,
                 fused=False, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.rot = rot or d
        half = self.rot // 2
        self.T, self.Hq, self.Hkv, self.d, self.bs, self.dtype, self.inter = T, Hq, Hkv, d, bs, dtype, inter
        self.NB = NB or -(-T // bs) + 3
        if fused:
            qkv = torch.randn(T, (Hq + 2 * Hkv) * d, generator=g).to(dtype).to(DEV)
            self.q = qkv[:, :Hq * d].view(T, Hq, d)
            self.k = qkv[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d)
            self.v = qkv[:, (Hq + Hkv) * d:].view(T, Hkv, d)
        else:
            self.q = torch.randn(T, Hq, d, generator=g).to(dtype).to(DEV)
            self.k = torch.randn(T, Hkv, d, generator=g).to(dtype).to(DEV)
            self.v = torch.randn(T, Hkv, d, generator=g).to(dtype).to(DEV)
        slots = np.random.default_rng(seed).permutation(self.NB * bs)[:T].astype(np.int64)
        if T > 4:
            slots[[1, T - 2]] = -1
        self.slots = torch.from_numpy(slots).to(DEV)
        pos = torch.randint(0, far, (axes, T), generator=g)
        if T > 1:
            pos[:, 0], pos[:, 1] = far - 1, 0
        self.pos = pos.to(DEV)
        self.inv = (10000.0 ** (-torch.arange(half).double() / half)).float().to(DEV)
        self.sections = (half,) if axes == 1 else (half // 4, 0, half - half // 4) if axes == 3 else \
            (half - 3, 1, 1, 1)
        shape = (self.NB, Hkv, bs, d)
        self.k_cache = torch.randn(shape, generator=g).to(dtype).to(DEV)
        self.v_cache = torch.randn(shape, generator=g).to(dtype).to(DEV)

    def rotated(self, x):
        """(64-bit rotation, |x| + |y| of each element's pair)"""
        half, x = self.rot // 2, x.double().cpu()
        axis = torch.repeat_interleave(torch.arange(len(self.sections)), torch.tensor(self.sections))
        a = self.pos.cpu().double()[axis].t() * self.inv.cpu().double()  # [T][half]
        c, s = a.cos()[:, None], a.sin()[:, None]
        y, mag = x.clone(), torch.zeros_like(x)
        i = torch.arange(half)
        ia, ib = (2 * i, 2 * i + 1) if self.inter else (i, i + half)
        u, w = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = u * c - w * s, u * s + w * c
        mag[..., ia] = mag[..., ib] = u.abs() + w.abs()
        return y, mag

    def run(self, **kw):
        from paged_kv_cache_192_gb300 import ops
        sec = {} if len(self.sections) == 1 else dict(sections=self.sections)
        pos = self.pos[0] if len(self.sections) == 1 else self.pos
        return ops.rope_reshape_and_cache(self.q, self.k, self.v, self.k_cache, self.v_cache,
                                          self.slots, pos, self.inv, interleaved=self.inter, **sec,
                                          **kw)

    def close(self, got, x):
        """The angle in half turns rounded to fp32 (pi 2^-25), cos and sin to an
        ulp (2^-24) and three roundings of products and their sum (2^-24 each):
        3.4e-7 < 2^-21 of |x| + |y|, then half a step of the type."""
        ref, mag = self.rotated(x)
        got = got.double().cpu()
        half_step = 2.0 ** -8 if self.dtype == bf16 else 2.0 ** -24
        tol = 2.0 ** -21 * mag + half_step * ref.abs() * (1 + 2.0 ** -8)
        err = (got - ref).abs()
        assert bool((err <= tol).all()), f"max excess {(err - tol).max():.3e}"
        assert torch.equal(got[..., self.rot:], x.double().cpu()[..., self.rot:])

    def check(self, q_out, q, k, kc0, vc0):
        from paged_kv_cache_192_gb300 import ops
        torch.cuda.synchronize()
        assert ops.device_error() == 0
        self.close(q_out, q)
        ok = self.slots >= 0
        blk, off = self.slots[ok] // self.bs, self.slots[ok] % self.bs
        self.close_k(self.k_cache[blk, :, off], k, ok)
        assert torch.equal(self.v_cache[blk, :, off], self.v[ok])
        kc0[blk, :, off] = self.k_cache[blk, :, off]
        vc0[blk, :, off] = self.v[ok]
        assert torch.equal(self.k_cache, kc0) and torch.equal(self.v_cache, vc0)  # the rest as it was

    def close_k(self, got, k, ok):
        full = k.clone()
        full[ok] = got
        ref, mag = self.rotated(k)
        skip = ~ok.cpu()
        half_step = 2.0 ** -8 if self.dtype == bf16 else 2.0 ** -24
        tol = 2.0 ** -21 * mag + half_step * ref.abs() * (1 + 2.0 ** -8)
        err = (full.double().cpu() - ref).abs()
        assert bool((err <= tol)[~skip].all()), f"max excess {(err - tol)[~skip].max():.3e}"

    def run_and_check(self, **kw):
        q0, k0, kc0, vc0 = self.q.clone(), self.k.clone(), self.k_cache.clone(), self.v_cache.clone()
        out = self.run(**kw)
        self.check(out, q0, k0, kc0, vc0)
        return out


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("T", [1, 2, 5, 64, 333])
@pytest.mark.parametrize("inter", [False, True])
def test_tokens(dtype, T, inter):
    Case(T, 8, 2, 128, 16, dtype, inter=inter, seed=T).run_and_check()


@pytest.mark.parametrize("d,rot,Hq,Hkv,bs", [(128, 64, 32, 8, 16), (64, 64, 4, 4, 8), (128, 96, 3, 1, 128),
                                             (64, 16, 1, 1, 1), (256, 256, 8, 1, 32), (96, 32, 6, 3, 64),
                                             (512, 512, 2, 2, 16), (80, 80, 5, 5, 16)])
@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("inter", [False, True])
def test_shapes(d, rot, Hq, Hkv, bs, dtype, inter):
    Case(37, Hq, Hkv, d, bs, dtype, rot=rot, inter=inter, seed=d + rot).run_and_check()


@pytest.mark.parametrize("axes", [3, 4])
@pytest.mark.parametrize("inter", [False, True])
def test_axes(axes, inter):
    Case(50, 8, 2, 128, 16, bf16, axes=axes, inter=inter).run_and_check()
    Case(50, 8, 2, 64, 16, f32, axes=axes, inter=inter).run_and_check()


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_far_positions(dtype):
    Case(40, 4, 2, 128, 16, dtype, far=2 ** 31).run_and_check()


def test_negative_positions():
    c = Case(40, 4, 2, 128, 16, f32)
    c.pos.neg_()
    c.run_and_check()


@pytest.mark.parametrize("inter", [False, True])
def test_fused_projection_and_in_place(inter):
    c = Case(45, 8, 2, 128, 16, bf16, fused=True, inter=inter)
    assert not c.q.is_contiguous()
    c.run_and_check()
    c = Case(45, 8, 2, 128, 16, bf16, fused=True, rot=64, inter=inter, seed=4)
    out = c.run_and_check(q_out=c.q)
    assert out.data_ptr() == c.q.data_ptr()


def test_same_as_the_plain_store_without_rotation():
    """At position 0 nothing turns: the pools are pa_reshape_and_cache's."""
    from paged_kv_cache_192_gb300 import ops
    c = Case(60, 8, 2, 128, 16, bf16)
    c.pos.zero_()
    kc, vc = c.k_cache.clone(), c.v_cache.clone()
    out = c.run()
    ops.reshape_and_cache(c.k, c.v, kc, vc, c.slots)
    assert torch.equal(out, c.q) and torch.equal(c.k_cache, kc) and torch.equal(c.v_cache, vc)


def test_slot_outside_the_pool_is_recorded():
    from paged_kv_cache_192_gb300 import ops
    c = Case(20, 4, 2, 64, 16, bf16)
    kc = c.k_cache.clone()
    c.slots[7] = c.NB * c.bs
    out = c.run()
    torch.cuda.synchronize()
    assert ops.device_error() == 1
    c.close(out, c.q)
    c.slots[7] = -1
    c2 = c.k_cache.clone()
    c.k_cache.copy_(kc)
    c.run()
    assert torch.equal(c.k_cache, c2)  # the other tokens were stored


def test_pool_past_4_gib():
    c = Case(30, 4, 2, 128, 16, bf16, NB=4)
    NB = 2 ** 32 // (2 * 16 * 128 * 2) + 100
    big_k = torch.empty(NB, 2, 16, 128, dtype=bf16, device=DEV)
    big_v = torch.empty_like(big_k)
    from paged_kv_cache_192_gb300 import ops
    shift = (NB - 4) * 16
    ops.rope_reshape_and_cache(c.q, c.k, c.v, big_k, big_v,
                               torch.where(c.slots < 0, c.slots, c.slots + shift), c.pos[0], c.inv)
    c.run()
    ok = c.slots >= 0
    blk, off = c.slots[ok] // 16, c.slots[ok] % 16
    assert torch.equal(big_k[NB - 4:][blk, :, off], c.k_cache[blk, :, off])
    assert torch.equal(big_v[NB - 4:][blk, :, off], c.v_cache[blk, :, off])


def test_graph_replay_and_stream():
    from paged_kv_cache_192_gb300 import ops
    c = Case(64, 8, 2, 128, 16, bf16)
    ref = c.run_and_check()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = c.run(stream=s)
    torch.cuda.synchronize()
    assert torch.equal(o, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = c.run()
    c.k_cache.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, ref) and ops.device_error() == 0
    ok = c.slots >= 0
    c.close_k(c.k_cache[c.slots[ok] // 16, :, c.slots[ok] % 16], c.k, ok)


def test_validate_mode():
    from paged_kv_cache_192_gb300 import ops
    from paged_kv_cache_192_gb300._lib import PAError
    c = Case(20, 4, 2, 64, 16, bf16)
    ops.set_validate(True)
    try:
        c.run_and_check()
        c.slots[3] = c.slots[4]
        with pytest.raises(PAError, match="duplicate"):
            c.run()
        c.slots[3] = c.NB * c.bs
        with pytest.raises(PAError, match="out of pool"):
            c.run()
    finally:
        ops.set_validate(False)
