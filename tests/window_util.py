"""Inputs and the 64-bit reference of the windowed attention tests (not a test
module).

A batch's pages hold only what is visible: table entries of blocks without a
visible token are -1, and every slot that no query sees holds NaN or an
infinity, so that any use of one shows in the output.
"""
import numpy as np
import torch

DEV = "cuda"


def visible_range(L, first, W):
    """First token of the window of the earliest query (position `first`)."""
    return max(0, first - W + 1)


class Batch:
    """Sequences of the given lengths; the queries of sequence b sit at
    positions L_b - n_b .. L_b - 1."""

    def __init__(self, lens, n_new, W, S, Hq, Hkv, d, bs, dtype, seed=0, extra_blocks=0,
                 num_blocks=None, device=DEV):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed + 1)
        self.lens, self.n_new, self.W, self.S = lens, n_new, W, S
        self.Hq, self.Hkv, self.d, self.bs, self.dtype = Hq, Hkv, d, bs, dtype
        MB = max(1, max((-(-L // bs) for L in lens), default=1)) + extra_blocks
        kept = []
        for L, n in zip(lens, n_new):
            lo = visible_range(L, L - n, W)
            kept.append([j for j in range(-(-L // bs))
                         if n > 0 and (j * bs < S or min((j + 1) * bs, L) > lo)])
        need = sum(map(len, kept))
        NB = num_blocks or need + 3
        ids = (rng.permutation(NB) if num_blocks is None else np.arange(NB - need, NB))[:need]
        self.table = np.full((len(lens), MB), -1, dtype=np.int32)
        poison = torch.tensor([float("nan"), float("inf"), -float("inf")])
        k_pool = poison[torch.randint(0, 3, (need + 1, Hkv, bs, d), generator=g)]
        v_pool = poison[torch.randint(0, 3, (need + 1, Hkv, bs, d), generator=g)]
        self.k, self.v = [], []
        at = 0
        for b, (L, n) in enumerate(zip(lens, n_new)):
            lo = visible_range(L, L - n, W)
            k = torch.randn(L, Hkv, d, generator=g).to(dtype)
            v = torch.randn(L, Hkv, d, generator=g).to(dtype)
            self.k.append(k)
            self.v.append(v)
            for j in kept[b]:
                self.table[b, j] = ids[at]
                for t in range(j * bs, min((j + 1) * bs, L)):
                    if t < S or t >= lo:
                        k_pool[at, :, t - j * bs] = k[t].float()
                        v_pool[at, :, t - j * bs] = v[t].float()
                at += 1
        self.q = torch.randn(sum(n_new), Hq, d, generator=g).to(dtype)
        if num_blocks is None:
            full_k = torch.full((NB, Hkv, bs, d), float("nan")).to(dtype)
            full_v = full_k.clone()
            full_k[ids], full_v[ids] = k_pool[:need].to(dtype), v_pool[:need].to(dtype)
            self.k_cache, self.v_cache = full_k.to(device), full_v.to(device)
        else:  # a pool too large to fill: only the pages in use are written
            self.k_cache = torch.empty(NB, Hkv, bs, d, dtype=dtype, device=device)
            self.v_cache = torch.empty_like(self.k_cache)
            if need:
                self.k_cache[NB - need:] = k_pool[:need].to(dtype).to(device)
                self.v_cache[NB - need:] = v_pool[:need].to(dtype).to(device)
        self.table_t = torch.from_numpy(self.table).to(device)
        self.lens_t = torch.tensor(lens, dtype=torch.int32, device=device)
        self.start_t = torch.tensor([0] + list(np.cumsum(n_new)), dtype=torch.int32, device=device)
        self.q_t = self.q.to(device)

    def reference(self, scale=None):
        """[sum n][Hq][d] in 64 bits; rows of empty sequences are zero."""
        scale = self.d ** -0.5 if scale is None else scale
        out, at, gq = [], 0, self.Hq // self.Hkv
        for b, (L, n) in enumerate(zip(self.lens, self.n_new)):
            q = self.q[at:at + n].double()
            at += n
            if L == 0 or n == 0:
                out.append(torch.zeros(n, self.Hq, self.d, dtype=torch.float64))
                continue
            k = self.k[b].double().repeat_interleave(gq, 1)
            v = self.v[b].double().repeat_interleave(gq, 1)
            s = torch.einsum("nhd,jhd->hnj", q, k) * scale
            j = torch.arange(L)
            pos = torch.arange(L - n, L)[:, None]
            sees = (j <= pos) & ((j < self.S) | (j > pos - self.W))
            w = torch.softmax(s.masked_fill(~sees, -float("inf")), -1)
            out.append(torch.einsum("hnj,jhd->nhd", w, v))
        return torch.cat(out)

    def check(self, got, scale=None):
        """bf16: half a step of the output (2^-8 of it) plus the weights' own
        error: a score in fp32 is off by at most d 2^-24 sum |q k| scale (about
        128 * 2^-24 * 8 = 6e-5 here), twice that relative in a weight with its
        sum, and the weights enter the product with 16 bits (2^-16): 1.3e-4 of
        sum w |v| <= max |v| in all, 2^-13 with nothing to spare for their
        coinciding.  fp32: 1e-5 + 1e-5 |o|, the library's bound."""
        ref = self.reference(scale)
        got = got.double().cpu()
        assert got.shape == ref.shape
        assert torch.isfinite(got).all(), "a slot that no query sees entered the result"
        vmax = max([float(v.abs().max()) for v in self.v if v.numel()], default=1.0)
        if self.dtype == torch.bfloat16:
            tol = 2.0 ** -8 * ref.abs() + 2.0 ** -13 * vmax
        else:
            tol = 1e-5 + 1e-5 * ref.abs()
        err = (got - ref).abs()
        assert bool((err <= tol).all()), f"max excess {(err - tol).max():.3e}, max err {err.max():.3e}"
        return float(err.max())
