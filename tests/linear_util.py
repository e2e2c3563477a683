"""Inputs, the 64-bit reference and the error bounds of the linear attention tests
(not a test module)."""
import torch


def _steps(q, k, v, S, lam, scale):
    """(o, S, A, B, oS) after each token of one request, in 64 bits: A sums the terms
    of the state by their amounts, B each times its age in tokens."""
    A, B = S.abs(), torch.zeros_like(S)
    outs, bound_a, bound_b = [], [], []
    l = lam[:, None, None]
    for t in range(q.shape[0]):
        kv = k[t][:, :, None] * v[t][:, None, :]
        S = l * S + kv
        B = l * (B + A)
        A = l * A + kv.abs()
        qq = q[t][:, None, :] * scale
        outs.append((qq @ S)[:, 0])
        bound_a.append((qq.abs() @ A)[:, 0])
        bound_b.append((qq.abs() @ B)[:, 0])
    return outs, S, A, B, bound_a, bound_b


class Linear:
    """Requests of n_new[r] tokens, prior[r] of them before; the states of requests
    without earlier tokens, and those that no request names, hold NaN."""

    def __init__(self, n_new, prior, H=3, d=64, dtype=torch.bfloat16, seed=0, log_decay=None, fused=True,
                 ids=None, num_states=None, gap=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.n, self.prior, self.H, self.d, self.dtype = n_new, prior, H, d, dtype
        R, T = len(n_new), sum(n_new) + gap
        NS = num_states or R + 2
        self.ids = torch.randperm(NS, generator=g)[:R].tolist() if ids is None else ids
        qkv = torch.randn(T, 3, H, d, generator=g).to(dtype)
        self.qkv = qkv.to(device)
        self.q, self.k, self.v = self.qkv.unbind(1) if fused else [x.contiguous() for x in self.qkv.unbind(1)]
        if log_decay is None:  # half-lives from 3 tokens to 3000, and no decay at all
            log_decay = [0.0 if h == H - 1 and H > 1 else -0.231 * 1000.0 ** (-h / max(1, H - 2)) for h in range(H)]
        self.decay = torch.tensor(log_decay, dtype=torch.float32)
        self.states0 = torch.randn(NS, H, d, d, generator=g) * 3
        held = {i for i, p, n in zip(self.ids, prior, n_new) if p > 0 and i >= 0}
        for i in range(NS):
            if i not in held:
                self.states0[i] = float("nan")
        self.states = self.states0.to(device)
        starts = [0]
        for n in n_new:
            starts.append(starts[-1] + n)
        i32 = dict(dtype=torch.int32, device=device)
        self.start = torch.tensor(starts, **i32)
        self.lens = torch.tensor([p + n for p, n in zip(prior, n_new)], **i32)
        self.ids_t = torch.tensor(self.ids, **i32)
        self.decay_t = self.decay.to(device)
        self.T = T

    def reference(self, scale=None, device="cuda"):
        """outputs [T][H][d] (NaN outside the requests), states, and their amounts A and
        ages B for the bounds."""
        scale = self.d ** -0.5 if scale is None else scale
        lam = self.decay.double().exp().to(device)
        q, k, v = (x.double().to(device) for x in self.qkv.unbind(1))
        nan = torch.full((self.T, self.H, self.d), float("nan"), dtype=torch.float64, device=device)
        out, oa, ob = nan, nan.clone(), nan.clone()
        states = self.states0.double().to(device)
        sa, sb = torch.zeros_like(states), torch.zeros_like(states)
        at = 0
        for r, n in enumerate(self.n):
            i = self.ids[r]
            if n and i >= 0:
                S = states[i] if self.prior[r] > 0 else torch.zeros_like(states[i])
                o, S, A, B, a, b = _steps(q[at:at + n], k[at:at + n], v[at:at + n], S, lam, scale)
                states[i], sa[i], sb[i] = S, A, B
                out[at:at + n], oa[at:at + n], ob[at:at + n] = torch.stack(o), torch.stack(a), torch.stack(b)
            at += n
        return out, states, oa, ob, sa, sb

    def check(self, out, states=None, scale=None, terms=(0.0, 0.0)):
        """Bounds.  A term of a state that is `age` tokens old has been multiplied by the
        decay `age` times: a factor in 32 bits (off by 2^-22: 2 ulp of exp2, and its
        argument) and a rounding (2^-24) each, after its own product's; sums of D
        terms in any order add D 2^-24 of their amounts.  `terms`: what else a term
        of an output, and of a state, may be off by (a kernel that takes products of
        16-bit terms).  An output is rounded to its type by half a step."""
        ref, rs, oa, ob, sa, sb = self.reference(scale)
        e, age = 2.0 ** -23, 2.0 ** -22 + 2.0 ** -24
        states = self.states if states is None else states
        touched = torch.zeros(len(rs), dtype=torch.bool)
        for i, n in zip(self.ids, self.n):
            if n and i >= 0:
                touched[i] = True
        t = touched.to(states.device)
        # states nobody named keep their bytes
        same = states[~t].view(torch.int32) == self.states0[~touched].to(states.device).view(torch.int32)
        assert bool(same.all())
        got = states[t].double()
        assert torch.isfinite(got).all()
        err = (got - rs[t]).abs()
        tol = (2 * e + 2.0 ** -24 * 16 + terms[1]) * sa[t] + age * sb[t]
        assert bool((err <= tol).all()), f"states: {(err / tol.clamp(min=1e-300)).max():.3f} of the bound"
        inside = ~torch.isnan(ref[:, 0, 0])
        got, ref, oa, ob = out[inside].double(), ref[inside], oa[inside], ob[inside]
        assert torch.isfinite(got).all(), "something that no token sees entered the result"
        err = (got - ref).abs()
        tol = torch.finfo(self.dtype).eps / 2 * ref.abs() + ((self.d + 20) * 2.0 ** -24 + terms[0]) * oa + age * ob
        worst = float((err / tol.clamp(min=1e-300)).max()) if err.numel() else 0.0
        assert worst <= 1, f"outputs: {worst:.3f} of the bound"
        return worst
