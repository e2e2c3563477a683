"""Operators of a bounded paged KV cache, each in a plain form and through the
framework's entry points: rotary positions with the store into pages, attention
with a sliding window and first tokens that stay visible (decode and chunked
prefill over pages), and the compaction of a sequence's kept tokens.

Pools are [num_blocks][Hkv][block_size][head_dim]; a block table maps logical
block i of a sequence to a physical block.  A table entry of -1 stands for a
page that was freed because none of its tokens is visible any more.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_ES = {"bf16": 2, "fp32": 4}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _rope(name, T, Hq, Hkv, d, bs, dtype, axes, rot, interleaved, far):
    return dict(name=name, op="rope", T=T, Hq=Hq, Hkv=Hkv, d=d, bs=bs, dtype=dtype, axes=axes,
                rot=rot, interleaved=interleaved, far=far)


def _decode(name, B, lo, hi, W, S, Hq, Hkv, d, bs, dtype):
    return dict(name=name, op="decode", B=B, lo=lo, hi=hi, W=W, S=S, Hq=Hq, Hkv=Hkv, d=d, bs=bs,
                dtype=dtype)


def _prefill(name, R, n_lo, n_hi, p_lo, p_hi, W, S, Hq, Hkv, d, bs):
    return dict(name=name, op="prefill", R=R, n_lo=n_lo, n_hi=n_hi, p_lo=p_lo, p_hi=p_hi, W=W, S=S,
                Hq=Hq, Hkv=Hkv, d=d, bs=bs, dtype="bf16")


def _compact(name, B, lo, hi, k_lo, k_hi, Hkv, d, bs, dtype):
    return dict(name=name, op="compact", B=B, lo=lo, hi=hi, k_lo=k_lo, k_hi=k_hi, Hkv=Hkv, d=d,
                bs=bs, dtype=dtype)


def listed():
    return [
        # a decode step of 64 sequences: one new token each, one position axis
        _rope("rope_step64", 64, 32, 8, 128, 16, "bf16", 1, 128, False, 32768),
        # a mixed step of image and text tokens: time, height and width positions
        _rope("rope_axes3_2k", 2048, 32, 8, 128, 16, "bf16", 3, 128, False, 32768),
        # a long prompt of a model that rotates half of each head, adjacent pairs
        _rope("rope_partial_20k", 20001, 64, 8, 128, 32, "bf16", 1, 64, True, 1 << 20),
        # one sequence deep into a long context: latency
        _decode("decode_one", 1, 33001, 33001, 1024, 4, 32, 8, 128, 16, "bf16"),
        # a serving batch of ragged contexts, some shorter than the window
        _decode("decode_batch64", 64, 128, 32768, 4096, 16, 32, 8, 128, 16, "bf16"),
        # long contexts of groups of 8 heads, the largest window
        _decode("decode_long", 64, 16384, 32768, 8192, 64, 64, 8, 128, 32, "bf16"),
        # the small full-precision model, odd window, pages shorter than a tile
        _decode("decode_fp32", 24, 5, 2001, 501, 3, 4, 4, 64, 8, "fp32"),
        # a short chunk late in a conversation
        _prefill("prefill_short", 1, 40, 40, 5000, 5000, 513, 4, 32, 8, 128, 16),
        # chunks of 512 tokens over growing contexts, as run next to decodes
        _prefill("prefill_chunks", 4, 512, 512, 0, 3584, 1024, 4, 32, 8, 128, 16),
        # one long prompt in one call
        _prefill("prefill_prompt", 1, 16384, 16384, 0, 0, 4096, 64, 32, 8, 128, 16),
        # one conversation pruned to a quarter of its tokens
        _compact("compact_one", 1, 4097, 4097, 1000, 1000, 8, 128, 16, "bf16"),
        # a batch pruned to a budget of about 4k tokens per head
        _compact("compact_batch64", 64, 5000, 12000, 3500, 4500, 8, 128, 16, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "decode", "prefill", "compact"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([2, 4, 8, 8])
    gq = rng.choice([1, 2, 4, 8])
    bs = rng.choice([8, 16, 16, 32, 64, 128])
    Hq = Hkv * gq
    if op == "rope":
        axes = rng.choice([1, 1, 3])
        rot = rng.choice([d, d, d // 2]) if axes == 1 else d
        return _case(_rope("", _log_int(rng, 1, 20000), Hq, Hkv, d, bs, rng.choice(["bf16", "bf16", "fp32"]),
                           axes, rot, rng.random() < 0.4, _log_int(rng, 64, 1 << 20)))
    if op == "decode":
        W, S = _log_int(rng, 16, 8192), rng.choice([0, 1, 4, 16, 37, 64])
        hi = _log_int(rng, 64, 32768)
        return _case(_decode("", _log_int(rng, 1, 64), max(1, hi // rng.randint(1, 8)), hi, W, S, Hq, Hkv, d,
                             bs, rng.choice(["bf16", "bf16", "bf16", "fp32"])))
    if op == "prefill":
        W, S = _log_int(rng, 16, 8192), rng.choice([0, 1, 4, 16, 37, 64])
        n, R = _log_int(rng, 1, 8192), _log_int(rng, 1, 16)
        p = _log_int(rng, 1, 16384) if rng.random() < 0.8 else 0
        while R > 1 and (R * n > 8192 or R * n * (n + p) * Hq > 1 << 32):
            R //= 2
        while n > 1 and n * (n + p) * Hq > 1 << 32:
            n, p = n * 2 // 3, p * 2 // 3
        return _case(_prefill("", R, max(1, n // rng.randint(1, 4)), n, p // 2, p, W, S, Hq, Hkv, d, bs))
    hi = _log_int(rng, 32, 12000)
    k = max(1, int(hi * rng.uniform(0.05, 0.45)))
    return _case(_compact("", _log_int(rng, 1, 64), max(2, hi // 2), hi, max(1, k // 2), k, Hkv, d, bs,
                          rng.choice(["bf16", "bf16", "fp32"])))


def _case(c):
    del c["name"]
    return c


def _spread(lo, hi, n):
    """n whole numbers over [lo, hi]: both ends (n > 1), the others scattered between them."""
    return [hi if i == 0 else lo if i == 1 else lo + int((hi - lo) * (i * 0.6180339887 % 1.0))
            for i in range(n)]


def _sections(case):
    half = case["rot"] // 2
    if case["axes"] == 1:
        return (half,)
    return (half // 4, half // 2 - half // 8, half - half // 4 - (half // 2 - half // 8))


def _prefill_sizes(case):
    R = case["R"]
    n, prior = _spread(case["n_lo"], case["n_hi"], R), _spread(case["p_lo"], case["p_hi"], R)[::-1]
    return n, prior


def _visible_blocks(L, first, case):
    """Blocks of [0, L) with a token visible to a query at `first` or later."""
    bs, lo = case["bs"], max(0, first - case["W"] + 1)
    return [j for j in range(-(-L // bs)) if j * bs < case["S"] or min((j + 1) * bs, L) > lo]


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _randn(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _pools(g, NB, case, dtype):
    shape = (NB, case["Hkv"], case["bs"], case["d"])
    return _randn(g, *shape, dtype=dtype), _randn(g, *shape, dtype=dtype)


def _table(g, rows, width):
    """Block table of `rows` (lists of logical blocks that are kept), the pages scattered over
    a pool a little larger than needed."""
    need = sum(len(r) for r in rows)
    NB = need + need // 20 + 1
    perm = torch.randperm(NB, generator=g, device="cuda")[:need].int().cpu()
    table = torch.full((len(rows), width), -1, dtype=torch.int32)
    at = 0
    for b, r in enumerate(rows):
        table[b, torch.tensor(r, dtype=torch.long)] = perm[at:at + len(r)]
        at += len(r)
    return table.cuda(), NB


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype, op = _DT[case["dtype"]], case["op"]
    st = dict(case)
    if op == "rope":
        T, Hq, Hkv, d, bs = case["T"], case["Hq"], case["Hkv"], case["d"], case["bs"]
        NB = -(-T // bs) + 8
        # one fused projection: q, k and v of a token lie next to each other
        qkv = _randn(g, T, (Hq + 2 * Hkv) * d, dtype=dtype)
        st["q"] = qkv[:, :Hq * d].view(T, Hq, d)
        st["k"] = qkv[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d)
        st["v"] = qkv[:, (Hq + Hkv) * d:].view(T, Hkv, d)
        st["k_cache"], st["v_cache"] = _pools(g, NB, case, dtype)
        st["slots"] = torch.randperm(NB * bs, generator=g, device="cuda")[:T]
        st["positions"] = torch.randint(0, case["far"], (case["axes"], T), generator=g, device="cuda")
        half = case["rot"] // 2
        st["inv_freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
        st["sections"] = _sections(case)
        return st
    if op == "compact":
        L = _spread(case["lo"], case["hi"], case["B"])
        n = [min(a, b) for a, b in zip(_spread(case["k_lo"], case["k_hi"], case["B"]), L)]
        bs, B, Hkv, Lm, nm = case["bs"], case["B"], case["Hkv"], max(L), max(n)
        width, wide = -(-Lm // bs), -(-nm // bs)
        # the old pages, and fresh ones for the kept tokens (the old ones are shared)
        rows = [list(range(-(-x // bs))) + [width + j for j in range(-(-y // bs))] for x, y in zip(L, n)]
        table, NB = _table(g, rows, width + wide)
        st["src_table"], st["dst_table"] = table[:, :width].contiguous(), table[:, width:].contiguous()
        st["k_cache"], st["v_cache"] = _pools(g, NB, case, dtype)
        lens, keep_lens = torch.tensor(L, device="cuda"), torch.tensor(n, device="cuda")
        # importance of each token to each head; the first four tokens always stay
        score = torch.rand(B, Hkv, Lm, generator=g, device="cuda")
        score[:, :, :4] = 2.0
        score.masked_fill_(torch.arange(Lm, device="cuda") >= lens[:, None, None], -1.0)
        order = score.argsort(-1, descending=True)[:, :, :nm]
        order = order.masked_fill(torch.arange(nm, device="cuda") >= keep_lens[:, None, None], 1 << 30)
        st["keep"] = order.sort(-1).values.int()
        st["keep_lens"] = keep_lens.int()
        return st
    if op == "decode":
        L = _spread(case["lo"], case["hi"], case["B"])
        rows = [_visible_blocks(x, x - 1, case) for x in L]
        tokens, T = L, case["B"]
    else:
        n, prior = _prefill_sizes(case)
        L = [a + b for a, b in zip(n, prior)]
        rows = [_visible_blocks(x, p, case) for x, p in zip(L, prior)]
        T = sum(n)
        starts = [0]
        for x in n:
            starts.append(starts[-1] + x)
        st["query_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        st["max_query_len"] = max(n)
    st["table"], NB = _table(g, rows, -(-max(L) // case["bs"]))
    st["k_cache"], st["v_cache"] = _pools(g, NB, case, dtype)
    st["context_lens"] = torch.tensor(L, dtype=torch.int32, device="cuda")
    st["q"] = _randn(g, T, case["Hq"], case["d"], dtype=dtype)
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(st):
    if own:
        from paged_kv_cache_192_gb300 import ops
        if st["op"] == "rope":
            q = ops.rope_reshape_and_cache(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"],
                                           st["slots"], st["positions"], st["inv_freq"],
                                           sections=st["sections"], interleaved=st["interleaved"])
            return q, st["k_cache"], st["v_cache"]
        if st["op"] == "decode":
            return ops.decode_window(st["q"], st["k_cache"], st["v_cache"], st["table"],
                                     st["context_lens"], window=st["W"], num_sinks=st["S"])
        if st["op"] == "prefill":
            return ops.prefill_window(st["q"], st["k_cache"], st["v_cache"], st["table"],
                                      st["query_start"], st["context_lens"], st["max_query_len"],
                                      window=st["W"], num_sinks=st["S"])
        ops.compact_cache(st["k_cache"], st["v_cache"], st["src_table"], st["dst_table"], st["keep"],
                          st["keep_lens"])
        return st["k_cache"], st["v_cache"]
    return {"rope": _run_rope, "decode": _run_decode, "prefill": _run_prefill,
            "compact": _run_compact}[st["op"]](st)


def _rotate(x, cos, sin, rot, interleaved):
    """x [T][H][d]: the first `rot` elements of each head rotated by the token's angles."""
    y = x.float()
    c, s = cos[:, None], sin[:, None]
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    u, v = a * c - b * s, a * s + b * c
    r = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((r, y[..., rot:]), -1).to(x.dtype)


def _run_rope(st):
    rot, bs = st["rot"], st["bs"]
    axis = torch.repeat_interleave(torch.arange(st["axes"], device="cuda"),
                                   torch.tensor(st["sections"], device="cuda"), output_size=rot // 2)
    # far positions: the product of position and frequency needs more than 24 bits
    ang = st["positions"].double().t()[:, axis] * st["inv_freq"].double()
    cos, sin = ang.cos().float(), ang.sin().float()
    q = _rotate(st["q"], cos, sin, rot, st["interleaved"])
    k = _rotate(st["k"], cos, sin, rot, st["interleaved"])
    blk, off = st["slots"] // bs, st["slots"] % bs
    st["k_cache"][blk, :, off] = k
    st["v_cache"][blk, :, off] = st["v"]
    return q, st["k_cache"], st["v_cache"]


def _softmax_av(s, hidden, v):
    """softmax of s where not hidden, times v (32 bits); s is overwritten."""
    s.masked_fill_(hidden, -math.inf)
    s.sub_(s.amax(-1, keepdim=True)).exp_()
    return (s @ v) / s.sum(-1, keepdim=True)


def _run_decode(st):
    q, bs, W, S = st["q"], st["bs"], st["W"], st["S"]
    B, Hq, d = q.shape
    Hkv, L = st["Hkv"], st["context_lens"].long()[:, None]
    n = min(int(st["table"].shape[1]) * bs, S + W)
    i = torch.arange(n, device="cuda")
    pos = torch.where(i < S, i, (L - W).clamp(min=S) + i - S)  # the i-th visible token
    seen = pos < L
    blk = st["table"].gather(1, torch.where(seen, pos, 0) // bs).clamp(min=0).long()
    at = (blk[:, None], torch.arange(Hkv, device="cuda")[:, None], (pos % bs)[:, None])
    k, v = st["k_cache"][at].float(), st["v_cache"][at].float()  # [B][Hkv][n][d]
    s = (q.float().view(B, Hkv, -1, d) / math.sqrt(d)) @ k.transpose(-1, -2)
    return _softmax_av(s, ~seen[:, None, None], v).view(B, Hq, d).to(q.dtype)


def _run_prefill(st):
    q, bs, W, S = st["q"], st["bs"], st["W"], st["S"]
    T, Hq, d = q.shape
    start, L, Hkv, R = st["query_start"].long(), st["context_lens"].long(), st["Hkv"], st["R"]
    n, nm = start.diff(), st["max_query_len"]
    j = torch.arange(st["table"].shape[1] * bs, device="cuda")
    blk = st["table"][:, j // bs].long()  # [R][keys]
    at = (blk.clamp(min=0)[:, None], torch.arange(Hkv, device="cuda")[:, None], (j % bs)[None, None])
    k = st["k_cache"][at].float()  # [R][Hkv][keys][d]
    v = st["v_cache"][at].float().masked_fill_((blk < 0)[:, None, :, None], 0.0)
    t = torch.arange(nm, device="cuda")
    row = (start[:-1, None] + t).clamp(max=T - 1)
    qp = (q[row].float() / math.sqrt(d)).view(R, nm, Hkv, -1, d).permute(0, 2, 3, 1, 4)
    s = qp.reshape(R, Hkv, -1, d) @ k.transpose(-1, -2)
    pos = torch.minimum((L - n)[:, None] + t, L[:, None] - 1)[:, :, None]  # [R][queries][1]
    hidden = (j > pos) | ((j >= S) & (j <= pos - W))
    o = _softmax_av(s.view(R, Hkv, Hq // Hkv, nm, -1), hidden[:, None, None], v[:, :, None])
    o = o.permute(0, 3, 1, 2, 4).reshape(R, nm, Hq, d)
    return o[t < n[:, None]].to(q.dtype)


def _run_compact(st):
    keep, bs = st["keep"].long(), st["bs"]
    i = torch.arange(keep.shape[2], device="cuda")
    b, h, i = (i < st["keep_lens"][:, None, None]).expand(keep.shape).nonzero(as_tuple=True)
    old = keep[b, h, i]
    src = st["src_table"][b, old // bs].long(), h, old % bs
    dst = st["dst_table"][b, i // bs].long(), h, i % bs
    st["k_cache"][dst] = st["k_cache"][src]
    st["v_cache"][dst] = st["v_cache"][src]
    return st["k_cache"], st["v_cache"]


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    es, d, Hkv, op = _ES[case["dtype"]], case["d"], case["Hkv"], case["op"]
    row = d * es
    if op == "rope":
        T, Hq = case["T"], case["Hq"]
        return {"bytes": T * ((2 * Hq + 4 * Hkv) * row + 8 * (case["axes"] + 1)) + 2 * case["rot"],
                "flops": T * (Hq + Hkv) * case["rot"] * 3}
    if op == "compact":
        n = sum(min(a, b) for a, b in zip(_spread(case["k_lo"], case["k_hi"], case["B"]),
                                          _spread(case["lo"], case["hi"], case["B"])))
        return {"bytes": n * Hkv * (4 * row + 4), "flops": 0}
    W, S, Hq = case["W"], case["S"], case["Hq"]
    if op == "decode":
        L = _spread(case["lo"], case["hi"], case["B"])
        vis = sum(min(x, S + W) for x in L)
        blocks = sum(len(_visible_blocks(x, x - 1, case)) for x in L)
        return {"bytes": vis * Hkv * 2 * row + 2 * case["B"] * Hq * row + 4 * blocks + 4 * case["B"],
                "flops": 4 * Hq * d * vis}
    n, prior = _prefill_sizes(case)
    pairs = keys = 0
    for m, p in zip(n, prior):
        full = max(0, S + W - p - 1)  # queries that see every earlier token
        a = min(m, full)
        pairs += a * p + a * (a + 1) // 2 + (m - a) * (S + W)
        keys += min(m + p, S + W + m - 1)
    return {"bytes": keys * Hkv * 2 * row + 2 * sum(n) * Hq * row, "flops": 4 * Hq * d * pairs}


# --------------------------------------------------------------------------
# the definition in 64 bits, sequence by sequence
# --------------------------------------------------------------------------
def _attend64(q, pos, st, b, scale):
    """q [m][Hq][d] of sequence b at positions pos, each over the tokens that it sees."""
    bs, Hkv, W, S = st["bs"], st["Hkv"], st["W"], st["S"]
    m, Hq, d = q.shape
    j = torch.arange(int(pos[-1]) + 1, device="cuda")
    j = j[(j < S) | (j > int(pos[0]) - W)]  # seen by one of them at least
    page = st["table"][b][j // bs].long()
    K = st["k_cache"].permute(0, 2, 1, 3)[page, j % bs].double().repeat_interleave(Hq // Hkv, 1)
    V = st["v_cache"].permute(0, 2, 1, 3)[page, j % bs].double().repeat_interleave(Hq // Hkv, 1)
    logit = torch.einsum("mhd,jhd->hmj", q.double(), K) * scale
    sees = (j <= pos[:, None]) & ((j < S) | (j > pos[:, None] - W))
    w = torch.where(sees, logit, -math.inf).softmax(-1)
    return torch.einsum("hmj,jhd->mhd", w, V)


def exact(case, seed):
    if case["op"] == "compact":
        return None  # moved, not computed
    st = prepare(case, seed)
    if case["op"] == "rope":
        T, half = case["T"], case["rot"] // 2
        axis = [a for a, s in enumerate(st["sections"]) for _ in range(s)]
        theta = torch.stack([st["positions"][a].double() for a in axis], 1) * st["inv_freq"].double()
        turn = torch.polar(torch.ones_like(theta), theta)[:, None]

        def rotated(x):
            x = x.double().clone()
            if case["interleaved"]:
                z = torch.complex(x[..., 0:2 * half:2], x[..., 1:2 * half:2]) * turn
                x[..., 0:2 * half:2], x[..., 1:2 * half:2] = z.real, z.imag
            else:
                z = torch.complex(x[..., :half], x[..., half:2 * half]) * turn
                x[..., :half], x[..., half:2 * half] = z.real, z.imag
            return x

        pools = []
        for pool, new in ((st["k_cache"], rotated(st["k"])), (st["v_cache"], st["v"].double())):
            flat = pool.double().permute(0, 2, 1, 3).reshape(-1, case["Hkv"], case["d"])
            flat[st["slots"]] = new
            pools.append(flat.view(-1, case["bs"], case["Hkv"], case["d"]).permute(0, 2, 1, 3).contiguous())
        return rotated(st["q"]), pools[0], pools[1]
    scale, parts = case["d"] ** -0.5, []
    L = st["context_lens"].tolist()
    if case["op"] == "decode":
        for b in range(case["B"]):
            parts.append(_attend64(st["q"][b:b + 1], torch.tensor([L[b] - 1], device="cuda"), st, b, scale))
        return torch.cat(parts)
    n, prior = _prefill_sizes(case)
    at = 0
    for r in range(case["R"]):
        for t in range(0, n[r], 512):
            m = min(512, n[r] - t)
            pos = prior[r] + t + torch.arange(m, device="cuda")
            parts.append(_attend64(st["q"][at:at + m], pos, st, r, scale))
            at += m
    return torch.cat(parts)
