"""Operators that a serving step runs beside paged causal attention, each in a
plain form and through the framework's entry points: the step's block tables,
slots and positions built on the GPU from the requests' lengths; attention to
an encoder's states in pages; linear attention with a decay for each head, its
state in a pool (single tokens, and prompts).

Pools are [num_blocks][Hkv][block_size][head_dim]; a block table maps logical
block i of a sequence to a physical block.  Pages that no sequence holds are in
a ring, [first, first + count) of it, taken at its front and given back behind
its end.  A state is a matrix of head_dim x head_dim per (sequence, head).
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_ES = {"bf16": 2, "fp32": 4}
_CHUNK = 128  # tokens per chunk of the plain form of linear attention


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _plan(name, R, S, lo, hi, n_lo, n_hi, fresh, idle, bs, width):
    """R rows (idle ones are padding) over S sequences of lo..hi tokens that grow by n_lo..n_hi;
    `fresh` of them hold nothing before the step."""
    return dict(name=name, op="plan", R=R, S=S, lo=lo, hi=hi, n_lo=n_lo, n_hi=n_hi, fresh=fresh, idle=idle,
                bs=bs, width=width)


def _cross(name, R, n_lo, n_hi, e_lo, e_hi, Hq, Hkv, d, bs):
    return dict(name=name, op="cross", R=R, n_lo=n_lo, n_hi=n_hi, e_lo=e_lo, e_hi=e_hi, Hq=Hq, Hkv=Hkv, d=d,
                bs=bs, dtype="bf16")


def _step(name, B, H, d, dtype, fresh):
    return dict(name=name, op="step", B=B, H=H, d=d, dtype=dtype, fresh=fresh)


def _prompt(name, R, n_lo, n_hi, H, d, fresh):
    return dict(name=name, op="prompt", R=R, n_lo=n_lo, n_hi=n_hi, H=H, d=d, dtype="bf16", fresh=fresh)


def listed():
    return [
        # a decode step of 64 sequences: a token each, planned and taken back
        _plan("plan_step64", 64, 64, 128, 4096, 1, 1, 0, 0, 16, 260),
        # decodes next to prompts that come and go, a batch padded to a multiple of 32
        _plan("plan_mixed", 160, 300, 256, 8192, 1, 512, 12, 9, 16, 560),
        # many long sequences with 20 drafted tokens each, all rejected
        _plan("plan_drafts1k", 1024, 1024, 2000, 32000, 20, 20, 0, 0, 16, 2048),
        # one token of a decoder over half a minute of encoded audio: latency
        _cross("cross_one", 1, 1, 1, 1500, 1500, 16, 16, 64, 16),
        # a step of 64 requests with up to 5 beams each over audio of several lengths
        _cross("cross_beams64", 64, 1, 5, 400, 1500, 16, 16, 64, 16),
        # short text prompts over the states of images, groups of 4 heads
        _cross("cross_prompts", 8, 20, 100, 1000, 4100, 32, 8, 128, 16),
        # long texts over long documents
        _cross("cross_long", 4, 2048, 2048, 2000, 8192, 32, 8, 128, 32),
        # one sequence of a small full-precision model: latency
        _step("linear_one", 1, 16, 64, "fp32", 0),
        # a decode step of 64 sequences, two of them at their first token
        _step("linear_step64", 64, 32, 128, "bf16", 2),
        # a short chunk late in a conversation
        _prompt("linear_short", 1, 100, 100, 32, 128, 0),
        # chunks of several lengths, half of them the first of their sequences
        _prompt("linear_chunks", 8, 65, 2048, 32, 128, 4),
        # one long prompt in one call
        _prompt("linear_prompt", 1, 16384, 16384, 32, 128, 1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "cross", "step", "prompt"])
    if op == "plan":
        R, bs = _log_int(rng, 1, 1024), rng.choice([8, 16, 16, 32, 64, 128])
        hi = _log_int(rng, 8, 32000)
        fresh, idle = (rng.randint(0, R // 3), rng.randint(0, R // 3)) if rng.random() < 0.6 else (0, 0)
        n_hi = _log_int(rng, 1, max(1, 20000 // R))
        return _case(_plan("", R, R + rng.randint(0, 200), max(1, hi // rng.randint(1, 8)), hi, rng.randint(1, n_hi),
                           n_hi, fresh, idle, bs, -(-(hi + n_hi) // bs) + rng.randint(0, 5)))
    d = rng.choice([64, 128])
    if op == "cross":
        Hkv, gq = rng.choice([2, 4, 8, 16]), rng.choice([1, 1, 2, 4, 8])
        R, n, e = _log_int(rng, 1, 64), _log_int(rng, 1, 2048), _log_int(rng, 1, 8192)
        while R * n * e * Hkv * gq > 1 << 31 or R * e * Hkv > 1 << 21:
            R, n, e = max(1, R * 2 // 3), max(1, n * 3 // 4), max(1, e * 4 // 5)
        return _case(_cross("", R, max(1, n // rng.randint(1, 5)), n, rng.choice([0, e // 4, e // 2]), e, Hkv * gq, Hkv,
                            d, rng.choice([8, 16, 16, 32, 64, 128])))
    H = rng.choice([1, 4, 8, 16, 32, 32])
    if op == "step":
        B = _log_int(rng, 1, 64)
        return _case(_step("", B, H, d, rng.choice(["bf16", "bf16", "fp32"]), rng.randint(0, B // 2)))
    R, n = _log_int(rng, 1, 16), _log_int(rng, 1, 16384)
    while R * n * H > 1 << 19:
        R, n = max(1, R * 2 // 3), max(1, n * 3 // 4)
    return _case(_prompt("", R, max(1, n // rng.randint(1, 8)), n, H, d, rng.randint(0, R)))


def _case(c):
    del c["name"]
    return c


def _spread(lo, hi, n):
    """n whole numbers over [lo, hi]: both ends (n > 1), the others scattered between them."""
    return [hi if i == 0 else lo if i == 1 else lo + int((hi - lo) * (i * 0.6180339887 % 1.0))
            for i in range(n)]


def _plan_rows(case):
    """(tokens held, tokens added) of each row; None for a row of padding."""
    R, work = case["R"], case["R"] - case["idle"]
    L = _spread(case["lo"], case["hi"], work)
    n = _spread(case["n_lo"], case["n_hi"], work)
    L[work - case["fresh"]:] = [0] * case["fresh"]
    return list(zip(L, n)) + [None] * (R - work)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _randn(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _perm(g, n):
    return torch.randperm(n, generator=g, device="cuda").int()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(n):
    return torch.cat((torch.zeros(1, dtype=torch.int64), torch.tensor(n).cumsum(0))).int().cuda()


def _prepare_plan(case, g, st):
    rows, S, bs, width = _plan_rows(case), case["S"], case["bs"], case["width"]
    held = [-(-r[0] // bs) if r else 0 for r in rows]
    need = sum(-(-(r[0] + r[1]) // bs) for r in rows if r)
    NB = need + need // 8 + 5
    ids = torch.randperm(S, generator=g, device="cuda")[:len(rows)].cpu()
    perm = _perm(g, NB).cpu()
    # one spare row, and a spare entry of the others, for what the plain form writes nowhere
    pages, lens = torch.zeros(S + 1, width, dtype=torch.int32), torch.zeros(S + 1, dtype=torch.int32)
    at = 0
    for i, r in enumerate(rows):
        if r is None:
            ids[i] = -1
            continue
        pages[ids[i], :held[i]] = perm[at:at + held[i]]
        lens[ids[i]] = r[0]
        at += held[i]
    first = int(torch.randint(0, NB, (1,), generator=g, device="cuda"))
    ring = torch.zeros(NB + 1, dtype=torch.int32)
    ring[(torch.arange(NB - at) + first) % NB] = perm[at:]
    st["all_pages"], st["all_lens"], st["all_ring"] = pages.cuda(), lens.cuda(), ring.cuda()
    st["pages"], st["lens"], st["ring"] = st["all_pages"][:S], st["all_lens"][:S], st["all_ring"][:NB]
    st["ring_state"] = _ints([first, NB - at, 0, 0])
    st["seq_ids"] = ids.int().cuda()
    st["grow"] = _ints([r[1] if r else 0 for r in rows])
    st["shrink"] = -st["grow"]
    st["max_tokens"] = sum(r[1] for r in rows if r) + 3
    return st


def _log_decay(H):
    """Half-lives from about 20 tokens to about 20,000."""
    return (-math.log(2.0) / 20.0 * 1000.0 ** (-torch.arange(H, dtype=torch.float64) / max(1, H - 1))).float().cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case)
    if case["op"] == "plan":
        return _prepare_plan(case, g, st)
    dtype, d = _DT[case["dtype"]], case["d"]
    if case["op"] == "cross":
        R, bs, Hkv = case["R"], case["bs"], case["Hkv"]
        n, e = _spread(case["n_lo"], case["n_hi"], R), _spread(case["e_lo"], case["e_hi"], R)[::-1]
        blocks = [-(-x // bs) for x in e]
        NB = sum(blocks) + sum(blocks) // 20 + 1
        perm, at = _perm(g, NB).cpu(), 0
        table = torch.zeros(R, max(1, max(blocks)), dtype=torch.int32)
        for r, m in enumerate(blocks):
            table[r, :m] = perm[at:at + m]
            at += m
        st["table"], st["query_start"], st["max_query_len"] = table.cuda(), _starts(n), max(n)
        st["encoder_lens"] = _ints(e)
        st["k_cache"], st["v_cache"] = (_randn(g, NB, Hkv, bs, d, dtype=dtype) for _ in range(2))
        st["q"] = _randn(g, sum(n), case["Hq"], d, dtype=dtype)
        return st
    H = case["H"]
    if case["op"] == "step":
        n = [1] * case["B"]
    else:
        n = _spread(case["n_lo"], case["n_hi"], case["R"])
        st["query_start"], st["max_query_len"] = _starts(n), max(n)
    R, T = len(n), sum(n)
    # the first `fresh` sequences begin with this call: what their states hold does not count
    prior = torch.randint(1, 30000, (R,), generator=g, device="cuda")
    prior[:case["fresh"]] = 0
    st["context_lens"] = (prior + torch.tensor(n, device="cuda")).int()
    st["state_ids"] = _perm(g, R + 3)[:R]
    st["states"] = _randn(g, R + 3, H, d, d, dtype=torch.float32)
    # one fused projection: q, k and v of a token lie next to each other
    qkv = _randn(g, T, 3, H, d, dtype=dtype)
    st["q"], st["k"], st["v"] = qkv.unbind(1)
    st["log_decay"] = _log_decay(H)
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(st):
    op = st["op"]
    if own:
        from paged_kv_cache_192_gb300 import ops
        if op == "plan":
            pages = ops.PageState(st["pages"], st["lens"], st["ring"], st["ring_state"])
            a = ops.plan_step(pages, st["seq_ids"], st["grow"], st["bs"], st["max_tokens"])
            b = ops.plan_step(pages, st["seq_ids"], st["shrink"], st["bs"], st["max_tokens"])
            return tuple(a), tuple(b), tuple(pages)
        if op == "cross":
            return ops.cross_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["query_start"],
                                       st["encoder_lens"], st["max_query_len"])
        if op == "step":
            o = ops.linear_decode(st["q"], st["k"], st["v"], st["states"], st["state_ids"], st["context_lens"],
                                  st["log_decay"])
        else:
            o = ops.linear_prefill(st["q"], st["k"], st["v"], st["states"], st["state_ids"], st["query_start"],
                                   st["context_lens"], st["max_query_len"], st["log_decay"])
        return o, st["states"]
    if op == "plan":
        return _run_plan(st, st["grow"]), _run_plan(st, st["shrink"]), (st["pages"], st["lens"], st["ring"],
                                                                       st["ring_state"])
    return {"cross": _run_cross, "step": _run_step, "prompt": _run_prompt}[op](st)


def _run_plan(st, change):
    """Every sequence grows or shrinks by its change: pages come from the front of the ring in the rows' order,
    those given up go behind its end."""
    bs, S, width, NB = st["bs"], st["S"], st["pages"].shape[1], st["ring"].shape[0]
    live = st["seq_ids"] >= 0
    row = torch.where(live, st["seq_ids"], S).long()
    old = torch.where(live, st["all_lens"][row], 0).long()
    new = torch.where(live, (old + change).clamp(min=0), 0)
    b0, b1 = (old + bs - 1) // bs, (new + bs - 1) // bs
    taken, given = (b1 - b0).clamp(min=0), (b0 - b1).clamp(min=0)
    first, count = st["ring_state"][0].long(), st["ring_state"][1].long()
    j = torch.arange(width, device="cuda")
    held = st["all_pages"][row]
    fresh = (j >= b0[:, None]) & (j < b1[:, None])
    source = (first + (taken.cumsum(0) - taken - b0)[:, None] + j) % NB
    table = torch.where(fresh, st["all_ring"][source], torch.where(j < b1[:, None], held, 0))
    gone = (j >= b1[:, None]) & (j < b0[:, None])
    back = (first + count + (given.cumsum(0) - given - b1)[:, None] + j) % NB
    st["all_ring"].scatter_(0, torch.where(gone, back, NB).view(-1), held.view(-1))
    st["all_pages"].view(-1).scatter_(0, torch.where(fresh, row[:, None] * width + j, S * width).view(-1), table.view(-1))
    st["all_lens"].scatter_(0, row, new.int())
    st["ring_state"][0] = (first + taken.sum()) % NB
    st["ring_state"][1] = count - taken.sum() + given.sum()
    more = (new - old).clamp(min=0)
    end = more.cumsum(0)
    t = torch.arange(st["max_tokens"], device="cuda")
    r = torch.searchsorted(end, t, right=True).clamp(max=len(end) - 1)
    inside = t < end[-1]
    pos = torch.where(inside, old[r] + t - (end - more)[r], 0)
    slots = torch.where(inside, table[r, pos // bs] * bs + pos % bs, -1)
    return table, new.int(), torch.cat((end[:1] * 0, end)).int(), slots, pos


def _run_cross(st):
    q, bs, Hkv, R, nm = st["q"], st["bs"], st["Hkv"], st["R"], st["max_query_len"]
    T, Hq, d = q.shape
    start, e = st["query_start"].long(), st["encoder_lens"].long()
    j = torch.arange(st["table"].shape[1] * bs, device="cuda")
    hidden = j >= e[:, None]
    at = (st["table"][:, j // bs].long()[:, None], torch.arange(Hkv, device="cuda")[:, None], (j % bs)[None, None])
    k = st["k_cache"][at].float()  # [R][Hkv][keys][d]
    v = st["v_cache"][at].float()
    t = torch.arange(nm, device="cuda")
    row = (start[:-1, None] + t).clamp(max=T - 1)
    qp = (q[row].float() / math.sqrt(d)).view(R, nm, Hkv, -1, d).permute(0, 2, 3, 1, 4)
    s = qp.reshape(R, Hkv, -1, d) @ k.transpose(-1, -2)
    s.masked_fill_(hidden[:, None, None], -math.inf)
    s.sub_(s.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()  # a row without states sums to 0
    o = (s @ v) / s.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.view(R, Hkv, Hq // Hkv, nm, d).permute(0, 3, 1, 2, 4).reshape(R, nm, Hq, d)
    return o[t < start.diff()[:, None]].to(q.dtype)


def _run_step(st):
    ids, d = st["state_ids"].long(), st["d"]
    q, k, v = (st[x].float() for x in "qkv")
    lam = st["log_decay"].exp()[:, None, None]
    held = (st["context_lens"] > 1)[:, None, None, None]
    s = torch.where(held, st["states"][ids] * lam, 0.0) + k[..., :, None] * v[..., None, :]
    st["states"][ids] = s
    o = (q[..., None, :] @ s)[..., 0, :] / math.sqrt(d)
    return o.to(st["q"].dtype), st["states"]


def _run_prompt(st):
    """Chunks of C tokens: each over its own tokens, and over the state before it, which follows from
    the chunks' own sums by one product with the decays between them."""
    ids, d, H, R, C = st["state_ids"].long(), st["d"], st["H"], st["R"], _CHUNK
    start, T = st["query_start"].long(), st["q"].shape[0]
    n = start.diff()
    N = -(-st["max_query_len"] // C)
    t = torch.arange(N * C, device="cuda")
    inside = t < n[:, None]
    row = torch.where(inside, start[:-1, None] + t, 0)
    # the requests' tokens at the ends of their rows, so that all states end together
    late = (row.shape[1] - n)[:, None]
    row, inside = row.gather(1, (t - late).clamp(min=0)), t >= late
    q, k, v = ((st[x][row].float() * inside[..., None, None]).view(R, N, C, H, d).permute(0, 3, 1, 2, 4) for x in "qkv")
    g = st["log_decay"].double()
    i = torch.arange(C, device="cuda")
    far = (i[:, None] - i).double()
    D = torch.where(far >= 0, (far.clamp(min=0) * g[:, None, None]).exp(), 0.0).float()  # [H][C][C]
    to_end = ((C - 1 - i) * g[:, None]).exp().float()[:, None, :, None]
    since = ((i + 1) * g[:, None]).exp().float()[:, None, :, None]
    own_sum = (k * to_end).transpose(-1, -2) @ v  # [R][H][N][d][d]
    c = torch.arange(N + 1, device="cuda")
    gap = (c[:, None] - 1 - c[:N]).double()
    A = torch.where(gap >= 0, (gap.clamp(min=0) * (C * g[:, None, None])).exp(), 0.0).float()  # [H][N + 1][N]
    s = (A @ own_sum.view(R, H, N, d * d)).view(R, H, N + 1, d, d)
    # the state before the call, decayed from its last token to the end of each chunk
    held = (st["context_lens"] > n)[:, None, None, None]
    s0 = torch.where(held, st["states"][ids], 0.0)
    since0 = (c * C - late).clamp(min=0)[:, None].double() * g[:, None]  # [R][H][N + 1]
    s = s + since0.exp().float()[..., None, None] * s0[:, :, None]
    # rows before a request's first token multiply it by 0, but its first chunk starts inside
    into = (t - late + 1).clamp(min=0)[:, None].double() * g[:, None]  # [R][H][N * C]
    since = torch.where((c[:N] * C - late < 0)[:, None, :, None], into.view(R, H, N, C).exp().float(), since[:, 0, :, 0][:, None])
    o = ((q @ k.transpose(-1, -2)) * D[:, None]) @ v + since[..., None] * (q @ s[:, :, :N])
    st["states"][ids] = s[:, :, N]
    o = (o / math.sqrt(d)).permute(0, 2, 3, 1, 4).reshape(R, N * C, H, d)
    return o[inside].to(st["q"].dtype), st["states"]


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "plan":
        rows, bs = _plan_rows(case), case["bs"]
        held = sum(-(-r[0] // bs) for r in rows if r)
        most = sum(-(-(r[0] + r[1]) // bs) for r in rows if r)
        tokens = sum(r[1] for r in rows if r) + 3
        # two calls: the sequences' pages in, tables out; pages taken and given back; rows; tokens
        return {"bytes": 4 * (held + most + 2 * case["R"] * case["width"]) + 4 * 4 * (most - held) + 2 * 24 * case["R"]
                         + 2 * 16 * tokens, "flops": 0}
    d, es = case["d"], _ES[case["dtype"]]
    if op == "cross":
        n = _spread(case["n_lo"], case["n_hi"], case["R"])
        e = _spread(case["e_lo"], case["e_hi"], case["R"])[::-1]
        return {"bytes": 2 * es * d * (sum(e) * case["Hkv"] + sum(n) * case["Hq"]) + 4 * sum(-(-x // case["bs"]) for x in e),
                "flops": 4 * case["Hq"] * d * sum(a * b for a, b in zip(n, e))}
    H = case["H"]
    if op == "step":
        B = case["B"]
        return {"bytes": H * d * (4 * B * es + (2 * B - case["fresh"]) * d * 4), "flops": 5 * B * H * d * d}
    n = _spread(case["n_lo"], case["n_hi"], case["R"])
    return {"bytes": H * d * (4 * sum(n) * es + (2 * case["R"] - case["fresh"]) * d * 4), "flops": 5 * sum(n) * H * d * d}


# --------------------------------------------------------------------------
# the definition in 64 bits, sequence by sequence
# --------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    st = prepare(case, seed)
    scale, parts = case["d"] ** -0.5, []
    if case["op"] == "cross":
        bs, gq = case["bs"], case["Hq"] // case["Hkv"]
        start = st["query_start"].tolist()
        for r, e in enumerate(st["encoder_lens"].tolist()):
            j = torch.arange(e, device="cuda")
            page = st["table"][r].long()[j // bs]
            K, V = (st[x].permute(0, 2, 1, 3)[page, j % bs].double().repeat_interleave(gq, 1) for x in ("k_cache", "v_cache"))
            for a in range(start[r], start[r + 1], 512):
                q = st["q"][a:min(a + 512, start[r + 1])].double()
                w = (torch.einsum("mhd,jhd->hmj", q, K) * scale).softmax(-1) if e else q.new_zeros(case["Hq"], len(q), 0)
                parts.append(torch.einsum("hmj,jhd->mhd", w, V))
        return torch.cat(parts)
    start = st["query_start"].tolist() if case["op"] == "prompt" else list(range(case["B"] + 1))
    states = st["states"].double()
    lam = st["log_decay"].double().exp()
    for r, slot in enumerate(st["state_ids"].tolist()):
        a, b = start[r], start[r + 1]
        S = states[slot] if int(st["context_lens"][r]) > b - a else torch.zeros_like(states[slot])
        for x in range(a, b, 64):
            q, k, v = (st[y][x:min(x + 64, b)].double().transpose(0, 1) for y in "qkv")
            m = q.shape[1]
            i = torch.arange(m, device="cuda", dtype=torch.float64)
            decay = (lam[:, None, None] ** (i[:, None] - i).clamp(min=0)).tril()
            o = (torch.einsum("hid,hjd->hij", q, k) * decay) @ v
            o += lam[:, None, None] ** (i[:, None] + 1) * (q @ S)
            S = lam[:, None, None] ** m * S + (k * lam[:, None, None] ** (m - 1 - i)[:, None]).transpose(1, 2) @ v
            parts.append(o.transpose(0, 1) * scale)
        states[slot] = S
    return torch.cat(parts), states
