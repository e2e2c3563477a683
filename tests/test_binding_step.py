"""Refusals of the calls of a serving step (plan, cross attention, linear attention):
mismatched tensors by the binding before any pointer reaches the library, bad sizes by
the library before it touches CUDA.  CPU only."""
import ctypes

import pytest
import torch

from paged_kv_cache_192_gb300 import layout, ops

bf16, f32, i32, i64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_192_gb300 import build
    build.build()
    from paged_kv_cache_192_gb300 import _lib
    return _lib.lib()


# ---- plan ------------------------------------------------------------------------
def plan_args(R=3, S=5):
    return dict(state=layout.page_state(S, 4, 20, device="cpu"), seq_ids=torch.zeros(R, dtype=i32),
                new_tokens=torch.zeros(R, dtype=i32), block_size=16, max_tokens=8)


def changed(**kw):
    st = layout.page_state(5, 4, 20, device="cpu")
    return dict(state=st._replace(**kw))


def outputs(R=3, W=4, T=8):
    return ops.StepPlan(torch.zeros(R, W, dtype=i32), torch.zeros(R, dtype=i32), torch.zeros(R + 1, dtype=i32),
                        torch.zeros(T, dtype=i64), torch.zeros(T, dtype=i64))


@pytest.mark.parametrize("bad,msg", [
    (changed(seq_pages=torch.zeros(5, dtype=i32)), "seq_pages must be"),
    (changed(seq_lens=torch.zeros(4, dtype=i32)), "seq_lens must be"),
    (changed(free_pages=torch.zeros(4, 5, dtype=i32)), "free_pages"),
    (changed(free_state=torch.zeros(2, dtype=i32)), "free_state must be"),
    (dict(seq_ids=torch.zeros(3, 1, dtype=i32)), "seq_ids"),
    (dict(new_tokens=torch.zeros(4, dtype=i32)), "new_tokens must be"),
    (dict(max_tokens=-1), "max_tokens"),
    (dict(table_blocks=-3), "table_blocks"),
    (dict(out=outputs(R=2)), "out must be"),
    (dict(out=outputs(T=7)), "out must be"),
    (dict(out=outputs(), table_blocks=5), "out must be"),
    (dict(out=outputs()[:4]), "StepPlan"),
    (dict(max_tokens=2 ** 31), "32 bits"),
    (dict(table_blocks=2 ** 40), "32 bits"),
])
def test_plan_rejects_mismatched_tensors(lib, bad, msg):
    with pytest.raises(ValueError, match=msg):
        ops.plan_step(**{**plan_args(), **bad})


def test_plan_then_device_check(lib):
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.plan_step(**plan_args())


P = ctypes.c_void_p


def c_plan(lib, **kw):
    a = dict(R=2, MB=4, S=5, NB=20, bs=16, W=4, T=8, ptr=None)
    a.update(kw)
    p = a["ptr"]
    return lib.pa_plan_step(p, p, a["R"], p, a["MB"], p, a["S"], p, p, a["NB"], a["bs"], p, a["W"], p, p, p, p,
                            a["T"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), 1), (dict(R=4097), 4), (dict(S=0), 1), (dict(S=2 ** 19 + 1), 4), (dict(MB=0), 1), (dict(W=0), 1),
    (dict(NB=0), 1), (dict(NB=2 ** 30 + 1), 4), (dict(T=-1), 1), (dict(T=2 ** 30 + 1), 1), (dict(bs=24), 4),
    (dict(bs=4), 4), (dict(bs=256), 4), (dict(MB=2 ** 27), 1), (dict(W=2 ** 27), 1), (dict(), 1),
    (dict(R=0, T=0), 1),  # query_start and the state are written even then
])
def test_plan_c_refusals(lib, kw, code):
    assert c_plan(lib, **kw) == code
    assert lib.pa_last_error_string()


# ---- cross attention ---------------------------------------------------------------
def cross_args(R=3, T=10):
    k = torch.zeros(8, 2, 16, 64, dtype=bf16)
    return dict(q=torch.zeros(T, 4, 64, dtype=bf16), k_cache=k, v_cache=k.clone(),
                block_table=torch.zeros(R, 4, dtype=i32), query_start=torch.zeros(R + 1, dtype=i32),
                encoder_lens=torch.ones(R, dtype=i32), max_query_len=10)


@pytest.mark.parametrize("bad,msg", [
    (dict(q=torch.zeros(10, 256, dtype=bf16)), "q must be"),
    (dict(out=torch.zeros(9, 4, 64, dtype=bf16)), "out must have the shape of q"),
    (dict(block_table=torch.zeros(2, 4, dtype=i32)), "block_table must be"),
    (dict(query_start=torch.zeros(3, dtype=i32)), "query_start must be"),
    (dict(encoder_lens=torch.ones(3, 1, dtype=i32)), "encoder_lens"),
    (dict(q=torch.zeros(10, 4, 128, dtype=bf16)), "head_dim"),
    (dict(v_cache=torch.zeros(8, 2, 8, 64, dtype=bf16)), "same shape"),
    (dict(max_query_len=2 ** 31), "32 bits"),
])
def test_cross_rejects_mismatched_tensors(lib, bad, msg):
    with pytest.raises(ValueError, match=msg):
        ops.cross_attention(**{**cross_args(), **bad})


def test_cross_then_device_check(lib):
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.cross_attention(**cross_args())


def c_cross(lib, **kw):
    a = dict(MB=4, R=2, T=10, mq=5, Hq=4, Hkv=4, d=64, bs=16, NB=8, scale=0.125, dtype=0, ptr=None)
    a.update(kw)
    p = a["ptr"]
    return lib.pa_cross_attention(p, p, p, p, p, a["MB"], p, p, a["R"], a["T"], a["mq"], a["Hq"], a["Hkv"], a["d"],
                                  a["bs"], a["NB"], a["scale"], a["dtype"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), 1), (dict(dtype=1), 4), (dict(d=96), 4), (dict(Hq=12, Hkv=8), 1), (dict(Hq=32, Hkv=2), 4),
    (dict(bs=24), 4), (dict(bs=256), 4), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(MB=0), 1), (dict(MB=2 ** 27), 1), (dict(NB=0), 1), (dict(NB=2 ** 25), 4),
    (dict(R=-1), 1), (dict(R=65536), 1), (dict(T=-1), 1), (dict(mq=-1), 1), (dict(), 1), (dict(ptr=P(8)), 1),
    (dict(T=2 ** 31 - 1, Hq=1024, Hkv=1024), 4), (dict(R=0), 0), (dict(T=0), 0), (dict(mq=0), 0),
])
def test_cross_c_refusals(lib, kw, code):
    assert c_cross(lib, **kw) == code
    assert bool(lib.pa_last_error_string()) == (code != 0)


# ---- linear attention ----------------------------------------------------------------
def decode_args(B=3, H=2, d=64):
    x = torch.zeros(B, H, d, dtype=bf16)
    return dict(q=x, k=x.clone(), v=x.clone(), states=torch.zeros(4, H, d, d), state_ids=torch.zeros(B, dtype=i32),
                context_lens=torch.ones(B, dtype=i32), log_decay=torch.zeros(H))


def prompt_args(R=2, T=3):
    a = decode_args(B=T)
    return dict(a, state_ids=torch.zeros(R, dtype=i32), context_lens=torch.ones(R, dtype=i32),
                query_start=torch.zeros(R + 1, dtype=i32), max_query_len=T)


BAD = [
    (dict(q=torch.zeros(3, 128, dtype=bf16)), "q must be"),
    (dict(k=torch.zeros(3, 3, 64, dtype=bf16)), "k must be"),
    (dict(v=torch.zeros(2, 2, 64, dtype=bf16)), "v must be"),
    (dict(k=torch.zeros(3, 2, 128, dtype=bf16)[..., ::2]), "contiguous"),
    (dict(v=torch.zeros(2, 3, 64, dtype=bf16).transpose(0, 1)), "contiguous"),
    (dict(states=torch.zeros(4, 2, 64, 32)), "states must be"),
    (dict(states=torch.zeros(4, 3, 64, 64)), "states must be"),
    (dict(context_lens=torch.ones(7, dtype=i32)), "context_lens must be"),
    (dict(log_decay=torch.zeros(3)), "log_decay must be"),
    (dict(out=torch.zeros(3, 2, 32, dtype=bf16)), "out must have the shape of q"),
]


@pytest.mark.parametrize("bad,msg", BAD + [(dict(state_ids=torch.zeros(2, dtype=i32),
                                                 context_lens=torch.ones(2, dtype=i32)), "state_ids must be")])
def test_linear_decode_rejects_mismatched_tensors(lib, bad, msg):
    with pytest.raises(ValueError, match=msg):
        ops.linear_decode(**{**decode_args(), **bad})


@pytest.mark.parametrize("bad,msg", BAD + [(dict(query_start=torch.zeros(4, dtype=i32)), "query_start must be"),
                                           (dict(max_query_len=-2 ** 40), "32 bits")])
def test_linear_prefill_rejects_mismatched_tensors(lib, bad, msg):
    with pytest.raises(ValueError, match=msg):
        ops.linear_prefill(**{**prompt_args(), **bad})


def test_linear_then_device_check(lib):
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.linear_decode(**decode_args())
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.linear_prefill(**prompt_args())


def c_decode(lib, **kw):
    a = dict(qs=256, ks=256, vs=256, NS=4, B=2, H=4, d=64, scale=0.125, dtype=0, ptr=None)
    a.update(kw)
    p = a["ptr"]
    return lib.pa_linear_decode(p, p, a["qs"], p, a["ks"], p, a["vs"], p, a["NS"], p, p, p, a["B"], a["H"], a["d"],
                                a["scale"], a["dtype"], None)


def c_prompt(lib, **kw):
    a = dict(qs=256, ks=256, vs=256, NS=4, R=2, T=20, mq=10, H=4, d=64, scale=0.125, ws=None, wb=0, dtype=0, ptr=None)
    a.update(kw)
    p = a["ptr"]
    return lib.pa_linear_prefill(p, p, a["qs"], p, a["ks"], p, a["vs"], p, a["NS"], p, p, p, p, a["R"], a["T"], a["mq"],
                                 a["H"], a["d"], a["scale"], a["ws"], a["wb"], a["dtype"], None)


BOTH = [(dict(dtype=7), 1), (dict(H=0), 1), (dict(H=1025), 1), (dict(NS=0), 1), (dict(d=96, qs=384, ks=384, vs=384), 4),
        (dict(qs=255), 1), (dict(ks=128), 1), (dict(vs=260), 1), (dict(qs=2 ** 29), 1), (dict(scale=0.0), 1),
        (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(), 1), (dict(ptr=P(8)), 1)]


@pytest.mark.parametrize("kw,code", BOTH + [(dict(B=-1), 1), (dict(B=65536), 1), (dict(B=0), 0)])
def test_linear_decode_c_refusals(lib, kw, code):
    assert c_decode(lib, **kw) == code
    assert bool(lib.pa_last_error_string()) == (code != 0)


@pytest.mark.parametrize("kw,code", BOTH + [(dict(R=-1), 1), (dict(R=65536), 1), (dict(T=-1), 1), (dict(mq=-1), 1),
                                            (dict(R=0), 0), (dict(T=0), 0), (dict(mq=0), 0)])
def test_linear_prefill_c_refusals(lib, kw, code):
    assert c_prompt(lib, **kw) == code
    assert bool(lib.pa_last_error_string()) == (code != 0)


def test_linear_workspace(lib):
    """None for fp32, short prompts and batches that fill the GPU; refused if too small."""
    size = ops.linear_prefill_workspace_size
    assert size(1, 16384, 16384, 32, 128, f32) == 0
    assert size(4, 40, 10, 32, 128) == 0
    assert size(64, 64 * 500, 500, 32, 128) == 0
    n = size(1, 16384, 16384, 32, 128)
    assert n > 0 and n % (32 * 128 * 128 * 4) == 0
    # never more segments than the tokens fill, and one per request
    for R, T, mq, H in ((1, 16384, 16384, 32), (3, 9000, 5000, 2), (1, 2 ** 20, 2 ** 20, 1), (2, 300, 299, 1)):
        assert size(R, T, mq, H, 64) <= (T // 64 + R) * H * 64 * 64 * 4
    out = ctypes.c_size_t(0)
    for bad in ((-1, 10, 10, 4, 64, 0), (1, -1, 10, 4, 64, 0), (1, 10, -1, 4, 64, 0), (1, 10, 10, 0, 64, 0),
                (1, 10, 10, 4, 96, 0), (1, 10, 10, 4, 64, 5)):
        assert lib.pa_linear_prefill_workspace_size(*bad, ctypes.byref(out)) == 1
    assert lib.pa_linear_prefill_workspace_size(1, 10, 10, 4, 64, 0, None) == 1
    big = dict(T=16384, mq=16384, R=1, H=1, qs=64, ks=64, vs=64, ptr=P(16))
    assert c_prompt(lib, **big) == 1 and b"needed" in lib.pa_last_error_string()
    assert c_prompt(lib, ws=P(16), wb=64, **big) == 1 and b"needed" in lib.pa_last_error_string()
    assert c_prompt(lib, ws=P(8), wb=2 ** 40, **big) == 1 and b"aligned" in lib.pa_last_error_string()
