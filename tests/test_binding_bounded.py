"""Refusals of the bounded-cache calls (rotary store, compaction, windowed
decode and prefill): mismatched shapes by the binding before any pointer reaches the
library, bad sizes by the library before it touches CUDA.  CPU only."""
import ctypes

import pytest
import torch

from paged_kv_cache_192_gb300 import ops

bf16, f32, i32, i64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_192_gb300 import build
    build.build()
    from paged_kv_cache_192_gb300 import _lib
    return _lib.lib()


def pools(NB=8, Hkv=2, bs=16, d=64):
    return torch.zeros(NB, Hkv, bs, d, dtype=bf16), torch.zeros(NB, Hkv, bs, d, dtype=bf16)


def rope_args(T=5):
    k, v = pools()
    return dict(q=torch.zeros(T, 4, 64, dtype=bf16), k_new=torch.zeros(T, 2, 64, dtype=bf16),
                v_new=torch.zeros(T, 2, 64, dtype=bf16), k_cache=k, v_cache=v,
                slot_mapping=torch.zeros(T, dtype=i64), positions=torch.zeros(T, dtype=i64),
                inv_freq=torch.zeros(32))


@pytest.mark.parametrize("bad,msg", [
    (dict(q=torch.zeros(5, 256, dtype=bf16)), "q must be"),
    (dict(q=torch.zeros(5, 4, 32, dtype=bf16)), "q must be"),
    (dict(k_new=torch.zeros(4, 2, 64, dtype=bf16)), "k_new must be"),
    (dict(v_new=torch.zeros(5, 3, 64, dtype=bf16)), "v_new must be"),
    (dict(v_cache=torch.zeros(8, 2, 8, 64, dtype=bf16)), "same shape"),
    (dict(slot_mapping=torch.zeros(4, dtype=i64)), "slot_mapping"),
    (dict(positions=torch.zeros(4, dtype=i64)), "positions"),
    (dict(positions=torch.zeros(3, 4, dtype=i64)), "positions"),
    (dict(positions=torch.zeros(3, 5, dtype=i64)), "sections"),
    (dict(sections=(16, 16)), "sections"),
    (dict(inv_freq=torch.zeros(2, 16)), "inv_freq"),
    (dict(q_out=torch.zeros(5, 4, 32, dtype=bf16)), "q_out must be"),
    (dict(q=torch.zeros(4, 5, 64, dtype=bf16).transpose(0, 1)), "contiguous"),
    (dict(k_new=torch.zeros(5, 2, 128, dtype=bf16)[..., ::2]), "contiguous"),
])
def test_rope_rejects_mismatched_tensors(bad, msg):
    with pytest.raises(ValueError, match=msg):
        ops.rope_reshape_and_cache(**{**rope_args(), **bad})


def test_rope_then_device_check():
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.rope_reshape_and_cache(**rope_args())


def compact_args(B=3):
    k, v = pools()
    return dict(k_cache=k, v_cache=v, src_table=torch.zeros(B, 4, dtype=i32),
                dst_table=torch.zeros(B, 2, dtype=i32), keep=torch.zeros(B, 2, 20, dtype=i32),
                keep_lens=torch.zeros(B, dtype=i32))


@pytest.mark.parametrize("bad,msg", [
    (dict(k_cache=torch.zeros(8, 2, 16, dtype=bf16)), "pools"),
    (dict(v_cache=torch.zeros(8, 2, 8, 64, dtype=bf16)), "same shape"),
    (dict(keep=torch.zeros(3, 1, 20, dtype=i32)), "keep must be"),
    (dict(keep=torch.zeros(3, 20, dtype=i32)), "keep must be"),
    (dict(src_table=torch.zeros(2, 4, dtype=i32)), "src_table"),
    (dict(dst_table=torch.zeros(3, 0, dtype=i32)), "dst_table"),
    (dict(keep_lens=torch.zeros(4, dtype=i32)), "keep_lens"),
])
def test_compact_rejects_mismatched_tensors(bad, msg):
    with pytest.raises(ValueError, match=msg):
        ops.compact_cache(**{**compact_args(), **bad})


def test_compact_then_device_check():
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.compact_cache(**compact_args())


def window_args(B=3):
    k, v = pools()
    return dict(q=torch.zeros(B, 4, 64, dtype=bf16), k_cache=k, v_cache=v,
                block_table=torch.zeros(B, 4, dtype=i32), context_lens=torch.ones(B, dtype=i32),
                window=16)


@pytest.mark.parametrize("bad,msg", [
    (dict(out=torch.zeros(2, 4, 64, dtype=bf16)), "out must have the shape of q"),
    (dict(block_table=torch.zeros(2, 4, dtype=i32)), "block_table must be"),
    (dict(context_lens=torch.ones(4, dtype=i32)), "context_lens must be"),
    (dict(q=torch.zeros(3, 4, 128, dtype=bf16)), "head_dim"),
    (dict(v_cache=torch.zeros(8, 2, 8, 64, dtype=bf16)), "same shape"),
])
def test_decode_window_rejects_mismatched_tensors(bad, msg):
    with pytest.raises(ValueError, match=msg):
        ops.decode_window(**{**window_args(), **bad})


def test_decode_window_then_device_check():
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.decode_window(**window_args())


def prefill_args(R=3, T=10):
    k, v = pools()
    return dict(q=torch.zeros(T, 4, 64, dtype=bf16), k_cache=k, v_cache=v,
                block_table=torch.zeros(R, 4, dtype=i32), query_start=torch.zeros(R + 1, dtype=i32),
                context_lens=torch.ones(R, dtype=i32), max_query_len=10, window=16)


@pytest.mark.parametrize("bad,msg", [
    (dict(out=torch.zeros(9, 4, 64, dtype=bf16)), "out must have the shape of q"),
    (dict(block_table=torch.zeros(2, 4, dtype=i32)), "block_table must be"),
    (dict(query_start=torch.zeros(3, dtype=i32)), "query_start must be"),
    (dict(context_lens=torch.ones(3, 1, dtype=i32)), "context_lens"),
    (dict(q=torch.zeros(10, 4, 128, dtype=bf16)), "head_dim"),
    (dict(v_cache=torch.zeros(8, 2, 8, 64, dtype=bf16)), "same shape"),
])
def test_prefill_window_rejects_mismatched_tensors(bad, msg):
    with pytest.raises(ValueError, match=msg):
        ops.prefill_window(**{**prefill_args(), **bad})


def test_prefill_window_then_device_check():
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.prefill_window(**prefill_args())


# ---- the C ABI ------------------------------------------------------------------
P = ctypes.c_void_p


def c_rope(lib, **kw):
    a = dict(qs=256, ks=128, vs=128, os=256, sections=(ctypes.c_int * 4)(32, 0, 0, 0), axes=1, T=3,
             NB=8, Hq=4, Hkv=2, bs=16, d=64, rot=64, dtype=0, ptr=None)
    a.update(kw)
    p = a["ptr"]
    return lib.pa_rope_reshape_and_cache(p, a["os"], p, a["qs"], p, a["ks"], p, a["vs"], p, p, p, p, p,
                                         a["sections"], a["axes"], 0, a["T"], a["NB"], a["Hq"],
                                         a["Hkv"], a["bs"], a["d"], a["rot"], a["dtype"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=5), 1), (dict(T=-1), 1), (dict(NB=0), 1), (dict(Hq=0), 1), (dict(bs=24), 1),
    (dict(d=60, rot=60), 1), (dict(rot=66), 1), (dict(rot=0), 1), (dict(rot=63), 1),
    (dict(rot=24, sections=(ctypes.c_int * 4)(12)), 4),  # half a rotation is no whole piece
    (dict(d=1024, rot=1024, qs=4096, os=4096, ks=2048, vs=2048,
          sections=(ctypes.c_int * 4)(512)), 4),
    (dict(axes=0), 1), (dict(axes=5), 1), (dict(sections=None), 1),
    (dict(sections=(ctypes.c_int * 4)(31)), 1), (dict(sections=(ctypes.c_int * 4)(33)), 1),
    (dict(axes=2, sections=(ctypes.c_int * 4)(33, -1)), 1),
    (dict(axes=2, sections=(ctypes.c_int * 4)(2 ** 31 - 1, 2 ** 31 - 1)), 1),
    (dict(qs=255), 1), (dict(ks=64), 1), (dict(vs=130), 1), (dict(os=0), 1), (dict(qs=2 ** 29), 1),
    (dict(), 1),                       # NULL pointers
    (dict(ptr=P(8)), 1),               # not 16-byte aligned
    (dict(T=0), 0),
])
def test_rope_c_refusals(lib, kw, code):
    assert c_rope(lib, **kw) == code
    assert bool(lib.pa_last_error_string()) == (code != 0)


def c_compact(lib, **kw):
    a = dict(MBs=4, MBd=2, mk=20, B=3, NB=8, Hkv=2, bs=16, d=64, dtype=0, ptr=None)
    a.update(kw)
    p = a["ptr"]
    return lib.pa_compact_cache(p, p, p, a["MBs"], p, a["MBd"], p, a["mk"], p, a["B"], a["NB"],
                                a["Hkv"], a["bs"], a["d"], a["dtype"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=5), 1), (dict(B=-1), 1), (dict(B=65536), 1), (dict(NB=0), 1), (dict(Hkv=0), 1),
    (dict(bs=12), 1), (dict(d=60), 1), (dict(MBs=0), 1), (dict(MBd=0), 1), (dict(mk=-1), 1),
    (dict(MBs=2 ** 27), 1), (dict(NB=2 ** 26), 4), (dict(), 1), (dict(ptr=P(8)), 1), (dict(B=0), 0),
    (dict(mk=0), 0),
])
def test_compact_c_refusals(lib, kw, code):
    assert c_compact(lib, **kw) == code
    assert bool(lib.pa_last_error_string()) == (code != 0)


def c_window(lib, **kw):
    a = dict(MB=4, B=2, Hq=4, Hkv=4, d=64, bs=16, NB=8, scale=0.125, window=8, sinks=0, dtype=0,
             ptr=None)
    a.update(kw)
    p = a["ptr"]
    return lib.pa_decode_window(p, p, p, p, p, a["MB"], p, a["B"], a["Hq"], a["Hkv"], a["d"],
                                a["bs"], a["NB"], a["scale"], a["window"], a["sinks"], a["dtype"],
                                None)


WINDOW_REFUSALS = [
    (dict(dtype=7), 1), (dict(d=96), 4), (dict(Hq=12, Hkv=8), 1), (dict(Hq=32, Hkv=2), 4),
    (dict(bs=24), 4), (dict(bs=256), 4), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(window=0), 1), (dict(window=-5), 1), (dict(sinks=-1), 1),
    (dict(MB=0), 1), (dict(MB=2 ** 27), 1), (dict(NB=0), 1),
    (dict(NB=2 ** 25), 4),  # 2^31 pool rows
    (dict(B=-1), 1), (dict(), 1), (dict(ptr=P(8)), 1), (dict(B=0), 0),
]


@pytest.mark.parametrize("kw,code", WINDOW_REFUSALS)
def test_decode_window_c_refusals(lib, kw, code):
    assert c_window(lib, **kw) == code
    assert bool(lib.pa_last_error_string()) == (code != 0)


def c_prefill(lib, **kw):
    a = dict(MB=4, R=2, T=10, mq=5, Hq=4, Hkv=4, d=64, bs=16, NB=8, scale=0.125, window=8, sinks=0,
             dtype=0, ptr=None)
    a.update(kw)
    p = a["ptr"]
    return lib.pa_prefill_window(p, p, p, p, p, a["MB"], p, p, a["R"], a["T"], a["mq"], a["Hq"],
                                 a["Hkv"], a["d"], a["bs"], a["NB"], a["scale"], a["window"],
                                 a["sinks"], a["dtype"], None)


@pytest.mark.parametrize("kw,code", [x for x in WINDOW_REFUSALS if "B" not in x[0]] + [
    (dict(dtype=1), 4), (dict(R=-1), 1), (dict(T=-1), 1), (dict(mq=-1), 1), (dict(R=0), 0),
    (dict(T=0), 0), (dict(mq=0), 0), (dict(T=2 ** 31 - 1, Hq=1024, Hkv=1024), 4),
])
def test_prefill_window_c_refusals(lib, kw, code):
    assert c_prefill(lib, **kw) == code
    assert bool(lib.pa_last_error_string()) == (code != 0)


@pytest.mark.parametrize("x", [2 ** 31, -2 ** 31 - 1, 2 ** 70])
@pytest.mark.parametrize("name", ["window", "num_sinks"])
def test_host_integers_that_would_wrap(x, name):
    with pytest.raises(ValueError, match="32 bits"):
        ops.decode_window(**{**window_args(), name: x})
    with pytest.raises(ValueError, match="32 bits"):
        ops.prefill_window(**{**prefill_args(), name: x})


@pytest.mark.parametrize("bad", [dict(window=3.5), dict(window=None), dict(scale="x")])
def test_host_arguments_of_other_types(bad):
    with pytest.raises(TypeError):
        ops.decode_window(**{**window_args(), **bad})


def test_things_that_are_no_tensors():
    with pytest.raises(ValueError, match="v_cache must be a CUDA tensor"):
        ops.decode_window(**{**window_args(), "v_cache": None})
    with pytest.raises(TypeError):
        ops.rope_reshape_and_cache(**{**rope_args(), "sections": 64})
    with pytest.raises(ValueError, match="1 to 4 axes"):
        ops.rope_reshape_and_cache(**{**rope_args(), "sections": (1, 1, 1, 1, 60)})


@pytest.mark.parametrize("args,code", [
    ((-1, 10, 5, 4, 4), 1), ((2, -1, 5, 4, 4), 1), ((2, 10, -1, 4, 4), 1), ((2, 10, 5, 0, 4), 1),
    ((2, 10, 5, 4, 0), 1), ((2, 10, 5, 6, 4), 1), ((2, 10, 5, 2048, 2048), 1), ((2, 10, 5, 64, 4), 4),
])
def test_prefill_window_kernel_for_refusals(lib, args, code):
    out = ctypes.c_int(-1)
    assert lib.pa_prefill_window_kernel_for(*args, ctypes.byref(out)) == code
    assert out.value == -1 and lib.pa_last_error_string()
    assert lib.pa_prefill_window_kernel_for(2, 10, 5, 4, 4, None) == 1


def test_prefill_window_kernel_for_needs_a_device(lib):
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")
    out = ctypes.c_int(-1)
    assert lib.pa_prefill_window_kernel_for(2, 10, 5, 4, 4, ctypes.byref(out)) == 3
    assert out.value == -1 and lib.pa_last_error_string()
