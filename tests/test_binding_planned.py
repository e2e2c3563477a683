"""Refusals of the single tokens of linear attention behind a plan.  CPU only."""
import pytest
import torch

from paged_kv_cache_192_gb300 import ops
from test_binding_step import BOTH, decode_args, lib  # noqa: F401


@pytest.mark.parametrize("start", [torch.zeros(3, dtype=torch.int32), torch.zeros(5, dtype=torch.int32),
                                   torch.zeros(4, 1, dtype=torch.int32), [0, 1, 2, 3]])
def test_query_start_has_an_entry_more_than_rows(lib, start):  # noqa: F811
    with pytest.raises(ValueError, match="query_start must be"):
        ops.linear_decode(**decode_args(), query_start=start)


def test_then_device_check(lib):  # noqa: F811
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.linear_decode(**decode_args(), query_start=torch.zeros(4, dtype=torch.int32))


@pytest.mark.parametrize("kw,code", BOTH + [(dict(B=-1), 1), (dict(B=65536), 1), (dict(B=0), 0)])
def test_c_refusals(lib, kw, code):  # noqa: F811
    a = dict(qs=256, ks=256, vs=256, NS=4, B=2, H=4, d=64, scale=0.125, dtype=0, ptr=None)
    a.update(kw)
    p = a["ptr"]
    assert lib.pa_linear_decode_planned(p, p, a["qs"], p, a["ks"], p, a["vs"], p, a["NS"], p, p, p, p, a["B"], a["H"],
                                        a["d"], a["scale"], a["dtype"], None) == code
    assert bool(lib.pa_last_error_string()) == (code != 0)
