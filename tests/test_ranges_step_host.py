"""What a step over a window, with groups or over a 4-bit cache refuses before anything is enqueued, without a GPU."""
import pytest

import paged_kv_gqa_08_gb300 as pa
from test_ranges_host import _groups, _step_args, enqueued  # noqa: F401 (a fixture)


def refused(enqueued, status, a):  # noqa: F811
    from paged_kv_gqa_08_gb300.step import run_step

    with pytest.raises(pa.PagedAttnError) as e:
        run_step(**a)
    assert e.value.status == status and not enqueued


@pytest.mark.parametrize("scale", [0.0, -0.1])
def test_shared_prefixes_need_a_positive_scale_without_groups_too(enqueued, scale):  # noqa: F811
    import torch

    a = _step_args(scale=scale, **_groups())
    a.update(cu_groups=torch.tensor([0], dtype=torch.int32))
    refused(enqueued, pa.PA_ERR_SHAPE, a)


def _odd(t):
    import torch
    return torch.zeros(t.numel() + 8, dtype=t.dtype)[1: 1 + t.numel()].view(t.shape)


ROWS = {
    "k's address": (lambda torch, a: a.update(k=_odd(a["k"])), pa.PA_ERR_ALIGN),
    "v's address": (lambda torch, a: a.update(v=_odd(a["v"])), pa.PA_ERR_ALIGN),
    "the cache's address": (lambda torch, a: a.update(v_cache=_odd(a["v_cache"])), pa.PA_ERR_ALIGN),
    "k's stride": (lambda torch, a: a.update(k=torch.zeros(a["k"].shape[0], 8 * 128 + 4, dtype=torch.bfloat16)[:, :1024]),
                   pa.PA_ERR_ALIGN),
    "v's rows": (lambda torch, a: a.update(v=torch.zeros(1024, dtype=torch.bfloat16).expand(a["v"].shape[0], 1024)),
                 pa.PA_ERR_SHAPE),
    "no cache": (lambda torch, a: a.update(k_cache=None), pa.PA_ERR_NULL),
}


@pytest.mark.parametrize("name", ROWS)
@pytest.mark.parametrize("how", ["window decode", "window prefill", "groups", "4-bit decode", "4-bit prefill"])
def test_rows_that_the_write_refuses_are_refused_before_their_slots_are_enqueued(enqueued, how, name):  # noqa: F811
    torch = pytest.importorskip("torch")

    kind = "prefill" if how.endswith("prefill") else "decode"
    if how.startswith("4-bit"):
        from test_q4_host import _step_args as q4_args
        a = q4_args(kind)
    else:
        a = _step_args(kind)
        a.update(_groups() if how == "groups" else dict(window=16, num_sinks=4))
    spoil, status = ROWS[name]
    spoil(torch, a)
    refused(enqueued, status, a)


@pytest.mark.parametrize("kind", ["prefill", "decode"])
def test_caches_that_hold_no_4_bit_rows_are_refused_first(enqueued, kind):  # noqa: F811
    torch = pytest.importorskip("torch")
    from test_q4_host import _step_args as q4_args

    for bad, status in ((torch.zeros(8, 16, 8, 128, dtype=torch.bfloat16), pa.PA_ERR_DTYPE),
                        (torch.zeros(8 * 16, 544, dtype=torch.uint8), pa.PA_ERR_SHAPE)):
        refused(enqueued, status, q4_args(kind, v_cache=bad))


@pytest.mark.parametrize("kind", ["prefill", "decode"])
@pytest.mark.parametrize("window,sinks", [(1 << 31, 4), ((1 << 32) + 16, 4), (16, 1 << 31), (16, (1 << 32) + 1)])
def test_windows_beyond_32_bits_are_refused_first(enqueued, kind, window, sinks):  # noqa: F811
    refused(enqueued, pa.PA_ERR_SHAPE, _step_args(kind, window=window, num_sinks=sinks))


def test_a_prefill_step_over_a_cache_that_its_kernel_does_not_take_is_refused_first(enqueued):  # noqa: F811
    a = _step_args("prefill", window=16)
    a["desc"].num_pages = 1 << 27
    refused(enqueued, pa.PA_ERR_UNSUPPORTED, a)
