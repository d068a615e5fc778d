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
