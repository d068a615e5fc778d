"""Windowed prefill and the calls over ranges of keys where the host's bounds and the lengths disagree, and where the bounds
choose the kernel."""
import pytest
import torch

import paged_kv_gqa_08_gb300 as pa
from range_reference import Paged, attend, check

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.mark.parametrize("dt,hd", [(BF16, 128), (BF16, 64), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("plan", [False, True])
@pytest.mark.parametrize("n", [33, 40, 150, 700])
def test_a_chunk_beyond_its_bound_is_skipped_and_flagged(cuda_lib, dt, hd, plan, n):
    """The rows of a chunk of more than max_seqlen_q tokens stay as they were; the others are computed."""
    lens, new, window, sinks, most = [60, n + 9, 200], [32, n, 7], 50, 4, 32
    c = Paged(lens, 4, 2, hd, 16, dt, seed=n)
    q = c.randn(sum(new), 4, hd)
    cu = torch.tensor([0, 32, 32 + n, 39 + n], dtype=torch.int32, device="cuda")
    nbytes = pa.pa_prefill_workspace_size(c.desc, 3, most, sum(new), max(lens)) if plan else 0
    ws = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda") if nbytes else None
    out = torch.full_like(q, NAN)
    pa.pa_prefill_varlen_window(c.desc, window, sinks, q, cu, 3, most, sum(new), c.k, c.v, c.bt, c.maxp, c.ctx,
                                max(lens), 0.1, out, ws)
    at = 0
    for b, (L, k) in enumerate(zip(lens, new)):
        if b == 1:
            assert torch.isnan(out[at: at + k].float()).all()
        else:
            p, j = torch.arange(L - k, L, device="cuda")[:, None], torch.arange(L, device="cuda")
            o, bound = attend(q[at: at + k], c.K[b], c.V[b], (j <= p) & ((j > p - window) | (j < sinks)), 0.1, dt)
            check(out[at: at + k], o, bound, f"request {b}")
        at += k
    assert pa.pa_read_device_errors(reset=True) == pa.PA_DEVERR_BAD_LENGTH
