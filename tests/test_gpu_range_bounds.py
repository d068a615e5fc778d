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


@pytest.mark.parametrize("dt,hd", [(BF16, 128), (BF16, 64), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("loose", [False, True])
def test_scores_that_are_no_numbers_reach_the_output_whatever_the_bounds(cuda_lib, dt, hd, loose):
    """Requests whose keys several CTAs share, a NaN in a key or in the queries: the same answer where the bounds say that
    nothing is left out (the plain kernel) as where they do not."""
    lens, Hq, Hkv = [3000, 40, 2000, 700], 8, 2
    c = Paged(lens, Hq, Hkv, hd, 16, dt, seed=3)
    c.bt = torch.nn.functional.pad(c.bt, (0, 70), value=-1)
    maxp = c.maxp + 70
    mx = maxp * 16 if loose else 3000
    q = c.randn(4, Hq, hd)
    q[2] = NAN
    c.K[0][1500] = NAN
    c.put(0, torch.arange(3000, device="cuda"), c.K[0], c.V[0])
    outs = {}
    ws = torch.full((pa.pa_decode_window_workspace_size(c.desc, 3000, 0, 4, mx),), 255, dtype=torch.uint8, device="cuda")
    outs["window"] = torch.zeros_like(q)
    pa.pa_decode_window(c.desc, 3000, 0, q, 4, c.k, c.v, c.bt, maxp, c.ctx, mx, 0.1, 0, outs["window"], ws)
    # the step's row is the one that the cache holds already
    rows = [torch.stack([x[b][L - 1].flatten() for b, L in enumerate(lens)]) for x in (c.K, c.V)]
    outs["window, with the write"] = torch.zeros_like(q)
    pa.pa_decode_kv_write_window(c.desc, 2990, 10, q, rows[0], Hkv * hd, rows[1], Hkv * hd, 4, c.k, c.v, c.bt, maxp,
                                 c.ctx, mx, 0.1, 0, None, outs["window, with the write"], ws)
    i32 = dict(dtype=torch.int32, device="cuda")
    for name, groups, most in (("no groups", 0, 0), ("nothing shared", 2, 0), ("a bound", 2, mx if loose else 16)):
        ws = torch.full((pa.pa_decode_shared_prefix_workspace_size(c.desc, groups, 4, most, mx),), 255, dtype=torch.uint8,
                        device="cuda")
        outs[name] = torch.zeros_like(q)
        pa.pa_decode_shared_prefix(c.desc, groups, torch.tensor([0, 2, 4], **i32), torch.zeros(2, **i32), most, q, 4, c.k,
                                   c.v, c.bt, maxp, c.ctx, mx, 0.1, 0, outs[name], ws)
    for name, out in outs.items():
        assert torch.isnan(out[0].float()).all() and torch.isnan(out[2].float()).all(), name
        for b in (1, 3):
            o, bound = attend(q[b: b + 1], c.K[b], c.V[b], torch.ones(1, lens[b], dtype=torch.bool, device="cuda"), 0.1,
                              dt)
            check(out[b: b + 1], o, bound, f"{name}, request {b}")
    assert pa.pa_read_device_errors(reset=True) == 0
