"""Prefill over a 4-bit cache with bad table entries: what a step attends to is the cache's, never what the staging cache
held before."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_08_gb300 as pa
from oracle import q4_cache as q4
from paged_kv_gqa_08_gb300.step import alloc_step_buffers, run_step
from test_gpu_bad_pages import close
from test_gpu_q4_step import DT, Model

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda_lib")]


@pytest.mark.parametrize("poison", ["nan", "large"])
@pytest.mark.parametrize("dtype,hq,hkv,hd,gs,P", [("bf16", 16, 8, 128, 32, 16), ("bf16", 8, 2, 128, 128, 64),
                                                  ("bf16", 12, 4, 64, 64, 16), ("f32", 4, 2, 64, 32, 16)])
def test_skipped_pages_are_not_attended_to(dtype, hq, hkv, hd, gs, P, poison):
    """Entries out of range among the pages of a prefix, of the new tokens, of a whole request: the step over the 4-bit
    cache answers as pa_prefill_varlen does over a cache of the dtype with the same rows and the same tables."""
    same = close if dtype == "bf16" and hd == 128 else torch.equal
    m = Model(dtype, hq, hkv, hd, gs, P, maxp=384 // P, batch=4, norm=False, seed=hq + gs)
    bufs = alloc_step_buffers(m.desc, "prefill", 500, 4, 384, "cuda", max_seqlen_q=200, group_size=gs)
    m.step("prefill", [150, 170, 90, 64], bufs)
    for x in (bufs.staging.k, bufs.staging.v):
        x.fill_(float("nan") if poison == "nan" else 1e3)
    good = m.bt.copy()
    m.bt[0, 1] = m.desc.num_pages                 # inside the prefix
    m.bt[1, 200 // P] = -1                        # the new tokens' page
    m.bt[3, :] = 1 << 30                          # every page
    new = np.array([20, 33, 1, 17])
    ctx = (m.lens + new).astype(np.int32)
    n = int(new.sum())
    q, k, v = m.rand(n, hq, hd), m.rand(n, hkv, hd), m.rand(n, hkv, hd)
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
    ctx_d, bt_d = torch.from_numpy(ctx).cuda(), torch.from_numpy(m.bt).cuda()
    bufs.out.fill_(7.0)
    run_step(m.desc, "prefill", bufs, q, k, v, cu, ctx_d, bt_d, *m.caches, m.scale, m.maxp, int(ctx.max()), 33)
    assert pa.pa_read_device_errors(reset=True) == pa.PA_DEVERR_BAD_PAGE
    slots = np.arange(m.caches[0].shape[0])
    plain = [torch.from_numpy(q4.row_values(c.cpu().numpy(), slots, hkv, hd, gs)).float().to(DT[dtype]).cuda()
             for c in m.caches]
    want = torch.full_like(bufs.out, 7.0)
    pa.pa_prefill_varlen(m.desc, q, cu, 4, 33, n, *plain, bt_d, m.maxp, ctx_d, int(ctx.max()), m.scale, want,
                         bufs.workspace)
    assert pa.pa_read_device_errors(reset=True) == pa.PA_DEVERR_BAD_PAGE
    assert same(bufs.out[:n], want[:n])
    assert torch.isfinite(bufs.out[:n]).all()
    m.bt[:] = good                                # the tables of the next step are its own
    bt_d.copy_(torch.from_numpy(good))
    run_step(m.desc, "prefill", bufs, q, k, v, cu, ctx_d, bt_d, *m.caches, m.scale, m.maxp, int(ctx.max()), 33)
    assert pa.pa_read_device_errors(reset=True) == 0
    plain = [torch.from_numpy(q4.row_values(c.cpu().numpy(), slots, hkv, hd, gs)).float().to(DT[dtype]).cuda()
             for c in m.caches]
    pa.pa_prefill_varlen(m.desc, q, cu, 4, 33, n, *plain, bt_d, m.maxp, ctx_d, int(ctx.max()), m.scale, want,
                         bufs.workspace)
    assert same(bufs.out[:n], want[:n])


@pytest.mark.parametrize("maxp,maxp_out", [(4, 4), (3, 6), (7, 2), (300, 301)])
def test_tables_of_the_rows_read_back(maxp, maxp_out):
    """Good and bad entries, requests with fewer rows than the tables have pages, rows that start late or below 0."""
    rng = np.random.default_rng(maxp)
    P, pages, B = 32, 50, 9
    room = rng.integers(0, maxp_out + 2, B) * P
    cu = np.concatenate([[0], np.cumsum(room)]).astype(np.int32)
    bt = rng.integers(-3, pages + 3, (B, maxp)).astype(np.int32)
    bt[0, 0], bt[1, -1] = 1 << 30, -(1 << 31)
    want = np.full((B, maxp_out), -1, np.int32)
    for b in range(B):
        for j in range(min(maxp, maxp_out, room[b] // P)):
            if 0 <= bt[b, j] < pages:
                want[b, j] = cu[b] // P + j
    desc = pa.cache_desc(2, 2, 64, P, pages, torch.float32)
    buf = torch.full((B * maxp_out + 64,), 77, dtype=torch.int32, device="cuda")
    args = [torch.from_numpy(x).cuda() for x in (cu, bt)]
    pa.pa_kv_read_q4_tables(desc, B, *args, maxp, buf, maxp_out)
    got = buf.cpu().numpy()
    assert (got[: B * maxp_out].reshape(B, maxp_out) == want).all() and (got[B * maxp_out:] == 77).all()
    args[0].sub_(cu[1] + P)                                # rows from below 0 on: none of such a request
    pa.pa_kv_read_q4_tables(desc, B, *args, maxp, buf, maxp_out)
    assert (buf[:maxp_out] == -1).all()
    assert pa.pa_read_device_errors(reset=True) == 0
