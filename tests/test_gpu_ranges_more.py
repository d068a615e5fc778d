"""Windows, shared prefixes and tables in calls that their documentation allows and the other tests do not make: rows normed
and rotated by the step, queries, rows and outputs in pinned host memory, tables of tens of thousands of rows."""
import random

import pytest
import torch

import paged_kv_gqa_08_gb300 as pa
from paged_kv_gqa_08_gb300.step import alloc_step_buffers, run_step
from range_reference import Paged
from test_gpu_tables import Dev, Ref, flags
from test_gpu_window_decode import decode

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dt,hd", [(BF16, 128), (BF16, 64), (F32, 128)])
@pytest.mark.parametrize("how", ["window decode", "window prefill", "groups"])
def test_steps_that_norm_and_rotate(cuda_lib, dt, hd, how):
    """The step is its calls, bit for bit: the write part with norm and rotary, then attention over what it wrote."""
    Hq, Hkv, B = 8, 2, 3
    lens = [70, 300, 41]
    new = [1] * B if how != "window prefill" else [33, 150, 41]
    n, mx = sum(new), max(lens)
    c = [Paged(lens, Hq, Hkv, hd, 16, dt, seed=1, fill=0.0) for _ in range(2)]
    q, k, v = c[0].randn(n, Hq, hd), c[0].randn(n, Hkv * hd), c[0].randn(n, Hkv * hd)
    wq, wk = (1 + 0.1 * c[0].randn(hd).float()).to(dt), (1 + 0.1 * c[0].randn(hd).float()).to(dt)
    cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32, device="cuda")
    kind = "prefill" if how.endswith("prefill") else "decode"
    i32 = dict(dtype=torch.int32, device="cuda")
    kw = dict(window=50, num_sinks=4)
    if how == "groups":
        for x in c:     # requests 0 and 1 begin with the same two pages
            x.bt[1, :2] = x.bt[0, :2]
        kw = dict(cu_groups=torch.tensor([0, 2], **i32), prefix_lens=torch.tensor([32], **i32), max_prefix_len=32)
    bufs = [alloc_step_buffers(x.desc, kind, n, B, mx, "cuda", norm=True, max_seqlen_q=max(new),
                               window=kw.get("window", 0), num_sinks=4, num_groups=how == "groups", max_prefix_len=32)
            for x in c]
    got = run_step(c[0].desc, kind, bufs[0], q, k, v, cu, c[0].ctx, c[0].bt, c[0].k, c[0].v, 0.1, c[0].maxp, mx, max(new),
                   wq, wk, 1e-6, 1e4, **kw)
    d, b = c[1], bufs[1]
    pa.pa_prefill_qk_norm_rope_kv_write(d.desc, q, Hq * hd, k, Hkv * hd, v, Hkv * hd, n, cu, B, d.ctx, d.bt, d.maxp, wq, wk,
                                        1e-6, 1e4, b.q_out, d.k, d.v, b.positions, b.slots)
    if how == "window decode":
        pa.pa_decode_window(d.desc, 50, 4, b.q_out, B, d.k, d.v, d.bt, d.maxp, d.ctx, mx, 0.1, 0, b.out, b.workspace)
    elif how == "groups":
        pa.pa_decode_shared_prefix(d.desc, 1, kw["cu_groups"], kw["prefix_lens"], 32, b.q_out, B, d.k, d.v, d.bt, d.maxp,
                                   d.ctx, mx, 0.1, 0, b.out, b.workspace)
    else:
        pa.pa_prefill_varlen_window(d.desc, 50, 4, b.q_out, cu, B, max(new), n, d.k, d.v, d.bt, d.maxp, d.ctx, mx, 0.1,
                                    b.out, b.workspace)
    assert not torch.isnan(got.float()).any() and got.float().abs().max() > 0
    for x, y in ((got, b.out), (c[0].k, d.k), (c[0].v, d.v), (bufs[0].q_out, b.q_out)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert flags() == 0


@pytest.mark.parametrize("window", [9, 120, 5000])
def test_windowed_decode_with_rows_and_output_in_pinned_host_memory(cuda_lib, window):
    lens = [1, 130, 700, 64, 0, 333]
    c = [Paged(lens, 8, 4, 128, 16, BF16, seed=window, fill=0.0) for _ in range(2)]
    q, k, v = c[0].randn(6, 8, 128), c[0].randn(6, 512), c[0].randn(6, 512)
    ws = torch.empty(pa.pa_decode_window_workspace_size(c[0].desc, window, 4, 6, 700), dtype=torch.uint8, device="cuda")
    outs = []
    for x, pinned in zip(c, (False, True)):
        rows = [t.cpu().pin_memory() if pinned else t for t in (q, k, v)]
        out = torch.zeros(6, 8, 128, dtype=BF16)
        out = out.pin_memory() if pinned else out.cuda()
        pa.pa_decode_kv_write_window(x.desc, window, 4, rows[0], rows[1], 512, rows[2], 512, 6, x.k, x.v, x.bt, x.maxp,
                                     x.ctx, 700, 0.1, 0, None, out, ws)
        torch.cuda.synchronize()
        outs.append(out.cpu().clone())
    assert torch.equal(outs[0].view(torch.uint8), outs[1].view(torch.uint8)) and outs[0].float().abs().max() > 0
    assert torch.equal(c[0].k.view(torch.uint8), c[1].k.view(torch.uint8))
    got = decode(c[0], window, 4, q, 0.1)
    live = torch.tensor(lens) > 0
    assert torch.equal(got.cpu()[live].view(torch.uint8), outs[1][live].view(torch.uint8))


@pytest.mark.parametrize("B", [12000, 32768])
def test_tables_of_many_rows(cuda_lib, B):
    """Sums over the rows that need more than a kernel's default shared memory."""
    r = random.Random(B)
    ref = Ref(3 * B, 16, B, 6, seed=B, start=5)
    dev = Dev(ref)
    new = [r.choice([0, 1, 16, 17, 30]) for _ in range(B)]
    want = ref.extend(new, sum(new) + 3)
    assert dev.extend(new, sum(new) + 3) == want[:3]
    ref.release_window(5, 0)
    dev.release_window(5, 0)
    dev.same(ref)
    first, end = [r.choice([0, 0, 1]) for _ in range(B)], [r.choice([0, 1, 2, 6]) for _ in range(B)]
    ref.release(first, end)
    dev.release(first, end)
    dev.same(ref)
    assert flags() == 0
