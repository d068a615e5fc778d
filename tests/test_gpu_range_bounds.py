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


@pytest.mark.parametrize("dt,hd", [(BF16, 128), (BF16, 64), (F32, 64), (F32, 128)])
def test_the_longest_contexts(cuda_lib, dt, hd):
    """Windows at the end of 2^31 - 128 tokens, whose pages are mostly the same ones; a longer context is skipped."""
    P, window, sinks, most = 1 << 20, 100, 5, 2 ** 31 - 1
    lens = [2 ** 31 - 128, 2 ** 31 - 127, 2 ** 31 - 1, 2 ** 31 - 200, 300]
    maxp = 2 ** 31 // P
    desc = pa.cache_desc(2, 1, hd, P, 3, dt)
    g = torch.Generator(device="cuda").manual_seed(hd)
    k, v = (torch.full((3, P, 1, hd), NAN, dtype=dt, device="cuda") for _ in range(2))
    for x in (k, v):   # the tails of page 1, the heads of pages 0 (the last requests' own) and 2 (everyone's sinks)
        x[1, -1024:] = torch.randn(1024, 1, hd, generator=g, device="cuda").to(dt)
        x[0, :1024] = torch.randn(1024, 1, hd, generator=g, device="cuda").to(dt)
        x[2, :sinks] = torch.randn(sinks, 1, hd, generator=g, device="cuda").to(dt)
    bt = torch.full((5, maxp), -1, dtype=torch.int32, device="cuda")
    bt[:, 0], bt[:, -1], bt[4, 0] = 2, 1, 0
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    new = [3, 3, 3, 70, 3]
    n = sum(new)
    cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32, device="cuda")
    q = torch.randn(n, 2, hd, generator=g, device="cuda").to(dt)

    def keys(b, x):  # the sinks and the last 300 tokens, with their positions
        L = lens[b]
        if L == 300:
            return x[0, :300], torch.arange(300, device="cuda")
        j = torch.cat([torch.arange(sinks, device="cuda"), torch.arange(L - 300, L, device="cuda")])
        return torch.cat([x[2, :sinks], x[1, j[sinks:] % P]]), j

    def compare(b, rows, out, qs):
        p = torch.arange(lens[b] - rows, lens[b], device="cuda")[:, None]
        (K, j), V = keys(b, k), keys(b, v)[0]
        o, bound = attend(qs, K, V, (j <= p) & ((j > p - window) | (j < sinks)), 0.1, dt)
        check(out, o, bound, f"request {b}")

    out = torch.full_like(q, NAN)
    pa.pa_prefill_varlen_window(desc, window, sinks, q, cu, 5, 70, n, k, v, bt, maxp, ctx, most, 0.1, out)
    assert pa.pa_read_device_errors(reset=True) == pa.PA_DEVERR_BAD_LENGTH
    assert torch.isnan(out[3:9].float()).all()
    for b in (0, 3, 4):
        compare(b, new[b], out[cu[b]: cu[b + 1]], q[cu[b]: cu[b + 1]])
    ws = torch.full((pa.pa_decode_window_workspace_size(desc, window, sinks, 5, most),), 255, dtype=torch.uint8,
                    device="cuda")
    out = torch.full_like(q[:5], NAN)
    pa.pa_decode_window(desc, window, sinks, q[:5], 5, k, v, bt, maxp, ctx, most, 0.1, 0, out, ws)
    assert pa.pa_read_device_errors(reset=True) == pa.PA_DEVERR_BAD_LENGTH
    assert torch.isnan(out[1:3].float()).all()
    for b in (0, 3, 4):
        compare(b, 1, out[b: b + 1], q[b: b + 1])
