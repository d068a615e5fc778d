"""Windowed and shared-prefix attention where requests must not reach each other: NaN in one of them, two streams at
once, hundreds of thousands of keys."""
import pytest
import torch

import paged_kv_gqa_08_gb300 as pa
from range_reference import Paged, attend, check
from test_gpu_shared_prefix import Groups
from test_gpu_window_decode import compare, decode, hide, seen_of
from test_gpu_window_prefill import prefill

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("dt,hd", [(BF16, 128), (BF16, 64), (F32, 128)])
@pytest.mark.parametrize("wide", [False, True])
def test_a_request_of_nan_leaves_its_group_alone(cuda_lib, dt, hd, wide):
    c = Groups([(300, [9, 20, 33, 1]), (150, [4, 5])], 8, 2, hd, 16, dt, 1, wide)
    q = c.randn(6, 8, hd)
    q[1], q[4] = NAN, INF                      # queries of two requests, and own tokens of a third
    j = torch.arange(300, 333, device="cuda")
    c.put(2, j, torch.full_like(c.K[2][:33], NAN), torch.full_like(c.V[2][:33], INF))
    out = c.call(q, 0.1)
    for b in (0, 3, 5):
        seen = torch.ones(1, c.lens[b], dtype=torch.bool, device="cuda")
        o, bound = attend(q[b: b + 1], c.K[b], c.V[b], seen, 0.1, dt)
        check(out[b: b + 1], o, bound, f"request {b}")
    assert not torch.isfinite(out[1].float()).any() and not torch.isfinite(out[2].float()).any()
    assert pa.pa_read_device_errors(reset=True) == 0


@pytest.mark.parametrize("dt,hd", [(BF16, 128), (BF16, 64), (F32, 128)])
def test_rows_of_nan_leave_a_chunk_alone(cuda_lib, dt, hd):
    lens, new, window, sinks = [400, 500, 90], [100, 60, 90], 70, 3
    c = Paged(lens, 8, 2, hd, 16, dt, seed=4)
    q = c.randn(250, 8, hd)
    q[10], q[77], q[130] = NAN, INF, -INF
    c.put(2, torch.arange(90, device="cuda"), torch.full_like(c.K[2], NAN), torch.full_like(c.V[2], NAN))
    for plan in (False, True):
        out = prefill(c, new, q, window, sinks, 0.1, plan)
        at = 0
        for b in (0, 1):
            L, n = lens[b], new[b]
            p, j = torch.arange(L - n, L, device="cuda")[:, None], torch.arange(L, device="cuda")
            good = torch.isfinite(q[at: at + n].float()).flatten(1).all(1)
            o, bound = attend(q[at: at + n][good], c.K[b], c.V[b],
                              ((j <= p) & ((j > p - window) | (j < sinks)))[good], 0.1, dt)
            check(out[at: at + n][good], o, bound, f"request {b}")
            assert torch.isnan(out[at: at + n][~good].float()).all()
            at += n
        assert torch.isnan(out[160:].float()).all()


@pytest.mark.parametrize("dt,hd", [(BF16, 128), (F32, 64)])
@pytest.mark.parametrize("per_request", [True, False])
def test_a_windowed_request_of_nan_leaves_the_batch_alone(cuda_lib, dt, hd, per_request):
    window, sinks = (9, 4) if per_request else (200, 4)
    lens = [250, 30, 251, 7, 300]
    c = Paged(lens, 4, 2, hd, 16, dt, seed=5)
    q = c.randn(5, 4, hd)
    hide(c, window, sinks, value=INF)
    q[1] = NAN
    j = torch.arange(250, 251, device="cuda")
    c.put(2, j, torch.full_like(c.K[2][:1], NAN), torch.full_like(c.V[2][:1], NAN))
    out = decode(c, window, sinks, q, 0.1)
    for b in (0, 3, 4):
        o, bound = attend(q[b: b + 1], c.K[b], c.V[b], seen_of(lens[b], window, sinks)[None], 0.1, dt)
        check(out[b: b + 1], o, bound, f"request {b}")
    assert torch.isnan(out[1].float()).all() and torch.isnan(out[2].float()).all()


def test_two_streams_at_once(cuda_lib):
    """Calls on two streams, each with its own workspace, over the same caches."""
    c = Groups([(2000, [50, 60, 70, 1, 2]), (400, [9, 8])], 16, 8, 128, 16, BF16, 7, True)
    w = Paged([3000, 100, 900, 5], 16, 8, 128, 16, BF16, seed=8)
    qc, qw = c.randn(7, 16, 128), w.randn(4, 16, 128)
    hide(w, 700, 4)
    want_c, want_w = c.call(qc, 0.1), decode(w, 700, 4, qw, 0.1)
    c.compare(qc, want_c, 0.1)
    compare(w, 700, 4, qw, want_w, 0.1)
    streams = [torch.cuda.Stream() for _ in range(2)]
    most = 65536 * 16
    ws = [torch.empty(pa.pa_decode_shared_prefix_workspace_size(c.desc, 2, 7, most, most), dtype=torch.uint8,
                      device="cuda") for _ in range(2)]
    ww = [torch.empty(pa.pa_decode_window_workspace_size(w.desc, 700, 4, 4, 3000), dtype=torch.uint8, device="cuda")
          for _ in range(2)]
    outs = [[torch.empty_like(want_c), torch.empty_like(want_w)] for _ in range(20)]
    torch.cuda.synchronize()
    for i, (oc, ow) in enumerate(outs):
        st = streams[i % 2]
        pa.pa_decode_shared_prefix(c.desc, 2, c.cu, c.pre, most, qc, 7, c.k, c.v, c.bt, c.maxp, c.ctx, most, 0.1, 0, oc,
                                   ws[i % 2], stream=st)
        pa.pa_decode_window(w.desc, 700, 4, qw, 4, w.k, w.v, w.bt, w.maxp, w.ctx, 3000, 0.1, 0, ow, ww[i % 2], stream=st)
    torch.cuda.synchronize()
    for oc, ow in outs:
        assert torch.equal(oc, want_c) and torch.equal(ow, want_w)
    assert pa.pa_read_device_errors(reset=True) == 0


@pytest.mark.parametrize("dt,Hq,Hkv,hd", [(BF16, 8, 2, 128), (BF16, 4, 1, 64), (F32, 4, 2, 64)])
def test_hundreds_of_thousands_of_keys(cuda_lib, dt, Hq, Hkv, hd):
    n = 300001
    c = Groups([(n, [5, 40, 0])], Hq, Hkv, hd, 64, dt, 3)
    q = c.randn(3, Hq, hd)
    for max_ctas in (0, 2):
        c.compare(q, c.call(q, 0.1, max_ctas), 0.1)
    w = Paged([n, 70000], Hq, Hkv, hd, 64, dt, seed=4)
    q = w.randn(2, Hq, hd)
    hide(w, 200003, 77)
    compare(w, 200003, 77, q, decode(w, 200003, 77, q, 0.1), 0.1)
    out = prefill(w, [1, 1], q, 200003, 77, 0.1, False)
    compare(w, 200003, 77, q, out, 0.1)
    assert pa.pa_read_device_errors(reset=True) == 0


@pytest.mark.parametrize("dt,hd", [(BF16, 128), (BF16, 64), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("G", [1, 3, 4, 5])
def test_results_repeat_whatever_ran_before(cuda_lib, dt, hd, G):
    """The same bits again after calls that leave huge values, infinities and NaN in every SM's memory."""
    Hkv, Hq = 2, 2 * G
    own, new, window, sinks = [1, 40, 200, 7, 90], [70, 1, 129, 300, 20], 100, 5
    c = Paged([400, 130, 600, 300, 333], Hq, Hkv, hd, 16, dt, seed=G)
    q = c.randn(sum(new), Hq, hd)
    g = [Groups([(777, own), (130, own[:3])], Hq, Hkv, hd, 16, dt, G, wide) for wide in (False, True)]
    gq = c.randn(8, Hq, hd)
    w = Paged([900] * 40, Hq, Hkv, hd, 16, dt, seed=9)  # as many pairs and requests as reach all SMs
    bad = [x.clone() for x in (w.k, w.v)]

    def calls():
        return [prefill(c, new, q, window, sinks, 0.1, plan) for plan in (False, True)] + \
            [x.call(gq, 0.1) for x in g] + [decode(c, window, sinks, q[:5], 0.1)]

    want = calls()
    for value in (3e4, -3e4, INF, NAN):
        for x in bad:
            x.fill_(value)
        w.k, w.v = bad
        for n in (1, 200):
            prefill(w, [n] * 40, torch.full((40 * n, Hq, hd), value, dtype=dt, device="cuda"), 512, 0, 0.1, False)
        for i, (a, b) in enumerate(zip(calls(), want)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), f"call {i} after {value}"
    assert pa.pa_read_device_errors(reset=True) == 0
