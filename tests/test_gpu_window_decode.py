"""Decode attention over a sliding window and sinks, against plain attention in 64 bits."""
import pytest
import torch

import paged_kv_gqa_08_gb300 as pa
from range_reference import Paged, attend, check

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def seen_of(L, window, sinks, dev="cuda"):
    j = torch.arange(L, device=dev)
    return (j >= L - window) | (j < sinks)


def hide(c, window, sinks, value=float("nan"), new=1):
    """Poison every token that no query sees, and leave the pages of only such tokens out of the tables."""
    for b, L in enumerate(c.lens):
        if L <= 0:
            continue
        first = max(0, L - new + 1 - window)
        j = torch.arange(L, device=c.dev)
        out = (j < first) & (j >= sinks)
        if out.any():
            bad = torch.full((int(out.sum()), *c.k.shape[2:]), value, dtype=c.dt, device=c.dev)
            c.put(b, j[out], bad, bad)
        for i in range(-(-L // c.P)):
            if i * c.P >= sinks and (i + 1) * c.P <= first:
                c.bt[b, i] = -1


def decode(c, window, sinks, q, scale, max_ctas=0, out=None):
    B = len(c.lens)
    mx = max(max(c.lens), 1)
    nbytes = pa.pa_decode_window_workspace_size(c.desc, window, sinks, B, mx, max_ctas)
    assert 0 < nbytes <= pa.pa_decode_workspace_size(c.desc, B, mx, max_ctas)
    ws = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, float("nan")) if out is None else out
    pa.pa_decode_window(c.desc, window, sinks, q, B, c.k, c.v, c.bt, c.maxp, c.ctx, mx, scale, max_ctas, out, ws)
    return out


def compare(c, window, sinks, q, out, scale, what=""):
    for b, L in enumerate(c.lens):
        if L <= 0:
            assert torch.isnan(out[b].float()).all()
            continue
        o, bound = attend(q[b: b + 1], c.K[b], c.V[b], seen_of(L, window, sinks)[None], scale, c.dt)
        check(out[b: b + 1], o, bound, f"{what} request {b} of {L}")


HEADS = [(BF16, 16, 8, 128), (BF16, 8, 1, 128), (BF16, 3, 1, 128), (BF16, 28, 4, 128), (BF16, 10, 2, 64),
         (BF16, 8, 8, 64), (F32, 4, 2, 64), (F32, 12, 2, 128), (F32, 8, 1, 128)]


@pytest.mark.parametrize("dt,Hq,Hkv,hd", HEADS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (15, 0), (16, 4), (33, 17), (100, 3), (257, 64), (5000, 5)])
def test_against_plain(cuda_lib, dt, Hq, Hkv, hd, window, sinks):
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 100, 0, 117, 118, 300, 1003]
    c = Paged(lens, Hq, Hkv, hd, 16 if sinks != 3 else 64, dt, seed=window + sinks)
    q = c.randn(len(lens), Hq, hd)
    hide(c, window, sinks)
    for max_ctas in (0, 1, 3):
        out = decode(c, window, sinks, q, hd ** -0.5, max_ctas)
        compare(c, window, sinks, q, out, hd ** -0.5, f"{max_ctas} CTAs")
    assert pa.pa_read_device_errors(reset=True) == 0


@pytest.mark.parametrize("dt,hd", [(BF16, 128), (BF16, 64), (F32, 128)])
@pytest.mark.parametrize("P", [16, 256])
def test_split_over_ctas(cuda_lib, dt, hd, P):
    """Few long requests: each one's window is cut over many CTAs."""
    lens, window, sinks = [40000, 9001, 4097], 4096, 100
    c = Paged(lens, 8, 2, hd, P, dt, seed=P)
    q = c.randn(3, 8, hd)
    hide(c, window, sinks)
    out = decode(c, window, sinks, q, 0.1)
    compare(c, window, sinks, q, out, 0.1)
    assert pa.pa_read_device_errors(reset=True) == 0


@pytest.mark.parametrize("dt,hd", [(BF16, 128), (F32, 64)])
@pytest.mark.parametrize("B", [512, 513, 700])
def test_planned_in_the_kernel_and_before(cuda_lib, dt, hd, B):
    lens = [(7 * i) % 330 for i in range(B)]
    c = Paged(lens, 4, 2, hd, 16, dt, seed=B)
    q = c.randn(B, 4, hd)
    hide(c, 40, 5)
    out = decode(c, 40, 5, q, 0.125)
    compare(c, 40, 5, q, out, 0.125)
    assert pa.pa_read_device_errors(reset=True) == 0


@pytest.mark.parametrize("dt,Hq,Hkv,hd", HEADS)
def test_a_window_of_everything_is_plain_decode(cuda_lib, dt, Hq, Hkv, hd):
    lens = [1, 17, 300, 2000, 0, 77]
    c = Paged(lens, Hq, Hkv, hd, 32, dt, seed=5)
    q = c.randn(len(lens), Hq, hd)
    full = torch.full_like(q, float("nan"))
    ws = torch.empty(pa.pa_decode_workspace_size(c.desc, len(lens), 2000), dtype=torch.uint8, device="cuda")
    pa.pa_decode(c.desc, q, len(lens), c.k, c.v, c.bt, c.maxp, c.ctx, 2000, 0.1, 0, full, ws)
    for window, sinks in ((2000, 0), (1 << 30, 7), (1500, 500), ((1 << 31) - 1, (1 << 31) - 1), (1, 2000)):
        out = decode(c, window, sinks, q, 0.1)
        assert torch.equal(out.view(torch.uint8), full.view(torch.uint8)), (window, sinks)
    assert pa.pa_read_device_errors(reset=True) == 0


@pytest.mark.parametrize("dt,Hq,Hkv,hd", HEADS[:1] + HEADS[4:7])
@pytest.mark.parametrize("window,sinks", [(1, 0), (50, 4), (10000, 0)])
def test_step_equals_the_separate_calls(cuda_lib, dt, Hq, Hkv, hd, window, sinks):
    lens = [1, 16, 17, 200, 0, 999, 64]
    B = len(lens)
    row = Hkv * hd
    c = Paged(lens, Hq, Hkv, hd, 16, dt, seed=9)
    hide(c, window, sinks)
    q = c.randn(B, Hq, hd)
    kv = c.randn(B, 2 * row + 32)  # k and v as views of one projection
    k, v = kv[:, :row], kv[:, row: 2 * row]
    ws = torch.empty(pa.pa_decode_window_workspace_size(c.desc, window, sinks, B, 999), dtype=torch.uint8,
                     device="cuda")
    one = [c.k.clone(), c.v.clone(), torch.full((B,), 7, dtype=torch.int64, device="cuda"), torch.zeros_like(q)]
    pa.pa_decode_kv_write_window(c.desc, window, sinks, q, k, kv.stride(0), v, kv.stride(0), B, one[0], one[1], c.bt,
                                 c.maxp, c.ctx, 999, 0.1, 0, one[2], one[3], ws)
    two = [c.k.clone(), c.v.clone(), torch.full((B,), 7, dtype=torch.int64, device="cuda"), torch.zeros_like(q)]
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    pa.pa_slot_mapping(c.desc, B, cu, c.ctx, c.bt, c.maxp, B, pos, two[2])
    pa.pa_kv_write(c.desc, k, kv.stride(0), v, kv.stride(0), B, two[2], two[0], two[1])
    pa.pa_decode_window(c.desc, window, sinks, q, B, two[0], two[1], c.bt, c.maxp, c.ctx, 999, 0.1, 0, two[3], ws)
    for a, b in zip(one, two):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for b, L in enumerate(lens):
        if L:
            c.K[b][L - 1], c.V[b][L - 1] = k[b].view(Hkv, hd), v[b].view(Hkv, hd)
    c.lens = [L if L else -1 for L in lens]
    one[3][4] = float("nan")
    compare(c, window, sinks, q, one[3], 0.1)
    assert pa.pa_read_device_errors(reset=True) == 0


def test_bad_pages_and_lengths_are_flagged(cuda_lib):
    lens, window, sinks = [300, 300, 300, 300], 64, 4
    c = Paged(lens, 4, 2, 128, 16, BF16, seed=1)
    q = c.randn(4, 4, 128)
    c.bt[1, 5] = 1 << 30           # a page of the range that is left out: not looked at
    out = decode(c, window, sinks, q, 0.1)
    compare(c, window, sinks, q, out, 0.1)
    assert pa.pa_read_device_errors(reset=True) == 0
    c.bt[2, 15] = c.num_pages      # a page of the window
    out = decode(c, window, sinks, q, 0.1)
    assert pa.pa_read_device_errors(reset=True) == pa.PA_DEVERR_BAD_PAGE
    for b in (0, 1, 3):
        o, bound = attend(q[b: b + 1], c.K[b], c.V[b], seen_of(300, window, sinks)[None], 0.1, BF16)
        check(out[b: b + 1], o, bound)
    c.ctx[3], c.ctx[0] = 301, -5
    out = decode(c, window, sinks, q, 0.1, out=torch.full_like(q, 3.0))
    assert pa.pa_read_device_errors(reset=True) == pa.PA_DEVERR_BAD_PAGE | pa.PA_DEVERR_BAD_LENGTH
    assert (out[3] == 3.0).all() and (out[0] == 3.0).all() and not (out[1] == 3.0).any()


def test_graph_and_stream(cuda_lib):
    lens, window, sinks = [900, 60, 3], 128, 4
    c = Paged(lens, 8, 4, 128, 16, BF16, seed=2)
    q = c.randn(3, 8, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.full_like(q, float("nan"))
    ws = torch.empty(pa.pa_decode_window_workspace_size(c.desc, window, sinks, 3, 900), dtype=torch.uint8,
                     device="cuda")
    args = (c.desc, window, sinks, q, 3, c.k, c.v, c.bt, c.maxp, c.ctx, 900, 0.1, 0, out, ws)
    pa.pa_decode_window(*args, stream=side)
    side.synchronize()
    first = out.clone()
    compare(c, window, sinks, q, first, 0.1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_decode_window(*args)
    c.lens = [700, 0, 2]
    c.ctx.copy_(torch.tensor(c.lens, dtype=torch.int32))
    out.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    c.K = [K[:L] for K, L in zip(c.K, c.lens)]
    c.V = [V[:L] for V, L in zip(c.V, c.lens)]
    compare(c, window, sinks, q, out, 0.1)
    assert pa.pa_read_device_errors(reset=True) == 0
