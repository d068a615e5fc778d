"""Chunked prefill over a sliding window and sinks, against plain attention in 64 bits."""
import random

import pytest
import torch

import paged_kv_gqa_08_gb300 as pa
from range_reference import Paged, attend, check

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


def hide(c, new, window, sinks):
    """Poison every token that no row sees, and leave the pages of only such tokens out of the tables."""
    for b, (L, n) in enumerate(zip(c.lens, new)):
        if L <= 0 or n <= 0:
            continue
        first = max(0, L - n + 1 - window)
        j = torch.arange(L, device=c.dev)
        out = (j < first) & (j >= sinks)
        if out.any():
            bad = torch.full((int(out.sum()), *c.k.shape[2:]), NAN, dtype=c.dt, device=c.dev)
            c.put(b, j[out], bad, bad)
        for i in range(-(-L // c.P)):
            if i * c.P >= sinks and (i + 1) * c.P <= first:
                c.bt[b, i] = -1


def prefill(c, new, q, window, sinks, scale, plan, out=None):
    cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32, device="cuda")
    mx, mq, n, B = max(max(c.lens), 1), max(new), int(sum(new)), len(new)
    ws = None
    if plan:
        nbytes = pa.pa_prefill_workspace_size(c.desc, B, mq, n, mx)
        ws = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda") if nbytes else None
    out = torch.full_like(q, NAN) if out is None else out
    pa.pa_prefill_varlen_window(c.desc, window, sinks, q, cu, B, mq, n, c.k, c.v, c.bt, c.maxp, c.ctx, mx, scale, out,
                                ws)
    return out


def compare(c, new, q, out, window, sinks, scale, what=""):
    at = 0
    for b, (L, n) in enumerate(zip(c.lens, new)):
        if L > 0 and n:
            p = torch.arange(L - n, L, device="cuda")[:, None]
            j = torch.arange(L, device="cuda")
            for r in range(0, n, 512):
                pr = p[r: r + 512]
                seen = (j <= pr) & ((j > pr - window) | (j < sinks))
                o, bound = attend(q[at + r: at + r + pr.shape[0]], c.K[b], c.V[b], seen, scale, c.dt)
                check(out[at + r: at + r + pr.shape[0]], o, bound, f"{what} request {b}, rows from {r}")
        elif n:
            assert torch.isnan(out[at: at + n].float()).all()
        at += n


def run(c, new, q, window, sinks, scale=0.088, what=""):
    hide(c, new, window, sinks)
    outs = [prefill(c, new, q, window, sinks, scale, plan) for plan in (False, True)]
    for out, how in zip(outs, ("unplanned", "planned")):
        compare(c, new, q, out, window, sinks, scale, f"{what} {how}")
    assert pa.pa_read_device_errors(reset=True) == 0


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 3), (128, 128), (129, 17), (300, 200),
                                          (1000, 0), (700, 1100)])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
def test_tensor_cores(cuda_lib, G, window, sinks):
    lens = [1, 130, 700, 1500, 2000, 0, 640]
    new = [1, 130, 33, 300, 1, 5, 128]
    c = Paged(lens, 2 * G, 2, 128, 16 if G % 2 else 64, BF16, seed=G)
    run(c, new, c.randn(sum(new), 2 * G, 128), window, sinks)


@pytest.mark.parametrize("dt,Hq,Hkv,hd", [(F32, 4, 2, 64), (F32, 8, 1, 128), (BF16, 6, 2, 64), (BF16, 8, 8, 64)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (33, 4), (128, 100), (400, 0)])
def test_cuda_cores(cuda_lib, dt, Hq, Hkv, hd, window, sinks):
    lens = [1, 70, 300, 513, 0]
    new = [1, 70, 17, 200, 3]
    c = Paged(lens, Hq, Hkv, hd, 32, dt, seed=window)
    run(c, new, c.randn(sum(new), Hq, hd), window, sinks)


@pytest.mark.parametrize("window,sinks", [(512, 4), (2048, 64), (4096, 0)])
def test_long_prompts_and_decode_rows(cuda_lib, window, sinks):
    """Several waves of q-tile pairs (ordered, not split), and decode rows as chunks of one token."""
    lens = [6000, 4097, 9000, 3000, 20000, 129]
    new = [2048, 4097, 1500, 1, 700, 1]
    c = Paged(lens, 16, 8, 128, 16, BF16, seed=window)
    run(c, new, c.randn(sum(new), 16, 128), window, sinks)


def test_split_key_ranges(cuda_lib):
    """A few tokens over a long window: the planner cuts the key range."""
    lens, new = [30000, 16000], [40, 3]
    c = Paged(lens, 8, 2, 128, 256, BF16, seed=3)
    run(c, new, c.randn(43, 8, 128), 12000, 300)


@pytest.mark.parametrize("seed", range(8))
def test_random_batches(cuda_lib, seed):
    r = random.Random(seed)
    B = r.randint(1, 9)
    lens = [int(2 ** r.uniform(0, 12)) for _ in range(B)]
    new = [r.randint(1, L) if r.random() < 0.7 else min(L, r.randint(1, 130)) for L in lens]
    G, Hkv = r.randint(1, 8), r.choice([1, 2, 4, 8])
    window, sinks = int(2 ** r.uniform(0, 11)), r.choice([0, 1, 4, 63, 130, 500])
    c = Paged(lens, G * Hkv, Hkv, 128, r.choice([16, 32, 128]), BF16, seed=seed)
    run(c, new, c.randn(sum(new), G * Hkv, 128), window, sinks, what=f"{lens} {new} {G} {Hkv} {window} {sinks}")


@pytest.mark.parametrize("dt,hd", [(BF16, 128), (BF16, 64), (F32, 64), (F32, 128)])
def test_a_window_of_everything_is_plain_prefill(cuda_lib, dt, hd):
    """The same bits where the same kernel runs; elsewhere two roundings of the same result."""
    lens, new = [700, 300, 1], [500, 1, 1]
    c = Paged(lens, 8, 2, hd, 16, dt, seed=1)
    q = c.randn(502, 8, hd)
    cu = torch.tensor([0, 500, 501, 502], dtype=torch.int32, device="cuda")
    full = torch.zeros_like(q)
    pa.pa_prefill_varlen(c.desc, q, cu, 3, 500, 502, c.k, c.v, c.bt, c.maxp, c.ctx, 700, 0.1, full)
    for window, sinks in ((700, 0), (1 << 30, 1 << 30), ((1 << 31) - 1, 5), ((1 << 31) - 1, (1 << 31) - 1), (300, 400)):
        out = prefill(c, new, q, window, sinks, 0.1, False)
        if (dt, hd) == (BF16, 128):
            assert torch.equal(out.view(torch.uint8), full.view(torch.uint8))
        compare(c, new, q, out, window, sinks, 0.1)
    # longer than the longest context, shorter than the bound that is given for it: the windowed kernel
    out = torch.zeros_like(q)
    pa.pa_prefill_varlen_window(c.desc, 701, 0, q, cu, 3, 500, 502, c.k, c.v, c.bt, c.maxp, c.ctx, c.maxp * 16, 0.1,
                                out)
    if (dt, hd) == (BF16, 128):
        assert torch.equal(out.view(torch.uint8), full.view(torch.uint8))
    compare(c, new, q, out, 701, 0, 0.1)


@pytest.mark.parametrize("dt,hd", [(BF16, 64), (F32, 64), (F32, 128)])
def test_bad_pages_of_the_other_types_are_left_out(cuda_lib, dt, hd):
    lens, new, window, sinks = [300, 300], [64, 64], 100, 4
    c = Paged(lens, 4, 2, hd, 16, dt, seed=1)
    q = c.randn(128, 4, hd)
    c.bt[0, 5] = 1 << 30   # between the sinks and the window: not looked at
    out = prefill(c, new, q, window, sinks, 0.1, True)
    compare(c, new, q, out, window, sinks, 0.1)
    assert pa.pa_read_device_errors(reset=True) == 0
    c.bt[1, 15] = -3       # in the window of some rows: keys 240 to 255 are left out
    out = prefill(c, new, q, window, sinks, 0.1, True)
    assert pa.pa_read_device_errors(reset=True) == pa.PA_DEVERR_BAD_PAGE
    p, j = torch.arange(236, 300, device="cuda")[:, None], torch.arange(300, device="cuda")
    seen = (j <= p) & ((j > p - window) | (j < sinks)) & ~((j >= 240) & (j < 256))
    o, bound = attend(q[64:], c.K[1], c.V[1], seen, 0.1, dt)
    check(out[64:], o, bound)


def test_bad_pages(cuda_lib):
    lens, new, window, sinks = [900, 900], [64, 64], 200, 4
    c = Paged(lens, 4, 2, 128, 16, BF16, seed=1)
    q = c.randn(128, 4, 128)
    c.bt[0, 20] = 1 << 30  # between the sinks and the window: not looked at
    out = prefill(c, new, q, window, sinks, 0.1, True)
    compare(c, new, q, out, window, sinks, 0.1)
    assert pa.pa_read_device_errors(reset=True) == 0
    c.bt[1, 50] = -3       # in the window: rows of zeros
    c.K[1][800:816], c.V[1][800:816] = 0, 0
    for plan in (False, True):
        out = prefill(c, new, q, window, sinks, 0.1, plan)
        compare(c, new, q, out, window, sinks, 0.1)
        assert pa.pa_read_device_errors(reset=True) == pa.PA_DEVERR_BAD_PAGE


def test_graph_and_stream(cuda_lib):
    lens, new, window, sinks = [900, 400], [300, 64], 128, 4
    c = Paged(lens, 8, 4, 128, 16, BF16, seed=2)
    q = c.randn(364, 8, 128)
    cu = torch.tensor([0, 300, 364], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, NAN)
    ws = torch.empty(pa.pa_prefill_workspace_size(c.desc, 2, 300, 364, 1000), dtype=torch.uint8, device="cuda")
    args = (c.desc, window, sinks, q, cu, 2, 300, 364, c.k, c.v, c.bt, c.maxp, c.ctx, 900, 0.1, out, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pa.pa_prefill_varlen_window(*args, stream=side)
    side.synchronize()
    compare(c, new, q, out, window, sinks, 0.1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_prefill_varlen_window(*args)
    out.fill_(NAN)
    c.lens, new = [650, 70], [290, 60]
    c.ctx.copy_(torch.tensor(c.lens, dtype=torch.int32))
    cu.copy_(torch.tensor([0, 290, 350], dtype=torch.int32))
    c.K, c.V = [[x[:L] for x, L in zip(y, c.lens)] for y in (c.K, c.V)]
    graph.replay()
    torch.cuda.synchronize()
    compare(c, new, q, out, window, sinks, 0.1)
    assert torch.isnan(out[350:].float()).all()
    assert pa.pa_read_device_errors(reset=True) == 0


@pytest.mark.parametrize("B,new,Hq,Hkv", [(24, 1300, 10, 2), (90, 2300, 16, 8), (300, 70, 8, 8)])
def test_many_blocks_without_rows(cuda_lib, B, new, Hq, Hkv):
    """A few long chunks between requests of one token: most of a grid has no rows, the rest fills several waves of
    CTAs, with and without a plan, on two streams at once and replayed."""
    r = random.Random(B)
    news = [new if b % 11 == 3 else r.choice([1, 1, 2, 40]) for b in range(B)]
    lens = [n + r.randint(0, 400) for n in news]
    lens[5] = 0
    c = Paged(lens, Hq, Hkv, 128, 16, BF16, seed=B)
    q = c.randn(sum(news), Hq, 128)
    run(c, news, q, 90, 5)
    want = prefill(c, news, q, 90, 5, 0.088, False)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(prefill(c, news, q, 90, 5, 0.088, False))
    torch.cuda.synchronize()
    cu = torch.tensor([0] + list(torch.tensor(news).cumsum(0)), dtype=torch.int32, device="cuda")
    out = torch.full_like(q, NAN)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_prefill_varlen_window(c.desc, 90, 5, q, cu, B, max(news), sum(news), c.k, c.v, c.bt, c.maxp, c.ctx,
                                    max(lens), 0.088, out)
    for _ in range(3):
        out.fill_(NAN)
        g.replay()
        torch.cuda.synchronize()
        outs.append(out.clone())
    for o in outs:
        assert torch.equal(o.view(torch.uint8), want.view(torch.uint8))
    assert pa.pa_read_device_errors(reset=True) == 0
