"""Windowed prefill and shared prefixes in tiles of rows (fp32; bf16 of 64 dims), where a window's start meets a key
tile's at every row of a tile: plain attention in 64 bits, and the same bits in every run."""
import pytest
import torch

import paged_kv_gqa_08_gb300 as pa
from range_reference import Paged, attend, check
from test_gpu_shared_prefix import Groups
from test_gpu_window_prefill import prefill

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
TYPES = [(F32, 64), (F32, 128), (BF16, 64)]


def rows_seen(L, n, window, sinks):
    p, j = torch.arange(L - n, L, device="cuda")[:, None], torch.arange(L, device="cuda")
    return (j <= p) & ((j > p - window) | (j < sinks))


@pytest.mark.parametrize("dt,hd", TYPES)
@pytest.mark.parametrize("G", range(1, 9))
@pytest.mark.parametrize("sinks", [0, 4])
def test_every_row_and_window_start(cuda_lib, dt, hd, G, sinks):
    """Chunks of 1 to 40 tokens, over 64 windows in a row: each row's window starts on every key of a tile."""
    new = list(range(1, 41))
    lens = [130 + n + 7 * n % 64 for n in new]
    c = Paged(lens, G, 1, hd, 16, dt, seed=10 * G + sinks)
    q = c.randn(sum(new), G, hd)
    windows = range(65, 129)
    outs = torch.stack([prefill(c, new, q, w, sinks, 0.088, False) for w in windows])
    at = 0
    for b, (L, n) in enumerate(zip(lens, new)):
        seen = torch.cat([rows_seen(L, n, w, sinks) for w in windows])
        o, bound = attend(q[at: at + n].repeat(len(windows), 1, 1), c.K[b], c.V[b], seen, 0.088, dt)
        check(outs[:, at: at + n].reshape(o.shape), o, bound, f"{n} tokens of {L}")
        at += n
    assert pa.pa_read_device_errors(reset=True) == 0


@pytest.mark.parametrize("dt,hd", TYPES)
@pytest.mark.parametrize("G,L,n,window,sinks", [
    (7, 200, 200, 101, 0), (1, 303, 4, 300, 0), (2, 131, 2, 66, 4), (7, 200, 200, 65, 0), (2, 165, 9, 100, 4),
    (4, 130, 13, 128, 0), (3, 300, 234, 105, 1), (5, 411, 394, 90, 1), (6, 160, 9, 95, 1), (8, 200, 200, 65, 0)])
def test_a_window_that_starts_with_a_tile(cuda_lib, dt, hd, G, L, n, window, sinks):
    """A tile's first key is the first that a row has lost, and that row the first of the next warp's."""
    c = Paged([L], 2 * G, 2, hd, 16, dt, seed=L)
    q = c.randn(n, 2 * G, hd)
    o, bound = attend(q, c.K[0], c.V[0], rows_seen(L, n, window, sinks), 0.088, dt)
    outs = [prefill(c, [n], q, window, sinks, 0.088, False) for _ in range(10)]
    for out in outs:
        check(out, o, bound)
        assert torch.equal(out.view(torch.uint8), outs[0].view(torch.uint8))
    assert pa.pa_read_device_errors(reset=True) == 0


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows", range(1, 9))
def test_prefixes_of_few_rows_repeat(cuda_lib, hd, rows):
    """A group of 1 to 8 rows a kv-head (requests of one q-head; one request of a group of q-heads)."""
    for own, G in (([5] * rows, 1), ([5], rows)):
        c = Groups([(5000, own)], 2 * G, 2, hd, 16, F32, rows, True)
        q = c.randn(len(own), 2 * G, hd)
        outs = [c.call(q, 0.1) for _ in range(5)]
        c.compare(q, outs[0], 0.1)
        for out in outs:
            assert torch.equal(out, outs[0])
    assert pa.pa_read_device_errors(reset=True) == 0
