"""Caches of more than 2^32 bytes: the requests' pages lie at their end."""
import pytest
import torch

import paged_kv_gqa_08_gb300 as pa
from range_reference import attend, check

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dt,hd", [(BF16, 128), (BF16, 64), (F32, 128)])
def test_pages_past_32_bits(cuda_lib, dt, hd):
    P, Hkv, Hq, window, sinks = 16, 8, 16, 70, 5
    row = Hkv * hd * (2 if dt == BF16 else 4)
    pages = (1 << 32) // (row * P) + 5000
    desc = pa.cache_desc(Hq, Hkv, hd, P, pages, dt)
    kc, vc = (torch.empty(pages, P, Hkv, hd, dtype=dt, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    lens, maxp = [333, 40, 200], 64
    bt = pages - 1 - torch.randperm(4000, generator=g, device="cuda")[: 3 * maxp].view(3, maxp).to(torch.int32)
    bt[1, :2], bt[2, :2] = bt[0, :2], bt[0, :2]           # 32 tokens that all share
    K, V = [rand(L, Hkv, hd) for L in lens], [rand(L, Hkv, hd) for L in lens]
    for b in (1, 2):
        K[b][:32], V[b][:32] = K[0][:32], V[0][:32]
    for b, L in enumerate(lens):
        j = torch.arange(L, device="cuda")
        kc[bt[b][j // P].long(), j % P], vc[bt[b][j // P].long(), j % P] = K[b], V[b]
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(512 << 20, dtype=torch.uint8, device="cuda")
    q, scale = rand(3, Hq, hd), 0.1

    def same(out, rows, seen_of):
        for b, L in enumerate(lens):
            n = rows[b]
            p, j = torch.arange(L - n, L, device="cuda")[:, None], torch.arange(L, device="cuda")
            at = sum(rows[:b])
            o, bound = attend(qs[at: at + n], K[b], V[b], seen_of(p, j), scale, dt)
            check(out[at: at + n], o, bound)

    win = lambda p, j: (j <= p) & ((j > p - window) | (j < sinks))  # noqa: E731
    full = lambda p, j: j <= p  # noqa: E731
    qs, out = q, torch.zeros_like(q)
    pa.pa_decode_window(desc, window, sinks, q, 3, kc, vc, bt, maxp, ctx, 333, scale, 0, out, ws)
    same(out, [1, 1, 1], win)
    groups = (torch.tensor([0, 3], dtype=torch.int32, device="cuda"), torch.tensor([32], dtype=torch.int32, device="cuda"))
    for bound_len in (32, 333):
        out.zero_()
        pa.pa_decode_shared_prefix(desc, 1, *groups, bound_len, q, 3, kc, vc, bt, maxp, ctx, 333, scale, 0, out, ws)
        same(out, [1, 1, 1], full)
    # the kernel over the prefixes: tables (and so bounds) of a million tokens
    wide = torch.full((3, 65536), -1, dtype=torch.int32, device="cuda")
    wide[:, :maxp] = bt
    out.zero_()
    pa.pa_decode_shared_prefix(desc, 1, *groups, 1 << 20, q, 3, kc, vc, wide, 65536, ctx, 1 << 20, scale, 0, out, ws)
    same(out, [1, 1, 1], full)
    new = [60, 40, 1]
    qs = rand(sum(new), Hq, hd)
    out = torch.zeros_like(qs)
    cu = torch.tensor([0, 60, 100, 101], dtype=torch.int32, device="cuda")
    for w in (None, ws):
        out.zero_()
        pa.pa_prefill_varlen_window(desc, window, sinks, qs, cu, 3, 60, 101, kc, vc, bt, maxp, ctx, 333, scale, out, w)
        same(out, new, win)
    kn, vn = rand(3, Hkv * hd), rand(3, Hkv * hd)
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    qs, out = q, torch.zeros_like(q)
    pa.pa_decode_kv_write_window(desc, window, sinks, q, kn, Hkv * hd, vn, Hkv * hd, 3, kc, vc, bt, maxp, ctx, 333, scale,
                                 0, slots, out, ws)
    for b, L in enumerate(lens):
        K[b][-1], V[b][-1] = kn[b].view(Hkv, hd), vn[b].view(Hkv, hd)
        assert int(slots[b]) == int(bt[b, (L - 1) // P]) * P + (L - 1) % P
        assert torch.equal(kc.view(-1, Hkv * hd)[slots[b]], kn[b]) and torch.equal(vc.view(-1, Hkv * hd)[slots[b]], vn[b])
    same(out, [1, 1, 1], win)
    assert pa.pa_read_device_errors(reset=True) == 0


def test_lengths_near_31_bits(cuda_lib):
    """A table whose pages hold more than 2^31 tokens: lengths stop where int32 does."""
    P, maxp = 1 << 20, 4096
    desc = pa.cache_desc(4, 2, 64, P, 4096, BF16)
    i32 = dict(dtype=torch.int32, device="cuda")
    top = (1 << 31) - 1
    ctx, new = torch.tensor([top - 3, top - 3], **i32), torch.tensor([4, 3], **i32)
    bt = torch.arange(2 * maxp, **i32).view(2, maxp) % 4096
    ring, pool = torch.arange(4096, **i32), torch.tensor([0, 0], device="cuda")
    cu, pos, slots = torch.zeros(3, **i32), torch.zeros(5, **i32), torch.zeros(5, dtype=torch.int64, device="cuda")
    pa.pa_extend_tables(desc, 2, new, ctx, bt, maxp, ring, pool, 5, cu, ctx, pos, slots, None, pool)
    assert pa.pa_read_device_errors(reset=True) == pa.PA_DEVERR_BAD_LENGTH
    assert ctx.tolist() == [top - 3, top] and cu.tolist() == [0, 0, 3] and pos.tolist() == [top - 3, top - 2, top - 1, 0, 0]
    last = int(bt[1, 2047]) * P
    assert slots.tolist() == [last + P - 4, last + P - 3, last + P - 2, -1, -1]
    # the pages that a window has left at such a length
    keep = bt.clone()
    refs = torch.ones(4096, **i32)
    refs += 1
    pa.pa_release_window_pages(desc, 5, 3, 2, ctx, bt, maxp, refs, ring, pool, pool)
    assert (bt[:, 1:2047] == -1).all() and torch.equal(bt[:, 2047:], keep[:, 2047:]) and torch.equal(bt[:, 0], keep[:, 0])
    assert pa.pa_read_device_errors(reset=True) == 0
