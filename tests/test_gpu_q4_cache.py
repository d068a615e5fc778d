"""Quantised writes and the read-back of a 4-bit cache on the GPU: rows byte for
byte against the oracle's, over types, head sets, group sizes, strides, skipped
and bad slots, and values at the edges of the format."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_08_gb300 as pa
from oracle import q4_cache as q4

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda_lib")]

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
FILL = 0xA5


def rows_of(n, hkv, hd, dtype, seed, spread=True):
    """K or V rows in the storage type: magnitudes from 1e-6 to 1e4 over the rows, some dims offset."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, hkv, hd, generator=g)
    if spread:
        x = x * torch.exp(torch.rand(n, hkv, 1, generator=g) * 23 - 14) + torch.randn(hkv, hd, generator=g) * 0.5
    return x.to(DT[dtype])


def stored(n, slots, x, num_slots, gs):
    """The oracle's cache after writing x into slots, over FILL bytes."""
    hkv, hd = x.shape[1:]
    cache = np.full((num_slots, q4.row_bytes(hkv, hd, gs)), FILL, np.uint8)
    live = slots >= 0
    u, s, c = q4.quantise(x.float().numpy()[live], gs)
    cache[slots[live]] = q4.pack_rows(u, s, c, slots[live])
    return cache


def blank_padding(cache, hkv, hd, gs):
    """The bytes of a row that hold nothing (parameters padded to 16 bytes), as FILL: their places do not move
    (parts of 16 bytes are not swizzled)."""
    used = hkv * hd // 2 + hkv * (hd // gs) * 4
    cache = cache.copy()
    cache[:, used:] = FILL
    return cache


SHAPES = [(8, 128, 32), (8, 128, 64), (8, 128, 128), (4, 128, 32), (2, 128, 64), (1, 128, 128), (1, 128, 32),
          (8, 64, 32), (4, 64, 64), (2, 64, 32), (1, 64, 64), (1, 64, 32)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hkv,hd,gs", SHAPES)
def test_written_rows_equal_the_oracles_byte_for_byte(dtype, hkv, hd, gs):
    n, pages, P = 45, 6, 16
    desc = pa.cache_desc(hkv, hkv, hd, P, pages, DT[dtype])
    k, v = rows_of(n, hkv, hd, dtype, 1), rows_of(n, hkv, hd, dtype, 2)
    slots = np.random.default_rng(3).permutation(pages * P)[:n].astype(np.int64)
    slots[[4, 17]] = -1
    R = pa.pa_q4_row_bytes(desc, gs)
    kc = torch.full((pages * P, R), FILL, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    # rows as views into a wider projection: two strides
    E = 16 // DT[dtype].itemsize
    wide = torch.zeros(n, 2 * hkv * hd + 3 * E, dtype=DT[dtype], device="cuda")
    wide[:, E: E + hkv * hd] = k.reshape(n, -1).cuda()
    vrow = v.reshape(n, -1).cuda().contiguous()
    pa.pa_kv_write_q4(desc, gs, wide[:, E:], wide.stride(0), vrow, hkv * hd, n, torch.from_numpy(slots).cuda(), kc, vc)
    torch.cuda.synchronize()
    for got, x in ((kc, k), (vc, v)):
        want = stored(n, slots, x, pages * P, gs)
        assert np.array_equal(blank_padding(got.cpu().numpy(), hkv, hd, gs), blank_padding(want, hkv, hd, gs))
    assert pa.pa_read_device_errors(reset=True) == 0


def test_many_tokens_written_by_one_call():
    """More tokens than one pass of the grid takes, the last warp's rows ragged."""
    hkv, hd, gs, P, n = 2, 64, 32, 64, 20001
    pages = n // P + 2
    desc = pa.cache_desc(hkv, hkv, hd, P, pages, torch.bfloat16)
    k = rows_of(n, hkv, hd, "bf16", 4)
    slots = np.random.default_rng(3).permutation(pages * P)[:n].astype(np.int64)
    kc = torch.full((pages * P, pa.pa_q4_row_bytes(desc, gs)), FILL, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    rows = k.reshape(n, -1).cuda()
    pa.pa_kv_write_q4(desc, gs, rows, hkv * hd, rows, hkv * hd, n, torch.from_numpy(slots).cuda(), kc, vc)
    torch.cuda.synchronize()
    want = stored(n, slots, k, pages * P, gs)
    assert np.array_equal(kc.cpu().numpy(), want) and torch.equal(kc, vc)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_edges_of_the_format(dtype):
    """Constants, zeros, NaN, infinities, values past the clamp, subnormals, ties between two codes."""
    hkv, hd, gs, P = 2, 128, 32, 16
    x = torch.zeros(8, hkv, hd)
    x[0] = 3.25
    x[1, 0, 7], x[1, 1, 40] = float("nan"), float("inf")
    x[2, 0, :32] = torch.linspace(-3e4, 3e4, 32)
    x[2, 1, 5], x[2, 1, 6] = 1e30, -1e30
    x[3] = torch.randn(hkv, hd, generator=torch.Generator().manual_seed(1)) * 1e-7
    x[4] = torch.arange(hd) % 32 * 0.5            # (x - c) / s falls between two codes
    x[5] = torch.arange(hd) % 16 - 7.5
    x[6] = -0.0
    x[7] = torch.randn(hkv, hd, generator=torch.Generator().manual_seed(2)) * 100 + 1000
    x = x.to(DT[dtype])
    desc = pa.cache_desc(hkv, hkv, hd, P, 1, DT[dtype])
    slots = np.arange(8, dtype=np.int64) + 3
    kc = torch.full((P, pa.pa_q4_row_bytes(desc, gs)), FILL, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    rows = x.reshape(8, -1).cuda()
    pa.pa_kv_write_q4(desc, gs, rows, hkv * hd, rows, hkv * hd, 8, torch.from_numpy(slots).cuda(), kc, vc)
    torch.cuda.synchronize()
    want = stored(8, slots, x, P, gs)
    w = [q4.unpack_rows(want[slots], slots, hkv, hd, gs), q4.unpack_rows(kc.cpu().numpy()[slots], slots, hkv, hd, gs)]
    assert np.array_equal(w[0][0], w[1][0])
    for i in (1, 2):  # parameters by value: any NaN is a NaN
        assert np.array_equal(w[0][i], w[1][i], equal_nan=True)
    assert torch.equal(kc, vc)


def test_bad_slots_are_skipped_and_flagged():
    hkv, hd, gs, P, pages = 8, 128, 64, 16, 2
    desc = pa.cache_desc(hkv, hkv, hd, P, pages, torch.bfloat16)
    k = rows_of(5, hkv, hd, "bf16", 7)
    slots = np.array([1, pages * P, -2, 1 << 40, 0], dtype=np.int64)
    # the caches lie inside a larger buffer: nothing around them may change
    R = pa.pa_q4_row_bytes(desc, gs)
    buf = torch.full(((pages * P + 2 * P) * R,), FILL, dtype=torch.uint8, device="cuda")
    kc = buf[P * R: (P + pages * P) * R]
    vc = torch.full((pages * P, R), FILL, dtype=torch.uint8, device="cuda")
    rows = k.reshape(5, -1).cuda()
    pa.pa_read_device_errors(reset=True)
    pa.pa_kv_write_q4(desc, gs, rows, hkv * hd, rows, hkv * hd, 5, torch.from_numpy(slots).cuda(), kc, vc)
    assert pa.pa_read_device_errors(reset=True) == pa.PA_DEVERR_BAD_SLOT
    good = np.where((slots >= 0) & (slots < pages * P), slots, -1)
    want = stored(5, good, k, pages * P, gs)
    assert np.array_equal(vc.cpu().numpy(), want)
    full = buf.cpu().numpy().reshape(-1, R)
    assert np.array_equal(full[P: P + pages * P], want)
    assert (full[:P] == FILL).all() and (full[P + pages * P:] == FILL).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,hd,gs", [(16, 8, 128, 32), (8, 8, 128, 64), (10, 2, 128, 128), (3, 1, 128, 32),
                                          (8, 4, 64, 32), (7, 1, 64, 64), (6, 2, 64, 32)])
def test_norm_rope_write_quantises_the_rows_of_the_plain_formula(dtype, hq, hkv, hd, gs):
    """q_out is the norm and rotary evaluated operation by operation in fp32, the cache rows those that pa_kv_write_q4
    makes of k so treated, bit for bit; so is the variant that maps the slots itself."""
    n, P, pages = 37, 16, 8
    dt = DT[dtype]
    desc = pa.cache_desc(hq, hkv, hd, P, pages, dt)
    g = torch.Generator(device="cuda").manual_seed(11)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    q, k, v, wq, wk = rnd(n, hq, hd), rnd(n, hkv, hd), rnd(n, hkv, hd), 1 + 0.1 * rnd(hd), 1 + 0.1 * rnd(hd)
    ctx = torch.tensor([20, 0, 50], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 5, 8, 37], dtype=torch.int32, device="cuda")   # request 1 is padding
    bt = torch.tensor([[3, 1, 0, 0], [0, 0, 0, 0], [7, 5, 2, 4]], dtype=torch.int32, device="cuda")
    pos = torch.empty(n, dtype=torch.int32, device="cuda")
    slots = torch.empty(n, dtype=torch.int64, device="cuda")
    pa.pa_slot_mapping(desc, 3, cu, ctx, bt, 4, n, pos, slots)
    row = hkv * hd
    R = pa.pa_q4_row_bytes(desc, gs)
    blank = lambda: [torch.full((pages * P, R), FILL, dtype=torch.uint8, device="cuda") for _ in range(2)]  # noqa: E731
    # k through q's place: its rows as the call norms and rotates them
    same = pa.cache_desc(hkv, hkv, hd, P, pages, dt)
    kn = torch.zeros_like(k)
    pa.pa_qk_norm_rope_kv_write_q4(same, gs, k, row, k, row, v, row, n, pos, wk, wk, 1e-6, 1e6, slots, kn, *blank())
    want = blank()
    pa.pa_kv_write_q4(desc, gs, kn, row, v, row, n, slots, *want)
    for mapped in (False, True):
        got = blank()
        qo = torch.zeros_like(q)
        if mapped:
            p2, s2 = torch.empty_like(pos), torch.empty_like(slots)
            pa.pa_prefill_qk_norm_rope_kv_write_q4(desc, gs, q, hq * hd, k, row, v, row, n, cu, 3, ctx, bt, 4, wq, wk,
                                                   1e-6, 1e6, qo, *got, p2, s2)
            assert torch.equal(p2, pos) and torch.equal(s2, slots)
        else:
            pa.pa_qk_norm_rope_kv_write_q4(desc, gs, q, hq * hd, k, row, v, row, n, pos, wq, wk, 1e-6, 1e6, slots,
                                           qo, *got)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        check_norm_rope(qo, plain_norm_rope(q, wq, pos, 1e-6, 1e6), dtype)
    check_norm_rope(kn, plain_norm_rope(k, wk, pos, 1e-6, 1e6), dtype)
    assert int((slots >= 0).sum()) == 34
    assert pa.pa_read_device_errors(reset=True) == 0


def plain_norm_rope(x, w, pos, eps, theta):
    """RMSNorm and rotary one fp32 operation at a time: squares 32 elements apart added first, then neighbours in pairs;
    sines and cosines those of the 64-bit angle, rounded."""
    dt, hd = x.dtype, x.shape[-1]
    x = x.float()
    t = (x * x).unflatten(-1, (hd // 32, 32))
    ss = t[..., 0, :]
    for i in range(1, hd // 32):
        ss = ss + t[..., i, :]
    while ss.shape[-1] > 1:
        ss = ss[..., 0::2] + ss[..., 1::2]
    r = torch.rsqrt(ss / hd + eps)
    x = ((x * r).to(dt).float() * w.float()).to(dt).float()
    f = theta ** (-2.0 * torch.arange(hd // 2, device=x.device, dtype=torch.float64) / hd)
    ang = pos.double()[:, None, None] * f
    c, s = torch.cos(ang).float(), torch.sin(ang).float()
    a, b = x[..., : hd // 2], x[..., hd // 2:]
    return torch.cat([a * c - b * s, b * c + a * s], -1).to(dt)


def check_norm_rope(got, want, dtype):
    """Equal but for the sines and cosines that round to the other neighbour: fewer than one in a thousand, and a value
    takes one of each (the bound: 1 in 100).  Those move a value by an ulp of its pair's size: 2^-23 of it in fp32, a
    rounding border crossed in bf16 (2^-7 of the value)."""
    g, w = got.float(), want.float()
    assert (g != w).float().mean() <= 0.01
    h = w.shape[-1] // 2
    size = torch.hypot(w[..., :h], w[..., h:])
    size = torch.cat([size, size], -1)
    assert ((g - w).abs() <= size * (2.0 ** -7 if dtype == "bf16" else 2.0 ** -22)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd", [64, 128])
def test_norm_rope_write_at_far_positions(dtype, hd):
    n, heads = 600, 4
    dt = DT[dtype]
    desc = pa.cache_desc(heads, heads, hd, 16, 40, dt)
    g = torch.Generator(device="cuda").manual_seed(2)
    x, w = torch.randn(n, heads, hd, generator=g, device="cuda").to(dt), torch.ones(hd, dtype=dt, device="cuda")
    pos = torch.randint(0, 131072, (n,), generator=g, device="cuda", dtype=torch.int32)
    pos[:4] = torch.tensor([0, 1, 131071, 65536], dtype=torch.int32)
    slots = torch.arange(n, dtype=torch.int64, device="cuda")
    out, row = torch.zeros_like(x), heads * hd
    caches = [torch.zeros(40 * 16, pa.pa_q4_row_bytes(desc, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
    pa.pa_qk_norm_rope_kv_write_q4(desc, 64, x, row, x, row, x, row, n, pos, w, w, 1e-6, 1e4, slots, out, *caches)
    check_norm_rope(out, plain_norm_rope(x, w, pos, 1e-6, 1e4), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hkv,hd,gs,P", [(8, 128, 32, 16), (8, 128, 64, 64), (2, 128, 128, 16), (1, 128, 32, 32),
                                         (8, 64, 32, 16), (4, 64, 64, 16), (1, 64, 64, 128)])
def test_read_back_rounds_each_value_once_and_leaves_other_rows(dtype, hkv, hd, gs, P):
    """Ragged requests (a padding one among them), starts inside, gaps between requests, rows behind the last."""
    rng = np.random.default_rng(5)
    lens = np.array([1, 3 * P + 7, 0, P, 2 * P + 1], dtype=np.int32)
    starts = np.array([0, P - 3, 0, P - 1, 0], dtype=np.int32)
    room = np.array([4, 2 * P + 20, 3, 5, 3 * P], dtype=np.int32)   # more rows than tokens: gaps
    npg = -(-lens // P)
    pages = int(npg.sum()) + 2
    bt = np.full((5, 4), pages - 1, dtype=np.int32)
    perm = rng.permutation(pages - 1)
    at = 0
    for b in range(5):
        bt[b, : npg[b]] = perm[at: at + npg[b]]
        at += npg[b]
    R = q4.row_bytes(hkv, hd, gs)
    caches, vals = [], []
    for seed in (1, 2):
        cache = rng.integers(0, 256, (pages * P, R)).astype(np.uint8)   # codes and parameters of every kind
        x = rows_of(pages * P, hkv, hd, "f32", seed, spread=seed == 1).numpy()
        slots = np.arange(pages * P)
        keep = np.isin(slots // P, perm[:at])
        cache[keep] = q4.pack_rows(*q4.quantise(x, gs), slots)[keep]
        caches.append(cache)
        vals.append(q4.row_values(cache, slots, hkv, hd, gs))
    cu = np.concatenate([[0], np.cumsum(room)]).astype(np.int32)
    rows = int(cu[-1]) + 6
    desc = pa.cache_desc(hkv, hkv, hd, P, pages, DT[dtype])
    dev = [torch.from_numpy(a).cuda() for a in (cu, starts, lens, bt)]
    outs = [torch.full((rows, hkv * hd + pad), 7.0, dtype=DT[dtype], device="cuda") for pad in (0, 8)]
    pa.pa_kv_read_q4(desc, gs, 5, dev[0], dev[1], dev[2], dev[3], 4, rows, *(torch.from_numpy(c).cuda() for c in caches),
                     outs[0], outs[0].stride(0), outs[1], outs[1].stride(0))
    torch.cuda.synchronize()
    for out, v in zip(outs, vals):
        want = torch.full((rows, hkv * hd), 7.0, dtype=DT[dtype])
        for b in range(5):
            for j in range(min(room[b], max(0, lens[b] - starts[b]))):
                p = starts[b] + j
                want[cu[b] + j] = torch.from_numpy(v[bt[b, p // P] * P + p % P].reshape(-1)).float().to(DT[dtype])
        assert torch.equal(out[:, : hkv * hd].cpu(), want)
        assert (out[:, hkv * hd:] == 7.0).all()
    assert pa.pa_read_device_errors(reset=True) == 0


def test_read_back_flags_bad_metadata():
    hkv, hd, gs, P, pages = 2, 128, 32, 16, 4
    desc = pa.cache_desc(hkv, hkv, hd, P, pages, torch.float32)
    kc = torch.zeros(pages * P, pa.pa_q4_row_bytes(desc, gs), dtype=torch.uint8, device="cuda")

    def read(cu, starts, lens, bt):
        out = torch.full((40, hkv * hd), 7.0, device="cuda")
        t = [torch.tensor(a, dtype=torch.int32, device="cuda") for a in (cu, starts, lens, bt)]
        pa.pa_kv_read_q4(desc, gs, len(lens), *t, 2, 40, kc, kc, out, hkv * hd, out.clone(), hkv * hd)
        flags = pa.pa_read_device_errors(reset=True)
        return flags, (out != 7.0).any(1).cpu().numpy()

    pa.pa_read_device_errors(reset=True)
    flags, wrote = read([0, 20, 40], [0, 0], [20, 20], [[0, 9], [2, -1]])   # second pages out of range
    assert flags == pa.PA_DEVERR_BAD_PAGE and wrote.sum() == 32
    flags, wrote = read([0, 20, 40], [-1, 0], [20, 33], [[0, 1], [2, 3]])   # a negative start, a length past the table
    assert flags == pa.PA_DEVERR_BAD_LENGTH and not wrote.any()
    flags, wrote = read([0, 20, 40], [30, 0], [20, -5], [[0, 1], [2, 3]])   # nothing left to read; a negative length
    assert flags == pa.PA_DEVERR_BAD_LENGTH and not wrote.any()
    flags, wrote = read([5, 20, 10], [0, 0], [20, 20], [[0, 1], [2, 3]])    # decreasing, rows before the first
    assert flags == pa.PA_DEVERR_BAD_LENGTH
