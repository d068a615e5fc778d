"""Decode for groups of requests that share a prefix, against plain attention in 64 bits over each request's keys."""
import random

import pytest
import torch

import paged_kv_gqa_08_gb300 as pa
from range_reference import Paged, attend, check

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


class Groups(Paged):
    """Requests of `groups` = [(prefix, [own tokens, ...]), ...] (None: a padding row), the prefix's whole pages
    shared, its last tokens copied; what the calls may not look at is left out or poisoned."""

    def __init__(self, groups, Hq, Hkv, hd, P, dt, seed, wide=False):
        lens = [0 if o is None else pre + o for pre, own in groups for o in own]
        super().__init__(lens, Hq, Hkv, hd, P, dt, seed)
        self.groups = groups
        if wide:  # tables, and so bounds, of a million tokens and more: the kernel over the prefixes, whatever is shared
            self.bt = torch.nn.functional.pad(self.bt, (0, 65536 - self.maxp), value=-1)
            self.maxp = 65536
        self.wide = wide
        self.cu = torch.tensor([0] + list(torch.tensor([len(o) for _, o in groups]).cumsum(0)), dtype=torch.int32,
                               device="cuda")
        self.pre = torch.tensor([p for p, _ in groups], dtype=torch.int32, device="cuda")
        b = 0
        for pre, own in groups:
            first = None
            for o in own:
                if o is not None:
                    if first is None:
                        first = b
                    else:
                        self.K[b][:pre], self.V[b][:pre] = self.K[first][:pre], self.V[first][:pre]
                        bad = torch.full_like(self.K[b][:pre], NAN)
                        if pre:  # the others' own copies of the prefix are not read, their entries not looked at
                            self.put(b, torch.arange(pre, device="cuda"), bad, bad)
                            self.bt[b, : pre // P] = 1 << 29
                b += 1

    def call(self, q, scale, max_ctas=0, out=None, max_ctx=None, max_pre=None):
        B, ng = len(self.lens), len(self.groups)
        mx = max_ctx or (65536 * self.P if self.wide else max(max(self.lens), 1))
        mp = max_pre if max_pre is not None else mx if self.wide else int(self.pre.max())
        nbytes = pa.pa_decode_shared_prefix_workspace_size(self.desc, ng, B, mp, mx, max_ctas)
        assert nbytes > 0
        ws = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
        out = torch.full_like(q, NAN) if out is None else out
        pa.pa_decode_shared_prefix(self.desc, ng, self.cu, self.pre, mp, q, B, self.k, self.v, self.bt, self.maxp,
                                   self.ctx, mx, scale, max_ctas, out, ws)
        return out

    def compare(self, q, out, scale, what=""):
        for b, L in enumerate(self.lens):
            if L <= 0:
                assert torch.isnan(out[b].float()).all()
                continue
            seen = torch.ones(1, L, dtype=torch.bool, device="cuda")
            o, bound = attend(q[b: b + 1], self.K[b], self.V[b], seen, scale, self.dt)
            # parts of up to 152 CTAs are merged: their rounding is within the bound's sums
            check(out[b: b + 1], o, bound, f"{what} request {b} of {L}")


HEADS = [(BF16, 16, 8, 128), (BF16, 1, 1, 128), (BF16, 6, 2, 128), (BF16, 28, 4, 128), (BF16, 40, 8, 128),
         (BF16, 8, 1, 128), (BF16, 10, 2, 64), (BF16, 24, 8, 64), (F32, 4, 2, 64), (F32, 12, 2, 128), (F32, 56, 8, 64)]
GROUPS = {
    "one": [(128, [1, 5, 70, 0, 33])],
    "alone": [(300, [17])],
    "none shared": [(0, [1, 50, None, 300])],
    "short": [(1, [1, 2, 3]), (15, [0, 16])],
    "ragged": [(129, [1] * 7), (1000, [3, None, 40, 200]), (0, [9, 90]), (17, [1, 1]), (640, [None, None]),
               (500, [None, 5, 0])],
    "many": [(700, [(7 * i) % 50 for i in range(150)]), (260, [(5 * i) % 33 for i in range(70)])],
}


@pytest.mark.parametrize("dt,Hq,Hkv,hd", HEADS)
@pytest.mark.parametrize("name", GROUPS)
@pytest.mark.parametrize("wide", [False, True])
def test_against_plain(cuda_lib, dt, Hq, Hkv, hd, name, wide):
    c = Groups(GROUPS[name], Hq, Hkv, hd, 16 if name != "ragged" else 64, dt, Hq, wide)
    q = c.randn(len(c.lens), Hq, hd)
    for max_ctas in (0, 1, 5):
        out = c.call(q, hd ** -0.5, max_ctas)
        c.compare(q, out, hd ** -0.5, f"{max_ctas} CTAs")
    assert pa.pa_read_device_errors(reset=True) == 0


@pytest.mark.parametrize("dt,Hq,Hkv,hd", [(BF16, 32, 8, 128), (BF16, 7, 1, 128), (F32, 8, 2, 64), (BF16, 16, 8, 64)])
def test_long_prefix(cuda_lib, dt, Hq, Hkv, hd):
    """A prefix cut over all CTAs, for few rows and for several units of rows."""
    for own in ([40, 1, 700], [(11 * i) % 90 for i in range(90)]):
        c = Groups([(20011, own)], Hq, Hkv, hd, 16, dt, seed=len(own))
        q = c.randn(len(own), Hq, hd)
        c.compare(q, c.call(q, 0.1), 0.1)
    assert pa.pa_read_device_errors(reset=True) == 0


@pytest.mark.parametrize("dt,hd", [(BF16, 128), (F32, 64)])
@pytest.mark.parametrize("wide", [False, True])
def test_batches_planned_before_the_kernel(cuda_lib, dt, hd, wide):
    groups = [(64 + i % 100, [(i * k) % 40 for k in range(1, 9)]) for i in range(70)]
    c = Groups(groups, 4, 2, hd, 16, dt, 1, wide)
    assert len(c.lens) > 512
    q = c.randn(len(c.lens), 4, hd)
    c.compare(q, c.call(q, 0.1), 0.1)
    assert pa.pa_read_device_errors(reset=True) == 0


@pytest.mark.parametrize("seed", range(10))
@pytest.mark.parametrize("wide", [False, True])
def test_random_groups(cuda_lib, seed, wide):
    r = random.Random(seed)
    groups = []
    for _ in range(r.randint(1, 12)):
        own = [None if r.random() < 0.1 else r.randint(0, 300) for _ in range(r.randint(1, 40))]
        pre = r.choice([0, 1, 127, 128, 129, int(2 ** r.uniform(0, 12))])
        groups.append((pre, [1 if o == 0 and pre == 0 else o for o in own]))
    G, Hkv = r.randint(1, 8), r.choice([1, 2, 4, 8])
    c = Groups(groups, G * Hkv, Hkv, 128, r.choice([16, 64, 256]), BF16, seed, wide)
    q = c.randn(len(c.lens), G * Hkv, 128)
    c.compare(q, c.call(q, 0.1, r.choice([0, 0, 7])), 0.1, f"{groups} {G} {Hkv}")
    assert pa.pa_read_device_errors(reset=True) == 0


@pytest.mark.parametrize("dt,hd", [(BF16, 128), (BF16, 64), (F32, 128)])
def test_no_groups_is_plain_decode(cuda_lib, dt, hd):
    c = Paged([300, 17, 0, 2000], 8, 2, hd, 16, dt, seed=1)
    q = c.randn(4, 8, hd)
    full, out = torch.full_like(q, NAN), torch.full_like(q, NAN)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    pa.pa_decode(c.desc, q, 4, c.k, c.v, c.bt, c.maxp, c.ctx, 2000, 0.1, 0, full, ws)
    pa.pa_decode_shared_prefix(c.desc, 0, None, None, 0, q, 4, c.k, c.v, c.bt, c.maxp, c.ctx, 2000, 0.1, 0, out, ws)
    assert torch.equal(out.view(torch.uint8), full.view(torch.uint8))
    # requests behind the last group, and groups without a prefix, alike
    cu = torch.tensor([0, 0, 2], dtype=torch.int32, device="cuda")
    pre = torch.tensor([100, 0], dtype=torch.int32, device="cuda")
    out.fill_(NAN)
    pa.pa_decode_shared_prefix(c.desc, 2, cu, pre, 100, q, 4, c.k, c.v, c.bt, c.maxp, c.ctx, 2000, 0.1, 0, out, ws)
    for b in (0, 1, 3):
        o, bound = attend(q[b: b + 1], c.K[b], c.V[b], torch.ones(1, c.lens[b], dtype=torch.bool, device="cuda"), 0.1,
                          dt)
        check(out[b: b + 1], o, bound)
    assert torch.isnan(out[2].float()).all()
    assert pa.pa_read_device_errors(reset=True) == 0


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dt,hd", [(BF16, 128), (BF16, 64), (F32, 128)])
def test_bad_lengths_and_pages(cuda_lib, dt, hd, wide):
    c = Groups([(256, [4, 40, 8]), (64, [9, 9])], 4, 2, hd, 16, dt, 1, wide)
    q = c.randn(5, 4, hd)
    c.ctx[1] = 255                      # shorter than its group's prefix
    out = c.call(q, 0.1, out=torch.full_like(q, 3.0))
    assert pa.pa_read_device_errors(reset=True) == pa.PA_DEVERR_BAD_LENGTH
    assert (out[1] == 3.0).all()
    c.lens[1] = -1
    out[1] = NAN
    c.compare(q, out, 0.1)
    c.lens[1], c.ctx[1] = 296, 296
    for bad in (-1, 1 << 30):               # out of range: the group's requests are skipped
        c.pre[1] = bad
        out = c.call(q, 0.1, out=torch.full_like(q, 3.0), max_pre=None if wide else 256)
        assert pa.pa_read_device_errors(reset=True) == pa.PA_DEVERR_BAD_LENGTH
        assert (out[3:] == 3.0).all()
        keep, c.lens[3], c.lens[4] = c.lens[3:], -1, -1
        out[3:] = NAN
        c.compare(q, out, 0.1)
        c.lens[3:] = keep
    c.pre[1] = 64
    c.bt[0, 3] = c.num_pages            # a page of the first group's prefix
    out = c.call(q, 0.1)
    assert pa.pa_read_device_errors(reset=True) == pa.PA_DEVERR_BAD_PAGE
    for b in range(5):
        seen = torch.ones(1, c.lens[b], dtype=torch.bool, device="cuda")
        if b < 3 and wide and (dt, hd) == (BF16, 128):
            c.K[b][48:64], c.V[b][48:64] = 0, 0
        elif b < 3:                     # the other kernels leave its keys out
            seen[:, 48:64] = False
        o, bound = attend(q[b: b + 1], c.K[b], c.V[b], seen, 0.1, dt)
        check(out[b: b + 1], o, bound, f"request {b}")


@pytest.mark.parametrize("wide", [False, True])
def test_graph_and_stream(cuda_lib, wide):
    c = Groups([(500, [30, 20, 10]), (100, [200, 300])], 8, 4, 128, 16, BF16, 2, wide)
    most = 65536 * 16 if wide else 530
    q = c.randn(5, 8, 128)
    out = torch.full_like(q, NAN)
    ws = torch.empty(pa.pa_decode_shared_prefix_workspace_size(c.desc, 2, 5, most, most), dtype=torch.uint8,
                     device="cuda")
    args = (c.desc, 2, c.cu, c.pre, most, q, 5, c.k, c.v, c.bt, c.maxp, c.ctx, most, 0.1, 0, out, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pa.pa_decode_shared_prefix(*args, stream=side)
    side.synchronize()
    c.compare(q, out, 0.1)
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_decode_shared_prefix(*args)
    with torch.cuda.graph(other):       # on the same workspace
        pa.pa_decode_shared_prefix(*args)
    c.lens = [525, 0, 505, 100, 333]
    c.ctx.copy_(torch.tensor(c.lens, dtype=torch.int32))
    c.K, c.V = [[x[:L] for x, L in zip(y, c.lens)] for y in (c.K, c.V)]
    for g in (graph, other, graph):
        out.fill_(NAN)
        g.replay()
        torch.cuda.synchronize()
        c.compare(q, out, 0.1)
    assert pa.pa_read_device_errors(reset=True) == 0


def test_the_same_bits_every_time(cuda_lib):
    c = Groups([(3000, [(13 * i) % 70 for i in range(40)]), (900, [7, 8, 9])], 32, 8, 128, 16, BF16, seed=3)
    q = c.randn(43, 32, 128)
    first = c.call(q, 0.1)
    for _ in range(20):
        assert torch.equal(c.call(q, 0.1), first)


@pytest.mark.parametrize("dt,hd", [(BF16, 128), (F32, 64)])
def test_a_workspace_for_the_largest_bounds_serves_smaller_ones(cuda_lib, dt, hd):
    desc = pa.cache_desc(32, 8, hd, 16, 1000, dt)
    sizes = [(g, b, p, c) for g in (0, 1, 3, 8, 64) for b in (1, 2, 8, 64) for p in (0, 1, 128, 4000, 40000)
             for c in (40000, 80000) if g <= b]
    need = {k: pa.pa_decode_shared_prefix_workspace_size(desc, *k) for k in sizes}
    for k in sizes:
        assert 0 < need[k] <= need[(64, 64, 40000, 80000)]
        assert all(need[k] <= need[m] for m in sizes if all(x <= y for x, y in zip(k, m)))
    for window, sinks in ((1, 0), (15, 1), (99, 0), (98, 1), (64, 30)):  # at most that of plain decode
        for b in (1, 3, 100):
            for mx in (1, 17, 100, 5000):
                assert (pa.pa_decode_window_workspace_size(desc, window, sinks, b, mx) <=
                        pa.pa_decode_workspace_size(desc, b, mx))
