"""Decode attention over a 4-bit cache on the GPU against the float64 oracle on
the values the rows stand for; the fused step; splits, padding, bad metadata,
graphs; prefill over the read-back."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_gqa_08_gb300 as pa
from oracle import q4_cache as q4

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda_lib")]

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


class Case:
    """A batch over a random 4-bit cache; slots no request owns hold random bytes (NaN and infinite scales among them)."""

    def __init__(self, dtype, hq, hkv, hd, gs, P, lens, seed=0, spread=0.0, vscale=1.0):
        rng = np.random.default_rng(seed)
        self.dtype, self.hq, self.hkv, self.hd, self.gs, self.P = dtype, hq, hkv, hd, gs, P
        self.lens = np.asarray(lens, dtype=np.int32)
        B = len(lens)
        npg = -(-self.lens // P)
        self.pages = int(npg.sum()) + 2
        self.maxp = max(int(npg.max()), 1)
        self.bt = np.full((B, self.maxp), self.pages - 1, dtype=np.int32)
        perm = rng.permutation(self.pages - 1)
        at, owned = 0, []
        for b in range(B):
            self.bt[b, : npg[b]] = perm[at: at + npg[b]]
            at += npg[b]
            for j in range(int(self.lens[b])):
                owned.append(self.bt[b, j // P] * P + j % P)
        owned = np.array(owned, dtype=np.int64)
        R = q4.row_bytes(hkv, hd, gs)
        self.desc = pa.cache_desc(hq, hkv, hd, P, self.pages, DT[dtype])
        self.cache, self.vals = [], []
        for scale in (1.0, vscale):
            cache = rng.integers(0, 256, (self.pages * P, R)).astype(np.uint8)
            x = rng.standard_normal((len(owned), hkv, hd)) * np.exp(spread * rng.standard_normal((len(owned), hkv, 1)))
            x = ((x + rng.standard_normal((hkv, hd)) * 0.3) * scale).astype(np.float32)
            u, s, c = q4.quantise(x, gs)
            cache[owned] = q4.pack_rows(u, s, c, owned)
            val = np.zeros((self.pages * P, hkv, hd))
            val[owned] = q4.values(u, s, c, gs)
            self.cache.append(torch.from_numpy(cache).cuda())
            self.vals.append(val)
        q = torch.from_numpy(rng.standard_normal((B, hq, hd)).astype(np.float32)).to(DT[dtype])
        self.q = q.cuda()
        self.q64 = q.double().numpy()
        self.scale = hd ** -0.5
        self.ctx = torch.from_numpy(self.lens).cuda()
        self.btd = torch.from_numpy(self.bt).cuda()
        self.max_ctx = max(int(self.lens.max()), 1)

    def reference(self):
        out = np.full((len(self.lens), self.hq, self.hd), np.nan)
        for b, L in enumerate(self.lens):
            if L < 1:
                continue
            slots = self.bt[b, np.arange(L) // self.P].astype(np.int64) * self.P + np.arange(L) % self.P
            out[b] = oracle.attend(self.q64[b: b + 1], self.vals[0][slots], self.vals[1][slots], [L - 1],
                                   self.scale)[0][0]
        return out

    def ws(self, max_ctas=0):
        n = pa.pa_decode_q4_workspace_size(self.desc, self.gs, len(self.lens), self.max_ctx, max_ctas)
        assert n > 0
        return torch.empty(n, dtype=torch.uint8, device="cuda")

    def decode(self, max_ctas=0, out=None):
        out = torch.full_like(self.q, 7.0) if out is None else out
        pa.pa_decode_q4(self.desc, self.gs, self.q, len(self.lens), *self.cache, self.btd, self.maxp, self.ctx,
                        self.max_ctx, self.scale, max_ctas, out, self.ws(max_ctas))
        return out

    def check(self, out, ref=None):
        """Tolerance.  fp32: the products and sums are fp32, so an output is off by a few 2^-24 of the values'
        magnitude per step: 1e-5 of it.  bf16: queries, values and probabilities enter the products as float16
        (2^-11 of each, the error of the scores scaled by their size of a few units) and the output is rounded to
        bf16 (2^-8 of it): 1e-2 of the largest output."""
        ref = self.reference() if ref is None else ref
        live = self.lens > 0
        got = out.double().cpu().numpy()
        assert (got[~live] == 7.0).all()
        err = np.abs(got[live] - ref[live]).max() if live.any() else 0.0
        top = np.abs(ref[live]).max() if live.any() else 1.0
        bound = 1e-5 * max(1.0, top) if self.dtype == "f32" else 1e-2 * top
        assert np.isfinite(err) and err <= bound, (err, bound)


SHAPES = [(16, 8, 128, 32, 16), (8, 8, 128, 64, 16), (24, 8, 128, 128, 32), (32, 8, 128, 32, 256), (40, 8, 128, 64, 16),
          (6, 1, 128, 32, 16), (14, 2, 128, 64, 64), (32, 4, 128, 128, 16), (64, 8, 128, 32, 16),
          (8, 8, 64, 32, 16), (4, 2, 64, 32, 16), (8, 1, 64, 64, 16), (12, 4, 64, 64, 128), (5, 1, 64, 32, 32)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,hd,gs,P", SHAPES)
def test_decode_matches_the_oracle(dtype, hq, hkv, hd, gs, P):
    c = Case(dtype, hq, hkv, hd, gs, P, [1, 2, 15, 16, 17, 0, 33, 64, 100, 257, 1001], seed=hq + hd + gs, spread=0.3)
    ref = c.reference()
    for max_ctas in (0, 1, 3, 7):
        c.check(c.decode(max_ctas), ref)
    assert pa.pa_read_device_errors(reset=True) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_contexts_split_over_the_gpu(dtype):
    c = Case(dtype, 16, 4, 128, 64, 64, [20011, 1, 9000], seed=5)
    ref = c.reference()
    for max_ctas in (0, 1, 31):
        c.check(c.decode(max_ctas), ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vscale", [1e-4, 300.0])
def test_small_and_large_values(dtype, vscale):
    c = Case(dtype, 8, 4, 128, 32, 16, [5, 300, 1111], seed=9, vscale=vscale)
    ref = c.reference()
    got = c.decode().double().cpu().numpy()
    top = np.abs(ref).max()
    assert np.abs(got - ref).max() <= (1e-5 if dtype == "f32" else 1e-2) * top


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("qscale", [1e-30, 1e-3, 40.0, 1e6])
def test_query_magnitudes(dtype, qscale):
    """Queries far outside a 16-bit float's range: uniform weights at one end, one key taking all at the other."""
    c = Case(dtype, 6, 2, 128, 64, 16, [40, 200], seed=3)
    c.q = (c.q.double() * qscale).to(DT[dtype])
    c.q64 = c.q.double().cpu().numpy()
    ref = c.reference()
    got = c.decode().double().cpu().numpy()
    if qscale <= 1.0:
        assert np.abs(got - ref).max() <= (1e-5 if dtype == "f32" else 1e-2) * max(1.0, np.abs(ref).max())
    else:
        # scores of size S carry an error of 2^-9 S (bf16) or some 2^-22 S (fp32): the weights between near keys are
        # not determined, but every output is a mean of values
        v = c.vals[1]
        assert np.isfinite(got).all() and np.abs(got).max() <= np.abs(v).max() * 1.01


def test_a_large_batch_is_planned_by_its_own_kernel():
    rng = np.random.default_rng(8)
    lens = rng.integers(1, 40, 700).astype(np.int32)
    lens[[3, 650]] = 0
    c = Case("bf16", 8, 4, 128, 32, 16, lens, seed=12)
    c.check(c.decode())
    lens = lens.copy()
    lens[5] = c.max_ctx + 1                      # longer than the bound: skipped and flagged
    c.ctx.copy_(torch.from_numpy(lens))
    c.lens = np.where(np.arange(700) == 5, 0, c.lens).astype(np.int32)
    pa.pa_read_device_errors(reset=True)
    out = torch.full_like(c.q, 7.0)
    pa.pa_decode_q4(c.desc, 32, c.q, 700, *c.cache, c.btd, c.maxp, c.ctx, c.max_ctx, c.scale, 0, out, c.ws())
    c.check(out)
    assert pa.pa_read_device_errors(reset=True) == pa.PA_DEVERR_BAD_LENGTH


def test_pages_may_lie_anywhere_and_the_output_is_the_same_bit_for_bit():
    c = Case("bf16", 16, 8, 128, 32, 16, [77, 500, 33], seed=2)
    a = c.decode()
    perm = torch.from_numpy(np.random.default_rng(1).permutation(c.pages)).cuda()
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(c.pages, device="cuda")
    R = c.cache[0].shape[1]
    c.cache = [x.reshape(c.pages, -1)[perm].reshape(-1, R).contiguous() for x in c.cache]
    c.btd = inv[c.btd.long()].to(torch.int32)
    assert torch.equal(a, c.decode())
    assert torch.equal(a, c.decode())


def test_bad_pages_are_skipped_and_flagged():
    c = Case("bf16", 8, 8, 128, 32, 16, [40, 50], seed=4)
    ref = c.reference()
    c.btd[1, 1] = c.pages
    pa.pa_read_device_errors(reset=True)
    out = c.decode()
    assert pa.pa_read_device_errors(reset=True) == pa.PA_DEVERR_BAD_PAGE
    assert torch.isfinite(out).all()
    top = np.abs(ref).max()
    assert np.abs(out[0].double().cpu().numpy() - ref[0]).max() <= 1e-2 * top


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd", [128, 64])
def test_nothing_past_a_context_reaches_the_output(dtype, hd):
    """The rest of a request's last page holds NaN and infinite scales; NaN queries of padding rows stay there."""
    c = Case(dtype, 16, 8, hd, 32, 64, [1, 33, 63, 65, 0], seed=6)
    c.q[4] = float("nan")
    for cache in c.cache:
        for b, L in enumerate(c.lens):
            for j in range(int(L), c.maxp * 64):
                page = c.bt[b, j // 64]
                if page != c.pages - 1:
                    cache[page * 64 + j % 64] = 0xFF     # codes 15, s = c = NaN
    for max_ctas in (0, 1):
        c.check(c.decode(max_ctas))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_group_that_holds_nan_makes_its_own_outputs_nan_only(dtype):
    c = Case(dtype, 4, 4, 128, 32, 16, [20, 20], seed=6)
    slot = int(c.bt[0, 0]) * 16 + 3
    row = c.cache[1][slot].cpu().numpy()
    u, s, p = q4.unpack_rows(row[None], [slot], 4, 128, 32)
    s[0, 2, 1], p[0, 2, 1] = 0, np.float16(np.nan)
    c.cache[1][slot] = torch.from_numpy(q4.pack_rows(u, s, p, [slot])[0]).cuda()
    nan = torch.isnan(c.decode()).cpu()
    want = torch.zeros_like(nan)
    want[0, 2, 32:64] = True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,hd,gs,P", [(16, 8, 128, 32, 16), (8, 2, 128, 64, 64), (7, 1, 128, 128, 16),
                                            (16, 8, 64, 64, 16), (6, 2, 64, 32, 32)])
def test_the_fused_step_equals_the_separate_calls(dtype, hq, hkv, hd, gs, P):
    c = Case(dtype, hq, hkv, hd, gs, P, [1, 16, 17, 0, 100, 300, 64, 2], seed=21)
    B, row = len(c.lens), hkv * hd
    g = torch.Generator().manual_seed(4)
    kn = torch.randn(B, row + 16, generator=g).to(DT[dtype]).cuda()
    vn = torch.randn(B, row, generator=g).to(DT[dtype]).cuda()
    vn[4, 5] = float("nan")       # a new row with a NaN: its group reads back as NaN, in both
    first = [x.clone() for x in c.cache]
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    pos = torch.empty(B, dtype=torch.int32, device="cuda")
    slots = torch.empty(B, dtype=torch.int64, device="cuda")
    pa.pa_slot_mapping(c.desc, B, cu, c.ctx, c.btd, c.maxp, B, pos, slots)
    pa.pa_kv_write_q4(c.desc, gs, kn, row + 16, vn, row, B, slots, *c.cache)
    for max_ctas in (0, 1, 5):
        out = c.decode(max_ctas)
        fused = [x.clone() for x in first]
        out2 = torch.full_like(out, 7.0)
        slot_out = torch.empty_like(slots)
        pa.pa_decode_kv_write_q4(c.desc, gs, c.q, kn, row + 16, vn, row, B, *fused, c.btd, c.maxp, c.ctx, c.max_ctx,
                                 c.scale, max_ctas, slot_out, out2, c.ws(max_ctas))
        assert torch.equal(slot_out, slots)
        assert torch.equal(fused[0], c.cache[0]) and torch.equal(fused[1], c.cache[1])
        assert torch.equal(out.view(torch.uint8), out2.view(torch.uint8))
        assert torch.isnan(out2[4]).any() and torch.isfinite(out2[[0, 1, 2, 5, 6, 7]]).all()
    assert pa.pa_read_device_errors(reset=True) == 0


@pytest.mark.parametrize("max_ctas", [0, 5])    # clusters; even shares and the merge kernel
def test_two_graphs_share_a_workspace_and_replay_with_new_inputs(max_ctas):
    """A captured step of each kind over one workspace, replayed in turn with other lengths, against fresh calls."""
    c = Case("bf16", 16, 8, 128, 32, 16, [300] * 21, seed=31)
    kn, vn = (torch.randn(21, 1024, device="cuda").bfloat16() for _ in range(2))
    ws = c.ws(max_ctas)
    outs = [torch.zeros_like(c.q) for _ in range(2)]
    slots = torch.zeros(21, dtype=torch.int64, device="cuda")

    def plain():
        pa.pa_decode_q4(c.desc, 32, c.q, 21, *c.cache, c.btd, c.maxp, c.ctx, c.max_ctx, c.scale, max_ctas, outs[0],
                        ws)

    def step():
        pa.pa_decode_kv_write_q4(c.desc, 32, c.q, kn, 1024, vn, 1024, 21, *c.cache, c.btd, c.maxp, c.ctx, c.max_ctx,
                                 c.scale, max_ctas, slots, outs[1], ws)

    plain()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(s):
        for f in (plain, step):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                f()
            graphs.append(g)
    torch.cuda.synchronize()
    for lens in ([300, 20, 150] * 7, [7, 0, 299] * 7, [1, 300, 17, 0, 33, 32, 256] * 3):
        c.ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        c.q.copy_(torch.randn(c.q.shape, device="cuda"))
        live = torch.tensor([x > 0 for x in lens])
        for o in outs:
            o.fill_(7.0)
        before = [x.clone() for x in c.cache]
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        after = c.cache
        c.cache = before
        want0 = c.decode(max_ctas)
        assert torch.equal(outs[0].view(torch.uint8), want0.view(torch.uint8))
        want1 = torch.full_like(want0, 7.0)
        pa.pa_decode_kv_write_q4(c.desc, 32, c.q, kn, 1024, vn, 1024, 21, *c.cache, c.btd, c.maxp, c.ctx, c.max_ctx,
                                 c.scale, max_ctas, None, want1, c.ws(max_ctas))
        torch.cuda.synchronize()
        assert torch.equal(outs[1].view(torch.uint8), want1.view(torch.uint8))
        assert torch.equal(after[0], c.cache[0]) and torch.equal(after[1], c.cache[1])
        c.cache = after     # the graphs hold these buffers
        assert bool((outs[0][~live] == 7.0).all())


def test_calls_on_a_stream_of_their_own_and_a_small_workspace():
    c = Case("bf16", 16, 8, 128, 64, 16, [200, 900], seed=14)
    ws, out = c.ws(), torch.full_like(c.q, 7.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pa.pa_decode_q4(c.desc, 64, c.q, 2, *c.cache, c.btd, c.maxp, c.ctx, c.max_ctx, c.scale, 0, out, ws, stream=s)
    s.synchronize()
    c.check(out)
    with pytest.raises(pa.PagedAttnError) as e:
        pa.pa_decode_q4(c.desc, 64, c.q, 2, *c.cache, c.btd, c.maxp, c.ctx, c.max_ctx, c.scale, 0, out, ws[:512])
    assert e.value.status == pa.PA_ERR_WORKSPACE


@pytest.mark.parametrize("hd", [128, 64])
def test_prefill_attends_to_the_read_back(hd):
    """A chunked prefill over a 4-bit cache as it is used: write the chunks, read the contexts back into a paged
    staging cache (each request's rows from a page boundary on), pa_prefill_varlen over it."""
    hq, hkv, gs, P = 8, 4, 32, 16
    lens, new = np.array([50, 16, 133]), np.array([20, 16, 70])
    c = Case("bf16", hq, hkv, hd, gs, P, lens, seed=17)
    n, row = int(new.sum()), hkv * hd
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(23)
    k, v = (torch.randn(n, hkv, hd, generator=g).bfloat16() for _ in range(2))
    q = torch.randn(n, hq, hd, generator=g).bfloat16()
    pos = torch.empty(n, dtype=torch.int32, device="cuda")
    slots = torch.empty(n, dtype=torch.int64, device="cuda")
    pa.pa_slot_mapping(c.desc, 3, cu, c.ctx, c.btd, c.maxp, n, pos, slots)
    pa.pa_kv_write_q4(c.desc, gs, k.cuda(), row, v.cuda(), row, n, slots, *c.cache)
    sl = slots.cpu().numpy()
    for val, x in zip(c.vals, (k, v)):
        val[sl] = q4.values(*q4.quantise(x.float().numpy(), gs), gs)
    pages = -(-lens // P)
    first = np.concatenate([[0], np.cumsum(pages)])
    stage = [torch.full((int(first[-1]), P, hkv, hd), float("nan"), dtype=torch.bfloat16, device="cuda")
             for _ in range(2)]
    pa.pa_kv_read_q4(c.desc, gs, 3, torch.tensor(first * P, dtype=torch.int32, device="cuda"), None, c.ctx, c.btd,
                     c.maxp, int(first[-1]) * P, *c.cache, stage[0], row, stage[1], row)
    bt2 = np.zeros((3, int(pages.max())), np.int32)
    for b in range(3):
        bt2[b, : pages[b]] = np.arange(first[b], first[b + 1])
    d2 = pa.cache_desc(hq, hkv, hd, P, int(first[-1]), torch.bfloat16)
    out = torch.zeros(n, hq, hd, dtype=torch.bfloat16, device="cuda")
    pa.pa_prefill_varlen(d2, q.cuda(), cu, 3, 70, n, stage[0], stage[1], torch.from_numpy(bt2).cuda(), bt2.shape[1],
                         c.ctx, 133, c.scale, out)
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    for b in range(3):
        L, m, s0 = int(lens[b]), int(new[b]), int(cu[b])
        at = c.bt[b, np.arange(L) // P].astype(np.int64) * P + np.arange(L) % P
        K, V = (torch.from_numpy(val[at]).float().bfloat16().double().numpy() for val in c.vals)
        ref = oracle.attend(q[s0: s0 + m].double().numpy(), K, V, np.arange(L - m, L), c.scale)[0]
        assert np.abs(got[s0: s0 + m] - ref).max() <= 1e-2 * np.abs(ref).max()
    assert pa.pa_read_device_errors(reset=True) == 0


@pytest.mark.parametrize("batch,longest", [(2, 600), (5, 600), (8, 600), (18, 600), (19, 600), (20, 600), (25, 600),
                                           (30, 600), (37, 600), (50, 600), (76, 500), (77, 256), (152, 256),
                                           (153, 256), (6, 64)])
def test_requests_by_clusters_of_every_size(batch, longest):
    """Short requests take a cluster of CTAs each where these fit the GPU and fill a good part of it (8 CTAs down to 1 as
    the batch grows): lengths below and above a cluster's CTAs, padding rows, a bad length and a bad page."""
    rng = np.random.default_rng(batch)
    lens = rng.integers(1, longest // 2, batch)
    lens[0], lens[-1] = longest, 33
    if batch > 4:
        lens[1:4] = 0, 1, longest // 2 + 1
    c = Case("bf16", 16, 8, 128, 64, 16, lens, seed=batch)
    ref = c.reference()
    c.check(c.decode(), ref)
    c.check(c.decode(max_ctas=1), ref)          # the same by one CTA
    assert pa.pa_read_device_errors(reset=True) == 0
    if batch > 4:
        c.ctx[4] = c.maxp * c.P + 1
        want = c.decode(max_ctas=1)
        got = c.decode()
        assert (got[4] == 7.0).all() and (want[4] == 7.0).all()
        keep = [i for i in range(batch) if i != 4]
        c2 = got[keep].double().cpu().numpy()
        live = lens[keep] > 0
        assert np.abs(c2[live] - ref[keep][live]).max() <= 1e-2 * np.nanmax(np.abs(ref))
        assert pa.pa_read_device_errors(reset=True) == pa.PA_DEVERR_BAD_LENGTH
        c.ctx[4] = int(lens[4])
    c.btd[0, :] = c.pages + 5                   # every page of a request: its output is zero
    out = c.decode()
    assert (out[0] == 0).all() and pa.pa_read_device_errors(reset=True) == pa.PA_DEVERR_BAD_PAGE
    got = out.double().cpu().numpy()
    live = np.arange(batch) > 0
    live &= lens > 0
    assert np.abs(got[live] - ref[live]).max() <= 1e-2 * np.abs(ref[live]).max()


@pytest.mark.parametrize("hq,hkv,hd,gs", [(64, 8, 128, 32), (5, 1, 64, 32), (14, 2, 128, 128), (12, 4, 64, 64)])
def test_the_fused_step_by_clusters_and_by_even_shares(hq, hkv, hd, gs):
    """The new token's row written by the cluster's last CTA, and by one CTA of an even split: the same bytes and the
    output of the separate calls."""
    lens = [1, 2, 33, 300, 0, 257, 64] * 3
    for max_ctas in (0, 3):
        c = Case("bf16", hq, hkv, hd, gs, 16, lens, seed=3)
        B = len(lens)
        g = torch.Generator().manual_seed(5)
        k, v = (torch.randn(B, hkv, hd, generator=g).bfloat16().cuda() for _ in range(2))
        row = hkv * hd
        other = [x.clone() for x in c.cache]
        out = torch.full_like(c.q, 7.0)
        slots = torch.full((B,), -9, dtype=torch.int64, device="cuda")
        pa.pa_decode_kv_write_q4(c.desc, gs, c.q, k, row, v, row, B, *c.cache, c.btd, c.maxp, c.ctx, c.max_ctx, c.scale,
                                 max_ctas, slots, out, c.ws(max_ctas))
        cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
        pos = torch.empty(B, dtype=torch.int32, device="cuda")
        s2 = torch.empty(B, dtype=torch.int64, device="cuda")
        pa.pa_slot_mapping(c.desc, B, cu, c.ctx, c.btd, c.maxp, B, pos, s2)
        pa.pa_kv_write_q4(c.desc, gs, k, row, v, row, B, s2, *other)
        assert (slots == s2).all()
        for a, b in zip(c.cache, other):
            assert (a == b).all()
        c.cache = other
        assert (c.decode(max_ctas) == out).all()
    assert pa.pa_read_device_errors(reset=True) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_key_that_is_not_a_number_makes_its_heads_outputs_nan_however_they_are_split(dtype):
    c = Case(dtype, 8, 4, 128, 32, 16, [900, 700] * 12, seed=6)
    ref = c.reference()
    slot = int(c.bt[0, 20]) * 16 + 3
    u, s, p = q4.unpack_rows(c.cache[0][slot].cpu().numpy()[None], [slot], 4, 128, 32)
    s[0, 2, 1], p[0, 2, 1] = 0, np.float16(np.nan)
    c.cache[0][slot] = torch.from_numpy(q4.pack_rows(u, s, p, [slot])[0]).cuda()
    want = torch.zeros(24, 8, 128, dtype=torch.bool)
    want[0, 4:6] = True                         # the two q-heads of kv-head 2
    for max_ctas in (0, 1, 24, 61):
        out = c.decode(max_ctas)
        assert torch.equal(torch.isnan(out).cpu(), want)
        ok = ~want.numpy()
        err = np.abs(out.double().cpu().numpy() - ref)[ok].max()
        assert err <= (1e-5 if dtype == "f32" else 1e-2) * np.abs(ref).max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gs", [32, 64, 128])
@pytest.mark.parametrize("order", ["growing", "falling", "one"])
def test_scales_that_change_along_the_context(gs, order, dtype):
    """V's magnitude rises or falls by 2^40 along the context, or is 2^20 times the others' in one token that no query
    looks at: the powers of two that keep p s in float16's range follow the largest scale."""
    c = Case(dtype, 4, 4, 128, gs, 16, [700, 90] * 8, seed=8)
    rng = np.random.default_rng(1)
    for b, L in enumerate(c.lens):
        slots = c.bt[b, np.arange(L) // 16].astype(np.int64) * 16 + np.arange(L) % 16
        x = rng.standard_normal((L, 4, 128))
        e = np.linspace(-28, 12, L)
        if order == "falling":
            e = e[::-1]
        if order == "one":
            e = np.full(L, -8.0)
            e[L // 2] = 12.0
            k = rng.standard_normal((1, 4, 128)) * 0.01 - 4 * c.q64[b][None]     # scores far below the others'
            c.cache[0][slots[L // 2]] = torch.from_numpy(q4.pack_rows(*q4.quantise(k.astype(np.float32), gs),
                                                                      slots[L // 2:L // 2 + 1])[0]).cuda()
            c.vals[0][slots[L // 2]] = q4.values(*q4.quantise(k.astype(np.float32), gs), gs)[0]
        x = (x * np.exp2(e)[:, None, None]).astype(np.float32)
        u, sc, off = q4.quantise(x, gs)
        c.cache[1][torch.from_numpy(slots).cuda()] = torch.from_numpy(q4.pack_rows(u, sc, off, slots)).cuda()
        c.vals[1][slots] = q4.values(u, sc, off, gs)
    ref = c.reference()
    for max_ctas in (0, 1, 2, 20):
        out = c.decode(max_ctas)
        c.check(out, ref)
        if dtype == "f32":      # small outputs, too
            assert np.abs(out.double().cpu().numpy() - ref).max() <= 1e-5 * np.abs(ref).max()


def test_two_streams_at_once_and_the_same_bits_every_time():
    """A clustered and a split decode, each on a stream and a workspace of its own, over and over side by side."""
    a = Case("bf16", 16, 8, 128, 64, 16, [300, 17, 1000, 0] * 4, seed=21)
    b = Case("bf16", 24, 4, 128, 32, 16, [3000, 5, 641], seed=22)
    wa, wb = a.decode(), b.decode(60)
    a.check(wa)
    b.check(wb)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    ws = [a.ws(), b.ws(60)]
    outs = [[torch.full_like(x.q, 7.0) for _ in range(40)] for x in (a, b)]
    torch.cuda.synchronize()
    for i in range(40):
        pa.pa_decode_q4(a.desc, a.gs, a.q, 16, *a.cache, a.btd, a.maxp, a.ctx, a.max_ctx, a.scale, 0, outs[0][i], ws[0],
                        stream=sa)
        pa.pa_decode_q4(b.desc, b.gs, b.q, 3, *b.cache, b.btd, b.maxp, b.ctx, b.max_ctx, b.scale, 60, outs[1][i], ws[1],
                        stream=sb)
    torch.cuda.synchronize()
    assert all(torch.equal(o, wa) for o in outs[0]) and all(torch.equal(o, wb) for o in outs[1])


def test_a_fork_and_join_in_one_graph():
    a = Case("bf16", 16, 8, 128, 64, 16, [300, 17, 1000, 0] * 4, seed=21)
    b = Case("f32", 8, 4, 64, 32, 16, [3000, 5, 641], seed=22)
    wa, wb = a.decode(), b.decode()
    oa, ob, ws = torch.full_like(a.q, 7.0), torch.full_like(b.q, 7.0), [a.ws(), b.ws()]
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        pa.pa_decode_q4(a.desc, a.gs, a.q, 16, *a.cache, a.btd, a.maxp, a.ctx, a.max_ctx, a.scale, 0, oa, ws[0])
        pa.pa_decode_q4(b.desc, b.gs, b.q, 3, *b.cache, b.btd, b.maxp, b.ctx, b.max_ctx, b.scale, 0, ob, ws[1],
                        stream=side)
        main.wait_stream(side)
    for _ in range(3):
        oa.fill_(7.0)
        ob.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(oa, wa) and torch.equal(ob, wb)
