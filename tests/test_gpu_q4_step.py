"""Whole steps over a 4-bit cache: the chunks of several prompts, then decode steps, through run_step."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_gqa_08_gb300 as pa
from oracle import q4_cache as q4
from paged_kv_gqa_08_gb300.step import alloc_step_buffers, run_step, write_rows

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda_lib")]

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


class Model:
    """One layer's requests over a 4-bit cache whose unused rows hold random bytes."""

    def __init__(self, dtype, hq, hkv, hd, gs, P, maxp, batch, norm, seed):
        self.dt, self.dtype, self.hq, self.hkv, self.hd, self.gs, self.P = DT[dtype], dtype, hq, hkv, hd, gs, P
        self.maxp, self.batch = maxp, batch
        self.rng = np.random.default_rng(seed)
        pages = maxp * batch + 3
        self.desc = pa.cache_desc(hq, hkv, hd, P, pages, self.dt)
        R = pa.pa_q4_row_bytes(self.desc, gs)
        self.caches = [torch.from_numpy(self.rng.integers(0, 256, (pages * P, R)).astype(np.uint8)).cuda()
                       for _ in range(2)]
        self.bt = self.rng.permutation(pages)[: batch * maxp].reshape(batch, maxp).astype(np.int32)
        self.lens = np.zeros(batch, np.int32)
        self.scale = hd ** -0.5
        self.w = [self.rand(hd) for _ in range(2)] if norm else [None, None]

    def rand(self, *shape):
        return torch.from_numpy(self.rng.standard_normal(shape).astype(np.float32)).to(self.dt).cuda()

    def step(self, kind, new, bufs, stream=None):
        """Run a step of ``new[b]`` tokens per request (-1: a padding request) and check what it wrote and answered."""
        new = np.asarray(new)
        pad = new < 0
        count = np.where(pad, 0, new) if kind != "decode" else np.ones_like(new)
        self.lens = self.lens + np.where(pad, 0, new).astype(np.int32)
        ctx = np.where(pad, 0, self.lens).astype(np.int32)
        n = int(count.sum())
        q, k, v = self.rand(n, self.hq, self.hd), self.rand(n, self.hkv, self.hd), self.rand(n, self.hkv, self.hd)
        cu = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
        before = [c.clone() for c in self.caches]
        bufs.out.fill_(7.0)
        out = run_step(self.desc, kind, bufs, q, k, v, torch.from_numpy(cu).cuda(), torch.from_numpy(ctx).cuda(),
                       torch.from_numpy(self.bt).cuda(), *self.caches, self.scale, self.maxp, int(ctx.max()),
                       int(count.max()), *self.w, 1e-6, 1e4, stream)
        torch.cuda.synchronize()
        assert pa.pa_read_device_errors(reset=True) == 0
        got = out.double().cpu().numpy()
        q64 = (q if self.w[0] is None else bufs.q_out[:n]).double().cpu().numpy()
        # the rows written: all of the new tokens', none other, and (without the norm) the oracle's codes and scales
        pos = np.concatenate([np.arange(ctx[b] - count[b], ctx[b]) for b in range(self.batch)])
        req = np.repeat(np.arange(self.batch), count)
        live = ctx[req] > 0
        slots = self.bt[req, np.maximum(pos, 0) // self.P].astype(np.int64) * self.P + pos % self.P
        other = np.ones(self.caches[0].shape[0], bool)
        other[slots[live]] = False
        raw = [c.cpu().numpy() for c in self.caches]
        for was, now, x, isk in zip(before, raw, (k, v), (True, False)):
            assert (was.cpu().numpy()[other] == now[other]).all()
            if self.w[0] is None or not isk:
                want = q4.quantise(x.float().cpu().numpy()[live], self.gs)
                for a, b in zip(q4.unpack_rows(now[slots[live]], slots[live], self.hkv, self.hd, self.gs), want):
                    assert (a.view(f"u{a.itemsize}") == b.view(f"u{b.itemsize}")).all()
        # The answer.  The decode kernel attends to the values of the codes; prefill to these rounded to the dtype (bf16:
        # 2^-8 of a value), with probabilities of that type, and every output is rounded to it: 1e-2 of the largest.
        for b in range(self.batch):
            r = slice(cu[b], cu[b + 1])
            if ctx[b] == 0:
                assert (got[r] == 7.0).all()
                continue
            if count[b] == 0:
                continue
            L = int(ctx[b])
            at = self.bt[b, np.arange(L) // self.P].astype(np.int64) * self.P + np.arange(L) % self.P
            K, V = (q4.row_values(c[at], at, self.hkv, self.hd, self.gs) for c in raw)
            if kind != "decode":
                K, V = (torch.from_numpy(x).to(self.dt).double().numpy() for x in (K, V))
            ref = oracle.attend(q64[r], K, V, np.arange(L - count[b], L), self.scale)[0]
            assert np.abs(got[r] - ref).max() <= (1e-5 if self.dtype == "f32" else 1e-2) * np.abs(ref).max()


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dtype,hq,hkv,hd,gs,P", [("bf16", 16, 8, 128, 32, 16), ("bf16", 8, 2, 128, 128, 64),
                                                  ("bf16", 12, 4, 64, 64, 16), ("f32", 4, 2, 64, 32, 16)])
def test_prompts_in_chunks_then_decode(dtype, hq, hkv, hd, gs, P, norm):
    m = Model(dtype, hq, hkv, hd, gs, P, maxp=384 // P, batch=4, norm=norm, seed=hq + gs)
    pre = alloc_step_buffers(m.desc, "prefill", 400, 4, 384, "cuda", norm=norm, max_seqlen_q=200, group_size=gs)
    dec = alloc_step_buffers(m.desc, "decode", 4, 4, 384, "cuda", norm=norm, group_size=gs)
    for new in ([1, 130, 16, -1], [17, 70, 0, 1], [1, 1, 200, 33]):
        m.step("prefill", new, pre)
    for new in ([1, 1, 1, 1], [1, -1, 1, 1], [1, 1, 1, 1]):
        m.step("decode", new, dec)
    m.step("prefill", [1, 33, 1, 5], pre)      # decode rows and chunks in one prefill launch
    m.step("decode", [1, 1, 1, 1], dec)


def test_a_step_on_a_stream_of_its_own():
    m = Model("bf16", 16, 8, 128, 64, 16, maxp=16, batch=2, norm=True, seed=3)
    pre = alloc_step_buffers(m.desc, "prefill", 200, 2, 256, "cuda", norm=True, group_size=64)
    dec = alloc_step_buffers(m.desc, "decode", 2, 2, 256, "cuda", norm=True, group_size=64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.step("prefill", [100, 7], pre)
        m.step("decode", [1, 1], dec)


def test_write_rows_and_limits():
    m = Model("bf16", 8, 4, 128, 32, 16, maxp=8, batch=2, norm=False, seed=4)
    k, v = m.rand(70, 4, 128), m.rand(70, 4, 128)
    cu = torch.tensor([0, 30, 70], dtype=torch.int32, device="cuda")
    lens = torch.tensor([30, 40], dtype=torch.int32, device="cuda")
    pos = torch.empty(70, dtype=torch.int32, device="cuda")
    slots = torch.empty(70, dtype=torch.int64, device="cuda")
    write_rows(m.desc, k, v, cu, lens, torch.from_numpy(m.bt).cuda(), m.maxp, pos, slots, *m.caches, group_size=32)
    sl = slots.cpu().numpy()
    for c, x in zip(m.caches, (k, v)):
        want = q4.pack_rows(*q4.quantise(x.float().cpu().numpy(), 32), sl)
        assert (c.cpu().numpy()[sl] == want).all()
    m.lens[:] = (30, 40)
    bufs = alloc_step_buffers(m.desc, "prefill", 20, 2, 64, "cuda", group_size=32)
    m.step("prefill", [9, 11], bufs)
    with pytest.raises(ValueError):
        m.step("prefill", [30, 1], bufs)       # a context of 69 tokens in a staging cache for 64
