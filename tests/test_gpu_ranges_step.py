"""Serving with the calls together: tables built on the GPU, steps over a window whose pages are handed back, and
branches that share their prompt's pages, each output against plain attention in 64 bits."""
import pytest
import torch

import paged_kv_gqa_08_gb300 as pa
from paged_kv_gqa_08_gb300.step import alloc_step_buffers, run_step
from range_reference import attend, check

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


class Server:
    """Rows of requests over one pool of pages; keeps every token's K and V for the check."""

    def __init__(self, B, Hq, Hkv, hd, P, dt, num_pages, maxp, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.Hq, self.Hkv, self.hd, self.P, self.dt, self.maxp = B, Hq, Hkv, hd, P, dt, maxp
        self.num_pages = num_pages
        self.desc = pa.cache_desc(Hq, Hkv, hd, P, num_pages, dt)
        nan = float("nan")
        self.kc = torch.full((num_pages, P, Hkv, hd), nan, dtype=dt, device="cuda")
        self.vc = self.kc.clone()
        i32 = dict(dtype=torch.int32, device="cuda")
        self.bt = torch.full((B, maxp), -1, **i32)
        self.ring = torch.randperm(num_pages, generator=self.g, device="cuda").to(torch.int32)
        self.pool = torch.tensor([0, num_pages], device="cuda")
        self.refs = torch.zeros(num_pages, **i32)
        self.ctx = torch.zeros(B, **i32)
        self.new = torch.zeros(B, **i32)
        self.cu = torch.zeros(B + 1, **i32)
        self.K = [torch.zeros(0, Hkv, hd, dtype=dt, device="cuda") for _ in range(B)]
        self.V = [k.clone() for k in self.K]

    def rand(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda").to(self.dt)

    def extend(self, rows):
        """On the device: pages for self.new; positions and slots of up to `rows` tokens."""
        pos = torch.zeros(rows, dtype=torch.int32, device="cuda")
        slots = torch.zeros(rows, dtype=torch.int64, device="cuda")
        pa.pa_extend_tables(self.desc, self.B, self.new, self.ctx, self.bt, self.maxp, self.ring, self.pool, rows,
                            self.cu, self.ctx, pos, slots, self.refs, self.pool)
        return pos, slots

    def poison_free_pages(self):
        free = self.refs == 0
        self.kc[free] = float("nan")
        self.vc[free] = float("nan")

    def remember(self, new, k, v):
        at = 0
        for b, n in enumerate(new):
            self.K[b] = torch.cat([self.K[b], k[at: at + n].view(n, self.Hkv, self.hd)])
            self.V[b] = torch.cat([self.V[b], v[at: at + n].view(n, self.Hkv, self.hd)])
            at += n

    def compare(self, new, q, out, scale, window, sinks, what):
        at = 0
        for b, n in enumerate(new):
            if not n:
                continue
            L = self.K[b].shape[0]
            p, j = torch.arange(L - n, L, device="cuda")[:, None], torch.arange(L, device="cuda")
            seen = (j <= p) & ((j > p - window) | (j < sinks))
            o, bound = attend(q[at: at + n], self.K[b], self.V[b], seen, scale, self.dt)
            check(out[at: at + n], o, bound, f"{what}, row {b}")
            at += n


@pytest.mark.parametrize("dt,Hq,Hkv,hd,P", [(BF16, 16, 8, 128, 16), (BF16, 6, 2, 64, 32), (F32, 4, 1, 128, 16)])
@pytest.mark.parametrize("window,sinks", [(40, 4), (200, 0), (100, 33)])
def test_windowed_serving(cuda_lib, dt, Hq, Hkv, hd, P, window, sinks):
    prompts = [1, 30, 300, 77, 161]
    B, scale = len(prompts), hd ** -0.5
    s = Server(B, Hq, Hkv, hd, P, dt, num_pages=80 + 10 * B, maxp=64, seed=window)

    def step(kind, new, what):
        n = sum(new)
        s.new.copy_(torch.tensor(new, dtype=torch.int32))
        s.extend(n)
        q, k, v = s.rand(n, Hq, hd), s.rand(n, Hkv * hd), s.rand(n, Hkv * hd)
        s.remember(new, k, v)
        bufs = alloc_step_buffers(s.desc, kind, n, B, 64 * P, "cuda", max_seqlen_q=max(new), window=window,
                                  num_sinks=sinks)
        out = run_step(s.desc, kind, bufs, q, k, v, s.cu, s.ctx, s.bt, s.kc, s.vc, scale, s.maxp, 64 * P, max(new),
                       window=window, num_sinks=sinks)
        s.compare(new, q, out, scale, window, sinks, what)
        pa.pa_release_window_pages(s.desc, window, sinks, B, s.ctx, s.bt, s.maxp, s.refs, s.ring, s.pool, s.pool)
        s.poison_free_pages()

    step("prefill", prompts, "prompts")
    step("prefill", [50, 1, 3, 64, 1], "second chunks")
    for i in range(2 * P):
        step("decode", [1] * B, f"decode {i}")
    # what is held: the sinks' pages and those of the window
    held = int((s.refs > 0).sum())
    assert held <= B * (-(-sinks // P) + -(-window // P) + 1)
    assert held + int(s.pool[1] - s.pool[0]) == s.num_pages
    assert pa.pa_read_device_errors(reset=True) == 0


@pytest.mark.parametrize("dt,Hq,Hkv,hd,P,prompt", [(BF16, 32, 8, 128, 16, 500), (BF16, 32, 8, 128, 64, 6000),
                                                   (BF16, 8, 8, 64, 16, 333), (F32, 6, 2, 64, 16, 200)])
def test_branches_of_prompts(cuda_lib, dt, Hq, Hkv, hd, P, prompt):
    """Two prompts; eight and five branches of them share their whole pages, take the rest of the prompt for
    themselves, decode, and go."""
    scale = hd ** -0.5
    of = [0] * 9 + [1] * 6            # the rows' prompts: row 0 and row 9 are the prompts themselves
    lens = (prompt, prompt // 2 + 3)
    heads = (0, 9)
    B = len(of)
    maxp = prompt // P + 8
    s = Server(B, Hq, Hkv, hd, P, dt, num_pages=3 * maxp + 8 * B, maxp=maxp, seed=prompt)
    whole = [n // P for n in lens]

    def step(kind, new, what, fill=None, **kw):
        n = sum(new)
        s.new.copy_(torch.tensor(new, dtype=torch.int32))
        s.extend(n)
        q = s.rand(n, Hq, hd)
        k, v = (s.rand(n, Hkv * hd), s.rand(n, Hkv * hd)) if fill is None else fill
        s.remember(new, k, v)
        bufs = alloc_step_buffers(s.desc, kind, n, B, maxp * P, "cuda", max_seqlen_q=max(new),
                                  num_groups=2 if kw else 0, max_prefix_len=max(lens))
        out = run_step(s.desc, kind, bufs, q, k, v, s.cu, s.ctx, s.bt, s.kc, s.vc, scale, s.maxp, maxp * P, max(new),
                       **kw)
        if kind == "decode":
            s.compare(new, q, out, scale, 1 << 30, 0, what)

    step("prefill", [lens[of[b]] if b in heads else 0 for b in range(B)], "prompts")
    parents = torch.tensor([-1 if b in heads else heads[of[b]] for b in range(B)], dtype=torch.int32, device="cuda")
    counts = torch.tensor([whole[of[b]] for b in range(B)], dtype=torch.int32, device="cuda")
    pa.pa_share_pages(s.desc, B, parents, counts, s.bt, s.maxp, s.refs)
    for b in range(B):
        if b not in heads:
            n = whole[of[b]] * P
            s.K[b], s.V[b] = s.K[heads[of[b]]][:n].clone(), s.V[heads[of[b]]][:n].clone()
    s.ctx = torch.where(parents >= 0, counts * P, s.ctx)
    # the rest of the prompt, in pages of their own
    rest = [0 if b in heads else lens[of[b]] - whole[of[b]] * P for b in range(B)]
    rows = [(s.K[heads[of[b]]][whole[of[b]] * P: lens[of[b]]], s.V[heads[of[b]]][whole[of[b]] * P: lens[of[b]]])
            for b in range(B) if b not in heads]
    if sum(rest):
        step("prefill", rest, "rest of the prompts",
             fill=tuple(torch.cat([r[i] for r in rows]).flatten(1).contiguous() for i in range(2)))
    groups = dict(cu_groups=torch.tensor([0, 9, 15], dtype=torch.int32, device="cuda"),
                  prefix_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), max_prefix_len=max(lens))
    for i in range(P + 3):
        step("decode", [1] * B, f"decode {i}", **groups)
    # the prompts' own rows go first: their shared pages stay, with the branches
    first, last = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.full((B,), maxp, dtype=torch.int32, device="cuda")
    own = torch.where(parents < 0, last, first)
    pa.pa_release_pages(s.desc, B, first, own, s.bt, s.maxp, s.refs, s.ring, s.pool, s.pool)
    s.ctx = torch.where(parents < 0, torch.zeros_like(s.ctx), s.ctx)
    s.poison_free_pages()
    new = [0 if b in heads else 1 for b in range(B)]
    n = sum(new)
    s.new.copy_(torch.tensor(new, dtype=torch.int32))
    s.extend(n)
    q, k, v = s.rand(n, Hq, hd), s.rand(n, Hkv * hd), s.rand(n, Hkv * hd)
    s.remember(new, k, v)
    # decode takes a row of queries for each row of the batch: the padding rows' are anything
    pad = torch.full((B, Hq, hd), float("nan"), dtype=dt, device="cuda")
    pad[torch.tensor(new, device="cuda") > 0] = q
    full = lambda x: torch.zeros(B, x.shape[1], dtype=dt, device="cuda").index_copy_(  # noqa: E731
        0, torch.tensor(new, device="cuda").nonzero()[:, 0], x)
    bufs = alloc_step_buffers(s.desc, "decode", B, B, maxp * P, "cuda", num_groups=2, max_prefix_len=max(lens))
    bufs.out.fill_(7.0)
    out = run_step(s.desc, "decode", bufs, pad, full(k), full(v), torch.arange(B + 1, dtype=torch.int32, device="cuda"),
                   s.ctx, s.bt, s.kc, s.vc, scale, s.maxp, maxp * P, 1, **groups)
    for b in heads:
        assert (out[b] == 7.0).all()
    s.compare(new, q, out[torch.tensor(new, device="cuda") > 0], scale, 1 << 30, 0, "after the prompts' rows went")
    pa.pa_release_pages(s.desc, B, first, last, s.bt, s.maxp, s.refs, s.ring, s.pool, s.pool)
    assert int(s.pool[1] - s.pool[0]) == s.num_pages and int(s.refs.abs().sum()) == 0
    assert sorted(s.ring.tolist()) == list(range(s.num_pages))
    assert pa.pa_read_device_errors(reset=True) == 0


def test_a_captured_windowed_step(cuda_lib):
    """Tables, rows written, attention and pages handed back in one graph, replayed while the contexts grow past their
    windows."""
    B, Hq, Hkv, hd, P, window, sinks = 3, 8, 4, 128, 16, 50, 4
    s = Server(B, Hq, Hkv, hd, P, BF16, num_pages=40, maxp=32, seed=1)
    q, k, v = torch.zeros(B, Hq, hd, dtype=BF16, device="cuda"), *torch.zeros(2, B, Hkv * hd, dtype=BF16, device="cuda")
    bufs = alloc_step_buffers(s.desc, "decode", B, B, 32 * P, "cuda", window=window, num_sinks=sinks)
    s.new.fill_(1)
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    slots = torch.zeros(B, dtype=torch.int64, device="cuda")

    def enqueue():
        pa.pa_extend_tables(s.desc, B, s.new, s.ctx, s.bt, s.maxp, s.ring, s.pool, B, s.cu, s.ctx, pos, slots, s.refs,
                            s.pool)
        pa.pa_decode_kv_write_window(s.desc, window, sinks, q, k, Hkv * hd, v, Hkv * hd, B, s.kc, s.vc, s.bt, s.maxp,
                                     s.ctx, 32 * P, 0.1, 0, None, bufs.out, bufs.workspace)
        pa.pa_release_window_pages(s.desc, window, sinks, B, s.ctx, s.bt, s.maxp, s.refs, s.ring, s.pool, s.pool)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        enqueue()
    for i in range(150):
        qi, ki, vi = s.rand(B, Hq, hd), s.rand(B, Hkv * hd), s.rand(B, Hkv * hd)
        q.copy_(qi)
        k.copy_(ki)
        v.copy_(vi)
        s.remember([1] * B, ki, vi)
        graph.replay()
        if i % 7 == 0:
            s.compare([1] * B, qi, bufs.out, 0.1, window, sinks, f"step {i}")
            s.poison_free_pages()
    assert int(s.pool[1] - s.pool[0]) >= 40 - B * 6
    assert pa.pa_read_device_errors(reset=True) == 0
