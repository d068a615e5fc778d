"""Block tables, positions and slots built on the GPU, against the rules written out in Python, request by request."""
import random

import pytest
import torch

import paged_kv_gqa_08_gb300 as pa
from paged_kv_gqa_08_gb300.block_manager import BlockManager

pytestmark = pytest.mark.gpu


class Ref:
    """The state on the host, and the calls' rules."""

    def __init__(self, num_pages, P, B, maxp, seed=0, start=0, refs=True):
        r = random.Random(seed)
        self.P, self.maxp, self.n = P, maxp, num_pages
        order = list(range(num_pages))
        r.shuffle(order)
        self.ring = [0] * num_pages
        for i, p in enumerate(order):
            self.ring[(start + i) % num_pages] = p
        self.pool = [start, start + num_pages]
        self.refs = [0] * num_pages if refs else None
        self.bt = [[-1] * maxp for _ in range(B)]
        self.ctx = [0] * B

    def extend(self, new, max_tokens):
        asked_p = asked_t = 0
        cu, pos, slots = [0], [], []
        flags = 0
        free = self.pool[1] - self.pool[0]
        for b, n in enumerate(new):
            L = self.ctx[b]
            if n < 0 or L < 0 or L + n > self.maxp * self.P:
                flags |= pa.PA_DEVERR_BAD_LENGTH
                n = 0
            need = -(-(L + n) // self.P) - -(-L // self.P)
            asked_p += need
            asked_t += n
            ok_t, ok_p = asked_t <= max_tokens, need == 0 or asked_p <= free
            if n and not (ok_t and ok_p):
                flags |= (0 if ok_t else pa.PA_DEVERR_BAD_LENGTH) | (0 if ok_p else pa.PA_DEVERR_NO_PAGES)
                n = 0
            for t in range(L, L + n):
                if t % self.P == 0:
                    page = self.ring[self.pool[0] % self.n]
                    self.pool[0] += 1
                    self.bt[b][t // self.P] = page
                    if self.refs:
                        self.refs[page] = 1
                pos.append(t)
                slots.append(self.bt[b][t // self.P] * self.P + t % self.P)
            self.ctx[b] = L + n
            cu.append(len(pos))
        pad = max_tokens - len(pos)
        return cu, pos + [0] * pad, slots + [-1] * pad, flags

    def share(self, parents, counts):
        for b, f in enumerate(parents):
            if f >= 0:
                for j in range(counts[b]):
                    self.bt[b][j] = self.bt[f][j]
                    if self.bt[b][j] >= 0:
                        self.refs[self.bt[b][j]] += 1

    def release(self, first, end):
        back = []
        for b, (f, e) in enumerate(zip(first, end)):
            for j in range(e - 1, f - 1, -1):
                if self.bt[b][j] >= 0:
                    back.append(self.bt[b][j])
                self.bt[b][j] = -1
        last = {p: i for i, p in enumerate(back)}
        for i, p in enumerate(back):
            if self.refs:
                self.refs[p] -= 1
        for i, p in enumerate(back):
            if last[p] == i and (not self.refs or self.refs[p] == 0):
                self.ring[self.pool[1] % self.n] = p
                self.pool[1] += 1

    def release_window(self, window, sinks):
        ends = [max(0, L + 1 - window) // self.P for L in self.ctx]
        self.release([min(-(-sinks // self.P), self.maxp)] * len(ends), [min(e, self.maxp) for e in ends])


class Dev:
    """The same state on the GPU."""

    def __init__(self, ref, alias=True):
        t = lambda x, dt=torch.int32: torch.tensor(x, dtype=dt, device="cuda")  # noqa: E731
        self.desc = pa.cache_desc(4, 2, 64, ref.P, ref.n, torch.bfloat16)
        self.B, self.maxp = len(ref.bt), ref.maxp
        self.bt, self.ring, self.ctx = t(ref.bt), t(ref.ring), t(ref.ctx)
        self.refs = t(ref.refs) if ref.refs is not None else None
        self.pool = t(ref.pool, torch.int64)
        self.alias = alias

    def out(self, x):
        return x if self.alias else torch.full_like(x, 12345)

    def extend(self, new, max_tokens, stream=None):
        new = torch.tensor(new, dtype=torch.int32, device="cuda")
        cu = torch.full((self.B + 1,), 9, dtype=torch.int32, device="cuda")
        pos = torch.full((max_tokens,), 9, dtype=torch.int32, device="cuda")
        slots = torch.full((max_tokens,), 9, dtype=torch.int64, device="cuda")
        ctx, pool = self.out(self.ctx), self.out(self.pool)
        pa.pa_extend_tables(self.desc, self.B, new, self.ctx, self.bt, self.maxp, self.ring, self.pool, max_tokens, cu,
                            ctx, pos if max_tokens else None, slots if max_tokens else None, self.refs, pool, stream)
        self.ctx, self.pool = ctx, pool
        return cu.tolist(), pos.tolist(), slots.tolist()

    def share(self, parents, counts):
        t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        pa.pa_share_pages(self.desc, self.B, t(parents), t(counts), self.bt, self.maxp, self.refs)

    def release(self, first, end):
        t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        pool = self.out(self.pool)
        pa.pa_release_pages(self.desc, self.B, t(first), t(end), self.bt, self.maxp, self.refs, self.ring, self.pool,
                            pool)
        self.pool = pool

    def release_window(self, window, sinks):
        pool = self.out(self.pool)
        pa.pa_release_window_pages(self.desc, window, sinks, self.B, self.ctx, self.bt, self.maxp, self.refs, self.ring,
                                   self.pool, pool)
        self.pool = pool

    def same(self, ref):
        assert self.ctx.tolist() == ref.ctx
        assert self.pool.tolist() == ref.pool
        assert self.bt.tolist() == ref.bt
        assert self.ring.tolist() == ref.ring
        if ref.refs is not None:
            assert self.refs.tolist() == ref.refs


def flags():
    return pa.pa_read_device_errors(reset=True)


def step(ref, dev, new, max_tokens):
    cu, pos, slots, fl = ref.extend(new, max_tokens)
    assert dev.extend(new, max_tokens) == (cu, pos, slots)
    assert flags() == fl
    dev.same(ref)
    return fl


@pytest.mark.parametrize("refs", [True, False])
@pytest.mark.parametrize("alias", [True, False])
@pytest.mark.parametrize("P", [16, 64, 1024])
@pytest.mark.parametrize("B", [1, 3, 64, 511, 512, 513, 1500])
def test_prompts_and_decode_steps(cuda_lib, B, P, alias, refs):
    r = random.Random(B * P)
    maxp = 400 // P + 2
    ref = Ref(B * maxp + 7, P, B, maxp, seed=B, start=(1 << 40) + 12345, refs=refs)
    dev = Dev(ref, alias)
    step(ref, dev, [r.choice([0, 1, P - 1, P, P + 1, r.randint(0, 380)]) for _ in range(B)], 400 * B)
    for _ in range(3):
        step(ref, dev, [1] * B, B + 5)
    step(ref, dev, [r.randint(0, 2) for _ in range(B)], 3 * B)
    step(ref, dev, [0] * B, 0)


def test_one_long_prompt(cuda_lib):
    ref = Ref(9000, 16, 3, 7000, seed=1)
    dev = Dev(ref)
    step(ref, dev, [5, 100003, 40], 100100)
    step(ref, dev, [1, 1, 1], 3)


def test_pool_runs_out(cuda_lib):
    ref = Ref(10, 16, 6, 8, seed=1, start=3)
    dev = Dev(ref)
    assert step(ref, dev, [40, 16, 100, 1, 0, 17], 200) == pa.PA_DEVERR_NO_PAGES   # 3 + 1 + 7 pages: the third and on
    assert ref.ctx == [40, 16, 0, 0, 0, 0]
    assert step(ref, dev, [8, 0, 90, 1, 1, 0], 200) == pa.PA_DEVERR_NO_PAGES       # six pages are left: the third takes them
    assert ref.ctx == [48, 16, 90, 0, 0, 0]
    step(ref, dev, [9, 1, 1, 1, 1, 1], 200)


def test_refusals_on_the_device(cuda_lib):
    ref = Ref(50, 16, 5, 4, seed=1)
    dev = Dev(ref)
    # a table too short, a negative count, more tokens than rows
    assert step(ref, dev, [65, -3, 20, 10, 30], 40) == pa.PA_DEVERR_BAD_LENGTH
    assert ref.ctx == [0, 0, 20, 10, 0]
    dev.pool.copy_(torch.tensor([5, 2]))                    # a state that is none
    keep = dev.bt.clone()
    out = dev.extend([16, 0, 1, 1, 16], 40)
    assert flags() == pa.PA_DEVERR_BAD_LENGTH | pa.PA_DEVERR_NO_PAGES
    assert out[0] == [0, 0, 0, 1, 2, 2] and torch.equal(dev.bt, keep) and dev.pool.tolist() == [5, 2]
    dev.pool.copy_(torch.tensor([0, 50]))
    dev.ring[0], dev.ring[1] = 50, -1                        # entries that are no pages
    out = dev.extend([0, 17, 0, 0, 0], 17)
    assert flags() == pa.PA_DEVERR_BAD_PAGE
    assert out[2] == [-1] * 17 and dev.bt[1].tolist() == [-1] * 4


@pytest.mark.parametrize("seed", range(6))
def test_random_serving(cuda_lib, seed):
    """Requests come, branch, grow, lose what their window leaves and go; pages are conserved throughout."""
    r = random.Random(seed)
    B, P, maxp = r.choice([5, 40, 300]), r.choice([16, 32]), 60
    ref = Ref(r.choice([B * 8, B * maxp]), P, B, maxp, seed=seed, start=r.randrange(1 << 45))
    dev = Dev(ref, alias=seed % 2 == 0)
    window, sinks = r.randint(1, 150), r.choice([0, 4, 40])
    for _ in range(12):
        free = [b for b in range(B) if ref.ctx[b] == 0]
        new = [0] * B
        for b in range(B):
            new[b] = r.choice([0, 1, 1, r.randint(1, 200)]) if ref.ctx[b] or r.random() < 0.3 else 0
        # branches: rows that hold nothing follow rows that hold whole pages
        parents, counts = [-1] * B, [0] * B
        for b in free:
            f = r.randrange(B)
            if new[b] == 0 and ref.ctx[f] >= P and r.random() < 0.5:
                parents[b], counts[b] = f, r.randint(1, ref.ctx[f] // P)
        ref.share(parents, counts)
        dev.share(parents, counts)
        for b in range(B):
            if parents[b] >= 0:
                ref.ctx[b] = counts[b] * P
        dev.ctx = torch.tensor(ref.ctx, dtype=torch.int32, device="cuda")
        step(ref, dev, new, sum(n for n in new) + r.choice([0, 5]))
        ref.release_window(window, sinks)
        dev.release_window(window, sinks)
        dev.same(ref)
        gone = [b for b in range(B) if ref.ctx[b] and r.random() < 0.2]
        end = [maxp if b in gone else 0 for b in range(B)]
        ref.release([0] * B, end)
        dev.release([0] * B, end)
        for b in gone:
            ref.ctx[b] = 0
        dev.ctx = torch.tensor(ref.ctx, dtype=torch.int32, device="cuda")
        dev.same(ref)
        assert flags() == 0
        held = {p for row in ref.bt for p in row if p >= 0}
        assert len(held) + ref.pool[1] - ref.pool[0] == ref.n
    ref.release([0] * B, [maxp] * B)
    dev.release([0] * B, [maxp] * B)
    dev.same(ref)
    assert ref.pool[1] - ref.pool[0] == ref.n and not any(ref.refs)


def test_many_entries_and_holders(cuda_lib):
    """A page held by every row goes back once, at its last entry's place; entries spread over the cluster's CTAs."""
    B, maxp = 700, 64
    ref = Ref(2000, 16, B, maxp, seed=4)
    dev = Dev(ref)
    step(ref, dev, [64 * 16] + [0] * (B - 1), 1024)
    parents, counts = [-1] + [0] * (B - 1), [0] + [1 + i % 64 for i in range(B - 1)]
    ref.share(parents, counts)
    dev.share(parents, counts)
    dev.same(ref)
    ref.release([0] * B, [0] + [64] * (B - 1))
    dev.release([0] * B, [0] + [64] * (B - 1))
    dev.same(ref)
    ref.share(parents, counts)
    dev.share(parents, counts)
    ref.release([0] * B, [64] * B)
    dev.release([0] * B, [64] * B)
    dev.same(ref)
    assert flags() == 0


def test_bad_releases_and_parents(cuda_lib):
    ref = Ref(20, 16, 4, 5, seed=1)
    dev = Dev(ref)
    step(ref, dev, [40, 20, 0, 0], 60)
    # a page that nobody holds: flagged, not in the ring; rows out of bounds are left alone
    free_page = ref.ring[ref.pool[0] % ref.n]
    dev.bt[2, 0] = free_page
    dev.bt[2, 1] = 99
    pool, ring = dev.pool.clone(), dev.ring.clone()
    dev.release([0, -1, 0, 0], [6, 2, 2, -4])
    assert flags() == pa.PA_DEVERR_BAD_PAGE | pa.PA_DEVERR_BAD_LENGTH
    assert torch.equal(dev.pool, pool) and torch.equal(dev.ring, ring)
    dev.same(ref)
    # the same page twice in rows that count it once: returned once, flagged
    dev.bt[3, 0] = ref.bt[1][0]
    dev.release([0, 0, 0, 0], [0, 1, 0, 1])
    assert flags() == pa.PA_DEVERR_BAD_PAGE
    ref.release([0] * 4, [0, 1, 0, 0])
    dev.same(ref)
    for parents, counts in (([-1, 4, -1, -1], [0, 1, 0, 0]), ([-1, 0, -1, -1], [0, 6, 0, 0]),
                            ([-1, -1, 2, -1], [0, 0, 1, 0]), ([-1, 0, 1, -1], [0, 0, 1, 0])):
        dev.share(parents, counts)
        assert flags() == pa.PA_DEVERR_BAD_LENGTH
        dev.same(ref)


def test_the_host_manager_hands_out_the_same_pages(cuda_lib):
    """Without shared prefixes, the host block manager's tables and slots."""
    P, B, n = 16, 6, 64
    m = BlockManager(n, P)
    ref = Ref(n, P, B, 10)
    ref.ring = list(range(n))
    dev = Dev(ref)
    r = random.Random(1)
    prompts = [[r.randrange(1 << 30) for _ in range(k)] for k in (5, 16, 17, 40, 33, 1)]
    for b, tokens in enumerate(prompts):
        m.allocate(b, tokens)
    cu, pos, slots = dev.extend([len(x) for x in prompts], 112)
    for _ in range(40):
        tables, lens = m.block_tables(list(range(B)), 10, -1)
        assert tables.tolist() == dev.bt.tolist() and lens.tolist() == dev.ctx.tolist()
        assert m.slot_mapping(list(range(B)), [1] * B).tolist() == [slots[c - 1] for c in cu[1:]]
        for b in range(B):
            m.append_token(b, 7)
        cu, pos, slots = dev.extend([1] * B, B)
    for b in (3, 0):
        m.free(b)
        dev.release([0] * B, [10 if i == b else 0 for i in range(B)])
    dev.ctx[3] = dev.ctx[0] = 0
    m.allocate(100, list(range(60)))
    dev.extend([60, 0, 0, 0, 0, 0], 60)
    tables, _ = m.block_tables([100, 1, 2, 4, 5], 10, -1)
    assert tables.tolist() == dev.bt[[0, 1, 2, 4, 5]].tolist()
    assert flags() == 0


def test_graph_replay(cuda_lib):
    """A captured step takes its pages from the pool's state of each replay."""
    ref = Ref(200, 16, 8, 20, seed=2, start=77)
    dev = Dev(ref)
    new = torch.ones(8, dtype=torch.int32, device="cuda")
    cu = torch.zeros(9, dtype=torch.int32, device="cuda")
    pos, slots = torch.zeros(10, dtype=torch.int32, device="cuda"), torch.zeros(10, dtype=torch.int64, device="cuda")
    args = (dev.desc, 8, new, dev.ctx, dev.bt, dev.maxp, dev.ring, dev.pool, 10, cu, dev.ctx, pos, slots, dev.refs,
            dev.pool)
    win = (dev.desc, 40, 4, 8, dev.ctx, dev.bt, dev.maxp, dev.refs, dev.ring, dev.pool, dev.pool)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_extend_tables(*args)
        pa.pa_release_window_pages(*win)
    for i in range(100):
        new.fill_(i % 4)
        if i % 4 > 1:
            new[2:] = 0
        graph.replay()
        want = ref.extend(new.tolist(), 10)
        ref.release_window(40, 4)
        assert (cu.tolist(), pos.tolist(), slots.tolist()) == want[:3]
        dev.same(ref)
    assert flags() == 0
