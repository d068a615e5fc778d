"""Pages handed back out of long tables, most of whose entries are -1 already: entries in runs and alone, held pages below
and above them, pages that rows share, against the rules in Python."""
import random

import pytest
import torch

import paged_kv_gqa_08_gb300 as pa
from test_gpu_tables import Dev, Ref, flags

pytestmark = pytest.mark.gpu


def sparse(B, maxp, P, held, seed):
    """Tables in which about `held` of the entries, in runs of any length, name pages; some pages in several rows."""
    r = random.Random(seed)
    rows, n = [], 0
    for _ in range(B):
        row, j = [-1] * maxp, 0
        while j < maxp:
            run = int(2 ** r.uniform(0, 9))
            if r.random() < held:
                for i in range(j, min(j + run, maxp)):
                    row[i] = n
                    n += 1
            j += run
        rows.append(row)
    pages = list(range(n))
    r.shuffle(pages)
    ref = Ref(n + 50, P, B, maxp, seed=seed, start=1 << 33)
    for b, row in enumerate(rows):
        for j, i in enumerate(row):
            if i >= 0:  # a page of its own, or (one in ten) another entry's
                page = pages[i] if r.random() < 0.9 else pages[r.randrange(n)]
                ref.bt[b][j] = page
                ref.refs[page] += 1
    free = [p for p, c in enumerate(ref.refs) if c == 0]
    ref.pool = [(1 << 33) + ref.n - len(free), (1 << 33) + ref.n]
    ref.ring = [0] * ref.n
    for i, p in enumerate(free):
        ref.ring[(ref.pool[0] + i) % ref.n] = p
    ref.ctx = [int(maxp * P * r.uniform(0.2, 0.6)) for _ in range(B)]
    return ref, Dev(ref, alias=seed % 2 == 0)


@pytest.mark.parametrize("B,maxp", [(1, 30000), (3, 9001), (40, 3001), (700, 200)])
@pytest.mark.parametrize("held", [0.03, 0.5])
def test_windows_leave_pages_of_sparse_tables(cuda_lib, B, maxp, held):
    ref, dev = sparse(B, maxp, 16, held, seed=B)
    r = random.Random(B)
    for _ in range(6):
        window, sinks = r.choice([1, 100, 5000]), r.choice([0, 5, 300])
        ref.release_window(window, sinks)
        dev.release_window(window, sinks)
        dev.same(ref)
        ref.ctx = [min(L + r.choice([0, 1, 16, 700]), maxp * 16) for L in ref.ctx]
        dev.ctx = torch.tensor(ref.ctx, dtype=torch.int32, device="cuda")
    assert flags() == 0
    ref.release([0] * B, [maxp] * B)
    dev.release([0] * B, [maxp] * B)
    dev.same(ref)
    assert ref.pool[1] - ref.pool[0] == ref.n and flags() == 0


def test_entries_that_are_none_become_minus_one(cuda_lib):
    """Negative entries are passed over, entries beyond the pages flagged; all of them are -1 afterwards."""
    ref, dev = sparse(30, 3000, 16, 0.0, seed=2)
    for b, j, page in ((0, 17, -5), (3, 2999, -(1 << 31)), (29, 0, ref.n), (29, 1500, (1 << 31) - 1)):
        dev.bt[b, j] = page
    dev.release([0] * 30, [3000] * 30)
    assert flags() == pa.PA_DEVERR_BAD_PAGE
    ref.release([0] * 30, [3000] * 30)
    dev.same(ref)
