"""Prefill over tables that name pages out of range: what the step before left in shared memory takes no part."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_gqa_08_gb300 as pa

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda_lib")]


def close(a, b):
    """Two answers of the tensor-core prefill to the same question.  Rows past a request's last share the other rows'
    reference of the exponentials, so equal inputs may round differently: bf16 outputs (2^-8 of each) of bf16
    probabilities (2^-8 of each, random: of unit values over tens of keys, below 2^-8 in all)."""
    a, b = a.double(), b.double()
    return bool(((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -8).all())


@pytest.mark.parametrize("planned", [False, True])
@pytest.mark.parametrize("hq,hkv,P", [(16, 8, 16), (8, 2, 64), (7, 1, 256)])
def test_tensor_core_prefill_takes_rows_of_bad_pages_as_zeros(hq, hkv, P, planned):
    hd, B, maxp, new = 128, 3, 768 // P, [40, 1, 150]
    ctx = [700, 500, 155]
    rng = np.random.default_rng(P)
    pages = B * maxp
    desc = pa.cache_desc(hq, hkv, hd, P, pages, torch.bfloat16)
    bt = rng.permutation(pages).reshape(B, maxp).astype(np.int32)
    cache = [torch.from_numpy(rng.standard_normal((pages, P, hkv, hd)).astype(np.float32)).bfloat16().cuda()
             for _ in range(2)]
    n = sum(new)
    q = torch.from_numpy(rng.standard_normal((n, hq, hd)).astype(np.float32)).bfloat16().cuda()
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    ws = None
    if planned:
        ws = torch.empty(pa.pa_prefill_workspace_size(desc, B, 150, n, 700), dtype=torch.uint8, device="cuda")

    def run(tables, caches):
        out = torch.full_like(q, 7.0)
        pa.pa_prefill_varlen(desc, q, torch.from_numpy(cu).cuda(), B, 150, n, *caches, torch.from_numpy(tables).cuda(),
                             maxp, torch.tensor(ctx, dtype=torch.int32, device="cuda"), 700, hd ** -0.5, out, ws)
        return out, pa.pa_read_device_errors(reset=True)

    bad = bt.copy()
    bad[0, 1], bad[0, 699 // P], bad[2, :] = pages, -1, 1 << 30    # inside a context, its ragged end, a whole request
    pa.pa_read_device_errors(reset=True)
    first = None
    for fill in (float("nan"), 1e4):
        run(bt, [torch.full_like(x, fill) for x in cache])         # leaves such rows in shared memory
        out, flags = run(bad, cache)
        assert flags == pa.PA_DEVERR_BAD_PAGE
        assert first is None or close(out, first)
        first = out
    got = first.double().cpu().numpy()
    assert (got[cu[2]:] == 0).all()
    raw = [x.double().cpu().numpy().reshape(pages * P, hkv, hd) for x in cache]
    for b in range(2):
        t = np.arange(ctx[b])
        page = bad[b, t // P]
        ok = (page >= 0) & (page < pages)
        K, V = (np.where(ok[:, None, None], x[np.where(ok, page, 0).astype(np.int64) * P + t % P], 0.0) for x in raw)
        r = slice(cu[b], cu[b + 1])
        ref = oracle.attend(q[r].double().cpu().numpy(), K, V, np.arange(ctx[b] - new[b], ctx[b]), hd ** -0.5)[0]
        # probabilities and outputs in bf16: 2^-8 of each
        assert np.abs(got[r] - ref).max() <= 2 * 2.0 ** -8 * np.abs(ref).max() + 2.0 ** -8 * np.abs(V).max() / np.sqrt(ctx[b])
