"""Planned prefill of head groups that do not divide a tile's 128 rows: the rows behind a tile's last token belong to no
token of its own, whatever order the parts are merged in."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_gqa_08_gb300 as pa

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda_lib")]


@pytest.mark.parametrize("G,hkv,new,ctx", [(3, 1, [90, 200], [1500, 900]), (5, 2, [60, 1], [1400, 300]),
                                           (6, 1, [50, 64], [1000, 1000]), (7, 1, [40, 1, 150], [700, 500, 155])])
def test_split_key_ranges_of_odd_groups(G, hkv, new, ctx):
    hd, P, B, n = 128, 16, len(new), sum(new)
    rng = np.random.default_rng(G)
    maxp = -(-max(ctx) // P)
    pages = B * maxp
    desc = pa.cache_desc(G * hkv, hkv, hd, P, pages, torch.bfloat16)
    bt = rng.permutation(pages).reshape(B, maxp).astype(np.int32)
    cache = [torch.from_numpy(rng.standard_normal((pages, P, hkv, hd)).astype(np.float32)).bfloat16().cuda()
             for _ in range(2)]
    q = torch.from_numpy(rng.standard_normal((n, G * hkv, hd)).astype(np.float32)).bfloat16().cuda()
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    ws = torch.zeros(pa.pa_prefill_workspace_size(desc, B, max(new), n, max(ctx)), dtype=torch.uint8, device="cuda")
    raw = [x.double().cpu().numpy().reshape(pages * P, hkv, hd) for x in cache]
    refs = []
    for b in range(B):
        t = np.arange(ctx[b])
        at = bt[b, t // P].astype(np.int64) * P + t % P
        refs.append(oracle.attend(q[cu[b]: cu[b + 1]].double().cpu().numpy(), raw[0][at], raw[1][at],
                                  np.arange(ctx[b] - new[b], ctx[b]), hd ** -0.5)[0])
    ref = np.concatenate(refs)
    args = [torch.from_numpy(x).cuda() for x in (cu, bt)] + [torch.tensor(ctx, dtype=torch.int32, device="cuda")]
    for fill in (7.0, float("nan"), 0.0, 1.0, 2.0):
        ws.random_()          # what a workspace held before takes no part
        out = torch.full_like(q, fill)
        pa.pa_prefill_varlen(desc, q, args[0], B, max(new), n, *cache, args[1], maxp, args[2], max(ctx), hd ** -0.5, out,
                             ws)
        torch.cuda.synchronize()
        assert ws[:16].view(torch.int32)[1] > 0        # some pair is split
        # outputs in bf16 (2^-8 of each) of probabilities in bf16 (2^-8 of each, random: of unit values over tens of
        # keys, or of the few keys that the first tokens of a whole prompt see, below 2^-7 in all)
        err = np.abs(out.double().cpu().numpy() - ref)
        assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -7).all(), err.max()
    assert pa.pa_read_device_errors(reset=True) == 0
