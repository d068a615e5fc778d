"""Decode over a 4-bit cache against float64, each output held to a bound of its own: what its rounding steps can do to
it, whatever the rest of the batch holds.  Contexts that one CTA sums alone, queries and keys of unequal magnitude, keys
that take nearly all the weight, tokens whose loss would show."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_08_gb300 as pa
from oracle import q4_cache as q4

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda_lib")]

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24


class Batch:
    """A decode batch over a 4-bit cache of given K and V rows: k[b], v[b] are fp32 [len, hkv, hd], q [batch, hq, hd]."""

    def __init__(self, dtype, hkv, gs, P, q, k, v, scale=None, seed=0):
        rng = np.random.default_rng(seed)
        B, hq, hd = q.shape
        self.dtype, self.gs, self.hq, self.hkv, self.hd, self.P = dtype, gs, hq, hkv, hd, P
        self.lens = np.array([len(x) for x in k], np.int32)
        npg = -(-self.lens // P)
        self.pages, self.maxp = int(npg.sum()) + 1, int(npg.max())
        self.bt = np.full((B, self.maxp), self.pages - 1, np.int32)
        perm = rng.permutation(self.pages - 1)
        at = np.concatenate([[0], np.cumsum(npg)])
        self.slots = []
        for b in range(B):
            self.bt[b, : npg[b]] = perm[at[b]: at[b + 1]]
            t = np.arange(self.lens[b])
            self.slots.append(self.bt[b, t // P].astype(np.int64) * P + t % P)
        self.desc = pa.cache_desc(hq, hkv, hd, P, self.pages, DT[dtype])
        self.caches, self.vals = [], []
        for x in (k, v):
            cache = rng.integers(0, 256, (self.pages * P, q4.row_bytes(hkv, hd, gs))).astype(np.uint8)
            vals = []
            for b in range(B):
                u, s, c = q4.quantise(np.asarray(x[b], np.float32), gs)
                cache[self.slots[b]] = q4.pack_rows(u, s, c, self.slots[b])
                m = np.repeat(16 * s.astype(np.float64) + c.astype(np.float64), gs, -1)
                vals.append((q4.values(u, s, c, gs), m))    # the values, and of each what its code 0 stands for
            self.caches.append(torch.from_numpy(cache).cuda())
            self.vals.append(vals)
        self.q = torch.from_numpy(np.asarray(q, np.float32)).to(DT[dtype]).cuda()
        self.scale = hd ** -0.5 if scale is None else scale
        self.ctx, self.btd = torch.from_numpy(self.lens).cuda(), torch.from_numpy(self.bt).cuda()

    def decode(self, max_ctas=0):
        longest = int(self.lens.max())
        n = pa.pa_decode_q4_workspace_size(self.desc, self.gs, len(self.lens), longest, max_ctas)
        out = torch.full_like(self.q, 7.0)
        pa.pa_decode_q4(self.desc, self.gs, self.q, len(self.lens), *self.caches, self.btd, self.maxp, self.ctx,
                        longest, self.scale, max_ctas, out, torch.empty(n, dtype=torch.uint8, device="cuda"))
        return out.double().cpu().numpy()

    def reference(self):
        """Outputs in float64 and their bounds.

        With p the weights (sum 1), v = s u + m a value, u = 2^-24.  Rounding to nearest errs to either side, so errors
        of many terms add like their squares; eight times that is allowed, and what a few terms can do at most.

        bf16: the output is rounded (2^-8 of it); p and p s are float16 (2^-11 each), the first in sum and products
        alike: 2^-11 p (|v - o| + |s u|) a term.  The products' sums are fp32 numbers that the tensor cores may cut off
        (2^-23 of a sum for every 16 tokens, to one side): for the output and the softmax sum, which grow evenly, half of
        that on the average and half as many terms in each of two sums, 2^-24 of the output for every 16 tokens; and of
        p s u, summed over 512 tokens before the rest joins, U * 64 of its sum.

        fp32: the two sums of 16 tokens round a few times (16 u of p (|s u| + |m|)); o grows by one addition for every
        16 tokens, each u / 2 of what it has come to (at most about the largest output of the head); a weight is off by
        the exponential's 4 u and by its score's rounding, some 10 u: 64 u of sqrt(sum p^2) times the largest value."""
        outs, bounds = [], []
        q64 = self.q.double().cpu().numpy()
        for b in range(len(self.lens)):
            K, (V, M) = self.vals[0][b][0], self.vals[1][b]
            G = self.hq // self.hkv
            o, e = np.empty((self.hq, self.hd)), np.empty((self.hq, self.hd))
            for h in range(self.hq):
                v, m = V[:, h // G], M[:, h // G]
                t = K[:, h // G] @ q64[b, h] * self.scale
                p = np.exp(t - t.max())
                p /= p.sum()
                o[h] = p @ v
                su = np.abs(v - m)
                if self.dtype == "bf16":
                    term = p[:, None] * (np.abs(v - o[h]) + su)
                    e[h] = 2.0 ** -8 * (np.abs(o[h]) + np.sqrt((term ** 2).sum(0))) + U * (
                        -(-len(v) // 16) * np.abs(o[h]) + 64 * (p @ (su + np.abs(m))))
                else:
                    n = np.sqrt(-(-len(v) // 16))
                    e[h] = U * (16 * (p @ (su + np.abs(m))) / n + 2 * n * np.abs(o[h]).max()
                                + 64 * np.sqrt((p ** 2).sum()) * np.abs(v).max())
            outs.append(o)
            bounds.append(e)
        return np.stack(outs), np.stack(bounds)

    def check(self, *splits):
        ref, bound = self.reference()
        for max_ctas in splits:
            ratio = np.abs(self.decode(max_ctas) - ref) / bound
            assert np.isfinite(ratio).all()
            worst = ratio.reshape(len(self.lens), -1).max(1)
            assert worst.max() <= 1, (max_ctas, worst)
        assert pa.pa_read_device_errors(reset=True) == 0


def normal(rng, lens, hkv, hd):
    return [rng.standard_normal((n, hkv, hd)).astype(np.float32) for n in lens]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,hd,gs,P", [(4, 4, 128, 32, 16), (8, 2, 128, 64, 64), (7, 1, 128, 128, 32),
                                            (8, 4, 64, 32, 16), (5, 1, 64, 64, 128)])
@pytest.mark.parametrize("lens", [[64, 1000, 1, 17], [4096, 33, 20000]])
def test_every_output_is_within_its_own_bound(dtype, hq, hkv, hd, gs, P, lens):
    """Values without a mean, so that outputs shrink as the context grows, summed by one CTA and by many."""
    rng = np.random.default_rng(hq + hd + gs)
    c = Batch(dtype, hkv, gs, P, rng.standard_normal((len(lens), hq, hd)), normal(rng, lens, hkv, hd),
              normal(rng, lens, hkv, hd))
    c.check(1, 0, 7)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hd,gs", [(4, 128, 32), (3, 128, 64), (8, 128, 128), (2, 64, 32), (1, 64, 64)])
@pytest.mark.parametrize("mean", [0.0, 2.0])
def test_a_share_of_a_hundred_thousand_tokens(dtype, hq, hd, gs, mean):
    rng = np.random.default_rng(hd + gs)
    lens = [100000, 40007]
    v = [x + np.float32(mean) for x in normal(rng, lens, 1, hd)]
    c = Batch(dtype, 1, gs, 64, rng.standard_normal((2, hq, hd)), normal(rng, lens, 1, hd), v)
    c.check(1, 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gs", [32, 64])
@pytest.mark.parametrize("ratio", [8, 11, 14])
def test_groups_of_unequal_query_magnitude(dtype, gs, ratio):
    """The queries of a head's first group are 2^ratio times the others', its keys as much smaller: every group counts
    alike in a score."""
    rng = np.random.default_rng(ratio)
    lens = [500, 77, 3000]
    a = np.full(128, 2.0 ** (-ratio / 2))
    a[:gs] = 2.0 ** (ratio / 2)
    k = [(x / a).astype(np.float32) for x in normal(rng, lens, 2, 128)]
    c = Batch(dtype, 2, gs, 16, rng.standard_normal((3, 6, 128)) * a, k, normal(rng, lens, 2, 128))
    c.check(1, 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_keys_far_below_the_largest_score_still_add_up(dtype):
    """One key's weight is 2^25 times each other's, of which there are 200000: together they hold half a percent."""
    n, hd = 200000, 64
    k, v = np.zeros((n, 1, hd), np.float32), np.ones((n, 1, hd), np.float32)
    k[1000], v[1000] = 25.2 * np.log(2) / 8, 0.0
    c = Batch(dtype, 1, 64, 256, np.ones((1, 4, hd)), [k], [v])
    c.check(1, 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("first", [True, False])
def test_values_far_below_the_largest_scale(dtype, first):
    """One token's values are 2^18 times the others', its weight next to nothing: the others' outputs keep their bits."""
    rng = np.random.default_rng(3)
    lens = [2000, 300]
    q = rng.standard_normal((2, 4, 128))
    k, v = normal(rng, lens, 2, 128), normal(rng, lens, 2, 128)
    for b in range(2):
        at = 0 if first else lens[b] // 2
        v[b] = v[b] * np.float32(2.0 ** -8)
        v[b][at] *= np.float32(2.0 ** 18)
        for h in range(2):
            k[b][at, h] = -60 * q[b, 2 * h: 2 * h + 2].sum(0) / 128      # scores of -100 and below
    c = Batch(dtype, 2, 64, 16, q, k, v, scale=0.18)
    c.check(1, 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,hd,gs,P", [(16, 8, 128, 32, 16), (8, 2, 128, 128, 64), (6, 2, 64, 64, 16)])
@pytest.mark.parametrize("lens,splits", [([20011, 1, 9000], (0, 1, 2, 31)), ([700, 33, 1000, 0, 65] * 5, (0, 1, 3, 24)),
                                         ([1000, 300, 31] * 50, (0, 7, 152))])
def test_every_chunk_counts_once(dtype, hq, hkv, hd, gs, P, lens, splits):
    """One token of every 32 has a value of 40 in a dim of its own (as many dims as the head has, in turn): a chunk lost
    or taken twice changes some dim's output by a good part of it, whatever the rest of the batch holds."""
    if max(lens) > 5000 and hkv == 8 and dtype == "f32":
        lens = [5011, 1, 3000]
    rng = np.random.default_rng(hd + gs)
    live = [n for n in lens if n]
    k, v = normal(rng, live, hkv, hd), normal(rng, live, hkv, hd)
    for b, n in enumerate(live):
        k[b] *= np.float32(0.3)
        v[b] *= np.float32(0.1)
        for i in range(0, -(-n // 32)):
            v[b][min(n - 1, 32 * i + int(rng.integers(32))), :, i % hd] += np.float32(40)
    c = Batch(dtype, hkv, gs, P, rng.standard_normal((len(live), hq, hd)), k, v)
    c.check(*splits)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd", [64, 128])
def test_rotary_angles_at_any_position(dtype, hd):
    """Positions up to the largest that an int32 holds.  A sine or cosine that rounds to its other neighbour moves a value
    by an ulp of its pair's size (2^-23, bf16 2^-7); the angle in 64 bits is off by two roundings, 2^-52 of it each."""
    from test_gpu_q4_cache import plain_norm_rope

    dt = DT[dtype]
    far = [131071, 131072, 140001, 200003, (1 << 20) + 3, (1 << 24) - 1, (1 << 24) + 1, (1 << 24) + 3, (1 << 27) + 5,
           (1 << 30) + 77, (1 << 31) - 1]
    n, heads = len(far), 4
    desc = pa.cache_desc(heads, heads, hd, 16, 4, dt)
    g = torch.Generator(device="cuda").manual_seed(2)
    x, w = torch.randn(n, heads, hd, generator=g, device="cuda").to(dt), torch.ones(hd, dtype=dt, device="cuda")
    pos = torch.tensor(far, dtype=torch.int32, device="cuda")
    slots = torch.arange(n, dtype=torch.int64, device="cuda")
    out, row = torch.zeros_like(x), heads * hd
    caches = [torch.zeros(4 * 16, pa.pa_q4_row_bytes(desc, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
    pa.pa_qk_norm_rope_kv_write_q4(desc, 64, x, row, x, row, x, row, n, pos, w, w, 1e-6, 1e4, slots, out, *caches)
    got, want = out.double(), plain_norm_rope(x, w, pos, 1e-6, 1e4).double()
    h = hd // 2
    size = torch.hypot(want[..., :h], want[..., h:])
    size = torch.cat([size, size], -1)
    bound = size * ((2.0 ** -7 if dtype == "bf16" else 2.0 ** -22) + 2.0 ** -51 * pos.double()[:, None, None])
    worst = ((got - want).abs() / bound).amax((1, 2))
    assert (worst <= 1).all(), dict(zip(far, worst.tolist()))
