"""Plain attention in 64 bits over the keys that a mask leaves, with a bound for each output of a kernel that works in
32 bits and rounds its probabilities and outputs to the type; and paged caches to run the kernels on.

The bound of an output o = sum_j p_j v_j, with A = sum_j p_j |v_j|:
  output rounding    h |o|                 h = 2^-8 for bf16, 2^-24 for fp32
  probabilities      h A                   bf16 kernels round each p_j to bf16 for the product (the sum keeps 32 bits)
  scores             2 e A                 e: error of an exponent, hd + 2 roundings of 2^-24 of scale * sum_d |q_d k_d|
                                           (the largest of the row), in the numerator and in the sum
  exp2               2 * 2^-21 A           ex2.approx (2^-22) and the rounding of its argument's maximum
  sums               2 (n / 8 + 40) 2^-24 A  additions in a row of n keys (chunks of 16 tokens and more, two or four terms of
                                           each added first, parts merged), numerator and sum; fp32 kernels add single
                                           tokens of a lane: a quarter of the keys at least
"""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def attend(q, K, V, seen, scale, dt):
    """q [n, Hq, hd], K and V [m, Hkv, hd], seen [n, m] (bool) -> float64 outputs and their bounds, [n, Hq, hd].
    Rows that see nothing give NaN."""
    n, Hq, hd = q.shape
    m, Hkv, _ = K.shape
    q = q.double().reshape(n, Hkv, Hq // Hkv, hd)
    K = torch.where(seen.any(0)[:, None, None], K.double(), 0.0)
    V = torch.where(seen.any(0)[:, None, None], V.double(), 0.0)
    s = torch.einsum("nhgd,mhd->nhgm", q, K) * scale
    big = torch.einsum("nhgd,mhd->nhgm", q.abs(), K.abs()) * abs(scale)
    mask = seen[:, None, None, :]
    p = torch.softmax(s.masked_fill(~mask, float("-inf")), -1)
    big = big.masked_fill(~mask, 0.0).amax(-1, keepdim=True)
    o = torch.einsum("nhgm,mhd->nhgd", p, V)
    A = torch.einsum("nhgm,mhd->nhgd", p, V.abs())
    h = HALF[dt]
    e = (hd + 2) * 2.0 ** -24 * big
    keys = seen.sum(1).double()[:, None, None, None]
    sums = (keys / (8 if dt == torch.bfloat16 else 4) + 40) * 2.0 ** -24
    bound = h * o.abs() + (h if dt == torch.bfloat16 else 0.0) * A + 2 * (e + 2.0 ** -21 + sums) * A
    # first-order terms; their products are below a hundredth of them for the scores of these tests
    return o.reshape(n, Hq, hd), 1.01 * bound.reshape(n, Hq, hd)


def check(got, ref, bound, what=""):
    err = (got.double() - ref).abs()
    worst = (err / bound).max().item() if err.numel() else 0.0
    assert not torch.isnan(got.double()).any(), f"{what}: NaN"
    assert worst <= 1.0, f"{what}: {worst:.3g} bounds off"
    return worst


class Paged:
    """A paged cache filled with `fill` but for the tokens that are put into it, on pages in random order."""

    def __init__(self, lens, Hq, Hkv, hd, P, dt, seed, fill=float("nan"), dev="cuda", spare=3):
        from paged_kv_gqa_08_gb300 import cache_desc
        self.g = torch.Generator(device=dev).manual_seed(seed)
        self.lens, self.P, self.dt, self.dev = list(lens), P, dt, dev
        pages = [-(-max(L, 0) // P) for L in lens]
        self.maxp = max(max(pages, default=1), 1)
        total = sum(pages)
        self.num_pages = total + spare
        self.desc = cache_desc(Hq, Hkv, hd, P, self.num_pages, dt)
        perm = torch.randperm(self.num_pages, generator=self.g, device=dev).to(torch.int32)
        self.bt = torch.full((len(pages), self.maxp), -1, dtype=torch.int32, device=dev)
        at = 0
        for b, n in enumerate(pages):
            self.bt[b, :n] = perm[at: at + n]
            at += n
        self.k = torch.full((self.num_pages, P, Hkv, hd), fill, dtype=dt, device=dev)
        self.v = self.k.clone()
        self.K, self.V = [], []
        for b, L in enumerate(lens):
            L = max(L, 0)
            K, V = (torch.randn(L, Hkv, hd, generator=self.g, device=dev).to(dt) for _ in range(2))
            self.K.append(K)
            self.V.append(V)
            self.put(b, torch.arange(L, device=dev), K, V)
        self.ctx = torch.tensor(self.lens, dtype=torch.int32, device=dev)

    def put(self, b, j, K, V):
        page = self.bt[b][j // self.P].long()
        self.k[page, j % self.P] = K
        self.v[page, j % self.P] = V

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g, device=self.dev).to(self.dt)
