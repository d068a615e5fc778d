"""Cases of the 4-bit paged KV cache: quantised writes, read-back, decode attention.

A cache row (one token, all kv-heads) holds 4-bit codes and, per kv-head and
group of ``gs`` dimensions, two float16 numbers s and c; a code u stands for
``s * (16 + u) + c``.  With mn and mx the least and largest value of a group,

    s = float16((mx - mn) / 15),  c = float16(mn - 16 s),
    16 + u = clamp(rint((x - c) / s), 16, 31)        (s = 0: u = 0)

``(mx - mn) / 15`` is the product with the fp32 number nearest to 1/15 and the
last quotient the product with the fp32 number nearest to 1/s, as the operator
defines them; values beyond +-16384 count as +-16384, and a group with a NaN
or an infinity has c = NaN.  Row layout: ``Hkv * hd / 2`` bytes of codes, then
``Hkv * hd / gs`` words (s low, c high half) padded to 16 bytes.  In each of
the two parts, within blocks of up to 128 bytes, the 16-byte piece j of slot t
lies at piece ``j ^ (t mod pieces)``.  16 bits of codes hold four consecutive
dimensions: u0 in bits 6-9, u1 in bits 14, 15, 0, 1, u2 in bits 2-5, u3 in
bits 10-13.

The kinds of pass:
  chunk   a prefill chunk's K/V rows are quantised into the cache, then the
          whole context is read back to rows (what chunked prefill attends to)
  norm    the same with the q/k RMSNorm and rotary embedding in the write
  read    a context is read back
  decode  one query per request attends to the 4-bit cache
  step    decode with the new token's K/V row quantised into the cache by the
          same call; the new rows are read back as the updated state
"""
import math

import numpy as np
import torch

own = False

NORM_EPS = 1e-6
ROPE_THETA = 1e6
KINDS = ("chunk", "norm", "read", "decode", "step")


def _case(name, kind, **kw):
    c = dict(name=name, kind=kind, dtype="bf16", B=1, Hq=16, Hkv=8, hd=128, P=16, gs=32, new_lo=1, new_hi=1,
             ctx_lo=1, ctx_hi=1, tail=False, lens=1)
    c.update(kw)
    return c


def listed():
    return [
        # one short prompt chunk of a single chat turn: latency
        _case("chunk_one", "chunk", B=1, new_lo=33, new_hi=33, ctx_lo=233, ctx_hi=233, lens=1),
        # eight requests in mixed chunked prefill, prefixes up to 4096 (Qwen3-0.6B heads, small pages)
        _case("chunk_mix", "chunk", B=8, new_lo=1, new_hi=512, ctx_lo=600, ctx_hi=4608, lens=2),
        # 2048 new tokens over 2048 cached, eight requests, with the model's q/k norm and rotary
        _case("norm_2k", "norm", B=8, new_lo=2048, new_hi=2048, ctx_lo=4096, ctx_hi=4096, gs=64, lens=3),
        # a decode batch's new tokens, normed, rotated, written, and only those rows read back
        _case("norm_tokens", "norm", B=256, ctx_lo=128, ctx_hi=2048, tail=True, lens=4),
        # contexts handed to another engine or staged for prefill: long, large pages, one scale per head
        _case("read_long", "read", B=16, ctx_lo=1024, ctx_hi=16384, P=256, gs=128, lens=5),
        # small fp32 model, odd lengths
        _case("read_f32", "read", dtype="f32", B=5, Hq=4, Hkv=2, hd=64, ctx_lo=1, ctx_hi=701, lens=6),
        # tiny fp32 decode, lengths down to a few tokens
        _case("decode_tiny_f32", "decode", dtype="f32", B=4, Hq=4, Hkv=2, hd=64, ctx_lo=5, ctx_hi=64, lens=7),
        # Qwen3-0.6B-shaped decode batch
        _case("decode_0p6b", "decode", B=256, ctx_lo=128, ctx_hi=2048, lens=8),
        # Qwen3-8B-shaped decode batch, large pages
        _case("decode_8b", "decode", B=64, Hq=32, P=256, gs=64, ctx_lo=1024, ctx_hi=8192, lens=9),
        # few long contexts: the key range of each request is split
        _case("decode_long", "decode", B=8, Hq=32, P=256, gs=128, ctx_lo=32768, ctx_hi=32768, lens=10),
        # two users' decode step: latency
        _case("step_two", "step", B=2, ctx_lo=301, ctx_hi=905, lens=11),
        # a step with groups of six q-heads, 64 dimensions, an odd batch
        _case("step_odd", "step", B=37, Hq=24, Hkv=4, hd=64, P=64, gs=64, ctx_lo=100, ctx_hi=2900, lens=12),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(KINDS)
    hd = rng.choice((64, 128, 128))
    hkv = rng.choice((1, 2, 4, 8, 8))
    g = rng.choice((1, 2, 3, 4, 5, 6, 7, 8))
    c = _case("", kind, dtype=rng.choice(("bf16", "bf16", "bf16", "f32")), Hq=hkv * g, Hkv=hkv, hd=hd,
              P=rng.choice((16, 32, 64, 128, 256)), gs=rng.choice([s for s in (32, 64, 128) if s <= hd]),
              lens=rng.randrange(1, 1 << 30))
    c["B"] = _spread(rng, 1, 256 if kind in ("decode", "step") else 24)
    # at most 160k context tokens in all where they are attended to, 100k where they are read back, 24k for fp32
    total = 24000 if c["dtype"] == "f32" else 160000 if kind in ("decode", "step") else 100000
    top = max(2, min(32768, total // c["B"]))
    c["ctx_hi"] = _spread(rng, 2, top)
    c["ctx_lo"] = _spread(rng, 1, c["ctx_hi"])
    if kind in ("chunk", "norm"):
        c["new_hi"] = _spread(rng, 1, min(2048, 16384 // c["B"], c["ctx_hi"]))
        c["new_lo"] = _spread(rng, 1, c["new_hi"])
        c["tail"] = rng.random() < 0.3
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# sizes of a case
# ---------------------------------------------------------------------------
def _lens(c):
    """Context lengths (with the new tokens) and new-token counts of the requests: both ends of the ranges occur."""
    r = np.random.RandomState(c["lens"])
    ctx = r.randint(c["ctx_lo"], c["ctx_hi"] + 1, c["B"])
    new = r.randint(c["new_lo"], c["new_hi"] + 1, c["B"])
    ctx[0], ctx[-1] = c["ctx_lo"], c["ctx_hi"]
    new[0], new[-1] = c["new_lo"], c["new_hi"]
    if c["kind"] == "read" or c["kind"] == "decode":
        new[:] = 0
    return ctx, np.minimum(new, ctx)


def _row_bytes(c):
    par = c["Hkv"] * (c["hd"] // c["gs"]) * 4
    return c["Hkv"] * c["hd"] // 2 + (par + 15) // 16 * 16


def work(c):
    ctx, new = _lens(c)
    e = 2 if c["dtype"] == "bf16" else 4
    row, heads = _row_bytes(c), c["Hkv"] * c["hd"]
    tokens, n = int(ctx.sum()), int(new.sum())
    pages = int(sum(-(-x // c["P"]) for x in ctx))
    nbytes, flops = 4 * pages, 0
    if n:
        nbytes += 2 * n * (heads * e + row)  # new rows in, cache rows out
        flops += 2 * n * heads * 8           # difference, product, rounding, clamps, minimum and maximum
    if c["kind"] == "norm":
        nbytes += 2 * n * c["Hq"] * c["hd"] * e
        flops += n * (c["Hq"] + c["Hkv"]) * c["hd"] * 10
    if c["kind"] in ("decode", "step"):
        # the new rows of a step are attended to as they come: not read from the cache again
        nbytes += 2 * (tokens - n) * row + 2 * c["B"] * c["Hq"] * c["hd"] * e
        flops += 4 * c["Hq"] * c["hd"] * tokens
    if c["kind"] != "decode":
        rows = n if (c["tail"] or c["kind"] == "step") else tokens
        # rows written in this pass need not come from memory again
        nbytes += 2 * (rows - n) * row + 2 * rows * heads * e if rows >= n else 2 * rows * heads * e
        flops += 2 * rows * heads * 2
    return {"bytes": float(nbytes), "flops": float(flops)}


# ---------------------------------------------------------------------------
# plain form: the packed rows
# ---------------------------------------------------------------------------
def _swizzle(part, slots):
    """Move the 16-byte pieces of `part` [n, bytes] to (or from: it is its own inverse) their places for `slots`."""
    n, size = part.shape
    pieces = min(8, size // 16)
    if pieces < 2:
        return part
    j = torch.arange(pieces, device=part.device)[None, :] ^ (slots[:, None] % pieces)
    p = part.reshape(n, size // (16 * pieces), pieces, 16)
    return torch.gather(p, 2, j[:, None, :, None].expand(-1, p.shape[1], -1, 16)).reshape(n, size)


def _params(x, c):
    """s, c (float16) of the groups of x [n, Hkv, hd] fp32, and x clamped, as [n, Hkv, groups, gs]."""
    x = x.reshape(x.shape[0], c["Hkv"], c["hd"] // c["gs"], c["gs"])
    good = torch.isfinite(x).all(-1)
    x = torch.where(good[..., None], x, torch.zeros_like(x)).clamp(-16384.0, 16384.0)
    mn, mx = x.amin(-1), x.amax(-1)
    s = ((mx - mn) * torch.tensor(1.0 / 15.0, dtype=torch.float32, device=x.device)).to(torch.float16)
    o = (mn - 16.0 * s.float()).to(torch.float16)
    return torch.where(good, s, 0.0), torch.where(good, o, float("nan")), x


def _pack(x, c, slots):
    """Cache rows (uint8) of fp32 K or V rows x [n, Hkv * hd]."""
    n = x.shape[0]
    s, o, x = _params(x, c)
    sf, of = s.float()[..., None], o.float()[..., None]
    r = torch.where(sf > 0, 1.0 / sf, torch.zeros_like(sf))
    u = torch.nan_to_num(torch.round((x - of) * r)).clamp(16.0, 31.0).to(torch.int32) - 16
    u = torch.where(sf > 0, u, torch.zeros_like(u)).reshape(n, -1, 4)
    h = (u[..., 0] << 6) | (u[..., 2] << 2) | (u[..., 3] << 10) | ((u[..., 1] & 3) << 14) | (u[..., 1] >> 2)
    codes = torch.stack([h & 255, h >> 8], -1).to(torch.uint8).reshape(n, -1)
    par = torch.stack([s, o], -1).reshape(n, -1).view(torch.uint8).reshape(n, -1)
    par = torch.nn.functional.pad(par, (0, -par.shape[1] % 16))
    return torch.cat([_swizzle(codes, slots), _swizzle(par, slots)], 1)


def _unpack(rows, c, slots):
    """fp32 values [n, Hkv, hd] of cache rows [n, row bytes] that lie in `slots`."""
    n, nc = rows.shape[0], c["Hkv"] * c["hd"] // 2
    b = _swizzle(rows[:, :nc], slots).reshape(n, -1, 2).to(torch.int32)
    h = b[..., 0] | (b[..., 1] << 8)
    u = torch.stack([(h >> 6) & 15, ((h >> 14) & 3) | ((h & 3) << 2), (h >> 2) & 15, (h >> 10) & 15], -1)
    groups = c["hd"] // c["gs"]
    par = _swizzle(rows[:, nc:], slots)[:, : c["Hkv"] * groups * 4].contiguous().view(torch.float16)
    par = par.reshape(n, c["Hkv"], groups, 1, 2).float()
    u = u.reshape(n, c["Hkv"], groups, c["gs"])
    return (par[..., 0] * (16 + u).float() + par[..., 1]).reshape(n, c["Hkv"], c["hd"])


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(c, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    ctx, new = _lens(c)
    B, P, heads, row = c["B"], c["P"], c["Hkv"] * c["hd"], _row_bytes(c)
    npg = -(-ctx // P)
    maxp = int(npg.max())
    total = int(npg.sum())
    num_pages = total + 1 + total // 16
    # physical pages in random order; the tables' unused entries name the last page
    perm = torch.randperm(num_pages - 1, generator=g, device=dev).to(torch.int32)
    bt = torch.full((B, maxp), num_pages - 1, dtype=torch.int32, device=dev)
    used = torch.arange(maxp, device=dev)[None, :] < torch.tensor(npg, device=dev)[:, None]
    bt[used] = perm[:total]

    tok_b = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(ctx, device=dev))
    first = torch.tensor(np.concatenate([[0], np.cumsum(ctx)]), device=dev)
    pos = torch.arange(int(ctx.sum()), device=dev) - first[tok_b]
    slots = bt[tok_b, pos // P].long() * P + pos % P
    ctx_t, new_t = torch.tensor(ctx, device=dev), torch.tensor(new, device=dev)
    is_new = pos >= (ctx_t - new_t)[tok_b]
    q_tokens = int(new.sum()) if c["kind"] == "norm" else B

    def rows(n):
        # K and V as a model has them: unit variance, a few dimensions of a head with an offset of their own
        off = torch.randn(heads, generator=g, device=dev) * 3.0
        off = torch.where(torch.rand(heads, generator=g, device=dev) < 1 / 16, off, torch.zeros_like(off))
        return (torch.randn(n, heads, generator=g, device=dev) + off).to(dt)

    # the caches start with what freed pages hold: any bytes
    caches = []
    for _ in range(2):
        cache = torch.randint(0, 256, (num_pages * P, row), generator=g, device=dev, dtype=torch.uint8)
        old = slots[~is_new]
        if old.numel():
            cache[old] = _pack(rows(old.numel()).float(), c, old)
        caches.append(cache)
    n = int(new.sum())
    read_n = new if (c["tail"] or c["kind"] == "step") else ctx
    cu_read = torch.tensor(np.concatenate([[0], np.cumsum(read_n)]), dtype=torch.int32, device=dev)
    reads = int(read_n.sum())
    s = {
        "c": dict(c), "dt": dt, "num_pages": num_pages, "maxp": maxp, "max_ctx": int(ctx.max()), "n": n,
        "reads": reads, "k_cache": caches[0], "v_cache": caches[1], "bt": bt,
        "ctx": ctx_t.to(torch.int32), "slots": slots[is_new].contiguous(),
        "positions": pos[is_new].to(torch.int32), "cu_read": cu_read,
        "starts": torch.tensor(ctx - read_n, dtype=torch.int32, device=dev),
        "q": torch.randn(q_tokens, c["Hq"], c["hd"], generator=g, device=dev).to(dt),
        "k": rows(n), "v": rows(n), "scale": c["hd"] ** -0.5,
        "wq": (1 + 0.1 * torch.randn(c["hd"], generator=g, device=dev)).to(dt),
        "wk": (1 + 0.1 * torch.randn(c["hd"], generator=g, device=dev)).to(dt),
        "k_out": torch.zeros(reads, heads, dtype=dt, device=dev),
        "v_out": torch.zeros(reads, heads, dtype=dt, device=dev),
        "q_out": torch.zeros(q_tokens, c["Hq"], c["hd"], dtype=dt, device=dev),
        "out": torch.zeros(B, c["Hq"], c["hd"], dtype=dt, device=dev),
        "slot_out": torch.zeros(B, dtype=torch.int64, device=dev),
        # a serving program's decode workspace, sized once for its largest step
        "ws": torch.empty(128 << 20, dtype=torch.uint8, device=dev) if c["kind"] in ("decode", "step") else None,
    }
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _token_slots(s, first, count):
    """Slots of tokens first[b] .. first[b] + count[b] - 1 of each request, packed, and their requests."""
    P, dev = s["c"]["P"], s["bt"].device
    b = torch.repeat_interleave(torch.arange(count.numel(), device=dev), count.long())
    start = torch.cumsum(count, 0) - count
    pos = torch.arange(b.numel(), device=dev) - start[b] + first[b]
    return s["bt"][b, pos // P].long() * P + pos % P, b


def _plain_read(s):
    slots, _ = _token_slots(s, s["starts"], s["cu_read"][1:] - s["cu_read"][:-1])
    c, dt = s["c"], s["dt"]
    return {"k": _unpack(s["k_cache"][slots], c, slots).flatten(1).to(dt),
            "v": _unpack(s["v_cache"][slots], c, slots).flatten(1).to(dt)}


def _plain_write(s, k):
    s["k_cache"][s["slots"]] = _pack(k.float(), s["c"], s["slots"])
    s["v_cache"][s["slots"]] = _pack(s["v"].float(), s["c"], s["slots"])


def _plain_norm_rope(x, w, positions, dt):
    """RMSNorm and rotary of x [n, heads, hd].  The operator's definition rounds to the type after the
    normalisation, after the weight and after the rotation; the angles are formed in 64 bits."""
    x = x.float()
    hd = x.shape[-1]
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + NORM_EPS)
    x = ((x * r).to(dt).float() * w.float()).to(dt).float()
    f = ROPE_THETA ** (-2.0 * torch.arange(hd // 2, device=x.device, dtype=torch.float64) / hd)
    ang = positions.double()[:, None] * f[None, :]
    cs, sn = torch.cos(ang).float()[:, None, :], torch.sin(ang).float()[:, None, :]
    a, b = x[..., : hd // 2], x[..., hd // 2:]
    return torch.cat([a * cs - b * sn, b * cs + a * sn], -1).to(dt)


def _plain_decode(s):
    c, ctx = s["c"], s["ctx"].long()
    B, L, G = c["B"], s["max_ctx"], c["Hq"] // c["Hkv"]
    slots, b = _token_slots(s, torch.zeros_like(ctx), ctx)
    pos = torch.arange(b.numel(), device=b.device) - (torch.cumsum(ctx, 0) - ctx)[b]
    K = torch.zeros(B, L, c["Hkv"], c["hd"], device=b.device)
    V = torch.zeros_like(K)
    K[b, pos] = _unpack(s["k_cache"][slots], c, slots)
    V[b, pos] = _unpack(s["v_cache"][slots], c, slots)
    q = s["q"].float().reshape(B, c["Hkv"], G, c["hd"])
    S = torch.matmul(q, K.permute(0, 2, 3, 1)) * s["scale"]
    live = torch.arange(L, device=b.device)[None, :] < ctx[:, None]
    S = torch.where(live[:, None, None, :], S, float("-inf"))
    p = torch.exp(S - S.amax(-1, keepdim=True))
    o = torch.matmul(p, V.permute(0, 2, 1, 3)) / p.sum(-1, keepdim=True)
    return o.reshape(B, c["Hq"], c["hd"]).to(s["dt"])


def _plain(s):
    c = s["c"]
    if c["kind"] == "chunk":
        _plain_write(s, s["k"])
        return _plain_read(s)
    if c["kind"] == "norm":
        k = _plain_norm_rope(s["k"].reshape(-1, c["Hkv"], c["hd"]), s["wk"], s["positions"], s["dt"])
        _plain_write(s, k.flatten(1))
        return {"q": _plain_norm_rope(s["q"], s["wq"], s["positions"], s["dt"]), **_plain_read(s)}
    if c["kind"] == "read":
        return _plain_read(s)
    if c["kind"] == "step":
        _plain_write(s, s["k"])
        return {"out": _plain_decode(s), **_plain_read(s)}
    return {"out": _plain_decode(s)}


def _own_read(pa, s, desc, gs):
    heads = desc.num_kv_heads * desc.head_dim
    pa.pa_kv_read_q4(desc, gs, s["c"]["B"], s["cu_read"], s["starts"], s["ctx"], s["bt"], s["maxp"], s["reads"],
                     s["k_cache"], s["v_cache"], s["k_out"], heads, s["v_out"], heads)
    return {"k": s["k_out"], "v": s["v_out"]}


def _own(s):
    import paged_kv_gqa_08_gb300 as pa

    c, gs = s["c"], s["c"]["gs"]
    if "desc" not in s:
        s["desc"] = pa.cache_desc(c["Hq"], c["Hkv"], c["hd"], c["P"], s["num_pages"], s["dt"])
    desc, heads = s["desc"], c["Hkv"] * c["hd"]
    if c["kind"] == "chunk":
        pa.pa_kv_write_q4(desc, gs, s["k"], heads, s["v"], heads, s["n"], s["slots"], s["k_cache"], s["v_cache"])
        return _own_read(pa, s, desc, gs)
    if c["kind"] == "norm":
        pa.pa_qk_norm_rope_kv_write_q4(desc, gs, s["q"], c["Hq"] * c["hd"], s["k"], heads, s["v"], heads, s["n"],
                                       s["positions"], s["wq"], s["wk"], NORM_EPS, ROPE_THETA, s["slots"],
                                       s["q_out"], s["k_cache"], s["v_cache"])
        return {"q": s["q_out"], **_own_read(pa, s, desc, gs)}
    if c["kind"] == "read":
        return _own_read(pa, s, desc, gs)
    if c["kind"] == "step":
        pa.pa_decode_kv_write_q4(desc, gs, s["q"], s["k"], heads, s["v"], heads, c["B"], s["k_cache"], s["v_cache"],
                                 s["bt"], s["maxp"], s["ctx"], s["max_ctx"], s["scale"], 0, s["slot_out"], s["out"],
                                 s["ws"])
        return {"out": s["out"], **_own_read(pa, s, desc, gs)}
    pa.pa_decode_q4(desc, gs, s["q"], c["B"], s["k_cache"], s["v_cache"], s["bt"], s["maxp"], s["ctx"],
                    s["max_ctx"], s["scale"], 0, s["out"], s["ws"])
    return {"out": s["out"]}


def run(s):
    return _own(s) if own else _plain(s)


# ---------------------------------------------------------------------------
# the definition in 64 bits, request by request
# ---------------------------------------------------------------------------
def _exact_values(x, c):
    """What rows x [n, Hkv * hd] stand for once quantised (float64)."""
    x = x.double().reshape(-1, c["gs"])
    lo, hi = x.min(1, keepdim=True).values, x.max(1, keepdim=True).values
    s = ((hi - lo) / 15.0).half().double()
    o = (lo - 16.0 * s).half().double()
    v = torch.clamp(torch.round((x - o) / torch.where(s > 0, s, torch.ones_like(s))), 16, 31)
    return (torch.where(s > 0, v, torch.full_like(v, 16.0)) * s + o).reshape(-1, c["Hkv"], c["hd"])


def _exact_row_values(raw, slot, c):
    """float64 [n, Hkv, hd] of raw rows, byte by byte from the layout."""
    n, hkv, hd, gs = raw.shape[0], c["Hkv"], c["hd"], c["gs"]
    nc = hkv * hd // 2
    npar = raw.shape[1] - nc
    dim = torch.arange(hkv * hd, device=raw.device)
    word = dim // 4

    def byte(part, size, i):  # byte i of a part, at its swizzled place
        pieces = min(8, size // 16)
        blk, j, low = i // (16 * pieces), (i // 16) % pieces, i % 16
        at = (blk * pieces)[None, :] * 16 + (j[None, :] ^ (slot[:, None] & (pieces - 1))) * 16 + low[None, :]
        return torch.gather(part, 1, at).long()

    h = byte(raw[:, :nc], nc, 2 * word) + 256 * byte(raw[:, :nc], nc, 2 * word + 1)
    k = (dim % 4)[None, :]
    u = torch.where(k == 0, (h // 64) % 16, torch.where(k == 2, (h // 4) % 16, torch.where(
        k == 3, (h // 1024) % 16, (h // 16384) + 4 * (h % 4))))
    at = (dim // gs) * 4
    par = raw[:, nc:]
    num = lambda i: (byte(par, npar, i) + 256 * byte(par, npar, i + 1)).to(torch.int16)  # noqa: E731
    s, o = num(at).view(torch.float16).double(), num(at + 2).view(torch.float16).double()
    return (s * (16 + u).double() + o).reshape(n, hkv, hd)


def _exact_norm_rope(x, w, pos, dt):
    x, w, hd = x.double(), w.double(), x.shape[-1]
    x = (x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / hd + NORM_EPS)).to(dt).double()
    x = (x * w).to(dt).double()
    z = torch.complex(x[..., : hd // 2], x[..., hd // 2:])
    i = torch.arange(hd // 2, device=x.device, dtype=torch.float64)
    ang = pos.double()[:, None, None] * torch.exp(-math.log(ROPE_THETA) * 2 * i / hd)
    z = z * torch.polar(torch.ones_like(ang), ang)
    return torch.cat([z.real, z.imag], -1).to(dt)


def exact(c, seed):
    s = prepare(c, seed)
    dt, G = s["dt"], c["Hq"] // c["Hkv"]
    k_new, v_new = s["k"], s["v"]
    res = {}
    if c["kind"] == "norm":
        res["q"] = _exact_norm_rope(s["q"], s["wq"], s["positions"], dt).double()
        k_new = _exact_norm_rope(k_new.reshape(-1, c["Hkv"], c["hd"]), s["wk"], s["positions"], dt).flatten(1)
    ctx, new = _lens(c)
    ks, vs, outs = [], [], []
    at = 0
    for b in range(c["B"]):
        L, n = int(ctx[b]), int(new[b])
        pos = torch.arange(L - n, device="cuda")
        slot = s["bt"][b][pos // c["P"]].long() * c["P"] + pos % c["P"]
        whole = not (c["tail"] or c["kind"] == "step")
        KV = []
        for cache, fresh in ((s["k_cache"], k_new), (s["v_cache"], v_new)):
            parts = []
            if L > n and (whole or c["kind"] == "step"):
                parts.append(_exact_row_values(cache[slot], slot, c))
            if n:
                parts.append(_exact_values(fresh[at: at + n], c))
            KV.append(torch.cat(parts))
        at += n
        K, V = KV
        if c["kind"] in ("decode", "step"):
            q = s["q"][b].double().reshape(c["Hkv"], G, c["hd"])
            logit = torch.einsum("hgd,lhd->hgl", q, K) * (c["hd"] ** -0.5)
            outs.append(torch.einsum("hgl,lhd->hgd", torch.softmax(logit, -1), V).reshape(c["Hq"], c["hd"]))
        if c["kind"] != "decode":
            keep = K.shape[0] if whole else n
            ks.append(K[K.shape[0] - keep:].flatten(1))
            vs.append(V[V.shape[0] - keep:].flatten(1))
    if outs:
        res["out"] = torch.stack(outs)
    if ks:
        res["k"], res["v"] = torch.cat(ks), torch.cat(vs)
    return res
