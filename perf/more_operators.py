"""Cases of attention over part of a paged K/V cache, and of the block tables that lead to it.

Four kinds of operator:

  window, step   decode attention in which a query at position p sees the tokens
                 j of its request with p - W < j <= p, and the first S tokens
                 (sinks); ``step`` also stores the new token's K/V row
  chunk          the same for the packed new tokens of prompt chunks
  shared         decode attention for groups of requests whose first tokens are
                 the same pages, attended to once for the group's queries
  tables         block tables, positions and slots of a batch's new tokens built
                 on the GPU from a ring of free pages; pages that rows share, and
                 pages handed back

A cache is ``[num_pages, P, Hkv, hd]``; token j of request b lies in page
``block_tables[b][j // P]`` at offset ``j % P``.  The ring of free pages holds
``num_pages`` entries; the two numbers of the pool's state count the pages taken
from it and put into it since the start, so the next page out is entry
``taken % num_pages`` and ``returned - taken`` pages are free.
"""
import math

import numpy as np
import torch

own = False

KINDS = ("window", "window", "step", "chunk", "chunk", "shared", "shared", "tables")
MODES = ("extend", "fork", "slide")


def _case(name, kind, **kw):
    c = dict(name=name, kind=kind, dtype="bf16", B=1, Hq=16, Hkv=8, hd=128, P=16, new_lo=1, new_hi=1, ctx_lo=1,
             ctx_hi=1, W=1, S=0, evict=False, groups=1, pre_lo=0, pre_hi=0, mode="", lens=1)
    c.update(kw)
    return c


def listed():
    return [
        # two users' decode over a short window: latency
        _case("window_two", "window", B=2, ctx_lo=301, ctx_hi=905, W=256, S=4, lens=1),
        # a full decode batch with small pages, contexts from inside the window to eight times it; the pages that the
        # window has left belong to others
        _case("window_batch", "window", B=256, ctx_lo=128, ctx_hi=8192, W=1024, S=4, evict=True, lens=2),
        # long contexts with large pages that keep all their pages (they are prefixes to other requests)
        _case("window_long", "window", B=64, Hq=32, P=256, ctx_lo=8192, ctx_hi=32768, W=4096, S=64, lens=3),
        # a small fp32 model's step, odd window, contexts from a single token
        _case("step_f32", "step", dtype="f32", B=5, Hq=4, Hkv=2, hd=64, ctx_lo=1, ctx_hi=701, W=101, S=3, lens=4),
        # one short prompt chunk of a chat turn: latency
        _case("chunk_one", "chunk", B=1, new_lo=33, new_hi=33, ctx_lo=633, ctx_hi=633, W=128, S=4, lens=5),
        # eight requests in mixed chunked prefill over contexts up to 4608
        _case("chunk_mix", "chunk", B=8, new_lo=1, new_hi=512, ctx_lo=600, ctx_hi=4608, W=1024, S=4, lens=6),
        # long prompts in chunks of 2048, every second key of theirs out of the window
        _case("chunk_2k", "chunk", B=8, new_lo=2048, new_hi=2048, ctx_lo=8192, ctx_hi=8192, W=2048, S=16, evict=True,
              lens=7),
        # four samples of one prompt: latency
        _case("shared_four", "shared", B=4, pre_lo=2048, pre_hi=2048, ctx_lo=1, ctx_hi=64, lens=8),
        # a batch behind three system prompts of different lengths
        _case("shared_groups", "shared", B=96, Hq=32, P=256, groups=3, pre_lo=3000, pre_hi=9000, ctx_lo=40, ctx_hi=700,
              lens=9),
        # many questions about one long document
        _case("shared_long", "shared", B=128, Hq=32, P=16, pre_lo=32768, pre_hi=32768, ctx_lo=20, ctx_hi=300, lens=10),
        # a decode batch's next token: one table entry and one slot a request
        _case("tables_decode", "tables", mode="extend", B=256, ctx_lo=128, ctx_hi=2048, new_lo=1, new_hi=1, lens=11),
        # branches of running requests: they share whole pages, get a chunk's pages of their own and are dropped again
        _case("tables_fork", "tables", mode="fork", B=64, ctx_lo=256, ctx_hi=8192, new_lo=1, new_hi=700, lens=12),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(KINDS)
    hkv = rng.choice((1, 2, 4, 8, 8))
    c = _case("", kind, dtype=rng.choice(("bf16", "bf16", "bf16", "f32")), Hkv=hkv,
              Hq=hkv * rng.choice((1, 2, 3, 4, 5, 6, 7, 8)), hd=rng.choice((64, 128, 128)),
              P=rng.choice((16, 32, 64, 128, 256)), lens=rng.randrange(1, 1 << 30))
    small = c["dtype"] == "f32" or c["hd"] == 64
    if kind == "tables":
        c["mode"] = rng.choice(MODES)
        c["B"] = _spread(rng, 1, 700)
        c["ctx_hi"] = _spread(rng, 1, 400000 // c["B"])
        c["ctx_lo"] = _spread(rng, 1, c["ctx_hi"])
        c["new_hi"] = _spread(rng, 1, min(4096, 60000 // c["B"]))
        c["new_lo"] = rng.choice((0, 1, c["new_hi"]))
        c["W"], c["S"] = _spread(rng, 1, 2000), rng.choice((0, 1, 4, 100))
    elif kind == "shared":
        c["B"] = _spread(rng, 2, 24 if small else 160)
        c["groups"] = min(c["B"], rng.choice((1, 1, 2, 3, 7)))
        c["pre_hi"] = _spread(rng, 16, 3000 if small else 24000)
        c["pre_lo"] = _spread(rng, 1, c["pre_hi"])
        c["ctx_hi"] = _spread(rng, 1, 600)
        c["ctx_lo"] = rng.choice((0, 1, c["ctx_hi"]))
    else:
        c["W"] = _spread(rng, 1, 6000)
        c["S"] = rng.choice((0, 1, 4, 17, 64, 300))
        c["evict"] = rng.random() < 0.5
        if kind == "chunk":
            c["B"] = _spread(rng, 1, 12)
            c["ctx_hi"] = _spread(rng, 2, 1500 if small else 12000)
            c["new_hi"] = _spread(rng, 1, min(c["ctx_hi"], (1200 if small else 16000) // c["B"]))
            c["new_lo"] = _spread(rng, 1, c["new_hi"])
        else:
            c["B"] = _spread(rng, 1, 256)
            c["ctx_hi"] = _spread(rng, 1, min(40000, (40000 if small else 400000) // c["B"]))
        c["ctx_lo"] = _spread(rng, 1, c["ctx_hi"])
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# sizes of a case
# ---------------------------------------------------------------------------
def _lens(c):
    """Context lengths (with the new tokens) and new tokens of the requests; both ends of the ranges occur.  For
    ``shared`` the context is the group's prefix and ctx_lo .. ctx_hi tokens of the request's own, for ``tables`` the
    tokens that a request has before its new ones."""
    r = np.random.RandomState(c["lens"])
    ctx = r.randint(c["ctx_lo"], c["ctx_hi"] + 1, c["B"])
    new = r.randint(c["new_lo"], c["new_hi"] + 1, c["B"])
    ctx[0], ctx[-1] = c["ctx_lo"], c["ctx_hi"]
    new[0], new[-1] = c["new_lo"], c["new_hi"]
    if c["kind"] == "shared":
        _, pre, of = _groups(c)
        ctx = ctx + pre[of]
    elif c["kind"] != "tables":
        new = np.minimum(new, ctx)
    return ctx, new


def _groups(c):
    """First request of each group, its prefix length, and the group of each request."""
    r = np.random.RandomState(c["lens"] + 1)
    cuts = np.sort(r.choice(np.arange(1, c["B"]), c["groups"] - 1, replace=False)) if c["groups"] > 1 else []
    cu = np.concatenate([[0], cuts, [c["B"]]]).astype(np.int64)
    pre = r.randint(c["pre_lo"], c["pre_hi"] + 1, c["groups"])
    pre[0], pre[-1] = c["pre_lo"], c["pre_hi"]
    return cu, pre, np.repeat(np.arange(c["groups"]), np.diff(cu))


def _first_seen(c, ctx, new):
    """The first token after the sinks that some new token of each request sees."""
    return np.maximum(np.minimum(c["S"], ctx), ctx - new + 1 - c["W"])


def _branches(c, ctx):
    """``fork``: the rows of odd index are branches of the row before them, which they follow for whole pages."""
    parent = np.full(c["B"], -1)
    parent[1::2] = np.arange(c["B"])[1::2] - 1
    pages = np.where(parent >= 0, np.minimum(ctx, ctx[parent]) // c["P"], 0)
    return parent, pages


def work(c):
    ctx, new = _lens(c)
    e = 2 if c["dtype"] == "bf16" else 4
    row, P = c["Hkv"] * c["hd"] * e, c["P"]
    q_row, flop = c["Hq"] * c["hd"] * e, 4 * c["Hq"] * c["hd"]
    if c["kind"] == "tables":
        old = _old(c, ctx)
        pages = int((-(-(old + new) // P) - -(-old // P)).sum())
        n = int(new.sum())
        back = 0
        if c["mode"] == "fork":
            parent, shared = _branches(c, ctx)
            end = -(-(old + new) // P)
            back = int(shared.sum()) * 5 * 4 + int(end[parent >= 0].sum()) * 4 * 4
        elif c["mode"] == "slide":
            back = int(np.maximum(0, _slid(c, old + new)[1] - _slid(c, old + new)[0]).sum()) * 5 * 4
        return {"bytes": float(16 * c["B"] + 12 * n + 12 * pages + back), "flops": float(4 * n + 8 * c["B"])}
    if c["kind"] == "shared":
        cu, pre, of = _groups(c)
        live = np.diff(cu) > 0
        tokens = int(pre[live].sum() + (ctx - pre[of]).sum())
        return {"bytes": float(2 * tokens * row + 2 * c["B"] * q_row + 4 * (tokens // P)),
                "flops": float(flop * int(ctx.sum()))}
    first = _first_seen(c, ctx, new)
    sinks = np.minimum(c["S"], ctx)
    if c["kind"] != "chunk":
        seen = int((sinks + ctx - first).sum())
        n = c["B"]
        nbytes = 2 * seen * row + 2 * n * q_row + 4 * (seen // P + 1)
        if c["kind"] == "step":
            nbytes += 2 * n * row  # the new rows in as they come, not from the cache, and out
        return {"bytes": float(nbytes), "flops": float(flop * seen)}
    seen = int((sinks + ctx - first).sum())
    pairs = 0
    for L, n in zip(ctx, new):
        p = np.arange(L - n, L)
        lo = np.maximum(0, p + 1 - c["W"])
        pairs += int((p + 1 - lo + np.minimum(c["S"], lo)).sum())
    return {"bytes": float(2 * seen * row + 2 * int(new.sum()) * q_row + 4 * (seen // P + 1)), "flops": float(flop * pairs)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _rows(c, n, g, dt):
    """K or V rows as a model has them: unit variance, a few dimensions of a head with an offset of their own."""
    heads = c["Hkv"] * c["hd"]
    off = torch.randn(heads, generator=g, device="cuda") * 3.0
    off = torch.where(torch.rand(heads, generator=g, device="cuda") < 1 / 16, off, torch.zeros_like(off)).to(dt)
    return torch.randn(n, heads, generator=g, device="cuda", dtype=dt).add_(off)


def _old(c, ctx):
    """``tables``: the tokens that each row has when its pages are taken."""
    if c["mode"] == "fork":
        parent, shared = _branches(c, ctx)
        return np.where(parent >= 0, shared * c["P"], ctx)
    return np.zeros_like(ctx) if c["mode"] == "slide" else ctx


def _slid(c, ctx):
    """``slide``: the pages [first, end) of contexts of `ctx` tokens that no later token sees."""
    return -(-c["S"] // c["P"]) + 0 * ctx, np.maximum(0, ctx + 1 - c["W"]) // c["P"]


def _prepare_tables(c, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    ctx, new = _lens(c)
    old = _old(c, ctx)
    parent = _branches(c, ctx)[0] if c["mode"] == "fork" else np.full(c["B"], -1)
    P, B = c["P"], c["B"]
    held = np.where(parent >= 0, 0, -(-old // P))
    need = -(-(old + new) // P) - -(-old // P)
    maxp = int(max(1, (-(-(old + new) // P)).max()))
    total, want = int(held.sum()), int(need.sum())
    others = want + 5  # held by rows of other batches
    num_pages = total + others + want + want // 8 + 3
    perm = torch.randperm(num_pages, generator=g, device=dev).to(torch.int32)
    bt = torch.full((B, maxp), -1, dtype=torch.int32, device=dev)
    bt[torch.arange(maxp, device=dev)[None, :] < torch.tensor(held, device=dev)[:, None]] = perm[:total]
    refs = torch.zeros(num_pages, dtype=torch.int32, device=dev)
    refs[perm[: total + others].long()] = 1
    # the ring has gone round before: the free pages start anywhere in it
    taken = int(torch.randint(0, 1 << 40, (1,), generator=g, device=dev).item())
    free = num_pages - total - others
    ring = torch.randint(0, num_pages, (num_pages,), generator=g, device=dev, dtype=torch.int32)
    ring[(taken + torch.arange(free, device=dev)) % num_pages] = perm[total + others:]
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)  # noqa: E731
    n = int(new.sum())
    s = {"c": dict(c), "num_pages": num_pages, "maxp": maxp, "n": n, "bt": bt, "refs": refs, "ring": ring,
         "pool": torch.tensor([taken, taken + free], dtype=torch.int64, device=dev),
         "pool_mid": torch.zeros(2, dtype=torch.int64, device=dev),
         "pool_out": torch.zeros(2, dtype=torch.int64, device=dev), "new": i32(new), "ctx": i32(old),
         "ctx_out": i32(0 * old), "cu": torch.zeros(B + 1, dtype=torch.int32, device=dev),
         "positions": torch.zeros(max(n, 1), dtype=torch.int32, device=dev),
         "slots": torch.zeros(max(n, 1), dtype=torch.int64, device=dev), "parent": i32(parent)}
    if c["mode"] == "fork":
        s["shared"] = i32(_branches(c, ctx)[1])
        s["first"], s["end"] = i32(0 * old), i32(np.where(parent >= 0, -(-(old + new) // P), 0))
    return s


def prepare(c, seed):
    if c["kind"] == "tables":
        return _prepare_tables(c, seed)
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    ctx, new = _lens(c)
    B, P = c["B"], c["P"]
    npg = -(-ctx // P)
    maxp = int(npg.max())
    page = np.arange(maxp)[None, :]
    has = page < npg[:, None]
    if c["kind"] == "shared":
        cu, pre, of = _groups(c)
        # whole pages of the prefix are the group's; the first request's are the ones that the others name, too
        whole = (pre // P)[of]
        first = cu[:-1][of]
        mine = has & ((page >= whole[:, None]) | (np.arange(B) == first)[:, None])
    else:
        mine = has
        if c["evict"]:
            seen = _first_seen(c, ctx, new)
            sinks = np.minimum(c["S"], ctx)
            mine = has & ((page * P < sinks[:, None]) | ((page + 1) * P > seen[:, None]))
    total = int(mine.sum())
    num_pages = total + 1 + total // 16
    perm = torch.randperm(num_pages, generator=g, device=dev).to(torch.int32)
    bt = torch.full((B, maxp), -1 if c["evict"] else num_pages - 1, dtype=torch.int32, device=dev)
    mine_t = torch.tensor(mine, device=dev)
    bt[mine_t] = perm[:total]
    if c["kind"] == "shared":
        of_first = torch.tensor(first, device=dev)
        take = torch.tensor(page < whole[:, None], device=dev)
        bt = torch.where(take, bt[of_first], bt)
    k_cache, v_cache = (_rows(c, num_pages * P, g, dt).view(num_pages, P, c["Hkv"], c["hd"]) for _ in range(2))
    if c["kind"] == "shared":
        # the rest of a prefix, in a page that the request goes on to write, is every request's own copy
        for b in range(B):
            f, w, r = int(first[b]), int(whole[b]), int(pre[of[b]] % P)
            if r and f != b:
                for cache in (k_cache, v_cache):
                    cache[int(bt[b, w]), :r] = cache[int(bt[f, w]), :r]
    n = int(new.sum()) if c["kind"] == "chunk" else B
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)  # noqa: E731
    s = {"c": dict(c), "dt": dt, "num_pages": num_pages, "maxp": maxp, "max_ctx": int(ctx.max()), "n": n,
         "k_cache": k_cache, "v_cache": v_cache, "bt": bt.contiguous(), "ctx": i32(ctx), "scale": c["hd"] ** -0.5,
         "q": torch.randn(n, c["Hq"], c["hd"], generator=g, device=dev).to(dt),
         "out": torch.zeros(n, c["Hq"], c["hd"], dtype=dt, device=dev),
         # a serving program's workspace, sized once for its largest step
         "ws": torch.empty(256 << 20, dtype=torch.uint8, device=dev)}
    if c["kind"] == "chunk":
        s["cu"] = i32(np.concatenate([[0], np.cumsum(new)]))
        s["max_q"] = int(new.max())
    if c["kind"] == "step":
        s["k"], s["v"] = _rows(c, B, g, dt), _rows(c, B, g, dt)
        s["slots"] = torch.zeros(B, dtype=torch.int64, device=dev)
    if c["kind"] == "shared":
        s["cu_groups"], s["prefix"], s["max_prefix"] = i32(cu), i32(pre), int(pre.max())
    return s


# ---------------------------------------------------------------------------
# one pass, plain
# ---------------------------------------------------------------------------
def _attend(q, K, V, seen, scale):
    """fp32 attention of q [.., Hkv, G, hd] over K, V [.., n, Hkv, hd]; ``seen`` broadcasts to [.., Hkv, G, n]."""
    axes = (1, 2, 0) if K.dim() == 3 else (0, 2, 3, 1)
    S = torch.matmul(q, K.permute(*axes)) * scale
    S = torch.where(seen, S, float("-inf"))
    m = S.amax(-1, keepdim=True)
    p = torch.exp(S - torch.where(m == float("-inf"), 0.0, m))
    return torch.matmul(p, V.transpose(-3, -2)) / p.sum(-1, keepdim=True)


def _at(s, cache, b, j):
    """fp32 rows of tokens j of requests b."""
    P = s["c"]["P"]
    return cache[s["bt"][b, j // P].long(), j % P].float()


def _plain_window(s):
    c, dev = s["c"], s["bt"].device
    B, G = c["B"], c["Hq"] // c["Hkv"]
    ctx = s["ctx"].long()[:, None]
    wide = min(c["W"], s["max_ctx"])
    first = torch.clamp(ctx - c["W"], min=0)
    sinks = torch.arange(min(c["S"], s["max_ctx"]), device=dev)[None, :].expand(B, -1)
    near = first + torch.arange(wide, device=dev)[None, :]
    j = torch.cat([sinks, near], 1)
    seen = torch.cat([sinks < first, near < ctx], 1)
    j = torch.where(seen, j, ctx - 1)
    b = torch.arange(B, device=dev)[:, None].expand_as(j)
    q = s["q"].float().view(B, c["Hkv"], G, c["hd"])
    o = _attend(q, _at(s, s["k_cache"], b, j), _at(s, s["v_cache"], b, j), seen[:, None, None, :], s["scale"])
    return o.reshape(B, c["Hq"], c["hd"]).to(s["dt"])


def _plain_step(s):
    c, ctx = s["c"], s["ctx"].long()
    b = torch.arange(c["B"], device=ctx.device)
    slot = s["bt"][b, (ctx - 1) // c["P"]].long() * c["P"] + (ctx - 1) % c["P"]
    for cache, rows in ((s["k_cache"], s["k"]), (s["v_cache"], s["v"])):
        cache.view(-1, rows.shape[1])[slot] = rows
    return {"out": _plain_window(s), "slots": slot, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_chunk(s):
    c, dev = s["c"], s["bt"].device
    G = c["Hq"] // c["Hkv"]
    ctx, new = _lens(c)
    outs, at = [], 0
    for b in range(c["B"]):
        L, n = int(ctx[b]), int(new[b])
        first = max(min(c["S"], L), L - n + 1 - c["W"])
        j = torch.cat([torch.arange(min(c["S"], L), device=dev), torch.arange(first, L, device=dev)])
        p = torch.arange(L - n, L, device=dev)[:, None]
        seen = ((j > p - c["W"]) | (j < c["S"])) & (j <= p)
        q = s["q"][at: at + n].float().view(n, c["Hkv"], G, c["hd"]).permute(1, 2, 0, 3)
        o = _attend(q.reshape(c["Hkv"], G * n, c["hd"]), _at(s, s["k_cache"], b, j), _at(s, s["v_cache"], b, j),
                    seen.repeat(G, 1), s["scale"])
        outs.append(o.view(c["Hkv"], G, n, c["hd"]).permute(2, 0, 1, 3).reshape(n, c["Hq"], c["hd"]).to(s["dt"]))
        at += n
    return torch.cat(outs)


def _plain_shared(s):
    c, dev = s["c"], s["bt"].device
    G = c["Hq"] // c["Hkv"]
    ctx, _ = _lens(c)
    seen = torch.ones((), dtype=torch.bool, device=dev)
    outs = []
    for b in range(c["B"]):
        j = torch.arange(int(ctx[b]), device=dev)
        q = s["q"][b].float().view(c["Hkv"], G, c["hd"])
        o = _attend(q, _at(s, s["k_cache"], b, j), _at(s, s["v_cache"], b, j), seen, s["scale"])
        outs.append(o.reshape(c["Hq"], c["hd"]).to(s["dt"]))
    return torch.stack(outs)


def _plain_extend(s):
    """Pages for the new tokens, in the order of the requests, and the tokens' positions and slots."""
    c, dev = s["c"], s["bt"].device
    P, B = c["P"], c["B"]
    old, new = s["ctx"].long(), s["new"].long()
    held, full = (old + P - 1) // P, (old + new + P - 1) // P
    need = full - held
    before = torch.cumsum(need, 0) - need
    page = torch.arange(s["maxp"], device=dev)[None, :]
    take = (page >= held[:, None]) & (page < full[:, None])
    nth = s["pool"][0] + before[:, None] + page - held[:, None]
    got = s["ring"][nth % s["num_pages"]]
    s["bt"] = torch.where(take, got, s["bt"])
    s["refs"][got[take].long()] = 1
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), torch.cumsum(new, 0)])
    t = torch.arange(s["n"], device=dev)
    b = torch.searchsorted(cu[1:], t, right=True)
    pos = old[b] + t - cu[b]
    slots = s["bt"][b, pos // P].long() * P + pos % P
    state = torch.stack([s["pool"][0] + need.sum(), s["pool"][1]])
    return {"cu": cu.int(), "ctx": (old + new).int(), "positions": pos.int(), "slots": slots, "pool": state}


def _plain_share(s):
    page = torch.arange(s["maxp"], device=s["bt"].device)[None, :]
    take = (page < s["shared"].long()[:, None]) & (s["parent"] >= 0)[:, None]
    s["bt"] = torch.where(take, s["bt"][s["parent"].clamp(min=0).long()], s["bt"])
    s["refs"].index_put_((s["bt"][take].long(),), torch.ones((), dtype=torch.int32, device=take.device), accumulate=True)


def _plain_release(s, first, end, state):
    """Entries [first, end) of the rows: a page that no row holds any longer goes back into the ring at the place of
    the last entry that named it, rows in order, each from its last page down."""
    dev = s["bt"].device
    page = torch.arange(s["maxp"], device=dev)[None, :]
    take = (page >= first[:, None]) & (page < end[:, None]) & (s["bt"] >= 0)
    pages = s["bt"].flip(1)[take.flip(1)].long()
    s["refs"].index_put_((pages,), torch.full((), -1, dtype=torch.int32, device=dev), accumulate=True)
    last = torch.full((s["num_pages"],), -1, dtype=torch.long, device=dev)
    at = torch.arange(pages.numel(), device=dev)
    last = last.scatter_reduce(0, pages, at, "amax")
    out = (last[pages] == at) & (s["refs"][pages] == 0)
    back = pages[out]
    s["ring"][(state[1] + torch.arange(back.numel(), device=dev)) % s["num_pages"]] = back.int()
    s["bt"] = torch.where(take, -1, s["bt"])
    return torch.stack([state[0], state[1] + back.numel()])


def _plain_tables(s):
    mode = s["c"]["mode"]
    if mode == "fork":
        _plain_share(s)
    r = _plain_extend(s)
    if mode == "fork":
        r["pool"] = _plain_release(s, s["first"].long(), s["end"].long(), r["pool"])
    elif mode == "slide":
        L, P = r["ctx"].long(), s["c"]["P"]
        first, end = torch.full_like(L, -(-s["c"]["S"] // P)), torch.clamp(L + 1 - s["c"]["W"], min=0) // P
        r["pool"] = _plain_release(s, first, end, r["pool"])
    return {**r, "tables": s["bt"], "refs": s["refs"], "ring": s["ring"]}


# ---------------------------------------------------------------------------
# one pass of the framework's calls
# ---------------------------------------------------------------------------
def _own(s):
    import paged_kv_gqa_08_gb300 as pa

    c = s["c"]
    if "desc" not in s:
        s["desc"] = pa.cache_desc(c["Hq"], c["Hkv"], c["hd"], c["P"], s["num_pages"],
                                  torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)
    desc = s["desc"]
    if c["kind"] == "tables":
        if c["mode"] == "fork":
            pa.pa_share_pages(desc, c["B"], s["parent"], s["shared"], s["bt"], s["maxp"], s["refs"])
        state = s["pool_out"] if c["mode"] == "extend" else s["pool_mid"]
        pa.pa_extend_tables(desc, c["B"], s["new"], s["ctx"], s["bt"], s["maxp"], s["ring"], s["pool"], s["n"],
                            s["cu"], s["ctx_out"], s["positions"], s["slots"], s["refs"], state)
        if c["mode"] == "fork":
            pa.pa_release_pages(desc, c["B"], s["first"], s["end"], s["bt"], s["maxp"], s["refs"], s["ring"], state,
                                s["pool_out"])
        elif c["mode"] == "slide":
            pa.pa_release_window_pages(desc, c["W"], c["S"], c["B"], s["ctx_out"], s["bt"], s["maxp"], s["refs"],
                                       s["ring"], state, s["pool_out"])
        return {"cu": s["cu"], "ctx": s["ctx_out"], "positions": s["positions"][: s["n"]],
                "slots": s["slots"][: s["n"]], "pool": s["pool_out"], "tables": s["bt"], "refs": s["refs"],
                "ring": s["ring"]}
    cache = (s["k_cache"], s["v_cache"], s["bt"], s["maxp"], s["ctx"], s["max_ctx"], s["scale"])
    if c["kind"] == "chunk":
        pa.pa_prefill_varlen_window(desc, c["W"], c["S"], s["q"], s["cu"], c["B"], s["max_q"], s["n"], *cache,
                                    s["out"], s["ws"])
    elif c["kind"] == "shared":
        pa.pa_decode_shared_prefix(desc, c["groups"], s["cu_groups"], s["prefix"], s["max_prefix"], s["q"], c["B"],
                                   *cache, 0, s["out"], s["ws"])
    elif c["kind"] == "step":
        row = c["Hkv"] * c["hd"]
        pa.pa_decode_kv_write_window(desc, c["W"], c["S"], s["q"], s["k"], row, s["v"], row, c["B"], *cache, 0,
                                     s["slots"], s["out"], s["ws"])
        return {"out": s["out"], "slots": s["slots"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    else:
        pa.pa_decode_window(desc, c["W"], c["S"], s["q"], c["B"], *cache, 0, s["out"], s["ws"])
    return s["out"]


def run(s):
    if own:
        return _own(s)
    kind = s["c"]["kind"]
    return {"window": _plain_window, "step": _plain_step, "chunk": _plain_chunk, "shared": _plain_shared,
            "tables": _plain_tables}[kind](s)


# ---------------------------------------------------------------------------
# the definitions, in 64 bits, request by request
# ---------------------------------------------------------------------------
def _exact_attention(s, c, ctx, new):
    G, dev = c["Hq"] // c["Hkv"], s["bt"].device
    windowed = c["kind"] != "shared"
    outs, row = [], 0
    for b in range(c["B"]):
        L, n = int(ctx[b]), int(new[b]) if c["kind"] == "chunk" else 1
        for r0 in range(0, n, 256):
            r1 = min(n, r0 + 256)
            p = torch.arange(L - n + r0, L - n + r1, device=dev)
            j = torch.arange(L, device=dev)
            if windowed:  # only what some of these rows see is looked up
                j = j[(j < c["S"]) | (j > int(p[0]) - c["W"])]
            j = j[j <= int(p[-1])]
            page = s["bt"][b][torch.div(j, c["P"], rounding_mode="floor")].long()
            K, V = s["k_cache"][page, j % c["P"]].double(), s["v_cache"][page, j % c["P"]].double()
            q = s["q"][row + r0: row + r1].double().reshape(r1 - r0, c["Hkv"], G, c["hd"])
            logit = torch.einsum("nhgd,jhd->hgnj", q, K) / math.sqrt(c["hd"])
            hidden = j[None, :] > p[:, None]
            if windowed:
                hidden = hidden | ((j[None, :] <= p[:, None] - c["W"]) & (j[None, :] >= c["S"]))
            logit = logit.masked_fill(hidden, float("-inf"))
            outs.append(torch.einsum("hgnj,jhd->nhgd", torch.softmax(logit, -1), V).reshape(-1, c["Hq"], c["hd"]))
        row += n
    return torch.cat(outs)


def _exact_tables(s, c, ctx, new):
    old, P = _old(c, ctx), c["P"]
    bt, refs, ring = (s[k].cpu().numpy().copy() for k in ("bt", "refs", "ring"))
    taken, returned = (int(x) for x in s["pool"].cpu())
    if c["mode"] == "fork":
        parent, shared = _branches(c, ctx)
        start = bt.copy()
        for b in range(c["B"]):
            for i in range(shared[b]):
                bt[b, i] = start[parent[b], i]
                refs[bt[b, i]] += 1
    cu, pos, slots = [0], [], []
    for b in range(c["B"]):
        for t in range(int(old[b]), int(old[b] + new[b])):
            if t % P == 0:
                bt[b, t // P] = ring[taken % len(ring)]
                refs[bt[b, t // P]] = 1
                taken += 1
            pos.append(t)
            slots.append(int(bt[b, t // P]) * P + t % P)
        cu.append(len(pos))
    lens = old + new
    back = []
    for b in range(c["B"]) if c["mode"] != "extend" else ():
        if c["mode"] == "fork":
            first, end = 0, -(-int(lens[b]) // P) if parent[b] >= 0 else 0
        else:
            first, end = -(-c["S"] // P), max(0, int(lens[b]) + 1 - c["W"]) // P
        for i in range(min(end, bt.shape[1]) - 1, first - 1, -1):
            if bt[b, i] >= 0:
                back.append(int(bt[b, i]))
                bt[b, i] = -1
    for i, page in enumerate(back):
        refs[page] -= 1
        if refs[page] == 0:
            ring[returned % len(ring)] = page
            returned += 1
    t = torch.tensor
    return {"cu": t(cu), "ctx": t(lens), "positions": t(pos), "slots": t(slots), "pool": t([taken, returned]),
            "tables": t(bt), "refs": t(refs), "ring": t(ring)}


def exact(c, seed):
    s = prepare(c, seed)
    ctx, new = _lens(c)
    if c["kind"] == "tables":
        return _exact_tables(s, c, ctx, new)
    if c["kind"] != "step":
        return _exact_attention(s, c, ctx, new)
    slots = []
    for b in range(c["B"]):
        at = divmod(int(ctx[b]) - 1, c["P"])
        page = int(s["bt"][b, at[0]])
        slots.append(page * c["P"] + at[1])
        s["k_cache"][page, at[1]] = s["k"][b].view(c["Hkv"], c["hd"])
        s["v_cache"][page, at[1]] = s["v"][b].view(c["Hkv"], c["hd"])
    return {"out": _exact_attention(s, c, ctx, new), "slots": torch.tensor(slots), "k_cache": s["k_cache"],
            "v_cache": s["v_cache"]}
