// How the attention of decode requests to prefixes that they share is cut over
// the CTAs of one launch, for the kernels that compute it (prefill_tc.cu,
// tile_attention.cu) and the merge.
//
// Group g is requests cu[g] .. cu[g+1]-1, whose first pre[g] keys are the same.
// For every kv-head its queries are n * G rows (n requests, G q-heads), cut into
// q-tiles of TQ requests; two q-tiles, or the last one alone, are a unit, and a
// unit has the prefix's key tiles of 128 to go through.  The key tiles of all
// units (groups, then kv-heads, then units) form one line on which a tile takes
// up its cost; CTA c of n takes the tiles that start in [c T / n, (c+1) T / n),
// T the line's length.  The cut depends only on the lengths, every CTA finds its
// own share from them, and no CTA waits for another.
//
// A unit cut over CTAs leaves a part (O / l and the base-2 log-sum-exp of each
// row) per CTA.  Parts are packed: CTA c's part of the rows of kv-head h of a
// group starts at row cu[g] Hq + h n G + R c, row (request, q-head) in order; a
// unit has at most R rows, so parts never overlap, and B Hq + R CTAs rows hold
// them all.
#pragma once

#include "pa_common.cuh"

namespace pa {

constexpr int kPrefixTile = 128;  // keys per tile

// a / b for a >= 0, b > 0: mostly small numbers, whose division is far shorter.
PA_DEVINL int64_t div_small(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

PA_DEVINL int32_t prefix_part_row(const PrefixShape& s, int s0, int n, int h, int c, int Hq, int G) {
  return s0 * Hq + h * n * G + c * s.unit_rows;
}

struct PrefixGroup {
  int s0, n;      // requests
  int prefix, nt; // keys, key tiles
  int rep;        // a request whose table names the prefix's pages, or -1
  int pairs, one; // units of two q-tiles per kv-head, and of one (0 or 1)
  int64_t head_cost, cost;
};

PA_DEVINL PrefixGroup prefix_group(const PrefixShape& s, int g) {
  PrefixGroup r;
  r.s0 = min(max(s.cu[g], 0), s.B);
  const int s1 = min(max(s.cu[g + 1], r.s0), s.B);
  r.n = s1 - r.s0;
  r.prefix = s.pre[g];
  r.rep = -1;
  if (r.prefix >= 1 && r.prefix <= s.max_prefix) {
    // the first live request that is as long as the prefix
    for (int b = r.s0; b < s1 && r.rep < 0; ++b)
      if (s.ctx[b] >= r.prefix && s.ctx[b] <= s.cap_ctx) r.rep = b;
  }
  r.nt = r.rep < 0 ? 0 : (r.prefix + kPrefixTile - 1) / kPrefixTile;
  const int q_tiles = (r.n + s.TQ - 1) / s.TQ;
  r.pairs = q_tiles / 2;
  r.one = q_tiles & 1;
  r.head_cost = static_cast<int64_t>(r.nt) * (r.pairs * s.cost_pair + r.one * s.cost_one);
  r.cost = r.head_cost * s.Hkv;
  return r;
}

// CTAs that take a share of a line of this length: as many as get min_share
// of it, at least the cost of a tile, so that every CTA between the ends of a
// unit has a tile of it.  (Fewer, with SMs left to the decode kernel over the
// requests' own keys from the start, was no faster: 64 -> 67 us for 96 requests
// in 3 groups, 96 -> 98 us for 128 behind 32768 keys.  A decode CTA streams 50
// GB/s at most, hardly more than its part of HBM's rate when all SMs stream.)
PA_DEVINL int prefix_ctas(const PrefixShape& s, int64_t total, int max_ctas) {
  return static_cast<int>(min(static_cast<int64_t>(max_ctas), max(div_small(total, s.min_share), int64_t(1))));
}

// The CTA that place x of the line belongs to.
PA_DEVINL int prefix_cta_of(int64_t x, int64_t total, int ctas) {
  return static_cast<int>(div_small((x + 1) * ctas + total - 1, total)) - 1;
}

struct PrefixShare {
  int64_t x, x1;  // what is left of the share
  int64_t base;   // where group g starts
  int g;
  PrefixGroup gr;  // group g, once looked up
};

// CTA c's share, found by one warp (all lanes); CTA 0 also writes where each
// group starts, the line's length and the number of CTAs to costs[0 .. n_groups + 1]
// for the merge.
PA_DEVINL PrefixShare prefix_share(const PrefixShape& s, int c, int max_ctas, int64_t* costs) {
  const int lane = threadIdx.x & 31;
  PrefixShare r{0, 0, 0, s.n_groups, {}};
  int64_t total = 0;
  for (int g = lane; g < s.n_groups; g += 32) {
    const PrefixGroup gr = prefix_group(s, g);
    if (g < 32) r.gr = gr;  // the lane's first one is used again
    total += gr.cost;
  }
  PrefixGroup mine = r.gr;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const int ctas = prefix_ctas(s, total, max_ctas);
  if (c < ctas && total > 0) {
    r.x = div_small(total * c, ctas);
    r.x1 = div_small(total * (c + 1), ctas);
  }
  int64_t carry = 0;
  for (int g0 = 0; g0 < s.n_groups; g0 += 32) {
    const int g = g0 + lane;
    if (g0 > 0) {
      mine.cost = 0;
      if (g < s.n_groups) mine = prefix_group(s, g);
    }
    int64_t incl = mine.cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    incl += carry;
    if (c == 0 && g < s.n_groups) costs[g] = incl - mine.cost;
    const unsigned past = __ballot_sync(0xffffffffu, incl > r.x);
    if (past && r.g == s.n_groups) {
      const int first = __ffs(past) - 1;
      auto from = [&](auto v) { return __shfl_sync(0xffffffffu, v, first); };
      r.g = g0 + first;
      r.base = from(incl - mine.cost);
      r.gr = PrefixGroup{from(mine.s0),  from(mine.n),   from(mine.prefix),    from(mine.nt),  from(mine.rep),
                         from(mine.pairs), from(mine.one), from(mine.head_cost), from(mine.cost)};
      if (c != 0) break;
    }
    carry = __shfl_sync(0xffffffffu, incl, 31);
  }
  if (c == 0 && lane == 0) {
    costs[s.n_groups] = total;
    costs[s.n_groups + 1] = ctas;
  }
  return r;
}

// A unit of a group: where it starts on the line, and its tiles' cost.
struct PrefixUnit {
  int64_t start;
  int qp, cost;
};
PA_DEVINL PrefixUnit prefix_unit(const PrefixShape& s, const PrefixGroup& gr, int64_t base, int h, int qp) {
  PrefixUnit u;
  u.qp = qp;
  u.cost = qp < gr.pairs ? s.cost_pair : s.cost_one;
  u.start = base + h * gr.head_cost + static_cast<int64_t>(qp) * gr.nt * s.cost_pair;
  return u;
}

// Tiles [lo, hi) of a unit that start in [x0, x1) of the line.
PA_DEVINL int prefix_tile_at(const PrefixUnit& u, int nt, int64_t x) {
  return x <= u.start ? 0 : static_cast<int>(min(static_cast<int64_t>(nt), div_small(x - u.start + u.cost - 1, u.cost)));
}

struct PrefixWork {
  int rep, s0, n, prefix;
  int h, qp, j_lo, j_hi;
};

// The share's next unit with tiles in it (one thread); false at the end.
PA_DEVINL bool next_prefix_work(const PrefixShape& s, PrefixShare& sh, PrefixWork& w) {
  while (sh.x < sh.x1 && sh.g < s.n_groups) {
    const PrefixGroup& gr = sh.gr;
    const int64_t rel = sh.x - sh.base;
    if (rel >= gr.cost) {
      sh.base += gr.cost;
      if (++sh.g < s.n_groups) sh.gr = prefix_group(s, sh.g);
      continue;
    }
    const int h = static_cast<int>(div_small(rel, gr.head_cost));
    const int64_t y = rel - h * gr.head_cost;
    const int qp = static_cast<int>(min(static_cast<int64_t>(gr.pairs), div_small(y, static_cast<int64_t>(gr.nt) * s.cost_pair)));
    const PrefixUnit u = prefix_unit(s, gr, sh.base, h, qp);
    const int j_lo = prefix_tile_at(u, gr.nt, sh.x), j_hi = prefix_tile_at(u, gr.nt, sh.x1);
    sh.x = u.start + static_cast<int64_t>(gr.nt) * u.cost;
    if (j_lo >= j_hi) continue;
    w.rep = gr.rep;
    w.s0 = gr.s0;
    w.n = gr.n;
    w.prefix = gr.prefix;
    w.h = h;
    w.qp = qp;
    w.j_lo = j_lo;
    w.j_hi = j_hi;
    return true;
  }
  return false;
}

}  // namespace pa
