// Attention of tiles of query rows to a paged K/V cache for the types that the
// tcgen05 kernel does not take (fp32; bf16 with head_dim 64): chunked prefill over
// a sliding window with sinks, and the prefixes that groups of decode requests
// share.
//
// A CTA has up to 64 rows (bf16; fp32 32) of one kv-head: tokens x the G q-heads
// that share it, so that a K/V tile in shared memory serves them all.  It goes
// through the tiles of 64 keys that some row sees, copied 16 bytes at a time
// (cp.async; bf16: the next tile while this one is at work; fp32: one tile, and
// more CTAs an SM instead -- 1200 tokens of 32 q-heads over 8 of 128 dims: 521 us
// with one stage and two CTAs, 670 with two stages and one CTA; 4 requests of 100
// to 300 tokens over 900 to 1500, 16 over 4 heads of 64 dims: 127 and 176), with
// an online softmax in base 2:
//   bf16   16 rows a warp, S = Q K^T and O += P V as mma.sync m16n8k16 with fp32
//          sums, K and V fragments by ldmatrix from swizzled rows.
//   fp32   8 rows a warp (4 or 2 where that leaves no row over), a lane two keys of
//          the tile for the scores (packed fp32 pairs) and head_dim / 32 dims for
//          the output: fp32 throughout; with 128 dims the fp32 pipe is busy 43% of
//          the time with 8 warps an SM, what its shared memory holds.
// Rows that no query sees are zero in shared memory and have probability 0; they
// are not read, and neither are table entries of pages that hold only such rows.
// Keys of a page that is out of range are left out.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "pa_common.cuh"
#include "prefix_plan.cuh"

namespace pa {
namespace {

constexpr int kTileKeys = 64;
constexpr int kTileThreads = 128;

template <typename T, int HD>
struct TileGeom {
  static constexpr bool kMma = sizeof(T) == 2;
  static constexpr int kRows = kMma ? 64 : 32;
  static constexpr int kWarpRows = kRows / (kTileThreads / 32);
  static constexpr int kPitch = kMma ? HD * 2 : (HD + 4) * 4;  // bytes of a K row (fp32: lanes' rows in different banks)
  static constexpr int kVPitch = HD * static_cast<int>(sizeof(T));
  static constexpr int kStage = kTileKeys * (kPitch + kVPitch);
  static constexpr int kStages = kMma ? 2 : 1;
  static constexpr int kOffQ = kStages * kStage;                         // fp32: the rows' queries, scaled
  static constexpr int kOffP = kOffQ + (kMma ? 0 : kRows * HD * 4);      // fp32: probabilities
  static constexpr int kOffWork = kOffP + (kMma ? 0 : kRows * kTileKeys * 4);
  static constexpr int kSmem = kOffWork + 64;
  static_assert(!kMma || HD == 64, "rows of 128 bytes: eight chunks, swizzled");
};

struct TileParams {
  const char* q;
  const char* k_cache;
  const char* v_cache;
  const int32_t* bt;
  unsigned int* err;
  int64_t num_pages;
  int32_t Hq, Hkv, G, maxp, log2P;
  float scale_log2;
  // chunked prefill over a window
  const int32_t* cu;
  const int32_t* ctx;
  char* out;
  int64_t num_tokens;
  int32_t max_ctx, max_q, window, sinks, q_tiles;
  // shared prefixes
  PrefixShape shape;
  int64_t* costs;
  float* o_part;
  float* lse_part;
};

// What a CTA works on: rows r (token tok0 + r / G, q-head h G + r % G) and keys.
struct TileItem {
  int64_t tok0;
  int h, rows;
  const int32_t* table;
  int pos0, pos_step;  // row r's last key is pos0 + pos_step (r / G)
  int kv_len;          // keys past the rows' last
  int gap_lo, gap_hi;  // keys that no row sees
  int window, sinks;   // of each row
};

PA_DEVINL void cp_async16(uint32_t dst, const void* src, bool live) {
  const int n = live ? 16 : 0;  // the rest is filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
PA_DEVINL void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
PA_DEVINL void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
PA_DEVINL float tile_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
PA_DEVINL void tile_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
PA_DEVINL void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
PA_DEVINL void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// The tiles of an item: those before the gap, then those after it; an item of a
// prefix has its share of them.
struct TileList {
  int first, before, skip, end;
  PA_DEVINL int key0(int j) const { return (j < before ? j : j + skip) * kTileKeys; }
};

// Page ids of a tile's four 16-row boxes: -1 where no row is seen, -2 (flagged)
// for a page out of range, whose keys are left out.
PA_DEVINL void tile_pages(const TileParams& p, const TileItem& it, int k0, int (&pg)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int a = k0 + 16 * i, z = min(a + 16, it.kv_len);
    pg[i] = -1;
    if (a < z && !(a >= it.gap_lo && z <= it.gap_hi)) {
      const int page = it.table[a >> p.log2P];
      pg[i] = page >= 0 && page < p.num_pages ? page : -2;
    }
  }
}

template <typename T, int HD>
PA_DEVINL void tile_copy(const TileParams& p, const TileItem& it, int k0, const int (&pg)[4], uint32_t stage) {
  using Gm = TileGeom<T, HD>;
  constexpr int E = sizeof(T), CH = HD * E / 16;  // 16-byte chunks of a row
  constexpr int PER = kTileKeys * CH / kTileThreads;
  const int64_t row_bytes = static_cast<int64_t>(p.Hkv) * HD * E;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = threadIdx.x + kTileThreads * j;
    const int r = i / CH, c = i % CH, key = k0 + r;
    const int page = pg[j * 4 / PER];  // (row r lies in box r / 16)
    const bool live = page >= 0 && key < it.kv_len && !(key >= it.gap_lo && key < it.gap_hi);
    const int64_t slot = live ? (static_cast<int64_t>(page) << p.log2P) + (key & ((1 << p.log2P) - 1)) : 0;
    const int64_t at = slot * row_bytes + it.h * HD * E + c * 16;
    const int cs = Gm::kMma ? c ^ (r & 7) : c;
    cp_async16(stage + r * Gm::kPitch + cs * 16, p.k_cache + at, live);
    cp_async16(stage + kTileKeys * Gm::kPitch + r * Gm::kVPitch + cs * 16, p.v_cache + at, live);
  }
  static_assert(PER % 4 == 0, "a quarter of a thread's chunks lies in each box");
}

// The rows' results: to the output, or as a part.
template <typename T, int HD, bool kPrefix>
struct TileOut {
  const TileParams& p;
  const TileItem& it;
  int64_t part_row;
  PA_DEVINL int64_t row(int r) const {
    return kPrefix ? part_row + r : (it.tok0 + r / p.G) * p.Hq + it.h * p.G + r % p.G;
  }
  PA_DEVINL void store2(int r, int d, float a, float b) const {
    const int64_t e = row(r) * HD + d;
    if constexpr (kPrefix)
      *reinterpret_cast<float2*>(p.o_part + e) = make_float2(a, b);
    else if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint32_t*>(p.out + e * 2) = pack_bf16x2(a, b);
    else
      *reinterpret_cast<float2*>(p.out + e * 4) = make_float2(a, b);
  }
  PA_DEVINL void store_lse(int r, float m, float l) const {
    if constexpr (kPrefix) p.lse_part[row(r)] = l != 0.f ? m + log2f(l) : -INFINITY;
  }
};

template <typename T, int HD, bool kPrefix>
PA_DEVINL void tile_run(const TileParams& p, const TileItem& it, const TileList& list, int64_t part_row,
                        unsigned char* smem) {
  using Gm = TileGeom<T, HD>;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t smem0 = smem_u32(smem);
  // rows of this warp: 16, or (fp32) 2, 4 or 8, as many as its loops work on: a row is one warp's
  const int nr = Gm::kMma ? Gm::kWarpRows : it.rows <= 8 ? 2 : it.rows <= 16 ? 4 : 8;
  const int row0 = warp * nr;
  const bool busy = row0 < it.rows;  // the warp has rows
  const TileOut<T, HD, kPrefix> out{p, it, part_row};
  auto seen = [&](int pos, int key) {
    return key <= pos && (kPrefix || key > pos - it.window || key < it.sinks);
  };
  auto pos_of = [&](int r) { return it.pos0 + it.pos_step * (r / p.G); };

  int pg[4], pg_next[4];
  tile_pages(p, it, list.key0(list.first), pg);
  if constexpr (Gm::kStages == 2) {
    tile_copy<T, HD>(p, it, list.key0(list.first), pg, smem0);
    cp_async_commit();
  }

  constexpr int KS = HD / 16;
  [[maybe_unused]] uint32_t qa[KS][4];
  [[maybe_unused]] float o4[HD / 8][4];
  constexpr int R = Gm::kMma ? 2 : Gm::kWarpRows;  // rows that a lane keeps the statistics of
  constexpr int DL = HD / 32;
  [[maybe_unused]] float o1[Gm::kMma ? 1 : R][DL];
  float m[R], l[R];
  int pos[R];
  const int gq = lane >> 2, tq = lane & 3;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
    pos[r] = pos_of(row0 + (Gm::kMma ? gq + 8 * r : r));
  }
  if constexpr (Gm::kMma) {
#pragma unroll
    for (int i = 0; i < HD / 8; ++i) o4[i][0] = o4[i][1] = o4[i][2] = o4[i][3] = 0.f;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = row0 + gq + 8 * half;
      const bool live = r < it.rows;
      const char* src = p.q + ((it.tok0 + (live ? r / p.G : 0)) * p.Hq + it.h * p.G + (live ? r % p.G : 0)) * HD * 2;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qa[ks][half] = live ? *reinterpret_cast<const uint32_t*>(src + (ks * 16 + 2 * tq) * 2) : 0u;
        qa[ks][2 + half] = live ? *reinterpret_cast<const uint32_t*>(src + (ks * 16 + 8 + 2 * tq) * 2) : 0u;
      }
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < DL; ++e) o1[r][e] = 0.f;
    float* qs = reinterpret_cast<float*>(smem + Gm::kOffQ);
    for (int i = tid; i < Gm::kRows * HD / 4; i += kTileThreads) {
      const int r = i / (HD / 4), d = i % (HD / 4) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < it.rows)
        v = *reinterpret_cast<const float4*>(
            p.q + (((it.tok0 + r / p.G) * p.Hq + it.h * p.G + r % p.G) * HD + d) * 4);
      *reinterpret_cast<float4*>(qs + r * HD + d) =
          make_float4(v.x * p.scale_log2, v.y * p.scale_log2, v.z * p.scale_log2, v.w * p.scale_log2);
    }
  }
  const int pos_min = pos_of(row0), pos_max = pos_of(min(it.rows, row0 + nr) - 1);

  for (int j = list.first; j < list.end; ++j) {
    const int k0 = list.key0(j), n = j - list.first;
    const bool more = j + 1 < list.end;
    if (more) tile_pages(p, it, list.key0(j + 1), pg_next);
    if constexpr (Gm::kStages == 2) {
      if (more) {
        tile_copy<T, HD>(p, it, list.key0(j + 1), pg_next, smem0 + ((n + 1) & 1) * Gm::kStage);
        cp_async_commit();
        cp_async_wait<1>();
      } else {
        cp_async_wait<0>();
      }
    } else {
      tile_copy<T, HD>(p, it, k0, pg, smem0);
      cp_async_commit();
      cp_async_wait<0>();
    }
    cta_sync();  // the tile (and, the first time, the queries) is in shared memory
    const bool bad = pg[0] == -2 || pg[1] == -2 || pg[2] == -2 || pg[3] == -2;
    if (bad && tid == 0) raise_flag(p.err, PA_DEVERR_BAD_PAGE);
    auto live_key = [&](int key) {  // not of a page that is out of range
      const int i = (key - k0) >> 4;
      return (i == 0 ? pg[0] : i == 1 ? pg[1] : i == 2 ? pg[2] : pg[3]) != -2;
    };
    // some row may not see some key: past its own, before its window, or left out
    const bool mask = bad || k0 + kTileKeys - 1 > pos_min ||
                      (!kPrefix && k0 <= pos_max - it.window && k0 + kTileKeys > it.sinks);
    const uint32_t kst = smem0 + (Gm::kStages == 2 ? (n & 1) * Gm::kStage : 0), vst = kst + kTileKeys * Gm::kPitch;
    if (busy) {
      if constexpr (Gm::kMma) {
        const int lrow = lane & 7, lmat = lane >> 3;
        float s[8][4];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
          const uint32_t row = kst + (t * 8 + lrow) * Gm::kPitch;
#pragma unroll
          for (int kk = 0; kk < KS / 2; ++kk) {
            uint32_t b[4];
            ldsm4(b, row + (((kk * 4 + lmat) ^ lrow) << 4));
            tile_mma(s[t], qa[2 * kk], b[0], b[1]);
            tile_mma(s[t], qa[2 * kk + 1], b[2], b[3]);
          }
        }
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[t][e] *= p.scale_log2;
            if (mask) {
              const int key = k0 + t * 8 + 2 * tq + (e & 1);
              if (!seen(pos[e >> 1], key) || (bad && !live_key(key))) s[t][e] = -INFINITY;
            }
            mx[e >> 1] = fmaxf(mx[e >> 1], s[t][e]);
          }
        float neg[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
          const float m_new = fmaxf(m[r], mx[r]), m_use = m_new == -INFINITY ? 0.f : m_new;
          const float alpha = tile_ex2(m[r] - m_use);
          m[r] = m_new;
          neg[r] = m_use;
          l[r] *= alpha;
#pragma unroll
          for (int i = 0; i < HD / 8; ++i) {
            o4[i][2 * r] *= alpha;
            o4[i][2 * r + 1] *= alpha;
          }
        }
#pragma unroll
        for (int ks = 0; ks < kTileKeys / 16; ++ks) {
          uint32_t pa[4];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float (&t)[4] = s[2 * ks + u];
#pragma unroll
            for (int e = 0; e < 4; ++e) t[e] = tile_ex2(t[e] - neg[e >> 1]);
            l[0] += t[0] + t[1];
            l[1] += t[2] + t[3];
            // the products take the probabilities rounded to bf16, the sum as they are
            pa[2 * u] = pack_bf16x2(t[0], t[1]);
            pa[2 * u + 1] = pack_bf16x2(t[2], t[3]);
          }
          const int r = ks * 16 + (lmat & 1) * 8 + lrow;
#pragma unroll
          for (int nn = 0; nn < HD / 16; ++nn) {
            uint32_t b[4];
            ldsm4_t(b, vst + r * Gm::kVPitch + (((nn * 2 + (lmat >> 1)) ^ lrow) << 4));
            tile_mma(o4[2 * nn], pa, b[0], b[1]);
            tile_mma(o4[2 * nn + 1], pa, b[2], b[3]);
          }
        }
      } else {
        // (for 2, 4 or 8 rows, so that few rows cost little and the sums stay in registers)
        auto tile_rows = [&](auto rows_c) {
          constexpr int NR = decltype(rows_c)::value;
          const float* qs = reinterpret_cast<const float*>(smem + Gm::kOffQ) + row0 * HD;
          float* ps = reinterpret_cast<float*>(smem + Gm::kOffP) + row0 * kTileKeys;
          const float* kf = reinterpret_cast<const float*>(smem + (kst - smem0));
          const float* vf = reinterpret_cast<const float*>(smem + (vst - smem0));
          float2 acc[NR][2];
#pragma unroll
          for (int r = 0; r < NR; ++r) acc[r][0] = acc[r][1] = make_float2(0.f, 0.f);
#pragma unroll 4
          for (int d = 0; d < HD; d += 4) {
            const float4 ka = *reinterpret_cast<const float4*>(kf + lane * (HD + 4) + d);
            const float4 kb = *reinterpret_cast<const float4*>(kf + (lane + 32) * (HD + 4) + d);
#pragma unroll
            for (int r = 0; r < NR; ++r) {
              const float4 qv = *reinterpret_cast<const float4*>(qs + r * HD + d);
              acc[r][0] = ffma2(make_float2(qv.x, qv.y), make_float2(ka.x, ka.y), acc[r][0]);
              acc[r][0] = ffma2(make_float2(qv.z, qv.w), make_float2(ka.z, ka.w), acc[r][0]);
              acc[r][1] = ffma2(make_float2(qv.x, qv.y), make_float2(kb.x, kb.y), acc[r][1]);
              acc[r][1] = ffma2(make_float2(qv.z, qv.w), make_float2(kb.z, kb.w), acc[r][1]);
            }
          }
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            float s0 = acc[r][0].x + acc[r][0].y, s1 = acc[r][1].x + acc[r][1].y;
            if (mask) {
              const int ka = k0 + lane, kb = ka + 32;
              if (!seen(pos[r], ka) || (bad && !live_key(ka))) s0 = -INFINITY;
              if (!seen(pos[r], kb) || (bad && !live_key(kb))) s1 = -INFINITY;
            }
            float mx = fmaxf(s0, s1);
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float m_new = fmaxf(m[r], mx), m_use = m_new == -INFINITY ? 0.f : m_new;
            const float alpha = tile_ex2(m[r] - m_use);
            m[r] = m_new;
            const float p0 = tile_ex2(s0 - m_use), p1 = tile_ex2(s1 - m_use);
            l[r] = l[r] * alpha + (p0 + p1);  // this lane's share of the sum
            ps[r * kTileKeys + lane] = p0;
            ps[r * kTileKeys + lane + 32] = p1;
#pragma unroll
            for (int e = 0; e < DL; ++e) o1[r][e] *= alpha;
          }
          __syncwarp();
#pragma unroll 4
          for (int k = 0; k < kTileKeys; k += 4) {
            float v[4][DL];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const float* src = vf + (k + u) * HD + lane * DL;
              if constexpr (DL == 4) {
                const float4 w = *reinterpret_cast<const float4*>(src);
                v[u][0] = w.x, v[u][1] = w.y, v[u][2] = w.z, v[u][3] = w.w;
              } else {
                const float2 w = *reinterpret_cast<const float2*>(src);
                v[u][0] = w.x, v[u][1] = w.y;
              }
            }
#pragma unroll
            for (int r = 0; r < NR; ++r) {
              const float4 pv = *reinterpret_cast<const float4*>(ps + r * kTileKeys + k);
#pragma unroll
              for (int e = 0; e < DL; ++e)
                o1[r][e] = fmaf(pv.w, v[3][e], fmaf(pv.z, v[2][e], fmaf(pv.y, v[1][e], fmaf(pv.x, v[0][e], o1[r][e]))));
            }
          }
        };
        if (nr <= 2) tile_rows(std::integral_constant<int, 2>{});
        else if (nr <= 4) tile_rows(std::integral_constant<int, 4>{});
        else tile_rows(std::integral_constant<int, 8>{});
      }
    }
    cta_sync();  // the stage may be filled again
#pragma unroll
    for (int i = 0; i < 4; ++i) pg[i] = pg_next[i];
  }

  if (!busy) return;
  if constexpr (Gm::kMma) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      const int row = row0 + gq + 8 * r;
      if (row < it.rows) {
        const float inv = l[r] > 0.f ? 1.f / l[r] : 0.f;
#pragma unroll
        for (int i = 0; i < HD / 8; ++i) out.store2(row, i * 8 + 2 * tq, o4[i][2 * r] * inv, o4[i][2 * r + 1] * inv);
        if (tq == 0) out.store_lse(row, m[r], l[r]);
      }
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
      if (r >= nr || row0 + r >= it.rows) continue;
      const float inv = l[r] > 0.f ? 1.f / l[r] : 0.f;
#pragma unroll
      for (int e = 0; e < DL; e += 2) out.store2(row0 + r, lane * DL + e, o1[r][e] * inv, o1[r][e + 1] * inv);
      if (lane == 0) out.store_lse(row0 + r, m[r], l[r]);
    }
  }
}

// Chunked prefill: CTA = (q-tile of a request, kv-head).
template <typename T, int HD>
__global__ void __launch_bounds__(kTileThreads) window_tile_kernel(const TileParams p) {
  extern __shared__ __align__(128) unsigned char tile_smem[];
  const int b = blockIdx.x / p.q_tiles, TQ = TileGeom<T, HD>::kRows / p.G;
  const int s0 = p.cu[b], s1 = p.cu[b + 1], n = s1 - s0, L = p.ctx[b];
  const int t0 = (blockIdx.x - b * p.q_tiles) * TQ;
  if (L == 0 && s0 >= 0 && s1 <= p.num_tokens) return;  // a padding row
  const int cap = static_cast<int>(min(static_cast<int64_t>(p.max_ctx), static_cast<int64_t>(p.maxp) << p.log2P));
  if (s0 < 0 || s1 > p.num_tokens || n < 0 || n > p.max_q || L < n || L > cap) {
    if (threadIdx.x == 0) raise_flag(p.err, PA_DEVERR_BAD_LENGTH);
    return;
  }
  if (t0 >= n) return;
  const int toks = min(TQ, n - t0);
  TileItem it;
  it.tok0 = static_cast<int64_t>(s0) + t0;
  it.h = blockIdx.y;
  it.rows = toks * p.G;
  it.table = p.bt + static_cast<int64_t>(b) * p.maxp;
  it.pos0 = L - n + t0;
  it.pos_step = 1;
  it.kv_len = it.pos0 + toks;
  it.gap_hi = max(0, it.pos0 - p.window + 1);
  it.gap_lo = min(p.sinks, it.gap_hi);
  it.window = p.window;
  it.sinks = p.sinks;
  TileList list;
  list.first = 0;
  list.before = (it.gap_lo + kTileKeys - 1) / kTileKeys;
  list.skip = max(0, it.gap_hi / kTileKeys - list.before);
  list.end = (it.kv_len + kTileKeys - 1) / kTileKeys - list.skip;
  tile_run<T, HD, false>(p, it, list, 0, tile_smem);
}

// Shared prefixes: each CTA has its share of the groups' tiles (prefix_plan.cuh).
template <typename T, int HD>
__global__ void __launch_bounds__(kTileThreads) prefix_tile_kernel(const TileParams p) {
  using Gm = TileGeom<T, HD>;
  extern __shared__ __align__(128) unsigned char tile_smem[];
  PrefixWork& work = *reinterpret_cast<PrefixWork*>(tile_smem + Gm::kOffWork);
  int& more = *reinterpret_cast<int*>(&work + 1);
  static_assert(sizeof(PrefixWork) + sizeof(int) <= 64, "the unit at work and the flag fit");
  pdl_trigger();  // the decode kernel over the requests' own keys may start
  PrefixShare share;
  if (threadIdx.x < 32) share = prefix_share(p.shape, blockIdx.x, gridDim.x, p.costs);
  for (;;) {
    if (threadIdx.x == 0) {
      PrefixWork w;
      more = next_prefix_work(p.shape, share, w);
      work = w;
    }
    cta_sync();
    if (!more) return;
    const PrefixWork w = work;
    const int t0 = 2 * w.qp * p.shape.TQ;  // the unit's first request in its group
    TileItem it;
    it.tok0 = static_cast<int64_t>(w.s0) + t0;
    it.h = w.h;
    it.rows = min(2 * p.shape.TQ, w.n - t0) * p.G;
    it.table = p.bt + static_cast<int64_t>(w.rep) * p.maxp;
    it.pos0 = w.prefix - 1;
    it.pos_step = 0;
    it.kv_len = w.prefix;
    it.gap_lo = it.gap_hi = 0;
    it.window = it.sinks = 0;
    constexpr int kSub = kPrefixTile / kTileKeys;
    TileList list;
    list.first = w.j_lo * kSub;
    list.before = list.skip = 0;
    list.end = min(w.j_hi * kSub, (w.prefix + kTileKeys - 1) / kTileKeys);
    // (every warp has copied `work` by the barriers of its tiles, before it is written again)
    tile_run<T, HD, true>(p, it, list, prefix_part_row(p.shape, w.s0, w.n, w.h, blockIdx.x, p.Hq, p.G) + t0 * p.G, tile_smem);
  }
}

TileParams tile_params(const pa_cache_desc& d, const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* bt, int32_t maxp, float scale, unsigned int* err) {
  TileParams p{};
  p.q = static_cast<const char*>(q);
  p.k_cache = static_cast<const char*>(k_cache);
  p.v_cache = static_cast<const char*>(v_cache);
  p.bt = bt;
  p.err = err;
  p.num_pages = d.num_pages;
  p.Hq = d.num_q_heads;
  p.Hkv = d.num_kv_heads;
  p.G = d.num_q_heads / d.num_kv_heads;
  p.maxp = maxp;
  while ((1 << p.log2P) < d.page_size) ++p.log2P;
  p.scale_log2 = scale * 1.4426950408889634f;
  return p;
}

// fn with its dynamic shared memory allowed (an attribute of the function, the same every time).
template <typename T, int HD>
cudaError_t launch_tile(const void* fn, dim3 grid, TileParams& p, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, TileGeom<T, HD>::kSmem);
  if (e != cudaSuccess) return e;
  void* args[] = {&p};
  return cudaLaunchKernel(fn, grid, dim3(kTileThreads), args, TileGeom<T, HD>::kSmem, s);
}

template <typename T, int HD>
cudaError_t launch_window(const pa_cache_desc& d, const PrefillArgs& a, cudaStream_t s) {
  TileParams p = tile_params(d, a.q, a.k_cache, a.v_cache, a.block_tables, a.max_pages, a.scale, a.err);
  p.cu = a.cu_seqlens_q;
  p.ctx = a.context_lens;
  p.out = static_cast<char*>(a.out);
  p.num_tokens = a.num_tokens;
  p.max_ctx = a.max_context_len;
  p.max_q = a.max_seqlen_q;
  p.window = a.window;
  p.sinks = a.sinks;
  const int TQ = TileGeom<T, HD>::kRows / p.G;
  p.q_tiles = (a.max_seqlen_q + TQ - 1) / TQ;
  const int64_t tiles = static_cast<int64_t>(p.q_tiles) * a.batch;
  if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(tiles), d.num_kv_heads);
  return launch_tile<T, HD>(reinterpret_cast<const void*>(window_tile_kernel<T, HD>), grid, p, s);
}

template <typename T, int HD>
cudaError_t launch_prefix(const pa_cache_desc& d, const SharedArgs& a, const SharedPlan& pl, cudaStream_t s) {
  TileParams p = tile_params(d, a.q, a.k_cache, a.v_cache, a.block_tables, a.max_pages, a.scale, a.err);
  char* ws = static_cast<char*>(a.workspace);
  p.shape = prefix_shape(d, a, pl);
  p.costs = reinterpret_cast<int64_t*>(ws + pl.off_costs);
  p.o_part = reinterpret_cast<float*>(ws + pl.off_o);
  p.lse_part = reinterpret_cast<float*>(ws + pl.off_lse);
  return launch_tile<T, HD>(reinterpret_cast<const void*>(prefix_tile_kernel<T, HD>), dim3(pl.prefix_ctas), p, s);
}

}  // namespace

int prefix_tile_rows(const pa_cache_desc& d) {
  return d.dtype == PA_BF16 ? TileGeom<__nv_bfloat16, 64>::kRows : TileGeom<float, 64>::kRows;
}

cudaError_t launch_prefill_window_tile(const pa_cache_desc& d, const PrefillArgs& a, cudaStream_t s) {
  if (a.num_tokens == 0 || a.batch == 0) return cudaSuccess;
  if (d.dtype == PA_BF16) return launch_window<__nv_bfloat16, 64>(d, a, s);
  return d.head_dim == 128 ? launch_window<float, 128>(d, a, s) : launch_window<float, 64>(d, a, s);
}

cudaError_t launch_prefix_tile(const pa_cache_desc& d, const SharedArgs& a, const SharedPlan& pl, cudaStream_t s) {
  if (d.dtype == PA_BF16) return launch_prefix<__nv_bfloat16, 64>(d, a, pl, s);
  return d.head_dim == 128 ? launch_prefix<float, 128>(d, a, pl, s) : launch_prefix<float, 64>(d, a, pl, s);
}

}  // namespace pa
