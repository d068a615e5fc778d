// Block tables on the GPU: pages for a batch's new tokens out of a ring of free
// pages, with the tokens' positions and slots; pages that rows share; pages
// handed back.  The host block manager's rules (nano-vLLM learning note,
// BlockManager.allocate, may_append, deallocate listings: first in, first out; a
// page counted by its holders; a sequence's last page returned first) as device
// calls that a captured step can make.
//
//   need_b   = ceil((L_b + n_b) / P) - ceil(L_b / P)
//   entry i  = ring[(taken + sum_{b'<b} need_b' + i - ceil(L_b / P)) mod num_pages]
//   slot     = table[pos / P] * P + pos mod P
//
// All of it is latency: a few kilobytes, prefix sums over the requests, a look-up
// for each new page and token.  One launch a call, of one thread block cluster (or
// a single CTA where there is little to do): every CTA works the prefix sums out
// for itself and takes its share of the pages, tokens or entries; the cluster's
// barrier separates the reads of the state from its update, so inputs and
// outputs may be the same arrays, and there is no workspace.  GPU us: the next
// token of 256 requests 5.2; 32 of 64 rows take over up to 512 pages of the others
// 2.3, 64 rows get 22000 tokens 8.6, those 32 hand 9000 entries back 10.
#include <algorithm>

#include "pa_common.cuh"

namespace pa {
namespace {

constexpr int kTabThreads = 512;  // also the requests per pass of the prefix sums
constexpr int kTabAhead = 4;       // look-ups that a thread has in flight
constexpr int kTabRun = 8;         // entries of a row that it goes through together
constexpr int kTabCluster = 8;
constexpr int kMaxReleaseRows = 32768;  // their prefix sums are in shared memory

PA_DEVINL void cluster_barrier(int cluster) {
  __syncwarp();
  if (cluster > 1)
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  else
    __syncthreads();
}

// Exclusive prefix sums of two numbers over the CTA, and their totals.
PA_DEVINL longlong2 scan2(longlong2 v, longlong2* sh, longlong2* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int NW = kTabThreads / 32;
  long long x = v.x, y = v.y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, x, o), b = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) x += a, y += b;
  }
  cta_sync();  // (the totals of an earlier scan have been read)
  if (lane == 31) sh[warp] = make_longlong2(x, y);
  cta_sync();
  longlong2 before = make_longlong2(0, 0), all = before;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const longlong2 t = sh[w];
    if (w < warp) before.x += t.x, before.y += t.y;
    all.x += t.x, all.y += t.y;
  }
  *total = all;
  return make_longlong2(before.x + x - v.x, before.y + y - v.y);
}

// The last i of [0, n) with sums[i] <= x (sums ascending, sums[0] <= x).
PA_DEVINL int last_at_or_below(const int32_t* sums, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sums[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kTabThreads) extend_tables_kernel(const ExtendParams p) {
  __shared__ longlong2 sh[kTabThreads / 32];
  __shared__ int32_t s_len[kTabThreads], s_tok[kTabThreads], s_page[kTabThreads];
  const int tid = threadIdx.x, rank = blockIdx.x, R = gridDim.x;
  const int64_t cap = min(static_cast<int64_t>(p.maxp) << p.log2P, static_cast<int64_t>(0x7fffffff));
  const int64_t taken = p.pool[0], returned = p.pool[1];
  int64_t free_pages = returned - taken;
  if (taken < 0 || free_pages < 0 || free_pages > p.num_pages) {
    if (rank == 0 && tid == 0) raise_flag(p.err, PA_DEVERR_BAD_LENGTH);
    free_pages = 0;
  }
  const int64_t ring0 = free_pages > 0 ? taken % p.num_pages : 0;  // the ring's first free entry
  int64_t pages_asked = 0, tokens_asked = 0, pages = 0, tokens = 0;  // of the requests before this pass
  for (int b0 = 0; b0 < p.batch; b0 += kTabThreads) {
    const int b = b0 + tid;
    int L = 0, n = 0, need = 0;
    unsigned int flag = 0;
    if (b < p.batch) {
      L = p.ctx[b];
      n = p.new_tokens[b];
      if (L < 0 || n < 0 || static_cast<int64_t>(L) + n > cap) {
        flag = PA_DEVERR_BAD_LENGTH;
        n = 0;
      }
      const int64_t P1 = (int64_t(1) << p.log2P) - 1;
      if (n > 0) need = static_cast<int>(((static_cast<int64_t>(L) + n + P1) >> p.log2P) - ((L + P1) >> p.log2P));
    }
    longlong2 total;
    const longlong2 before = scan2(make_longlong2(need, n), sh, &total);
    const bool room = tokens_asked + before.y + n <= p.max_tokens;
    const bool fits = need == 0 || pages_asked + before.x + need <= free_pages;
    const bool refused = n > 0 && !(room && fits);
    if (refused) flag |= (room ? 0u : PA_DEVERR_BAD_LENGTH) | (fits ? 0u : PA_DEVERR_NO_PAGES);
    if (rank == 0 && flag) raise_flag(p.err, flag);
    const int granted = refused ? 0 : n;
    // Pages are refused from some request on, so those granted lie where they
    // were asked for; tokens in a row's last page may follow a refusal.
    longlong2 got = before, got_total = total;
    __syncwarp();
    if (__syncthreads_or(refused)) got = scan2(make_longlong2(refused ? 0 : need, granted), sh, &got_total);
    s_len[tid] = L;
    s_tok[tid] = static_cast<int>(got.y);
    s_page[tid] = static_cast<int>(got.x);
    cluster_barrier(R);  // every CTA has read these requests' lengths (and its sums are complete)
    if (rank == 0 && b < p.batch) {
      p.ctx_out[b] = L + granted;
      p.cu[b + 1] = static_cast<int>(tokens + got.y + granted);
    }
    const int rows = min(kTabThreads, p.batch - b0);
    auto page_at = [&](int64_t k) {  // page k of those granted in this pass
      int64_t i = ring0 + pages + k;
      if (i >= p.num_pages) i -= p.num_pages;
      return p.ring[i];
    };
    for (int64_t k = static_cast<int64_t>(rank) * kTabThreads + tid; k < got_total.x;
         k += static_cast<int64_t>(R) * kTabThreads) {
      const int i = last_at_or_below(s_page, rows, static_cast<int>(k));
      const int held = (static_cast<int64_t>(s_len[i]) + (1 << p.log2P) - 1) >> p.log2P;
      int page = page_at(k);
      if (page < 0 || page >= p.num_pages) {
        raise_flag(p.err, PA_DEVERR_BAD_PAGE);
        page = -1;
      } else if (p.refs) {
        p.refs[page] = 1;
      }
      p.bt[static_cast<int64_t>(b0 + i) * p.maxp + held + (k - s_page[i])] = page;
    }
    const int64_t step = static_cast<int64_t>(R) * kTabThreads;
    for (int64_t t0 = static_cast<int64_t>(rank) * kTabThreads + tid; t0 < got_total.y; t0 += kTabAhead * step) {
      int pos[kTabAhead], page[kTabAhead];
#pragma unroll
      for (int u = 0; u < kTabAhead; ++u) {
        const int64_t t = t0 + u * step;
        if (t >= got_total.y) break;
        const int i = last_at_or_below(s_tok, rows, static_cast<int>(t));
        pos[u] = s_len[i] + static_cast<int>(t - s_tok[i]);
        const int held = (static_cast<int64_t>(s_len[i]) + (1 << p.log2P) - 1) >> p.log2P, at = pos[u] >> p.log2P;
        page[u] = at < held ? p.bt[static_cast<int64_t>(b0 + i) * p.maxp + at] : page_at(s_page[i] + at - held);
      }
#pragma unroll
      for (int u = 0; u < kTabAhead; ++u) {
        const int64_t t = t0 + u * step;
        if (t >= got_total.y) break;
        int64_t slot = -1;
        if (page[u] >= 0 && page[u] < p.num_pages)
          slot = (static_cast<int64_t>(page[u]) << p.log2P) + (pos[u] & ((1 << p.log2P) - 1));
        else
          raise_flag(p.err, PA_DEVERR_BAD_PAGE);
        p.positions[tokens + t] = pos[u];
        p.slots[tokens + t] = slot;
      }
    }
    pages_asked += total.x;
    tokens_asked += total.y;
    pages += got_total.x;
    tokens += got_total.y;
    cta_sync();  // the pass's sums have been read
  }
  cluster_barrier(R);  // every CTA has read the pool's state
  if (rank == 0 && tid == 0) {
    p.cu[0] = 0;
    p.pool_out[0] = taken + pages;
    p.pool_out[1] = returned;
  }
  for (int64_t t = tokens + static_cast<int64_t>(rank) * kTabThreads + tid; t < p.max_tokens;
       t += static_cast<int64_t>(R) * kTabThreads) {
    p.positions[t] = 0;
    p.slots[t] = -1;
  }
}

__global__ void __launch_bounds__(128) share_pages_kernel(const ShareParams p) {
  const int b = blockIdx.x;
  const int from = p.parents[b];
  if (from < 0) return;
  const int n = p.num_pages_shared[b];
  // (a row whose own entries are being written cannot be followed)
  if (from >= p.batch || n < 0 || n > p.maxp || p.parents[from] >= 0) {
    if (threadIdx.x == 0) raise_flag(p.err, PA_DEVERR_BAD_LENGTH);
    return;
  }
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    int page = p.bt[static_cast<int64_t>(from) * p.maxp + j];
    if (page >= p.num_pages) {
      raise_flag(p.err, PA_DEVERR_BAD_PAGE);
      page = -1;
    }
    if (page >= 0) atomicAdd(&p.refs[page], 1);
    p.bt[static_cast<int64_t>(b) * p.maxp + j] = max(page, -1);
  }
}

// Entries that name the same page may be handed back together.  The page returns
// to the ring at the place of the last of them (rows in order, each from its
// last page down), whatever the order in which the GPU gets to them: an entry
// that takes the count from 1 marks the page, then the marked page's count keeps
// the largest entry, which is the one that returns it.
constexpr int kReturned = -(1 << 30);

__global__ void __launch_bounds__(kTabThreads) release_pages_kernel(const ReleaseParams p) {
  extern __shared__ int32_t s_sums[];  // [batch + 1] entries of the rows before
  __shared__ longlong2 sh[kTabThreads / 32];
  __shared__ int32_t s_count;
  const int tid = threadIdx.x, rank = blockIdx.x, R = gridDim.x;
  const int64_t taken = p.pool[0], returned = p.pool[1];
  int64_t room = p.num_pages - (returned - taken);  // entries of the ring that are not free pages
  if (taken < 0 || returned < taken || room < 0) {
    if (rank == 0 && tid == 0) raise_flag(p.err, PA_DEVERR_BAD_LENGTH);
    room = 0;
  }
  // a row's entries [first, end)
  auto range = [&](int b) {
    int64_t first, end;
    if (p.ctx) {  // what no token from position L on sees
      const int L = p.ctx[b];
      first = (static_cast<int64_t>(p.sinks) + (1 << p.log2P) - 1) >> p.log2P;
      end = max(static_cast<int64_t>(L) + 1 - p.window, int64_t(0)) >> p.log2P;
      if (L < 0 || L > (static_cast<int64_t>(p.maxp) << p.log2P)) {
        if (rank == 0) raise_flag(p.err, PA_DEVERR_BAD_LENGTH);
        first = end = 0;
      }
    } else {
      first = p.first[b];
      end = p.end[b];
      if (first < 0 || end > p.maxp) {
        if (rank == 0) raise_flag(p.err, PA_DEVERR_BAD_LENGTH);
        first = end = 0;
      }
    }
    const int64_t most = p.maxp;
    return make_int2(static_cast<int>(min(first, most)), static_cast<int>(min(end, most)));
  };
  int n_all = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kTabThreads) {
    const int b = b0 + tid;
    int n = 0;
    if (b < p.batch) {
      const int2 r = range(b);
      n = max(r.y - r.x, 0);
    }
    longlong2 total;
    const int before = static_cast<int>(scan2(make_longlong2(n, 0), sh, &total).x);
    if (b < p.batch) s_sums[b] = n_all + before;
    n_all += static_cast<int>(total.x);
  }
  if (tid == 0) s_sums[p.batch] = n_all;
  cta_sync();
  // this CTA's entries, and of those this thread's: [lo, hi), in order
  const int e0 = static_cast<int>(static_cast<int64_t>(n_all) * rank / R);
  const int e1 = static_cast<int>(static_cast<int64_t>(n_all) * (rank + 1) / R);
  const int per = (e1 - e0 + kTabThreads - 1) / kTabThreads;
  const int lo = min(e1, e0 + tid * per), hi = min(e1, lo + per);
  auto end_of = [&](int b) {
    return p.ctx ? static_cast<int>(min(max(static_cast<int64_t>(p.ctx[b]) + 1 - p.window, int64_t(0)) >> p.log2P,
                                        static_cast<int64_t>(p.maxp)))
                 : p.end[b];
  };
  auto entry = [&](int e) {  // the place of entry e in the tables
    const int b = last_at_or_below(s_sums, p.batch, e);
    return p.bt + static_cast<int64_t>(b) * p.maxp + end_of(b) - 1 - (e - s_sums[b]);
  };
  auto valid = [&](int page) { return page >= 0 && page < p.num_pages; };
  // A thread's first entries stay in registers from step to step, with their
  // look-ups in flight together; the others are looked up again.
  int32_t* place_of[kTabAhead];
  int page_of[kTabAhead];
#pragma unroll
  for (int u = 0; u < kTabAhead; ++u) place_of[u] = lo + u < hi ? entry(lo + u) : nullptr;
#pragma unroll
  for (int u = 0; u < kTabAhead; ++u) page_of[u] = place_of[u] ? *place_of[u] : -1;
  // The others, looked up again: in order, along their rows, kTabRun at a time.
  int others = lo + kTabAhead, others_end = hi;
  auto for_others = [&](auto&& f) {
    int e = others;
    if (e >= others_end) return;
    for (int b = last_at_or_below(s_sums, p.batch, e); e < others_end; ++b) {
      const int stop = min(others_end, s_sums[b + 1]);
      int32_t* place = p.bt + static_cast<int64_t>(b) * p.maxp + end_of(b) - 1 - (e - s_sums[b]);
      while (e < stop) {
        const int n = min(kTabRun, stop - e);
        int page[kTabRun];
#pragma unroll
        for (int u = 0; u < kTabRun; ++u) page[u] = u < n ? place[-u] : -1;
#pragma unroll
        for (int u = 0; u < kTabRun; ++u)
          if (u < n) f(e + u, page[u], place - u);
        e += n;
        place -= n;
      }
    }
  };
  auto for_entries = [&](auto&& f) {  // f(entry, page, place)
#pragma unroll
    for (int u = 0; u < kTabAhead; ++u)
      if (place_of[u]) f(lo + u, page_of[u], place_of[u]);
    for_others(f);
  };
  // 1. the counts
  int held = hi, held_end = 0;
  for_entries([&](int e, int page, int32_t*) {
    if (e - lo >= kTabAhead && page != -1) held = min(held, e), held_end = e + 1;
    if (page >= p.num_pages) raise_flag(p.err, PA_DEVERR_BAD_PAGE);
    if (!valid(page) || !p.refs) return;
    const int old = atomicSub(&p.refs[page], 1);
    if (old == 1) {
      atomicAdd(&p.refs[page], kReturned);
    } else if (old < 1) {  // nobody holds it any longer
      atomicAdd(&p.refs[page], 1);
      raise_flag(p.err, PA_DEVERR_BAD_PAGE);
    }
  });
  // (those that a window left in earlier calls are -1: gone through once.  256 rows
  // of 32768 tokens in pages of 16, window 1024, 16 pages handed back: 342 -> 34 us)
  others = held;
  others_end = held_end;
  if (p.refs) {
    cluster_barrier(R);
    // 2. the last entry of each page that nobody holds any longer
    for_entries([&](int e, int page, int32_t*) {
      if (valid(page) && __ldcg(&p.refs[page]) <= kReturned) atomicMin(&p.refs[page], kReturned - 1 - e);
    });
  }
  cluster_barrier(R);
  // 3. how many of this thread's entries return a page, and where in the ring
  auto returns = [&](int e, int page) {
    return valid(page) && (!p.refs || __ldcg(&p.refs[page]) == kReturned - 1 - e);
  };
  int mine = 0;
  uint32_t out_of = 0;  // those kept in registers
  for_entries([&](int e, int page, int32_t*) {
    const bool out = returns(e, page);
    mine += out;
    if (e - lo < kTabAhead) out_of |= static_cast<uint32_t>(out) << (e - lo);
  });
  longlong2 total;
  const int64_t before = scan2(make_longlong2(mine, 0), sh, &total).x;
  if (tid == 0) s_count = static_cast<int>(total.x);
  cluster_barrier(R);
  int64_t at = before, all = 0;
  for (int r = 0; r < R; ++r) {
    int n = s_count;
    if (R > 1) {
      uint32_t a;
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(&s_count)), "r"(r));
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(n) : "r"(a) : "memory");
    }
    at += r < rank ? n : 0;
    all += n;
  }
  int64_t to = (returned + at) % p.num_pages;
  for_entries([&](int e, int page, int32_t* place) {
    if (e - lo < kTabAhead ? (out_of >> (e - lo)) & 1 : returns(e, page)) {
      if (at < room) p.ring[to] = page;
      else raise_flag(p.err, PA_DEVERR_BAD_LENGTH);  // more pages than there are
      if (p.refs) p.refs[page] = 0;
      ++at;
      if (++to == p.num_pages) to = 0;
    }
    *place = -1;
  });
  if (rank == 0 && tid == 0) {
    p.pool_out[0] = taken;
    p.pool_out[1] = returned + min(all, room);
  }
  cluster_barrier(R);  // no CTA leaves while its count is read
}

cudaError_t launch_cluster(const void* fn, int ctas, size_t smem, cudaStream_t s, void** args) {
  if (ctas == 1) return cudaLaunchKernel(fn, dim3(1), dim3(kTabThreads), args, smem, s);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kTabThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

// the descriptor as the calls here need it: 32-bit page ids
pa_status check_tables(const pa_cache_desc* d, int32_t batch, int32_t max_pages_per_seq) {
  pa_status st = check_desc(d);
  if (st != PA_OK) return st;
  if (batch < 0 || max_pages_per_seq < 1) return PA_ERR_SHAPE;
  if (d->num_pages >= int64_t(1) << 31) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

pa_status release(const pa_cache_desc* desc, ReleaseParams& p, int32_t batch, int32_t* block_tables,
                  int32_t max_pages_per_seq, int32_t* ref_counts, int32_t* free_pages, const int64_t* pool_state,
                  int64_t* pool_state_out, pa_stream_t stream) {
  // entries are numbered in the counts' range below kReturned
  if (batch > kMaxReleaseRows || static_cast<int64_t>(batch) * max_pages_per_seq >= int64_t(1) << 30)
    return PA_ERR_UNSUPPORTED;
  if (!free_pages || !pool_state || !pool_state_out) return PA_ERR_NULL;
  if (batch > 0 && !block_tables) return PA_ERR_NULL;
  p.bt = block_tables;
  p.refs = ref_counts;
  p.ring = free_pages;
  p.pool = pool_state;
  p.pool_out = pool_state_out;
  p.num_pages = desc->num_pages;
  p.batch = batch;
  p.maxp = max_pages_per_seq;
  p.log2P = log2_of(desc->page_size);
  pa_status st = prepare(&p.err);
  if (st != PA_OK) return st;
  const size_t smem = (static_cast<size_t>(batch) + 1) * 4;
  cudaError_t e = cudaSuccess;
  if (smem > 40 * 1024)
    e = cudaFuncSetAttribute(release_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (kMaxReleaseRows + 1) * 4);
  if (e != cudaSuccess) return cuda_fail(e);
  // a CTA alone goes through some thousand entries as fast as a cluster starts
  const int ctas = static_cast<int64_t>(batch) * max_pages_per_seq > 4096 ? kTabCluster : 1;
  void* args[] = {&p};
  e = launch_cluster(reinterpret_cast<const void*>(release_pages_kernel), ctas, smem,
                     static_cast<cudaStream_t>(stream), args);
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

pa_status pa_extend_tables(const pa_cache_desc* desc, int32_t batch, const int32_t* new_tokens,
                           const int32_t* context_lens, int32_t* block_tables, int32_t max_pages_per_seq,
                           const int32_t* free_pages, const int64_t* pool_state, int64_t max_tokens,
                           int32_t* cu_seqlens_q, int32_t* context_lens_out, int32_t* positions,
                           int64_t* slot_mapping, int32_t* ref_counts, int64_t* pool_state_out, pa_stream_t stream) {
  pa_status st = check_tables(desc, batch, max_pages_per_seq);
  if (st != PA_OK) return st;
  if (max_tokens < 0 || max_tokens > 0x7fffffff) return PA_ERR_SHAPE;
  if (!free_pages || !pool_state || !pool_state_out || !cu_seqlens_q) return PA_ERR_NULL;
  if (batch > 0 && (!new_tokens || !context_lens || !context_lens_out || !block_tables)) return PA_ERR_NULL;
  if (max_tokens > 0 && (!positions || !slot_mapping)) return PA_ERR_NULL;
  ExtendParams p{};
  p.new_tokens = new_tokens;
  p.ctx = context_lens;
  p.bt = block_tables;
  p.ring = free_pages;
  p.pool = pool_state;
  p.cu = cu_seqlens_q;
  p.ctx_out = context_lens_out;
  p.positions = positions;
  p.slots = slot_mapping;
  p.refs = ref_counts;
  p.pool_out = pool_state_out;
  p.num_pages = desc->num_pages;
  p.max_tokens = max_tokens;
  p.batch = batch;
  p.maxp = max_pages_per_seq;
  p.log2P = log2_of(desc->page_size);
  if ((st = prepare(&p.err)) != PA_OK) return st;
  // a CTA alone writes some thousand slots as fast as a cluster starts
  const int ctas = max_tokens > 2048 ? kTabCluster : 1;
  void* args[] = {&p};
  cudaError_t e = launch_cluster(reinterpret_cast<const void*>(extend_tables_kernel), ctas, 0,
                                 static_cast<cudaStream_t>(stream), args);
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

pa_status pa_share_pages(const pa_cache_desc* desc, int32_t batch, const int32_t* parents,
                         const int32_t* num_shared_pages, int32_t* block_tables, int32_t max_pages_per_seq,
                         int32_t* ref_counts, pa_stream_t stream) {
  pa_status st = check_tables(desc, batch, max_pages_per_seq);
  if (st != PA_OK || batch == 0) return st;
  if (!parents || !num_shared_pages || !block_tables || !ref_counts) return PA_ERR_NULL;
  ShareParams p{};
  p.parents = parents;
  p.num_pages_shared = num_shared_pages;
  p.bt = block_tables;
  p.refs = ref_counts;
  p.num_pages = desc->num_pages;
  p.batch = batch;
  p.maxp = max_pages_per_seq;
  if ((st = prepare(&p.err)) != PA_OK) return st;
  share_pages_kernel<<<batch, 128, 0, static_cast<cudaStream_t>(stream)>>>(p);
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

pa_status pa_release_pages(const pa_cache_desc* desc, int32_t batch, const int32_t* first_pages,
                           const int32_t* end_pages, int32_t* block_tables, int32_t max_pages_per_seq,
                           int32_t* ref_counts, int32_t* free_pages, const int64_t* pool_state,
                           int64_t* pool_state_out, pa_stream_t stream) {
  pa_status st = check_tables(desc, batch, max_pages_per_seq);
  if (st != PA_OK) return st;
  if (batch > 0 && (!first_pages || !end_pages)) return PA_ERR_NULL;
  ReleaseParams p{};
  p.first = first_pages;
  p.end = end_pages;
  return release(desc, p, batch, block_tables, max_pages_per_seq, ref_counts, free_pages, pool_state, pool_state_out,
                 stream);
}

pa_status pa_release_window_pages(const pa_cache_desc* desc, int32_t window, int32_t num_sinks, int32_t batch,
                                  const int32_t* context_lens, int32_t* block_tables, int32_t max_pages_per_seq,
                                  int32_t* ref_counts, int32_t* free_pages, const int64_t* pool_state,
                                  int64_t* pool_state_out, pa_stream_t stream) {
  pa_status st = check_tables(desc, batch, max_pages_per_seq);
  if (st != PA_OK) return st;
  if (window < 1 || num_sinks < 0) return PA_ERR_SHAPE;
  if (batch > 0 && !context_lens) return PA_ERR_NULL;
  ReleaseParams p{};
  p.ctx = context_lens;
  p.window = window;
  p.sinks = num_sinks;
  return release(desc, p, batch, block_tables, max_pages_per_seq, ref_counts, free_pages, pool_state, pool_state_out,
                 stream);
}

}  // extern "C"
