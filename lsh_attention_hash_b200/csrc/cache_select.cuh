// Choice of the pages a new token attends to, by the cheap score that the hash
// already gives: in how many (round, cached token) pairs of the page the query
// and the token share a bucket.
//
// score(page) = sum over the query heads of the cached head, over the rounds and
// over the page's admissible positions of [tag == bucket of the query].  Whole
// numbers, so the choice is the same however the sum is split.
//
// Scoring reads 2 bytes per token and round and is bound by that: a warp takes up to 16
// pages of a head, all 16-byte loads of a page (and of the next ones) in flight, and compares two
// tags an instruction: min(tag ^ bucket, 1) counts those that differ.  The choice is one CTA per
// query row over its scores in shared memory: a binary search for the lowest score that gets
// in, then one pass that writes the chosen pages in ascending order, of equal scores those of the
// lowest pages.
//
// Measured on the device, inputs not in L2: 64 heads x 65536 tokens, 8 rounds (67 MB of tags, floor 10 us) 20 us for
// both kernels; 8 heads x 1 M tokens, 4 rounds (67 MB) 26 us.  What does not fit the batches of pages (several query
// heads, other numbers of tags) takes the general loop, a page at a time: 64 heads x 65536 tokens, 6 rounds 30 us
// (50 MB), 2 rounds 18 us (17 MB), 8 rounds with 4 query heads a head 49 us; 5 rows in the batches, which read the tags
// for each, 53 us.
#pragma once

#include "cache_common.cuh"

namespace lsh {
namespace cache {

constexpr int kScoreThreads = 256;
constexpr int kWarpPages = 16;  // most pages of a warp (at most 32: a lane each)
constexpr int kPickThreads = 1024;
constexpr int kMaxPickPages = 49152;  // scores of one row in shared memory (192 KB)

struct SelectArgs {
  const uint16_t* tags;      // [n_pages, H, n_rounds, page]
  const int32_t* q_buckets;  // [B, H * G, n_rounds, T]
  int32_t* scores;           // [B, H, T, max_pages]
  int32_t* selected;         // [B, H, T, n_select]
  int B, G, n_rounds, n_select, n_local, causal;
  int warp_pages, fused;     // pages of a scoring warp; the picking CTA scores its row itself
  Pages pg;
};

// Positions [0, limit) are admissible to row t.
__device__ __forceinline__ int select_limit(const SelectArgs& a, int b, int t) {
  const int pos = row_pos(a.pg, b, t);
  if (pos < 0) return 0;
  return a.causal ? pos + 1 : ctx_of(a.pg, b);
}

// How many of the tags in a word's two halves differ from q's (a count in each half).
__device__ __forceinline__ uint32_t differ2(uint32_t tags, uint32_t q2) {
  return __vminu2(tags ^ q2, 0x00010001u);
}

// Score of one page (whole warp): any sizes, query heads, and a limit inside the page.  ph < 0: missing.
__device__ __forceinline__ int page_score(const SelectArgs& a, const int32_t* qb, int ph, int h, int first, int limit,
                                          int lane) {
  const int cl = a.pg.page_log2 - 3;  // log2 of the 16-byte chunks of a round
  const int n_chunks = ph >= 0 ? a.n_rounds << cl : 0;
  const uint4* src = reinterpret_cast<const uint4*>(
      a.tags + ((((long long)max(ph, 0) * a.pg.H + h) * a.n_rounds) << a.pg.page_log2));
  uint32_t acc = 0;
  for (int c = lane; c < n_chunks; c += 32) {
    const uint4 u = __ldg(src + c);
    const int n = c >> cl;
    const int ok = limit - first - ((c & ((1 << cl) - 1)) << 3);  // admissible tokens of the chunk
    const uint32_t m0 = ok >= 2 ? 0x10001u : (ok == 1 ? 1u : 0u);
    const uint32_t m1 = ok >= 4 ? 0x10001u : (ok == 3 ? 1u : 0u);
    const uint32_t m2 = ok >= 6 ? 0x10001u : (ok == 5 ? 1u : 0u);
    const uint32_t m3 = ok >= 8 ? 0x10001u : (ok == 7 ? 1u : 0u);
    for (int g = 0; g < a.G; ++g) {
      const uint32_t q = (uint32_t)__ldg(qb + ((long long)g * a.n_rounds + n) * a.pg.T);
      if (q > 65535u) continue;  // no tag holds it
      const uint32_t qq = q * 0x10001u;
      acc += (~differ2(u.x, qq) & m0) + (~differ2(u.y, qq) & m1) + (~differ2(u.z, qq) & m2) +
             (~differ2(u.w, qq) & m3);
    }
  }
  // a lane's halves stay below 2^16 (checked on the host)
  return (int)__reduce_add_sync(0xffffffffu, (acc & 0xffffu) + (acc >> 16));
}

// NC: 16-byte chunks of a page per lane (n_rounds * page / 256) when the page is whole and there is one
// query head, so that the lane's buckets stay in registers; 0: any number.
template <int NC>
__global__ void __launch_bounds__(kScoreThreads) cache_score_kernel(const SelectArgs a, int groups) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the choice may be set up; it waits below
  const int lane = threadIdx.x & 31;
  const Pages& pg = a.pg;
  const unsigned w = blockIdx.x * (kScoreThreads / 32) + (threadIdx.x >> 5);  // (head, its pages)
  const unsigned bh = w / groups;
  if (bh >= (unsigned)(a.B * pg.H)) return;
  const int lp0 = (int)(w - bh * groups) * a.warp_pages;
  const int b = bh / pg.H, h = bh - b * pg.H;
  const int page = 1 << pg.page_log2;
  const int cl = pg.page_log2 - 3;  // log2 of the 16-byte chunks of a round
  const int mine = lp0 + lane;      // the first lanes have a page each
  const bool has = lane < a.warp_pages && mine < pg.max_pages;
  int phys = -2;                    // of the lane's page, once it is wanted
  const long long row_bytes = (long long)a.n_rounds * page * 2;
  for (int t = 0; t < pg.T; ++t) {
    const int limit = select_limit(a, b, t);
    if (has && phys == -2 && (mine << pg.page_log2) < limit) phys = page_of(pg, b, mine);
    const int32_t* qb = a.q_buckets + ((long long)bh * a.G * a.n_rounds) * pg.T + t;
    int score = has && (mine << pg.page_log2) < limit ? 0 : -1;
    const int whole = min(a.warp_pages, max(0, (limit >> pg.page_log2) - lp0));  // pages below the limit
    int i = 0;
    if (NC > 0) {
      uint32_t q2[NC > 0 ? NC : 1];
      bool bad = false;  // a bucket that no tag holds: then the general loop
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        const uint32_t q = (uint32_t)qb[(long long)((lane + 32 * k) >> cl) * pg.T];
        bad |= q > 65535u;
        q2[k] = q * 0x10001u;
      }
      if (pg.n_pages > 0 && !__any_sync(0xffffffffu, bad)) {
        constexpr int kBatch = NC == 1 ? 8 : NC == 2 ? 4 : 2;  // pages whose loads are in flight together
        for (; i < whole; i += kBatch) {
          uint4 u[kBatch][NC > 0 ? NC : 1];
#pragma unroll
          for (int p = 0; p < kBatch; ++p) {
            // (a page that is missing, or behind the last whole one, reads page 0 for nothing)
            const int ph = max(__shfl_sync(0xffffffffu, phys, min(i + p, 31)), 0);
            const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(a.tags) +
                                                              ((long long)ph * pg.H + h) * row_bytes) + lane;
#pragma unroll
            for (int k = 0; k < NC; ++k) u[p][k] = __ldg(src + 32 * k);
          }
#pragma unroll
          for (int p = 0; p < kBatch; ++p) {
            uint32_t acc = NC * 0x00040004u;
#pragma unroll
            for (int k = 0; k < NC; ++k)
              acc -= differ2(u[p][k].x, q2[k]) + differ2(u[p][k].y, q2[k]) + differ2(u[p][k].z, q2[k]) +
                     differ2(u[p][k].w, q2[k]);
            const int sum = __reduce_add_sync(0xffffffffu, (acc & 0xffffu) + (acc >> 16));
            if (lane == i + p && i + p < whole) score = phys >= 0 ? sum : 0;
          }
        }
        i = whole;
      }
    }
    // the page that the limit cuts, other sizes, several query heads
    for (; i < a.warp_pages && ((lp0 + i) << pg.page_log2) < limit; ++i) {
      const int ph = __shfl_sync(0xffffffffu, phys, i);
      const int sum = page_score(a, qb, ph, h, (lp0 + i) << pg.page_log2, limit, lane);
      if (lane == i) score = sum;
    }
    if (has) a.scores[((long long)bh * pg.T + t) * pg.max_pages + mine] = score;
  }
}

__global__ void __launch_bounds__(kPickThreads) cache_pick_kernel(const SelectArgs a) {
  extern __shared__ __align__(16) int sc[];
  __shared__ int cell[4];  // the largest score; counts of three steps in turn
  static_assert(kPickThreads == 1024, "a lane for every warp in the second scan");
  __shared__ int2 scan[kPickThreads / 32];
  const Pages& pg = a.pg;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // what follows waits for this kernel's end
  asm volatile("griddepcontrol.wait;" ::: "memory");               // the scores are there
  if (threadIdx.x < 4) cell[threadIdx.x] = 0;
  const long long row = blockIdx.x;
  const int t = (int)(row % pg.T);
  const int b = (int)(row / pg.T / pg.H);
  const int limit = select_limit(a, b, t);
  const int n = limit > 0 ? ((limit - 1) >> pg.page_log2) + 1 : 0;  // candidate pages
  int32_t* out = a.selected + row * a.n_select;
  if (a.fused) {  // the row's scores: every warp a page at a time
    const long long bh = row / pg.T;
    const int h = (int)(bh % pg.H), lane = threadIdx.x & 31;
    const int32_t* qb = a.q_buckets + bh * a.G * a.n_rounds * pg.T + t;
    for (int i = threadIdx.x >> 5; i < pg.max_pages; i += kPickThreads / 32) {
      int score = -1;
      if (i < n) score = page_score(a, qb, page_of(pg, b, i), h, i << pg.page_log2, limit, lane);
      if (lane == 0) {
        a.scores[row * pg.max_pages + i] = score;
        sc[i] = score;
      }
    }
  }
  if (n <= a.n_select) {
    for (int i = threadIdx.x; i < a.n_select; i += kPickThreads) out[i] = i < n ? i : -1;
    return;
  }
  const int n_free = n - a.n_local;          // pages that the score decides about
  const int want = a.n_select - a.n_local;   // of which so many get in (want < n_free)
  // scores to shared memory, four at a time, with -1 behind the last (max_pages is padded there)
  int best = 0;
  const int n4 = (n_free + 3) / 4;
  if (a.fused) {
    __syncthreads();
    for (int i = threadIdx.x; i < n_free; i += kPickThreads) best = max(best, sc[i]);
    __syncthreads();
    for (int i = n_free + threadIdx.x; i < 4 * n4; i += kPickThreads) sc[i] = -1;
  } else {
    const int* from = a.scores + row * pg.max_pages;
    if ((pg.max_pages & 3) == 0) {
#pragma unroll 4
      for (int i = threadIdx.x; i < n4; i += kPickThreads) {
        int4 u = *reinterpret_cast<const int4*>(from + 4 * i);
        if (4 * i + 1 >= n_free) u.y = -1;
        if (4 * i + 2 >= n_free) u.z = -1;
        if (4 * i + 3 >= n_free) u.w = -1;
        reinterpret_cast<int4*>(sc)[i] = u;
        best = max(best, max(max(u.x, u.y), max(u.z, u.w)));
      }
    } else {
#pragma unroll 4
      for (int i = threadIdx.x; i < 4 * n4; i += kPickThreads) {
        const int v = i < n_free ? from[i] : -1;
        sc[i] = v;
        best = max(best, v);
      }
    }
  }
  for (int i = threadIdx.x; i < a.n_local; i += kPickThreads) out[want + i] = n_free + i;
  if (!a.fused) __syncthreads();  // cell is cleared
  best = __reduce_max_sync(0xffffffffu, best);
  if ((threadIdx.x & 31) == 0) atomicMax(cell, best);
  __syncthreads();  // (and sc is there)
  best = cell[0];
  // the largest v with at least `want` scores >= v
  int lo = 0, hi = best + 1, step = 0;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    int cnt = 0;
    for (int i = threadIdx.x; i < n4; i += kPickThreads) {
      const int4 u = reinterpret_cast<const int4*>(sc)[i];
      cnt += (u.x >= mid) + (u.y >= mid) + (u.z >= mid) + (u.w >= mid);
    }
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    if ((threadIdx.x & 31) == 0) atomicAdd(cell + 1 + step, cnt);
    const int next = step == 2 ? 0 : step + 1;
    if (threadIdx.x == 0) cell[1 + next] = 0;  // (last read two barriers ago)
    __syncthreads();
    if (cell[1 + step] >= want) lo = mid; else hi = mid;
    step = next;
  }
  // a thread's stretch of pages: how many score above lo, how many equal it
  const int per = ((n_free + kPickThreads - 1) / kPickThreads) | 1;  // odd: no shared-memory bank conflicts
  const int i0 = min((int)threadIdx.x * per, n_free), i1 = min(i0 + per, n_free);
  int above = 0, equal = 0;
  for (int i = i0; i < i1; ++i) {
    above += sc[i] > lo;
    equal += sc[i] == lo;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int pa = above, pe = equal;  // inclusive sums over the warp
  for (int o = 1; o < 32; o <<= 1) {
    const int xa = __shfl_up_sync(0xffffffffu, pa, o), xe = __shfl_up_sync(0xffffffffu, pe, o);
    if (lane >= o) {
      pa += xa;
      pe += xe;
    }
  }
  if (lane == 31) scan[warp] = make_int2(pa, pe);
  __syncthreads();
  int2 w = scan[lane];  // (kPickThreads / 32 warps: a lane each)
  for (int o = 1; o < 32; o <<= 1) {
    const int xa = __shfl_up_sync(0xffffffffu, w.x, o), xe = __shfl_up_sync(0xffffffffu, w.y, o);
    if (lane >= o) {
      w.x += xa;
      w.y += xe;
    }
  }
  const int total_above = __shfl_sync(0xffffffffu, w.x, 31);
  int ba = pa - above, be = pe - equal;
  if (warp > 0) {
    ba += __shfl_sync(0xffffffffu, w.x, warp - 1);
    be += __shfl_sync(0xffffffffu, w.y, warp - 1);
  }
  const int need = want - total_above;  // of the equal ones, the first so many
  for (int i = i0; i < i1; ++i) {
    const bool gt = sc[i] > lo, eq = sc[i] == lo;
    if (gt || (eq && be < need)) out[ba + min(be, need)] = i;
    ba += gt;
    be += eq;
  }
}

}  // namespace cache
}  // namespace lsh
