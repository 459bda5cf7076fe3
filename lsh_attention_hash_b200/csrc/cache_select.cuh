// Choice of the pages a new token attends to, by the cheap score that the hash
// already gives: in how many (round, cached token) pairs of the page the query
// and the token share a bucket.
//
// score(page) = sum over the query heads of the cached head, over the rounds and
// over the page's admissible positions of [tag == bucket of the query].  Whole
// numbers, so the choice is the same however the sum is split.
//
// Scoring reads 2 bytes per token and round and is bound by that: one warp per
// (page, head), 16-byte loads, two tags per comparison.  The choice is one CTA per
// query row over its scores in shared memory: a binary search for the lowest score
// that gets in, then one pass that writes the chosen pages in ascending order, of
// equal scores those of the lowest pages.
#pragma once

#include "cache_common.cuh"

namespace lsh {
namespace cache {

constexpr int kScoreThreads = 256;
constexpr int kPickThreads = 512;
constexpr int kMaxPickPages = 49152;  // scores of one row in shared memory (192 KB)

struct SelectArgs {
  const uint16_t* tags;      // [n_pages, H, n_rounds, page]
  const int32_t* q_buckets;  // [B, H * G, n_rounds, T]
  int32_t* scores;           // [B, H, T, max_pages]
  int32_t* selected;         // [B, H, T, n_select]
  int B, G, n_rounds, n_select, n_local, causal;
  Pages pg;
};

// Positions [0, limit) are admissible to row t.
__device__ __forceinline__ int select_limit(const SelectArgs& a, int b, int t) {
  const int pos = row_pos(a.pg, b, t);
  if (pos < 0) return 0;
  return a.causal ? pos + 1 : ctx_of(a.pg, b);
}

__global__ void __launch_bounds__(kScoreThreads) cache_score_kernel(const SelectArgs a) {
  const long long w = (long long)blockIdx.x * (kScoreThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const Pages& pg = a.pg;
  const long long bh = w / pg.max_pages;
  if (bh >= (long long)a.B * pg.H) return;
  const int lp = (int)(w - bh * pg.max_pages);
  const int b = (int)(bh / pg.H), h = (int)(bh - (long long)b * pg.H);
  const int page = 1 << pg.page_log2, first = lp << pg.page_log2;
  const int chunks_log2 = pg.page_log2 - 3;  // 16-byte chunks of a round
  const int n_chunks = a.n_rounds << chunks_log2;
  int phys = -2;
  for (int t = 0; t < pg.T; ++t) {
    const int limit = select_limit(a, b, t);
    int score = -1;
    if (first < limit) {
      if (phys == -2) phys = page_of(pg, b, lp);
      uint32_t acc = 0;
      if (phys >= 0) {
        const uint4* src = reinterpret_cast<const uint4*>(
            a.tags + (((long long)phys * pg.H + h) * a.n_rounds) * page);
        for (int c = lane; c < n_chunks; c += 32) {
          const uint4 u = __ldg(src + c);
          const int n = c >> chunks_log2;
          const int ok = limit - first - ((c & ((1 << chunks_log2) - 1)) << 3);  // admissible tokens of the chunk
          const uint32_t m0 = ok >= 2 ? 0x10001u : (ok == 1 ? 1u : 0u);
          const uint32_t m1 = ok >= 4 ? 0x10001u : (ok == 3 ? 1u : 0u);
          const uint32_t m2 = ok >= 6 ? 0x10001u : (ok == 5 ? 1u : 0u);
          const uint32_t m3 = ok >= 8 ? 0x10001u : (ok == 7 ? 1u : 0u);
          const int32_t* qb = a.q_buckets + (((long long)b * pg.H + h) * a.G * a.n_rounds + n) * pg.T + t;
          for (int g = 0; g < a.G; ++g) {
            const uint32_t q = (uint32_t)__ldg(qb + (long long)g * a.n_rounds * pg.T);
            if (q > 65535u) continue;  // no tag holds it
            const uint32_t qq = q * 0x10001u;
            acc += (__vseteq2(u.x, qq) & m0) + (__vseteq2(u.y, qq) & m1) + (__vseteq2(u.z, qq) & m2) +
                   (__vseteq2(u.w, qq) & m3);
          }
        }
      }
      // halves hold at most 4 * G per chunk; the sum of a lane stays below 2^16 (checked on the host)
      score = (int)__reduce_add_sync(0xffffffffu, (acc & 0xffffu) + (acc >> 16));
    }
    if (lane == 0) a.scores[(bh * pg.T + t) * pg.max_pages + lp] = score;
  }
}

// Sum over the block; every thread gets it.
__device__ __forceinline__ int block_max(int v, int* red) {
  v = __reduce_max_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  int m = red[0];
  for (int i = 1; i < kPickThreads / 32; ++i) m = max(m, red[i]);
  __syncthreads();
  return m;
}

__device__ __forceinline__ int block_count(int v, int* red) {
  v = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  int m = 0;
  for (int i = 0; i < kPickThreads / 32; ++i) m += red[i];
  __syncthreads();
  return m;
}

__global__ void __launch_bounds__(kPickThreads) cache_pick_kernel(const SelectArgs a) {
  extern __shared__ int sc[];
  __shared__ int red[kPickThreads / 32];
  __shared__ int2 scan[kPickThreads / 32];
  const Pages& pg = a.pg;
  const long long row = blockIdx.x;
  const int t = (int)(row % pg.T);
  const int b = (int)(row / pg.T / pg.H);
  const int limit = select_limit(a, b, t);
  const int n = limit > 0 ? ((limit - 1) >> pg.page_log2) + 1 : 0;  // candidate pages
  int32_t* out = a.selected + row * a.n_select;
  if (n <= a.n_select) {
    for (int i = threadIdx.x; i < a.n_select; i += kPickThreads) out[i] = i < n ? i : -1;
    return;
  }
  const int n_free = n - a.n_local;          // pages that the score decides about
  const int want = a.n_select - a.n_local;   // of which so many get in (want < n_free)
  int best = 0;
  for (int i = threadIdx.x; i < n_free; i += kPickThreads) {
    const int s = a.scores[row * pg.max_pages + i];
    sc[i] = s;
    best = max(best, s);
  }
  for (int i = threadIdx.x; i < a.n_local; i += kPickThreads) out[want + i] = n_free + i;
  best = block_max(best, red);  // (its barriers also publish sc)
  // the largest v with at least `want` scores >= v
  int lo = 0, hi = best + 1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    int cnt = 0;
    for (int i = threadIdx.x; i < n_free; i += kPickThreads) cnt += sc[i] >= mid;
    if (block_count(cnt, red) >= want) lo = mid; else hi = mid;
  }
  // a thread's stretch of pages: how many score above lo, how many equal it
  const int per = (n_free + kPickThreads - 1) / kPickThreads;
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
  int total_above = 0, ba = pa - above, be = pe - equal;
  for (int i = 0; i < kPickThreads / 32; ++i) {
    if (i < warp) {
      ba += scan[i].x;
      be += scan[i].y;
    }
    total_above += scan[i].x;
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
