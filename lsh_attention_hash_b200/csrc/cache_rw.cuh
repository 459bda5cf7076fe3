// Writing rows into the 4-bit cache and reading them back.
//
// Quantiser, per row and group of GROUP dims with lo = min, hi = max:
//   z = the largest bf16 <= lo,  s = the nearest bf16 to (hi - z) / 15,
//   code = min(15, nearest integer to (x - z) / s, ties to even),  value = z + s code.
// s and z are kept in bf16: 4 bytes for a group instead of 8, and since the codes
// are taken against the rounded s and z, their rounding costs no more than a clip
// of the group's ends.  Both quotients are those of the real numbers: a float
// quotient that lies so near a border that its rounding could decide is settled by
// the exact remainder, so a code depends on nothing but its inputs.
//
// D/8 lanes own a row, 8 dims each (one 16-byte load in bf16); the codes change
// lanes by a byte transpose (K) and a nibble transpose (V) and leave as whole words.
#pragma once

#include "cache_common.cuh"

namespace lsh {
namespace cache {

constexpr int kRwThreads = 256;

// A group whose scale would be below this counts as constant (codes 0).
constexpr float kMinScale = 7.8886090522101181e-31f;  // 2^-100

struct GroupParams {
  float s, z;
  uint32_t word;
};

// The largest bf16 not above x.
__device__ __forceinline__ float floor_bf16(float x) {
  const uint32_t b = __float_as_uint(x);
  uint32_t t = b & 0xffff0000u;
  if ((b & 0xffffu) && (b >> 31)) t += 0x10000u;
  return __uint_as_float(t);
}

// Scale of a group from hi - z (see above); s = NaN when the group holds a non-finite value or its
// range overflows.  lo is -inf for a group with a NaN.
__device__ __forceinline__ GroupParams group_params(float lo, float hi) {
  GroupParams g;
  g.z = floor_bf16(lo);
  const float span = hi - g.z;
  const float q = span / 15.f;
  uint32_t b = __float_as_uint(q);
  const uint32_t low = b & 0xffffu;
  if (low - 0x7ffeu <= 4u) {  // within the float quotient's error of the middle of two bf16
    const double d = (double)hi - (double)g.z;
    const double mid = 15.0 * (double)__uint_as_float((b & 0xffff0000u) | 0x8000u);
    const bool up = d > mid || (d == mid && (b & 0x10000u));
    b = (b & 0xffff0000u) + (up ? 0x10000u : 0u);
  } else {
    b = (b + 0x7fffu + ((b >> 16) & 1u)) & 0xffff0000u;
  }
  g.s = __uint_as_float(b);
  if (g.s < kMinScale) g.s = 0.f;
  if (!(span < INFINITY)) g.s = __uint_as_float(0x7fc00000u);
  g.word = (__float_as_uint(g.s) >> 16) | (__float_as_uint(g.z) & 0xffff0000u);
  return g;
}

// Code of x; inv = 1 / s, or 0 for a constant or non-finite group.
__device__ __forceinline__ uint32_t code_of(float x, const GroupParams& g, float inv) {
  const float d = x - g.z;
  const float t = d * inv;  // error below 3e-6: 15 * 3 roundings
  float k = rintf(t);
  if (fabsf(t - k) > 0.49997f) {
    // near a border: the sign of x - z - (f + 1/2) s decides, with the rounding of x - z put back
    const float f = floorf(t);
    const float q = (f + 0.5f) * g.s;  // exact: 5 + 8 bits
    const float bp = d - x;
    const float e = (x - (d - bp)) + (-g.z - bp);
    const float r = (d - q) + e;
    const bool odd = (int)f & 1;
    k = (r > 0.f || (r == 0.f && odd)) ? f + 1.f : f;
  }
  return (uint32_t)(int)fminf(k, 15.f);  // NaN (a non-finite group) gives 15; masked by the caller
}

// Quantises the lane's 8 dims: params of its group and the 8 codes.
template <int GROUP>
__device__ __forceinline__ GroupParams quantise8(const float (&x)[8], uint32_t (&c)[8]) {
  float lo = x[0], hi = x[0], poison = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    poison = fmaf(x[i], 0.f, poison);  // NaN if any x is infinite or NaN
  }
  if (poison != 0.f) lo = -INFINITY;
#pragma unroll
  for (int o = 1; o < GROUP / 8; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const GroupParams g = group_params(lo, hi);
  const bool codes = g.s > 0.f;
  const float inv = codes ? 1.f / g.s : 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = codes ? code_of(x[i], g, inv) : 0u;
  return g;
}

struct WriteArgs {
  const void *k, *v;        // [B, H, T, D]
  const int32_t* buckets;   // [B, H, n_rounds, T] or null
  uint8_t* cache;           // [n_pages, H, block]
  uint16_t* tags;           // [n_pages, H, n_rounds, page] or null
  long long rows;           // B * H * T
  int n_rounds;
  Pages pg;
};

template <typename T, int D, int GROUP>
__global__ void __launch_bounds__(kRwThreads) cache_write_kernel(const WriteArgs a) {
  using F = Fmt<D, GROUP>;
  constexpr int kLanes = D / 8;  // lanes of a row
  const long long gt = (long long)blockIdx.x * kRwThreads + threadIdx.x;
  const long long row = gt / kLanes;
  const int j = (int)(gt % kLanes), lane = threadIdx.x & 31;
  const bool live = row < a.rows;
  float xk[8], xv[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) xk[i] = xv[i] = 0.f;
  int pos = -1, phys = -1, h = 0, b = 0, tok = 0;
  long long bh = 0;
  if (live) {
    load8(static_cast<const T*>(a.k) + row * D + j * 8, xk);
    load8(static_cast<const T*>(a.v) + row * D + j * 8, xv);
    bh = row / a.pg.T;
    tok = (int)(row - bh * a.pg.T);
    b = (int)(bh / a.pg.H);
    h = (int)(bh - (long long)b * a.pg.H);
    pos = row_pos(a.pg, b, tok);
    if (pos >= 0) phys = page_of(a.pg, b, pos >> a.pg.page_log2);
  }
  uint32_t ck[8], cv[8];
  const GroupParams gk = quantise8<GROUP>(xk, ck);
  const GroupParams gv = quantise8<GROUP>(xv, cv);
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) sq = fmaf(xk[i], xk[i], sq);
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
  uint32_t wk = 0, wv = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    wk |= ck[i] << (4 * i);
    wv |= cv[i] << (4 * i);
  }
  wk = transpose_bytes4(wk, lane);
  wv = transpose_nibbles8(wv, lane);
  if (phys < 0) return;
  const int r = pos & 15, pair = r >> 1, e = r & 1;
  uint8_t* tile = a.cache + tile_offset(a.pg, phys, h, pos, F::kTile);
  *reinterpret_cast<uint32_t*>(tile + r * (D / 2) + (j & 3) * (D / 8) + (j >> 2) * 4) = wk;
  *reinterpret_cast<uint32_t*>(tile + F::kOffV + pair * D + ((j & 7) ^ (2 * (pair & 3))) * (D / 8) + (j >> 3) * 8 +
                               e * 4) = wv;
  if (j % (GROUP / 8) == 0) {
    const int grp = j / (GROUP / 8);
    reinterpret_cast<uint32_t*>(tile + F::kOffKp)[grp * 16 + r] = gk.word;
    reinterpret_cast<uint32_t*>(tile + F::kOffVp)[grp * 16 + r] = gv.word;
  }
  if (j == 0) reinterpret_cast<float*>(tile + F::kOffInv)[r] = 1.f / fmaxf(sqrtf(sq), 1e-12f);
  if (a.tags) {
    const int page = 1 << a.pg.page_log2;
    for (int n = j; n < a.n_rounds; n += kLanes) {
      const int32_t bk = a.buckets[(bh * a.n_rounds + n) * a.pg.T + tok];
      if ((uint32_t)bk > 65535u) record_error(LSH_ERR_INVALID_ARG);
      a.tags[(((long long)phys * a.pg.H + h) * a.n_rounds + n) * page + (pos & (page - 1))] = (uint16_t)bk;
    }
  }
}

struct ReadArgs {
  const uint8_t* cache;
  void *k, *v;      // [B, H, T, D]
  float* inv;       // [B, H, T] or null
  long long rows;
  Pages pg;
};

template <typename T, int D, int GROUP>
__global__ void __launch_bounds__(kRwThreads) cache_read_kernel(const ReadArgs a) {
  using F = Fmt<D, GROUP>;
  constexpr int kLanes = D / 8;
  const long long gt = (long long)blockIdx.x * kRwThreads + threadIdx.x;
  const long long row = gt / kLanes;
  const int j = (int)(gt % kLanes), lane = threadIdx.x & 31;
  const bool live = row < a.rows;
  uint32_t wk = 0, wv = 0, pk = 0, pv = 0;
  float inv = 0.f;
  if (live) {
    const long long bh = row / a.pg.T;
    const int tok = (int)(row - bh * a.pg.T);
    const int b = (int)(bh / a.pg.H), h = (int)(bh - (long long)b * a.pg.H);
    const int pos = row_pos(a.pg, b, tok);
    const int phys = pos >= 0 ? page_of(a.pg, b, pos >> a.pg.page_log2) : -1;
    if (phys >= 0) {
      const int r = pos & 15, pair = r >> 1, e = r & 1, grp = j / (GROUP / 8);
      const uint8_t* tile = a.cache + tile_offset(a.pg, phys, h, pos, F::kTile);
      wk = *reinterpret_cast<const uint32_t*>(tile + r * (D / 2) + (j & 3) * (D / 8) + (j >> 2) * 4);
      wv = *reinterpret_cast<const uint32_t*>(tile + F::kOffV + pair * D + ((j & 7) ^ (2 * (pair & 3))) * (D / 8) +
                                              (j >> 3) * 8 + e * 4);
      pk = reinterpret_cast<const uint32_t*>(tile + F::kOffKp)[grp * 16 + r];
      pv = reinterpret_cast<const uint32_t*>(tile + F::kOffVp)[grp * 16 + r];
      inv = reinterpret_cast<const float*>(tile + F::kOffInv)[r];
    }
  }
  wk = transpose_bytes4(wk, lane);
  wv = transpose_nibbles8(wv, lane);
  if (!live) return;
  const float sk = bf16_bits(pk & 0xffffu), zk = __uint_as_float(pk & 0xffff0000u);
  const float sv = bf16_bits(pv & 0xffffu), zv = __uint_as_float(pv & 0xffff0000u);
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = fmaf(sk, (float)((wk >> (4 * i)) & 15u), zk);
  store8(static_cast<T*>(a.k) + row * D + j * 8, x);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = fmaf(sv, (float)((wv >> (4 * i)) & 15u), zv);
  store8(static_cast<T*>(a.v) + row * D + j * 8, x);
  if (a.inv && j == 0) a.inv[row] = inv;
}

}  // namespace cache
}  // namespace lsh
