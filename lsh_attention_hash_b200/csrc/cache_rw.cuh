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
// No clamp to 15 is needed: s is off by 2^-9 of itself at most, so (hi - z) / s <= 15.03.
//
// D/16 lanes own a row, 16 dims each of K and of V; the codes change lanes by one (K) and four
// (V) shuffles and leave as whole words.  Both kernels are streams bound by instruction issue
// before they are bound by memory, so a code costs few: the three-input minimum and maximum of
// sm_100, the integer taken from a float's mantissa, packing by multiply-add.
//
// Measured, 8 x 8 heads x 16384 rows: D 128 bf16 writing 198 us (3.5 TB/s: 630 instructions a warp for its
// 1024 values bind it, three quarters of the issue slots), reading 111 us (6.25 TB/s, 95 % of the measured copy
// rate); 8 heads x 262144 rows of 64 in fp32: writing 226 us (5.5 TB/s), reading 191 us (6.5 TB/s).
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

// The largest bf16 not above x (bf16 rows: x itself).
__device__ __forceinline__ float floor_bf16(float x, const float*) {
  const uint32_t b = __float_as_uint(x);
  uint32_t t = b & 0xffff0000u;
  if ((b & 0xffffu) && (b >> 31)) t += 0x10000u;
  return __uint_as_float(t);
}
__device__ __forceinline__ float floor_bf16(float x, const __nv_bfloat16*) { return x; }

// Minimum and maximum of three; a NaN stays.
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Scale of a group from hi - z (see above); s = NaN when the group holds a non-finite value or its
// range overflows (lo and hi are NaN for a group with a NaN).
template <typename T>
__device__ __forceinline__ GroupParams group_params(float lo, float hi) {
  GroupParams g;
  g.z = floor_bf16(lo, static_cast<const T*>(nullptr));
  const float span = hi - g.z;
  const float q = span * (1.f / 15.f);  // off by 3 units of its last place at most
  uint32_t b = __float_as_uint(q);
  if ((b & 0xffffu) - 0x7ffcu <= 8u) {  // the middle of two bf16 is that near: the exact quotient decides
    const double h = (double)hi, z = (double)g.z, d = h - z;
    // what d leaves out of hi - z (bf16: where it leaves something out, d is next to a number of 8 bits, and the
    // middle, 15 times an odd one of 9 bits, is not)
    double lost = 0.0;
    if (sizeof(T) == 4) {
      const double back = d - h;
      lost = (h - (d - back)) + (-z - back);
    }
    const double mid = 15.0 * (double)__uint_as_float((b & 0xffff0000u) | 0x8000u);
    const bool up = d > mid || (d == mid && (lost > 0.0 || (lost == 0.0 && (b & 0x10000u))));
    b = (b & 0xffff0000u) + (up ? 0x10000u : 0u);
  } else {
    b = (b + 0x8000u) & 0xffff0000u;
  }
  g.s = __uint_as_float(b);
  if (g.s < kMinScale) g.s = 0.f;
  if (!(span < INFINITY)) g.s = __uint_as_float(0x7fc00000u);
  g.word = (__float_as_uint(g.s) >> 16) | (__float_as_uint(g.z) & 0xffff0000u);
  return g;
}

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: the low mantissa bits of kMagic + k are k

// kMagic plus the code of x, from the exact remainder at the border next to t = (x - z) / s.
__device__ __forceinline__ float code_exact(float x, float z, float s, float t) {
  const float f = floorf(t);
  if (fabsf(t - f - 0.5f) < 1e-4f) {
    // the sign of x - z - (f + 1/2) s decides, with the rounding of x - z put back
    const float d = x - z;
    const float q = (f + 0.5f) * s;  // exact: 5 + 8 bits
    const float bp = d - x;
    const float e = (x - (d - bp)) + (-z - bp);
    const float r = (d - q) + e;
    const bool odd = (int)f & 1;
    return ((r > 0.f || (r == 0.f && odd)) ? f + 1.f : f) + kMagic;
  }
  return t + kMagic;
}

// The 16 codes of a lane as kMagic + code, over x.  s > 0, inv = 1 / s to 2^-22; `rows` is where x came from.
//
// t = (x - z) inv is off by 1e-5 at most, so only quotients that near a border are in doubt.
// fp32: those are rare, found by one comparison for the 16, and settled exactly.  bf16: many values lie
// exactly on a border.  There one Newton step makes t the nearest float to the quotient, which is
// k + 1/2 for a true tie and, if x - z is a short number, for nothing else: x, z and s have 8 bits, so
// only an x or z below 2^-11 s can put the quotient within 2^-20 of a border without being on it (or
// make x - z inexact).  Such an x lies within 2^-11 of -z / s in codes, so groups where that is
// near a border, and those with such a z, settle their codes exactly.
__device__ __forceinline__ void codes16(float (&x)[16], const GroupParams& g, float inv, const float* rows) {
  float worst = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float t = (x[i] - g.z) * inv;
    x[i] = t + kMagic;  // ties to even
    worst = fmaxf(worst, fabsf(t - (x[i] - kMagic)));
  }
  if (worst > 0.4999f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float y = rows[i];
      x[i] = code_exact(y, g.z, g.s, (y - g.z) * inv);
    }
  }
}

__device__ __forceinline__ void codes16(float (&x)[16], const GroupParams& g, float inv, const __nv_bfloat16*) {
  const float t0 = -g.z * inv;
  if (fabsf(t0 - ((t0 + kMagic) - kMagic)) > 0.499f || (g.z != 0.f && fabsf(g.z) < g.s * 4.8828125e-4f)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = code_exact(x[i], g.z, g.s, (x[i] - g.z) * inv);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float d = x[i] - g.z;
      const float t = d * inv;
      x[i] = fmaf(fmaf(-t, g.s, d), inv, t) + kMagic;
    }
  }
}

// 32 bytes (one sector) at a time where the buffers allow it, else 2 x 16: a lane's 16-byte halves of a
// sector are two requests.
__device__ __forceinline__ void ld32(uint4 (&u)[2], const void* p, bool wide) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(u[0].x), "=r"(u[0].y), "=r"(u[0].z), "=r"(u[0].w), "=r"(u[1].x), "=r"(u[1].y), "=r"(u[1].z),
                   "=r"(u[1].w)
                 : "l"(p));
  } else {
    u[0] = ld16(p);
    u[1] = ld16(reinterpret_cast<const uint4*>(p) + 1);
  }
}
__device__ __forceinline__ void st32(void* p, const uint4& a, const uint4& b, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    st16(p, a);
    st16(reinterpret_cast<uint4*>(p) + 1, b);
  }
}

// A lane's 16 dims as they lie in memory.
template <typename T>
struct Raw {
  uint4 u[sizeof(T)];
  __device__ __forceinline__ Raw(const T* p, bool live, bool wide) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) u[i] = make_uint4(0u, 0u, 0u, 0u);
    if (live)
#pragma unroll
      for (int i = 0; i < (int)sizeof(T); i += 2)
        ld32(*reinterpret_cast<uint4(*)[2]>(u + i), reinterpret_cast<const uint4*>(p) + i, wide);
  }
};

// The lane's 16 dims, quantised: params of its group and the codes, nibble i of w[0] dim i, of w[1] dim 8 + i.
// SQUARES: adds up the squares.
template <typename T, int GROUP, bool SQUARES>
__device__ __forceinline__ GroupParams quantise16(const Raw<T>& raw, const T* rows, uint32_t sixteen, uint32_t (&w)[2],
                                                  float& squares) {
  float x[16];
  load8(reinterpret_cast<const T*>(raw.u), *reinterpret_cast<float(*)[8]>(x));
  load8(reinterpret_cast<const T*>(raw.u) + 8, *reinterpret_cast<float(*)[8]>(x + 8));
  float lo = min3(x[0], x[1], x[2]), hi = max3(x[0], x[1], x[2]);
#pragma unroll
  for (int i = 3; i < 15; i += 2) {
    lo = min3(lo, x[i], x[i + 1]);
    hi = max3(hi, x[i], x[i + 1]);
  }
  lo = min3(lo, x[15], x[15]);
  hi = max3(hi, x[15], x[15]);
  if (SQUARES) {
    squares = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) squares = fmaf(x[i], x[i], squares);
  }
#pragma unroll
  for (int o = 1; o < GROUP / 16; o <<= 1) {
    const float l2 = __shfl_xor_sync(0xffffffffu, lo, o), h2 = __shfl_xor_sync(0xffffffffu, hi, o);
    lo = min3(lo, l2, l2);
    hi = max3(hi, h2, h2);
  }
  const GroupParams g = group_params<T>(lo, hi);
  w[0] = w[1] = 0u;
  if (g.s > 0.f) {
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(g.s));  // s is 2^-100 .. 2^125
    codes16(x, g, inv, rows);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      // sum of (0x4B400000 + code) 16^i; what the floats' upper bits add up to is taken off again.  (16 comes in
      // as a value: as a literal it would be a shift and add at half the rate of multiply-add)
      uint32_t sum = __float_as_uint(x[8 * j + 7]);
#pragma unroll
      for (int i = 6; i >= 0; --i) sum = sum * sixteen + __float_as_uint(x[8 * j + i]);
      w[j] = sum - 0x4B400000u * 0x11111111u;
    }
  }
  return g;
}

// The codes of 32 (K) or 64 (V) dims between "16 dims of a lane" and "words of the tile" (the same
// exchange leads back).  K: two lanes; of words t = 0..3 lane `half` has 2 half and 2 half + 1.
__device__ __forceinline__ void k_to_words(uint32_t (&w)[2], int half) {
  const uint32_t a = __byte_perm(w[0], w[1], 0x5410), b = __byte_perm(w[0], w[1], 0x7632);
  const uint32_t r = __shfl_xor_sync(0xffffffffu, half ? a : b, 1);
  const uint32_t lo = half ? r : a, hi = half ? b : r;
  w[0] = __byte_perm(lo, hi, 0x6420);
  w[1] = __byte_perm(lo, hi, 0x7531);
}
__device__ __forceinline__ void words_to_k(uint32_t (&w)[2], int half) {
  const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[0], w[1], 0x7362);
  const uint32_t r = __shfl_xor_sync(0xffffffffu, half ? a : b, 1);
  const uint32_t lo = half ? r : a, hi = half ? b : r;
  w[0] = __byte_perm(lo, hi, 0x5410);
  w[1] = __byte_perm(lo, hi, 0x7632);
}
// V: four lanes; lane u has the words of chunks 2 u and 2 u + 1.
__device__ __forceinline__ void v_to_words(uint32_t (&w)[2], int lane) {
  const uint32_t even = (w[0] & 0x0f0f0f0fu) | ((w[1] & 0x0f0f0f0fu) << 4);
  const uint32_t odd = ((w[0] >> 4) & 0x0f0f0f0fu) | (w[1] & 0xf0f0f0f0u);
  w[0] = transpose_bytes4(even, lane);
  w[1] = transpose_bytes4(odd, lane);
}
__device__ __forceinline__ void words_to_v(uint32_t (&w)[2], int lane) {
  const uint32_t even = transpose_bytes4(w[0], lane), odd = transpose_bytes4(w[1], lane);
  w[0] = (even & 0x0f0f0f0fu) | ((odd & 0x0f0f0f0fu) << 4);
  w[1] = ((even >> 4) & 0x0f0f0f0fu) | (odd & 0xf0f0f0f0u);
}

// Offsets in a tile of a lane's two words of K and of V, for token r and dims 16 j .. 16 j + 15.
template <int D>
struct LaneWords {
  int k0, v0, v1;
  __device__ __forceinline__ LaneWords(int r, int j) {
    k0 = r * (D / 2) + (j & 1) * 2 * (D / 8) + (j >> 1) * 4;  // the second word D/8 further
    const int pair = r >> 1, x = 2 * (pair & 3), c = 2 * (j & 3);
    const int base = 8 * D + pair * D + (j >> 2) * 8 + (r & 1) * 4;
    v0 = base + (c ^ x) * (D / 8);
    v1 = base + ((c + 1) ^ x) * (D / 8);
  }
};

// A row of the call and its place: (b, h, t) of row = (b H + h) T + t, its position and physical page
// (-1: padding, or a page that is missing).
struct Row {
  int b, h, t, pos, phys;
  unsigned bh;
};

__device__ __forceinline__ Row row_of(const Pages& p, unsigned row) {
  Row r;
  r.bh = p.div_t.of(row);
  r.t = (int)(row - r.bh * p.T);
  r.b = (int)p.div_h.of(r.bh);
  r.h = (int)(r.bh - (unsigned)r.b * p.H);
  r.pos = row_pos(p, r.b, r.t);
  r.phys = -1;
  return r;
}

// Looks the row's page up (apart from row_of so that a row's own loads need not wait for it).
__device__ __forceinline__ void look_up_page(const Pages& p, Row& r) {
  if (r.pos >= 0) r.phys = page_of(p, r.b, r.pos >> p.page_log2);
}

struct WriteArgs {
  const void *k, *v;        // [B, H, T, D]
  const int32_t* buckets;   // [B, H, n_rounds, T] or null
  uint8_t* cache;           // [n_pages, H, block]
  uint16_t* tags;           // [n_pages, H, n_rounds, page] or null
  unsigned rows;            // B * H * T
  int n_rounds;
  bool wide;                // k and v on 32-byte boundaries
  uint32_t sixteen;         // 16
  Pages pg;
};

// 1 / length of a row whose squares overflow a float (it is longer than 1.8e19), from the row scaled by 2^-96; 0 for a
// row with an infinity, NaN for one with a NaN.  One lane reads the row again: the common case pays a comparison (bf16
// nothing that shows, fp32 217 -> 226 us for 8 heads x 262144 rows of 64, as its registers are full; the whole warp by
// a vote 222, but bf16 5 % more).
template <typename T, int D>
__device__ __noinline__ float long_row_inv(const T* row) {
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int d = 0; d < D; d += 8) {
    float x[8];
    load8(row + d, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = fmaf(x[i] * 0x1p-96f, x[i] * 0x1p-96f, s[i]);
  }
  return 1.f / sqrtf(((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]))) * 0x1p-96f;
}

template <typename T, int D, int GROUP>
__global__ void __launch_bounds__(kRwThreads, 4) cache_write_kernel(const WriteArgs a) {
  using F = Fmt<D, GROUP>;
  constexpr int kLanes = D / 16;  // lanes of a row
  const unsigned row = blockIdx.x * (kRwThreads / kLanes) + threadIdx.x / kLanes;
  const int j = threadIdx.x % kLanes, lane = threadIdx.x & 31;
  Row r;
  r.pos = r.phys = -1;
  if (row < a.rows) r = row_of(a.pg, row);
  uint32_t wk[2], wv[2];
  const long long from = (long long)row * D + j * 16;
  float sq, none;
  const T *k = static_cast<const T*>(a.k) + from, *v = static_cast<const T*>(a.v) + from;
  const Raw<T> raw_k(k, r.pos >= 0, a.wide), raw_v(v, r.pos >= 0, a.wide);  // of padding nothing is read
  look_up_page(a.pg, r);
  const GroupParams gk = quantise16<T, GROUP, true>(raw_k, k, a.sixteen, wk, sq);
  const GroupParams gv = quantise16<T, GROUP, false>(raw_v, v, a.sixteen, wv, none);
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
  k_to_words(wk, j & 1);
  v_to_words(wv, lane);
  if (r.phys < 0) return;
  const int t = r.pos & 15;
  uint8_t* tile = a.cache + tile_offset(a.pg, r.phys, r.h, r.pos, F::kTile);
  const LaneWords<D> at(t, j);
  *reinterpret_cast<uint32_t*>(tile + at.k0) = wk[0];
  *reinterpret_cast<uint32_t*>(tile + at.k0 + D / 8) = wk[1];
  *reinterpret_cast<uint32_t*>(tile + at.v0) = wv[0];
  *reinterpret_cast<uint32_t*>(tile + at.v1) = wv[1];
  if (j % (GROUP / 16) == 0) {
    const int grp = j / (GROUP / 16);
    reinterpret_cast<uint32_t*>(tile + F::kOffKp)[grp * 16 + t] = gk.word;
    reinterpret_cast<uint32_t*>(tile + F::kOffVp)[grp * 16 + t] = gv.word;
  }
  if (j == 0) {
    float inv = 1.f / fmaxf(sqrtf(sq), 1e-12f);
    if (!(sq < INFINITY)) inv = long_row_inv<T, D>(static_cast<const T*>(a.k) + (long long)row * D);
    reinterpret_cast<float*>(tile + F::kOffInv)[t] = inv;
  }
  if (a.tags) {
    const int page = 1 << a.pg.page_log2;
    for (int n = j; n < a.n_rounds; n += kLanes) {
      const int32_t bk = a.buckets[((long long)r.bh * a.n_rounds + n) * a.pg.T + r.t];
      if ((uint32_t)bk > 65535u) record_error(LSH_ERR_INVALID_ARG);
      a.tags[(((long long)r.phys * a.pg.H + r.h) * a.n_rounds + n) * page + (r.pos & (page - 1))] = (uint16_t)bk;
    }
  }
}

struct ReadArgs {
  const uint8_t* cache;
  void *k, *v;      // [B, H, T, D]
  float* inv;       // [B, H, T] or null
  unsigned rows;
  bool wide;        // k and v on 32-byte boundaries
  Pages pg;
};

// z + s code of the 16 codes, rounded once, to 16 consecutive elements.
__device__ __forceinline__ void store16(float* p, const uint32_t (&w)[2], uint32_t params, bool wide) {
  const float s = bf16_bits(params & 0xffffu), z = __uint_as_float(params & 0xffff0000u);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    alignas(16) float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = fmaf(s, __uint_as_float(((w[j] >> (4 * i)) & 15u) | 0x4B000000u) - 8388608.f, z);
    const float4* y = reinterpret_cast<const float4*>(x);
    st32(p + 8 * j, *reinterpret_cast<const uint4*>(y), *reinterpret_cast<const uint4*>(y + 1), wide);
  }
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const uint32_t (&w)[2], uint32_t params, bool wide) {
  const uint32_t s2 = __byte_perm(params, 0, 0x1010), z2 = __byte_perm(params, 0, 0x3232);
  const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162*>(&s2), z = *reinterpret_cast<const __nv_bfloat162*>(&z2);
  const uint32_t c128 = 0x43004300u;  // 0x4300 | code is 128 + code in bf16
  uint4 u[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t y[4];  // dims i and i + 4
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t c = ((w[j] >> (4 * i)) & 0x000f000fu) | c128;
      const __nv_bfloat162 v = __hfma2(s, __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&c),
                                                  *reinterpret_cast<const __nv_bfloat162*>(&c128)), z);
      y[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    u[j].x = __byte_perm(y[0], y[1], 0x5410);
    u[j].y = __byte_perm(y[2], y[3], 0x5410);
    u[j].z = __byte_perm(y[0], y[1], 0x7632);
    u[j].w = __byte_perm(y[2], y[3], 0x7632);
  }
  st32(p, u[0], u[1], wide);
}

template <typename T, int D, int GROUP>
__global__ void __launch_bounds__(kRwThreads) cache_read_kernel(const ReadArgs a) {
  using F = Fmt<D, GROUP>;
  constexpr int kLanes = D / 16;
  const unsigned row = blockIdx.x * (kRwThreads / kLanes) + threadIdx.x / kLanes;
  const int j = threadIdx.x % kLanes, lane = threadIdx.x & 31;
  const bool live = row < a.rows;
  uint32_t wk[2] = {0u, 0u}, wv[2] = {0u, 0u}, pk = 0, pv = 0;
  float inv = 0.f;
  if (live) {
    Row r = row_of(a.pg, row);
    look_up_page(a.pg, r);
    if (r.phys >= 0) {
      const int t = r.pos & 15, grp = j / (GROUP / 16);
      const uint8_t* tile = a.cache + tile_offset(a.pg, r.phys, r.h, r.pos, F::kTile);
      const LaneWords<D> at(t, j);
      wk[0] = *reinterpret_cast<const uint32_t*>(tile + at.k0);
      wk[1] = *reinterpret_cast<const uint32_t*>(tile + at.k0 + D / 8);
      wv[0] = *reinterpret_cast<const uint32_t*>(tile + at.v0);
      wv[1] = *reinterpret_cast<const uint32_t*>(tile + at.v1);
      pk = reinterpret_cast<const uint32_t*>(tile + F::kOffKp)[grp * 16 + t];
      pv = reinterpret_cast<const uint32_t*>(tile + F::kOffVp)[grp * 16 + t];
      inv = reinterpret_cast<const float*>(tile + F::kOffInv)[t];
    }
  }
  words_to_k(wk, j & 1);
  words_to_v(wv, lane);
  if (!live) return;
  const long long at = (long long)row * D + j * 16;
  store16(static_cast<T*>(a.k) + at, wk, pk, a.wide);
  store16(static_cast<T*>(a.v) + at, wv, pv, a.wide);
  if (a.inv && j == 0) a.inv[row] = inv;
}

}  // namespace cache
}  // namespace lsh
