// The 4-bit paged cache of decoding: format, addresses, and the quantiser.
//
// A page holds `page` consecutive positions of one sequence for every head; the
// block of one (page, head) is page / 16 tiles of 16 tokens.  A tile keeps all
// that attention needs of its tokens side by side, so that any number of
// consecutive tiles is one bulk copy:
//
//   K codes   16 rows of D/2 bytes: byte t*(D/8) + 4w + b, low nibble dim
//             32w + 8b + 2t, high nibble the next dim (t, b = 0..3, w < D/32)
//   V codes   8 token pairs of D bytes: the D/8-byte chunk number
//             g ^ (2 * (pair & 3)) holds, for word q < D/64 and token e of the
//             pair, at byte 8q + 4e, nibble i = dim 64q + 8i + g
//   K params  [D/group][16] words: scale (bf16) | zero (bf16) << 16
//   V params  the same
//   K inv     16 floats: 1 / max(||row||, 1e-12)
//
// Both code layouts are what the lanes of a 16 x 8 x 32 product of 8-bit integers hold:
// lane 4g + t takes D/8 consecutive bytes of K row g, of which a word's low nibbles and its
// high nibbles are two registers of its A fragment, and D/8 consecutive bytes of V's token
// pair t, whose bytes are dealt out to fragments by dims.  The chunk
// XOR keeps the latter free of shared-memory bank conflicts.
#pragma once

#include "common.cuh"

namespace lsh {
namespace cache {

constexpr int kTileTokens = 16;

template <int D, int GROUP>
struct Fmt {
  static constexpr int kGroups = D / GROUP;
  static constexpr int kOffV = 8 * D;
  static constexpr int kOffKp = 16 * D;
  static constexpr int kOffVp = kOffKp + 64 * kGroups;
  static constexpr int kOffInv = kOffVp + 64 * kGroups;
  static constexpr int kTile = kOffInv + 64;
  static_assert(kTile % 16 == 0, "tiles are copied in 16-byte units");
};

__host__ __device__ constexpr int tile_bytes(int D, int group) { return 16 * D + 128 * (D / group) + 64; }

// Division of numbers below 2^31 by a fixed one: n / d = (n m) >> (32 + s) with s = ceil(log2 d) - 1 (0 for
// d = 1) and m = ceil(2^(32 + s) / d), which fits 32 bits for d > 1; the error n / 2^(32 + s) of
// the rounded-up m stays below 1 / d.
struct FastDiv {
  uint32_t m, s;
  __host__ static FastDiv by(uint32_t d) {
    FastDiv f{0, 0};
    if (d <= 1) return f;
    while ((1ull << (f.s + 1)) < d) ++f.s;
    f.m = (uint32_t)(((1ull << (32 + f.s)) + d - 1) / d);
    return f;
  }
  __device__ __forceinline__ uint32_t of(uint32_t n) const { return m ? __umulhi(n, m) >> s : n; }
};

// Where a sequence's pages lie.  Page ids are checked against n_pages at every use.
struct Pages {
  const int32_t* table;  // [B, max_pages]
  const int32_t* ctx_len;  // [B]
  const int32_t* new_len;  // [B] or null (T for every sequence)
  int max_pages, page_log2, n_pages, H, T;
  FastDiv div_t, div_h;    // by T and by H
};

// Tokens of sequence b in the cache.  A count that is negative or more than its table has room
// for is the caller's error: recorded, and the sequence is treated as empty.
__device__ __forceinline__ int ctx_of(const Pages& p, int b) {
  const int c = p.ctx_len[b];
  if (c >= 0 && c <= ((long long)p.max_pages << p.page_log2)) return c;
  record_error(LSH_ERR_INVALID_ARG);
  return 0;
}

// Rows of this call that belong to sequence b, and the position of row 0 (negative when
// ctx_len is smaller than the number of rows: those rows have no position).
__device__ __forceinline__ int new_of(const Pages& p, int b) {
  if (!p.new_len) return p.T;
  const int n = p.new_len[b];
  return n < 0 ? 0 : (n > p.T ? p.T : n);
}

// Position of row i of sequence b, or -1.
__device__ __forceinline__ int row_pos(const Pages& p, int b, int i) {
  const int n = new_of(p, b);
  const int pos = ctx_of(p, b) - n + i;
  return (i < n && pos >= 0) ? pos : -1;
}

// Physical page of a position's logical page, or -1 (recorded) when the table's entry is bad.
__device__ __forceinline__ int page_of(const Pages& p, int b, int logical) {
  const int phys = p.table[(long long)b * p.max_pages + logical];
  if ((unsigned)phys < (unsigned)p.n_pages) return phys;
  record_error(LSH_ERR_INVALID_ARG);
  return -1;
}

// Byte offset of the tile of (physical page, head h, position).
__device__ __forceinline__ long long tile_offset(const Pages& p, int phys, int h, int pos, int tile) {
  const int in_page = pos & ((1 << p.page_log2) - 1);
  const long long block = (long long)tile << (p.page_log2 - 4);
  return ((long long)phys * p.H + h) * block + (long long)(in_page >> 4) * tile;
}

// 4 x 4 byte transpose over 4 neighbouring lanes: byte b of lane i becomes byte i of lane b.
__device__ __forceinline__ uint32_t transpose_bytes4(uint32_t x, int lane) {
  uint32_t y = __shfl_xor_sync(0xffffffffu, x, 2);
  x = __byte_perm(x, y, (lane & 2) ? 0x3276 : 0x5410);
  y = __shfl_xor_sync(0xffffffffu, x, 1);
  return __byte_perm(x, y, (lane & 1) ? 0x3715 : 0x6240);
}

__device__ __forceinline__ float bf16_bits(uint32_t b) { return __uint_as_float(b << 16); }

}  // namespace cache
}  // namespace lsh
