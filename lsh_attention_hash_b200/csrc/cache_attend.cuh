// Attention of new tokens over the 4-bit cache: one pass with the running maximum
// and sum of the softmax, the keys of all sequences dealt out evenly over the SMs and the
// pieces joined by a second small kernel.
//
// With K = z + s c by groups of dims, a query's logit needs only whole codes on the
// matrix units:  q . K = sum_grp ( s_grp sum_d q_d c_d + z_grp sum_d q_d ),  and
// the output  O_d = sum_j (p_j s_j) c_jd + sum_j p_j z_j.  So codes are the A operand and
// the queries (then the weights p_j s_j) the B operand: S^T = K Q^T and O^T = V^T P^T,
// 8 columns wide.  With keys as the 16 rows, a group of query heads or several new tokens
// share every key that is unpacked.
//
// What bounds it after memory is unpacking: integer instructions issue at half rate, so
// their number per code decides.
//   K: mma.m16n8k32 of 8-bit integers.  A word's 8 codes are two masks and a shift.  The query
//      is a fixed-point number of the column's largest |q|: 16 bits (an upper and a lower
//      byte, two products) for bf16 queries, 24 bits (three) for fp32 ones.  The sums are
//      exact; the rounding of q is 2^-16 (2^-24) of its largest entry.
//   V: mma.m16n8k16 in bf16, since weights need a float's range.  0x4300 | c is 128 + c in
//      bf16; the 128 is taken out by one more product per group with a constant -128 operand,
//      so a code costs no arithmetic beyond its mask.  In fp32 the weights are three bf16
//      pieces (24 bits), 128 is subtracted from the codes, and the sums leave the matrix
//      unit after every stage, so that its accumulation does not show.
//
// A single token has one or two query columns, and all that follows the products (scales,
// exponentials, weights) would be done for 8.  So a fragment's 8 columns are CW query columns
// of each of TP = 8 / CW tiles: tile i's products use a B operand that is zero outside its
// own CW columns, and add into the same fragment.  Column n = i CW + c is a stream of its
// own with its own maximum and sum; the streams are joined with the warps at the end.
//
// Every warp is a pipeline of its own: a lane copies ST tiles (cp.async.bulk, codes
// and parameters together, one copy for tiles that lie side by side) into the warp's ring,
// and the warp consumes them without a block barrier.  A piece's warps meet once, at its end.
// The maximum moves only when a logit exceeds it by 2^8: weights up to 256 cost nothing
// in float, and the 32-lane maximum and the rescaling of O are left out of most steps.
//
// The work is the list of all (cached head, column tile) items, with the row too when pages are
// selected, each of ceil(keys / 128) blocks; CTA c of NC takes blocks [c W / NC, (c + 1) W / NC) of
// it, whatever the lengths are, so one wave of CTAs ends together.  An item inside one CTA is
// written out there; the pieces of any other go to the workspace (a CTA has two at most: its
// first and its last) and the join adds them up in order.
#pragma once

#include <type_traits>

#include "cache_common.cuh"
#include "tc_common.cuh"

namespace lsh {
namespace cache {

constexpr int kAttWarps = 4;
constexpr int kAttThreads = kAttWarps * 32;
constexpr int kMaxEntries = 256;     // pages looked up at a time
constexpr int kBlockTiles = 8;       // 128 tokens: what the work is dealt out in
constexpr float kLazyMax = 8.f;

struct AttendArgs {
  const void* q;            // [B, H * G, T, D]
  const uint8_t* cache;
  const int32_t* selected;  // [B, H, T, n_select] or null
  void* out;                // [B, H * G, T, D]
  float* lse;               // [B, H * G, T]
  float *part_o, *part_ml;  // [NC, 2, cols of a tile, D], [NC, 2, cols of a tile, 2]
  int B, G, n_select;
  int causal, self_mask, unit_keys, out_f32;
  float scale_log2;         // scale * log2(e)
  int nc, n_ct, cols, tile_cols;  // CTAs; column tiles, all columns, columns of a tile
  uint32_t nibbles, c128;   // 0x000f000f, 0x43004300 (see codes2)
  Pages pg;
};

// A sequence's part of the work: items of nb blocks each.  Without selection an item is (cached
// head, column tile); with it (cached head, row, column tile) for the rows that have a position.
struct Seq {
  int ctx, n_new, start;   // tokens in the cache, rows of this call, position of row 0
  int row0, n_rows;        // with selection: first row with a position, and how many
  int n_list, items, nb;   // keys of an item in list order, number of items, blocks of an item
};

__device__ __forceinline__ Seq seq_of(const AttendArgs& a, int b) {
  Seq s;
  s.ctx = ctx_of(a.pg, b);
  s.n_new = new_of(a.pg, b);
  s.start = s.ctx - s.n_new;
  s.row0 = s.start < 0 ? -s.start : 0;
  s.n_rows = max(0, s.n_new - s.row0);
  const bool sel = a.selected != nullptr;
  if (!sel && s.n_rows > 0) {
    s.row0 = 0;
    s.n_rows = 1;
  }
  s.n_list = s.n_rows > 0 ? (sel ? a.n_select << a.pg.page_log2 : s.ctx) : 0;
  s.items = a.pg.H * s.n_rows * a.n_ct;
  s.nb = (s.n_list + kBlockTiles * kTileTokens - 1) / (kBlockTiles * kTileTokens);
  return s;
}

// Whether row t is one of the sequence's tokens (padding is answered with zeros).
__device__ __forceinline__ bool row_live(const Seq& s, int t) { return t < s.n_new && s.start + t >= 0; }

// Sum of v over the lanes up to and including this one.
__device__ __forceinline__ long long warp_scan(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

// Blocks of all sequences, and of those before b (whole warp).
__device__ __forceinline__ void work_before(const AttendArgs& a, int b, int lane, long long& total, long long& before) {
  total = before = 0;
  for (int i0 = 0; i0 < a.B; i0 += 32) {
    long long v = 0;
    if (i0 + lane < a.B) {
      const Seq s = seq_of(a, i0 + lane);
      v = (long long)s.items * s.nb;
    }
    const long long sum = warp_scan(v, lane);
    if (b >= i0 && b < i0 + 32) before = total + __shfl_sync(0xffffffffu, sum - v, b - i0);
    total += __shfl_sync(0xffffffffu, sum, 31);
  }
}

// The sequence that block x of the work belongs to, and the blocks before it (whole warp).
__device__ __forceinline__ int work_find(const AttendArgs& a, long long x, int lane, long long& before) {
  before = 0;
  for (int i0 = 0; i0 < a.B; i0 += 32) {
    long long v = 0;
    if (i0 + lane < a.B) {
      const Seq s = seq_of(a, i0 + lane);
      v = (long long)s.items * s.nb;
    }
    const long long sum = warp_scan(v, lane);
    const unsigned over = __ballot_sync(0xffffffffu, before + sum > x);
    if (over) {
      const int l = __ffs(over) - 1;
      before += __shfl_sync(0xffffffffu, sum - v, l);
      return i0 + l;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  return a.B;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes (unsigned bytes) times signed (BS) or unsigned bytes.
template <bool BS>
__device__ __forceinline__ void imma16832(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  if (BS)
    asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.u8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Two codes (the low nibbles of both halves of w >> 4 i) as bf16: 128 + c, or c with SUB.  The
// constants come in as values (kernel arguments): as literals the mask and the exponent would be
// two instructions, since one instruction holds one literal.
template <bool SUB>
__device__ __forceinline__ uint32_t codes2(uint32_t w, int i, uint32_t nibbles, uint32_t c128) {
  uint32_t x;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(x) : "r"(w >> (4 * i)), "r"(nibbles), "r"(c128));  // (w & n) | c
  if (SUB) {
    __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&c128));
    x = *reinterpret_cast<uint32_t*>(&r);
  }
  return x;
}

// N consecutive words of shared memory (8 or 16 byte loads).
template <int N>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x; w[1] = u.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 u = *reinterpret_cast<const uint4*>(p + 16 * i);
      w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
    }
  }
}

// CW: query columns of a tile in a fragment (2, 4 or 8); NT: fragments side by side (CW 8 only).
template <typename TQ, int D, int GROUP, int CW, int NT>
struct AttendCfg {
  using F = Fmt<D, GROUP>;
  static_assert(CW == 8 || NT == 1, "more than 8 columns go in whole fragments");
  static constexpr bool kF32 = sizeof(TQ) == 4;
  static constexpr int kPieces = kF32 ? 3 : 1;   // bf16 pieces of a weight
  static constexpr int kBytes = kF32 ? 3 : 2;    // bytes of a query's fixed-point number,
  static constexpr int kTop = kF32 ? 0x7fffff : 0x7fff;  // and its largest value
  // 128 taken out of V's codes: always in fp32; at D 256 the -128 products' accumulators would not fit
  static constexpr bool kSub = kF32 || D == 256;
  static constexpr int kKs = D / 16;             // m tiles of V^T P^T
  static constexpr int kTp = 8 / CW;             // tiles of a fragment
  static constexpr int kSt = kTp > 2 ? kTp : 2;  // tiles of a stage
  static constexpr int kSf = kSt / kTp;          // fragments of a stage
  static constexpr int kQ = CW * NT;             // query columns of a CTA
  static constexpr int kCols = 8 * NT;           // streams of a warp
  // four tiles fill the time of their own copies with the other warps' work; two take a second stage
  static constexpr int kStages = kSt > 2 ? 1 : 2;
  static constexpr int kStageBytes = kSt * F::kTile;
  static constexpr int kRing = kAttWarps * kStages * kStageBytes;
  static constexpr int kMerge = kAttWarps * kCols * D * 4;
  static constexpr int kOffQ = (kRing > kMerge ? kRing : kMerge);
  static constexpr int kOffQs = kOffQ + kBytes * NT * kTp * (D / 32) * 32 * 8;
  static constexpr int kOffMl = kOffQs + kQ * (F::kGroups + 1) * 4;
  static constexpr int kOffEnt = kOffMl + kAttWarps * kCols * 8;
  static constexpr int kOffBar = kOffEnt + kMaxEntries * 8;
  static constexpr int kOffDesc = kOffBar + kAttWarps * kStages * 8;
  static constexpr int kSmem = kOffDesc + kAttWarps * kStages * kSt * 4;
  static_assert(kOffMl % 8 == 0 && kOffBar % 8 == 0 && kOffDesc % 8 == 0, "alignment");
  static_assert(kBlockTiles % kSt == 0, "blocks are whole stages");
  // CTAs of an SM: what registers allow (128 threads each) and what shared memory does
  static constexpr int kByRegs = D == 256 ? 2 : NT == 2 ? (D == 64 ? 3 : 2) : D == 64 ? (kF32 ? 4 : 5)
                                 : kF32 || GROUP == 32 ? 3 : 4;
  static constexpr int kBySmem = 227 * 1024 / (kSmem + 1024);
  static constexpr int kCtas = kByRegs < kBySmem ? kByRegs : kBySmem;
};

template <typename TQ, int D, int GROUP, int CW, int NT>
__global__ void __launch_bounds__(kAttThreads, AttendCfg<TQ, D, GROUP, CW, NT>::kCtas)
cache_attend_kernel(const __grid_constant__ AttendArgs a) {
  using C = AttendCfg<TQ, D, GROUP, CW, NT>;
  using F = Fmt<D, GROUP>;
  constexpr int NG = F::kGroups, KS = C::kKs, P = C::kPieces, TP = C::kTp, ST = C::kSt, SF = C::kSf;
  constexpr bool SUB = C::kSub;
  constexpr int kStages = C::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int abort_flag;
  uint4* qf = reinterpret_cast<uint4*>(smem + C::kOffQ);
  float* qs = reinterpret_cast<float*>(smem + C::kOffQs);
  float* qstep = qs + C::kQ * NG;
  float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);
  int2* ent = reinterpret_cast<int2*>(smem + C::kOffEnt);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  int* descs = reinterpret_cast<int*>(smem + C::kOffDesc);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const bool sel = a.selected != nullptr;
  const int pl = a.pg.page_log2;
  const uint32_t nibbles = a.nibbles, c128 = a.c128;
  uint8_t* ring = smem + warp * kStages * C::kStageBytes;
  uint64_t* bar = bars + warp * kStages;
  int* desc = descs + warp * kStages * ST;
  if (tid < kAttWarps * kStages) tc::mbar_init(bars + tid, 1);
  if (tid == 0) abort_flag = 0;
  tc::fence_mbar_init();
  int slot = 0;
  uint32_t phase = 0;

  // ---- the CTA's stretch of the work -----------------------------------------------------------------
  long long total, before;
  work_before(a, 0, lane, total, before);
  const long long nc = min((long long)a.nc, total);  // CTAs with work: a block each at least
  if (blockIdx.x >= nc) return;
  long long x = blockIdx.x * total / nc;
  const long long x_end = (blockIdx.x + 1) * total / nc;
  int b = work_find(a, x, lane, before);
  Seq u = seq_of(a, b);

  while (x < x_end) {
  while (x >= before + (long long)u.items * u.nb) {  // the next sequence with anything to do
    before += (long long)u.items * u.nb;
    u = seq_of(a, ++b);
  }
  const int item = (int)((x - before) / u.nb);
  const int blk0 = (int)((x - before) - (long long)item * u.nb);
  const int blk1 = (int)min((long long)u.nb, blk0 + (x_end - x));
  x += blk1 - blk0;
  const int ct = item % a.n_ct, rest = item / a.n_ct;
  const int row_t = sel ? u.row0 + rest % u.n_rows : 0;  // the row, with selection
  const int h = sel ? rest / u.n_rows : rest;
  const int col0 = ct * C::kQ;
  const int tile_lo = blk0 * kBlockTiles;
  const int tile_hi = min(blk1 * kBlockTiles, (u.n_list + kTileTokens - 1) / kTileTokens);
  tc::fence_proxy_async_smem();  // (the last item's sums lay where copies go now)
  __syncthreads();

  // ---- set-up of the item: query operands and sums -----------------------------------------------------
  const int32_t* picks = sel ? a.selected + (((long long)b * a.pg.H + h) * a.pg.T + row_t) * a.n_select : nullptr;
  auto q_row = [&](int col) -> const TQ* {
    const int tt = sel ? row_t : col / a.G, gg = sel ? col : col - tt * a.G;
    return static_cast<const TQ*>(a.q) + (((long long)b * a.pg.H + h) * a.G + gg) * (long long)a.pg.T * D +
           (long long)tt * D;
  };
  // 16 threads a column: sums by group, and the step of the fixed-point numbers
  for (int cc = tid >> 4; cc < C::kQ; cc += kAttThreads / 16) {
    const int j = tid & 15;
    const uint32_t half = 0xffffu << (tid & 16);
    float sum = 0.f, top = 0.f;
    if (col0 + cc < a.cols) {
      const TQ* q = q_row(col0 + cc) + j * (D / 16);
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        const float v = to_f32<TQ>(q[d]);
        sum += v;
        // a NaN counts as infinity: the step is then infinite and so is, or NaN, every logit
        top = fmaxf(top, v == v ? fabsf(v) : INFINITY);
      }
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
      if (o < 16 / NG) sum += __shfl_xor_sync(half, sum, o);
      top = fmaxf(top, __shfl_xor_sync(half, top, o));
    }
    if (j % (16 / NG) == 0) qs[cc * NG + j / (16 / NG)] = sum;
    if (j == 0) qstep[cc] = top / C::kTop;
  }
  __syncthreads();
  // B operands of K's products, byte by byte: fragment column n = i CW + c holds query column c for
  // tile i and zero for the others; word w covers dims 32 w .. 32 w + 31
  for (int i = tid; i < NT * (D / 32) * 32; i += kAttThreads) {
    const int l = i & 31, w = (i >> 5) % (D / 32), nt = (i >> 5) / (D / 32);
    const int n = l >> 2, cc = nt * CW + n % CW, col = col0 + cc;
    const float step = qstep[cc];
    const float inv = step > 0.f ? 1.f / step : 0.f;
    uint32_t v[C::kBytes][2];
#pragma unroll
    for (int p = 0; p < C::kBytes; ++p) v[p][0] = v[p][1] = 0u;
    if (col < a.cols) {
      const TQ* q = q_row(col) + 32 * w + 2 * (l & 3);
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x = to_f32<TQ>(q[8 * k + e]);
          // x / step; a step too small to invert (denormal queries) is divided by
          const float y = inv < INFINITY ? x * inv : x / step;
          const int f = max(-C::kTop, min(C::kTop, __float2int_rn(y)));
#pragma unroll
          for (int p = 0; p < C::kBytes; ++p) v[p][e] |= ((f >> (8 * p)) & 255) << (8 * k);
        }
    }
#pragma unroll
    for (int p = 0; p < C::kBytes; ++p)
#pragma unroll
      for (int t = 0; t < TP; ++t)
        reinterpret_cast<uint2*>(qf + (((p * NT + nt) * TP + t) * (D / 64) + (w >> 1)) * 32 + l)[w & 1] =
            n / CW == t ? make_uint2(v[p][0], v[p][1]) : make_uint2(0u, 0u);
  }
  __syncthreads();

  // ---- the lane's streams (C fragment: columns 2 t4 and 2 t4 + 1 of each 8) -------------------------
  const int my_tile = 2 * t4 / CW;  // the tile of a fragment that both belong to
  int pos[NT][2], last[NT][2];  // position; largest admissible position
  bool self[NT][2];             // whether its own key is masked
  int fast = u.ctx;             // tiles that end at or below are admissible to every column
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int col = col0 + nt * CW + (2 * t4 + k) % CW;
      const int tt = sel ? row_t : col / a.G;
      const bool live = col < a.cols && row_live(u, tt);
      pos[nt][k] = live ? u.start + tt : -1;
      last[nt][k] = !live ? -1 : (a.causal ? pos[nt][k] : u.ctx - 1);
      self[nt][k] = live && a.self_mask;
      if (live && a.self_mask) {
        // its own key counts when nothing else is admissible
        bool other;
        if (!sel) {
          other = last[nt][k] > 0;
        } else {
          other = false;
          for (int i = 0; i < a.n_select && !other; ++i) {
            const int lp = picks[i];
            if (lp < 0 || lp >= a.pg.max_pages) continue;
            const long long f = (long long)lp << pl;
            const long long e = min((long long)last[nt][k], f + (1 << pl) - 1);  // last admissible of the page
            other = f <= e && (e > f || f != pos[nt][k]);
          }
        }
        self[nt][k] = other;
      }
      if (live && (a.causal || a.self_mask)) fast = min(fast, pos[nt][k]);
    }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) fast = min(fast, __shfl_xor_sync(0xffffffffu, fast, o));

  float qsum[NT][NG][2], step[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) qsum[nt][n][k] = qs[(nt * CW + (2 * t4 + k) % CW) * NG + n];

#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int k = 0; k < 2; ++k) step[nt][k] = qstep[nt * CW + (2 * t4 + k) % CW];

  float m[NT][2], base[NT][2], bar_m[NT][2], l[NT][2];  // maximum; what is subtracted; where it has to move
  float o[NT][KS][4], zs[NT][NG][2], cb[SUB ? 1 : NT][SUB ? 1 : NG][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      m[nt][k] = bar_m[nt][k] = -INFINITY;
      base[nt][k] = l[nt][k] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[nt][i][k] = 0.f;
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      zs[nt][n][0] = zs[nt][n][1] = 0.f;
      if (!SUB)
#pragma unroll
        for (int k = 0; k < 4; ++k) cb[SUB ? 0 : nt][SUB ? 0 : n][k] = 0.f;
    }
  }

  // ---- the warp's pipeline ------------------------------------------------------------------------
  int tile0 = tile_lo, tile1 = tile_lo, e0 = 0;  // the tiles whose pages are looked up, in list order
  auto issue = [&](int st, int slot) {  // lane 0: copies of stage st, and the positions of its tiles (-1: none)
    uint32_t bytes = 0;
    const uint8_t* src[ST];
#pragma unroll
    for (int k = 0; k < ST; ++k) {
      const int tile = tile0 + st * ST + k;
      src[k] = nullptr;
      int first = -1;
      if (tile < tile1) {
        const int2 e = ent[((tile << 4) >> pl) - e0];
        const int p = e.y + ((tile << 4) & ((1 << pl) - 1));
        if (e.x >= 0 && p < u.ctx) {
          src[k] = a.cache + tile_offset(a.pg, e.x, h, p, F::kTile);
          bytes += F::kTile;
          first = p;
        }
      }
      desc[slot * ST + k] = first;
    }
    tc::mbar_arrive_expect_tx(bar + slot, bytes);
    const uint32_t dst = tc::smem_u32(ring + slot * C::kStageBytes);
    int from = 0;  // runs of tiles side by side
#pragma unroll
    for (int k = 1; k <= ST; ++k) {
      if (k < ST && src[k] && src[k] == src[k - 1] + F::kTile) continue;
      if (src[k - 1]) bulk_load(dst + from * F::kTile, src[k - 1] - (k - 1 - from) * F::kTile, (k - from) * F::kTile, bar + slot);
      from = k;
    }
  };
  // One stage of ST tiles.  MASKED: a tile may be missing, and every key is tested against the columns.
  auto consume = [&](const uint8_t* buf, const int* first, auto masked_c) {  // first: positions, in shared memory
    constexpr bool MASKED = decltype(masked_c)::value;
    // ---- logits: s[f][nt][0,1]: key g of the lane's tile, columns 2 t4, +1;  [2,3]: key g + 8
    float s[SF][NT][4];
#pragma unroll
    for (int f = 0; f < SF; ++f) {
      int part[C::kBytes][NT][NG][4];
#pragma unroll
      for (int p = 0; p < C::kBytes; ++p)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) part[p][nt][n][c] = 0;
#pragma unroll
      for (int i = 0; i < TP; ++i) {
        const int k = f * TP + i;
        if (MASKED && first[k] < 0) continue;
        const uint8_t* tb = buf + k * F::kTile;
        uint32_t wa[D / 32], wb[D / 32];
        lds_words<D / 32>(tb + g * (D / 2) + t4 * (D / 8), wa);
        lds_words<D / 32>(tb + (g + 8) * (D / 2) + t4 * (D / 8), wb);
#pragma unroll
        for (int w = 0; w < D / 32; w += 2) {
          uint32_t y[2][4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            y[e][0] = wa[w + e] & 0x0f0f0f0fu;
            y[e][1] = wb[w + e] & 0x0f0f0f0fu;
            y[e][2] = (wa[w + e] >> 4) & 0x0f0f0f0fu;
            y[e][3] = (wb[w + e] >> 4) & 0x0f0f0f0fu;
          }
#pragma unroll
          for (int p = 0; p < C::kBytes; ++p)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint4 q = qf[(((p * NT + nt) * TP + i) * (D / 64) + w / 2) * 32 + lane];
              constexpr int kLast = C::kBytes - 1;
              if (p == kLast) {
                imma16832<true>(part[p][nt][w * 32 / GROUP], y[0][0], y[0][1], y[0][2], y[0][3], q.x, q.y);
                imma16832<true>(part[p][nt][(w + 1) * 32 / GROUP], y[1][0], y[1][1], y[1][2], y[1][3], q.z, q.w);
              } else {
                imma16832<false>(part[p][nt][w * 32 / GROUP], y[0][0], y[0][1], y[0][2], y[0][3], q.x, q.y);
                imma16832<false>(part[p][nt][(w + 1) * 32 / GROUP], y[1][0], y[1][1], y[1][2], y[1][3], q.z, q.w);
              }
            }
        }
      }
      const int mine = f * TP + my_tile;
      const int first_mine = MASKED ? first[mine] : 0;
      const uint8_t* tb = buf + mine * F::kTile;
      const uint32_t* kp = reinterpret_cast<const uint32_t*>(tb + F::kOffKp);
      float acc[NT][4], zero[NT][4];  // sum of s (codes . q) in steps of q, and of z (sum of q)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[nt][c] = zero[nt][c] = 0.f;
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const uint32_t pa = kp[n * 16 + g], pb = kp[n * 16 + g + 8];
        const float sa = bf16_bits(pa), za = __uint_as_float(pa & 0xffff0000u);
        const float sb = bf16_bits(pb), zb = __uint_as_float(pb & 0xffff0000u);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            // at most 64 * 15 * 2^15 in 16 bits; the third byte joins in float
            const int v16 = part[C::kBytes - 1][nt][n][c] * 256 + part[C::kBytes - 2][nt][n][c];
            float v = (float)v16;
            if (C::kBytes == 3) v = fmaf(v, 256.f, (float)part[0][nt][n][c]);
            acc[nt][c] = fmaf(c < 2 ? sa : sb, v, acc[nt][c]);
            zero[nt][c] = fmaf(c < 2 ? za : zb, qsum[nt][n][c & 1], zero[nt][c]);
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[nt][c] = fmaf(acc[nt][c], step[nt][c & 1], zero[nt][c]);
      float fa = a.scale_log2, fb = a.scale_log2;
      if (a.unit_keys) {
        const float* inv = reinterpret_cast<const float*>(tb + F::kOffInv);
        fa *= inv[g];
        fb *= inv[g + 8];
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float x = acc[nt][c] * (c < 2 ? fa : fb);
          if (MASKED) {
            const int key = first_mine + g + (c < 2 ? 0 : 8);
            if (first_mine < 0 || key > last[nt][c & 1] || (key == pos[nt][c & 1] && self[nt][c & 1])) x = -INFINITY;
          }
          s[f][nt][c] = x;
        }
    }
    // ---- the running maximum, moved only when a logit is 2^8 above it
    float top[NT][2];
    bool raise = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = fmaxf(s[0][nt][c], s[0][nt][c + 2]);
#pragma unroll
        for (int f = 1; f < SF; ++f) x = fmaxf(fmaxf(x, s[f][nt][c]), s[f][nt][c + 2]);
        top[nt][c] = x;
        raise |= x > bar_m[nt][c];
      }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float x = top[nt][c];
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          const float mn = fmaxf(m[nt][c], x);
          const float al = m[nt][c] == mn ? 1.f : exp2f(m[nt][c] - mn);
          m[nt][c] = mn;
          base[nt][c] = mn == -INFINITY ? 0.f : mn;
          bar_m[nt][c] = mn == -INFINITY ? mn : mn + kLazyMax;
          l[nt][c] *= al;
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            o[nt][i][c] *= al;
            o[nt][i][c + 2] *= al;
          }
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            zs[nt][n][c] *= al;
            if (!SUB) {
              cb[SUB ? 0 : nt][SUB ? 0 : n][c] *= al;
              cb[SUB ? 0 : nt][SUB ? 0 : n][c + 2] *= al;
            }
          }
        }
    }
    float fresh[P > 1 ? NT : 1][P > 1 ? KS : 1][4];  // fp32: this stage's sums
    if (P > 1) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) fresh[P > 1 ? nt : 0][P > 1 ? i : 0][c] = 0.f;
    }
#pragma unroll
    for (int f = 0; f < SF; ++f) {
      float p[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float x = s[f][nt][c] - base[nt][c & 1];
          p[nt][c] = P > 1 ? exp2f(x) : tc::ex2_approx(x);
          l[nt][c & 1] += p[nt][c];
        }
      const uint32_t* vp = reinterpret_cast<const uint32_t*>(buf + (f * TP + my_tile) * F::kTile + F::kOffVp);
      uint32_t pf[P][NG][NT][2];  // B fragments of (p s): [0] keys 0..7, [1] keys 8..15 of every column's tile
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const uint32_t pa = vp[n * 16 + g], pb = vp[n * 16 + g + 8];
        const float sa = bf16_bits(pa), za = __uint_as_float(pa & 0xffff0000u);
        const float sb = bf16_bits(pb), zb = __uint_as_float(pb & 0xffff0000u);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const bool out = MASKED && s[f][nt][c] == -INFINITY;  // whatever lies in a masked place
            w[c] = out ? 0.f : p[nt][c] * (c < 2 ? sa : sb);
            if (!out) zs[nt][n][c & 1] = fmaf(p[nt][c], c < 2 ? za : zb, zs[nt][n][c & 1]);
          }
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const uint32_t lo = tc::pack_bf16x2(w[0], w[1]), hi = tc::pack_bf16x2(w[2], w[3]);
            pf[i][n][nt][0] = movmatrix(lo);
            pf[i][n][nt][1] = movmatrix(hi);
            if (i + 1 < P) {
              w[0] -= bf16_bits(lo); w[1] -= __uint_as_float(lo & 0xffff0000u);
              w[2] -= bf16_bits(hi); w[3] -= __uint_as_float(hi & 0xffff0000u);
            }
          }
        }
      }
      if (!SUB) {
        const uint32_t c = 0xc300c300u;  // -128 twice
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(cb[SUB ? 0 : nt][SUB ? 0 : n], c, c, c, c, pf[0][n][nt][0], pf[0][n][nt][1]);
      }
#pragma unroll
      for (int i = 0; i < TP; ++i) {
        const int k = f * TP + i;
        if (MASKED && first[k] < 0) continue;
        const uint8_t* tb = buf + k * F::kTile;
        uint32_t pb[P][NG][NT][2];  // the tile's own columns
#pragma unroll
        for (int pc = 0; pc < P; ++pc)
#pragma unroll
          for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) pb[pc][n][nt][e] = TP == 1 || g / CW == i ? pf[pc][n][nt][e] : 0u;
        const uint8_t* vrow = tb + F::kOffV + t4 * D + (g ^ (2 * t4)) * (D / 8);
        uint32_t w0[D / 32], w1[D / 32];  // token pairs t4 and t4 + 4
        lds_words<D / 32>(vrow, w0);
        lds_words<D / 32>(vrow + 4 * D, w1);
#pragma unroll
        for (int q = 0; q < D / 64; ++q) {
          // the two tokens of a pair side by side: 16 dims in two words
          uint32_t r0[2], r1[2];
          r0[0] = __byte_perm(w0[2 * q], w0[2 * q + 1], 0x5410);
          r0[1] = __byte_perm(w0[2 * q], w0[2 * q + 1], 0x7632);
          r1[0] = __byte_perm(w1[2 * q], w1[2 * q + 1], 0x5410);
          r1[1] = __byte_perm(w1[2 * q], w1[2 * q + 1], 0x7632);
#pragma unroll
          for (int mm = 0; mm < 4; ++mm) {
            const int mt = 4 * q + mm, n = mt * 16 / GROUP, x = (mm & 1) * 2;
            const uint32_t a0 = codes2<SUB>(r0[mm >> 1], x, nibbles, c128);
            const uint32_t a1 = codes2<SUB>(r0[mm >> 1], x + 1, nibbles, c128);
            const uint32_t a2 = codes2<SUB>(r1[mm >> 1], x, nibbles, c128);
            const uint32_t a3 = codes2<SUB>(r1[mm >> 1], x + 1, nibbles, c128);
#pragma unroll
            for (int pc = P - 1; pc >= 0; --pc)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float(&dst)[4] = P > 1 ? fresh[P > 1 ? nt : 0][P > 1 ? mt : 0] : o[nt][mt];
                mma16816(dst, a0, a1, a2, a3, pb[pc][n][nt][0], pb[pc][n][nt][1]);
              }
          }
        }
      }
    }
    if (P > 1) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[nt][i][c] += fresh[P > 1 ? nt : 0][P > 1 ? i : 0][c];
    }
  };

  while (tile1 < tile_hi) {
  // pages of the next tiles (the table and, with selection, the list), as many as are held at a time
  tile0 = tile1;
  e0 = (tile0 << 4) >> pl;
  tile1 = (int)min((long long)tile_hi, ((long long)(e0 + kMaxEntries) << pl) >> 4);
  const int n_ent = (((tile1 - 1) << 4) >> pl) - e0 + 1;
  if (tile0 != tile_lo) __syncthreads();
  for (int i = tid; i < n_ent; i += kAttThreads) {
    int logical = e0 + i;
    if (sel) logical = picks[e0 + i];
    int phys = -1;
    if (logical >= 0 && logical < a.pg.max_pages && ((long long)logical << pl) < u.ctx) phys = page_of(a.pg, b, logical);
    ent[i] = make_int2(phys, logical << pl);
  }
  __syncthreads();
  const int n_stage = (tile1 - tile0 + ST - 1) / ST;
  if (lane == 0)
    for (int i = 0, s2 = slot; i < kStages; ++i) {
      if (warp + i * kAttWarps < n_stage) issue(warp + i * kAttWarps, s2);
      s2 = s2 + 1 == kStages ? 0 : s2 + 1;
    }
  __syncwarp();
  for (int st = warp; st < n_stage; st += kAttWarps) {
    if (!tc::mbar_wait(bar + slot, phase, &abort_flag)) {
      // give the copies in flight the same time each, then leave
      for (int i = 0, s2 = slot; i < kStages; ++i) {
        if (st + i * kAttWarps < n_stage) {
          const unsigned long long t0 = tc::globaltimer();
          while (!tc::mbar_try_wait(bar + s2, (s2 < slot) ? phase ^ 1 : phase) && tc::globaltimer() - t0 < tc::kWaitNs) {
          }
        }
        s2 = s2 + 1 == kStages ? 0 : s2 + 1;
      }
      break;
    }
    const int* first = desc + slot * ST;
    int lo = first[0], hi = lo;
#pragma unroll
    for (int k = 1; k < ST; ++k) {
      lo = min(lo, first[k]);
      hi = max(hi, first[k]);
    }
    const uint8_t* buf = ring + slot * C::kStageBytes;
    if (lo >= 0 && hi + kTileTokens <= fast)
      consume(buf, first, std::false_type());
    else if (hi >= 0)
      consume(buf, first, std::true_type());
    __syncwarp();
    if (lane == 0 && st + kStages * kAttWarps < n_stage) issue(st + kStages * kAttWarps, slot);
    if (++slot == kStages) {
      slot = 0;
      phase ^= 1;
    }
  }
  }

  // ---- join the warps -----------------------------------------------------------------------------
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], x);
#pragma unroll
        for (int n = 0; n < NG; ++n) zs[nt][n][c] += __shfl_xor_sync(0xffffffffu, zs[nt][n][c], x);
      }
      if (g == 0) ml[warp * C::kCols + nt * 8 + 2 * t4 + c] = make_float2(m[nt][c], l[nt][c]);
    }
  __syncthreads();  // the ring is free
  float* om = reinterpret_cast<float*>(smem);  // [warp][col][D]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      const int n = i * 16 / GROUP;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float x = o[nt][i][c] + zs[nt][n][c & 1];
        if (!SUB) x += cb[SUB ? 0 : nt][SUB ? 0 : n][c];
        om[(warp * C::kCols + nt * 8 + 2 * t4 + (c & 1)) * D + i * 16 + g + (c < 2 ? 0 : 8)] = x;
      }
    }
  __syncthreads();
  for (int i = tid; i < C::kQ * D; i += kAttThreads) {
    const int cc = i / D, d = i - cc * D, col = col0 + cc;
    if (col >= a.cols) break;
    const int n0 = NT > 1 ? cc : cc % CW;  // its first stream; the others CW further each
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kAttWarps * TP; ++w) mx = fmaxf(mx, ml[w / TP * C::kCols + n0 + w % TP * CW].x);
    float sum = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kAttWarps * TP; ++w) {
      const int j = w / TP * C::kCols + n0 + w % TP * CW;
      const float2 v = ml[j];
      const float f = v.x == mx ? 1.f : exp2f(v.x - mx);
      sum = fmaf(v.y, f, sum);
      y = fmaf(om[j * D + d], f, y);
    }
    if (blk0 == 0 && blk1 == u.nb) {
      const int tt = sel ? row_t : col / a.G, gg = sel ? col : col - tt * a.G;
      const long long row = (((long long)b * a.pg.H + h) * a.G + gg) * a.pg.T + tt;
      if (!row_live(u, tt)) sum = 0.f;
      y = sum == 0.f ? 0.f : y / sum;
      if (a.out_f32)
        static_cast<float*>(a.out)[row * D + d] = y;
      else
        static_cast<__nv_bfloat16*>(a.out)[row * D + d] = __float2bfloat16_rn(y);
      if (d == 0) a.lse[row] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * 0.6931471805599453f;
    } else {
      const long long pi = ((long long)blockIdx.x * 2 + (blk0 == 0 ? 1 : 0)) * C::kQ + cc;
      a.part_o[pi * D + d] = y;
      if (d == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * pi) = make_float2(mx, sum);
    }
  }
  }
}

// Joins the pieces of a column: out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i, and answers the
// rows that no item has (padding).
constexpr int kJoinThreads = 128;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) cache_join_kernel(const __grid_constant__ AttendArgs a) {
  constexpr int kLanes = D / 4, kParts = kJoinThreads / kLanes;  // 4 dims a thread, the pieces dealt out
  __shared__ float4 so[kParts][kLanes];
  __shared__ float2 sml[kParts];
  const bool sel = a.selected != nullptr;
  const int unit = blockIdx.x / a.cols, col = blockIdx.x - unit * a.cols;
  const int bh = sel ? unit / a.pg.T : unit;
  const int b = bh / a.pg.H, h = bh - b * a.pg.H;
  const int tt = sel ? unit - bh * a.pg.T : col / a.G, gg = sel ? col : col - tt * a.G;
  const int j = threadIdx.x % kLanes, part = threadIdx.x / kLanes;
  const Seq u = seq_of(a, b);
  float mx = -INFINITY, sum = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  const int ct = col / a.tile_cols, cc = col - ct * a.tile_cols;
  int c0 = 0, c1 = -1;  // the CTAs that have pieces
  if (u.n_rows > 0 && (!sel || row_live(u, tt))) {
    long long total, before;
    work_before(a, b, threadIdx.x & 31, total, before);
    const long long item = ((sel ? (long long)h * u.n_rows + tt - u.row0 : h) * a.n_ct) + ct;
    const long long first = before + item * u.nb;
    // CTA of block y: the largest c with floor(c total / nc) <= y
    const long long nc = min((long long)a.nc, total);
    c0 = (int)(((first + 1) * nc - 1) / total);
    c1 = (int)(((first + u.nb) * nc - 1) / total);
  }
  // before any thread leaves: the stream must not go on while the CTAs still write
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (c0 == c1) return;  // written by its CTA
  {
    for (int c = c0 + part; c <= c1; c += kParts) {
      const long long pi = ((long long)c * 2 + (c == c0 ? 1 : 0)) * a.tile_cols + cc;
      const float2 v = *reinterpret_cast<const float2*>(a.part_ml + 2 * pi);
      const float4 y = *reinterpret_cast<const float4*>(a.part_o + pi * D + 4 * j);
      const float mn = fmaxf(mx, v.x);
      const float f = mx == mn ? 1.f : exp2f(mx - mn), e = v.x == mn ? 1.f : exp2f(v.x - mn);
      mx = mn;
      sum = sum * f + v.y * e;
      x.x = x.x * f + y.x * e;
      x.y = x.y * f + y.y * e;
      x.z = x.z * f + y.z * e;
      x.w = x.w * f + y.w * e;
    }
  }
  so[part][j] = x;
  if (j == 0) sml[part] = make_float2(mx, sum);
  __syncthreads();
  if (part) return;
  float M = -INFINITY;
#pragma unroll
  for (int i = 0; i < kParts; ++i) M = fmaxf(M, sml[i].x);
  sum = 0.f;
  float r[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    const float f = sml[i].x == M ? 1.f : exp2f(sml[i].x - M);
    sum = fmaf(sml[i].y, f, sum);
    r[0] = fmaf(so[i][j].x, f, r[0]);
    r[1] = fmaf(so[i][j].y, f, r[1]);
    r[2] = fmaf(so[i][j].z, f, r[2]);
    r[3] = fmaf(so[i][j].w, f, r[3]);
  }
  const long long row = (((long long)b * a.pg.H + h) * a.G + gg) * a.pg.T + tt;
  if (!row_live(u, tt)) sum = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = sum == 0.f ? 0.f : r[i] / sum;
  if (a.out_f32)
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * D + 4 * j) = make_float4(r[0], r[1], r[2], r[3]);
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * D + 4 * j) =
        make_uint2(tc::pack_bf16x2(r[0], r[1]), tc::pack_bf16x2(r[2], r[3]));
  if (j == 0) a.lse[row] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace cache
}  // namespace lsh
