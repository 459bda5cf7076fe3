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
// their number per code decides.  Both products are mma.m16n8k32 of 8-bit integers: a word's 8
// codes become bytes by two masks and at most one shift (16 codes as bf16 took 15 instructions,
// as bytes 6 for K and 8 for V, and one product covers twice the depth).
//   K: the query is a fixed-point number of 24 bits of the column's largest |q|.  The sums are
//      exact; the rounding of q is 2^-24 of its largest entry.  (16 bits would save a product in
//      three, but their rounding, the same for every key, moves the log-sum-exp by 1e-4.)
//   V: the weights p_j s_j of a stage's 64 keys are fixed-point numbers in steps of 2^(e - 22), 2^e the
//      power of two at or below the largest of them: 22 to 23 bits, as much as float products keep, and a weight
//      with a short mantissa (a lone key's is its scale) is exact.  (16 bits save a product in three; the
//      outputs were then off by 3e-4 of their size, so that one bf16 result in fifty was rounded to its
//      neighbour.)  The sums go into float accumulators after every stage.  A step for each
//      stage and not for the whole sequence: however many
//      small weights there are, what rounding takes from a stage is at most 64 half steps of its
//      own largest weight.  The upper nibbles stay where they are (16 c); their scale takes
//      the 16 out.  An accumulator that starts at 0x4B400000 is, read as a float, 1.5 * 2^23
//      plus the sum, so the integers become floats by one subtraction.
//
// A number's two upper bytes are two columns of the product (the third bytes of two fragments are a product more), so a
// fragment's 8 columns are 4 numbers: CW queries of each of TP = 4 / CW tiles, tile i's
// products using a B operand that is zero outside its own columns.  A single query thus
// fills all lanes: lane 4 g + t4 has keys g and g + 8 of tile t4, and scales, exponentials and
// weights are done once per key and not for 8 columns.  Slot t4 = i CW + c is a stream of its
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
// first and its last) and the join adds them up in order.  Where no item has more than 1024 keys,
// each has a CTA to itself and there is nothing to join (8 heads of 1021 keys: 9.0 us on the device and
// 17.5 us a call; with two kernels 8.3 us, but another launch and a workspace, 21 to 23 us a call).
//
// Measured on the device, one new token, bf16: 8 x 8 heads x 65536 keys of 128 (621 MB) 103 us, 6.0 TB/s, 92 %
// of the measured copy rate; 8 heads x 1 M keys of 64 (638 MB) 104 us, 6.1 TB/s, 93 %.  (In runs of a second, at the
// power cap's 1.65 GHz, 114.5 and 118.4 us: instructions weigh there too.)  Queries a cached head of
// the former: 2 107 us, 4 114 us, 8 161 us, 16 294 us: from 4 on
// the integer products and the unpacking (198 instructions a tile for one query, set-up and join included) bind.
// The ring is two stages of 64 tokens a warp and 8 warps an SM at D 128: one stage and 16 warps took as long
// there and 11 % more at D 64; three stages leave one CTA an SM (42 % more).
#pragma once

#include <type_traits>

#include "attend_tc.cuh"
#include "cache_common.cuh"
#include "cache_ring.cuh"
#include "tc_common.cuh"

namespace lsh {
namespace cache {

constexpr int kAttWarps = 4;
constexpr int kAttThreads = kAttWarps * 32;
constexpr int kMaxEntries = 256;     // pages looked up at a time
constexpr int kBlockTiles = 8;       // 128 tokens: what the work is dealt out in
constexpr float kLazyMax = 8.f;
constexpr float kPlainUnit = 0x1p-26f;  // of plain keys' scales: 2^-100 of them is still a normal number

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
  int direct;               // one CTA per item (short key lists): no pieces, no join
  int nc, n_ct, cols, tile_cols;  // CTAs; column tiles, all columns, columns of a tile
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

// A page looked up: its block of the item's head (null: missing) and its first position.
struct __align__(16) Entry {
  const uint8_t* src;
  int pos, pad;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
               : "memory");
}

// Bounded wait for a stage's copies: true for the whole warp or for none of it, as its lanes go on to shuffles and
// matrix products together.  (att_tc::warp_wait sleeps with a long hint: 2 % slower here, as copies are mostly there.)
__device__ __forceinline__ bool stage_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity))) return true;
  const unsigned long long t0 = tc::globaltimer();
  for (uint32_t i = 1;; ++i) {
    if (__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity))) return true;
    if ((i & 31u) == 0) {
      int bail = 0;
      if ((threadIdx.x & 31) == 0) {
        bail = *abort_flag;
        if (!bail && tc::globaltimer() - t0 > tc::kWaitNs) {
          *abort_flag = bail = 1;
          record_error(LSH_ERR_TIMEOUT);
        }
      }
      if (__shfl_sync(0xffffffffu, bail, 0)) return false;
    }
  }
}

// d = (first ? start : d) + codes (unsigned bytes) times signed (BS) or unsigned bytes.
template <bool BS>
__device__ __forceinline__ void imma16832(int (&d)[4], bool first, int start, uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  const int c0 = first ? start : d[0], c1 = first ? start : d[1], c2 = first ? start : d[2], c3 = first ? start : d[3];
  if (BS)
    asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(c0), "r"(c1), "r"(c2), "r"(c3));
  else
    asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.u8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(c0), "r"(c1), "r"(c2), "r"(c3));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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

// CW: queries of a tile in a fragment (1, 2 or 4); NT: fragments side by side (CW 4 only).
template <typename TQ, int D, int GROUP, int CW, int NT>
struct AttendCfg {
  using F = Fmt<D, GROUP>;
  static_assert(CW == 4 || NT == 1, "more than 4 queries go in whole fragments");
  static constexpr bool kF32 = sizeof(TQ) == 4;
  // products for the bytes of queries or weights: NT of (upper, lower) columns, then the third bytes of two
  // fragments as one
  static constexpr int kFrag = NT + (NT + 1) / 2;
  // a query's largest number: signed bytes, 127 in each
  static constexpr int kTop = 127 * 65536 + 127 * 256 + 127;
  static constexpr int kMt = D / 16;       // m tiles of V^T P^T
  static constexpr int kTp = 4 / CW;       // tiles of a fragment
  static constexpr int kSt = 4;            // tiles of a stage
  static constexpr int kSf = kSt / kTp;    // fragments of a stage
  static constexpr int kQ = CW * NT;       // query columns of a CTA
  static constexpr int kStreams = 4 * NT;  // of a warp
  static constexpr int kStages = 2;
  static constexpr int kStageBytes = kSt * F::kTile;
  static constexpr int kRing = kAttWarps * kStages * kStageBytes;
  static constexpr int kMerge = kAttWarps * kStreams * D * 4;
  static constexpr int kOffQ = (kRing > kMerge ? kRing : kMerge);
  static constexpr int kOffQs = kOffQ + kFrag * kTp * (D / 32) * 32 * 8;
  static constexpr int kOffMl = kOffQs + (kQ * (F::kGroups + 1) * 4 + 15) / 16 * 16;
  static constexpr int kOffEnt = kOffMl + kAttWarps * kStreams * 8;
  static_assert(kOffEnt % 16 == 0, "16-byte entries");
  static constexpr int kOffDesc = kOffEnt + kMaxEntries * 16;
  static constexpr int kOffBar = kOffDesc + kAttWarps * kStages * kSt * 4;
  static constexpr int kSmem = kOffBar + kAttWarps * kStages * 8;
  static_assert(kBlockTiles % kSt == 0, "blocks are whole stages");
  // CTAs of an SM: what registers allow (128 threads each) and what shared memory does
  static constexpr int kByRegs = D == 256 ? 2 : D == 64 ? 4 : 3;
  static constexpr int kBySmem = 227 * 1024 / (kSmem + 1024);
  static constexpr int kCtas = kByRegs < kBySmem ? kByRegs : kBySmem;
};

template <typename TQ, int D, int GROUP, int CW, int NT>
__global__ void __launch_bounds__(kAttThreads, AttendCfg<TQ, D, GROUP, CW, NT>::kCtas)
cache_attend_kernel(const __grid_constant__ AttendArgs a) {
  using C = AttendCfg<TQ, D, GROUP, CW, NT>;
  using F = Fmt<D, GROUP>;
  constexpr int NG = F::kGroups, MT = C::kMt, FQ = C::kFrag, TP = C::kTp, ST = C::kSt, SF = C::kSf;
  constexpr int kStages = C::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int abort_flag;
  uint4* qf = reinterpret_cast<uint4*>(smem + C::kOffQ);
  float* qs = reinterpret_cast<float*>(smem + C::kOffQs);
  float* qstep = qs + C::kQ * NG;
  float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);
  Entry* ent = reinterpret_cast<Entry*>(smem + C::kOffEnt);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  int4* descs = reinterpret_cast<int4*>(smem + C::kOffDesc);  // positions of a stage's tiles, -1: missing

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const bool sel = a.selected != nullptr;
  const int pl = a.pg.page_log2;
  uint8_t* ring = smem + warp * kStages * C::kStageBytes;
  uint64_t* bar = bars + warp * kStages;
  int4* desc = descs + warp * kStages;
  if (tid < kAttWarps * kStages) tc::mbar_init(bars + tid, 1);
  if (tid == 0) abort_flag = 0;
  tc::fence_mbar_init();
  int slot = 0;
  uint32_t phase = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // what ran before is done: lengths, pages, rows, workspace

  // ---- the CTA's stretch of the work -----------------------------------------------------------------
  long long before = 0, x = 0, x_end = 1;
  int b, own_item = 0;
  Seq u;
  if (a.direct) {
    const int unit = blockIdx.x / a.n_ct, ct = blockIdx.x - unit * a.n_ct;
    const int bh = sel ? unit / a.pg.T : unit, t = sel ? unit - bh * a.pg.T : 0;
    b = bh / a.pg.H;
    const int h = bh - b * a.pg.H;
    u = seq_of(a, b);
    if (u.n_rows == 0 || (sel && !row_live(u, t))) {  // padding: zeros
      const int col0 = ct * C::kQ, n = min(C::kQ, a.cols - col0);
      for (int i = tid; i < n * D; i += kAttThreads) {
        const int col = col0 + i / D, d = i % D;
        const int tt = sel ? t : col / a.G, gg = sel ? col : col - tt * a.G;
        const long long row = ((long long)bh * a.G + gg) * a.pg.T + tt;
        if (a.out_f32)
          static_cast<float*>(a.out)[row * D + d] = 0.f;
        else
          static_cast<__nv_bfloat16*>(a.out)[row * D + d] = __float2bfloat16_rn(0.f);
        if (d == 0) a.lse[row] = -INFINITY;
      }
      return;
    }
    own_item = (sel ? h * u.n_rows + t - u.row0 : h) * a.n_ct + ct;
  } else {
    // the join may be set up (it waits for this kernel's end before it reads): every CTA is resident
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    long long total;
    work_before(a, 0, lane, total, before);
    const long long nc = min((long long)a.nc, total);  // CTAs with work: a block each at least
    if (blockIdx.x >= nc) return;
    x = blockIdx.x * total / nc;
    x_end = (blockIdx.x + 1) * total / nc;
    b = work_find(a, x, lane, before);
    u = seq_of(a, b);
  }

  while (x < x_end) {
  int item = own_item, blk0 = 0, blk1 = u.nb;
  if (a.direct) {
    x = x_end;
  } else {
    while (x >= before + (long long)u.items * u.nb) {  // the next sequence with anything to do
      before += (long long)u.items * u.nb;
      u = seq_of(a, ++b);
    }
    item = (int)((x - before) / u.nb);
    blk0 = (int)((x - before) - (long long)item * u.nb);
    blk1 = (int)min((long long)u.nb, blk0 + (x_end - x));
    x += blk1 - blk0;
  }
  const int ct = item % a.n_ct, rest = item / a.n_ct;
  const int row_t = sel ? u.row0 + rest % u.n_rows : 0;  // the row, with selection
  const int h = sel ? rest / u.n_rows : rest;
  const int col0 = ct * C::kQ;
  const int tile_lo = blk0 * kBlockTiles;
  const int tile_hi = min(blk1 * kBlockTiles, (u.n_list + kTileTokens - 1) / kTileTokens);
  tc::fence_proxy_async_smem();  // (the last item's sums lay where copies go now)
  __syncthreads();

  const int32_t* picks = sel ? a.selected + (((long long)b * a.pg.H + h) * a.pg.T + row_t) * a.n_select : nullptr;
  // ---- pages and copies: first of all, so that the first copies run under the rest of the set-up --------
  int tile0 = tile_lo, tile1 = tile_lo, e0 = 0;  // the tiles whose pages are looked up, in list order
  auto look_up = [&]() {  // the next ones, as many pages as are held at a time (table and, with selection, list)
    tile0 = tile1;
    e0 = (tile0 << 4) >> pl;
    tile1 = (int)min((long long)tile_hi, ((long long)(e0 + kMaxEntries) << pl) >> 4);
    const int n_ent = (((tile1 - 1) << 4) >> pl) - e0 + 1;
    for (int i = tid; i < n_ent; i += kAttThreads) {
      int logical = e0 + i;
      if (sel) logical = picks[e0 + i];
      int phys = -1;
      if (logical >= 0 && logical < a.pg.max_pages && ((long long)logical << pl) < u.ctx) phys = page_of(a.pg, b, logical);
      Entry e;
      e.src = phys >= 0 ? a.cache + tile_offset(a.pg, phys, h, 0, F::kTile) : nullptr;
      e.pos = logical << pl;
      e.pad = 0;
      ent[i] = e;
    }
  };
  auto issue = [&](int st, int slot) {  // lane 0: copies of stage st
    const int tile = tile0 + st * ST;
    const uint32_t dst = tc::smem_u32(ring + slot * C::kStageBytes);
    if (pl >= 6) {  // a stage lies inside a page
      const Entry e = ent[((tile << 4) >> pl) - e0];
      const int in_page = tile & ((1 << (pl - 4)) - 1);
      const int p = e.pos + (in_page << 4);
      // tiles that hold tokens of the sequence (in list order the sequence may end before the list)
      const int n = e.src ? min(min(ST, tile1 - tile), max(0, (u.ctx - p + kTileTokens - 1) >> 4)) : 0;
      desc[slot] = make_int4(n > 0 ? p : -1, n > 1 ? p + 16 : -1, n > 2 ? p + 32 : -1, n > 3 ? p + 48 : -1);
      tc::mbar_arrive_expect_tx(bar + slot, n * F::kTile);
      if (n > 0) bulk_load(dst, e.src + in_page * F::kTile, n * F::kTile, bar + slot);
      return;
    }
    const uint8_t* src[ST];
    int first[ST];
    uint32_t bytes = 0;
#pragma unroll
    for (int k = 0; k < ST; ++k) {
      src[k] = nullptr;
      first[k] = -1;
      if (tile + k < tile1) {
        const Entry e = ent[(((tile + k) << 4) >> pl) - e0];
        const int in_page = (tile + k) & ((1 << (pl - 4)) - 1);
        const int p = e.pos + (in_page << 4);
        if (e.src && p < u.ctx) {
          src[k] = e.src + in_page * F::kTile;
          first[k] = p;
          bytes += F::kTile;
        }
      }
    }
    desc[slot] = make_int4(first[0], first[1], first[2], first[3]);
    tc::mbar_arrive_expect_tx(bar + slot, bytes);
#pragma unroll
    for (int k = 0; k < ST; ++k)
      if (src[k]) bulk_load(dst + k * F::kTile, src[k], F::kTile, bar + slot);
  };
  auto start = [&]() {  // the warp's first copies
    const int n_stage = (tile1 - tile0 + ST - 1) / ST;
    if (lane == 0)
      for (int i = 0, s2 = slot; i < kStages; ++i) {
        if (warp + i * kAttWarps < n_stage) issue(warp + i * kAttWarps, s2);
        s2 = s2 + 1 == kStages ? 0 : s2 + 1;
      }
    __syncwarp();
  };

  // ---- set-up of the item: query operands and sums -----------------------------------------------------
  look_up();
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
  start();
  // B operands of K's products: columns 2 k, 2 k + 1 of a fragment are the upper and lower byte (behind
  // those, of fragments nt and nt + 1 the third byte) of slot k = i CW + c, that is of query column c for tile i,
  // and zero for the other tiles; word w covers dims 32 w .. 32 w + 31.  Bytes are signed, so a lower
  // byte is -128..127 and the rest is rounded to it.
  for (int i = tid; i < NT * (D / 32) * 32; i += kAttThreads) {
    const int l = i & 31, w = (i >> 5) % (D / 32), nt = (i >> 5) / (D / 32);
    const int k = l >> 3, cc = nt * CW + k % CW, col = col0 + cc;
    const bool lower = (l >> 2) & 1;
    const float step = qstep[cc];
    const float inv = step > 0.f ? 1.f / step : 0.f;
    const bool third = lower == (nt & 1);  // this lane's column of the third bytes
    uint32_t v[2][2] = {{0u, 0u}, {0u, 0u}};
    if (col < a.cols) {
      const TQ* q = q_row(col) + 32 * w + 2 * (l & 3);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x = to_f32<TQ>(q[8 * j + e]);
          // x / step; a step too small to invert (denormal queries) is divided by
          const float y = inv < INFINITY ? x * inv : x / step;
          int f = max(-C::kTop, min(C::kTop, __float2int_rn(y)));
          const int b0 = (int8_t)f;  // the third byte
          if (third) v[1][e] |= (uint32_t)(b0 & 255) << (8 * j);
          f = (f - b0) >> 8;
          const int b1 = (int8_t)f, b2 = (f - b1) >> 8;
          v[0][e] |= (uint32_t)((lower ? b1 : b2) & 255) << (8 * j);
        }
    }
    auto put = [&](int frag, const uint32_t (&u)[2]) {
#pragma unroll
      for (int t = 0; t < TP; ++t)
        reinterpret_cast<uint2*>(qf + ((frag * TP + t) * (D / 64) + (w >> 1)) * 32 + l)[w & 1] =
            k / CW == t ? make_uint2(u[0], u[1]) : make_uint2(0u, 0u);
    };
    put(nt, v[0]);
    if (third || (nt % 2 == 0 && nt + 1 == NT)) put(NT + nt / 2, v[1]);  // (an unpaired column: zero)
  }
  __syncthreads();

  // ---- the lane's streams: slot t4 of each fragment -----------------------------------------------------
  const int my_tile = t4 / CW;  // the tile of a fragment that it belongs to
  int pos[NT], last[NT];        // position; largest admissible position
  bool self[NT];                // whether its own key is masked
  int fast = u.ctx;             // tiles that end at or below are admissible to every column
  float qsum[NT][NG], step[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int cc = nt * CW + t4 % CW, col = col0 + cc;
    const int tt = sel ? row_t : col / a.G;
    const bool live = col < a.cols && row_live(u, tt);
    pos[nt] = live ? u.start + tt : -1;
    last[nt] = !live ? -1 : (a.causal ? pos[nt] : u.ctx - 1);
    self[nt] = live && a.self_mask;
    if (live && a.self_mask) {
      // its own key counts when nothing else is admissible
      bool other;
      if (!sel) {
        other = last[nt] > 0;
      } else {
        other = false;
        for (int i = 0; i < a.n_select && !other; ++i) {
          const int lp = picks[i];
          if (lp < 0 || lp >= a.pg.max_pages) continue;
          const long long f = (long long)lp << pl;
          const long long e = min((long long)last[nt], f + (1 << pl) - 1);  // last admissible of the page
          other = f <= e && (e > f || f != pos[nt]);
        }
      }
      self[nt] = other;
    }
    if (live && (a.causal || a.self_mask)) fast = min(fast, pos[nt]);
    step[nt] = a.unit_keys ? qstep[cc] : qstep[cc] * (1.f / kPlainUnit);
#pragma unroll
    for (int n = 0; n < NG; ++n) qsum[nt][n] = qs[cc * NG + n];
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) fast = min(fast, __shfl_xor_sync(0xffffffffu, fast, o));

  float m[NT], base[NT], bar_m[NT], l[NT];  // maximum; what is subtracted; where it has to move; sum
  float o[NT][MT][2], zs[NT][NG];           // dims 16 i + g, + 8; sums of p z
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt] = bar_m[nt] = -INFINITY;
    base[nt] = l[nt] = 0.f;
#pragma unroll
    for (int i = 0; i < MT; ++i) o[nt][i][0] = o[nt][i][1] = 0.f;
#pragma unroll
    for (int n = 0; n < NG; ++n) zs[nt][n] = 0.f;
  }

  // One stage of ST tiles.  MASKED: a tile may be missing, and every key is tested against the columns.
  auto consume = [&](const uint8_t* buf, const int* first, auto masked_c) {  // first: positions, in shared memory
    constexpr bool MASKED = decltype(masked_c)::value;
    // ---- logits of keys g and g + 8 of the lane's tile
    float s[SF][NT][2];
#pragma unroll
    for (int f = 0; f < SF; ++f) {
      int part[FQ][NG][4];
#pragma unroll
      for (int i = 0; i < TP; ++i) {
        const uint8_t* tb = buf + (f * TP + i) * F::kTile;  // (a missing tile's sums are replaced below)
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
          for (int p = 0; p < FQ; ++p) {
            const uint4 q = qf[((p * TP + i) * (D / 64) + w / 2) * 32 + lane];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int n = (w + e) * 32 / GROUP;
              const bool fresh = i == 0 && (w + e) * 32 % GROUP == 0;
              imma16832<true>(part[p][n], fresh, 0, y[e][0], y[e][1], y[e][2], y[e][3], e ? q.z : q.x, e ? q.w : q.y);
            }
          }
        }
      }
      const int mine = f * TP + my_tile;
      const int first_mine = MASKED ? first[mine] : 0;
      const uint8_t* tb = buf + mine * F::kTile;
      const uint32_t* kp = reinterpret_cast<const uint32_t*>(tb + F::kOffKp);
      float acc[NT][2], zero[NT][2];  // sum of s (codes . q) in steps of q, and of z (sum of q)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = zero[nt][0] = zero[nt][1] = 0.f;
      // The key's length goes into s and z, which leaves them below 1 whatever the row's size; of plain keys s is taken
      // in units that leave room for a sum of codes and queries, up to 2^36 (step has the factor back).
      float ks[2] = {kPlainUnit, kPlainUnit}, kz[2] = {1.f, 1.f};
      if (a.unit_keys) {
        ks[0] = kz[0] = reinterpret_cast<const float*>(tb + F::kOffInv)[g];
        ks[1] = kz[1] = reinterpret_cast<const float*>(tb + F::kOffInv)[g + 8];
      }
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t pw = kp[n * 16 + g + 8 * r];
          const float sc = bf16_bits(pw) * ks[r], ze = __uint_as_float(pw & 0xffff0000u) * kz[r];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            // at most 64 * 15 * 2^15; the third byte joins in float
            float v = (float)(part[nt][n][2 * r] * 256 + part[nt][n][2 * r + 1]);
            v = fmaf(v, 256.f, (float)part[NT + nt / 2][n][2 * r + nt % 2]);
            acc[nt][r] = fmaf(sc, v, acc[nt][r]);
            zero[nt][r] = fmaf(ze, qsum[nt][n], zero[nt][r]);
          }
        }
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float x = fmaf(acc[nt][r], step[nt], zero[nt][r]) * a.scale_log2;
          if (MASKED) {
            const int key = first_mine + g + 8 * r;
            if (first_mine < 0 || key > last[nt] || (key == pos[nt] && self[nt])) x = -INFINITY;
          }
          s[f][nt][r] = x;
        }
    }
    // ---- the running maximum, moved only when a logit is 2^8 above it
    float top[NT];
    bool raise = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x = fmaxf(s[0][nt][0], s[0][nt][1]);
#pragma unroll
      for (int f = 1; f < SF; ++f) x = fmaxf(fmaxf(x, s[f][nt][0]), s[f][nt][1]);
      top[nt] = x;
      raise |= x > bar_m[nt];
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x = top[nt];
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        const float mn = fmaxf(m[nt], x);
        const float al = m[nt] == mn ? 1.f : exp2f(m[nt] - mn);
        m[nt] = mn;
        base[nt] = mn == -INFINITY ? 0.f : mn;
        bar_m[nt] = mn == -INFINITY ? mn : mn + kLazyMax;
        l[nt] *= al;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          o[nt][i][0] *= al;
          o[nt][i][1] *= al;
        }
#pragma unroll
        for (int n = 0; n < NG; ++n) zs[nt][n] *= al;
      }
    }
    // ---- weights p, and what they take from the zeros
    float p[SF][NT][2];
#pragma unroll
    for (int f = 0; f < SF; ++f)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float y = s[f][nt][r] - base[nt];
          p[f][nt][r] = C::kF32 ? exp2f(y) : tc::ex2_approx(y);
          l[nt] += p[f][nt][r];
        }
    // ---- O += weights . codes, 64 dims at a time: p s of their groups, the largest of the stage, fixed-point
    // numbers of it, then 16 dims of 64 keys in a product
    constexpr int NQ = 64 / GROUP;  // groups of 64 dims
#pragma unroll
    for (int q = 0; q < D / 64; ++q) {
      float unit[NT][NQ];              // what a step of the weights is worth
      uint32_t pb[SF][NQ][FQ];         // their bytes in column g: keys 2 t4, +1, 2 t4 + 8, +9 of the column's tile
#pragma unroll
      for (int u = 0; u < NQ; ++u) {
        const int n = q * NQ + u;
        float wt[SF][NT][2];
        uint32_t top_w[NT];  // bits of a float that is not negative order as integers do, NaN above all
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) top_w[nt] = 0u;
#pragma unroll
        for (int f = 0; f < SF; ++f) {
          const uint32_t* vp = reinterpret_cast<const uint32_t*>(buf + (f * TP + my_tile) * F::kTile + F::kOffVp);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t pw = vp[n * 16 + g + 8 * r];
            const float sc = bf16_bits(pw), ze = __uint_as_float(pw & 0xffff0000u);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const bool out = MASKED && s[f][nt][r] == -INFINITY;  // whatever lies in a masked place
              const float w = out ? 0.f : p[f][nt][r] * sc;
              if (!out) zs[nt][n] = fmaf(p[f][nt][r], ze, zs[nt][n]);
              wt[f][nt][r] = w;
              top_w[nt] = max(top_w[nt], __float_as_uint(w));
            }
          }
        }
        float inv[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t t = top_w[nt];
          t = max(t, __shfl_xor_sync(0xffffffffu, t, 4));
          t = max(t, __shfl_xor_sync(0xffffffffu, t, 8));
          t = max(t, __shfl_xor_sync(0xffffffffu, t, 16));
          // with 2^e the power of two at or below the largest, 2^-105 at least: a step is 2^(e - 22), so numbers end at
          // 2^23; unit is the step times 2^16, and NaN where the largest is NaN or infinite
          const uint32_t e = max(t & 0x7f800000u, 22u << 23);
          inv[nt] = __uint_as_float((276u << 23) - e);
          unit[nt][u] = __uint_as_float(e == 0x7f800000u ? 0x7fffffffu : e - (6u << 23));
        }
#pragma unroll
        for (int f = 0; f < SF; ++f) {
          uint32_t x[NT][2];  // the number in the low bits of a float's mantissa (2^23 itself, as 0x4B800000, too)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r) x[nt][r] = __float_as_uint(fmaf(wt[f][nt][r], inv[nt], 8388608.f));
          // its bytes as columns: the upper two as those of its slot, the lowest beside another fragment's.  (What
          // stands in the odd bytes goes no further.)
          auto column = [&](uint32_t lo, uint32_t hi) { return __byte_perm(movmatrix(lo), movmatrix(hi), 0x6420); };
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            pb[f][u][nt] = column(__byte_perm(x[nt][0], 0u, 0x4142), __byte_perm(x[nt][1], 0u, 0x4142));
#pragma unroll
          for (int nt = 0; nt < NT; nt += 2) {
            const bool pair = nt + 1 < NT;
            const uint32_t(&y)[2] = x[nt + pair];
            pb[f][u][NT + nt / 2] = column(__byte_perm(x[nt][0], pair ? y[0] : 0u, 0x4400),
                                           __byte_perm(x[nt][1], pair ? y[1] : 0u, 0x4400));
          }
        }
      }
      uint32_t by[ST][4];  // byte j of the four keys of a lane: dims 16 j + g (low nibble), 16 j + 8 + g
#pragma unroll
      for (int k = 0; k < ST; ++k) {
        const uint8_t* vrow = buf + k * F::kTile + F::kOffV + t4 * D + (g ^ (2 * t4)) * (D / 8) + 8 * q;
        const uint2 u0 = *reinterpret_cast<const uint2*>(vrow), u1 = *reinterpret_cast<const uint2*>(vrow + 4 * D);
        const uint32_t a01 = __byte_perm(u0.x, u0.y, 0x5140), b01 = __byte_perm(u1.x, u1.y, 0x5140);
        const uint32_t a23 = __byte_perm(u0.x, u0.y, 0x7362), b23 = __byte_perm(u1.x, u1.y, 0x7362);
        by[k][0] = __byte_perm(a01, b01, 0x5410);
        by[k][1] = __byte_perm(a01, b01, 0x7632);
        by[k][2] = __byte_perm(a23, b23, 0x5410);
        by[k][3] = __byte_perm(a23, b23, 0x7632);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int mt = 4 * q + j, u = j * 16 / GROUP;
        int sum[FQ][4];
#pragma unroll
        for (int k = 0; k < ST; k += 2) {  // two tiles: the depth of a product
          const uint32_t a0 = by[k][j] & 0x0f0f0f0fu, a1 = by[k][j] & 0xf0f0f0f0u;
          const uint32_t a2 = by[k + 1][j] & 0x0f0f0f0fu, a3 = by[k + 1][j] & 0xf0f0f0f0u;
#pragma unroll
          for (int e = 0; e < FQ; ++e) {
            // a tile's own columns only
            const uint32_t b0 = TP == 1 || (g >> 1) / CW == k % TP ? pb[k / TP][u][e] : 0u;
            const uint32_t b1 = TP == 1 || (g >> 1) / CW == (k + 1) % TP ? pb[(k + 1) / TP][u][e] : 0u;
            imma16832<false>(sum[e], k == 0, 0x4B400000, a0, a1, a2, a3, b0, b1);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float v = fmaf(__int_as_float(sum[NT + nt / 2][2 * r + nt % 2]) - 12582912.f, 1.f / 256.f,
                           __int_as_float(sum[nt][2 * r + 1]) - 12582912.f);
            v = fmaf(v, 1.f / 256.f, __int_as_float(sum[nt][2 * r]) - 12582912.f);
            o[nt][mt][r] = fmaf(v, unit[nt][u] * (r ? 0.0625f : 1.f), o[nt][mt][r]);  // upper nibbles: 16 c
          }
      }
    }
  };

  bool ok = true;  // whether every wait of this warp ended in time
  for (;;) {
    ok = run_stages<kStages, kAttWarps>(
        warp, (tile1 - tile0 + ST - 1) / ST, slot, phase,
        [&](int s, uint32_t parity) { return stage_wait(bar + s, parity, &abort_flag); },
        [&](int s, uint32_t parity) { att_tc::drain_wait(bar + s, parity); },
        [&](int, int s) {
          const int4 at = desc[s];
          const int* first = reinterpret_cast<const int*>(desc + s);
          const int lo = min(min(at.x, at.y), min(at.z, at.w)), hi = max(max(at.x, at.y), max(at.z, at.w));
          const uint8_t* buf = ring + s * C::kStageBytes;
          if (lo >= 0 && hi + kTileTokens <= fast)
            consume(buf, first, std::false_type());
          else if (hi >= 0)
            consume(buf, first, std::true_type());
          __syncwarp();
        },
        [&](int st, int s) {
          if (lane == 0) issue(st, s);
        });
    if (tile1 >= tile_hi) break;
    if (__syncthreads_or(!ok)) return;  // a wait gave up (the status word says so): every warp leaves
    look_up();
    __syncthreads();
    start();
  }

  // ---- join the warps -----------------------------------------------------------------------------
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int y = 4; y < 32; y <<= 1) {
      l[nt] += __shfl_xor_sync(0xffffffffu, l[nt], y);
#pragma unroll
      for (int n = 0; n < NG; ++n) zs[nt][n] += __shfl_xor_sync(0xffffffffu, zs[nt][n], y);
    }
    if (g == 0) ml[warp * C::kStreams + nt * 4 + t4] = make_float2(m[nt], l[nt]);
  }
  if (__syncthreads_or(!ok)) return;  // (else the ring is free)
  float* om = reinterpret_cast<float*>(smem);  // [warp][stream][D]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        om[(warp * C::kStreams + nt * 4 + t4) * D + i * 16 + g + 8 * r] = o[nt][i][r] + zs[nt][i * 16 / GROUP];
  __syncthreads();
  for (int i = tid; i < C::kQ * D; i += kAttThreads) {
    const int cc = i / D, d = i - cc * D, col = col0 + cc;
    if (col >= a.cols) break;
    // its streams: slot cc of every warp, and CW further for each other tile of a fragment
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kAttWarps * TP; ++w) mx = fmaxf(mx, ml[w / TP * C::kStreams + cc + w % TP * CW].x);
    float sum = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kAttWarps * TP; ++w) {
      const int j = w / TP * C::kStreams + cc + w % TP * CW;
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
constexpr int kJoinThreads = 512;

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
#pragma unroll 4
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
#pragma unroll 8
  for (int i = 0; i < kParts; ++i) M = fmaxf(M, sml[i].x);
  sum = 0.f;
  float r[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
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
