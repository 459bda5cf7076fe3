// C entry points of the 4-bit cache: argument checks, launch plans, dispatch.
// Included at the end of lsh_api.cu (one translation unit).
#pragma once

#include "cache_attend.cuh"
#include "cache_rw.cuh"
#include "cache_select.cuh"

namespace {

// Form of a cache: what every entry point checks first.
inline lsh_status check_cache_form(int H, int D, int page, int group, int n_pages, int B, int max_pages) {
  if (B < 0 || H < 0 || n_pages < 0 || max_pages < 0) return LSH_ERR_SHAPE;
  if (D < 8 || D > 256 || (D % 8) != 0) return LSH_ERR_SHAPE;
  if (page < 16 || page > 256 || (page & (page - 1)) != 0) return LSH_ERR_SHAPE;
  if (group < 8 || group > D || D % group != 0) return LSH_ERR_SHAPE;
  if ((long long)max_pages * page > (1ll << 30)) return LSH_ERR_SHAPE;
  if ((D != 64 && D != 128 && D != 256) || (group != 32 && group != 64)) return LSH_ERR_UNSUPPORTED;
  return LSH_OK;
}

// Whether a product of sizes (not negative, so at most 2^124) is below 2^31, the reach of rows and columns.
inline bool fits_31_bits(int a, int b, int c, int d = 1) { return (__int128)a * b * c * d < ((__int128)1 << 31); }

inline int log2_of(int p) {
  int l = 0;
  while ((1 << l) < p) ++l;
  return l;
}

inline lsh::cache::Pages pages_of(const int32_t* table, const int32_t* ctx_len, const int32_t* new_len, int max_pages,
                                  int page, int n_pages, int H, int T) {
  lsh::cache::Pages p;
  p.table = table;
  p.ctx_len = ctx_len;
  p.new_len = new_len;
  p.max_pages = max_pages;
  p.page_log2 = log2_of(page);
  p.n_pages = n_pages;
  p.H = H;
  p.T = T;
  p.div_t = lsh::cache::FastDiv::by((uint32_t)T);
  p.div_h = lsh::cache::FastDiv::by((uint32_t)H);
  return p;
}

// Calls f(integral_constant D, integral_constant GROUP) for a form check_cache_form accepts.
template <typename Fn>
lsh_status cache_form_dispatch(int D, int group, Fn f) {
#define LSH_CF(DD, GG) \
  if (D == DD && group == GG) return f(std::integral_constant<int, DD>(), std::integral_constant<int, GG>())
  LSH_CF(64, 32);
  LSH_CF(64, 64);
  LSH_CF(128, 32);
  LSH_CF(128, 64);
  LSH_CF(256, 32);
  LSH_CF(256, 64);
#undef LSH_CF
  return LSH_ERR_UNSUPPORTED;
}

// How an attention call is cut: query columns per cached head in tiles of cw * nt, the work over
// at most max_ctas CTAs (what the kernel's registers and shared memory allow may be fewer).
struct AttendPlan {
  long long units, blocks;  // (cached head [, row]) of all sequences; blocks of all items with full tables
  int cols, cw, nt, n_ct, max_ctas;
  bool direct;  // one CTA per item, no workspace
};

constexpr int kMaxCtasPerSm = 6;

inline AttendPlan attend_plan(int B, int H, int G, int T, int D, int max_pages, int page, int n_select) {
  AttendPlan p;
  const bool sel = n_select > 0;
  p.units = (long long)B * H * (sel ? T : 1);
  p.cols = sel ? G : G * T;
  // one or two columns: four or two tiles share a fragment; beyond four, two fragments side by side, so that a
  // cached token is unpacked once for up to 8 columns.  16 queries of 64 heads of 64K, D 128: 305 us so, 309 us with
  // four fragments, whose sums do not fit the registers.  At D 256 two do not either (8 queries of 32 heads
  // of 64K: 297 us, with one 285 us).
  const int most = D == 256 ? 1 : 2;
  p.cw = p.cols >= 3 ? 4 : p.cols == 2 ? 2 : 1;
  p.nt = p.cols <= 4 ? 1 : most;
  const long long keys = (long long)(sel ? n_select : max_pages) * page;
  p.direct = keys <= 1024;
  const int block = lsh::cache::kBlockTiles * lsh::cache::kTileTokens;
  const int sms = dev_info().sms > 0 ? dev_info().sms : 148;
  p.n_ct = (p.cols + p.cw * p.nt - 1) / (p.cw * p.nt);
  p.blocks = p.units * p.n_ct * ((keys + block - 1) / block);
  p.max_ctas = (int)std::max<long long>(1, std::min<long long>(p.blocks, (long long)sms * kMaxCtasPerSm));
  return p;
}

// Two pieces per CTA: unnormalised outputs, then (maximum, sum).
inline size_t attend_plan_bytes(const AttendPlan& p, int D) {
  if (p.direct) return 0;
  const size_t n = (size_t)p.max_ctas * 2 * p.cw * p.nt;
  return n * D * sizeof(float) + n * 2 * sizeof(float);
}

// Sets a kernel's dynamic shared memory limit once per device (the call costs as much as a launch).
inline lsh_status allow_smem(const void* fn, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return LSH_ERR_CUDA;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (bit && (done.load(std::memory_order_relaxed) & bit)) return LSH_OK;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
    cudaGetLastError();  // (reported here, not by whatever launches next)
    return LSH_ERR_CUDA;
  }
  done.fetch_or(bit, std::memory_order_relaxed);
  return LSH_OK;
}

// Launches a kernel that may be set up before the one ahead of it on the stream has ended: it executes
// griddepcontrol.wait before it reads or writes anything that others do.
template <typename Args>
lsh_status launch_early(void (*fn)(Args), unsigned grid, int threads, int smem, cudaStream_t s,
                        const std::remove_const_t<Args>& args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, fn, args) == cudaSuccess) return LSH_OK;
  cudaGetLastError();  // (reported here, not by whatever launches next)
  return LSH_ERR_CUDA;
}

template <typename TQ, int D, int GROUP, int CW, int NT>
lsh_status launch_cache_attend(lsh::cache::AttendArgs& a, const AttendPlan& p, cudaStream_t s) {
  using namespace lsh::cache;
  using C = AttendCfg<TQ, D, GROUP, CW, NT>;
  auto kfn = cache_attend_kernel<TQ, D, GROUP, CW, NT>;
  static std::atomic<uint64_t> done{0};
  const lsh_status st = allow_smem((const void*)kfn, C::kSmem, done);
  if (st != LSH_OK) return st;
  static_assert(C::kCtas >= 1 && C::kCtas <= kMaxCtasPerSm, "workspace is sized for it");
  const int sms = dev_info().sms > 0 ? dev_info().sms : 148;
  a.direct = p.direct;
  a.nc = p.direct ? (int)(p.units * p.n_ct) : std::min(p.max_ctas, sms * C::kCtas);
  const lsh_status run = launch_early(kfn, (unsigned)a.nc, kAttThreads, C::kSmem, s, a);
  if (run != LSH_OK || p.direct) return run;
  // set up while the last CTAs run; it waits for them before it reads
  return launch_early(cache_join_kernel<D>, (unsigned)(p.units * p.cols), kJoinThreads, 0, s, a);
}

}  // namespace

extern "C" {

size_t lsh_cache_block_bytes(int page, int D, int group) {
  if (check_cache_form(1, D, page, group, 1, 1, 1) != LSH_OK) return 0;
  return (size_t)(page / 16) * lsh::cache::tile_bytes(D, group);
}

lsh_status lsh_cache_write(const void* k, const void* v, int dtype, int B, int H, int T, int D,
                           const int32_t* buckets, int n_rounds, const int32_t* ctx_len, const int32_t* new_len,
                           const int32_t* page_table, int max_pages, int page, int group, void* cache, int n_pages,
                           uint16_t* tags, void* stream) {
  if (!valid_dtype(dtype)) return LSH_ERR_DTYPE;
  const lsh_status st = check_cache_form(H, D, page, group, n_pages, B, max_pages);
  if (st != LSH_OK) return st;
  if (T < 0 || !fits_31_bits(B, H, T)) return LSH_ERR_SHAPE;
  if ((buckets == nullptr) != (tags == nullptr)) return LSH_ERR_INVALID_ARG;
  if (tags && (n_rounds < 1 || n_rounds > 64)) return LSH_ERR_SHAPE;
  if (!k || !v || !ctx_len || !page_table || !cache) return LSH_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(ctx_len) || !aligned16(page_table) || !aligned16(cache) ||
      (new_len && !aligned16(new_len)) || (tags && (!aligned16(tags) || !aligned16(buckets))))
    return LSH_ERR_ALIGN;
  lsh::cache::WriteArgs a;
  a.k = k;
  a.v = v;
  a.buckets = buckets;
  a.cache = static_cast<uint8_t*>(cache);
  a.tags = tags;
  a.rows = (unsigned)B * H * T;
  a.n_rounds = n_rounds;
  a.sixteen = 16;
  a.wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31u) == 0;
  a.pg = pages_of(page_table, ctx_len, new_len, max_pages, page, n_pages, H, T);
  if (a.rows == 0 || max_pages == 0) return LSH_OK;
  cudaStream_t s = as_stream(stream);
  return cache_form_dispatch(D, group, [&](auto DC, auto GC) {
    constexpr int DD = decltype(DC)::value, GG = decltype(GC)::value;
    const unsigned per = lsh::cache::kRwThreads / (DD / 16);  // rows of a CTA
    const unsigned grid = (a.rows + per - 1) / per;
    if (dtype == LSH_F32)
      lsh::cache::cache_write_kernel<float, DD, GG><<<grid, lsh::cache::kRwThreads, 0, s>>>(a);
    else
      lsh::cache::cache_write_kernel<__nv_bfloat16, DD, GG><<<grid, lsh::cache::kRwThreads, 0, s>>>(a);
    return launch_status();
  });
}

lsh_status lsh_cache_read(const void* cache, int n_pages, int B, int H, int T, int D, const int32_t* ctx_len,
                          const int32_t* new_len, const int32_t* page_table, int max_pages, int page, int group,
                          void* k, void* v, int out_dtype, float* key_inv, void* stream) {
  if (!valid_dtype(out_dtype)) return LSH_ERR_DTYPE;
  const lsh_status st = check_cache_form(H, D, page, group, n_pages, B, max_pages);
  if (st != LSH_OK) return st;
  if (T < 0 || !fits_31_bits(B, H, T)) return LSH_ERR_SHAPE;
  if (!k || !v || !ctx_len || !page_table || !cache) return LSH_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(ctx_len) || !aligned16(page_table) || !aligned16(cache) ||
      (new_len && !aligned16(new_len)) || (key_inv && !aligned16(key_inv)))
    return LSH_ERR_ALIGN;
  lsh::cache::ReadArgs a;
  a.cache = static_cast<const uint8_t*>(cache);
  a.k = k;
  a.v = v;
  a.inv = key_inv;
  a.wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31u) == 0;
  a.rows = (unsigned)B * H * T;
  a.pg = pages_of(page_table, ctx_len, new_len, max_pages, page, n_pages, H, T);
  if (a.rows == 0) return LSH_OK;
  cudaStream_t s = as_stream(stream);
  return cache_form_dispatch(D, group, [&](auto DC, auto GC) {
    constexpr int DD = decltype(DC)::value, GG = decltype(GC)::value;
    const unsigned per = lsh::cache::kRwThreads / (DD / 16);  // rows of a CTA
    const unsigned grid = (a.rows + per - 1) / per;
    if (out_dtype == LSH_F32)
      lsh::cache::cache_read_kernel<float, DD, GG><<<grid, lsh::cache::kRwThreads, 0, s>>>(a);
    else
      lsh::cache::cache_read_kernel<__nv_bfloat16, DD, GG><<<grid, lsh::cache::kRwThreads, 0, s>>>(a);
    return launch_status();
  });
}

lsh_status lsh_cache_select(const uint16_t* tags, int n_pages, const int32_t* q_buckets, int B, int Hq, int H, int T,
                            int n_rounds, const int32_t* ctx_len, const int32_t* new_len, const int32_t* page_table,
                            int max_pages, int page, int n_select, int n_local, int mask, int32_t* selected,
                            int32_t* scores, void* stream) {
  const lsh_status st = check_cache_form(H, 128, page, 64, n_pages, B, max_pages);
  if (st != LSH_OK) return st;
  if (T < 0 || Hq < 0 || (H == 0 ? Hq != 0 : (Hq % H != 0 || Hq == 0))) return LSH_ERR_SHAPE;
  if (n_rounds < 1 || n_rounds > 64 || n_select < 1 || n_local < 0 || n_local > n_select) return LSH_ERR_SHAPE;
  if ((long long)n_select * page > (1ll << 30)) return LSH_ERR_SHAPE;
  if (!fits_31_bits(B, H, T, n_select) || !fits_31_bits(B, H, T, std::max(1, max_pages)) ||
      !fits_31_bits(B, Hq, n_rounds, T))
    return LSH_ERR_SHAPE;
  if (mask & ~LSH_MASK_CAUSAL) return LSH_ERR_INVALID_ARG;
  if (!tags || !q_buckets || !ctx_len || !page_table || !selected || !scores) return LSH_ERR_INVALID_ARG;
  if (!aligned16(tags) || !aligned16(q_buckets) || !aligned16(ctx_len) || !aligned16(page_table) ||
      !aligned16(selected) || !aligned16(scores) || (new_len && !aligned16(new_len)))
    return LSH_ERR_ALIGN;
  const long long rows = (long long)B * H * T;
  if (rows == 0) return LSH_OK;
  // a lane's 16-bit counters and the scores of a row in shared memory
  if (Hq / H > 128 || max_pages > lsh::cache::kMaxPickPages) return LSH_ERR_UNSUPPORTED;
  lsh::cache::SelectArgs a;
  a.tags = tags;
  a.q_buckets = q_buckets;
  a.scores = scores;
  a.selected = selected;
  a.B = B;
  a.G = Hq / H;
  a.n_rounds = n_rounds;
  a.n_select = n_select;
  a.n_local = n_local;
  a.causal = (mask & LSH_MASK_CAUSAL) ? 1 : 0;
  a.pg = pages_of(page_table, ctx_len, new_len, max_pages, page, n_pages, H, T);
  cudaStream_t s = as_stream(stream);
  const int per = lsh::cache::kScoreThreads / 32;
  // up to 64 KB of tags a head: the CTA that picks scores them itself (8 heads of 4093 tokens in 4 rounds:
  // 8.3 us on the device and 18 us a call as two kernels, 6.6 us and 15.5 us as one)
  const bool fused = (long long)max_pages * page * n_rounds * 2 <= 64 * 1024;
  if (!fused && max_pages > 0) {
    // pages a warp: 16, fewer where that would leave the device with less than 16 warps an SM
    const int sms = dev_info().sms > 0 ? dev_info().sms : 148;
    int wp = lsh::cache::kWarpPages;
    while (wp > 1 && (long long)B * H * max_pages / wp < 16ll * sms) wp /= 2;
    a.warp_pages = wp;
    const int groups = (max_pages + wp - 1) / wp;
    const unsigned grid = (unsigned)(((long long)B * H * groups + per - 1) / per);
    const int threads = lsh::cache::kScoreThreads;
    // a lane's chunks of a page in registers for one query head and up to 8 rounds of 128 tokens
    const int chunks = a.G == 1 && n_rounds * page % 256 == 0 ? n_rounds * page / 256 : 0;
    if (chunks == 1) lsh::cache::cache_score_kernel<1><<<grid, threads, 0, s>>>(a, groups);
    else if (chunks == 2) lsh::cache::cache_score_kernel<2><<<grid, threads, 0, s>>>(a, groups);
    else if (chunks == 4) lsh::cache::cache_score_kernel<4><<<grid, threads, 0, s>>>(a, groups);
    else lsh::cache::cache_score_kernel<0><<<grid, threads, 0, s>>>(a, groups);
    const lsh_status run = launch_status();
    if (run != LSH_OK) return run;
  }
  const int smem = fused || max_pages > n_select ? std::max(16, (max_pages + 3) / 4 * 16) : 16;
  a.fused = fused;
  if (smem > 32 * 1024) {
    // 48 KB are free to use, the kernel's static shared memory among them; beyond, the largest choice's limit is set
    // once: one for each call's size could be lowered by another thread's call before the launch
    static std::atomic<uint64_t> done{0};
    const lsh_status lim = allow_smem((const void*)lsh::cache::cache_pick_kernel, lsh::cache::kMaxPickPages * 4, done);
    if (lim != LSH_OK) return lim;
  }
  return launch_early(lsh::cache::cache_pick_kernel, (unsigned)rows, lsh::cache::kPickThreads, smem, s, a);
}

size_t lsh_cache_attend_workspace_bytes(int dtype, int B, int Hq, int H, int T, int D, int max_pages, int page,
                                        int n_select) {
  if (!valid_dtype(dtype) || check_cache_form(H, D, page, 32, 1, B, max_pages) != LSH_OK) return 0;
  if (H <= 0 || Hq <= 0 || Hq % H != 0 || T <= 0 || B <= 0 || n_select < 0) return 0;
  if (!fits_31_bits(B, Hq, T) || !fits_31_bits(B, H, T, std::max(1, n_select))) return 0;
  if ((long long)n_select * page > (1ll << 30)) return 0;
  return attend_plan_bytes(attend_plan(B, H, Hq / H, T, D, max_pages, page, n_select), D);
}

lsh_status lsh_cache_attend(const void* q, int dtype, int B, int Hq, int H, int T, int D, const void* cache,
                            int n_pages, const int32_t* ctx_len, const int32_t* new_len, const int32_t* page_table,
                            int max_pages, int page, int group, const int32_t* selected, int n_select, int mask,
                            int unit_keys, float scale, void* out, int out_dtype, float* lse, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (!valid_dtype(dtype) || !valid_dtype(out_dtype)) return LSH_ERR_DTYPE;
  const lsh_status st = check_cache_form(H, D, page, group, n_pages, B, max_pages);
  if (st != LSH_OK) return st;
  if (T < 0 || Hq < 0 || (H == 0 ? Hq != 0 : (Hq % H != 0 || Hq == 0))) return LSH_ERR_SHAPE;
  if (!fits_31_bits(B, Hq, T)) return LSH_ERR_SHAPE;
  if (selected ? n_select < 1 : n_select != 0) return LSH_ERR_INVALID_ARG;
  if ((long long)n_select * page > (1ll << 30) || !fits_31_bits(B, H, T, std::max(1, n_select))) return LSH_ERR_SHAPE;
  if (mask & ~(LSH_MASK_SELF | LSH_MASK_CAUSAL)) return LSH_ERR_INVALID_ARG;
  if (unit_keys != 0 && unit_keys != 1) return LSH_ERR_INVALID_ARG;
  if (!q || !cache || !ctx_len || !page_table || !out || !lse) return LSH_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(cache) || !aligned16(ctx_len) || !aligned16(page_table) || !aligned16(out) ||
      !aligned16(lse) || (new_len && !aligned16(new_len)) || (selected && !aligned16(selected)))
    return LSH_ERR_ALIGN;
  if ((long long)B * Hq * T == 0) return LSH_OK;
  const AttendPlan p = attend_plan(B, H, Hq / H, T, D, max_pages, page, n_select);
  if (p.units * p.cols >= (1ll << 31) || p.units * p.n_ct >= (1ll << 31)) return LSH_ERR_SHAPE;
  const size_t need = attend_plan_bytes(p, D);
  if (need > 0 && (!workspace || workspace_bytes < need)) return LSH_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return LSH_ERR_ALIGN;
  if (!(scale > 0.f)) scale = 1.0f / sqrtf((float)D);
  lsh::cache::AttendArgs a;
  a.q = q;
  a.cache = static_cast<const uint8_t*>(cache);
  a.selected = selected;
  a.out = out;
  a.lse = lse;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = need ? a.part_o + (size_t)p.max_ctas * 2 * p.cw * p.nt * D : nullptr;
  a.B = B;
  a.G = Hq / H;
  a.n_select = n_select;
  a.causal = (mask & LSH_MASK_CAUSAL) ? 1 : 0;
  a.self_mask = (mask & LSH_MASK_SELF) ? 1 : 0;
  a.unit_keys = unit_keys;
  a.out_f32 = out_dtype == LSH_F32;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.n_ct = p.n_ct;
  a.cols = p.cols;
  a.tile_cols = p.cw * p.nt;
  a.pg = pages_of(page_table, ctx_len, new_len, max_pages, page, n_pages, H, T);
  cudaStream_t s = as_stream(stream);
  return cache_form_dispatch(D, group, [&](auto DC, auto GC) -> lsh_status {
    constexpr int DD = decltype(DC)::value, GG = decltype(GC)::value;
    using bf = __nv_bfloat16;
#define LSH_CA(TQ)                                                              \
  do {                                                                          \
    if (p.cw == 1) return launch_cache_attend<TQ, DD, GG, 1, 1>(a, p, s);       \
    if (p.cw == 2) return launch_cache_attend<TQ, DD, GG, 2, 1>(a, p, s);       \
    if (p.nt == 1) return launch_cache_attend<TQ, DD, GG, 4, 1>(a, p, s);       \
    if constexpr (DD <= 128) return launch_cache_attend<TQ, DD, GG, 4, 2>(a, p, s); \
  } while (0)
    if (dtype == LSH_F32)
      LSH_CA(float);
    else
      LSH_CA(bf);
#undef LSH_CA
    return LSH_ERR_UNSUPPORTED;
  });
}

}  // extern "C"
