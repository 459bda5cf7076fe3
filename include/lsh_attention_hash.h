/*
 * lsh_attention_hash.h -- C ABI of the B200 (sm_100a) shared-QK LSH attention
 * (the Reformer's LSH attention): forward pass, backward, and decoding over a 4-bit cache.
 *
 * The method, as the pages state it:
 *   - Ultralytics glossary "Reformer", section "Atencao LSH": one shared
 *     projection for queries and keys; each vector is hashed by multiplying
 *     with a random matrix R and taking as bucket the position of the largest
 *     value of [xR, -xR]; tokens are sorted by bucket, the sorted sequence is
 *     cut into equal blocks and each token attends to its own block and the
 *     previous one; several hash rounds run in parallel.
 *   - twgreatdaily ICLR 2020 Reformer article, section "1 LSH Attention":
 *     attention of a query as a sum over its admissible key set divided by the
 *     set's partition function; Q = K with length-normalised keys; two-level
 *     sort by (bucket, position); a later chunk looks back one chunk; several
 *     rounds with different hash functions.
 *   - ai-scholar.tech Reformer article, "Transformerの問題点とは": the
 *     1/sqrt(d_k) logit scale.
 *
 * Conventions shared by every call:
 *   - Tensors are dense, row-major, caller-owned device buffers; every pointer
 *     must be 16-byte aligned.  The library never allocates or frees device
 *     memory: scratch space is passed in by the caller (size from the matching
 *     *_workspace_bytes query).
 *   - Shapes: B batch, H heads, L sequence length, D head dim, n_rounds hash
 *     rounds.  Index tensors are int32, so B*H*n_rounds*L < 2^31.
 *   - dtype codes: LSH_F32 (float) or LSH_BF16 (bfloat16); accumulation is
 *     always fp32.
 *   - Every call is asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *     default stream) and does no host synchronisation, except
 *     lsh_get_device_status.
 *   - Argument, shape, dtype and alignment errors are returned before any
 *     launch and leave every output untouched.  A failed launch returns
 *     LSH_ERR_CUDA.  Errors that kernels detect (an exhausted bounded wait)
 *     are recorded in a per-device status word read by lsh_get_device_status.
 *   - An empty problem (B*H*L == 0) returns LSH_OK without launching.
 *   - No C++ exception crosses this boundary.
 */
#ifndef LSH_ATTENTION_HASH_H
#define LSH_ATTENTION_HASH_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define LSH_API __attribute__((visibility("default")))
#else
#define LSH_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum lsh_status {
  LSH_OK = 0,
  LSH_ERR_INVALID_ARG = 1, /* null required pointer, bad flag or parameter */
  LSH_ERR_SHAPE = 2,       /* size out of range, L % chunk != 0, odd n_buckets */
  LSH_ERR_DTYPE = 3,       /* unknown dtype code */
  LSH_ERR_ALIGN = 4,       /* a pointer is not 16-byte aligned */
  LSH_ERR_WORKSPACE = 5,   /* workspace missing or smaller than required */
  LSH_ERR_CUDA = 6,        /* a CUDA launch or runtime call failed */
  LSH_ERR_TIMEOUT = 7,     /* a device-side bounded wait ran out */
  LSH_ERR_UNSUPPORTED = 8  /* valid request that no kernel of this build serves */
} lsh_status;

typedef enum lsh_dtype { LSH_F32 = 0, LSH_BF16 = 1 } lsh_dtype;

/* Mask bits of lsh_chunk_attend. */
typedef enum lsh_mask {
  LSH_MASK_SELF = 1,    /* a slot does not see itself unless it is its only key */
  LSH_MASK_CAUSAL = 2,  /* a key after the query's original position is not admissible */
  LSH_MASK_BUCKET = 4,  /* a key in another bucket than the query's (this round) is not admissible */
  LSH_MASK_UNION = 8    /* lower each logit by log(#rounds sharing the bucket); needs LSH_MASK_BUCKET */
} lsh_mask;

/* Version of this ABI (incremented on any signature change). */
LSH_API int lsh_abi_version(void);

/* Human-readable name of a status code (static storage, never NULL). */
LSH_API const char* lsh_status_string(int status);

/*
 * lsh_hash -- angular LSH of every shared query/key row, all rounds at once.
 * (Ultralytics glossary "Reformer", "Atencao LSH": bucket = position of the
 * largest value of [xR, -xR].)
 *
 *   qk        [B, H, L, D]  dtype          shared query/key rows
 *   R         [n_rounds, D, n_buckets/2] dtype   one random projection per round,
 *                                          shared by all batches and heads
 *   buckets   [B, H, n_rounds, L] int32    out: bucket in [0, n_buckets); entry k
 *                                          (< n_buckets/2) means +p_k was largest,
 *                                          k + n_buckets/2 means -p_k was
 *   near_tie  [B, H, n_rounds, L] uint8    out, nullable: 1 when the two largest
 *                                          values u1 >= u2 of [p, -p] satisfy
 *                                          u1 - u2 < 1e-5 * max(u1, 1e-30)
 *
 * p = x R is computed from the raw row (the argmax does not depend on the
 * row's length); products are exact and sums are fp32.  Exact ties go to the
 * lowest bucket index.  Requires n_buckets even, 2 <= n_buckets <= 65536,
 * D % 8 == 0, 8 <= D <= 256.
 */
LSH_API lsh_status lsh_hash(const void* qk, int dtype, int B, int H, int L, int D,
                    const void* R, int n_rounds, int n_buckets,
                    int32_t* buckets, uint8_t* near_tie, void* stream);

/*
 * Bytes of scratch that lsh_sort_permute needs for these sizes (0 when none).
 */
LSH_API size_t lsh_sort_workspace_bytes(int B, int H, int L, int n_rounds, int n_buckets);

/*
 * lsh_sort_permute -- stable sort of each (b, h, round) segment by the key
 * (bucket, position), and an optional gather of the sorted rows.
 * (twgreatdaily ICLR 2020 Reformer article, "1 LSH Attention": two-level
 * sort by bucket number and position inside the bucket.)
 *
 *   buckets    [B, H, n_rounds, L] int32   in, values in [0, n_buckets)
 *   perm       [B, H, n_rounds, L] int32   out: perm[s] = original position of
 *                                          sorted slot s
 *   inv        [B, H, n_rounds, L] int32   out, nullable: inv[perm[s]] = s
 *   qk, v      [B, H, L, D] dtype          in, nullable (both or neither): rows
 *                                          to gather in sorted order
 *   qk_sorted, v_sorted [B, H, n_rounds, L, D] dtype  out, nullable with qk/v:
 *                                          qk_sorted[..., s, :] = qk[..., perm[s], :]
 *   workspace  device scratch of at least lsh_sort_workspace_bytes(...) bytes,
 *              contents undefined on entry and on exit
 *
 * A bucket id outside [0, n_buckets) is a caller error: the kernels skip that
 * element, leave the slot it would have filled unwritten, and record
 * LSH_ERR_INVALID_ARG in the device status word (lsh_get_device_status).
 */
LSH_API lsh_status lsh_sort_permute(const int32_t* buckets, int B, int H, int L, int n_rounds,
                            int n_buckets, int32_t* perm, int32_t* inv,
                            const void* qk, const void* v, int dtype, int D,
                            void* qk_sorted, void* v_sorted,
                            void* workspace, size_t workspace_bytes, void* stream);

/*
 * lsh_sort_permute_noalloc -- lsh_sort_permute (without the optional row
 * gather) for callers that cannot hand the library any scratch memory.
 * The pages have no counterpart of this call; it exists for this library's
 * users only.
 *
 * Some callers cannot allocate device memory while they run: a plugin that a
 * host application gives only its input and output buffers, a process whose
 * device memory another framework's pool has already reserved, or a code path
 * that must not pay cudaMalloc's implicit synchronisation.  This entry point
 * takes no workspace and allocates nothing (no cudaMalloc, no cudaFree, no
 * allocating library call): its scratch is a 16 MiB array of static device
 * memory inside the library, which every GPU that loads the library holds
 * until the process exits.
 *
 *   buckets, perm, inv: as for lsh_sort_permute (inv nullable).
 *
 * Shapes with L <= 65536 and n_buckets <= 1024 (the 64K workload among them)
 * are sorted by one CTA per segment entirely in shared memory and touch the
 * array not at all.  Larger shapes run the radix sort (one counting pass per
 * 8-bit digit of the bucket id), which takes, with S = B*H*n_rounds segments,
 * S * 256 * ceil(L / 4096) counter words, at most S * 64 + S + 3 more, and, when
 * n_buckets > 256, 2 * S * L words for the first pass's ids and positions; the
 * call returns LSH_ERR_WORKSPACE, before any launch, when that exceeds the
 * array's 4 Mi words (16 MiB).  All other argument rules and errors are those
 * of lsh_sort_permute.
 *
 * The first call on a device that needs the array looks up its device
 * address (with that device current) and keeps it for the life of the
 * process, so make that first call before any stream capture, and do not use
 * this call after cudaDeviceReset (the kept address would be stale).  Every
 * call on a device shares the one array and leaves its contents behind; the
 * call clears what must start at zero itself.  Calls whose work overlaps on
 * the GPU (different streams, or graphs running at the same time) race on the
 * array: order them, for example on one stream.
 */
LSH_API lsh_status lsh_sort_permute_noalloc(const int32_t* buckets, int B, int H, int L,
                                            int n_rounds, int n_buckets, int32_t* perm,
                                            int32_t* inv, void* stream);

/*
 * lsh_chunk_attend -- attention of every sorted slot to its own chunk and the
 * previous chunk, per round, scattered back to original token order.
 * (twgreatdaily ICLR 2020 Reformer article, "1 LSH Attention": sum over the
 * admissible set divided by its partition function, masked keys, Q = K with
 * normalised keys, later chunk looks back one chunk; rdly.ru Reformer summary,
 * "Разделение на блоки": fixed-size blocks of the sorted sequence.)
 *
 *   qk, v      [B, H, L, D] dtype          in: shared query/key rows and values
 *   perm       [B, H, n_rounds, L] int32   in: from lsh_sort_permute
 *   buckets    [B, H, n_rounds, L] int32   in, nullable: from lsh_hash (by original
 *              position); required by LSH_MASK_BUCKET and LSH_MASK_UNION, else unread
 *   qk_sorted, v_sorted  nullable [B, H, n_rounds, L, D] dtype: when given, the
 *              rows are read in sorted order from them instead of through perm
 *   chunk      chunk length c, L % c == 0.  Chunk k = sorted slots
 *              [k c, (k+1) c); its queries see the slots of chunk k-1 (none
 *              for k = 0: no wrap-around) and of chunk k
 *   mask       bits of lsh_mask: LSH_MASK_SELF (1): a slot does not see itself
 *              unless it is its only key; LSH_MASK_CAUSAL (2): a key whose
 *              original position perm[t] is after the query's perm[s] is not
 *              admissible (the pages' character-level language model; the self
 *              rule then applies to what remains, so a query with no earlier key
 *              in its window sees only itself); LSH_MASK_BUCKET (4): a key whose
 *              bucket buckets[r][perm[t]] differs from the query's is not
 *              admissible (the article's admissible set: the query's own bucket,
 *              batched by chunks; self rule as for causal); LSH_MASK_UNION (8,
 *              only with 4): each admissible logit is lowered by log N, N = the
 *              number of rounds r' with buckets[r'][i] == buckets[r'][j] (the
 *              article's multi-round union: lsh_combine_rounds then counts each
 *              shared key once).  Every mask runs on the tensor-core path
 *              (UNION there for up to 8 rounds, with a stream-ordered scratch
 *              buffer of 16 bytes per token, cudaMallocAsync / cudaFreeAsync on
 *              `stream`, holding each token's buckets in all rounds as fp16
 *              codes; a bucket id outside [0, 30720) has no code and records
 *              LSH_ERR_UNSUPPORTED in the device status word, its pairs then
 *              counting no shared round) and on the CUDA-core path
 *   scale      logit scale; <= 0 selects 1/sqrt(D).  logit(s, t) =
 *              scale * qk[perm[s]] . qk[perm[t]] / ||qk[perm[t]]||
 *   out_rounds [B, H, n_rounds, L, D] out_dtype  out: per-round softmax-weighted
 *              values, at the original position perm[s]
 *   lse        [B, H, n_rounds, L] float   out: per-round log-sum-exp of the
 *              logits, at the original position
 *
 * A key row of zero length contributes logit 0.  Requires D % 8 == 0,
 * 8 <= D <= 256, 1 <= chunk <= L.
 */
LSH_API lsh_status lsh_chunk_attend(const void* qk, const void* v, int dtype, int B, int H, int L,
                            int D, int n_rounds, const int32_t* perm, const int32_t* buckets,
                            const void* qk_sorted, const void* v_sorted, int chunk,
                            int mask, float scale, void* out_rounds, int out_dtype,
                            float* lse, void* stream);

/*
 * lsh_combine_rounds -- merge the rounds of every query by their log-sum-exp
 * weights: out = sum_r exp(lse_r - LSE) o_r with LSE = log sum_r exp(lse_r).
 * (twgreatdaily ICLR 2020 Reformer article, "1 LSH Attention": several hash
 * rounds, each with its own admissible set; weighting by each round's
 * partition function gives the softmax over the union of the rounds' key sets
 * counted with multiplicity.)
 *
 *   out_rounds [B, H, n_rounds, L, D] in_dtype
 *   lse        [B, H, n_rounds, L] float
 *   out        [B, H, L, D] out_dtype       out
 *   lse_out    [B, H, L] float              out, nullable: LSE
 */
LSH_API lsh_status lsh_combine_rounds(const void* out_rounds, int in_dtype, const float* lse,
                              int B, int H, int L, int D, int n_rounds, void* out,
                              int out_dtype, float* lse_out, void* stream);

/*
 * lsh_chunk_attend_backward -- gradients of sum(dout * out) with respect to the
 * shared rows and the values, where out is lsh_combine_rounds' merge of
 * lsh_chunk_attend's rounds.  (Training through LSH attention recomputes from
 * the stored hash: twgreatdaily ICLR 2020 Reformer article, "1 LSH Attention";
 * Ultralytics glossary "Reformer", "Atencao LSH".)  The hash, the sort and the
 * masks are held fixed; per admissible pair (i, j) of every round, with
 * p~ = exp(logit - LSE_i):
 *     dv_j += p~ dout_i,  dz = p~ (dout_i . v_j - dout_i . out_i),
 *     dqk_i += scale dz k_j,  and through k_j = qk_j / ||qk_j|| the key side.
 *
 *   qk, v, perm, buckets, chunk, mask, scale   as given to lsh_chunk_attend
 *   out        [B, H, L, D] out_dtype   in: the merged output (lsh_combine_rounds)
 *   lse        [B, H, L] float          in: its LSE (lse_out of lsh_combine_rounds)
 *   dout       [B, H, L, D] out_dtype   in: gradient of the loss w.r.t. out
 *   dqk, dv    [B, H, L, D] float       out: overwritten (zeroed, then accumulated
 *                                       over the rounds in order; deterministic)
 *
 * Every mask runs.  bf16 rows with bf16 out / dout, D = 128, chunk = 64 and
 * L % 128 == 0 run on the tensor cores of sm_100 with every mask (the union
 * correction up to 8 rounds): a per-token pass (LSE, dout . out, key lengths)
 * into a stream-ordered scratch buffer of 16 bytes per token, with masks a
 * per-slot pass (bucket, and whether the window leaves the token alone) into
 * 4 bytes per token and round, with the union correction each token's buckets
 * in all rounds (16 bytes per token; bucket ids below 30720, as for
 * lsh_chunk_attend) (cudaMallocAsync / cudaFreeAsync on
 * `stream`; LSH_ERR_CUDA if they cannot be had), then one launch per round.
 * Everything else runs on the CUDA cores (one launch per round after zeroing
 * dqk / dv).  Both keep the rounds in order, so the
 * result is deterministic.  A key row of zero length takes the clamp's linear
 * branch (its gradient is scaled by 1e12).
 * Requires what lsh_chunk_attend requires and B * H <= 65535.
 */
LSH_API lsh_status lsh_chunk_attend_backward(const void* qk, const void* v, int dtype, int B, int H, int L,
                                     int D, int n_rounds, const int32_t* perm, const int32_t* buckets,
                                     int chunk, int mask, float scale, const void* out, const float* lse,
                                     const void* dout, int out_dtype, float* dqk, float* dv, void* stream);

/*
 * ---- Decoding: a paged cache in 4 bits, attention over it, hash-selected pages ----
 * The pages describe training; generating token by token needs the keys and values
 * of every earlier position again at each step.  These calls keep them in 4 bits and
 * attend to them, with the shared-QK conventions of lsh_chunk_attend (the query is the
 * token's own qk row, keys are length-normalised, a token does not see itself unless
 * it is its only key).
 *
 * The cache is one buffer [n_pages, H, block], block = lsh_cache_block_bytes(page, D,
 * group) bytes.  A page holds `page` consecutive positions of one sequence (a power
 * of two from 16 to 256); page_table [B, max_pages] names the physical page of each of
 * a sequence's logical pages, in any order, and sequences may share pages that are only
 * read.  Entries of logical pages that lie behind a sequence are not looked at.
 *
 * A stored value is z + s c with a code c of 0..15 and, per row and group of `group`
 * dims, z = the largest bf16 not above the group's smallest value and s = the bf16 nearest to
 * (largest - z) / 15; c = min(15, nearest integer to (x - z) / s, ties to even).  The
 * quotients are the real numbers', so equal rows are stored equally by every kernel.
 * A group whose s would be below 2^-100 is stored as z; a group that holds an infinity or a
 * NaN, whose range overflows a float or whose smallest value lies below every bf16, reads back
 * as NaN.  Each K row also keeps 1 / max(||row||, 1e-12) of the row as it came, in fp32 (0 with an
 * infinity, NaN with a NaN).  At D = 128 and group = 64 a token takes 148 bytes per head.
 *
 * Positions: ctx_len [B] int32 counts the tokens of each sequence in the cache, this
 * call's among them.  Of the T rows of a call the first new_len[b] belong to sequence b
 * (new_len null: all T) and are its last tokens: row i is position ctx_len[b] -
 * new_len[b] + i.  Rows at or behind new_len[b], and rows whose position would be
 * negative, are padding (a new_len above T counts as T).  All three arrays are read on the
 * device, so a captured graph replays with their current contents.
 *
 * Caller errors that only the device can see are recorded as LSH_ERR_INVALID_ARG in the
 * device status word, and no access leaves a buffer: a ctx_len outside
 * [0, max_pages * page] makes its sequence count as empty; a page id outside
 * [0, n_pages) makes its page count as missing (not written, read back as zeros, not
 * attended to); a bucket outside [0, 65536) is stored by its low 16 bits.
 *
 * Requires D of 64, 128 or 256 and group of 32 or 64 (LSH_ERR_UNSUPPORTED otherwise).
 */

/* Bytes of one (page, head) block of the cache, a multiple of 16; 0 for a form that no
 * kernel serves. */
LSH_API size_t lsh_cache_block_bytes(int page, int D, int group);

/*
 * lsh_cache_write -- quantise rows into the cache at their positions.
 *
 *   k, v       [B, H, T, D] dtype          in: key (shared qk) and value rows
 *   buckets    [B, H, n_rounds, T] int32   in, nullable (with tags): lsh_hash's buckets
 *   ctx_len, new_len, page_table           see above
 *   cache      [n_pages, H, block]         in/out: only the rows' own bytes change
 *   tags       [n_pages, H, n_rounds, page] 16-bit  in/out, nullable (with buckets): the
 *              buckets by position, for lsh_cache_select; 1 <= n_rounds <= 64
 *
 * Two rows with the same place in one call (sequences that share a page they write to)
 * leave that place with either row's bytes or a mixture.
 */
LSH_API lsh_status lsh_cache_write(const void* k, const void* v, int dtype, int B, int H, int T, int D,
                                   const int32_t* buckets, int n_rounds, const int32_t* ctx_len,
                                   const int32_t* new_len, const int32_t* page_table, int max_pages, int page,
                                   int group, void* cache, int n_pages, uint16_t* tags, void* stream);

/*
 * lsh_cache_read -- the stored values of each sequence's last new_len[b] tokens (all of
 * them with new_len = ctx_len), rounded once to out_dtype.
 *
 *   k, v       [B, H, T, D] out_dtype      out: K rows are not length-normalised; padding 0
 *   key_inv    [B, H, T] float             out, nullable: 1 / length of the original K row;
 *                                          padding 0
 */
LSH_API lsh_status lsh_cache_read(const void* cache, int n_pages, int B, int H, int T, int D,
                                  const int32_t* ctx_len, const int32_t* new_len, const int32_t* page_table,
                                  int max_pages, int page, int group, void* k, void* v, int out_dtype,
                                  float* key_inv, void* stream);

/*
 * lsh_cache_select -- the pages each new token attends to, by shared buckets.
 *
 *   tags       [n_pages, H, n_rounds, page] 16-bit  in: from lsh_cache_write
 *   q_buckets  [B, Hq, n_rounds, T] int32  in: buckets of the T rows' queries (lsh_hash);
 *              Hq a multiple of H, query heads h Hq/H .. (h + 1) Hq/H - 1 use cached head h
 *   mask       LSH_MASK_CAUSAL or 0: whether positions after the row's own count
 *   scores     [B, H, T, max_pages] int32  out: per page the number of (query head of h,
 *              round, admissible position) with equal buckets, the row's own position
 *              included; -1 for pages without an admissible position
 *   selected   [B, H, T, n_select] int32   out: the last n_local pages with an admissible
 *              position and those of the highest scores, of equal scores the lowest pages;
 *              n_select in all (or as many as there are), ascending, then -1
 *
 * 1 <= n_rounds <= 64, 0 <= n_local <= n_select; at most 128 query heads per cached head
 * and 49152 logical pages (LSH_ERR_UNSUPPORTED beyond).
 */
LSH_API lsh_status lsh_cache_select(const uint16_t* tags, int n_pages, const int32_t* q_buckets, int B, int Hq, int H,
                                    int T, int n_rounds, const int32_t* ctx_len, const int32_t* new_len,
                                    const int32_t* page_table, int max_pages, int page, int n_select, int n_local,
                                    int mask, int32_t* selected, int32_t* scores, void* stream);

/*
 * Bytes of scratch that lsh_cache_attend needs for these sizes (0 when none, as for short contexts);
 * n_select 0 without selection.
 */
LSH_API size_t lsh_cache_attend_workspace_bytes(int dtype, int B, int Hq, int H, int T, int D, int max_pages, int page,
                                                int n_select);

/*
 * lsh_cache_attend -- attention of the T rows over their sequences' cached tokens, which
 * include the rows themselves once lsh_cache_write has stored them.
 *
 *   q          [B, Hq, T, D] dtype         in: queries; Hq as for lsh_cache_select
 *   selected   [B, H, T, n_select] int32   in, nullable (n_select 0 then): logical pages
 *              that each row attends to, in any order; entries outside [0, max_pages) or
 *              behind the sequence are skipped, a page listed twice counts twice
 *   mask       LSH_MASK_SELF (a token does not see itself unless nothing else is
 *              admissible to it) and LSH_MASK_CAUSAL (no later position); else 0
 *   unit_keys  1: logits are divided by the key rows' original lengths (shared QK); 0: not
 *   scale      logit scale; <= 0 selects 1/sqrt(D)
 *   out        [B, Hq, T, D] out_dtype     out: softmax-weighted stored values; 0 for padding
 *                                          and rows without an admissible key
 *   lse        [B, Hq, T] float            out: log-sum-exp of the logits; -inf for those
 *   workspace  device scratch of at least lsh_cache_attend_workspace_bytes(...) bytes,
 *              contents undefined on entry and on exit; calls that may overlap on the GPU
 *              (other streams, graphs replayed at the same time) need one each
 *
 * The products with the codes are exact integer sums of fixed-point numbers: a query in steps of
 * its largest entry / 8355711, a weight (softmax numerator times the value's scale) in steps of 2^-22 of
 * the power of two at or below the largest of its 64 keys' weights, 2^-127 at the finest.  Everything
 * else is fp32; keys in any order give the same result only up to rounding, the same call the same bits.
 *
 * Range.  A query row with an infinity or a NaN answers NaN; its largest entry lies between 1e-30 and
 * 1e36 (below, its entries count with fewer digits).  Keys may reach 1e36 in size; of plain keys
 * (unit_keys 0) sum_d |q_d K_d|, before the scale, stays below 1e38.  The size of the stored values times
 * the number of a row's keys may reach 1e35 (beyond, the sum before its division by the weights' sum,
 * which are up to 2^8, can overflow: infinities or NaN).
 *
 * lse makes the result joinable with other key sets by lsh_combine_rounds, where one of
 * them has a key for the row.
 */
LSH_API lsh_status lsh_cache_attend(const void* q, int dtype, int B, int Hq, int H, int T, int D, const void* cache,
                                    int n_pages, const int32_t* ctx_len, const int32_t* new_len,
                                    const int32_t* page_table, int max_pages, int page, int group,
                                    const int32_t* selected, int n_select, int mask, int unit_keys, float scale,
                                    void* out, int out_dtype, float* lse, void* workspace, size_t workspace_bytes,
                                    void* stream);

/*
 * Synchronises `stream`, then returns and clears the current device's status
 * word (LSH_OK when no kernel recorded an error).  Returns LSH_ERR_CUDA if the
 * synchronisation itself fails.
 */
LSH_API lsh_status lsh_get_device_status(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LSH_ATTENTION_HASH_H */
