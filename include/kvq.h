/*
 * kvq.h -- C ABI of the compressed-KV-cache attention library (sm_103a).
 *
 * The cache follows "KV殘差窗口：最近Token一定值得高精度嗎？" (huhohoo.com,
 * kv-residual-window), section 固定預算，先問它保護了誰: the tokens before the
 * last R are stored as grouped symmetric int4 (group 32, no zero point, K per
 * channel over 32-token groups, V per token over 32-feature groups) and the
 * last R tokens stay in floating point. Attention always covers the whole
 * context, or exactly a listed set of candidate keys (MiniCPM5-2B study,
 * bjdmk.com.cn/news/5855973, sections 6 and 9). The chunk layout and the
 * per-row region mass follow "Catnip Week 10 KV Cache Attention Study"
 * (cappuccino.cafe/kv-attn.html), section "KV Cache 的实际作用"; MXFP8 Q/K
 * (E4M3 elements, one E8M0 scale per 32 along the head dim) follows its section
 * "Q/K 与 probability quantization 的影响".
 *
 * Conventions for every call:
 *  - All tensor pointers are DEVICE pointers owned by the caller; the library
 *    never allocates, never frees and never synchronises. Every pointer must be
 *    16-byte aligned (else KVQ_ERR_ALIGN).
 *  - Tensors are dense, row-major, in the index order written beside them.
 *  - GQA: query head h reads KV head h / (q_heads / kv_heads); q_heads must be
 *    a multiple of kv_heads.
 *  - Work is enqueued on `stream` (a cudaStream_t; NULL = the legacy default
 *    stream) and runs asynchronously.
 *  - Argument errors are returned before anything is enqueued. Errors a kernel
 *    detects are OR-ed as KVQ_DEV_* bits into *dev_status (a device int32 the
 *    caller zeroes beforehand and reads after synchronising); kernels never
 *    trap and every wait in them is bounded.
 *  - sm_scale <= 0 selects 1/sqrt(head_dim). Only kv_attend_tree masks keys.
 *  - Calls that may run at the same time (on several streams, or replayed from
 *    several captured graphs) need a workspace each, and their outputs and a
 *    summary or list that one of them writes must not overlap.
 *  - head_dim is a multiple of 32 in [32, 256].
 */
#ifndef KVQ_H
#define KVQ_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define KVQ_API __attribute__((visibility("default")))
#else
#define KVQ_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *kvq_stream_t; /* same type as cudaStream_t */

typedef enum {
  KVQ_OK = 0,
  KVQ_ERR_ARG = 1,         /* bad shape, dtype, count or NULL pointer */
  KVQ_ERR_ALIGN = 2,       /* a pointer is not 16-byte aligned */
  KVQ_ERR_UNSUPPORTED = 3, /* a valid combination this build has no kernel for */
  KVQ_ERR_WORKSPACE = 4,   /* workspace given but smaller than required */
  KVQ_ERR_CUDA = 5         /* a launch failed (cudaGetLastError) */
} kvq_status;

/* Bits OR-ed into *dev_status by kernels. */
enum {
  KVQ_DEV_INDEX = 1,   /* a candidate index outside [0, n_tokens), a listed block or a parent
                          that does not exist (that key, block or row is skipped) */
  KVQ_DEV_DUP = 2,     /* a candidate list holds the same index twice (validate only), or a
                          list of blocks does not increase */
  KVQ_DEV_TIMEOUT = 4, /* a bounded wait ran out; the outputs of that launch are invalid */
  KVQ_DEV_BOUNDS = 8,  /* an address range a kernel derived lay outside the call's buffers
                          (checked in the KVQ_DEBUG build, kvq_debug_checks); outputs invalid */
  KVQ_DEV_PAGES = 16   /* kv_page_tables: a request's new tokens got no pages (none left, or its
                          row of the table is full); the request stays as it was */
};

typedef enum { KVQ_F32 = 0, KVQ_BF16 = 1, KVQ_MXFP8 = 2 } kvq_dtype;

/*
 * A packed cache of `batch` sequences x `kv_heads` heads, each holding
 * `n_tokens` (N) tokens of `head_dim` (D) features, the last `recent` (R)
 * tokens kept in the window. With cut = N - R and Gk = ceil(cut / 32):
 *
 *   k_codes  [batch][kv_heads][Gk][32][D/2]   uint8: token-group major; byte i
 *            of a token row holds channels 2i (low nibble) and 2i+1 (high
 *            nibble) as code + 8 (codes in [-7, 7]); padding tokens of the last
 *            group hold code 0.
 *   k_scales [batch][kv_heads][Gk][D]         float: one scale per (group, channel).
 *   v_codes  [batch][kv_heads][cut][D/2]      uint8: same nibble order, per token.
 *   v_scales [batch][kv_heads][cut][D/32]     float: one scale per (token, 32 features).
 *   k_window [batch][kv_heads][R][D]          kwin_dtype: F32, BF16, or MXFP8
 *            (E4M3 bytes, with k_window_e8m0 [batch][kv_heads][R][D/32] holding
 *            the E8M0 block-scale bytes, exponent + 127).
 *   v_window [batch][kv_heads][R][D]          vwin_dtype: F32 or BF16.
 *   header   {N, D, R, 32}: the 16 bytes of shape metadata, filled by kv_pack.
 *
 * Pointers for empty arrays (cut == 0 or R == 0) may be NULL.
 */
typedef struct kvq_cache {
  int32_t batch, kv_heads, n_tokens, head_dim, recent;
  int32_t kwin_dtype, vwin_dtype;
  uint8_t *k_codes;
  float *k_scales;
  uint8_t *v_codes;
  float *v_scales;
  void *k_window;
  void *v_window;
  uint8_t *k_window_e8m0;
  uint32_t header[4];
  /* Room reserved per (sequence, head) for kv_append; 0 and 0 = a tight cache
   * whose arrays are exactly the sizes above. With cap_groups > 0 the
   * per-(sequence, head) strides become cap_groups K groups (k_codes,
   * k_scales), 32 * cap_groups V rows (v_codes, v_scales) and cap_window
   * window rows (k_window, v_window, k_window_e8m0); rows past Gk, cut and R
   * are unused. Both are then required, with cap_groups >= Gk and
   * cap_window >= R. */
  int32_t cap_groups;
  int32_t cap_window;
} kvq_cache;

/* Array sizes of a cache, in bytes (host only, no GPU needed):
 * sizes[0..7] = k_codes, k_scales, v_codes, v_scales, k_window, v_window,
 * k_window_e8m0, header. Returns KVQ_ERR_ARG for an invalid shape. */
KVQ_API kvq_status kvq_cache_sizes(int32_t batch, int32_t kv_heads, int32_t n_tokens,
                                   int32_t head_dim, int32_t recent, int32_t kwin_dtype,
                                   int32_t vwin_dtype, size_t sizes[8]);

/* Array sizes of a cache laid out for kv_append, with cap_groups >= 1 K groups
 * (and 32 * cap_groups V rows) and cap_window window rows reserved per
 * (sequence, head); same order as kvq_cache_sizes. KVQ_ERR_ARG for an invalid
 * shape. */
KVQ_API kvq_status kvq_cache_sizes_reserved(int32_t batch, int32_t kv_heads, int32_t head_dim,
                                            int32_t kwin_dtype, int32_t vwin_dtype,
                                            int32_t cap_groups, int32_t cap_window,
                                            size_t sizes[8]);

/* Total payload in bytes: the sum of kvq_cache_sizes (header included). */
KVQ_API size_t kvq_cache_bytes(int32_t batch, int32_t kv_heads, int32_t n_tokens,
                               int32_t head_dim, int32_t recent, int32_t kwin_dtype,
                               int32_t vwin_dtype);

/*
 * kv_pack -- quantize K and V into `cache` (residual-window page, section
 * 固定預算). k, v: [batch][kv_heads][N][D] in in_dtype (F32 or BF16), device.
 * For each (sequence, head): tokens [0, cut) are quantized, tokens [cut, N)
 * are copied into the window (rounded to nearest even when the window type is
 * narrower; E4M3 with an E8M0 scale per 32 features for an MXFP8 K window).
 * int4 rule: scale = amax / 7 rounded to fp32, code = clamp(rint(x / scale),
 * -7, 7) with the division correctly rounded in fp32 and ties to even; a zero
 * scale gives all-zero codes. Inputs are expected finite: the code of a NaN
 * or infinite element is unspecified (the group's other elements follow the
 * rule; a NaN does not enter amax). The cache's shape fields and array
 * pointers are read; header[] is written. dev_status may be NULL.
 */
KVQ_API kvq_status kv_pack(const void *k, const void *v, int32_t in_dtype, kvq_cache *cache,
                           int32_t *dev_status, kvq_stream_t stream);

/*
 * kv_append -- add n_new tokens per (sequence, head) to a cache laid out with
 * reserved room (cap_groups > 0), as decoding produces them. The pages build
 * the cache once and leave this online update out ("KV殘差窗口", section
 * 適用邊界：本輪沒有測在線更新: the oldest window entries are not migrated
 * into the quantized part token by token); this call is that update, with
 * the cache layout and quantization rule of kv_pack.
 * k_new, v_new: [batch][kv_heads][n_new][D] in in_dtype (F32 or BF16), device.
 * The window grows by n_new; then, while it holds at least `window` + 32
 * tokens, its oldest 32 become one more int4 K group and 32 more V rows (the
 * kv_pack rule applied to the window's values, so the result equals kv_pack
 * of the whole sequence whenever the window type holds the inputs exactly --
 * BF16 inputs with a BF16 window, or an F32 window). Afterwards N - R is the
 * largest multiple of 32 leaving at least `window` tokens in the window (and
 * never less than before), so R lies in [window, window + 31] once
 * N >= window.
 * On success the call updates cache->n_tokens, cache->recent and header[]
 * (host fields) and enqueues the kernels on `stream`.
 * Errors: KVQ_ERR_UNSUPPORTED for a tight cache (cap_groups == 0), an MXFP8
 * K window, an int4 part whose last K group is padded ((N - R) % 32 != 0) or
 * more than 65,535 (sequence, head) pairs when groups migrate;
 * KVQ_ERR_WORKSPACE when the reserved room (cap_groups, cap_window) is too
 * small for the result; the cache is then left unchanged.
 */
KVQ_API kvq_status kv_append(kvq_cache *cache, const void *k_new, const void *v_new,
                             int32_t in_dtype, int32_t n_new, int32_t window,
                             int32_t *dev_status, kvq_stream_t stream);

/*
 * kv_attend -- O = softmax(sm_scale * Q K^T) V over all N tokens of the cache,
 * with K, V dequantized (int4 part) or taken from the window.
 * q:   [batch][q_heads][n_q][D] in q_dtype (F32 or BF16), device.
 * out: [batch][q_heads][n_q][D] in out_dtype (F32 or BF16), device.
 * region_bounds: HOST array of n_regions + 1 increasing token positions
 *   starting at 0 and ending at N, or NULL; region_mass: device float
 *   [batch][q_heads][n_q][n_regions] receiving, per query row, the softmax
 *   mass on tokens [b_k, b_{k+1}) (n_regions <= 16). For an MXFP8 K window, Q
 *   is quantized the same way (E4M3 + E8M0 per 32) before QK^T.
 * workspace: device scratch of *ws_bytes bytes. With workspace == NULL the
 *   call only stores the required size in *ws_bytes and returns KVQ_OK
 *   (enqueueing nothing); to run, pass a non-NULL workspace even when the
 *   required size is 0.
 * Kernel choice: one query row per (sequence, head) with 8 query heads per KV
 *   head and D = 128 runs the split-K decode kernels; with bf16 q, D = 128
 *   and at least 64 query rows, a bf16 or MXFP8 window covering all tokens,
 *   or an int4 part followed by a bf16 window (the key tiles holding int4
 *   tokens are expanded to bf16 in the workspace, the others read in place),
 *   runs the tensor-core chunk kernel (when batch * q_heads <= 65,535);
 *   everything else runs the fp32 kernel, which needs q_heads and batch
 *   <= 65,535 (else KVQ_ERR_UNSUPPORTED).
 */
KVQ_API kvq_status kv_attend(const kvq_cache *cache, const void *q, int32_t q_dtype,
                             int32_t q_heads, int32_t n_q, float sm_scale, void *out,
                             int32_t out_dtype, const int32_t *region_bounds, int32_t n_regions,
                             float *region_mass, void *workspace, size_t *ws_bytes,
                             int32_t *dev_status, kvq_stream_t stream);

/* Columns of kv_attend_stats' output, one row of KVQ_N_STATS floats per query. */
enum {
  KVQ_STAT_ENTROPY = 0,  /* H = -sum p ln p (nats) */
  KVQ_STAT_SUPPORT = 1,  /* exp(H) / N: entropy-equivalent share of the keys */
  KVQ_STAT_TOP1 = 2,     /* mass of the ceil(1 % of N) largest probabilities */
  KVQ_STAT_TOP5 = 3,     /* ... ceil(5 %) */
  KVQ_STAT_TOP10 = 4,    /* ... ceil(10 %) */
  KVQ_STAT_ZERO = 5,     /* share of probabilities exactly 0 in fp32 */
  KVQ_STAT_P_ZERO = 6,   /* share of keys nonzero in fp32 but 0 on the MXFP8 P path */
  KVQ_STAT_P_TV = 7,     /* 0.5 sum |p_mx - p| on the MXFP8 P path */
  KVQ_STAT_P_SUM = 8,    /* sum p_mx (the P-path proxy row sum) */
  KVQ_STAT_QK_TV = 9,    /* 0.5 sum |p_qk - p|, p_qk from MXFP8 Q/K */
  KVQ_STAT_QK_AGREE = 10, /* 1 when p_qk and p have the same argmax (first index), else 0 */
  KVQ_N_STATS = 11
};

/*
 * kv_attend_stats -- observer statistics of attention rows (Catnip study,
 * "Catnip Week 10 KV Cache Attention Study", section 实验设计 step 5 with its
 * Structural / Effective / Numerical MXFP8 notes, and section "Q/K 与
 * probability quantization 的影响"). For each query row, p is the fp32
 * softmax of sm_scale * q K^T over all N keys of the cache, K as kv_attend
 * reads it. The MXFP8 P path rounds p to E4M3 with one E8M0 scale per 32
 * consecutive keys (the scale rule of the MXFP8 K window). The MXFP8 Q/K path
 * rotates q and every key by the signed Hadamard transform
 * x -> (x * signs) H / sqrt(D) (H the Sylvester Hadamard matrix of order D)
 * when hadamard_signs is not NULL, rounds both to MXFP8 along D and takes the
 * softmax of their scores (p_qk).
 * q: [batch][q_heads][n_q][D] in q_dtype (F32 or BF16), device; typically a
 *   sample of query rows. hadamard_signs: device float [D] of +-1, or NULL.
 * stats: device float [batch][q_heads][n_q][KVQ_N_STATS], see KVQ_STAT_*.
 * workspace/ws_bytes as kv_attend (it holds every key twice in fp32, as
 * attention reads it and on the MXFP8 Q/K path, and both score rows of
 * every query row: about 8 x B x Hkv x N x D + 8 x B x q_heads x n_q x N
 * bytes).
 * Restrictions (else KVQ_ERR_UNSUPPORTED): D in {32, 64, 128, 256},
 * N <= 1,048,576, batch * q_heads <= 65,535. A row's reference scores are
 * swept in shared memory up to 16,384 keys, longer rows in place in the
 * workspace (slower).
 */
KVQ_API kvq_status kv_attend_stats(const kvq_cache *cache, const void *q, int32_t q_dtype,
                                   int32_t q_heads, int32_t n_q, float sm_scale,
                                   const float *hadamard_signs, float *stats, void *workspace,
                                   size_t *ws_bytes, int32_t *dev_status, kvq_stream_t stream);

/*
 * kv_attend_candidates -- exact attention of each query row over its own
 * candidate keys only (MiniCPM5-2B study, sections 6 and 9): row (b, h, i)
 * attends the n_cand token positions idx[b][h][i][:] (int32, device) and no
 * other key. Lists hold distinct positions in any order. An index outside
 * [0, N) is skipped and flagged KVQ_DEV_INDEX; with validate != 0 duplicate
 * positions are flagged KVQ_DEV_DUP (the output of that row is then invalid).
 * An MXFP8 K window, n_cand > 65,536 and q_heads or batch above 65,535 are
 * not supported (KVQ_ERR_UNSUPPORTED). Other arguments as for kv_attend.
 * Kernel choice: with D = 128, bf16 q, one query row, 8 query heads per KV
 * head, a bf16 window (or none) and 8 x n_cand <= 4096, one pass per
 * (sequence, KV head) covers the union of its 8 query heads' lists, reading
 * each distinct row and K-scale group once and scoring it for all 8 heads on
 * the tensor cores (bf16 operands, the int4 rows rounded once to bf16); it
 * needs workspace for per-slice partials (query it with workspace == NULL).
 * Other shapes run a per-row fp32 kernel and need none.
 */
KVQ_API kvq_status kv_attend_candidates(const kvq_cache *cache, const void *q, int32_t q_dtype,
                                        int32_t q_heads, int32_t n_q, const int32_t *idx,
                                        int32_t n_cand, int32_t validate, float sm_scale,
                                        void *out, int32_t out_dtype, void *workspace,
                                        size_t *ws_bytes, int32_t *dev_status,
                                        kvq_stream_t stream);

/*
 * kv_attend_candidates_topk -- the two-stage form of candidate attention
 * (MiniCPM5-2B study, section 6: a predictor proposes top-C candidates, then
 * the true top-32 inside them is taken by exact score): each query row scores
 * its n_cand listed keys exactly (sm_scale * q . k, keys as kv_attend reads
 * them), keeps the top_k highest (equal scores: the key listed first) and
 * attends exactly over those. q, idx, out as kv_attend_candidates; positions
 * outside [0, N) score -inf (flagged KVQ_DEV_INDEX) and are never kept.
 * selected: device int32 [batch][q_heads][n_q][top_k] receiving the kept
 *   positions in score order (-1 past the valid ones), or NULL.
 * Restrictions: 1 <= top_k <= n_cand <= 4096 (else KVQ_ERR_ARG /
 * KVQ_ERR_UNSUPPORTED); an MXFP8 K window is not supported. No workspace.
 */
KVQ_API kvq_status kv_attend_candidates_topk(const kvq_cache *cache, const void *q,
                                             int32_t q_dtype, int32_t q_heads, int32_t n_q,
                                             const int32_t *idx, int32_t n_cand, int32_t top_k,
                                             float sm_scale, void *out, int32_t out_dtype,
                                             int32_t *selected, int32_t *dev_status,
                                             kvq_stream_t stream);

/*
 * kv_attend_candidates_block -- candidate attention for many query rows
 * (prefill) with one candidate list per block of block_q consecutive query
 * rows of a head. The MiniCPM5-2B study (section 9) found its prefill kernel,
 * which gathered a head's candidate rows again for every query block, slower
 * than dense attention, and names the fix: a block-shared candidate layout
 * with the rows tiled through on-chip memory. Row i of head h of sequence b
 * attends exactly over the keys of list idx[b][h][i / block_q][0 .. n_cand).
 * idx: device int32 [batch][q_heads][ceil(n_q / block_q)][n_cand] of distinct
 *   positions in [0, N) (others are flagged KVQ_DEV_INDEX; such a list's rows
 *   are then invalid). q, out as kv_attend.
 * With D = 128, bf16 q, block_q a multiple of 128 and no MXFP8 K window,
 * every list's K and V rows are gathered once into workspace as bf16 and the
 * rows attend them on the tensor cores; otherwise the fp32 candidate kernel
 * runs with the shared lists (no workspace). workspace/ws_bytes as kv_attend.
 */
KVQ_API kvq_status kv_attend_candidates_block(const kvq_cache *cache, const void *q,
                                              int32_t q_dtype, int32_t q_heads, int32_t n_q,
                                              const int32_t *idx, int32_t n_cand, int32_t block_q,
                                              float sm_scale, void *out, int32_t out_dtype,
                                              void *workspace, size_t *ws_bytes,
                                              int32_t *dev_status, kvq_stream_t stream);

/*
 * kv_attend_region_drop -- the local output ablation the Catnip study
 * recommends ("Catnip Week 10 KV Cache Attention Study", section
 * 当前判断与下一步优化空间: drop sink, drop recent or drop all history,
 * renormalise P, compare the attention output): O over the keys of the regions
 * NOT set in drop_mask only, the softmax renormalised over them.
 * region_bounds: HOST array of n_regions + 1 increasing positions from 0 to N
 * (n_regions <= 16); bit r of drop_mask drops region r (at least one key must
 * remain). q, out, workspace/ws_bytes as kv_attend. The kept keys of every
 * (sequence, KV head) are gathered once to bf16 in workspace and attended on
 * the tensor cores: D = 128, bf16 q and no MXFP8 K window, else
 * KVQ_ERR_UNSUPPORTED.
 */
KVQ_API kvq_status kv_attend_region_drop(const kvq_cache *cache, const void *q, int32_t q_dtype,
                                         int32_t q_heads, int32_t n_q, float sm_scale,
                                         const int32_t *region_bounds, int32_t n_regions,
                                         uint32_t drop_mask, void *out, int32_t out_dtype,
                                         void *workspace, size_t *ws_bytes, int32_t *dev_status,
                                         kvq_stream_t stream);

/*
 * kv_attend_decode_static -- the decode case of kv_attend (one query row per
 * sequence and head, 8 query heads per KV head, D = 128, bf16 or no window)
 * for callers that cannot allocate device memory: a serving runtime that has
 * already handed all free HBM to its KV-cache pool (any further cudaMalloc
 * fails), or a latency-critical caller that cannot afford cudaMalloc's
 * implicit device synchronisation. The pages have no counterpart; it exists
 * only for those callers.
 * Same q / out / dtype / dev_status / stream rules as kv_attend; no
 * workspace argument. The split-K partials go to a scratch array of
 * KVQ_DECODE_STATIC_SCRATCH_BYTES (8 MiB) that the library keeps in device
 * memory on every GPU that loads it, until the process exits. A call whose
 * partials need more (batch * kv_heads above 992 on a
 * 152-SM GPU) returns KVQ_ERR_WORKSPACE and enqueues nothing; other
 * unsupported shapes return KVQ_ERR_UNSUPPORTED. Nothing is allocated, by
 * the library or by any library it calls.
 * The array's device address is looked up (cudaGetSymbolAddress) once per
 * device, with that device current, by the first kv_pack or kv_append on the
 * device, or else by the first call of this entry point; make that first call
 * before any stream capture. The lookup loads the library's decode module on
 * the device (CUDA loads modules lazily by default), and that load is what
 * takes the 8 MiB: a runtime that hands all free HBM to its KV-cache pool
 * should pack (or append to) a cache first, as it must before decoding anyway.
 * If the lookup fails, the call returns KVQ_ERR_CUDA with the CUDA error
 * cleared. The looked-up address is kept for the life of the process: do not
 * use the library across a cudaDeviceReset on that device.
 * Every call reads scratch it wrote itself in the
 * same call, so nothing needs clearing between calls, but all calls share
 * the one array: calls that overlap on the GPU (different streams, no
 * ordering between them) race and corrupt each other's results.
 */
#define KVQ_DECODE_STATIC_SCRATCH_BYTES (8u << 20)
KVQ_API kvq_status kv_attend_decode_static(const kvq_cache *cache, const void *q,
                                           int32_t q_dtype, int32_t q_heads, float sm_scale,
                                           void *out, int32_t out_dtype, int32_t *dev_status,
                                           kvq_stream_t stream);

/*
 * Rotary positions. Pair i of a head (of rotary_dim / 2 pairs) turns by the
 * angle pos * f_i, f_i = base^(-2 i / rotary_dim) before scaling; features past
 * rotary_dim pass through. KVQ_ROPE_HALF pairs features i and
 * i + rotary_dim / 2, KVQ_ROPE_INTERLEAVED features 2i and 2i + 1.
 * Scaling for contexts longer than the trained one:
 *   NONE    f_i as above; the other fields are ignored.
 *   LINEAR  f_i / factor.
 *   BASE    base * factor^(rotary_dim / (rotary_dim - 2)) in place of base
 *           (rotary_dim >= 4).
 *   RAMP    pairs that turn often over the original context keep f_i, pairs
 *           that turn seldom take f_i / factor, linear in i between
 *           floor(x(p0)) and ceil(x(p1)) (both clamped to [0, rotary_dim - 1];
 *           a step behind that pair where they meet),
 *           x(r) = rotary_dim ln(original / (2 pi r)) / (2 ln base) the pair
 *           that makes r turns; the rotation is multiplied by
 *           0.1 ln(factor) + 1.
 *   BANDS   with r = original f_i / (2 pi) turns, w = (r - p0) / (p1 - p0)
 *           clamped to [0, 1]: w f_i + (1 - w) f_i / factor.
 */
typedef enum { KVQ_ROPE_HALF = 0, KVQ_ROPE_INTERLEAVED = 1 } kvq_rope_layout;
typedef enum {
  KVQ_ROPE_NONE = 0,
  KVQ_ROPE_LINEAR = 1,
  KVQ_ROPE_BASE = 2,
  KVQ_ROPE_RAMP = 3,
  KVQ_ROPE_BANDS = 4
} kvq_rope_scaling_kind;

typedef struct kvq_rope_scaling {
  int32_t kind;    /* kvq_rope_scaling_kind */
  double factor;   /* >= 1 */
  double original; /* RAMP, BANDS: tokens of the trained context (> 0) */
  double p0, p1;   /* RAMP: turns kept from / scaled to, p0 > p1 > 0; BANDS: p1 > p0 >= 0 */
} kvq_rope_scaling;

/*
 * The frequency table of kv_rope: turns[i] = f_i / (2 pi) as a 64-bit binary
 * fraction of a turn, so that pos * turns[i] modulo 2^64 is the phase of any
 * position, to |pos| * 2^-53 turns (the entries are made from doubles). turns:
 * HOST array of rotary_dim / 2 entries (the caller copies it to the device
 * once); *amplitude receives the factor on the rotation. scaling may be NULL
 * (NONE). Host only. KVQ_ERR_ARG for an odd or non-positive rotary_dim, one
 * above 256, base <= 1 or a scaling outside the limits above.
 */
KVQ_API kvq_status kvq_rope_turns(int32_t rotary_dim, double base, const kvq_rope_scaling *scaling,
                                  uint64_t *turns, float *amplitude);

/* One tensor of kv_rope: element (b, h, t, d) of the input lies at
 * in[b * stride_b + h * stride_h + t * stride_t + d] (strides in elements);
 * the output is dense [batch][heads][n][head_dim], as the other calls read q
 * and new keys and values. rotate == 0 only copies (values that come out of
 * the same projection). in == out is allowed with the dense strides; other
 * overlaps are not. */
typedef struct kvq_rope_tensor {
  const void *in;
  void *out;
  int32_t heads;
  int32_t rotate;
  int64_t stride_b, stride_h, stride_t;
} kvq_rope_tensor;

/*
 * kv_rope -- rotary positions of up to three tensors (q, k and, copied, v of
 * one projection) in one kernel: y0 = a (x0 cos - x1 sin), y1 = a (x0 sin +
 * x1 cos) per pair, a the amplitude, computed in fp32 and rounded once.
 * tensors: HOST array of n_tensors (1..3) entries, all of `dtype` (F32 or
 * BF16), read before the call returns. positions: device int32 [batch][n], any
 * values (negative ones turn backwards). turns: device copy of kvq_rope_turns'
 * table. inverse != 0 applies the transposed rotation (angle negated, same
 * amplitude): the gradient of the call with respect to its input, and with
 * amplitude 1 what takes a position off a key.
 * rotary_dim: even, 2 <= rotary_dim <= head_dim; head_dim as everywhere.
 * Strides must be >= 0 and multiples of 16 bytes (KVQ_ERR_ALIGN).
 * KVQ_ERR_UNSUPPORTED when batch * n exceeds 2^31 - 1. n == 0 and batch == 0
 * are valid and enqueue nothing.
 */
KVQ_API kvq_status kv_rope(const kvq_rope_tensor *tensors, int32_t n_tensors, int32_t dtype,
                           int32_t batch, int32_t n, int32_t head_dim, int32_t rotary_dim,
                           int32_t layout, const uint64_t *turns, float amplitude,
                           int32_t inverse, const int32_t *positions, int32_t *dev_status,
                           kvq_stream_t stream);

/*
 * kv_attend_tree -- attention of drafted tokens that are not in the cache yet:
 * n_tree (T) tokens per sequence, a forest given by parents: device int32
 * [batch][T]. parents[b][i] is the drafted token that token i follows (below
 * i), -1 when it follows the cache's last token, or -2 when row i holds no
 * token (a smaller tree in a padded batch): such a row's output is left as it
 * was and no row sees it. Token i attends every token of the cache, itself
 * and its ancestors, with K and V of the drafted tokens taken from
 * k_tree, v_tree: [batch][kv_heads][T][D] in tree_dtype (F32 or BF16). A
 * chain (parents[i] = i - 1) is causal attention of T new tokens.
 * q: [batch][q_heads][T][D], out likewise, as kv_attend (their row i is token
 * i). Contents of k_tree, v_tree and q where a row holds no token, and of any
 * drafted token for the rows that do not see it, never reach an output,
 * infinities and NaN included.
 * A parent outside [-2, i), or that is itself no token, is flagged
 * KVQ_DEV_INDEX and its row treated as holding no token.
 * 1 <= T <= KVQ_TREE_MAX (else KVQ_ERR_ARG); an MXFP8 K window rounds Q to
 * MXFP8 for every key, drafted ones included.
 * workspace/ws_bytes as kv_attend.
 * Kernel choice: D = 128, bf16 q and tree and a bf16 window (or none) run on
 * the tensor cores with fp16 operands: the int4 part as code * scale (the
 * scale and the product each rounded once to fp16, 11 bits), q, window and
 * drafted rows converted from bf16 (exact within fp16's normal range, 6e-5 to
 * 65504; of 2^16 and more q and keys count as NaN, values as infinite), products
 * and sums in fp32.
 * Scales of the int4 part belong in that range too: smaller ones keep
 * fewer bits, and 7 * scale above 65504 overflows. Probabilities are rounded to
 * fp16 against a reference near the row's maximum: those of keys more than 15.9
 * nats below the maximum keep fewer than 11 bits, and those of keys more than 23
 * nats below it may be dropped from the output (the sum keeps them).
 * Other shapes run an fp32 kernel (q_heads and batch <= 65,535).
 */
#define KVQ_TREE_MAX 256
KVQ_API kvq_status kv_attend_tree(const kvq_cache *cache, const void *q, int32_t q_dtype,
                                  int32_t q_heads, int32_t n_tree, const void *k_tree,
                                  const void *v_tree, int32_t tree_dtype, const int32_t *parents,
                                  float sm_scale, void *out, int32_t out_dtype, void *workspace,
                                  size_t *ws_bytes, int32_t *dev_status, kvq_stream_t stream);

/*
 * Block summaries: for every block of `block` (32, 64 or 128) consecutive
 * tokens of a cache's int4 part one int8 mean key, from which
 * kv_select_blocks scores the block. There are n_blocks = ceil((N - R) / block)
 * of them; the last may hold fewer tokens.
 *   codes  [batch][kv_heads][cap_blocks][D]  int8, in [-127, 127]
 *   scales [batch][kv_heads][cap_blocks]     float
 * Entries past n_blocks are not read or written.
 */
typedef struct kvq_summary {
  int8_t *codes;
  float *scales;
  int32_t block;
  int32_t cap_blocks;
} kvq_summary;

/*
 * kv_block_summary -- (re)compute the summaries of blocks [first_block,
 * n_blocks) from the cache's K codes and scales. With c the int4 codes of a
 * group and s its scale of a channel: part_g = fl(s * sum c) per 32-token
 * group, the groups' parts added in order in fp32, mean = fl(sum / tokens),
 * scale = fl(max over D of |mean| / 127), code = rint(fl(mean / scale)), ties
 * to even, held to [-127, 127] (a subnormal scale is rounded coarsely; 0 for a
 * zero scale): integers and single fp32 roundings, so the result does not
 * depend on the order of the work. After kv_append moved
 * groups out of the window, the blocks from floor(old cut / block) on are
 * new; first_block >= n_blocks enqueues nothing.
 * KVQ_ERR_ARG: block not 32, 64 or 128, first_block < 0; KVQ_ERR_WORKSPACE:
 * cap_blocks < n_blocks.
 */
KVQ_API kvq_status kv_block_summary(const kvq_cache *cache, const kvq_summary *summary,
                                    int32_t first_block, int32_t *dev_status,
                                    kvq_stream_t stream);

/*
 * kv_block_values -- the mean keys that the summaries of blocks [first_block,
 * n_blocks) stand for, code * scale: values, device float
 * [batch][kv_heads][n_blocks - first_block][D]. Errors as kv_block_summary.
 */
KVQ_API kvq_status kv_block_values(const kvq_cache *cache, const kvq_summary *summary,
                                   int32_t first_block, float *values, int32_t *dev_status,
                                   kvq_stream_t stream);

/*
 * kv_select_blocks -- for each query token of each KV head the top_k blocks by
 * a cheap score. Each query row is rounded to int8 (scale s_q = fl(max|q| /
 * 127), code = rint(fl(q / s_q)) held to [-127, 127]); a block's score for a head is
 * fl(fl(s_q * s_b) * d), d the integer product of the codes, and its score
 * for the KV head the largest over the query heads that share it. Equal
 * scores: the lower block first. The first n_sink blocks are always taken
 * (before the others, n_sink <= top_k). Every step is exact or a single fp32
 * rounding, so the choice is the same whatever the order of the work.
 * q: [batch][q_heads][n_q][D] in q_dtype (F32 or BF16), finite.
 * The summaries of all n_blocks blocks must be there (kv_block_summary, again
 * for the new blocks after appends).
 * selected: device int32 [batch][kv_heads][n_q][top_k], the chosen blocks in
 * increasing order, then -1 when the cache has fewer than top_k blocks.
 * workspace/ws_bytes as kv_attend. KVQ_ERR_UNSUPPORTED for q_heads / kv_heads
 * above 64, batch * kv_heads * n_q above 65,535.
 */
KVQ_API kvq_status kv_select_blocks(const kvq_cache *cache, const kvq_summary *summary,
                                    const void *q, int32_t q_dtype, int32_t q_heads, int32_t n_q,
                                    int32_t top_k, int32_t n_sink, int32_t *selected,
                                    void *workspace, size_t *ws_bytes, int32_t *dev_status,
                                    kvq_stream_t stream);

/*
 * kv_attend_blocks -- exact attention of each query token over the tokens of
 * its listed blocks and the whole window. selected: device int32
 * [batch][kv_heads][n_q][top_k] as kv_select_blocks writes it (any list of
 * increasing blocks in [0, n_blocks), closed by -1 entries, may be passed).
 * All query heads of a KV head share a list. An entry outside the blocks
 * (other than -1) is skipped and flagged KVQ_DEV_INDEX; one that does not
 * exceed the entry before it is skipped and flagged KVQ_DEV_DUP (the list's
 * rows are then invalid). Entries past the n_blocks-th are not looked at (a
 * valid list holds -1 there). Rows with no key at all (no window, an empty
 * list) are zero; a row with an infinite q has no defined value (NaN or zero).
 * q, out, workspace/ws_bytes as kv_attend.
 * Kernel choice: D = 128, bf16 q, a bf16 window (or none) and at most 8 query
 * heads per KV head run the decode kernels over the listed blocks; other
 * shapes run an fp32 kernel (q_heads and batch <= 65,535). The decode kernels
 * round q times the K scales, the int4 values and the probabilities to fp16, the
 * last against a reference near the row's maximum: those of keys more than 14.5
 * nats below the maximum may keep fewer than 11 bits, and those of keys more than
 * 21 nats below it may be dropped from the output.
 */
KVQ_API kvq_status kv_attend_blocks(const kvq_cache *cache, const void *q, int32_t q_dtype,
                                    int32_t q_heads, int32_t n_q, const int32_t *selected,
                                    int32_t top_k, int32_t block, float sm_scale, void *out,
                                    int32_t out_dtype, void *workspace, size_t *ws_bytes,
                                    int32_t *dev_status, kvq_stream_t stream);

/*
 * The paged cache: requests of different lengths that come and go, each in a slot.
 * Request s holds lengths[s] = L tokens. With W = window, the first
 *   cut(L) = 32 * floor((L - W) / 32) for L >= W, else 0
 * tokens are int4 groups (the kv_pack rule) in pages of `page` tokens taken from a
 * pool, and the tokens [cut, L), between W and W + 31 once L >= W, are floats in the
 * slot's window, a ring of T = floor((W + 63) / 32) tiles of 32 rows: token p lies in
 * row p % 32 of tile (p / 32) % T. What a token is stored as depends on its request's
 * tokens alone, not on the steps they came in: every value is first rounded to the
 * window's type and the groups are made from the rounded values.
 *
 * kvq_page_state is shared by the caches of all layers of a model:
 *   table      [slots][max_pages] int32: entry j of row s is the page that holds tokens
 *              [j * page, (j + 1) * page) of request s below cut; entries behind a
 *              request's pages hold nothing.
 *   lengths    [slots] int32
 *   free_pages [n_pages] int32: a stack of the pages no request holds, n_free[0] of them
 *              (the rest of the array is scratch); n_free: 4 int32, only the first used.
 * An empty state has lengths 0, n_free[0] = n_pages and free_pages any permutation of
 * the pages. The arrays may be saved and restored by the caller, all together.
 * Calls on a state and its caches are ordered by the caller (one stream, or events): a
 * step's kv_page_tables and kv_append_pages do not overlap calls that read the lengths,
 * pages or windows. Calls that only read may overlap, with a workspace each.
 *
 * kvq_paged_cache adds one layer's memory, laid out for the attention kernel:
 *   pool  [n_pages][kv_heads][page / 32][40 * D] bytes: one record per 32-token group
 *         and head, so that every group is one copy:
 *           K codes  16 D bytes, [32][D/2] as in kvq_cache
 *           K scales 4 D bytes, float of channel (D/4) t + 8 i + k (t < 4, i < D/32, k < 8)
 *                    at [2 i + (k >> 1 & 1)][t][2 (k & 1) + (k >> 2)]
 *           V codes  16 D bytes: words of 8 codes + 8, word (m, g, t, f), m < 2, g < 8, t < 4,
 *                    f < D/16; nibbles from the lowest: tokens x, x + 8 of feature y, tokens x,
 *                    x + 8 of feature y + 8, the same of token x + 1, x = 16 m + 2 t,
 *                    y = 16 f + g; at [m][f / c][g][t][f % c], c = 4 (2 when D % 64 != 0)
 *           V scales 4 D bytes, float of (token, 32-feature block b) at
 *                    [token / 8][token % 8 / 2][b][token % 2]
 *   ring  [slots][kv_heads][T][2][32 * D] elements of win_dtype (F32 or BF16), K then V:
 *           K of (row r, channel (D/4) t + 8 i + k) at [r][i ^ x][t][2 (k & 3) + (k >> 2)],
 *             x = r & 1 when D % 64 == 0, else 0
 *           V of (row r, feature 32 b + 8 j + g) at [r / 16][r / 8 % 2][b][g][r % 8 / 2][j][r % 2]
 */
typedef struct kvq_page_state {
  int32_t slots;     /* 1 .. KVQ_PAGES_MAX_SLOTS */
  int32_t n_pages;   /* of the pool, 1 .. 2^28 */
  int32_t page;      /* tokens: 32, 64 or 128 */
  int32_t max_pages; /* of one request */
  int32_t window;    /* W, 0 .. 65,536 */
  int32_t *table;
  int32_t *lengths;
  int32_t *free_pages;
  int32_t *n_free;
} kvq_page_state;

typedef struct kvq_paged_cache {
  kvq_page_state state;
  int32_t kv_heads; /* 1 .. 65,535 */
  int32_t head_dim; /* 32 .. 256, a multiple of 32 */
  int32_t win_dtype;
  uint8_t *pool;
  void *ring;
} kvq_paged_cache;

#define KVQ_PAGES_MAX_SLOTS 8192

/* Sizes in bytes (host only; pointers are not read): sizes[0..5] = table, lengths,
 * free_pages, n_free, pool, ring. KVQ_ERR_ARG for a shape outside the limits above or a
 * request that could hold more than 2^31 - 1 tokens. */
KVQ_API kvq_status kvq_paged_sizes(const kvq_paged_cache *cache, size_t sizes[6]);

/* What kv_page_tables makes of one step: device arrays of the caller's, written by it and
 * read by kv_append_pages (and by the caller).
 *   offsets   [slots + 1]: first row of each request's new tokens in the step's tensors
 *             (sums above 2^30 are 2^30)
 *   before    [slots], after [slots]: the requests' lengths
 *   row_slot  [rows]: the request of each row, -1 for a row of none
 *   positions [rows]: its token's position (0 for a row of none); what kv_rope takes
 *   work      [cap_work][8]: of every 32-token group the step writes, in the pages or in
 *             the windows: slot, group, the page it goes to (-1: the window), its
 *             request's before, after and first row, and two unused;
 *             cap_work >= kvq_page_work(state, rows)
 *   counts    [4]: pages free after the step, groups in work, and scratch that has to
 *             be zero before the first call (it is left zero)
 */
typedef struct kvq_page_plan {
  int32_t rows;
  int32_t cap_work;
  int32_t *offsets, *before, *after, *row_slot, *positions, *work, *counts;
} kvq_page_plan;

/* Entries `work` needs for a step of `rows` token rows; 0 for an invalid state or rows
 * outside [0, 2^28]. */
KVQ_API int32_t kvq_page_work(const kvq_page_state *state, int32_t rows);

/*
 * kv_page_tables -- the tables of one step, built on the GPU from the requests' lengths.
 * n_new: device int32 [slots]: tokens that each request adds, 0 for one that rests, -1
 * for one that ends: its pages go back and its length becomes 0. The step's tensors hold
 * the new tokens of the requests one behind the other in slot order, `plan->rows` rows
 * in all; rows behind the last request's belong to none.
 * The pages of ended requests go on top of the free ones (in slot order, each request's
 * in table order) and requests that grow take theirs from the top (in slot order). A
 * request whose pages are not there (the sum of the pages asked for by it and the ones
 * before it exceeds the free ones, or max_pages is exceeded) is flagged KVQ_DEV_PAGES
 * and stays as it was; its rows belong to none. A request with n_new below -1, more new
 * tokens than rows are left, or a length that its table cannot hold is flagged
 * KVQ_DEV_INDEX and stays as it was.
 * advance != 0: lengths and the free pages become what they are after the step, as the
 * steps of a model need it (once a step, before the layers' kv_append_pages). advance ==
 * 0 looks ahead: the plan is the one the step would have (counts[0] >= 0 pages would be
 * left), and only scratch of the state is written.
 */
KVQ_API kvq_status kv_page_tables(const kvq_page_state *state, const int32_t *n_new,
                                  const kvq_page_plan *plan, int32_t advance,
                                  int32_t *dev_status, kvq_stream_t stream);

/*
 * kv_append_pages -- the new tokens' keys and values into one layer's pages and windows,
 * as the plan of kv_page_tables says; whole groups that leave the windows are quantized.
 * k_new, v_new: in_dtype (F32 or BF16), element (row, head, d) at [row * stride_row +
 * head * stride_head + d] (strides in elements, multiples of 16 bytes, 0 .. 2^31 - 1: rows of
 * a projection are read in place). Rows of none are not read. May be called again with the
 * same plan, for other layers or, while no token of the step took the window row of
 * an older one that moved (steps of one token never do), for the same layer.
 * A page outside the pool is flagged KVQ_DEV_INDEX and not written.
 */
typedef struct kvq_page_rows {
  const void *k_new, *v_new;
  int64_t k_stride_row, k_stride_head, v_stride_row, v_stride_head;
} kvq_page_rows;
KVQ_API kvq_status kv_append_pages(const kvq_paged_cache *cache, const kvq_page_plan *plan,
                                   const kvq_page_rows *rows, int32_t in_dtype,
                                   int32_t *dev_status, kvq_stream_t stream);

/*
 * kv_page_values -- keys and values of listed tokens as attention reads them: code * scale,
 * or the window's value, rounded to out_dtype (F32 or BF16). row_slot, positions: device
 * int32 [n_rows]; k, v: [n_rows][kv_heads][D]. A row with slot -1 is left as it was; one
 * with another slot that does not exist, or a position outside the request, is flagged
 * KVQ_DEV_INDEX and left as it was. n_rows <= 2^28.
 */
KVQ_API kvq_status kv_page_values(const kvq_paged_cache *cache, const int32_t *row_slot,
                                  const int32_t *positions, int32_t n_rows, void *k, void *v,
                                  int32_t out_dtype, int32_t *dev_status, kvq_stream_t stream);

/*
 * kv_attend_pages -- attention of new tokens, one query row each, over their requests'
 * pages and windows. q, out: [n_rows][q_heads][D]. row_slot: device int32 [n_rows], the
 * request of each row, or NULL for row i = request i (n_rows <= slots). positions: device
 * int32 [n_rows]: row i attends the tokens [0, positions[i]] of its request, so that
 * several new tokens of one request each see the ones before them; NULL: all tokens of
 * the request. Lengths are read on the device: a captured call serves every later step.
 * A row with slot -1 is left as it was (a batch padded to a captured size); one of a
 * request without tokens is zero. A slot outside [-1, slots), a length that the table
 * cannot hold or a position outside the request is flagged KVQ_DEV_INDEX and the row left
 * as it was; a page outside the pool is flagged KVQ_DEV_INDEX and its tokens skipped.
 * workspace/ws_bytes as kv_attend (the size depends on n_rows, q_heads and the cache's shape
 * alone). n_rows <= 65,535; 0 rows are valid.
 * Kernel choice: D = 64 or 128 with BF16 windows runs on the tensor cores, other shapes an
 * fp32 kernel. Either reads a request's cache once for every row and every eight query
 * heads of a KV head. On the tensor cores:
 *   Roundings to 11 bits, fp16's: q * sm_scale * log2(e), F32 q too; a K scale; their
 *   product (times 4 or 1/4); a probability; a V scale; their product. In the window the
 *   rounded q is used as well, probabilities keep 15 bits, keys and values all. Sums are fp32.
 *   q * sm_scale * log2(e), a K scale and their product belong below 2^14 (either factor
 *   below 2^-12 has an absolute error of up to 2^-23).
 *   The reference of the probabilities puts the largest product of a key's probability and
 *   its 32-token group's largest V scale near 2^7, whatever the size of the values: keys
 *   whose product lies more than 11.8 nats below the largest may keep fewer bits, as may V
 *   scales below 2^-10 of their group's largest, and keys more than 18 nats below may be
 *   dropped from the output (the sum keeps them).
 *   The largest of 32 features of a token's values in the int4 part belongs between 2.4e-17
 *   and 5e17 (or is zero): smaller ones keep fewer bits, and larger or infinite ones make those
 *   32 features NaN in the rows that attend the token.
 *   Infinite keys and values in the window give what the formula gives (a score of -inf
 *   leaves its token out, one of +inf makes the row NaN, an infinite value is infinite in the
 *   output), but where q rounds to zero.
 * Tokens that a row does not attend have no part in it, whatever they hold (but that the
 * tokens of a group share its K scales). A row whose scores are all -inf is zero.
 */
KVQ_API kvq_status kv_attend_pages(const kvq_paged_cache *cache, const void *q, int32_t q_dtype,
                                   int32_t q_heads, int32_t n_rows, const int32_t *row_slot,
                                   const int32_t *positions, float sm_scale, void *out,
                                   int32_t out_dtype, void *workspace, size_t *ws_bytes,
                                   int32_t *dev_status, kvq_stream_t stream);

/* Number of kernel launches the last successful call on this thread enqueued. */
KVQ_API int32_t kvq_last_launch_count(void);

/* Name of the kernel family the last successful call on this thread used
 * ("pack", "decode", "chunk_bf16", "chunk_mxfp8", "generic", "candidates",
 * "rope", "tree_tensor", "tree_rows", "block_summary", "block_values",
 * "select_blocks", "blocks_decode", "blocks_rows", "page_tables", "append_pages",
 * "page_values", "pages_tensor", "pages_rows", ...); a static string. */
KVQ_API const char *kvq_last_path(void);

/*
 * Test hook: bound every mbarrier wait of the next launches on this thread to
 * `wait_limit_ns` nanoseconds (0 restores the default of one second), and,
 * when drop_item >= 0, make the loader of the decode kernel (over listed
 * blocks too) and of the bf16 kv_pack kernel skip the copy of that work item,
 * and the tree kernel withhold the keys of that one (row block * tiles + tile),
 * so that the wait on it can only run out. Used by the failure tests.
 */
KVQ_API void kvq_debug_set(uint32_t wait_limit_ns, int32_t drop_item);

/*
 * 1 when this library was built with KVQ_DEBUG (libkvq_debug.so), else 0. In
 * that build every kernel checks each global address range it derives from
 * its indices (a row, a chunk, a bulk copy) against the device buffers the
 * call passed -- the cache's arrays at the sizes its shape gives, q, the
 * outputs, index lists and the workspace at the size given in *ws_bytes --
 * and, for a range outside them, sets KVQ_DEV_BOUNDS in *dev_status and
 * leaves the access out (a load reads zeros, a store is dropped, a bulk copy
 * is neither issued nor waited for), so a wrong index is reported instead of
 * faulting. TMA tile copies are bounded by their tensor maps. The checks cost
 * time; the outputs of a call that reports no error are those of the other
 * build.
 */
KVQ_API int32_t kvq_debug_checks(void);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_H */
