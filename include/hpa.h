/*
 * hpa.h -- load-balanced split-KV GQA decode attention for NVIDIA GB300 (sm_103a).
 *
 * C ABI.  Every pointer argument named *_dev is a device pointer allocated by
 * the caller; the library never allocates or frees memory and never
 * synchronises a stream.  All work is enqueued on the caller's stream in
 * stream order, so the three calls below can be captured in a CUDA graph.
 *
 * The method (sources are web pages, cited by title and section):
 *   [Notes §3.1]  "Hy3 Preview AI Infra 推理优化精读笔记", §3.1 "Attention：动态切分和
 *                 负载均衡" -- cut every request's KV into uniform tiles, join all
 *                 tiles into one stream, give each CTA an equal (or +1) budget of
 *                 it, build a task map before the step, have the attention
 *                 kernel take its tiles from the map, merge split results in a
 *                 combine kernel.  Worked example: lengths 1024/5120/2048, tile
 *                 512 -> 2/10/4 tiles, 4 CTAs x 4 tiles, the long request spans
 *                 CTAs.
 *   [HPC-Ops §二.1] "腾讯混元AI Infra进化：HPC-Ops推理核心算子全面升级", §二.1
 *                 "Attention：动态调度负载均衡" -- a Task Assign module builds the
 *                 map once per inference step; the attention kernel of every
 *                 layer reads it; a Combine kernel merges the split-KV results.
 *   [Stack §二.1]  "大模型推理性能优化新范式：Hy3架构下的全栈优化技术拆解", §二.1 --
 *                 budget base = T / C, the first T % C CTAs get one more tile.
 *   [Notes §2]    same notes page, §2 -- 64 query heads, 8 KV heads, head dim 128.
 *
 * Units used below: B requests; L_r the KV length of request r (counting its
 * q_len new tokens); T the total number of tiles; C = num_ctas, the number of
 * partitions of the tile stream; each partition runs once per KV head, so
 * the attention grid has C x Hkv CTAs.
 *
 * Error behaviour: every call validates its host-visible arguments first and
 * returns a negative HPA_ERR_* code without launching anything when one is
 * wrong.  Problems only the device can see (sequence lengths, page ids, a
 * task map built for another shape or corrupted after it was built, a
 * pipeline wait that ran past its time bound) set bits in the task map's
 * status word (int32 word 6 of the map, HPA_STATUS_*); the attention kernel
 * then does no work for what it cannot trust and the combine kernel writes
 * NaN to every output element, so a bad step cannot pass silently.  The
 * kernels check every index they take from the map before following it, so
 * a corrupted map is reported rather than read or written out of bounds.
 * Asynchronous CUDA faults surface at the caller's next sync.
 */
#ifndef HPA_H
#define HPA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t (the runtime's stream handle); NULL is the legacy default stream. */
typedef struct CUstream_st *hpa_stream_t;

/* ---- return codes (host) ---- */
#define HPA_OK 0
#define HPA_ERR_INVALID (-1)     /* NULL pointer or out-of-range size; nothing launched */
#define HPA_ERR_UNSUPPORTED (-2) /* a shape these kernels do not implement */
#define HPA_ERR_WORKSPACE (-3)   /* task map buffer smaller than required */
#define HPA_ERR_ALIGN (-4)       /* a pointer lacks the alignment stated below */
#define HPA_ERR_CUDA (-5)        /* a CUDA runtime call or launch failed */
#define HPA_ERR_NOALLOC_CAPACITY (-6) /* the problem needs more than the fixed no-alloc scratch */

/* ---- status bits written by the kernels into task map word 6 ---- */
#define HPA_STATUS_BAD_SEQLEN 1 /* some L_r < 1 (plan) or L_r < q_len (attention) */
#define HPA_STATUS_MISMATCH 2   /* map built for another B / num_ctas / tile */
#define HPA_STATUS_BAD_PAGE 4   /* a page id outside [0, num_pages); page 0 was read instead */
#define HPA_STATUS_TIMEOUT 8    /* a shared-memory pipeline wait exceeded ~2 s; CTA gave up */
#define HPA_STATUS_OVERFLOW 16  /* total tile count does not fit int32; hpa_plan_window and
                                   hpa_evict_select: a length whose positions do not */
#define HPA_STATUS_BAD_MAP 32   /* a malformed map: a partition's segment range, a segment row
                                   (request, owner, tile range) or a request's segment range
                                   out of bounds; the row was skipped, never followed */
#define HPA_STATUS_BAD_BUDGET 64 /* hpa_evict_select: a budget below 1, below sinks + recent of a
                                    longer request, or beyond kept_stride */
#define HPA_STATUS_NO_PAGES 128 /* hpa_assign_pages: a request asked for more pages than are free */

/* ---- KV element types ---- */
#define HPA_KV_BF16 0 /* bfloat16 */
#define HPA_KV_E4M3 1 /* OCP FP8 E4M3 code; value = code * scale[kv head] */
#define HPA_KV_E2M1 2 /* 4-bit: OCP FP4 E2M1 code; value = code * block scale * scale[kv head],
                         with an E4M3 block scale for every 16 elements of a row */

/* A 4-bit pool holds, for each page and KV head, HPA_E2M1_PAGE_BYTES bytes: 64 rows of 64 bytes
 * of codes (byte i of a row: element 2i in the low nibble, 2i + 1 in the high one), then the
 * block scales, 64 rows of 8 bytes (byte j of a row: elements [16j, 16j + 16)).  Taken by
 * hpa_decode_attn, hpa_decode_attn_window, hpa_decode_attn_combine_noalloc, hpa_store_qkv and
 * hpa_default_num_ctas(_window); every other call with a kv_dtype refuses it. */
#define HPA_E2M1_PAGE_BYTES 4608

/*
 * Task map: an opaque int32 blob in device memory, written by hpa_plan or
 * hpa_plan_static and read by hpa_decode_attn and hpa_combine.  One map
 * serves every layer of a decode step ([HPC-Ops §二.1]).  Layout (int32 words):
 *   [0,16)  header: T, base, rem, C, B, S (segments), status, tile, kind
 *           (0 dynamic / 1 static / 2 token-weighted / 3 window), splits, S_cap,
 *           then window, sinks, q_len of a window map, and two words that
 *           hpa_key_weights uses while it runs (0 before and after)
 *   lens[B]            copy of the sequence lengths
 *   cu_tiles[B+1]      exclusive running sum of tiles per request
 *   cta_begin[C+1]     first stream tile of each partition
 *   cta_seg[C+1]       first segment of each partition
 *   seg_off[B+1]       first segment of each request
 *   (padding to a multiple of 4 words)
 *   seg[S_cap][4]      {request, tile_lo, tile_hi, partition}; tiles are
 *                      request-local, [tile_lo, tile_hi); unused rows are -1.
 *                      In a window map tiles count the pages the window reaches.
 * A segment is the part of one request that one partition owns.
 */

/* Bytes of the dynamic task map for B requests over num_ctas partitions
 * (segment capacity B + num_ctas - 1).  0 if an argument is out of range. */
size_t hpa_taskmap_bytes(int32_t B, int32_t num_ctas);

/* Segment capacity of the dynamic map: B + num_ctas - 1 (0 if out of range).
 * partial_o needs capacity * q_len * Hq * d floats, partial_lse capacity *
 * q_len * Hq floats. */
int32_t hpa_max_segments(int32_t B, int32_t num_ctas);

/* Static comparator: num_ctas = B * splits partitions, capacity B * splits. */
int32_t hpa_static_num_ctas(int32_t B, int32_t splits);
size_t hpa_static_taskmap_bytes(int32_t B, int32_t splits);

/* Partitions per KV head that fill the current device once with the kernel
 * hpa_decode_attn picks for this shape: hpa_default_num_ctas_mma up to 16
 * query rows per KV head (G * q_len), hpa_default_num_ctas_tc above; for 4-bit
 * pages that of their kernels.  Returns <= 0 on a CUDA error or unsupported
 * arguments. */
int32_t hpa_default_num_ctas(int32_t Hq, int32_t Hkv, int32_t q_len, int32_t kv_dtype);

/* Partitions per KV head for hpa_decode_attn_mma: SMs x resident CTAs per SM /
 * (Hkv x query-row groups), at least 1, where a group is 16 of the G * q_len
 * query rows of a KV head. */
int32_t hpa_default_num_ctas_mma(int32_t Hq, int32_t Hkv, int32_t q_len, int32_t kv_dtype);

/*
 * hpa_plan -- the Task Assign step ([Notes §3.1] steps 1-4, [HPC-Ops §二.1],
 * [Stack §二.1]).  One device kernel:
 *   n_r = ceil(L_r / tile); cu_tiles = exclusive scan of n_r; T = cu_tiles[B];
 *   base = T / C, rem = T % C; partition c owns stream tiles
 *   [c*base + min(c, rem), (c+1)*base + min(c+1, rem)); its range is split at
 *   request boundaries into segments.
 * seq_lens_dev: int32[B] device, L_r >= 1.  tile: a positive multiple of 64
 * (the page size).  num_ctas >= 1 (more partitions than tiles leaves the
 * surplus empty).  taskmap_dev: >= hpa_taskmap_bytes(B, num_ctas) bytes,
 * 16-byte aligned.
 */
int hpa_plan(const int32_t *seq_lens_dev, int32_t B, int32_t tile, int32_t num_ctas,
             void *taskmap_dev, size_t taskmap_bytes, hpa_stream_t stream);

/*
 * hpa_plan_weighted -- the token-weighted variant of hpa_plan (a reading the
 * pages leave open: a partial last tile costs its fill, not a whole tile).
 * Same stream, same contiguous partitions and map format (kind 2), with
 * budgets in keys: with K = sum L_r, P_t the keys before stream tile t and w_t
 * the keys in it, tile t goes to partition floor(C (2 P_t + w_t) / (2 K)) --
 * the partition whose equal share of the key stream holds the tile's middle
 * key.  Header words base / rem hold K / C and K % C.  Sizes as hpa_plan;
 * requires (B + C) small enough for the plan's 40 KB shared-memory staging
 * (about B + C <= 3400), else HPA_ERR_UNSUPPORTED; K > 2^40 sets
 * HPA_STATUS_OVERFLOW.
 */
int hpa_plan_weighted(const int32_t *seq_lens_dev, int32_t B, int32_t tile, int32_t num_ctas,
                      void *taskmap_dev, size_t taskmap_bytes, hpa_stream_t stream);

/*
 * hpa_plan_static -- the static split-KV comparator the pages contrast the
 * method with ([Notes §3.1] 问题): request r is cut into min(splits, n_r)
 * contiguous chunks of near-equal tile counts (the first n_r % chunks get
 * one more); partition r * splits + s owns chunk s, or nothing.  Same map
 * format, so the same attention and combine kernels run it.
 * taskmap_dev: >= hpa_static_taskmap_bytes(B, splits) bytes.
 */
int hpa_plan_static(const int32_t *seq_lens_dev, int32_t B, int32_t tile, int32_t splits,
                    void *taskmap_dev, size_t taskmap_bytes, hpa_stream_t stream);

/*
 * hpa_plan_window -- the dynamic plan for attention with a sliding window and sink
 * tokens (the pages have no counterpart to it).  With W = window >= 1 and
 * S = sinks >= 0, token j of request r, at position a = L_r - q_len + j, sees key
 * i <= a when i > a - W or i < S.  The map (kind 3) cuts into tiles only the pages
 * that hold such a key: those of the sinks and those from position
 * max(0, L_r - q_len + 1 - W) on, joined without the pages between them; so the
 * budget of a partition is what it reads, whatever the length.  window, sinks and
 * q_len are kept in the map, and the calls that read it follow them:
 * hpa_decode_attn_window, hpa_combine and hpa_key_weights.  The other attention
 * calls report such a map as HPA_STATUS_BAD_MAP.  L_r < q_len sets
 * HPA_STATUS_BAD_SEQLEN, L_r > 2^31 - 65 HPA_STATUS_OVERFLOW.  Sizes as hpa_plan; a
 * tile of 64 (one page) balances short windows best.
 */
int hpa_plan_window(const int32_t *seq_lens_dev, int32_t B, int32_t q_len, int32_t window,
                    int32_t sinks, int32_t tile, int32_t num_ctas, void *taskmap_dev,
                    size_t taskmap_bytes, hpa_stream_t stream);

/*
 * hpa_decode_attn -- the split-KV attention kernel ([Notes §3.1] steps 4-5).
 * Up to 16 query rows per KV head (G * q_len <= 16: one new token at any
 * GQA ratio up to 16, or two at 8 heads per KV head) it runs the kernel
 * described here, which is the one that streams the KV at the copy peak
 * there; above 16 rows (MTP with several draft tokens) it runs the same step
 * as hpa_decode_attn_tc, which takes all rows in one pass.  Size num_ctas with
 * hpa_default_num_ctas, which follows the same choice.  hpa_decode_attn_mma
 * runs the kernel described here at any row count.
 *
 * Grid num_ctas x Hkv x ceil(G q_len / 16); the CTA of (partition c, KV
 * head h, row group z) walks c's segments in order and, for each, computes
 * over the segment's keys
 *   s = sm_scale * q . k,  m = max s,  l = sum exp(s - m),  o = sum exp(s - m) v / l
 * for query rows [16 z, 16 z + 16) of the G * q_len rows (row j * G + g:
 * query head g of the G = Hq / Hkv heads of h, token j of the q_len new ones,
 * which sees keys [0, L_r - q_len + 1 + j)), and writes
 *   partial_o[seg][j][head][d] = o,  partial_lse[seg][j][head] = m + ln l
 * (natural log; -inf and o = 0 for a row that sees no key of the segment).
 *
 * q_dev:        bf16 [B][q_len][Hq][d], 16-byte aligned.
 * k_pool_dev, v_pool_dev: [num_pages][Hkv][page_size][d] of bf16 or E4M3
 *               bytes, 16-byte aligned (read with TMA tensor copies).
 * k_scale_dev, v_scale_dev: fp32 [Hkv] for HPA_KV_E4M3 and HPA_KV_E2M1, ignored for bf16.
 *               With E4M3 pages the products run in f16: each query row is
 *               scaled by a power of two that puts its largest |element| in
 *               [2^14, 2^15) (taken back out of the scores), so any finite bf16
 *               query converts exactly, down to 2^-28 of its row's largest.
 *               With HPA_KV_E2M1 pages (layout above, pools 16-byte aligned) kernels of
 *               their own run at every row count, in passes of up to 32 rows (up to 32 rows
 *               per KV head 4-bit pages are faster than E4M3 ones, or level; above, the second
 *               pass over a long cache takes up to 1.6 times E4M3's time), with the
 *               precision of E4M3 pages here: codes times block scales and queries enter the
 *               products exactly, in f16, sums and softmax statistics are fp32 and the
 *               probabilities are rounded to f16 (2^-11 of each; those below 2^-21 of the
 *               row's largest to 2^-32 of that one).  NaN block scales of keys that a row does
 *               not see do not reach it; a row that sees one is NaN in the result, of a value's
 *               block in its 16 elements, of a key's in all of them and in the lse, as is a row
 *               with a score of NaN or +inf (its partial lse is +inf); scores of -inf are
 *               those of keys that are not seen.
 * page_indptr_dev: int32 [B+1]; page_indices_dev: int32; key i of request r
 *               is slot i % page_size of page page_indices[page_indptr[r] + i / page_size].
 *               page_indptr has to be right when the kernel reads it: no call is told how
 *               many indices there are (page ids themselves are checked).
 * Supported: d == 128, page_size == 64, Hq % Hkv == 0, (Hq / Hkv) * q_len <= 64,
 *               num_pages * Hkv < 2^31.  Row groups past the first re-read the
 *               pages (through L2 when they run together).
 * taskmap_dev:  a map from hpa_plan / hpa_plan_static for these B and num_ctas.
 * partial_o_dev: fp32, >= (B + num_ctas - 1) * q_len * Hq * d, 16-byte aligned (one
 *               row per segment; no map has more than B + num_ctas - 1 segments);
 * partial_lse_dev: fp32, >= (B + num_ctas - 1) * q_len * Hq.
 */
int hpa_decode_attn(const void *q_dev, const void *k_pool_dev, const void *v_pool_dev,
                    int32_t kv_dtype, const float *k_scale_dev, const float *v_scale_dev,
                    int64_t num_pages, const int32_t *page_indptr_dev,
                    const int32_t *page_indices_dev, int32_t page_size, int32_t B,
                    int32_t q_len, int32_t Hq, int32_t Hkv, int32_t d, float sm_scale,
                    void *taskmap_dev, int32_t num_ctas, float *partial_o_dev,
                    float *partial_lse_dev, hpa_stream_t stream);
int hpa_decode_attn_mma(const void *q_dev, const void *k_pool_dev, const void *v_pool_dev,
                        int32_t kv_dtype, const float *k_scale_dev, const float *v_scale_dev,
                        int64_t num_pages, const int32_t *page_indptr_dev,
                        const int32_t *page_indices_dev, int32_t page_size, int32_t B,
                        int32_t q_len, int32_t Hq, int32_t Hkv, int32_t d, float sm_scale,
                        void *taskmap_dev, int32_t num_ctas, float *partial_o_dev,
                        float *partial_lse_dev, hpa_stream_t stream);

/*
 * hpa_decode_attn_tc -- the same split-KV attention step ([Notes §3.1] steps
 * 4-5), computed by a kernel that runs both products on the 5th-generation
 * tensor cores (tcgen05.mma with accumulators in tensor memory).  Grid
 * num_ctas x Hkv: one CTA covers all G * q_len query rows of its KV head
 * (up to 64) in a single pass over the keys, where hpa_decode_attn makes one
 * pass per group of up to 16 rows.  It pays for MTP with more than 16 rows per KV
 * head, and hpa_decode_attn runs it there (on the E4M3 MTP workload at 64/8
 * heads: 1.9x the mma.sync kernel at q_len 3-4, 2.7x at q_len 6, 2.6x at
 * q_len 8).  With up to 16 rows, or with many short segments per partition
 * (hundreds of short requests), the mma.sync kernel is as fast or faster.
 * Arguments, layouts, supported shapes, outputs and errors are exactly those
 * of hpa_decode_attn; the partials feed hpa_combine unchanged.  E4M3 pages
 * enter the MMA as 8-bit operands; the query rows and the probabilities are
 * each carried as two E4M3 terms (about 8 significant bits, as bf16).  Each
 * query row is scaled by a power of two (its largest element into [128, 256))
 * and its residual term by a fixed 16, so rows of any bf16 magnitude are
 * carried exactly as long as their elements lie within about 2^-12 of the
 * row's largest; smaller elements lose bits and those below about 2^-21 of it
 * are dropped (hpa_decode_attn_mma keeps bf16 precision down to 2^-28).
 */
int hpa_decode_attn_tc(const void *q_dev, const void *k_pool_dev, const void *v_pool_dev,
                       int32_t kv_dtype, const float *k_scale_dev, const float *v_scale_dev,
                       int64_t num_pages, const int32_t *page_indptr_dev,
                       const int32_t *page_indices_dev, int32_t page_size, int32_t B,
                       int32_t q_len, int32_t Hq, int32_t Hkv, int32_t d, float sm_scale,
                       void *taskmap_dev, int32_t num_ctas, float *partial_o_dev,
                       float *partial_lse_dev, hpa_stream_t stream);

/* Partitions per KV head that fill the current device once with
 * hpa_decode_attn_tc CTAs (SMs x resident CTAs per SM / Hkv), or -1. */
int32_t hpa_default_num_ctas_tc(int32_t Hq, int32_t Hkv, int32_t q_len, int32_t kv_dtype);

/*
 * hpa_decode_attn_window -- hpa_decode_attn over a map of hpa_plan_window: the same
 * step for the keys the window and the sinks show to each token (see there), reading
 * only their pages.  Arguments, layouts, supported shapes, partials and errors are
 * those of hpa_decode_attn; q_len is the one the map was planned with
 * (HPA_STATUS_MISMATCH).  What lies in hidden places of a page, NaN included, does
 * not enter the result.  hpa_combine merges the partials.  The kernel is that of
 * hpa_decode_attn_mma, and a window that hides nothing gives its bits: sums and softmax
 * statistics are fp32, and the probabilities are rounded to the type of the second product
 * (bf16 pages: bf16, each off by at most 2^-8 of itself; E4M3 pages: f16, 2^-11).
 */
int hpa_decode_attn_window(const void *q_dev, const void *k_pool_dev, const void *v_pool_dev,
                           int32_t kv_dtype, const float *k_scale_dev, const float *v_scale_dev,
                           int64_t num_pages, const int32_t *page_indptr_dev,
                           const int32_t *page_indices_dev, int32_t page_size, int32_t B,
                           int32_t q_len, int32_t Hq, int32_t Hkv, int32_t d, float sm_scale,
                           void *taskmap_dev, int32_t num_ctas, float *partial_o_dev,
                           float *partial_lse_dev, hpa_stream_t stream);

/* Partitions per KV head that fill the current device once with
 * hpa_decode_attn_window, or <= 0 as hpa_default_num_ctas. */
int32_t hpa_default_num_ctas_window(int32_t Hq, int32_t Hkv, int32_t q_len, int32_t kv_dtype);

/*
 * hpa_decode_attn_traced -- hpa_decode_attn (the same kernel choice) that
 * also records, for every CTA, four uint64 words at trace_dev[4 * (h * num_ctas
 * + c)]: the %globaltimer (ns) at kernel entry, after the task map was read,
 * after the CTA's last segment was stored, and (smid | segments << 32).  Used
 * to measure SM busy time and the tail idle of the last CTA (the pages watch
 * "attention kernel tail idle", "Hy3 Preview AI Infra 推理优化精读笔记", §3.1
 * 对我们的启发).  trace_dev: device, 8-byte aligned, >= 4 * num_ctas * Hkv *
 * row groups words; CTA (c, h, z) of the mma.sync kernel (up to 16 rows) at
 * word 4 * ((z * Hkv + h) * num_ctas + c), CTA (c, h) of the tcgen05 kernel
 * (above 16 rows, no row-group axis) at word 4 * (h * num_ctas + c).
 */
int hpa_decode_attn_traced(const void *q_dev, const void *k_pool_dev, const void *v_pool_dev,
                           int32_t kv_dtype, const float *k_scale_dev, const float *v_scale_dev,
                           int64_t num_pages, const int32_t *page_indptr_dev,
                           const int32_t *page_indices_dev, int32_t page_size, int32_t B,
                           int32_t q_len, int32_t Hq, int32_t Hkv, int32_t d, float sm_scale,
                           void *taskmap_dev, int32_t num_ctas, float *partial_o_dev,
                           float *partial_lse_dev, uint64_t *trace_dev, hpa_stream_t stream);

/*
 * hpa_decode_attn_allheads -- hpa_decode_attn with the KV heads inside the CTA
 * instead of on a grid axis (the pages do not say how heads map to CTAs,
 * "Hy3 Preview AI Infra 推理优化精读笔记" §3.1 方案 step 3; this is the other
 * reading, kept as an A/B).  Grid num_ctas x 1 x row groups: the CTA of
 * partition c walks c's segments and, for each, every KV head in turn
 * (heads innermost), so num_ctas counts partitions of the tile stream for the
 * whole grid (hpa_default_num_ctas_allheads: SMs x resident CTAs per SM /
 * row groups) and the task map must be planned with that count.  Arguments,
 * layouts, partials and errors are those of hpa_decode_attn; trace_dev is
 * NULL or, as for hpa_decode_attn_traced, 4 uint64 words per CTA at
 * trace_dev[4 * (z * num_ctas + c)].
 */
int hpa_decode_attn_allheads(const void *q_dev, const void *k_pool_dev, const void *v_pool_dev,
                             int32_t kv_dtype, const float *k_scale_dev,
                             const float *v_scale_dev, int64_t num_pages,
                             const int32_t *page_indptr_dev, const int32_t *page_indices_dev,
                             int32_t page_size, int32_t B, int32_t q_len, int32_t Hq,
                             int32_t Hkv, int32_t d, float sm_scale, void *taskmap_dev,
                             int32_t num_ctas, float *partial_o_dev, float *partial_lse_dev,
                             uint64_t *trace_dev, hpa_stream_t stream);
int32_t hpa_default_num_ctas_allheads(int32_t Hq, int32_t Hkv, int32_t q_len, int32_t kv_dtype);

/*
 * hpa_decode_attn_fused -- hpa_decode_attn with the combine folded in (one
 * launch instead of two).  Same arguments and layouts, plus the combine's
 * outputs out_dev (bf16 [B][q_len][Hq][d], 8-byte aligned) and out_lse_dev
 * (fp32 [B][q_len][Hq] or NULL), and arrivals_dev: int32 [B][Hkv][row groups]
 * (hpa_arrivals_elems), zero before the first call.
 *   - A request with one segment is written straight to out_dev.
 *   - Otherwise every CTA stores its partial, then counts itself in
 *     arrivals[r][h][z] with an atomic add (after a fence); the CTA whose add
 *     completes the count merges the request's partials for that KV head,
 *     exactly as hpa_combine does, and resets the counter to zero.  No CTA
 *     waits for another.
 * After a call whose map reports a non-zero status, re-zero arrivals_dev
 * before the next call.  A bad map makes every output NaN, as with
 * hpa_combine.  This is the fused combine the pages' three-module design
 * leaves as a later step ("Hy3 Preview AI Infra 推理优化精读笔记", §3.1 step 5:
 * a combine merges the split-KV results).
 */
size_t hpa_arrivals_elems(int32_t B, int32_t Hq, int32_t Hkv, int32_t q_len);
int hpa_decode_attn_fused(const void *q_dev, const void *k_pool_dev, const void *v_pool_dev,
                          int32_t kv_dtype, const float *k_scale_dev, const float *v_scale_dev,
                          int64_t num_pages, const int32_t *page_indptr_dev,
                          const int32_t *page_indices_dev, int32_t page_size, int32_t B,
                          int32_t q_len, int32_t Hq, int32_t Hkv, int32_t d, float sm_scale,
                          void *taskmap_dev, int32_t num_ctas, float *partial_o_dev,
                          float *partial_lse_dev, void *out_dev, float *out_lse_dev,
                          int32_t *arrivals_dev, hpa_stream_t stream);

/*
 * hpa_combine -- the Combine kernel ([Notes §3.1] step 5, [HPC-Ops §二.1]).
 * For every (request r, token j, head g) over r's segments s:
 *   M = max_s lse_s,  w_s = exp(lse_s - M),
 *   out = sum_s w_s o_s / sum_s w_s  (rounded to bf16),  out_lse = M + ln sum_s w_s.
 * out_dev: bf16 [B][q_len][Hq][d], 8-byte aligned; out_lse_dev: fp32
 * [B][q_len][Hq] or NULL.  d == 128.
 */
int hpa_combine(const float *partial_o_dev, const float *partial_lse_dev, void *taskmap_dev,
                int32_t B, int32_t num_ctas, int32_t q_len, int32_t Hq, int32_t d,
                void *out_dev, float *out_lse_dev, hpa_stream_t stream);

/*
 * hpa_store_kv -- the fused KV-cache writer that feeds the decode path
 * ("Hy3 Preview AI Infra 推理优化精读笔记", §4.1 "Rope + Norm + Hadamard + Quant +
 * Store KV": the element-wise chain after the QKV projection in one pass,
 * written straight to the low-bit cache).  For request r, new token j (at
 * position pos = L_r - q_len + j) and KV head h:
 *   key:   rotate-half RoPE with cos_sin[pos] (cos in columns [0, d/2), sin in
 *          [d/2, d)), then RMSNorm over d (x / sqrt(mean x^2 + eps) * norm_w),
 *          then, if use_hadamard, the orthonormal Sylvester Walsh-Hadamard
 *          transform of order d; stored as bf16, or as E4M3 codes of
 *          x / k_scale[h] (round to nearest even, saturating at +-448);
 *   value: stored as bf16, or as E4M3 codes of v / v_scale[h];
 * into slot pos % page_size of page page_indices[page_indptr[r] + pos / page_size]
 * of k_pool_dev / v_pool_dev ([num_pages][Hkv][page_size][d]).
 * k_new_dev, v_new_dev: bf16 [B][q_len][Hkv][d], 16-byte aligned (pools too).  seq_lens_dev:
 * int32 [B], lengths including the new tokens.  cos_sin_dev: fp32 [max_pos][d],
 * 16-byte aligned.  norm_w_dev: fp32 [d], 16-byte aligned.  d == 128,
 * page_size == 64.  status_dev: optional int32; a position outside
 * [0, max_pos) sets HPA_STATUS_BAD_SEQLEN, a missing or out-of-range page
 * HPA_STATUS_BAD_PAGE, and that token is not written.
 */
int hpa_store_kv(const void *k_new_dev, const void *v_new_dev, const int32_t *seq_lens_dev,
                 const int32_t *page_indptr_dev, const int32_t *page_indices_dev,
                 int64_t num_pages, int32_t page_size, const float *cos_sin_dev, int32_t max_pos,
                 const float *norm_w_dev, float eps, int32_t use_hadamard, int32_t kv_dtype,
                 const float *k_scale_dev, const float *v_scale_dev, void *k_pool_dev,
                 void *v_pool_dev, int32_t B, int32_t q_len, int32_t Hkv, int32_t d,
                 int32_t *status_dev, hpa_stream_t stream);

/*
 * hpa_store_kv_at -- hpa_store_kv for a cache that evicts (below): the slot of token j
 * is still position L_r - q_len + j of the cache, and its rotation is that of position
 * text_pos_dev[r] + j of the text, which the evictions have left ahead of it.
 * text_pos_dev: int32 [B], the text position of each request's first new token.  A
 * text position outside [0, max_pos) sets HPA_STATUS_BAD_SEQLEN.
 */
int hpa_store_kv_at(const void *k_new_dev, const void *v_new_dev, const int32_t *seq_lens_dev,
                    const int32_t *text_pos_dev, const int32_t *page_indptr_dev,
                    const int32_t *page_indices_dev, int64_t num_pages, int32_t page_size,
                    const float *cos_sin_dev, int32_t max_pos, const float *norm_w_dev, float eps,
                    int32_t use_hadamard, int32_t kv_dtype, const float *k_scale_dev,
                    const float *v_scale_dev, void *k_pool_dev, void *v_pool_dev, int32_t B,
                    int32_t q_len, int32_t Hkv, int32_t d, int32_t *status_dev,
                    hpa_stream_t stream);

/*
 * The calls below keep a cache bounded by the attention its keys receive (the
 * pages have no counterpart to them).  Accumulated weights live in pools of their own,
 * fp32 [num_pages][Hkv][page_size], paged by the same table as K and V.  Each call
 * writes what it names for the pages of a request, so a page that is listed twice (a
 * prefix shared by two requests) is not for these calls: its results are unspecified.
 * Copy such a prefix first (hpa_evict_compact to pages of the request's own).
 *
 * hpa_key_weights -- adds one attention step's weights to the accumulators.  With
 * lse_dev the step's out_lse (fp32 [B][q_len][Hq], natural log), for every key
 * i < L_r that some token sees:
 *   acc_out[i] = (i < L_r - q_len ? decay * acc_in[i] : 0)
 *              + sum over the rows (j, g) of the KV head that see i of
 *                exp(sm_scale * q . k_i - lse[j][g]),
 * in fp32, the same order on every run.  The q_len new keys start from zero, whatever
 * their slots held.  Other slots are not written (with a window map: keys no token
 * sees; they keep their weight and do not decay, so an eviction by these weights may keep
 * keys that no window shows any more).  acc_in_dev may equal acc_out_dev
 * (the usual, in place), be another pool that does not overlap it (draft tokens that may
 * yet be rejected) or be NULL for zero; decay 0 does not read it.  A row whose lse is
 * -inf adds nothing.
 * taskmap_dev: the map of the attention step, of any plan; num_ctas as planned.  Both
 * pools 16-byte aligned.  q, K, shapes and errors as hpa_decode_attn, but with E4M3 pages
 * the query rows are carried as in hpa_decode_attn_tc at every row count: exactly down to
 * about 2^-12 of a row's largest element, then to an absolute 2^-21 of it.  The pages of a
 * bad page id, the keys of a request shorter than q_len and those of a malformed segment
 * are not written, all others are updated in full, and the bits are in the status once the
 * call has run.  A status that an earlier call left in the map (the plan, the attention
 * step, hpa_key_weights) stops the whole call: nothing is written.  After
 * HPA_STATUS_TIMEOUT the accumulators are undefined.  Calls that run at the same time over
 * one map need the same Hkv, as they count their blocks in it together, and an error in one
 * of them may stop blocks of the others.
 */
int hpa_key_weights(const void *q_dev, const float *lse_dev, const void *k_pool_dev,
                    int32_t kv_dtype, const float *k_scale_dev, int64_t num_pages,
                    const int32_t *page_indptr_dev, const int32_t *page_indices_dev,
                    int32_t page_size, int32_t B, int32_t q_len, int32_t Hq, int32_t Hkv,
                    int32_t d, float sm_scale, float decay, void *taskmap_dev, int32_t num_ctas,
                    const float *acc_in_dev, float *acc_out_dev, hpa_stream_t stream);

/*
 * hpa_evict_select -- which keys each KV head keeps.  For request r with budget
 * budgets_dev[r] and every KV head: if L_r is within the budget, all of them; else the
 * first `sinks` keys, the last `recent` keys and, of the others, the
 * budget - sinks - recent with the largest weight in acc_dev, ties to the lower index
 * (-0 equals 0; NaN ranks above every number).  Writes their indices in ascending
 * order to kept_dev[(r * Hkv + h) * kept_stride + t], t < new_lens_dev[r] =
 * min(L_r, budget); entries past that are left as they were.  A request that cannot
 * be served gets new_lens -1, which hpa_evict_compact passes over, and sets bits in
 * status_dev (optional int32, 4-byte aligned): L_r < 1 HPA_STATUS_BAD_SEQLEN; L_r above
 * 2^31 - 65537 HPA_STATUS_OVERFLOW; a budget below 1, min(L_r, budget) > kept_stride, or
 * sinks + recent > budget < L_r HPA_STATUS_BAD_BUDGET; a missing or out-of-range page
 * HPA_STATUS_BAD_PAGE.
 * kept_dev: int32, B * Hkv * kept_stride.  new_lens_dev: int32 [B], overlapping neither
 * seq_lens_dev nor budgets_dev.  acc_dev 16-byte aligned.
 */
int hpa_evict_select(const float *acc_dev, const int32_t *seq_lens_dev,
                     const int32_t *page_indptr_dev, const int32_t *page_indices_dev,
                     int64_t num_pages, int32_t page_size, const int32_t *budgets_dev,
                     int32_t sinks, int32_t recent, int32_t B, int32_t Hkv, int32_t *kept_dev,
                     int64_t kept_stride, int32_t *new_lens_dev, int32_t *status_dev,
                     hpa_stream_t stream);

/*
 * hpa_evict_compact -- moves the kept rows of K, V and (unless NULL) the accumulated
 * weights together: position t of the request's new cache gets the row of position
 * kept[t], for t < new_lens[r] and every KV head.  With dst_indptr_dev and
 * dst_indices_dev NULL the new cache is the front of the request's own pages; the pages
 * past ceil(new_len / page_size) are then free.  Otherwise it is the pages that this
 * second table lists, none of them among the pages being read: the old cache stays as
 * it was (a shared prefix, say).  Order is kept, so sinks and causal masks mean the same as
 * before; a window counts cache slots, so after an eviction it reaches further back in the
 * text than its number of keys (no call masks by text position).  kept must ascend, as hpa_evict_select writes it.  new_lens[r]
 * below 1 or beyond kept_stride: the request is passed over.  A position without a
 * valid page sets HPA_STATUS_BAD_PAGE in status_dev (optional), and that row is not
 * moved.  k_pool_dev, v_pool_dev 16-byte aligned, apart from each other.
 */
int hpa_evict_compact(void *k_pool_dev, void *v_pool_dev, int32_t kv_dtype, float *acc_dev,
                      int64_t num_pages, const int32_t *page_indptr_dev,
                      const int32_t *page_indices_dev, const int32_t *dst_indptr_dev,
                      const int32_t *dst_indices_dev, int32_t page_size, const int32_t *kept_dev,
                      int64_t kept_stride, const int32_t *new_lens_dev, int32_t B, int32_t Hkv,
                      int32_t d, int32_t *status_dev, hpa_stream_t stream);

/*
 * hpa_evict -- hpa_evict_select followed by hpa_evict_compact of K, V and the weights
 * (acc_dev, not NULL) in one call, with their arguments, results and checks (those of the
 * arguments all made before the first launch).  With a second table the selection checks it
 * too: a request whose new pages are not all listed with valid ids gets new_lens -1 and
 * HPA_STATUS_BAD_PAGE, and none of its rows moves.
 */
int hpa_evict(void *k_pool_dev, void *v_pool_dev, int32_t kv_dtype, float *acc_dev,
              int64_t num_pages, const int32_t *seq_lens_dev, const int32_t *page_indptr_dev,
              const int32_t *page_indices_dev, const int32_t *dst_indptr_dev,
              const int32_t *dst_indices_dev, int32_t page_size, const int32_t *budgets_dev,
              int32_t sinks, int32_t recent, int32_t B, int32_t Hkv, int32_t d, int32_t *kept_dev,
              int64_t kept_stride, int32_t *new_lens_dev, int32_t *status_dev,
              hpa_stream_t stream);

/*
 * hpa_store_qkv -- queries and the cache from the projections of num_tokens tokens in one pass:
 * RMSNorm of every query and key head, position rotation in the same pass, an optional
 * transform, and the quantised paged store.  hpa_store_kv ("Hy3 Preview AI Infra 推理优化精读
 * 笔记", §4.1) does the keys and values of [B][q_len] tokens; this call takes any list of tokens
 * (prompt chunks, decode steps, both) by the slots and positions of hpa_assign_pages, does the
 * queries too, and writes 4-bit caches.  Token t, head h, row x of d = 128 elements:
 *   query, key: norm and rotation, the norm first, or last with HPA_QKV_NORM_AFTER (the order of
 *           hpa_store_kv).  Norm: x / sqrt(mean(x^2) + eps) * w, w = q_norm or k_norm (fp32 [d],
 *           NULL: no norm).  Rotation of the first rot_dim elements (0, 16, 32, 64 or 128):
 *           pair i, (x_i, x_{i + rot_dim/2}) or with HPA_QKV_INTERLEAVED (x_2i, x_{2i+1}), turned
 *           by cos_sin[positions[t]][i] (cosine) and [rot_dim/2 + i] (sine).  With
 *           HPA_QKV_HADAMARD then the orthonormal Sylvester transform of order d, on queries and
 *           keys alike, which leaves their products as they were;
 *   query:  rounded to bf16 into q_out[t][h];
 *   key, value: into place slots[t] % 64 of page slots[t] / 64 of the pools: bf16; E4M3 codes of
 *           x / scale[h] (round to nearest even, saturating); or 4-bit: with y = x / scale[h], for
 *           every 16 elements the block scale b = E4M3(max |y| / 6) and codes E2M1(y / b), both to
 *           nearest even and saturating (codes 0 where b is 0; a NaN makes b NaN).
 * All arithmetic is fp32; nothing is rounded between the steps.
 * q_dev, k_dev, v_dev: bf16, token t's heads from t * stride elements on (so they may be parts
 * of one packed projection), 16-byte aligned, strides multiples of 8.  q_out_dev likewise; it may
 * be q_dev with its stride (in place), and other columns of the rows that hold keys and values;
 * otherwise what the call writes overlaps neither itself nor what it reads.  q_dev NULL: no
 * queries; k_dev and v_dev NULL: no cache (num_pages then only bounds the slots).  positions_dev
 * int32, slots_dev int64 [num_tokens].
 * cos_sin_dev: fp32 [max_pos][rot_dim], 16-byte aligned.
 * A token of slot -1 is passed over, its q_out row left as it was (rows of a captured batch that
 * hold no token, requests that got no pages); so is one of another slot outside the pool
 * (HPA_STATUS_BAD_PAGE in status_dev, optional int32) or of a position outside [0, max_pos)
 * (HPA_STATUS_BAD_SEQLEN).  Two tokens of one slot: which one its row holds, or parts of both,
 * is unspecified.  d == 128, page_size == 64; num_tokens may be 0.
 */
#define HPA_QKV_NORM_AFTER 1
#define HPA_QKV_INTERLEAVED 2
#define HPA_QKV_HADAMARD 4
int hpa_store_qkv(const void *q_dev, int64_t q_stride, const void *k_dev, int64_t k_stride,
                  const void *v_dev, int64_t v_stride, int32_t num_tokens, int32_t Hq, int32_t Hkv,
                  int32_t d, const int32_t *positions_dev, const int64_t *slots_dev,
                  const float *cos_sin_dev, int32_t max_pos, int32_t rot_dim,
                  const float *q_norm_dev, const float *k_norm_dev, float eps, int32_t flags,
                  void *q_out_dev, int64_t q_out_stride, int32_t kv_dtype,
                  const float *k_scale_dev, const float *v_scale_dev, void *k_pool_dev,
                  void *v_pool_dev, int64_t num_pages, int32_t page_size, int32_t *status_dev,
                  hpa_stream_t stream);

/*
 * hpa_assign_pages -- page tables and slot maps from request lengths, on the device (the pages
 * have no counterpart to it).  The state of a pool of num_pages pages:
 *   table_dev       int32 [num_rows][table_stride]: the pages that each row (a session) holds,
 *                   in order;
 *   held            int32 [num_rows]: how many;
 *   free_pages_dev  int32 [num_pages]: a stack of the pages that no row holds;
 *   free_count      int32: its height.
 * A page belongs to one row or to the stack, so one that several sessions share (a prefix) is
 * not for this call.  One step, for the B requests of a batch in rows rows_dev[r] (NULL: row r):
 *   n_r = ceil(L_r / page_size) pages from now on, for L_r = seq_lens_dev[r] >= 0 tokens, the
 *   new ones included (0: the session has ended).  Pages past n_r go back on the stack, in the
 *   order of the requests and of their pages; then missing ones come off it, request by request,
 *   the top first.  A request that asks for more than is left after the requests before it
 *   gets none and keeps what it holds, as does every later one that needs a page
 *   (HPA_STATUS_NO_PAGES).
 * held_in_dev and held_out_dev, free_count_in_dev and free_count_out_dev may each be one array
 * (the usual, in place).  Where they differ, the state before the step stays whole -- entries
 * of the table past a row's count and of the stack past its height mean nothing -- so that a
 * step can be taken again from it with other lengths (draft tokens that were rejected).
 * held_out is written for the rows of the batch alone.  Results:
 *   page_indptr_dev [B+1], page_indices_dev [indices_cap]: the page lists of the batch, as the
 *                   attention calls read them; entries past the last are left as they were;
 *   with new_tokens_dev (int32 [B], 0 <= new_tokens[r] <= L_r, the last tokens of r; or NULL)
 *   slots_dev (int64) and positions_dev (int32) [max_tokens]: for each of them, request by
 *                   request, page * page_size + place in the page, and L_r - new_tokens[r] + j
 *                   plus pos_offset_dev[r] (NULL: 0; the tokens that evictions removed).  A
 *                   refused request's tokens have slot -1; behind the last token slots are -1
 *                   and positions 0, so a captured step can be replayed with fewer tokens.
 * status_dev (optional int32) gets bits, and the request in question keeps its pages:
 * HPA_STATUS_BAD_SEQLEN (L_r < 0, new_tokens outside [0, L_r]), HPA_STATUS_OVERFLOW (n_r beyond
 * table_stride; page lists beyond indices_cap or tokens beyond max_tokens, which are cut),
 * HPA_STATUS_BAD_MAP (a row outside [0, num_rows), one that an earlier request of the batch
 * lists, a count outside its range), HPA_STATUS_BAD_PAGE (a page id out of range in the state).
 * workspace_dev: >= hpa_assign_pages_workspace(B, num_rows) bytes, 16-byte aligned; calls that
 * may run at the same time need one each.  page_size == 64.  slots_dev 8-byte aligned.  The
 * arrays written overlap neither each other nor those read.
 */
size_t hpa_assign_pages_workspace(int32_t B, int32_t num_rows);
int hpa_assign_pages(const int32_t *seq_lens_dev, const int32_t *new_tokens_dev,
                     const int32_t *rows_dev, const int32_t *pos_offset_dev, int32_t B,
                     int32_t num_rows, int32_t *table_dev, int32_t table_stride,
                     const int32_t *held_in_dev, int32_t *held_out_dev, int32_t *free_pages_dev,
                     const int32_t *free_count_in_dev, int32_t *free_count_out_dev,
                     int32_t num_pages, int32_t page_size, int32_t *page_indptr_dev,
                     int32_t *page_indices_dev, int32_t indices_cap, int64_t *slots_dev,
                     int32_t *positions_dev, int32_t max_tokens, void *workspace_dev,
                     size_t workspace_bytes, int32_t *status_dev, hpa_stream_t stream);

/*
 * hpa_selftest_wait_timeout -- diagnostic for the failure path of the
 * attention pipeline (no counterpart on the pages).  One thread waits on an
 * mbarrier phase that nothing completes, using the same time-bounded wait
 * as hpa_decode_attn, for limit_ns nanoseconds (1e3 .. 5e9); on expiry it ORs
 * HPA_STATUS_TIMEOUT into status_dev[0] and returns, leaving the context
 * usable.  status_dev: one int32 in device memory, 4-byte aligned.
 */
int hpa_selftest_wait_timeout(int32_t *status_dev, int64_t limit_ns, hpa_stream_t stream);

/*
 * hpa_decode_attn_combine_noalloc -- hpa_decode_attn followed by hpa_combine,
 * for callers that cannot allocate device memory; the pages have no
 * counterpart to it.  Such callers include a plugin running inside another
 * runtime that owns the whole device memory pool and hands out no
 * workspace, and a serving loop that must not call cudaMalloc/cudaFree in the
 * middle of a step (cudaFree synchronises the device; either can fail under
 * memory pressure).  Instead of caller-provided partial_o / partial_lse, the
 * split partials live in one fixed array inside the library's device image,
 * HPA_NOALLOC_SCRATCH_BYTES (16 MiB) per GPU, held by every GPU that loads
 * the library until the process exits.  The call itself allocates nothing.
 *
 * Arguments are those of hpa_decode_attn (minus the partial buffers) and of
 * hpa_combine (out_dev, out_lse_dev), with the same layouts and checks.  The
 * partials need (B + num_ctas - 1) * q_len * Hq * (d + 1) floats; a problem
 * larger than the array returns HPA_ERR_NOALLOC_CAPACITY before any launch
 * (e.g. 64 requests x 2 tokens x 64 heads with 38 partitions uses 6.7 MB).
 *
 * The first call on a device resolves the array's device address with that
 * device current (cudaGetSymbolAddress, which may load the module); make that
 * first call before any stream capture.  The address belongs to the CUDA
 * context that was current, so it is cached per context (keyed by the
 * context's process-unique id): a call under another context of the same
 * device, or after cudaDeviceReset, repeats that set-up once for the new
 * context and should likewise come before any capture there.  All calls
 * share the one array and it keeps the last call's contents: nothing in it
 * needs to start at zero (each call writes every partial it reads), but
 * calls that overlap on the GPU -- on different streams, or from several
 * host threads -- race on it and must be serialised by the caller.
 */
#define HPA_NOALLOC_SCRATCH_BYTES (16u << 20)
int hpa_decode_attn_combine_noalloc(const void *q_dev, const void *k_pool_dev,
                                    const void *v_pool_dev, int32_t kv_dtype,
                                    const float *k_scale_dev, const float *v_scale_dev,
                                    int64_t num_pages, const int32_t *page_indptr_dev,
                                    const int32_t *page_indices_dev, int32_t page_size,
                                    int32_t B, int32_t q_len, int32_t Hq, int32_t Hkv,
                                    int32_t d, float sm_scale, void *taskmap_dev,
                                    int32_t num_ctas, void *out_dev, float *out_lse_dev,
                                    hpa_stream_t stream);

/* Static description of a return code. */
const char *hpa_error_string(int code);

/* The last CUDA error the library saw on this thread (cudaError_t value), 0 if none. */
int hpa_last_cuda_error(void);

#ifdef __cplusplus
}
#endif
#endif /* HPA_H */
