/*
 * sd_ops.h -- op-level C ABI of libsd.so: the individual decode-step kernels,
 * exposed so that each can be checked on its own at full workload shapes.
 * Same conventions as sd.h (SD_* return codes; *_dev pointers are device
 * memory owned by the caller; `stream` is a cudaStream_t or NULL for the
 * legacy default stream).  Errors are reported through sd_last_error(NULL).
 */
#ifndef SD_OPS_H
#define SD_OPS_H

#include "sd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A block-quantised matrix [rows][cols] (one row per output feature, cols
 * contiguous: the orientation of "Chatterbox -> ggml Port: Development
 * Journal", section 3.2, issue 5) repacked into the device layout the GEMV
 * streams: codes of a row contiguous (16-byte units) and the fp16 scales (and
 * affine biases) in a separate array.  `canon` holds the canonical blob
 * bytes of one tensor: Q8_0 34-byte blocks, Q4_0 18-byte blocks (journal
 * section 3.23), Q5_0 22-byte blocks (fp16 d, 32 fifth bits, 16 nibble
 * bytes), or affine codes (8-bit: one per byte; 4-bit: element 2i in the low
 * nibble of byte i) + fp16 scales + fp16 biases; host memory, or device memory
 * when on_device != 0.  cols must be a multiple of 32 (64 for SD_A8G64 and
 * SD_A4G64). */
typedef struct sd_qmat sd_qmat;
int sd_qmat_create(int quant, const void* canon, int64_t rows, int64_t cols, int on_device, int device,
                   sd_qmat** out);
void sd_qmat_destroy(sd_qmat* m);

/* Dequantise to fp32 out_dev[rows][cols]: Q8_0 d*q, Q4_0 d*(q-8), Q5_0
 * d*(q-16), affine fma(scale, q, bias) -- bit-exact definitions of the formats. */
int sd_qmat_dequant(const sd_qmat* m, float* out_dev, void* stream);

/* y_dev[b][r] = sum_k W[r][k] x_dev[b][k] (+ bias_dev[r]) for b < nb (nb 1 or
 * 2), fp32 accumulation.  bias_dev may be NULL. */
int sd_qmat_gemv(const sd_qmat* m, const float* x_dev, int32_t nb, const float* bias_dev, float* y_dev,
                 void* stream);

/* Epilogues of sd_qmat_gemm. */
enum { SD_EPI_LINEAR = 0, SD_EPI_GELU = 1, SD_EPI_SWIGLU = 2 };

/* Tensor-core GEMM for prompt prefill and batched rows ("Chatterbox -> ggml
 * Port: Development Journal", section 3.2: the prompt graph applies every
 * layer to all prompt positions at once):
 *   t[i][r] = sum_k W[r][k] x_dev[i][k] for i < M (x_dev [M][cols], fp32);
 *   SD_EPI_LINEAR: y_dev[i][r] = t[i][r] (+ bias_dev[r]) (+ resid_dev[i][r]);
 *   SD_EPI_GELU:   y_dev[i][r] = gelu_tanh(t[i][r] (+ bias_dev[r])) (+ resid_dev[i][r]);
 *   SD_EPI_SWIGLU: rows are interleaved gate/up pairs (row 2j gate j, row
 *     2j+1 up j), y_dev[i][j] = silu(t[i][2j]) * t[i][2j+1] (+ resid_dev[i][j]),
 *     j < rows/2; bias_dev must be NULL; rows must be even.
 * y_dev and resid_dev have leading dimension rows (rows/2 for SwiGLU); resid_dev
 * may equal y_dev; bias_dev and resid_dev may be NULL.  The codes of a
 * quantisation block enter the tensor cores exactly (fp16 integers), the
 * fp32 activations as an fp16 high + low pair, and the block scale (and
 * affine bias times the group's activation sum) is applied in fp32.
 * Device pointers; enqueued on `stream`; returns SD_ERR_INVALID_ARG on a NULL
 * pointer, M < 1 or a bad epilogue. */
int sd_qmat_gemm(const sd_qmat* m, const float* x_dev, int32_t M, int32_t epilogue, const float* bias_dev,
                 const float* resid_dev, float* y_dev, void* stream);

/* As sd_qmat_gemm, on the 5th-generation tensor cores (tcgen05 MMA with a
 * tensor-memory accumulator, operands loaded by TMA), the form the prompt
 * prefill uses.  The weights are dequantised once (kept with the matrix,
 * device memory rows*cols*4 bytes, allocated on the first call) and, like the
 * activations, split into fp16 high and low parts; three fp16 products per
 * K step (hi*hi + hi*lo + lo*hi) accumulate in fp32.  cols must be a multiple
 * of 64 (else SD_ERR_UNSUPPORTED).  Synchronises `stream` before returning;
 * allocates and frees a scratch buffer of M*cols*4 bytes per call.  A kernel
 * wait that runs out of its time budget returns SD_ERR_TIMEOUT. */
int sd_qmat_gemm_tc(sd_qmat* m, const float* x_dev, int32_t M, int32_t epilogue, const float* bias_dev,
                    const float* resid_dev, float* y_dev, void* stream);

/* As sd_qmat_gemm for 1 <= M <= 16 rows (the G rollouts of "Every Frame Is a
 * Memory Read", section 8, which share one read of the weights per step):
 * the form the decode step uses for more than two rows.  The weights stream
 * once from memory straight into the tensor cores (mma.sync m16n8k16, the same
 * exact-code / fp16 hi+lo / fp32-scale arithmetic); K is split over CTAs and
 * the partial sums are added in a fixed order, so results are reproducible.
 * x_dev must be 16-byte aligned.  A workspace of partial sums and column-tile
 * counters is kept with the matrix (allocated on the first call, at most
 * 16 * rows * cols / 32 floats).  Calls on one matrix must not run
 * concurrently on different streams.  Returns SD_ERR_INVALID_ARG on a NULL
 * pointer, M outside [1, 16], a bad epilogue or a misaligned x_dev. */
int sd_qmat_gemm16(sd_qmat* m, const float* x_dev, int32_t M, int32_t epilogue, const float* bias_dev,
                   const float* resid_dev, float* y_dev, void* stream);

/* Sample one token per row from logits_dev[rows][V] with draws u_dev[rows];
 * tokens to out_dev[rows].  Sampler semantics as in sd.h.  V <= 16384. */
int sd_sample_rows(const float* logits_dev, int32_t rows, int32_t V, const sd_sampler* sampler,
                   const float* u_dev, int32_t* out_dev, void* stream);

/* (sd_sampler_ladder, the ladder's parameters, is declared in sd.h.) */

/* Sampler ladder of the multilingual T3 ("Chatterbox -> ggml Port: Development
 * Journal", the multilingual port's sampling path): classifier-free-guidance
 * combine -> repetition penalty -> temperature -> min_p -> top-p -> top-k ->
 * draw in vocabulary order.  Per row b:
 *   z_i = c_i + w (c_i - u_i)      (c = logits_cond_dev[b], u = logits_uncond_dev[b]; w ignored when NULL)
 *   seen_dev[b][i] != 0: z_i / penalty if z_i > 0, else z_i * penalty   (seen_dev may be NULL)
 *   z_i / T; p_i proportional to exp(z_i); min_p keeps p_i >= min_p * max p;
 *   top-p keeps the shortest (p desc, index asc) prefix of those whose
 *   renormalised mass reaches top_p; top-k keeps the ones whose value is >= the
 *   k-th largest remaining (ties kept); the token is the smallest vocabulary
 *   index whose cumulative kept mass exceeds u_dev[b] times the kept total.
 * Layouts: logits [rows][V] fp32, seen [rows][V] bytes, u [rows], out [rows] int32;
 * device pointers; 1 <= V <= 16384.  Double-precision arithmetic, one CTA per row.
 * This entry is an op-level form of the ladder: the decode step's own sampler
 * is temperature -> top-k -> top-p (sd.h).  Synchronises `stream`; returns
 * SD_ERR_INVALID_ARG on a NULL required pointer or a parameter out of range. */
int sd_sample_rows_ladder(const float* logits_cond_dev, const float* logits_uncond_dev, int32_t rows, int32_t V,
                          const sd_sampler_ladder* sampler, const uint8_t* seen_dev, const float* u_dev,
                          int32_t* out_dev, void* stream);

/* Decode attention for one query per head against n cached positions
 * (journal section 3.13 flash attention over a cache laid out
 * [head][pos][dim]): out[b][h] = softmax(q[b][h] . K[b][g][0:n] / sqrt(hd))
 * V[b][g][0:n] with g = h / (H / Hkv).  q_dev [B][H][hd] fp32, k_dev/v_dev
 * [B][Hkv][n_ctx][hd] fp16, out_dev [B][H][hd] fp32.  Split-KV over
 * `nsplit` chunks per (row, kv head) then a log-sum-exp combine.  hd is 64 or
 * 128; 1 <= n <= n_ctx. */
int sd_attend_rows(const float* q_dev, const uint16_t* k_dev, const uint16_t* v_dev, int32_t B, int32_t H,
                   int32_t Hkv, int32_t hd, int32_t n_ctx, int32_t n, int32_t nsplit, float* out_dev,
                   void* stream);

/* The decode attention of sd_attend_rows for callers that may not allocate
 * device memory while they run -- for instance a host thread with a hard
 * latency budget (cudaMalloc can synchronise the whole device) or a host
 * framework that owns all device memory through its own pool.  This entry has
 * no counterpart in the pages; it exists for those callers.  Arguments,
 * layouts and the values written to out_dev are those of sd_attend_rows.
 *
 * Unlike sd_attend_rows, the call is stream-ordered: it queues a counter clear
 * (cudaMemsetAsync) and the attention kernel on `stream` and returns without
 * waiting.  out_dev is ready, and the inputs may be released, only after the
 * caller synchronises the stream (or orders later work after it); an error
 * raised by the kernel appears at that synchronisation, not in this call's
 * return value, which reports only argument and launch errors.
 *
 * Instead of allocating, the split-KV partial results and one counter per
 * (row, kv head) go to one fixed array of 1048576 floats (4 MiB) that every
 * device loading the library keeps until the process exits.  A call needs
 * B * H * nsplit * (hd + 4) + B * Hkv floats of it; a larger request returns
 * SD_ERR_INVALID_ARG.  The call allocates nothing: no cudaMalloc, cudaFree or
 * allocating library routine.  The first call on each device (with that device
 * current) looks up the array's device address; make that first call before
 * any stream capture.  All calls share the one array: calls that overlap on
 * the GPU (different streams, or different threads on the same device) race on
 * it and must be serialised by the caller.  Every partial record a call reads
 * is written earlier in the same call; the counters, which must start at zero,
 * are cleared by the call itself on `stream` before the kernel runs. */
int sd_attend_rows_static(const float* q_dev, const uint16_t* k_dev, const uint16_t* v_dev, int32_t B, int32_t H,
                          int32_t Hkv, int32_t hd, int32_t n_ctx, int32_t n, int32_t nsplit, float* out_dev,
                          void* stream);

/* ---- Requests of different lengths: a cache in pages, and attention to an
 * encoder's states.  These entries have no counterpart in the pages; they are
 * the forms of the step's rotary write and attention for callers that serve
 * requests of their own lengths (the contexts of sd.h keep one position counter
 * for all rows) or that attend to states other than the own past (the T3's
 * conditioning).  All of them are stream-ordered: they queue their kernel on
 * `stream` and return; nothing is allocated, copied or waited for, so they may be
 * captured into a graph.  They run on the calling thread's current device (the
 * attention entries: on their workspace's device); the stream and every pointer
 * belong to that device.  Return values report arguments and launches.  A call of the
 * write or of attention with no rows (n, R, B or Lq 0) returns SD_OK and does nothing,
 * whatever its other arguments; sd_page_plan, which has something to write even then, refuses R 0. */

/* Element types.  E4M3 is a cache type only. */
enum { SD_F32 = 1, SD_F16 = 2, SD_BF16 = 3, SD_E4M3 = 4 };

/* The pages of one layer's cache.  Element d of position j of a page, for kv
 * head g, is at page * page_stride + g * head_stride + j * pos_stride + d
 * (elements, the same for k_dev and v_dev).  All three strides 0: the order
 * [page][kv_head][pos][dim], as in the contexts' cache; [page][pos][kv_head][dim]
 * and pages of all layers in one pool are given by their strides.  Pointers are
 * 16-byte aligned and strides positive multiples of 16 bytes (below 2^40; not used where
 * there is one element).  dtype SD_F16, SD_BF16, or
 * SD_E4M3 (stored value times k_scale_dev[g] / v_scale_dev[g]; NULL: 1; the scale
 * pointers are NULL for the other types).  head_dim is 64 or 128, page_size 1 to
 * 65536, n_pages * page_size at most 2^31 - 1. */
typedef struct sd_pages {
    void* k_dev;
    void* v_dev;
    const float* k_scale_dev;
    const float* v_scale_dev;
    int64_t page_stride, head_stride, pos_stride;
    int32_t dtype, n_pages, page_size, n_kv_head, head_dim, reserved;
} sd_pages;

/* Block tables and slot maps of a step from the requests' lengths.  Request r
 * (0 <= r < R) has len_dev[r] positions in the cache and brings new_dev[r] >= 0
 * new tokens.  The pages it needs beyond the ceil(len / page_size) it has are
 * taken from free_dev[n_free], in request order, first to last, and written to
 * its row of table_dev [R][table_stride]; the row's other entries stay.  Outputs:
 *   total_dev[R]     len + new
 *   start_dev[R + 1] new tokens of the requests before r; [R]: of all
 *   slot_dev[rows]   of new token i of the step: page id * page_size + place in
 *                    the page; -1 behind the last token
 *   pos_dev[rows]    its position in its request (0 behind the last token)
 *   req_dev[rows]    its request (-1 behind the last token)
 *   info_dev[4]      new tokens; pages taken; what went wrong (bits); longest total
 * `rows` is the capacity of the step, known to the host.  Bits of info_dev[2]:
 *   1 more than `rows` new tokens (the first `rows` are mapped, and the pages
 *     that begin with a later token stay out of the table);
 *   2 the free list is too short (info_dev[1] says how many pages are needed;
 *     the table entries without a page are -1, as are their tokens' slots);
 *   4 a request is longer than its table row (the tokens behind it: slot -1, and
 *     no page is taken for them);
 *   8 a negative length or count (read as 0).
 * A table entry that a token falls into and that is negative gives slot -1.
 * Calling again with the same inputs gives the same outputs: the new lengths
 * take effect when the caller passes total_dev as len_dev of the next step.
 * Counts are held in 64 bits and limited to 2^31 - 1 where they are stored.
 * free_dev may be NULL when n_free is 0; slot_dev, pos_dev and req_dev when rows
 * is 0.  The buffers must not overlap. */
int sd_page_plan(const int32_t* len_dev, const int32_t* new_dev, int32_t R, const int32_t* free_dev, int32_t n_free,
                 int32_t page_size, int32_t* table_dev, int32_t table_stride, int32_t rows, int32_t* total_dev,
                 int32_t* start_dev, int32_t* slot_dev, int32_t* pos_dev, int32_t* req_dev, int32_t* info_dev,
                 void* stream);

/* Rotary frequencies: pair i (elements i and i + head_dim/2, NEOX) turns by
 * pos[axis[i]] * theta^(-2i/head_dim) radians.  turn[i] holds theta^(-2i/head_dim)
 * / (2 pi) in units of 2^-64 of a turn, so that a position times it, modulo 2^64, is
 * the angle without a reduction error at any position. */
typedef struct sd_rope {
    uint64_t turn[64];
    uint8_t axis[64];
    int32_t head_dim, n_axes;
} sd_rope;

/* Fill *out (host memory) for head_dim 64 or 128, theta > 1, and n_axes (1 to 4)
 * position axes: pairs[a] of the head_dim/2 pairs belong to axis a (time, height,
 * width, ...).  interleaved 0: the first pairs[0] pairs are axis 0's, the next
 * pairs[1] axis 1's, and so on; otherwise the axes take turns pair by pair, an
 * axis without pairs left being passed over.  pairs may be NULL for one axis. */
int sd_rope_init(int32_t head_dim, double theta, int32_t n_axes, const int32_t* pairs, int32_t interleaved,
                 sd_rope* out);

/* Rotate n tokens' queries and keys and write keys and values into the pages
 * (journal section 3.13's write at n_past, for tokens of any request): token i,
 * with positions pos_dev[a * pos_stride + i] on axis a (any int32), goes to slot
 * slot_dev[i].  A token whose slot is negative or not below n_pages * page_size is
 * skipped: nothing of it is written.  q_dev [n][n_head][head_dim] (rows q_stride
 * elements apart) is rotated to q_out_dev (rows q_out_stride apart; may be q_dev
 * with the same stride); q_dev NULL: no queries (n_head 0).  k_dev / v_dev
 * [n][n_kv_head][head_dim], rows kv_stride apart: parts of one fused projection's
 * rows are given by their strides.  dtype (q, k, v and q_out): SD_F32, SD_F16 or
 * SD_BF16.  Pointers are 16-byte aligned, strides multiples of 16 bytes.  rope
 * NULL: nothing is rotated (pos_dev NULL; q_out is a copy of q).  Rotated in
 * fp32 and rounded once; SD_E4M3: value / scale, limited to +-448.  Slots of
 * a call are distinct (of two tokens with one slot either may remain). */
int sd_rope_write_pages(const sd_rope* rope, const int32_t* pos_dev, int64_t pos_stride, const int32_t* slot_dev,
                        int32_t n, int32_t dtype, const void* q_dev, int64_t q_stride, void* q_out_dev,
                        int64_t q_out_stride, int32_t n_head, const void* k_dev, const void* v_dev,
                        int64_t kv_stride, const sd_pages* cache, void* stream);

/* Workspace of the attention entries below: the partial results of split
 * lengths and of groups, fixed at about 80 MB, allocated here on `device` (-1: the current one).
 * Calls with one workspace, replays of graphs that captured one among them, must
 * not overlap: one workspace for each stream.  A kernel whose bounded waits (about
 * two seconds each) expire leaves its results unfinished; every later call with the
 * workspace returns SD_ERR_TIMEOUT, and what was captured or queued before runs on
 * but writes NaN to all its results (out_dev and lse_dev). */
typedef struct sd_attn_ws sd_attn_ws;
/* Not while a stream is being captured. */
int sd_attn_ws_create(int32_t device, sd_attn_ws** out);
void sd_attn_ws_destroy(sd_attn_ws* ws);

/* Attention of one new token per request over the paged cache: with g = h / (n_head /
 * n_kv_head) and len = len_dev[r],
 *   out[r][h] = sum_{j < len} softmax_j(scale * q[r][h] . K[g][j]) V[g][j],
 * position j in page table_dev[r * table_stride + j / page_size]. len 0 (or negative)
 * gives zeros; a len beyond table_stride * page_size (or 2^31 - 1024) is limited to it;
 * the positions of a page id outside [0, n_pages) are left out, as if masked. Nothing
 * behind len is used, whatever it holds. (An infinite or NaN element of V at a used
 * position makes its output element infinite or NaN.) out_dev overlaps no other
 * argument. (A row whose scores are all -inf gives zeros, like one without positions.)
 * dtype (q and out): SD_F32 (with an SD_F16 or SD_E4M3 cache), SD_F16 or
 * SD_BF16. q_dev [R][n_head][head_dim] with rows q_stride elements apart, out_dev the
 * same with out_stride; pointers are 16-byte aligned, strides multiples of 16 bytes.
 * lse_dev [R][n_head] (may be NULL): the natural logarithm of the softmax's denominator,
 * -inf for len 0. n_head is a multiple of n_kv_head; an SD_E4M3 cache of head_dim 64
 * needs an even page_size. SD_F32 q enters the products with 22 bits (elements below
 * 2^-14 of their row's largest with an error of 2^-37 of it), 16-bit types exactly (SD_BF16
 * with other caches: elements below 2^-17 with an error of 2^-25 of the largest).
 * Probabilities enter with 22 bits for SD_F32 results, 16 on SD_BF16 caches, 11 otherwise
 * (on SD_F16 and SD_E4M3 caches small ones have an error of up to 2^-40 of the largest);
 * sums and statistics are fp32. */
int sd_attend_pages(sd_attn_ws* ws, const sd_pages* cache, const int32_t* table_dev, int32_t table_stride,
                    const int32_t* len_dev, int32_t R, int32_t dtype, const void* q_dev, int64_t q_stride,
                    int32_t n_head, float scale, void* out_dev, int64_t out_stride, float* lse_dev, void* stream);

/* Keys and values of an encoder's states, [B][n_pos][n_kv_head][head_dim] by
 * default (all three strides 0); other orders by their strides (elements, positive
 * multiples of 16 bytes; pointers 16-byte aligned).  len_dev[b] states of row b
 * are used (limited to [0, n_pos]; NULL: n_pos).  dtype SD_F16 or SD_BF16. */
typedef struct sd_states {
    const void* k_dev;
    const void* v_dev;
    const int32_t* len_dev;
    int64_t batch_stride, head_stride, pos_stride;
    int32_t dtype, B, n_pos, n_kv_head, head_dim, reserved;
} sd_states;

/* Cross attention: every query i < Lq of row b attends to all len[b] states of its row,
 * whatever Lq is (masks, values that are not finite and overlap as in sd_attend_pages),
 *   out[b][i][h] = sum_{j < len} softmax_j(scale * q[b][i][h] . K[b][g][j]) V[b][g][j].
 * q_dev [B][Lq][n_head][head_dim]: batch rows q_batch elements apart (unused for B 1),
 * queries q_stride apart; out_dev the same with out_batch, out_stride. A row without
 * states gives zeros. States behind len are not used, whatever they hold. dtype (q and
 * out): SD_F32 (with SD_F16 states), SD_F16 or SD_BF16. lse_dev [B][Lq][n_head] (may be
 * NULL) as in sd_attend_pages. Precision as there; many queries of one 16-bit type with
 * their states enter probabilities with that type's bits (SD_BF16: 8): never with up to
 * 16 query rows to a kv head (Lq * n_head / n_kv_head) over SD_BF16 states, always from
 * 24 queries on, if the scale is positive. */
int sd_attend_cross(sd_attn_ws* ws, const sd_states* states, int32_t dtype, const void* q_dev, int64_t q_batch,
                    int64_t q_stride, int32_t Lq, int32_t n_head, float scale, void* out_dev, int64_t out_batch,
                    int64_t out_stride, float* lse_dev, void* stream);

/* ---- Rollouts: rows that continue one another's cache, and what picks among them.  Conventions as
 * above: stream-ordered, nothing allocated or waited for, buffers of the current device
 * (sd_attend_shared: of its workspace's device).  The buffers of a call must not overlap,
 * but for what is said. */

/* int32 words of work_dev (8-byte aligned, any contents; one for each call that may run beside another) for sd_page_fork with R rows, N new rows and n_pages
 * pages, and for sd_page_compact (N 0).  0 for negative counts or n_pages below 1. */
int64_t sd_page_work(int32_t R, int32_t N, int32_t n_pages);

/* Rows of the next step from rows of this one (rollouts of a prompt, beams, requests that end).  New row
 * i < N continues old row p = parent_dev[i], any number of new rows the same one; a parent outside
 * [0, R) gives an empty row.  Row p has len_dev[p] positions in the pages table_dev [R][table_stride]
 * names.  Their full pages are shared.  The partly filled page stays with the lowest of the rows that
 * continue p; each other one takes the next page of free_dev[n_free], in the order of the rows, and the
 * positions have to be copied there.  Outputs:
 *   table_out_dev [N][table_stride]  pages of the new rows, -1 behind their last
 *   len_out_dev [N]        their positions
 *   copy_dev [N][3]        source page, destination page and positions of each copy (sd_page_copy)
 *   ref_dev [n_pages]      how many new rows name the page
 *   free_out_dev [n_pages] the free pages from now on: the rest of free_dev, then the pages that
 *                          old rows named and no new row does, in ascending order
 *   info_dev [4]           copies; free pages; what went wrong (bits); longest new row
 * What lies behind the copies and the free pages stays as it was.  Bits of info_dev[2]:
 *   2 the free list is too short: the rows it does not serve end before their partly filled page
 *   4 a row is longer than its table row (limited to it)
 *   8 a negative length (read as 0)
 *  16 a page id outside [0, n_pages) in use or taken: -1 in the new row, counted nowhere; a copy
 *     from or to it names -1, and a row that took it ends before that page
 * A partly filled page belongs to one old row, and no free page is in use.  R, N and n_free may be 0 (the
 * pointers that belong to them may be NULL then).  page_size 1 to 65536, n_pages * page_size at most 2^31 - 1,
 * n_pages at most 2^26, N at most 2^20, table_stride at most 2^30. */
int sd_page_fork(const int32_t* table_dev, int32_t table_stride, const int32_t* len_dev, int32_t R,
                 const int32_t* parent_dev, int32_t N, const int32_t* free_dev, int32_t n_free, int32_t page_size,
                 int32_t n_pages, int32_t* table_out_dev, int32_t* len_out_dev, int32_t* copy_dev, int32_t* ref_dev,
                 int32_t* free_out_dev, int32_t* info_dev, int32_t* work_dev, void* stream);

/* The pages in use moved to the front of the pool: with L of them, the page in use with the k-th lowest id
 * from L on moves to the k-th lowest id below L that is not in use.  A page is in use if one of
 * the R rows names it.  Outputs:
 *   table_out_dev [R][table_stride]  the rows with the new ids, -1 behind their last page
 *   copy_dev [n_pages / 2][3]  the moves: source, destination, page_size (sd_page_copy); the
 *                              rest stays as it was
 *   ref_dev [n_pages]          how many rows name the page now
 *   free_out_dev [n_pages]     L, L + 1, ..., n_pages - 1; the rest stays as it was
 *   info_dev [4]               moves; n_pages - L; bits 4, 8 and 16 as in sd_page_fork; L
 * Sizes as in sd_page_fork. */
int sd_page_compact(const int32_t* table_dev, int32_t table_stride, const int32_t* len_dev, int32_t R,
                    int32_t page_size, int32_t n_pages, int32_t* table_out_dev, int32_t* copy_dev, int32_t* ref_dev,
                    int32_t* free_out_dev, int32_t* info_dev, int32_t* work_dev, void* stream);

/* Copies pages within each of n_caches (up to 128; the layers') caches of one type, shape and strides: for each
 * c < min(count_dev[0], max_copies), positions [0, copy_dev[c][2]) of page copy_dev[c][0] to page
 * copy_dev[c][1], keys and values of all heads.  The positions are limited to [0, page_size]; a copy
 * from or to a page id outside [0, n_pages) is skipped, one of a page to itself does nothing.
 * No copy's destination is another copy's source or destination.  max_copies or n_caches 0 does nothing. */
int sd_page_copy(const sd_pages* caches, int32_t n_caches, const int32_t* copy_dev, const int32_t* count_dev,
                 int32_t max_copies, void* stream);

/* sd_attend_pages for requests that share their first pages (rollouts of one prompt): the same results, with the
 * common keys and values read once for a group instead of once a request.  Group x is
 * requests group_dev[x] to group_dev[x + 1] - 1 (x < n_groups <= R; ascending, between 0 and R; group_dev has
 * n_groups + 1 numbers, all on the device), whose table rows name the same pages in their first
 * shared_dev[x] entries; the page ids are taken from any of those rows.  A request in no group, or with shorter
 * length than the group's pages, is served too.  n_groups 0: sd_attend_pages.  Everything else as in sd_attend_pages.
 * (With SD_F32 queries an infinite key at a shared position may give NaN.)  Groups are served together where that saves
 * reading enough: 150 MB of keys and values, 75 MB with SD_F32 queries (the device decides, from the groups).  Each
 * request is served by itself below that, with SD_E4M3 pages, a scale of 0 or outside 2^-60 to 2^60, and
 * more than 65536 query heads in all (R * n_head). */
int sd_attend_shared(sd_attn_ws* ws, const sd_pages* cache, const int32_t* table_dev, int32_t table_stride,
                     const int32_t* len_dev, int32_t R, const int32_t* group_dev, const int32_t* shared_dev,
                     int32_t n_groups, int32_t dtype, const void* q_dev, int64_t q_stride, int32_t n_head, float scale,
                     void* out_dev, int64_t out_stride, float* lse_dev, void* stream);

/* Scores of rows of logits [rows][V] (rows `stride` elements apart, dtype SD_F32, SD_F16 or SD_BF16, any
 * alignment of whole elements), p = softmax(z / temperature):
 *   logp_dev[r]     log p of token token_dev[r]
 *   rank_dev[r]     how many entries are ahead of it: with a larger logit, or the same and a lower index
 *   entropy_dev[r]  -sum p log p (natural logarithms)
 *   top_id_dev, top_logp_dev [rows][top_n]   the first top_n entries in that order, and their log p
 * logp_dev, rank_dev and entropy_dev may be NULL; token_dev if the first two are.  A token outside [0, V)
 * (padding) has logp 0 and rank -1.  A logit of -inf (masked) has p 0 and is no alternative: places without one
 * hold -1 and -inf.  A row of -inf alone: logp -inf, entropy 0.  NaN or +inf in a row makes its
 * logp, entropy and top_logp NaN; NaN is ahead of nothing and no alternative.  Sums are fp32.  1 <= V <= 262144,
 * 0 <= top_n <= 32, temperature between 1e-30 and 1e30. */
int sd_score_rows(const void* logits_dev, int64_t stride, int32_t dtype, int32_t rows, int32_t V, float temperature,
                  const int32_t* token_dev, float* logp_dev, int32_t* rank_dev, float* entropy_dev, int32_t top_n,
                  int32_t* top_id_dev, float* top_logp_dev, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SD_OPS_H */
