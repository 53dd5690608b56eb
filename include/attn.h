/*
 * attn.h — C ABI of the GB300 (sm_103a) attention-forward library.
 *
 * One call computes, for every batch b, query head h and query row i,
 *
 *   O[b,h,i,:] = softmax_j( scale * Q[b,h,i,:] . K[b,kvh,j,:] ) V[b,kvh,j,:]
 *
 * over the keys j that are visible to row i, plus the row's log-sum-exp.
 * Sources (web pages this library restates):
 *   - "Flash Attention in CUDA Tile (cuTile)" (NVIDIA blog), sections
 *     "What is attention?" and "Understanding online softmax": the operation
 *     and the tiled online-softmax method that computes it exactly;
 *   - same page, section "Causal attention" and the kernel listing's
 *     "Applying the causal mask" step: key j is visible to query row i iff
 *     j <= input_pos + i (queries sit at absolute positions input_pos + i,
 *     the KV-cache offset of the listing's "Initializing accumulators" step);
 *   - same page, section "Grouped-query attention": kvh = h / (Hq / Hkv);
 *   - same page, host-launcher section: [B, H, S, D] contiguous tensors,
 *     the scale defaulting to 1/sqrt(D) on the Python side.
 *
 * No function here allocates device memory; the caller owns every buffer.
 * (attn_fwd_splitkv_noalloc's scratch is a fixed array compiled into the
 * library, which every GPU that loads it holds, not an allocation.)
 */
#ifndef ATTN_FWD_GB300_ATTN_H
#define ATTN_FWD_GB300_ATTN_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t / CUstream; NULL is the legacy default stream. */
struct CUstream_st;
typedef struct CUstream_st* attn_stream_t;

/* Element type of Q, K, V and O. */
typedef enum {
  ATTN_F16 = 0,  /* IEEE binary16 */
  ATTN_BF16 = 1, /* bfloat16 */
  ATTN_E4M3 = 2  /* OCP FP8 E4M3 ("e4m3fn") inputs with a bfloat16 O: only
                    attn_fwd_fp8, attn_splitkv_plan and attn_tile_config
                    take it; elsewhere ATTN_ERR_INVALID_ARG (ATTN_ERR_-
                    UNSUPPORTED for attn_bwd) */
} attn_dtype_t;

/* Return codes.  Everything but ATTN_OK leaves O and LSE untouched. */
typedef enum {
  ATTN_OK = 0,
  ATTN_ERR_INVALID_ARG = 1,  /* bad size, NULL or host pointer, bad dtype   */
  ATTN_ERR_UNSUPPORTED = 2,  /* valid but not implemented (D not 64 or 128) */
  ATTN_ERR_ALIGNMENT = 3,    /* Q/K/V/O not 16-byte or LSE not 4-byte aligned */
  ATTN_ERR_CUDA = 4,         /* a CUDA runtime/driver call failed            */
  ATTN_ERR_TIMEOUT = 5       /* a kernel pipeline wait ran out (device status) */
} attn_status_t;

/*
 * attn_fwd — scaled-dot-product attention forward on the GPU.
 *
 * Q    device, [B, Hq,  Sq,  D] contiguous, dtype      (read)
 * K    device, [B, Hkv, Skv, D] contiguous, dtype      (read)
 * V    device, [B, Hkv, Skv, D] contiguous, dtype      (read)
 * O    device, [B, Hq,  Sq,  D] contiguous, dtype      (written)
 * LSE  device, [B, Hq,  Sq] float32, or NULL to skip   (written)
 *      LSE[b,h,i] = ln( sum over visible j of exp(scale * q_i . k_j) ),
 *      natural log, scale included.
 * B >= 0, Hq > 0, Hkv > 0 with Hq % Hkv == 0, Sq >= 0, Skv >= 1,
 * D in {64, 128}.  B == 0 or Sq == 0 is a successful no-op.
 * scale     finite; any sign (0 gives uniform weights over visible keys).
 * causal    0: every key is visible and input_pos is ignored;
 *           non-zero: key j is visible to query row i iff j <= input_pos + i.
 *           Queries with input_pos + i >= Skv - 1 see every key.
 * input_pos >= 0, and input_pos + Sq + 512 must fit in a signed 32-bit int.
 * dtype     ATTN_F16 or ATTN_BF16 (Q, K, V and O share it).
 * stream    the CUDA stream the kernel is enqueued on.
 *
 * Q/K/V/O must be 16-byte aligned (tensor-memory-accelerator copies), LSE
 * 4-byte aligned; O must not overlap Q, K or V.  The call is asynchronous:
 * the return code covers argument checks and the launch only.  A device
 * side pipeline timeout is reported later by attn_device_status().
 * Results are deterministic for a given shape and dtype.
 */
attn_status_t attn_fwd(const void* Q, const void* K, const void* V, void* O,
                       float* LSE, int B, int Hq, int Hkv, int Sq, int Skv,
                       int D, float scale, int causal, int input_pos,
                       attn_dtype_t dtype, attn_stream_t stream);

/*
 * attn_fwd_window — attn_fwd with a causal sliding window: the query at
 * absolute position p = input_pos + i sees the keys j with
 * p - window < j <= p (its last `window` positions, itself included).
 * "Flash Attention from Scratch", section "What's Next", names sliding
 * window attention for ultra-long sequences as future work without
 * defining it; this is the plain reading consistent with the causal offset
 * rule above.  Key tiles wholly before a query tile's window are skipped
 * like those past its causal horizon.
 *
 * Arguments as attn_fwd, plus:
 * window   >= 0 keys; 0 means no window (the result of attn_fwd).  A
 *          window needs causal != 0, and every query must see a key
 *          (input_pos + Sq - window < Skv); otherwise
 *          ATTN_ERR_INVALID_ARG.
 */
attn_status_t attn_fwd_window(const void* Q, const void* K, const void* V,
                              void* O, float* LSE, int B, int Hq, int Hkv,
                              int Sq, int Skv, int D, float scale, int causal,
                              int input_pos, int window, attn_dtype_t dtype,
                              attn_stream_t stream);

/*
 * attn_fwd_splitkv — the same operation as attn_fwd, with the key range cut
 * into num_splits pieces of equal length (multiples of 128 keys) that are
 * processed in parallel, then merged by their log-sum-exps: for a row with
 * partial results (O_c, lse_c), O = sum_c w_c O_c / sum_c w_c and
 * LSE = M + ln(sum_c w_c) with w_c = exp(lse_c - M), M = max_c lse_c.
 * This is the KV-cache decoding shape (few query rows, long key range)
 * where attn_fwd alone would leave most SMs idle; it is the online-softmax
 * rescaling of "Flash Attention in CUDA Tile (cuTile)", section "The online
 * softmax algorithm", applied across key ranges.
 *
 * Arguments as attn_fwd, plus:
 * num_splits       1..128, a value returned by attn_splitkv_plan for the
 *                  same shape (other counts give ATTN_ERR_INVALID_ARG);
 * workspace        device memory owned by the caller, 256-byte aligned,
 *                  of at least the size attn_splitkv_plan reports: fp32
 *                  partial outputs [num_splits, B, Hq, Sq, D], fp32
 *                  partial LSEs [num_splits, B, Hq, Sq]; its contents
 *                  need no initialisation (every value read is written
 *                  first by the same call);
 * workspace_bytes  its size.
 * Enqueued on `stream`: the forward kernel, and unless its key ranges merge
 * inside thread-block clusters (GQA-packed launches whose units all run at
 * once, at most 8 ranges), a merge kernel after it (a programmatic
 * dependent launch: its blocks start once every forward block has and wait
 * for the forward grid to complete).  The workspace must not be used by
 * another call until this one has run.
 */
attn_status_t attn_fwd_splitkv(const void* Q, const void* K, const void* V,
                               void* O, float* LSE, int B, int Hq, int Hkv,
                               int Sq, int Skv, int D, float scale, int causal,
                               int input_pos, attn_dtype_t dtype,
                               int num_splits, void* workspace,
                               size_t workspace_bytes, attn_stream_t stream);

/*
 * attn_fwd_splitkv_window — attn_fwd_splitkv with the sliding window of
 * attn_fwd_window (same `window` rule).  Plan with attn_splitkv_plan (the
 * plan does not depend on the window); ranges wholly outside a row
 * block's window are skipped.
 */
attn_status_t attn_fwd_splitkv_window(const void* Q, const void* K,
                                      const void* V, void* O, float* LSE,
                                      int B, int Hq, int Hkv, int Sq, int Skv,
                                      int D, float scale, int causal,
                                      int input_pos, int window,
                                      attn_dtype_t dtype, int num_splits,
                                      void* workspace, size_t workspace_bytes,
                                      attn_stream_t stream);

/*
 * attn_fwd_fp8 — attention forward with 8-bit floating-point inputs.
 * "Flash Attention from Scratch", section "What's Next", names FP8 tensor
 * cores as future work without defining a format; the reading taken: Q, K
 * and V hold OCP E4M3 codes (sign, 4-bit exponent with bias 7, 3-bit
 * mantissa, no infinities, S.1111.111 is NaN; torch.float8_e4m3fn) with one
 * fp32 descale factor per tensor, and the call computes the operation of
 * attn_fwd_window on the real values
 *   Q = q_descale * Q8,  K = k_descale * K8,  V = v_descale * V8.
 * Both products run on the FP8 tensor cores with fp32 accumulation; the
 * softmax weights are rounded to E4M3 for the P.V product (the row sums
 * use them unrounded), which bounds the accuracy: each weight carries up to
 * 2^-4 relative rounding (absolute 2^-10 below 2^-6).  The LSE is exact to
 * fp32 rounding.
 *
 * Q, K, V  device, layouts as attn_fwd, one byte per element (read);
 * O        device, [B, Hq, Sq, D] bfloat16 (written);
 * LSE      device fp32 [B, Hq, Sq] or NULL: ln-sum-exp of the scores
 *          scale * q_descale * k_descale * Q8.K8 (written);
 * D        128 only (else ATTN_ERR_UNSUPPORTED);
 * scale, q_descale, k_descale, v_descale  finite, any sign; the product
 *          scale * q_descale * k_descale must be finite in fp32;
 * causal, input_pos, window  as attn_fwd_window;
 * num_splits  0: one pass (workspace ignored); >= 1: the split-KV form of
 *          attn_fwd_splitkv_window with a count from attn_splitkv_plan
 *          (dtype ATTN_E4M3) and its workspace rules;
 * Other rules and errors as attn_fwd.
 */
attn_status_t attn_fwd_fp8(const void* Q, const void* K, const void* V,
                           void* O, float* LSE, int B, int Hq, int Hkv,
                           int Sq, int Skv, int D, float scale,
                           float q_descale, float k_descale, float v_descale,
                           int causal, int input_pos, int window,
                           int num_splits, void* workspace,
                           size_t workspace_bytes, attn_stream_t stream);

/*
 * attn_splitkv_plan — split count and workspace size for attn_fwd_splitkv.
 * *num_splits in: the requested count, or <= 0 to choose the count with
 * the shortest estimated time on the current device's SMs (152, a GB300's,
 * when the calling thread has no CUDA device): waves of units times key
 * tiles per range plus fixed per-unit and merge costs, bounded below by
 * streaming K and V once from HBM; out: the count attn_fwd_splitkv accepts
 * (requests are clamped to the number of 128-key tiles, and trailing empty
 * ranges are dropped).  Host only: launches nothing.
 * *workspace_bytes (may be NULL) receives the workspace size.
 */
attn_status_t attn_splitkv_plan(int B, int Hq, int Hkv, int Sq, int Skv, int D,
                                int causal, int input_pos, attn_dtype_t dtype,
                                int* num_splits, size_t* workspace_bytes);

/*
 * attn_fwd_splitkv_noalloc — attn_fwd_splitkv for callers that cannot
 * allocate device memory (code running where the allocator must not be
 * entered, or inside a host that owns every allocation): the partial
 * results go to a fixed scratch array compiled into this library (its size
 * is attn_noalloc_scratch_bytes(), 16 MiB, held on every GPU that loads the
 * library until the process exits) instead of a caller workspace.  The
 * pages have no counterpart; this is a deployment convenience.
 *
 * Arguments as attn_fwd_splitkv without the workspace: num_splits <= 0
 * lets the library choose, and a positive count must be one that
 * attn_splitkv_plan keeps (otherwise ATTN_ERR_INVALID_ARG).  Returns
 * ATTN_ERR_UNSUPPORTED when the partial results of that split count need
 * more than the scratch holds.  The first call on a device (and the first
 * after a device reset, which replaces the context) looks up the scratch
 * address on that device (no allocation); make that first call before any
 * stream capture.  All calls share the one scratch array and it keeps the
 * last call's contents (nothing in it has to start at zero): calls whose
 * kernels overlap on the GPU race on it, so issue them on one stream or
 * otherwise order them.
 */
attn_status_t attn_fwd_splitkv_noalloc(const void* Q, const void* K,
                                       const void* V, void* O, float* LSE,
                                       int B, int Hq, int Hkv, int Sq, int Skv,
                                       int D, float scale, int causal,
                                       int input_pos, attn_dtype_t dtype,
                                       int num_splits, attn_stream_t stream);

/* Bytes of the fixed scratch array attn_fwd_splitkv_noalloc uses. */
size_t attn_noalloc_scratch_bytes(void);

/*
 * attn_bwd — backward pass: gradients dQ, dK, dV of the forward output O
 * for an upstream gradient dO.  "Flash Attention from Scratch", section
 * "What's Next", lists the backward pass as future work without formulas;
 * this is the chain rule on the forward's definition, recomputing P tile
 * by tile from the forward's LSE instead of storing it:
 *   P_ij = exp(scale q_i.k_j - LSE_i) on visible keys (0 elsewhere),
 *   D_i = sum_d dO_id O_id,  dV_j = sum_i P_ij dO_i,
 *   dS_ij = P_ij (dO_i.v_j - D_i),
 *   dQ_i = scale sum_j dS_ij k_j,  dK_j = scale sum_i dS_ij q_i,
 * with the query heads of a GQA group adding into the same dK, dV.
 *
 * Q, K, V, O, dO   device, same dtype and layouts as attn_fwd (O and LSE
 *                  are the forward's outputs for these Q, K, V and scale,
 *                  causal, input_pos, window);
 * LSE              device fp32 [B, Hq, Sq] (required);
 * dQ               device [B, Hq, Sq, D]; dK, dV device [B, Hkv, Skv, D];
 *                  outputs, same dtype, 16-byte aligned, overlapping no
 *                  input, each other or the workspace;
 * window           as attn_fwd_window (0: none);
 * workspace        device, 256-byte aligned, at least
 *                  attn_bwd_workspace_bytes(B, Hq, Sq) bytes (per-row
 *                  lse2 and D); contents need no initialisation;
 * Three kernels: the row pass and the dK/dV kernel on `stream`, the dQ
 * kernel on an internal stream forked from `stream` after the row pass and
 * joined back into it (event record / wait), so the two run concurrently
 * and later work on `stream` waits for both; this works under stream
 * capture.  The first call on a host thread and device creates that
 * internal stream and its two events (make it before any capture).  Every
 * output element has one writer, so results are deterministic.  Sq = 0
 * writes zero dK, dV.  Errors as attn_fwd.
 */
attn_status_t attn_bwd(const void* Q, const void* K, const void* V,
                       const void* O, const float* LSE, const void* dO,
                       void* dQ, void* dK, void* dV, int B, int Hq, int Hkv,
                       int Sq, int Skv, int D, float scale, int causal,
                       int input_pos, int window, attn_dtype_t dtype,
                       void* workspace, size_t workspace_bytes,
                       attn_stream_t stream);

/* Workspace bytes attn_bwd needs for B x Hq x Sq query rows: two fp32
 * values per row, Sq padded to a multiple of 128 (0 on negative sizes). */
size_t attn_bwd_workspace_bytes(int B, int Hq, int Sq);

/*
 * attn_kv8_t — a KV cache held in 8 bits: E4M3 codes with one fp32 scale for
 * each block of `block` consecutive tokens of a (batch, K/V head), separate
 * for K and V.  Token j of head (b, h) stands for the numbers
 *   k[b,h,j,:] = k_scale[b,h, j / block] * K8[b,h,j,:]   (V likewise).
 * "Flash Attention from Scratch", section "What's Next", names FP8 without a
 * format; attn_fwd_fp8 above takes one factor per tensor, this cache one per
 * block, so that late tokens do not have to share the range of early ones.
 *
 * k, v       device, [B, Hkv, capacity, D] one byte per element, 16-byte
 *            aligned;
 * k_scale, v_scale  device fp32 [B, Hkv, ceil(capacity / block)], 4-byte
 *            aligned; positive normal numbers for every block that holds a
 *            token (attn_kv8_append and attn_kv8_evict write powers of two,
 *            2^-126 to 2^120);
 * lens       device int32 [B]: tokens of sequence b in the cache, the new
 *            tokens of the current step included, 0 <= lens[b] <= capacity.
 *            One array may serve the caches of all layers; no function
 *            changes the lens of a cache it reads or appends to.  A value
 *            outside the range is taken as the nearer end of it and reported
 *            by attn_device_status (bit 1 of the code).
 * B >= 0, Hkv > 0, 1 <= capacity < 2^31 - 2^16 - 1, D in {64, 128}, block in
 * {16, 32, 64, 128}; B * Hkv < 2^24.  Codes and scales of tokens at lens[b] or later are never
 * read: they need no initialisation.
 */
typedef struct {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int* lens;
  int B, Hkv, capacity, D, block;
} attn_kv8_t;

/*
 * attn_kv8_append — quantise the K and V of new tokens into the cache.
 * The new tokens of sequence b are its last n_b tokens, positions
 * lens[b] - n_b .. lens[b] - 1, with n_b = Sq, or new_lens[b].
 *
 * K, V      device, [B, Hkv, Sq, D] contiguous, dtype, 16-byte aligned (read);
 *           rows i >= n_b are ignored;
 * new_lens  device int32 [B] or NULL (n_b = Sq): 0 <= n_b <= Sq and
 *           n_b <= lens[b]; values outside are taken as the nearer end and
 *           reported like lens;
 * dtype     ATTN_F16 or ATTN_BF16.
 *
 * Let a be the largest finite magnitude among the new tokens of one block of
 * one head, and tight(a) the smallest power of two (2^-126 at least, 2^127 at
 * most) with a <= 448 * tight(a).  A block that holds no earlier token gets the
 * scale tight(a).  A block begun by earlier calls keeps its scale when
 * a <= 448 * scale; else its scale becomes tight(a) and the codes it holds
 * are requantised, round(code * old / new) -- with powers of two an exponent
 * shift, exact unless the result is subnormal.  New codes are
 * round(x / scale): to nearest, ties to even (a scale of other origin: after
 * the fp32 rounding of the quotient); infinities become +-448, NaN
 * stays NaN.  Nothing else of the cache is written.  Sq <= capacity.
 * Deterministic.
 */
attn_status_t attn_kv8_append(const attn_kv8_t* cache, const void* K,
                              const void* V, int Sq, const int* new_lens,
                              attn_dtype_t dtype, attn_stream_t stream);

/*
 * attn_kv8_fwd — attention of Sq query rows per sequence over an 8-bit
 * cache, in the scores, softmax and sums of attn_fwd (fp32), on the numbers
 * the cache stands for.  As there, the softmax's weights are rounded to 16
 * bits for their product with V: to fp16, 2^-11 relative down to 2^-21 of the
 * row's largest.
 *
 * Q         device, [B, Hq, Sq, D] contiguous, dtype (read);
 * O         device, [B, Hq, Sq, D] contiguous, dtype (written);
 * LSE       device fp32 [B, Hq, Sq] or NULL (written);
 * weights   device fp32 [B, Hkv, capacity] or NULL: the attention weight each
 *           cached token receives is added to it,
 *             weights[b,h,j] += sum over the query heads of K/V head h and
 *                               the rows i of softmax_ij;
 *           entries of tokens nobody sees keep their bits;
 * new_lens  device int32 [B] or NULL (n_b = Sq): rows i < n_b are computed,
 *           0 <= n_b <= Sq; O and LSE of rows i >= n_b are left as they are
 *           and their Q is ignored;
 * causal    non-zero: row i of sequence b sits at position
 *           lens[b] - n_b + i and sees the tokens up to it (the new tokens
 *           are the cache's last n_b); 0: every row sees all lens[b] tokens
 *           (cross attention to cached encoder states).
 *           A row that sees no token gets O = 0 and LSE = -inf.
 * Hq        a multiple of the cache's Hkv; scale finite, any sign;
 * dtype     ATTN_F16 or ATTN_BF16;
 *           NaN: a row of Q with NaN gets NaN and leaves the others alone; a
 *           NaN code of K reaches the rows that see its token; a NaN code of V
 *           may reach every row of its sequence and head in the call, also
 *           rows before its token (0 * NaN, as in attn_fwd).  A V scale
 *           more than 2^22 (2^64 where Hq / Hkv * Sq <= 16) below the
 *           largest one among the lens[b] tokens of its sequence and head
 *           costs precision: its numbers are then off by up to 2^-23 of the
 *           largest scale.  V scales that are no powers of two add two
 *           roundings of 2^-11 where Hq / Hkv * Sq > 16;
 * workspace device, 256-byte aligned, at least attn_kv8_workspace_bytes(...)
 *           bytes; contents need no initialisation.  It must not be used by
 *           another call until this one has run.  Where weights are
 *           accumulated under 16 or fewer query rows per K/V head it holds
 *           their scores: 4 bytes for every row (of Hq / Hkv * Sq, rounded up
 *           to a power of two) and every one of the capacity's tokens of a
 *           head, up to 64 bytes a token against 2 D of codes.
 * One to three kernels on `stream` (one over short caches, three with weights
 * of more than 16 query rows per K/V head).  O, LSE, weights and workspace must
 * not overlap each other or any input.  B == 0 or Sq == 0 is a successful
 * no-op.  Deterministic for a given device, shape and lengths; O and LSE are
 * the same with and without weights.
 */
attn_status_t attn_kv8_fwd(const attn_kv8_t* cache, const void* Q, void* O,
                           float* LSE, float* weights, int Hq, int Sq,
                           const int* new_lens, float scale, int causal,
                           attn_dtype_t dtype, void* workspace,
                           size_t workspace_bytes, attn_stream_t stream);

/* Workspace bytes attn_kv8_fwd needs (0 on bad sizes); `weights` non-zero
 * when the call accumulates attention weights.  Host only; the value is for
 * the current device's SM count (152 without a device). */
size_t attn_kv8_workspace_bytes(int B, int Hq, int Hkv, int Sq, int capacity,
                                int D, int weights);

/*
 * attn_kv8_evict — keep the tokens of a cache that received the most
 * attention.  For every sequence with lens[b] > keep and every K/V head,
 * the `recent` last tokens stay, and of the others the keep - recent with
 * the largest weights (equal weights: the earlier token; NaN counts as less
 * than every number).  Kept tokens keep their order and become tokens
 * 0 .. keep - 1 of the same head of `dst`: per block of dst the scale is
 * tight(largest magnitude of its kept numbers) and the codes are
 * requantised as in attn_kv8_append.  Sequences with lens[b] <= keep are
 * copied bit for bit.
 *
 * src          the cache (read);
 * dst          the cache written: its k, v, scales, and lens (lens[b]
 *              becomes min(lens[b], keep)).  Either all of k, v and both
 *              scales are other memory than src's (any capacity >= keep), or
 *              all four are src's own (in place, same capacity).
 *              dst->lens is always other memory than src->lens.  B, Hkv, D
 *              and block must agree.
 * weights      device fp32 [B, Hkv, src capacity] (read);
 * dst_weights  device fp32 [B, Hkv, dst capacity] (written): the kept
 *              tokens' weights, then zeros to the capacity.  In place it may
 *              be `weights` itself; else it must not overlap it;
 * keep, recent 1 <= keep <= dst capacity, 0 <= recent <= keep;
 * indices      device int32 [B, Hkv, keep] (written): the place in src of
 *              each kept token, ascending; -1 behind the last one.
 * Two kernels on `stream`.  Codes and scales of dst behind the kept tokens'
 * last block are left as they are.  Deterministic.
 */
attn_status_t attn_kv8_evict(const attn_kv8_t* src, const attn_kv8_t* dst,
                             const float* weights, float* dst_weights,
                             int keep, int recent, int* indices,
                             attn_stream_t stream);

/*
 * attn_rope_t — a rotation of heads by position, on one or several axes.
 * The pages' listings take Q and K as they come; this is what a decoder does
 * to them before.  The first `rot` of a head's D elements form rot / 2 pairs:
 * (i, i + rot / 2), or with `interleaved` (2i, 2i + 1).  At position t_a on
 * axis a, pair i with axis[i] = a turns by the angle t_a * freq[i]:
 *   (x, y) -> (x cos - y sin, x sin + y cos).
 *
 * phase  device, [rot / 2]: freq[i] in units of 2^-64 of a turn, from
 *        attn_rope_phase.  Positions are multiplied with it modulo 2^64, so
 *        that the fraction of a turn is exact at any distance; the angle, in
 *        (-pi, pi], is then off by 2^-23 of itself and a unit of the phase per
 *        position;
 * axis   device, [rot / 2] values below `axes`; not read when axes is 1.
 * D in {64, 128}, rot a multiple of 8 from 0 (norm only) to D, 1 <= axes <=
 * 255.
 */
typedef struct {
  const unsigned long long* phase;
  const unsigned char* axis;
  int D, rot, axes, interleaved;
} attn_rope_t;

/* A strided view [B, S, H, D] of 16-bit elements on the device, as a
 * projection gives them: p 16-byte aligned, strides in elements, multiples of
 * 8 and not negative (those of dimensions of one element are not read). */
typedef struct {
  void* p;
  long long stride_b, stride_s, stride_h;
} attn_heads_t;

/* Frequencies (radians per position, host, |freq| <= 2^32) to the phases of
 * attn_rope_t (host).  Host only. */
attn_status_t attn_rope_phase(const double* freq, int n,
                              unsigned long long* phase);

/*
 * attn_qk_rope — norm of queries and keys per head, their rotation, and the
 * layout that attention reads, in one pass: for every row x of D elements of
 * q and k
 *   n = x / sqrt(mean(x^2) + eps) * weight      (n = x without a weight)
 * and then the rotation above; v is copied.
 *
 * q          view with Hq heads; k, v  views with Hkv heads (read);
 * v          NULL (with v_out NULL): no values;
 * q_weight, k_weight  device [D] or NULL (no norm); float32 if weight_f32,
 *            else dtype;
 * eps        positive and finite (not looked at without a norm);
 * q_out      device, [B, Hq, S, D] contiguous (written);
 * k_out, v_out  device, [B, Hkv, capacity, D] contiguous (written), capacity
 *            >= S: row i of a sequence goes to place i, or with lens to place
 *            lens[b] - n_b + i, the last n_b of a cache whose length already
 *            counts them (attn_prefix_cache_t's k and v are such);
 * lens, new_lens  device int32 [B] or NULL: n_b = S, or new_lens[b] rows,
 *            0 <= n_b <= S, n_b <= lens[b] <= capacity.  Values outside are
 *            taken as the nearer end and reported by attn_device_status (bit 1
 *            of the code).  Rows i >= n_b are ignored and nothing is written
 *            for them;
 * positions  device int32 [axes, B, S] or NULL: then a row's position on every
 *            axis is its place (i, or lens[b] - n_b + i), plus *offset;
 * offset     device int32 [1] or NULL (0), only without positions.  (The
 *            length of a shared prefix ahead of the cache.)
 * dtype      ATTN_F16 or ATTN_BF16: of all views and outputs.
 *
 * Computed in fp32 and rounded once.  Rows whose squares pass fp32's largest
 * number are scaled by a power of two first.  Outputs must not overlap each
 * other nor the range of memory that a view spans.  B == 0 or S == 0 is a
 * successful no-op.  Deterministic.
 */
attn_status_t attn_qk_rope(const attn_rope_t* rope, const attn_heads_t* q,
                           const attn_heads_t* k, const attn_heads_t* v,
                           const void* q_weight, const void* k_weight,
                           int weight_f32, float eps, const int* positions,
                           const int* lens, const int* new_lens,
                           const int* offset, void* q_out, void* k_out,
                           void* v_out, int B, int S, int Hq, int Hkv,
                           int capacity, attn_dtype_t dtype,
                           attn_stream_t stream);

/*
 * attn_qk_rope_bwd — backward pass of attn_qk_rope without lens (every
 * sequence has S rows): from the gradients of its outputs, as attn_bwd leaves
 * them, those of its inputs and weights.  With dn the rotation of the upstream
 * gradient by the opposite angles, r = 1 / sqrt(mean(x^2) + eps) and g = dn *
 * weight:
 *   dx = r * (g - x r^2 mean(g x)),  dweight = sum over rows of dn * x r;
 * without a weight dx = dn.
 *
 * dq_out, dk_out, dv_out  device, [B, Hq or Hkv, S, D] contiguous (read);
 *            dv_out may be NULL (with dv NULL);
 * q, k       the forward's views (read where they were normed; else NULL
 *            will do);
 * dq, dk, dv views (written): the gradients of q, k and v.  No two of their
 *            places may share an element; they may be parts of one packed
 *            buffer: side by side within each token, as the forward's inputs
 *            may, or behind one another in each sequence or altogether
 *            (refused where no order of the strides shows them apart);
 * dq_weight, dk_weight  device float32 [D] (written), given exactly where the
 *            weight is; summed in fp32 in a fixed order;
 * workspace  device, 256-byte aligned, at least
 *            attn_qk_rope_bwd_workspace_bytes(D) bytes; contents need no
 *            initialisation; not looked at without weights.  It must not be
 *            used by another call until this one has run.
 * Other arguments as attn_qk_rope.  One kernel on `stream`, two with weights.
 * Outputs and workspace must not overlap each other or any input.  B == 0 or
 * S == 0 writes zeros to the weights' gradients.  Deterministic.
 */
attn_status_t attn_qk_rope_bwd(
    const attn_rope_t* rope, const void* dq_out, const void* dk_out,
    const void* dv_out, const attn_heads_t* q, const attn_heads_t* k,
    const void* q_weight, const void* k_weight, int weight_f32, float eps,
    const int* positions, const int* offset, const attn_heads_t* dq,
    const attn_heads_t* dk, const attn_heads_t* dv, float* dq_weight,
    float* dk_weight, int B, int S, int Hq, int Hkv, attn_dtype_t dtype,
    void* workspace, size_t workspace_bytes, attn_stream_t stream);

/* Workspace bytes attn_qk_rope_bwd needs (0 for another D than 64 and 128).
 * Host only; the value is for the current device's SM count (152 without a
 * device). */
size_t attn_qk_rope_bwd_workspace_bytes(int D);

/*
 * attn_prefix_cache_t — 16-bit keys and values of a batch whose sequences
 * share a prefix (a system prompt, a document, one prompt of many samples):
 * the prefix's are held once, each sequence's own behind it in a cache of its
 * own.  The pages' listings read one K and V per batch entry; here the B
 * sequences' query rows meet the prefix's keys together, so that these are
 * read once.
 *
 * prefix_k, prefix_v  device, [Hkv, prefix_capacity, D], 16-byte aligned;
 * prefix_len  device int32 [1]: tokens of the prefix, 0 <= *prefix_len <=
 *             prefix_capacity;
 * k, v        device, [B, Hkv, capacity, D], 16-byte aligned;
 * lens        device int32 [B]: a sequence's own tokens in k and v, the new
 *             ones of the current step included, 0 <= lens[b] <= capacity.
 * Lengths outside their range are taken as the nearer end of it and reported
 * by attn_device_status (bit 1 of the code).  What lies behind a length is not
 * used: it needs no initialisation.
 * B >= 0, Hkv > 0, B * Hkv < 2^24, capacities from 1 to below 2^31 - 2^16 - 1,
 * D in {64, 128}.
 */
typedef struct {
  const void* prefix_k;
  const void* prefix_v;
  const int* prefix_len;
  const void* k;
  const void* v;
  const int* lens;
  int B, Hkv, prefix_capacity, capacity, D;
} attn_prefix_cache_t;

/*
 * attn_prefix_fwd — attention of Sq query rows per sequence over the prefix
 * and the sequence's own tokens behind it, one softmax over both, in the
 * scores, softmax and sums of attn_fwd (fp32; the weights are rounded to the
 * inputs' type for their product with V).  For that product they are held
 * times a power of two.  In bf16 it is 2^-24: sums over 2^16 keys (2^24 of like
 * weights) stay within fp32 for every finite V, and a key's share of O is off by
 * 2^-126 at most, by which values of V below 2^-100 lose bits.  In fp16 it is
 * 2^7: weights down to 2^-21 of the row's largest keep their bits.
 *
 * Q         device, [B, Hq, Sq, D] contiguous, dtype (read);
 * O         device, [B, Hq, Sq, D] contiguous, dtype (written);
 * LSE       device fp32 [B, Hq, Sq] or NULL (written);
 * new_lens  device int32 [B] or NULL (n_b = Sq): rows i < n_b are computed,
 *           0 <= n_b <= Sq; O and LSE of rows i >= n_b are left as they are
 *           and their Q is ignored;
 * causal    non-zero: row i of sequence b is its own token lens[b] - n_b + i
 *           and sees the prefix and its own tokens up to it (the new tokens
 *           are its last n_b); 0: every row sees all lens[b] of them.
 *           A row that sees no token gets O = 0 and LSE = -inf.
 * Hq        a multiple of the cache's Hkv, 128 times it at most (else
 *           ATTN_ERR_UNSUPPORTED); scale finite, any sign;
 * dtype     ATTN_F16 or ATTN_BF16, of Q, O and the cache;
 *           NaN: a row of Q with NaN gets NaN and leaves the others alone; a
 *           NaN of K reaches the rows that see its token; a NaN or infinity of
 *           V may reach every row of the sequences that hold its token, also
 *           rows before it (0 * NaN, as in attn_fwd).
 * workspace device, 256-byte aligned, at least
 *           attn_prefix_workspace_bytes(...) bytes; contents need no
 *           initialisation.  It must not be used by another call until this
 *           one has run.
 * Two kernels on `stream`.  O, LSE and workspace must not overlap each
 * other or any input.  B == 0 or Sq == 0 is a successful no-op.  Deterministic
 * for a given device, shape and lengths.
 */
attn_status_t attn_prefix_fwd(const attn_prefix_cache_t* cache, const void* Q,
                              void* O, float* LSE, int Hq, int Sq,
                              const int* new_lens, float scale, int causal,
                              attn_dtype_t dtype, void* workspace,
                              size_t workspace_bytes, attn_stream_t stream);

/* Workspace bytes attn_prefix_fwd needs (0 on bad sizes).  Host only; the
 * value is for the current device's SM count (152 without a device). */
size_t attn_prefix_workspace_bytes(int B, int Hq, int Hkv, int Sq,
                                   int prefix_capacity, int capacity, int D);

/* Short English description of a status code (static storage). */
const char* attn_status_string(attn_status_t status);

/*
 * attn_device_status — synchronises the current device, then reads and
 * clears the library's device status word.  *code receives 0 when no kernel
 * wait has run out since the last call; otherwise a non-zero code
 * (bit 0: a wait timed out, bits 8-15 then name the pipeline role that gave
 * up; bit 1: a call that reads lengths on the device, attn_kv8_*, attn_qk_rope
 * or attn_prefix_fwd, met one outside its range and clamped it) and the function
 * returns ATTN_ERR_TIMEOUT, or ATTN_ERR_INVALID_ARG
 * when bit 1 alone is set.  code may be NULL.
 * Every wait of every kernel in flight ORs into the one word, so the
 * device-wide form sees them all; attn_stream_status below waits for one
 * stream only.
 */
attn_status_t attn_device_status(unsigned int* code);

/*
 * attn_stream_status — the same query ordered on one stream: waits for the
 * work already enqueued on `stream` (cudaStreamSynchronize of that stream
 * only; other streams keep running), reads the status word and enqueues on
 * `stream` the clearing of exactly the bits it reports.  The word is one
 * per device, shared by every stream and call, so a wait that ran out in a
 * kernel of another stream, finished before the read, is reported here too;
 * bits 8-15 name the role that gave up (in the forward kernel 1 producer,
 * 2 MMA issuer, 3 softmax, 4 epilogue; OR-ed when several gave up).  Not for use while `stream` is being captured.  code
 * may be NULL.
 */
attn_status_t attn_stream_status(attn_stream_t stream, unsigned int* code);

/*
 * attn_selftest_wait_timeout — exercises the kernel's bounded-wait abort
 * path on demand.  Launches the attn_fwd kernel for these arguments (same
 * meaning and checks as attn_fwd) with two changes: every pipeline wait
 * gives up after timeout_ns (> 0) instead of the library default, and the
 * first CTA never loads its first K tile, so its MMA issuer waits for a
 * tile that cannot arrive.  That wait runs out, the CTA's roles stop,
 * drain what they have in flight (bounded), free TMEM and exit; the other
 * CTAs finish normally.  Nothing faults or hangs and the context stays
 * usable: the timeout is reported by the next attn_device_status() or
 * attn_stream_status() (ATTN_ERR_TIMEOUT, bit 0 set, role bits non-zero),
 * and the rows of the first CTA's work units in O and LSE are left
 * undefined.  For tests of the failure path only.
 */
attn_status_t attn_selftest_wait_timeout(const void* Q, const void* K,
                                         const void* V, void* O, float* LSE,
                                         int B, int Hq, int Hkv, int Sq,
                                         int Skv, int D, float scale,
                                         int causal, int input_pos,
                                         attn_dtype_t dtype,
                                         unsigned long long timeout_ns,
                                         attn_stream_t stream);

/*
 * attn_selftest_prefix_timeout — the same of attn_prefix_fwd: its arguments and
 * checks, every wait gives up after timeout_ns (> 0), and thread block `block`
 * (>= 0) waits in vain for its first key tile, or with query_rows non-zero for
 * its first query rows.  That block's copies and products end before it does.
 * The rows it works on are left undefined, those of the other blocks are right.
 * A block that has no key tiles gives up nothing.  For tests of the failure path
 * only.
 */
attn_status_t attn_selftest_prefix_timeout(
    const attn_prefix_cache_t* cache, const void* Q, void* O, float* LSE,
    int Hq, int Sq, const int* new_lens, float scale, int causal,
    attn_dtype_t dtype, void* workspace, size_t workspace_bytes, int block,
    int query_rows, unsigned long long timeout_ns, attn_stream_t stream);

/*
 * attn_tile_config — the tile configuration attn_fwd would launch for these
 * arguments (host only, no GPU needed).  Fills, when non-NULL:
 *   block_m   query rows per CTA, block_n keys per K/V tile,
 *   stages    K/V tiles the shared-memory ring holds,
 *   grid      work units (each 2 x 128 query rows); the launch runs
 *             min(grid, SM count) persistent CTAs that walk them,
 *   smem_bytes dynamic shared memory per CTA.
 * Returns the same validation code attn_fwd would (pointers not checked).
 */
attn_status_t attn_tile_config(int B, int Hq, int Hkv, int Sq, int Skv, int D,
                               int causal, int input_pos, attn_dtype_t dtype,
                               int* block_m, int* block_n, int* stages,
                               int* grid, int* smem_bytes);

/*
 * attn_dispatch_t / attn_dispatch — the forward dispatch-table entry a call
 * with these arguments runs, spelled out (host only, no GPU needed).  The
 * entry is keyed on D, dtype, causal / window, the GQA group size and Sq
 * (the tile shape and work unit) and on num_splits (one pass or split-KV):
 *   q_tiles 2, paired 1   two query heads of one K/V group at the same 128
 *                         rows per unit (even group size);
 *   q_tiles 2, paired 0   256 consecutive rows of one head per unit;
 *   q_tiles 1             the group * Sq <= 128 query rows of all heads of
 *                         a K/V group packed into one tile (few query rows);
 *   s_buffers             score tiles in TMEM: 2, or 3 rotating between the
 *                         two Q tiles at D = 64 (O needs only 128 columns);
 *   order 0               heaviest causal row block first, the heads of a
 *                         row block in turn (longest-processing-time order
 *                         over the persistent CTAs); order 1: the row blocks
 *                         of one head in turn (non-causal: equal units, K/V
 *                         of the few heads in flight stays in L2); order 2:
 *                         causal units assigned to the CTAs by a plan packed
 *                         on the host (one-pass launches of more units than
 *                         SMs and at most 1024, when the plan beats the
 *                         order-0 rounds; see attn_unit_plan), so the entry
 *                         depends on Sq through the unit count;
 *   o_store 1             O leaves through a 128-byte-swizzled shared-memory
 *                         box stored by TMA; 0: each softmax thread stores
 *                         its row (packed tiles, split-KV fp32 partials);
 *   hold_scores 1         the softmax keeps a row's 128 scores in registers
 *                         between its max and exp passes (register split).
 * units is the number of work units (the launch runs min(units, SM count)
 * persistent CTAs), stages the K/V tiles in flight, smem_bytes the dynamic
 * shared memory per CTA.  name is a static string naming the entry.
 * num_splits: 0 for the one-pass forward, else as attn_fwd_splitkv
 * (planned count; units then count (rows, key range) pairs).  merge: how
 * the key ranges are merged -- 0 no split; 1 inside the forward kernel,
 * the ranges of a K/V group forming one thread-block cluster (packed tiles,
 * units <= SM count, at most 8 ranges; one kernel per call); 2 by a merge
 * kernel enqueued after the forward kernel (two kernels per call).  The
 * SM count is the current device's (152 without one).  Returns the
 * validation code the call would; out must be non-NULL.
 */
typedef struct {
  int block_m, block_n, q_tiles, paired, s_buffers, stages;
  int order, o_store, hold_scores, num_splits, units, smem_bytes, merge;
  const char* name;
} attn_dispatch_t;

attn_status_t attn_dispatch(int B, int Hq, int Hkv, int Sq, int Skv, int D,
                            int causal, int input_pos, int window,
                            attn_dtype_t dtype, int num_splits,
                            attn_dispatch_t* out);

/*
 * attn_unit_plan — how a one-pass forward call of this shape assigns its
 * work units to `grid` persistent CTAs (host only, no GPU needed; the call
 * itself uses grid = min(units, SM count)).  Has no counterpart in the
 * method's description: it exposes the launch's load balancing.
 * Causal two-tile launches (not the packed few-row mode) of more units
 * than CTAs and at most 1024 units are packed on the host: units heaviest
 * first into the first CTA with room under a capacity searched from the
 * mean upwards (first-fit decreasing, the MULTIFIT method), kept only when
 * its busiest CTA beats the zigzag rounds the kernel otherwise walks.
 *   planned      out: 1 when such a plan assigns the units, else 0 (the
 *                rounds: non-causal or packed launches, units <= grid,
 *                more than 1024 units, or no better plan);
 *   work_max     out: the busiest CTA's work under the assignment the
 *                call uses, in half K/V steps (each unit counts 2 per K/V
 *                step its later Q tile visits, plus 3 for its boundary);
 *                0 when not computed (a launch the plan never considers);
 *   work_rounds  out: the same under the zigzag rounds (0 likewise);
 *   unit_order   optional (NULL: not written), room for the unit count:
 *                CTA c walks units unit_order[cta_start[c] ..
 *                cta_start[c + 1]) in order (written only when planned);
 *   cta_start    optional, room for min(units, grid) + 1 entries.
 * Returns the validation code of attn_fwd for the shape (bf16), or
 * ATTN_ERR_INVALID_ARG for grid < 1 or a NULL output.
 */
attn_status_t attn_unit_plan(int B, int Hq, int Hkv, int Sq, int Skv, int D,
                             int causal, int input_pos, int window, int grid,
                             int* planned, long long* work_max,
                             long long* work_rounds, int* unit_order,
                             int* cta_start);

/* Library version as major*10000 + minor*100 + patch. */
int attn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_FWD_GB300_ATTN_H */
