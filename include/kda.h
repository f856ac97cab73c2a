/*
 * kda.h -- C ABI of libkda: Kimi Delta Attention (KDA) prefill and decode on
 * AMD MI355X (gfx950).
 *
 * The operation (Kimi Linear paper notes, section 2 "KDA recurrence"): per
 * (sequence, head) a fixed dk x dv fp32 state S is updated token by token as
 *
 *     S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T
 *     o_t = S_t^T q_t
 *
 * where alpha_t = exp(log_alpha_t) is a per-key-channel decay vector and
 * beta_t the write strength.  kda_prefill evaluates whole sequences with the
 * chunkwise-parallel form (paper notes, section 3: dense WY/UT form of each
 * chunk's rank-1 transitions, inter-chunk plus intra-chunk output, only the
 * fixed-size state passed between chunks); kda_decode_step applies the
 * recurrence to one token (the fused recurrent decode path).  Both compute
 * the same function.
 *
 * Conventions shared by every call
 *   Layout     dense row-major.  Tokens of all sequences are packed along the
 *              first axis; head h of token t of a [T,H,d] tensor is row
 *              (t*H + h).  The state is [N,H,dk,dv], key channel major (row c
 *              of a head's state is key channel c).
 *   Dtypes     q, k, v and o share one dtype (KDA_DTYPE_F32 or KDA_DTYPE_BF16);
 *              log_alpha, beta and states are always fp32; accumulation is fp32.
 *   Sizes      dk, dv in {64, 128} (any pairing); H >= 1; num_seqs >= 1.
 *   Alignment  every pointer 16-byte aligned.
 *   Ownership  the caller owns every buffer (device memory).  The library
 *              keeps no pointer after a call returns.
 *   Streams    work is enqueued on `stream` (a hipStream_t; NULL = the null
 *              stream).  KDA_OK means "enqueued"; faults during execution
 *              surface at the caller's next synchronisation.
 *   Errors     a call returns a status and never aborts, prints or throws.
 *              Host-checkable argument errors are reported before any HIP
 *              call is made; kda_last_error_message() gives detail (per
 *              thread).  The contents of device-resident cu_seqlens are a
 *              precondition and are not read on the host, except with the
 *              environment variable KDA_DEBUG_SYNC=1: then every call copies
 *              them, returns KDA_ERR_INVALID_ARGUMENT unless
 *              0 = c_0 <= c_1 <= ... <= c_N = T, and synchronises the stream
 *              after each kernel so that execution faults surface as
 *              KDA_ERR_HIP from the call that caused them.
 *   Threads    calls are reentrant and may come from several threads.  The
 *              library keeps no mutable state shared between threads: the
 *              error text and the optional kernel timing are per thread.
 *   Values     log_alpha must be finite and <= 0 (alpha in (0, 1]).  Within
 *              every aligned 16-token block of a 64-token chunk the summed
 *              log_alpha of one channel must stay above -80; inside that range
 *              results match the recurrence up to rounding, outside it they
 *              are unspecified.  NaN/Inf inputs propagate.
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARGUMENT = 1, /* NULL/misaligned pointer, bad size or dtype */
    KDA_ERR_UNSUPPORTED = 2,      /* a head size the library has no kernels for */
    KDA_ERR_WORKSPACE = 3,        /* caller workspace smaller than required     */
    KDA_ERR_HIP = 4               /* a HIP runtime call or launch failed        */
} kda_status;

typedef enum { KDA_DTYPE_F32 = 0, KDA_DTYPE_BF16 = 1 } kda_dtype;

/*
 * Input preprocessing the layer may leave to the kernels (Kimi Linear paper
 * notes, section 3 on the FLA implementation: the layer L2-normalises q and
 * k and passes beta through a sigmoid, optionally inside the kernel).  Flags
 * for kda_prefill_ex and kda_decode_tokens; any other bit is rejected.
 *   KDA_FLAG_L2NORM_QK    q_t <- q_t / sqrt(q_t . q_t + 1e-6) per (token,
 *                         head) over the dk channels, the same for k_t
 *   KDA_FLAG_BETA_SIGMOID beta holds logits x; beta_t = 1 / (1 + exp(-x))
 */
enum { KDA_FLAG_L2NORM_QK = 1u, KDA_FLAG_BETA_SIGMOID = 2u };

/*
 * Device workspace kda_prefill needs for these sizes (bytes, 256-aligned).
 * It holds one record per (chunk, head) built from the chunk intermediates of
 * the chunkwise form (paper notes, section 3 and its list of chunk
 * intermediates: g, A_qk, A_kk, w, u, decayed q and k): the chunk's state
 * transition and read-out with W and U folded in, in the dtype of q/k/v, plus
 * the chunk-end decay in fp32; and the chunk table of the batch.  Returns 0
 * for invalid sizes.
 */
size_t kda_prefill_workspace_bytes(int64_t total_tokens, int32_t num_seqs, int32_t H,
                                   int32_t dk, int32_t dv, kda_dtype dtype);

/*
 * Chunkwise prefill of a packed batch (paper notes, sections 2-3).
 *
 *   q, k          [T,H,dk] dtype; v [T,H,dv] dtype      (device, read)
 *   log_alpha     [T,H,dk] fp32, log of the per-channel decay (device, read)
 *   beta          [T,H] fp32 write strength              (device, read)
 *   initial_state [N,H,dk,dv] fp32, or NULL = zero state (device, read)
 *   cu_seqlens    [N+1] int32 offsets 0 = c_0 <= c_1 <= ... <= c_N = T
 *                 (device; zero-length sequences allowed), or NULL = N equal
 *                 contiguous sequences of T/N tokens (T % N must be 0).  The
 *                 offsets are a precondition and are not read on the host.
 *   total_tokens  T >= 0; num_seqs N >= 1
 *   o             [T,H,dv] dtype (device, written; must not alias an input)
 *   final_state   [N,H,dk,dv] fp32 (device, written), or NULL.  May be the
 *                 same buffer as initial_state (state carried in place).
 *   workspace     device buffer of at least kda_prefill_workspace_bytes(), or
 *                 NULL with workspace_bytes 0: the library then allocates and
 *                 frees one stream-ordered on `stream`.
 * A sequence of length 0 writes final_state = initial_state (or zeros).
 */
kda_status kda_prefill(const void *q, const void *k, const void *v,
                       const float *log_alpha, const float *beta,
                       const float *initial_state, const int32_t *cu_seqlens,
                       int64_t total_tokens, int32_t num_seqs, int32_t H,
                       int32_t dk, int32_t dv, kda_dtype dtype,
                       void *o, float *final_state,
                       void *workspace, size_t workspace_bytes, void *stream);

/*
 * kda_prefill without a workspace argument, for callers that cannot allocate
 * device memory: code under HIP graph capture, tight serving loops and
 * harnesses that forbid hipMalloc.  The call allocates nothing (no hipMalloc,
 * no stream-ordered allocation, no allocating library routine).  Its
 * workspace is a fixed array of KDA_NOALLOC_SCRATCH_BYTES in the library's
 * device code: every GPU the library is loaded on holds one copy of it from
 * module load until the process ends.
 *   Limit    sizes for which kda_prefill_workspace_bytes() exceeds
 *            KDA_NOALLOC_SCRATCH_BYTES return KDA_ERR_WORKSPACE before any
 *            HIP call (at H = 32, dk = dv = 128, bf16 that is beyond 1,280
 *            tokens of one sequence; smaller H or head sizes allow more).
 *   Sharing  every call on one GPU uses that GPU's one array and leaves its
 *            contents behind; nothing in it needs to start at zero.  Calls
 *            that overlap on one GPU (concurrent streams, or threads without
 *            an order between them) race on the array: the caller must order
 *            them, e.g. by issuing them on one stream.
 * Arguments, results and errors otherwise as for kda_prefill.
 */
#define KDA_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
kda_status kda_prefill_noalloc(const void *q, const void *k, const void *v,
                               const float *log_alpha, const float *beta,
                               const float *initial_state, const int32_t *cu_seqlens,
                               int64_t total_tokens, int32_t num_seqs, int32_t H,
                               int32_t dk, int32_t dv, kda_dtype dtype,
                               void *o, float *final_state, void *stream);

/*
 * kda_prefill with options.  The extra arguments:
 *   flags         KDA_FLAG_* bits (0 = kda_prefill)
 *   chunk_states  fp32 [NC,H,dk,dv] (device, written), or NULL: the state
 *                 entering every 64-token chunk of every sequence, i.e. after
 *                 64c of its tokens for c = 0 .. ceil(len/64) - 1 (c = 0 is
 *                 the initial state).  Rows run over the sequences in order,
 *                 ceil(len_s/64) rows for sequence s (none for an empty one):
 *                 NC = sum_s ceil(len_s/64) <= ceil(T/64) + N.  With
 *                 final_state, a caller can roll back to any 64-token boundary
 *                 of a sequence and prefill again from there (paper notes,
 *                 section 3: the chunk states h of the chunkwise form).
 */
kda_status kda_prefill_ex(const void *q, const void *k, const void *v,
                          const float *log_alpha, const float *beta,
                          const float *initial_state, const int32_t *cu_seqlens,
                          int64_t total_tokens, int32_t num_seqs, int32_t H,
                          int32_t dk, int32_t dv, kda_dtype dtype, uint32_t flags,
                          void *o, float *final_state, float *chunk_states,
                          void *workspace, size_t workspace_bytes, void *stream);

/*
 * One recurrent token for each of N sequences (fused recurrent decode,
 * paper notes, section 3; the state is the only memory a KDA layer keeps per
 * sequence).  The state is updated in place:
 *
 *   state      [N,H,dk,dv] fp32 (device, read and written)
 *   q, k       [N,H,dk] dtype; v [N,H,dv] dtype (device, read)
 *   log_alpha  [N,H,dk] fp32; beta [N,H] fp32   (device, read)
 *   o          [N,H,dv] dtype (device, written; must not alias an input)
 */
kda_status kda_decode_step(float *state, const void *q, const void *k, const void *v,
                           const float *log_alpha, const float *beta,
                           int32_t num_seqs, int32_t H, int32_t dk, int32_t dv,
                           kda_dtype dtype, void *o, void *stream);

/*
 * The recurrent form over a few tokens per sequence, on pooled states
 * (paper notes, section 3: FLA's fused recurrent mode, used for short inputs
 * and decoding; one fixed-size state per sequence).  Each sequence s runs
 * its tokens in order starting from state_pool[slot_s] and leaves its final
 * state there; the state never leaves the registers in between.
 *
 *   state_pool     [num_slots,H,dk,dv] fp32 (device, read and written)
 *   num_slots      >= 1
 *   state_indices  [N] int32 slot per sequence (device), or NULL = slot s for
 *                  sequence s (then num_slots >= N).  A slot outside
 *                  [0, num_slots) marks a padding sequence: its o rows are
 *                  zeroed and no state is read or written.  Sequences must
 *                  name distinct slots (with a repeated slot the results
 *                  are undefined).
 *   q, k, v, log_alpha, beta, cu_seqlens, total_tokens, num_seqs, flags:
 *                  as for kda_prefill_ex (tokens packed, cu_seqlens NULL = N
 *                  equal rows)
 *   o              [T,H,dv] dtype (device, written)
 * Meant for short runs (speculative verification, chunked decoding).  For
 * bf16 with dk = dv = 128 and more tokens than sequences the tokens of a
 * sequence are taken 16 at a time in the chunkwise form (section 3; bf16
 * products, fp32 state, the precision of kda_prefill); otherwise they are
 * processed one by one.  One token per sequence given as equal rows
 * (cu_seqlens NULL, total_tokens = num_seqs) with no flags runs
 * kda_decode_step's kernel through the slots: with identity slots its
 * results are kda_decode_step's, bit for bit.
 */
kda_status kda_decode_tokens(float *state_pool, int32_t num_slots, const int32_t *state_indices,
                             const void *q, const void *k, const void *v,
                             const float *log_alpha, const float *beta,
                             const int32_t *cu_seqlens, int64_t total_tokens, int32_t num_seqs,
                             int32_t H, int32_t dk, int32_t dv, kda_dtype dtype,
                             uint32_t flags, void *o, void *stream);

/*
 * Device workspace kda_backward needs for these sizes (bytes, 256-aligned;
 * 0 for invalid sizes).  It covers a forward recomputation of the chunk
 * states (used when the caller passes none) and either the per-chunk records
 * and bf16 gradients leaving every chunk of the chunkwise path or the
 * per-slice partial gradients and per-workgroup scratch of the token walk.
 */
size_t kda_backward_workspace_bytes(int64_t total_tokens, int32_t num_seqs, int32_t H,
                                    int32_t dk, int32_t dv, kda_dtype dtype);

/*
 * Gradients of kda_prefill (the recurrence of paper notes section 2; the
 * FLA implementation the pages describe trains through the chunkwise form
 * with a backward pass, section 3).  For a loss L with dL/do = d_o and
 * dL/dfinal_state = d_final_state it writes dL/dq, dL/dk, dL/dv, dL/dlog_alpha,
 * dL/dbeta and dL/dinitial_state.
 *
 *   q, k, v, log_alpha, beta, initial_state, cu_seqlens, total_tokens,
 *   num_seqs, H, dk, dv, dtype   as for kda_prefill (the forward's inputs;
 *                 no preprocessing flags: the gradients are with respect to
 *                 the q, k and beta the recurrence sees)
 *   d_o           [T,H,dv] dtype (device, read)
 *   d_final_state [N,H,dk,dv] fp32, or NULL = zero
 *   chunk_states  the forward's chunk states as kda_prefill_ex writes them
 *                 ([NC,H,dk,dv] fp32), or NULL: recomputed here
 *   dq, dk_out    [T,H,dk] dtype; dv_out [T,H,dv] dtype (device, written)
 *   dlog_alpha    [T,H,dk] fp32; dbeta [T,H] fp32 (device, written)
 *   d_initial_state [N,H,dk,dv] fp32 (device, written), or NULL
 *   workspace     at least kda_backward_workspace_bytes(), or NULL with 0
 *                 (then allocated stream-ordered on `stream`)
 * Outputs must not alias inputs.  The result is deterministic.  bf16 with
 * dk = dv = 128 runs the chunkwise backward: a reverse pass over the chunks
 * (the transpose of each chunk's transition, from the last chunk to the
 * first) gives the gradient leaving every chunk, then every chunk's input
 * gradients are formed in parallel from its entry state and that gradient.
 * Other configurations walk the tokens backwards (recomputed forward from the
 * chunk states, 8 tokens at a time).  KDA_BACKWARD_SERIAL=1 in the
 * environment selects the token walk for bf16 too.
 */
kda_status kda_backward(const void *q, const void *k, const void *v,
                        const float *log_alpha, const float *beta,
                        const float *initial_state, const int32_t *cu_seqlens,
                        int64_t total_tokens, int32_t num_seqs, int32_t H,
                        int32_t dk, int32_t dv, kda_dtype dtype,
                        const void *d_o, const float *d_final_state, const float *chunk_states,
                        void *dq, void *dk_out, void *dv_out, float *dlog_alpha, float *dbeta,
                        float *d_initial_state, void *workspace, size_t workspace_bytes,
                        void *stream);

/*
 * ---------------------------------------------------------------------------
 * Latent attention: the full-attention layer that a hybrid model puts between
 * its KDA layers.  A token leaves one latent vector c (dl channels, RMS
 * normalised) and one rotary key part (dr channels) shared by all heads.  Its
 * per-head keys [c Wk_h, k_pe] and values c Wv_h are expanded from the latent
 * by a matrix product of the caller's (kda_latent_attention and its
 * gradients), or Wk_h and Wv_h are multiplied into the query and the output,
 * so that every head reads the one latent row (kda_latent_decode, over the
 * paged cache that kda_latent_append writes).  The conventions at the top of
 * this file hold, with these differences:
 *   Strides    where a tensor takes strides they count elements; the last axis
 *              is dense, and strides and pointers are multiples of 16 bytes.
 *   Offsets    cu_seqlens may end before the last row (c_N <= T): the rows
 *              behind the last sequence are neither read nor written.  Offsets
 *              outside [0, T] are clamped to it.  They must not decrease
 *              (all that KDA_DEBUG_SYNC=1 checks of them).
 *   Empty rows a query row that sees no key gets o = 0, lse = -inf and zero
 *              gradients.
 *   Values     NaN and Inf propagate from the keys a row sees to its result, and
 *              from a row to the gradients of the keys it sees, and no further:
 *              keys that the mask hides, rows behind a sequence's end and unused
 *              cache rows may hold anything.  In kda_latent_attention a value of
 *              v that is not finite reaches its own channel of o only, and never
 *              lse.  Elsewhere how far it spreads is not specified: a latent of
 *              the cache may turn all of o and lse of the rows that see it into
 *              NaN where the formula gives some of it as Inf or finite, and an
 *              input of the backward pass any gradient that it takes part in.
 * ---------------------------------------------------------------------------
 */

/*
 * Inputs of the expanded form (all device memory):
 *   q      [total_q, H, dn + dr]: the dn channels that meet k, then the dr
 *          channels that meet k_pe (already rotated, see kda_rotary)
 *   k, v   [total_k, H, dn], [total_k, H, dv]: strided, so that both may be
 *          halves of one [total_k, H, dn + dv] product
 *   k_pe   [total_k, dr], shared by the heads; NULL with dr = 0
 *   cu_seqlens_q, cu_seqlens_k   [num_seqs + 1] int32 offsets of each
 *          sequence's queries and keys; cu_seqlens_k NULL = the queries'
 *          offsets (then total_k = total_q); both NULL = num_seqs equal rows
 *   causal nonzero: query i of a sequence with n queries and m keys sees the
 *          keys j <= i + (m - n), i.e. the last query sees all of them; with
 *          m < n the first n - m queries see none
 *   scale  finite and > 0, multiplies q . k
 * dn = dv in {64, 128}; dr in {0, 64}; token strides and H * dv below 2^23;
 * (rows / 64 + num_seqs) * H below 2^24.
 */
typedef struct {
    const void *q;
    const void *k;
    const void *v;
    const void *k_pe;
    int64_t q_token_stride, q_head_stride;
    int64_t k_token_stride, k_head_stride;
    int64_t v_token_stride, v_head_stride;
    int64_t k_pe_token_stride;
    const int32_t *cu_seqlens_q;
    const int32_t *cu_seqlens_k;
    int64_t total_q, total_k;
    int32_t num_seqs, H, dn, dr, dv;
    int32_t dtype;               /* kda_dtype */
    int32_t causal;
    float scale;
} kda_latent_inputs;

/*
 * Expanded latent attention over packed sequences, one pass over the keys with
 * the running maximum and sum of the softmax:
 *
 *     z_ij = scale (q_i . [k_j, k_pe_j]),   o_i = sum_j softmax(z_i)_j v_j,
 *     lse_i = log sum_j exp(z_ij)           over the keys j that i sees
 *
 *   o    [total_q, H, dv] dtype (written; must not alias an input)
 *   lse  [total_q, H] fp32 (written), or NULL; the backward pass needs it
 */
kda_status kda_latent_attention(const kda_latent_inputs *in, void *o, float *lse, void *stream);

/*
 * Device workspace that suffices for kda_latent_attention_backward with either
 * dtype (bytes, 256-aligned; 0 for invalid sizes).  It never falls as an argument
 * grows: a workspace for the largest batch serves every smaller one.
 */
size_t kda_latent_attention_backward_workspace_bytes(int64_t total_q, int64_t total_k, int32_t H,
                                                     int32_t dr);

/*
 * Gradients of kda_latent_attention for dL/do = d_o, from the forward's o and
 * lse.  Deterministic; the gradient of the shared k_pe is summed over the heads
 * in order, in fp32.
 *   o, d_o   [total_q, H, dv] dtype; lse [total_q, H] fp32   (read)
 *   dq       [total_q, H, dn + dr] dtype, dense (written)
 *   dk, dv   strided like k and v, dtype (written): both may be halves of one
 *            [total_k, H, dn + dv] gradient
 *   dk_pe    [total_k, dr] dtype, dense (written; NULL with dr = 0)
 *   workspace at least kda_latent_attention_backward_workspace_bytes(), or
 *            NULL with 0 (then allocated stream-ordered on `stream`)
 * Keys of a sequence without queries get zero gradients.  Outputs must not
 * alias inputs.
 */
kda_status kda_latent_attention_backward(const kda_latent_inputs *in, const void *o,
                                         const float *lse, const void *d_o, void *dq, void *dk,
                                         int64_t dk_token_stride, int64_t dk_head_stride, void *dv,
                                         int64_t dv_token_stride, int64_t dv_head_stride,
                                         void *dk_pe, void *workspace, size_t workspace_bytes,
                                         void *stream);

/*
 * Device workspace kda_latent_decode needs (bytes, 256-aligned; 0 for invalid
 * sizes): the partial results of rows whose keys are split over workgroups.  It
 * depends on dl only, so that one workspace serves batches of any size.
 */
size_t kda_latent_decode_workspace_bytes(int64_t total_tokens, int32_t num_seqs, int32_t H,
                                         int32_t dl, int32_t dr, kda_dtype dtype);

/*
 * Absorbed latent attention of one or more new tokens per sequence over a
 * paged cache of latents (single-token decode, speculative tokens, a chunk of
 * a prompt over its cached prefix).  All heads read the same cached row:
 *
 *     z_ij = scale (q_i . [c_j, k_pe_j]),   o_i = sum_j softmax(z_i)_j c_j
 *
 *   q            [T, H, dl + dr] dtype, strided: the query multiplied by Wk_h
 *                (dl channels), then its rotated part (dr)
 *   cache        [num_pages, page_size, dl + dr] dtype, dense: rows [c, k_pe]
 *   block_table  [N, max_pages] int32: sequence s's token j is row
 *                j % page_size of page block_table[s][j / page_size].  A page
 *                outside [0, num_pages) is not read: its tokens count as
 *                absent.  num_pages * page_size < 2^31.
 *   seq_lens     [N] int32 cached tokens of every sequence, the new ones
 *                included (they are appended first); clamped to
 *                [0, max_pages * page_size]
 *   cu_seqlens   [N+1] int32 offsets of the new tokens, or NULL = T / N each
 *                (T % N must be 0).  New token i of n sees the tokens
 *                j <= seq_len - n + i.
 *   o            [T, H, dl] dtype (written); lse [T, H] fp32 (written), or NULL
 *   workspace    at least kda_latent_decode_workspace_bytes(), or NULL with 0
 *                (then allocated stream-ordered on `stream`).  Two calls that
 *                may overlap need one each.
 * dl in {256, 512}; dr in {0, 64}; H * T <= 2^31 - 4096.  The result is
 * deterministic: how the keys are split depends on the sizes and lengths only.
 */
kda_status kda_latent_decode(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                             const void *cache, int32_t num_pages, int32_t page_size,
                             const int32_t *block_table, int32_t max_pages,
                             const int32_t *seq_lens, const int32_t *cu_seqlens,
                             int64_t total_tokens, int32_t num_seqs, int32_t H, int32_t dl,
                             int32_t dr, kda_dtype dtype, float scale, void *o, float *lse,
                             void *workspace, size_t workspace_bytes, void *stream);

/*
 * Rotary layouts: which channels of the rotated part form pair i of dr / 2.
 * The default is the half layout (i, i + dr / 2).
 *   KDA_ROTARY_INTERLEAVED  channels 2i and 2i + 1
 *   KDA_ROTARY_INVERSE      rotate by minus the angle (the gradient of the
 *                           rotation; kda_rotary only)
 */
enum { KDA_ROTARY_INTERLEAVED = 1u, KDA_ROTARY_INVERSE = 2u };

/*
 * Writes the new tokens' rows of the paged cache:
 *
 *     row = [ c / sqrt(mean(c^2) + eps) * norm_weight,  amplitude R(p f) k_pe ]
 *
 * Token i of the n new ones of sequence s sits at position p = seq_len - n + i,
 * in the row that kda_latent_decode reads for it; a token whose position is
 * negative or whose page is outside [0, num_pages) is not written to the cache.
 *   cache, num_pages, page_size, block_table, max_pages, seq_lens, cu_seqlens,
 *   total_tokens, num_seqs, dl, dr, dtype: as for kda_latent_decode (dl a
 *                multiple of 64 up to 1024, dr an even number up to 256, a
 *                multiple of 16 bytes)
 *   c            [T, dl] dtype and k_pe [T, dr] dtype (read), rows
 *                c_token_stride and k_pe_token_stride apart: both may be parts
 *                of one [T, dl + dr] product.  k_pe NULL with dr = 0.
 *   norm_weight  [dl] fp32, or NULL: c is written as it is
 *   eps          >= 0, finite
 *   inv_freq     [dr/2] fp32 radians per position, or NULL: k_pe is written as
 *                it is (no positions)
 *   amplitude    finite; multiplies the rotated part (long-context scaling)
 *   flags        KDA_ROTARY_INTERLEAVED or 0
 *   c_out        [T, dl] dtype, dense, or NULL: the normalised latents, for
 *                their expansion (written for every token of a sequence,
 *                whether or not it has a cache row)
 *   k_pe_out     [T, dr] dtype, dense, or NULL: the rotated key parts, alike
 */
kda_status kda_latent_append(void *cache, int32_t num_pages, int32_t page_size,
                             const int32_t *block_table, int32_t max_pages,
                             const int32_t *seq_lens, const int32_t *cu_seqlens,
                             int64_t total_tokens, int32_t num_seqs, int32_t dl, int32_t dr,
                             kda_dtype dtype, const void *c, int64_t c_token_stride,
                             const void *k_pe, int64_t k_pe_token_stride,
                             const float *norm_weight, float eps, const float *inv_freq,
                             float amplitude, uint32_t flags, void *c_out, void *k_pe_out,
                             void *stream);

/*
 * Rotary positions on channels [start, start + dr) of every head:
 * y = amplitude R(p f) x per pair, the other channels copied.  The angle
 * p f is reduced in 64 bits, so far positions keep their accuracy.
 *   x          [T, H, d] dtype, strided in tokens and heads (read)
 *   y          [T, H, d] dtype, strided (written).  y = x with x's strides
 *              rotates in place and leaves the other channels untouched; any
 *              other overlap is not allowed.
 *   positions  [T] int32
 *   inv_freq   [dr/2] fp32 radians per position (see kda_rotary_frequencies)
 *   flags      KDA_ROTARY_* bits
 * dr even and >= 2, start >= 0, start + dr <= d <= 4096.  Pointers and strides
 * need the alignment of one element only (wider accesses are used where they
 * allow it).
 */
kda_status kda_rotary(const void *x, int64_t x_token_stride, int64_t x_head_stride, void *y,
                      int64_t y_token_stride, int64_t y_head_stride, const int32_t *positions,
                      const float *inv_freq, int64_t total_tokens, int32_t H, int32_t d,
                      int32_t start, int32_t dr, kda_dtype dtype, float amplitude, uint32_t flags,
                      void *stream);

/*
 * Rotary frequencies, computed on the host into host memory inv_freq[dr/2]:
 * f_i = base^(-2i/dr).  With factor > 1 the context is stretched by `factor`:
 *   original_context = 0  every f_i / factor (linear interpolation)
 *   original_context > 0  by parts: a pair that makes at least 32 full turns
 *                         over the original context keeps f_i, one that makes
 *                         at most one gets f_i / factor, with a linear ramp in
 *                         the number of turns in between; the amplitude that
 *                         goes with it is 0.1 ln(factor) + 1
 * *amplitude (or NULL) receives the amplitude, 1 otherwise.
 */
kda_status kda_rotary_frequencies(int32_t dr, double base, double factor,
                                  int64_t original_context, float *inv_freq, float *amplitude);

/* Static description of a status code. */
const char *kda_status_string(kda_status status);

/* Detail of the last non-OK status returned on the calling thread ("" if none). */
const char *kda_last_error_message(void);

/* Library version, major*10000 + minor*100 + patch. */
int32_t kda_version(void);

/*
 * Kernel timing for measurement (not needed for normal use), per calling
 * thread.  While enabled on a thread, kda_prefill called from that thread
 * has each of its kernels record its own start and end in a pair of HIP
 * events (hipExtLaunchKernelGGL; timing-only events without a system-scope
 * fence, created on first use and kept until the process ends), so a
 * kernel's time excludes the gap to the work queued before it.
 * kda_prefill_kernel_times() waits for the events of the last call timed on
 * the calling thread and writes, for up to max_kernels kernels in launch
 * order, the elapsed milliseconds (ms) and a static kernel name (names, may
 * be NULL).  It returns the number of kernels of that call, or -1 when
 * nothing was recorded on this thread or a HIP call failed.
 */
kda_status kda_set_kernel_timing(int32_t enabled);
int32_t kda_prefill_kernel_times(float *ms, const char **names, int32_t max_kernels);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
