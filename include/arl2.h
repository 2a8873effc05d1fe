/*
 * arl2.h -- C ABI of libarl2.so: the per-frame hot path of the ARL2 hybrid
 * attention module on NVIDIA B200 (sm_100a).
 *
 * Sources.  "ARL2 summary" is the technical summary on the page "Attend
 * Locally, Remember Linearly: Linear Attention as Cross-Frame Memory for
 * Autoregressive Video Diffusion" (gist.science; German, Italian, Japanese and
 * Korean editions carry the same text).  "ARL2 abstract" is the authors'
 * English abstract of arXiv 2605.16579v2 (fugumt.com paper_check page).
 *
 * What one hybrid layer computes, per stream b and head h, for frame N:
 *   intra-frame branch   O_intra = softmax(Q K^T * scale) V over the frame's
 *                        L tokens, bidirectional, no mask
 *                        (ARL2 summary, section 2.1, intra-frame branch);
 *   feature maps         Q' = Q phi_q, K' = rownorm2(K phi_k), V' = V phi_v
 *                        (section 2.1, adaptation by per-head grouped 1x1 maps);
 *   inter-frame read-out O_inter = Q' S_{N-1}   (section 2.1, output);
 *   output               O = O_intra + O_inter;
 *   state write          S_N = alpha S_{N-1} + c K'^T diag(beta)(V' - K' S_{N-1})
 *                        (section 2.1, state update), once per frame on the clean
 *                        pass only, every token reading the same S_{N-1}
 *                        (section 2.2, frame-level access and clean-pass updates;
 *                        ARL2 abstract).
 *
 * Conventions shared by every call:
 *   - Tensor pointers are DEVICE pointers owned by the caller, 16-byte
 *     aligned, contiguous, in the handle's dtype (float32 or bf16).
 *       Q, K, V, O : [B, L, H, d] token-major (row = token, then head, then
 *                    channel); O must not overlap Q, K or V.
 *       phi_*      : [H, d, d] row-major, Q' = Q phi (q'_j = sum_i q_i phi[i][j]).
 *       alpha      : float32 [B, H]      (one decay gate per stream and head).
 *       beta       : float32 [B, H, L]   (one write strength per token).
 *       state      : float32 [B, H, d, d], S[b][h][i][j] with i over K' and
 *                    j over V' channels.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *     Calls are asynchronous on that stream; their return value covers argument
 *     and launch errors only.  Errors raised inside kernels (a bounded wait that
 *     ran out) are recorded in the handle and returned by arl2_last_error().
 *   - A handle must not be used from two streams at once; calls on one handle
 *     execute in stream order.  The attention and projection-GEMM kernels are
 *     launched with programmatic stream serialisation: their CTAs may start
 *     (barrier and tensor-memory set-up only) while the kernel ahead of them
 *     on the stream finishes, and wait for its completion before any global
 *     memory access, so the stream's ordering of memory effects is unchanged.
 *   - No C++ exception crosses this interface.
 *   - Supported shapes: bf16 needs head_dim = 128; float32 needs head_dim <= 128
 *     and tokens_per_frame <= 4096.  Anything else returns ARL2_ERR_UNSUPPORTED.
 */
#ifndef ARL2_H
#define ARL2_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ARL2_OK = 0,
  ARL2_ERR_INVALID_ARGUMENT = 1, /* null or misaligned pointer, bad handle, bad size */
  ARL2_ERR_UNSUPPORTED = 2,      /* a shape or dtype outside the supported set */
  ARL2_ERR_OUT_OF_MEMORY = 3,    /* a device allocation of the library failed */
  ARL2_ERR_CUDA = 4,             /* a CUDA runtime call or kernel launch failed */
  ARL2_ERR_TIMEOUT = 5,          /* a bounded device-side wait ran out */
  ARL2_ERR_NO_DEVICE = 6,        /* no usable CUDA device / driver */
  ARL2_ERR_SCRATCH_LIMIT = 7,    /* sizes need more than the fixed scratch of
                                    arl2_state_write_noalloc */
  ARL2_ERR_BOUNDS = 8,           /* debug builds (libarl2_debug.so) only: a
                                    kernel's index check failed and the access
                                    was skipped; surfaced by arl2_last_error */
  ARL2_ERR_PAGE = 9              /* paged cache: a page number, length or offset
                                    that a kernel read from device memory is out
                                    of range; surfaced by arl2_paged_last_error */
} arl2_status;

typedef enum { ARL2_F32 = 0, ARL2_BF16 = 1 } arl2_dtype;

/* Test-only flags of arl2_config.flags: return only one branch of O. */
#define ARL2_INTRA_ONLY 1u
#define ARL2_INTER_ONLY 2u

typedef struct {
  int32_t batch;            /* B independent streams, >= 1 */
  int32_t heads;            /* H, >= 1 */
  int32_t head_dim;         /* d */
  int32_t tokens_per_frame; /* L, >= 1 */
  int32_t dtype;            /* arl2_dtype of Q, K, V, O and phi */
  float softmax_scale;      /* 0 => 1/sqrt(head_dim) */
  float corr_scale;         /* c of the state write; < 0 => 1/L (mean over the frame's tokens) */
  uint32_t flags;           /* 0, or ARL2_INTRA_ONLY / ARL2_INTER_ONLY (tests only) */
} arl2_config;

typedef struct arl2_state* arl2_state_t;
typedef struct arl2_kv* arl2_kv_t;

/* Create a hybrid-layer handle with S_0 = 0 and frame counter 0.
 * phi_q, phi_k, phi_v: device [H, d, d] in cfg->dtype; the library copies them
 * (the caller may free them after the call returns).  The handle owns its
 * state double buffer and work space on the current device.
 * Errors: INVALID_ARGUMENT (null pointers, bad sizes), UNSUPPORTED (shape),
 * OUT_OF_MEMORY (no partial handle is left behind), CUDA. */
arl2_status arl2_state_init(const arl2_config* cfg, const void* phi_q, const void* phi_k,
                            const void* phi_v, void* stream, arl2_state_t* out);

/* One denoising step of a frame (ARL2 summary, section 2.2, clean-pass updates:
 * denoising steps query the state and never write it):
 *   O = softmax(Q K^T * scale) V + (Q phi_q) S_{N-1}.
 * Reads the state, writes only O. */
arl2_status arl2_frame_query(arl2_state_t h, const void* q, const void* k, const void* v, void* o,
                             void* stream);

/* The clean pass of frame N: O as in arl2_frame_query from S_{N-1}, then the
 * frame's single state write
 *   S_N = alpha S_{N-1} + c K'^T diag(beta) (V' - K' S_{N-1}),
 * then the frame counter increments (ARL2 summary, sections 2.1 and 2.2). */
arl2_status arl2_frame_commit(arl2_state_t h, const void* q, const void* k, const void* v,
                              const float* alpha, const float* beta, void* o, void* stream);

/* Query and commit with Q, K and V as strided views of wider token rows, as
 * a fused QKV projection writes them ([B, L, 3 * H * d] with K and V at column
 * offsets H*d and 2*H*d): token rows are `ld` elements apart instead of H*d.
 * bf16 handles only; ld >= H * d and a multiple of 8 (16-byte pitch); ld = 0
 * means contiguous, the same as arl2_frame_query / arl2_frame_commit, which
 * these calls equal bit for bit on the same values.  O stays contiguous and
 * must not overlap the views' spans.  Errors: INVALID_ARGUMENT (also for an
 * f32 handle with ld != 0), CUDA. */
arl2_status arl2_frame_query_strided(arl2_state_t h, const void* q, const void* k, const void* v, int64_t ld,
                                     void* o, void* stream);
arl2_status arl2_frame_commit_strided(arl2_state_t h, const void* q, const void* k, const void* v, int64_t ld,
                                      const float* alpha, const float* beta, void* o, void* stream);

/* Token-level access: the access rule that the ablation of the ARL2 summary
 * (section 4) reports as worse than frame-level access (section 2.2).  Within
 * the pass, token t reads the state left by the tokens before it, and the
 * update of section 2.1 runs one token at a time with a per-token decay:
 *   o_t   = O_intra,t + q'_t S^(t-1),   S^(0) = the handle's current state,
 *   S^(t) = a_t S^(t-1) + c beta_t k'_t^T (v'_t - k'_t S^(t-1)),
 * c being the handle's corr_scale.  The frame-level gate alpha corresponds to
 * a = (alpha, 1, ..., 1).
 * alpha_tok, beta: device float32 [B, H, L], 16-byte aligned.
 * arl2_token_query leaves the state as it is (denoising passes never write
 * it); arl2_token_commit makes S^(L) the current state, advances the frame
 * counter, and refreshes what the frame-level calls read, so the two kinds of
 * call may follow one another on one handle.
 * bf16 handles only.  The first token-level call on a handle allocates its
 * scratch (about 5.2 KB per token and head) with cudaMalloc and adds it to
 * arl2_state_device_bytes, so that first call must not be made while a
 * stream is being captured into a CUDA graph (it fails there with
 * OUT_OF_MEMORY or CUDA); later calls allocate nothing.  The arithmetic past the intra-frame
 * branch is float32.  Errors: INVALID_ARGUMENT, UNSUPPORTED (an f32 handle),
 * OUT_OF_MEMORY, CUDA. */
arl2_status arl2_token_query(arl2_state_t h, const void* q, const void* k, const void* v, const float* alpha_tok,
                             const float* beta, void* o, void* stream);
arl2_status arl2_token_commit(arl2_state_t h, const void* q, const void* k, const void* v, const float* alpha_tok,
                              const float* beta, void* o, void* stream);

/* Copy the current state (float32 [B, H, d, d]) to device memory `dst` and the
 * frame counter to *frame (host pointer, may be null).  Synchronous with
 * respect to `stream` for *frame only; the copy is enqueued on `stream`. */
arl2_status arl2_state_get(arl2_state_t h, float* dst, int64_t* frame, void* stream);

/* Replace the current state with device memory `src` (float32 [B, H, d, d]) and
 * set the frame counter: checkpoint / resume of a stream. */
arl2_status arl2_state_set(arl2_state_t h, const float* src, int64_t frame, void* stream);

/* Wait for the handle's device, whatever streams its calls and the replays of
 * captured ones ran on, and return (and clear) the first error recorded by its
 * kernels, ARL2_OK if none. */
arl2_status arl2_last_error(arl2_state_t h);

/* Device bytes held by the handle.  Fixed at init and independent of the
 * frame index, with one exception: the first token-level call
 * (arl2_token_query / arl2_token_commit) allocates that call's scratch and
 * adds it to the count, which then stays constant again. */
int64_t arl2_state_device_bytes(arl2_state_t h);

/* Wall-clock limit of one device-side wait in the handle's kernels (default
 * 1 second).  0 restores the default. */
arl2_status arl2_state_set_wait_limit(arl2_state_t h, uint64_t limit_ns);

arl2_status arl2_state_destroy(arl2_state_t h);

/* ---- Softmax layers kept from the teacher, with a growing KV cache --------
 * (ARL2 summary, section 1: the KV cache grows with every generated block.)
 * The queries of frame n attend, with no mask, to the clean keys and values
 * of frames 0..n-1 followed by the current pass's own K and V.  A query pass
 * leaves the cache's committed frames unchanged; a commit appends its K and V
 * as frame n.  The cache is [B, max_frames * L, H, d] in cfg->dtype. */
arl2_status arl2_kv_init(const arl2_config* cfg, int32_t max_frames, void* stream, arl2_kv_t* out);
arl2_status arl2_kv_query(arl2_kv_t kv, const void* q, const void* k, const void* v, void* o,
                          void* stream);
arl2_status arl2_kv_commit(arl2_kv_t kv, const void* q, const void* k, const void* v, void* o,
                           void* stream);
/* As arl2_kv_query / arl2_kv_commit with Q, K and V read as strided views
 * (token rows `ld` elements apart; bf16 only; ld >= H * d, a multiple of 8;
 * 0 = contiguous), bit-identical to the contiguous calls on the same values.
 * Errors as arl2_frame_query_strided. */
arl2_status arl2_kv_query_strided(arl2_kv_t kv, const void* q, const void* k, const void* v, int64_t ld,
                                  void* o, void* stream);
arl2_status arl2_kv_commit_strided(arl2_kv_t kv, const void* q, const void* k, const void* v, int64_t ld,
                                   void* o, void* stream);
int64_t arl2_kv_frames(arl2_kv_t kv);
int64_t arl2_kv_device_bytes(arl2_kv_t kv);
arl2_status arl2_kv_last_error(arl2_kv_t kv);
arl2_status arl2_kv_destroy(arl2_kv_t kv);

/* ---- Norm and rotation of queries and keys ---------------------------------
 * What a DiT or language-model block does to Q and K between its projection
 * and its attention, in one pass: per token and head
 *   y = x * rsqrt(mean(x^2) + eps) * w                     (over head_dim)
 * and then the rotation of pairs of channels by the token's position:
 *   (y0, y1) -> (y0 cos a - y1 sin a, y0 sin a + y1 cos a),
 *   a = pos[token][axis] * theta^(-2 i / axis_dim[axis]).
 * The axes take their axis_dim / 2 pairs one after the other (1 axis: a text
 * or frame position; 3 axes: frame, row and column of a video token); i counts
 * within the axis.  Pair p is channels (2p, 2p + 1), or with halves = 1
 * channels (p, p + R/2), R = sum of axis_dim; channels from R on are not
 * rotated.  Angles come from 64-bit fractions of a turn, so they stay exact to
 * 2^-24 of a turn over all int32 positions (negative ones too).  The arithmetic
 * is float32, rounded once to the tensors' type. */
typedef struct {
  int32_t n_axes;       /* 0 (no rotation) to 3 */
  int32_t axis_dim[3];  /* even, >= 2 for axes < n_axes; their sum R <= head_dim */
  int32_t halves;       /* 0: pairs of neighbours, 1: pairs R/2 apart (then R/2 is a
                           multiple of 8 in bf16, of 4 in float32) */
  float theta;          /* base of the rotation, in [1, 1e12] (ignored with n_axes = 0) */
  float eps;            /* >= 0, finite */
  const void* w_q;      /* device [head_dim] norm weights in the tensors' type, */
  const void* w_k;      /* both null: no norm; one null is INVALID_ARGUMENT */
} arl2_qk_prep;

/* q_out, k_out = prep(q, k) for `tokens` tokens.
 *   dtype    : ARL2_BF16 (head_dim a multiple of 8, <= 128) or ARL2_F32
 *              (head_dim a multiple of 4, <= 128).
 *   q, k     : device [tokens, heads, head_dim] and [tokens, kv_heads, head_dim];
 *              token rows are ld elements apart (views into the rows of a
 *              fused projection; 0: each contiguous), ld a multiple of 16 bytes.
 *   pos      : device int32 [tokens, n_axes] (null when n_axes = 0).
 *   q_out, k_out : the same shapes, token rows ld_out apart (0: contiguous).
 *              An output may be its own input (equal pointer and pitch: in
 *              place) and may otherwise share no byte with any input or the
 *              other output -- except that two outputs, or an output and the
 *              other input, may interleave in the rows of one pitch, as Q and K
 *              of a fused row do.
 * tokens = 0 does nothing.  Errors: INVALID_ARGUMENT, UNSUPPORTED (head_dim, or
 * R/2 with halves), CUDA. */
arl2_status arl2_qk_norm_rope(const arl2_qk_prep* prep, int32_t dtype, int32_t heads, int32_t kv_heads,
                              int32_t head_dim, int64_t tokens, const void* q, const void* k, int64_t ld,
                              const int32_t* pos, void* q_out, void* k_out, int64_t ld_out, void* stream);

/* ---- Softmax layers on a paged KV cache -----------------------------------
 * The cache of many streams in one pool of pages, next to the contiguous
 * arl2_kv layers: streams of different lengths, chunks of one to many new
 * tokens, shared key heads (grouped queries), and eviction.
 *
 * The pools are the caller's device memory in the handle's dtype, both
 * [n_pages, kv_heads, page_size, head_dim], 16-byte aligned; they must outlive
 * the handle.  Key j of a stream is row j % page_size of page pages[j / page_size].
 * The handle owns work space only (fixed at init), and as everywhere must not
 * be used from two streams at once: two captured graphs of one handle share it,
 * so their replays must be ordered.
 *
 * A batch of streams lives in device memory and is read by the kernels alone,
 * so that a captured graph may be replayed with other lengths and pages:
 *   q_start : int32 [n_seqs + 1], the streams' first rows among the new tokens;
 *             non-decreasing; rows from q_start[n_seqs] on are left as they were;
 *   kv_len  : int32 [n_seqs], keys cached per stream, the new tokens' included;
 *   pages   : int32 [n_seqs, pages_ld], the streams' pages in order (entries
 *             past the last page are not read).
 * The host gives bounds that size the launches: tokens (rows of the new-token
 * tensors), max_q and max_kv (at least any stream's new tokens and kv_len).
 * They may be loose: attend and weights count work in 32 bits, which always suffice
 * where (tokens * heads / 32 + n_seqs * kv_heads) * (max_kv / 64 + 8) is below
 * 2^31 - 2^14, whatever max_q is, and answer UNSUPPORTED where they might not.
 * What the kernels find out of range they do not access: a stream whose rows
 * or lengths break a bound is left out (its outputs stay as they were, but for
 * arl2_paged_evict's), a page number outside [0, n_pages) reads as zeros and is
 * not written; both record ARL2_ERR_PAGE for arl2_paged_last_error.  (Calls that
 * launch nothing record nothing: append and attend with tokens = 0, attend with
 * max_q = 0.) */
typedef struct {
  int32_t heads;        /* H query heads */
  int32_t kv_heads;     /* Hk: divides heads; heads / kv_heads <= 64 */
  int32_t head_dim;     /* bf16: 128; float32: a multiple of 4, <= 128 */
  int32_t page_size;    /* a multiple of 8, <= 4096 */
  int32_t n_pages;      /* >= 1; n_pages * kv_heads * page_size < 2^31 */
  int32_t dtype;        /* arl2_dtype */
  float softmax_scale;  /* 0 => 1/sqrt(head_dim) */
} arl2_paged_config;

typedef struct {
  int32_t n_seqs;  /* 0: every call returns at once */
  int32_t tokens;
  int32_t max_q;
  int32_t max_kv;
  int32_t pages_ld;
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* pages;
} arl2_paged_batch;

typedef struct arl2_paged* arl2_paged_t;

/* Waits for the stream: what it clears is clear for any stream's first call. */
arl2_status arl2_paged_init(const arl2_paged_config* cfg, void* k_pool, void* v_pool, void* stream,
                            arl2_paged_t* out);

/* Store the new tokens' K and V as the last rows of their streams (keys
 * kv_len - n .. kv_len - 1 of a stream with n new tokens), with prep's norm and
 * rotation of K in the same pass, and Q's into q_out.
 *   prep  : null stores K as it is; then q and q_out must be null.
 *   q, k, v : [tokens, H or Hk, head_dim], token rows ld elements apart (0:
 *           contiguous); q and q_out may both be null.  pos: int32 [tokens, n_axes].
 *   q_out : [tokens, H, head_dim] contiguous; may be q itself when q is
 *           contiguous, and otherwise shares no byte with an input.
 * Tokens before key 0 (kv_len < n) are ARL2_ERR_PAGE and not stored.  Streams may
 * share the pages that they read (a common prefix); a row that is stored to must
 * be one stream's. */
arl2_status arl2_paged_append(arl2_paged_t h, const arl2_paged_batch* batch, const arl2_qk_prep* prep, const void* q,
                              const void* k, const void* v, int64_t ld, const int32_t* pos, void* q_out,
                              void* stream);

/* O = softmax(Q K^T * scale) V of the new tokens over their streams' cached keys.
 *   mask_block m: 0: every new token sees all kv_len keys (a frame's pass).
 *     m > 0: new token t (from 0) of a stream with n new tokens sees the keys
 *     before the chunk and the chunk's blocks of m tokens up to its own:
 *     keys < clamp(kv_len - n + (floor(t / m) + 1) * m, 0, kv_len).  m = 1 is
 *     causal, m = tokens per frame is causal by frames.
 *   q   : [tokens, H, head_dim], token rows ld_q elements apart (0: contiguous).
 *   o   : [tokens, H, head_dim] contiguous, shares no byte with q, lse or the pools.
 *   lse : float32 [tokens, H], log sum exp of a row's scaled logits; may be null.
 * A row that sees no key gets O = 0 and lse = -inf; one whose query is no number
 * gets NaN for both, and others are not touched by it.  K and V of the cached
 * keys (those below kv_len) must be finite; what lies past kv_len in the pool is
 * not used, whatever it is.  A query pass that is not to be kept appends to
 * scratch pages of its own table, as the calls take the pages anew each time. */
arl2_status arl2_paged_attend(arl2_paged_t h, const arl2_paged_batch* batch, const void* q, int64_t ld_q,
                              int32_t mask_block, void* o, float* lse, void* stream);

/* The attention weight that every cached key received from the new tokens,
 * summed over their rows and the query heads of the key head, on top of the
 * decayed sum so far:
 *   w_out[b][hk][j] = decay * w_in[b][hk][j] + sum exp(q k_j * scale - lse[row])
 * over the rows that see key j.  lse is arl2_paged_attend's for the same
 * batch, q and mask_block (rows with lse = -inf, and finite q, add nothing).  w_in, w_out:
 * float32 [n_seqs, Hk, w_ld], w_ld >= max_kv; w_out may be w_in (equal pointer)
 * and otherwise shares no byte with it.  Entries from kv_len on are set to 0
 * in w_out (not read in w_in), so that tokens appended later start from 0. */
arl2_status arl2_paged_weights(arl2_paged_t h, const arl2_paged_batch* batch, const void* q, int64_t ld_q,
                               int32_t mask_block, const float* lse, float decay, const float* w_in, float* w_out,
                               int64_t w_ld, void* stream);

/* Cut every stream to at most `budget` keys, per key head: the first `sink`
 * and the last `recent` keys, and of the others the budget - sink - recent
 * with the largest weights w_in (equal weights: the lower index; NaN counts as
 * the lowest), in their old order.  A stream of at most budget keys keeps all.
 * The kept K and V rows are copied to the pages of dst_pages (int32 [n_seqs,
 * dst_ld], ceil(min(kv_len, budget) / page_size) used per stream), which must
 * be pages that no stream of `batch` uses and no two entries may share; a
 * destination page that the stream itself reads is ARL2_ERR_PAGE and not
 * written.  The old pages stay as they are: they may be shared with other
 * streams, and belong to the caller again afterwards.
 *   w_out      : float32 [n_seqs, Hk, w_ld]: the kept keys' weights, then 0;
 *                shares no byte with w_in.
 *   kept       : int32 [n_seqs, Hk, budget]: the kept keys' old indices, then -1.
 *   kv_len_out : int32 [n_seqs]: min(kv_len, budget).
 * A stream whose length breaks a bound (ARL2_ERR_PAGE) has no keys afterwards:
 * its kv_len_out is 0, its kept -1 and its w_out 0.
 * No output shares a byte with an input, another output or the batch's arrays.
 * q_start, tokens and max_q of the batch are not used.
 * budget >= 1, sink and recent >= 0, sink + recent <= budget. */
arl2_status arl2_paged_evict(arl2_paged_t h, const arl2_paged_batch* batch, const float* w_in, int64_t w_ld,
                             int32_t budget, int32_t sink, int32_t recent, const int32_t* dst_pages, int32_t dst_ld,
                             float* w_out, int32_t* kept, int32_t* kv_len_out, void* stream);

/* Wait for the handle's device, whatever streams its calls and the replays of
 * captured ones ran on, and return (and clear) the first error recorded by its
 * kernels (ARL2_ERR_PAGE, ARL2_ERR_TIMEOUT), ARL2_OK if none.  After
 * ARL2_ERR_TIMEOUT, or a q_start that decreases, a call's outputs are undefined,
 * and so are those of later calls until this one has returned. */
arl2_status arl2_paged_last_error(arl2_paged_t h);
int64_t arl2_paged_device_bytes(arl2_paged_t h);
/* As arl2_state_set_wait_limit. */
arl2_status arl2_paged_set_wait_limit(arl2_paged_t h, uint64_t limit_ns);
arl2_status arl2_paged_destroy(arl2_paged_t h);

/* ---- Hybrid attention block (the layer around the hot path) ----------------
 * One hybrid layer with the projections a DiT attention block puts around it
 * (ARL2 summary, section 2.1: the frozen pretrained Q/K/V projections feed
 * both branches; alpha and beta are per-token learned projections), bf16 with
 * fp32 accumulation, for a hidden size D = H * 128:
 *   Q = X W_qkv[:, 0:D],  K = X W_qkv[:, D:2D],  V = X W_qkv[:, 2D:3D]
 *   O = the hybrid layer's output on (Q, K, V)  (arl2_frame_query / commit)
 *   Y = O W_o
 * and, on the commit (clean) pass, the gates from the tokens:
 *   alpha[b][h]   = sigmoid( mean over t of (X W_gate)[b][t][h] )
 *   beta[b][h][t] = sigmoid( (X W_gate)[b][t][H + h] )
 * (the pages fix neither the gates' inputs nor their pooling; a head-wise
 * alpha from the frame's mean token and a per-token beta are this build's
 * reading).  No position encoding is applied: Q and K enter the layer as
 * projected.  The projections are plain GEMMs (this library's tcgen05 GEMM,
 * arl2_gemm_bf16: fp32 accumulate, bf16 results): one against
 * [W_qkv | W_gate] (the layer reads Q, K and V as strided views of its rows),
 * one against W_o.
 *   cfg     : bf16 configuration with head_dim 128 (hidden D = heads * 128).
 *   w_qkv   : device bf16 [D, 3D] row-major (X W: y_j = sum_i x_i W[i][j]);
 *   w_o     : device bf16 [D, D];  w_gate : device bf16 [D, 2H] (alpha columns
 *             first, then beta columns);  phi_q, phi_k, phi_v as for
 *             arl2_state_init.  Every weight is copied at init.
 *   x, y    : device bf16 [B, L, D] (token-major; y must not overlap x).
 * The block owns one hybrid-layer handle (its state, KV-free) and its work
 * space (Q, K, V, O, gates: about 5 * B * L * D * 2 bytes, fixed at init).  arl2_block_layer() returns that handle
 * for state get/set, last_error and the device-byte count; it is destroyed
 * with the block.  Errors: INVALID_ARGUMENT, UNSUPPORTED (not bf16 / d != 128),
 * OUT_OF_MEMORY, CUDA. */
typedef struct arl2_block* arl2_block_t;
arl2_status arl2_block_init(const arl2_config* cfg, const void* w_qkv, const void* w_o, const void* w_gate,
                            const void* phi_q, const void* phi_k, const void* phi_v, void* stream,
                            arl2_block_t* out);
arl2_status arl2_block_query(arl2_block_t blk, const void* x, void* y, void* stream);
arl2_status arl2_block_commit(arl2_block_t blk, const void* x, void* y, void* stream);
arl2_state_t arl2_block_layer(arl2_block_t blk);
arl2_status arl2_block_destroy(arl2_block_t blk);

/* The attention block's projection GEMM on its own: C = A B with A [M, K],
 * B [K, N] and C [M, N] row-major bf16 device matrices (leading dimensions
 * lda >= K, ldb >= N, ldc >= N elements, each a multiple of 8; pointers
 * 16-byte aligned), fp32 accumulation, C rounded to bf16.  This is the
 * token-by-weight product that turns the block's input X into Q | K | V | gate
 * logits and the layer's output O into Y (ARL2 summary, section 2.1: the frozen
 * Q/K/V projections feed both branches).  C must not overlap A or B.
 * Errors: INVALID_ARGUMENT (null or misaligned pointers, bad sizes or leading
 * dimensions, overlap), NO_DEVICE, CUDA.  A device-side wait that runs out is
 * not reported here: the call has no handle; the block reports it through its
 * layer (arl2_last_error of arl2_block_layer). */
arl2_status arl2_gemm_bf16(const void* a, int64_t lda, const void* b, int64_t ldb, void* c, int64_t ldc, int64_t m,
                           int64_t n, int64_t k, void* stream);

/* Diagnostic, host only (no device is touched): the work partition the
 * attention kernel uses for `batch` streams of `heads` heads with q_len query
 * rows and kv_len keys on `pairs` CTA pairs.  The (stream, head) slabs are cut
 * into blocks of 256 query rows, each block into key tiles of 128; every pair
 * walks its own list of segments (a run [j0, j1) of key tiles of one block).
 * A block split across pairs is finished by the pair holding key tile 0, which
 * merges the pieces of the n_contrib pairs right after it.  On return
 * *n_pairs is the pairs used (<= pairs), *n_segs the segments, seg_first
 * [*n_pairs + 1] the offsets of each pair's list and segs [*n_segs][5] the
 * segments as (slab = stream * heads + head, block, j0, j1, n_contrib).
 * segs must hold max_segs segments, seg_first 97 entries.
 * Errors: INVALID_ARGUMENT (null pointers, sizes < 1, pairs > 96),
 * UNSUPPORTED (the problem does not fit the partition's encoding or more than
 * max_segs segments). */
arl2_status arl2_attn_partition(int batch, int heads, int q_len, int kv_len, int pairs, int32_t* segs, int max_segs,
                                int32_t* seg_first, int* n_segs, int* n_pairs);

/* ---- State write without allocation ---------------------------------------
 * The paper has no counterpart to this call; it is a deployment aid.  Some
 * callers cannot call cudaMalloc: code that runs while a CUDA graph is being
 * captured, a host that must keep a fixed device-memory budget for the
 * process's whole life, or an embedding runtime whose allocator owns the
 * device and forbids allocations behind its back.  For them this call
 * computes one frame's state write,
 *   S_next = alpha S_prev + c K'^T diag(beta) (V' - K' S_prev),
 * K' = rownorm2(K phi_k), V' = V phi_v, with the same kernels as
 * arl2_frame_commit, but with no handle and without allocating anything: its
 * work space (transposed phi_k and phi_v, a bf16 copy of S_prev, and the
 * per-128-token partial sums) lives in one static device array of
 * ARL2_NOALLOC_SCRATCH_BYTES that every GPU loading the library holds until
 * the process exits.
 *   cfg       : bf16 configuration (head_dim 128); flags and softmax_scale are
 *               ignored; corr_scale < 0 means c = 1/L.
 *   k, v      : device bf16 [B, L, H, 128];  phi_k, phi_v : device bf16 [H, 128, 128]
 *               as given to arl2_state_init;
 *   S_prev    : device float32 [B, H, 128, 128];  alpha : float32 [B, H];
 *   beta      : float32 [B, H, L];  S_next : device float32 [B, H, 128, 128];
 *   dev_error : device uint32, set to 0 by the call and to an arl2_status by a
 *               kernel whose bounded wait ran out (read it after a sync).
 * S_next and dev_error may share no byte with any input or with each other
 * (INVALID_ARGUMENT otherwise).
 * All pointers are caller-owned and 16-byte aligned.  The scratch needed is
 *   2 * H * 32768 + 2 * B * H * 32768 + B * H * ceil(L / 128) * 65536 bytes
 * (each part rounded up to 1 KiB); more than ARL2_NOALLOC_SCRATCH_BYTES returns
 * ARL2_ERR_SCRATCH_LIMIT before any CUDA call.  The first call on a device
 * looks up the array's device address (once per device, with that device
 * current); make that first call before any stream capture begins.  The
 * library keeps that address for the life of the process, so it must not
 * outlive the device context it was looked up in: after cudaDeviceReset (or
 * any other teardown of the device's primary context) do not call this entry
 * point again in the same process.  Every
 * call shares the one array and leaves its contents behind, so calls whose
 * kernels overlap on the GPU (other streams, other host threads) race:
 * serialise them.  Errors: INVALID_ARGUMENT, UNSUPPORTED, SCRATCH_LIMIT, CUDA. */
#define ARL2_NOALLOC_SCRATCH_BYTES (16u << 20)
arl2_status arl2_state_write_noalloc(const arl2_config* cfg, const void* k, const void* v,
                                     const void* phi_k, const void* phi_v, const float* S_prev,
                                     const float* alpha, const float* beta, float* S_next,
                                     uint32_t* dev_error, void* stream);

/* ---- Diagnostics -----------------------------------------------------------
 * Run one kernel whose bounded wait is on a barrier that nothing completes,
 * with the given limit; returns ARL2_ERR_TIMEOUT when the limit worked (the
 * kernel returned and reported it) -- used by the failure-detection tests. */
arl2_status arl2_selftest_wait_timeout(uint64_t limit_ns, void* stream);

/* y[i] = 2^x[i] (device float32 arrays of n values) through the FMA-pipe
 * exponential the attention kernel uses for part of its softmax (a degree-3
 * polynomial after rounding x to an integer; inputs clamped to [-125, 125];
 * relative error <= 1.0e-4).  The attention kernel takes it for 3 of the 16
 * column pairs of every 32-column chunk, in a paired form with the same
 * operations, and the MUFU for the rest.  For accuracy tests of that routine. */
arl2_status arl2_selftest_exp2(const float* x, float* y, int64_t n, void* stream);

const char* arl2_status_string(arl2_status s);
int32_t arl2_abi_version(void);

/* 1 in the debug build (libarl2_debug.so, kernels compiled with
 * -DARL2_DEBUG_BOUNDS: each checks the indices it takes from its parameters and
 * launch shape before it uses them, skips the access when a check fails and
 * records ARL2_ERR_BOUNDS, which arl2_last_error returns), 0 in the release
 * build (libarl2.so), whose kernels carry no such checks.  Needs no device. */
int32_t arl2_debug_bounds_enabled(void);

#ifdef __cplusplus
}
#endif

#endif /* ARL2_H */
