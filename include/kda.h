/*
 * libkda -- Kimi Delta Attention (KDA) operator for AMD Instinct MI355X (gfx950).
 *
 * The operator is the per-head gated delta-rule recurrence defined in the
 * "Kimi K3 Technical Report review" (jw9603.github.io), sections 3.2-3.3:
 *
 *     Sbar_{t-1} = Diag(alpha_t) S_{t-1}            (key channel i kept at rate alpha_t[i])
 *     S_t        = Sbar_{t-1} + beta_t k_t (v_t - Sbar_{t-1}^T k_t)^T
 *     o_t        = S_t^T q_t                          (read from the updated state)
 *
 * with S_t in R^{d_k x d_v}.  Decay is applied before the write.  There is no
 * readout scale and keys are used as given (the library does not normalise them).
 *
 * Conventions shared by every call:
 *  - All tensor pointers are DEVICE pointers (HIP global memory) owned by the
 *    caller.  The bf16 prefill with d_k in {64, 128} (kda_chunk_fwd, its
 *    snapshot, packed-batch and gated forms, and a split of one part) keeps its
 *    per-chunk intermediates ("chunk records", about 1 KB per token and head) in
 *    device memory it takes from a memory pool the library creates on each
 *    device at first use and keeps: allocated and freed in stream order on
 *    `stream` around the call, at most 1 GiB of records per buffer (2 GiB when a
 *    long batch's blocks overlap); when that memory cannot be had, or a packed
 *    batch's records exceed the cap, the call runs a kernel that needs none.
 *    kda_chunk_fwd_split_noalloc never allocates.  Beyond that pool the library
 *    keeps, per device, its compute-unit count and the address of the
 *    allocation-free call's array, and a thread-local copy of the last HIP
 *    error.  Calls are reentrant.
 *  - `stream` is the hipStream_t the work is enqueued on (NULL = the default
 *    stream).  Each call only enqueues work on that stream and returns without
 *    synchronising; a device-side fault surfaces at the caller's next
 *    synchronisation.
 *  - Layouts are dense, row-major, token-major: [B][T][H][d] for per-token
 *    tensors and [B][H][d_k][d_v] for states.
 *  - Every pointer must be 16-byte aligned.
 *  - Arguments are validated before any HIP call; on error nothing is enqueued
 *    and no output is touched.  Calls never abort and never throw.
 *  - Supported sizes: d_k, d_v in {16, 32, 64, 128}, for bf16 and fp32 q/k/v.
 *  - Arithmetic.  The state is carried in fp32 and every product accumulates in
 *    fp32.  With fp32 q/k/v all matrix-core operands are fp32.  With bf16 q/k/v
 *    the matrix-core operands are fp16: the decayed keys and queries, the
 *    factors of the intra-chunk key products (each bounded by |k| or |q|: every
 *    decay ratio inside a chunk is split at a power-of-two block boundary into
 *    two products of decays; the single-kernel form used without a workspace
 *    takes inverse-decayed keys, at most e^10 |k|, and processes a chunk whose
 *    decay would exceed that as shorter exact segments), and the state and
 *    values rescaled by a power of two per state column, so their magnitude is
 *    not restricted.  q and k entries should stay below 6.5e4 in magnitude.
 *    (Head sizes served by the generic kernel form the intra-chunk key products
 *    from bf16 high/low pairs instead, about 16 significant bits.)
 *  - Input domain: alpha in [exp(-5), 1] (the lower-bounded decay of section 3.5
 *    of the same page); results outside it are not guaranteed, except that the
 *    bf16 prefill with d_k in {64, 128} on its chunk-record path accepts any
 *    alpha in [0, 1].  beta may be any finite value (it is not clamped).
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>

#include <hip/hip_runtime_api.h> /* hipStream_t */

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  KDA_F32 = 0,  /* IEEE binary32 */
  KDA_BF16 = 1, /* bfloat16; outputs are rounded to nearest even */
  KDA_E4M3 = 2  /* 8 bits (4 exponent, 3 mantissa; largest 448, no infinity): of cached keys and values only */
} kda_dtype;

typedef enum {
  KDA_OK = 0,
  KDA_ERR_NULL = 1,        /* a required pointer is NULL */
  KDA_ERR_SHAPE = 2,       /* B, H < 1, T < 0, or a size overflows 2^31 elements per row index */
  KDA_ERR_DTYPE = 3,       /* qkv_dtype or o_dtype is not a kda_dtype */
  KDA_ERR_UNSUPPORTED = 4, /* d_k/d_v not in {16,32,64,128} or chunk not in {16,32,64} */
  KDA_ERR_MISALIGNED = 5,  /* a pointer is not 16-byte aligned */
  KDA_ERR_ALIAS = 6,       /* an output overlaps an input it may not overlap */
  KDA_ERR_HIP = 7          /* the launch failed; kda_last_hip_error() holds the hipError_t */
} kda_status;

/*
 * Chunkwise-parallel prefill over T tokens for B sequences and H heads.
 *
 * The sequence is cut into chunks of `chunk` tokens (the chunkwise form of the
 * second page, "Kimi 모델 분석", rlaope.github.io, section on putting the
 * recurrence on the GPU: chunk size 64, WY representation, UT transform, only
 * the state carried between chunks).  The result equals the token recurrence
 * above up to rounding, for any chunk size.
 *
 *   q, k   : [B][T][H][d_k]  qkv_dtype          (read)
 *   v      : [B][T][H][d_v]  qkv_dtype          (read)
 *   alpha  : [B][T][H][d_k]  fp32, per-channel retention   (read)
 *   beta   : [B][T][H]       fp32, write strength          (read)
 *   S0     : [B][H][d_k][d_v] fp32 initial state, or NULL for zeros   (read)
 *   o      : [B][T][H][d_v]  o_dtype, o_t for every token             (written)
 *   o_dtype: KDA_F32 or KDA_BF16 (the q/k/v dtype is the usual choice).  A
 *            bf16 o is exactly the fp32 result rounded to nearest even; that
 *            rounding alone can reach 2^-8 of |o_t|, so an fp32 o keeps the full
 *            accuracy of the fp32 state.
 *   S_T    : [B][H][d_k][d_v] fp32 final state, or NULL to skip       (written)
 *   chunk  : 16, 32 or 64 (64 is the size the second page names).  The chunk
 *            size a call actually runs: 32 for chunk 32 or 64 with bf16 q/k/v,
 *            d_k in {64, 128} and d_v a multiple of 32 (the pipelined kernel,
 *            whose stage rings of 64-token chunks would not fit the 160 KB of
 *            LDS), and for chunk 64 with fp32 q/k/v and d_k in {64, 128} (same
 *            reason); the requested size otherwise.  The result does not depend
 *            on the chunk size beyond rounding.
 *
 * S0 == S_T (the same buffer) is allowed and updates the state in place; any
 * other overlap between an output and an input returns KDA_ERR_ALIAS.
 * T == 0 writes S_T = S0 (zeros when S0 is NULL) and touches nothing else.
 * Any T >= 1 is accepted; a partial last chunk is masked.
 */
kda_status kda_chunk_fwd(const void* q, const void* k, const void* v, kda_dtype qkv_dtype,
                         const float* alpha, const float* beta, const float* S0,
                         void* o, kda_dtype o_dtype, float* S_T,
                         int B, int T, int H, int d_k, int d_v, int chunk, hipStream_t stream);

/*
 * The chunk size a kda_chunk_fwd call with these arguments runs (see `chunk`
 * above), written to *run_chunk.  Host only: enqueues nothing and touches no
 * device.  Errors: KDA_ERR_DTYPE, KDA_ERR_SHAPE (H < 1), KDA_ERR_UNSUPPORTED
 * (a size or chunk that kda_chunk_fwd would refuse), KDA_ERR_NULL.
 */
kda_status kda_chunk_fwd_run_chunk(kda_dtype qkv_dtype, int H, int d_k, int d_v, int chunk, int* run_chunk);

/* Most positions one kda_chunk_fwd_snapshots call records. */
#define KDA_MAX_SNAPSHOTS 128

/*
 * kda_chunk_fwd that also records the state at caller-chosen positions, for
 * prefix caching.  A KDA layer keeps no per-token keys and values: resuming a
 * shared prompt prefix needs the state at exactly that position, and saving it
 * at every token is too costly, so a server saves it at positions it selects --
 * at a fixed interval, or where a prompt ends (the second page, "Kimi 모델
 * 분석", section on prefix caching breaking and its parts on separating block
 * size from caching granularity and on where to store the summaries).
 *
 * Every argument of kda_chunk_fwd keeps its meaning; in addition:
 *   snap_tokens: HOST array of n_snap token counts, strictly increasing, each
 *                in [1, T] and a multiple of `chunk` or equal to T.  Entry j
 *                asks for the state after the first snap_tokens[j] tokens of
 *                every sequence, S_{snap_tokens[j]} (read during the call only).
 *   n_snap     : 0 .. KDA_MAX_SNAPSHOTS (0: identical to kda_chunk_fwd).
 *   snaps      : [B][H][n_snap][d_k][d_v] fp32, device (written).  Snapshot j
 *                of (b, h) is the same value kda_chunk_fwd's S_T would hold for
 *                the first snap_tokens[j] tokens with the same S0 (bit for bit:
 *                the chunks before it are computed identically).
 *
 * Errors, in addition to kda_chunk_fwd's: KDA_ERR_SHAPE for n_snap outside
 * [0, KDA_MAX_SNAPSHOTS] or a position list that breaks the rules above;
 * KDA_ERR_NULL for a NULL snap_tokens or snaps with n_snap > 0;
 * KDA_ERR_MISALIGNED / KDA_ERR_ALIAS for snaps as for the other outputs.
 */
kda_status kda_chunk_fwd_snapshots(const void* q, const void* k, const void* v, kda_dtype qkv_dtype,
                                   const float* alpha, const float* beta, const float* S0,
                                   void* o, kda_dtype o_dtype, float* S_T,
                                   const int* snap_tokens, int n_snap, float* snaps,
                                   int B, int T, int H, int d_k, int d_v, int chunk, hipStream_t stream);

/*
 * One batched decode step: one new token for each of B sequences and H heads,
 * i.e. exactly one step of the recurrence, applied to the state in place.
 *
 *   q, k   : [B][H][d_k] qkv_dtype        v: [B][H][d_v] qkv_dtype   (read)
 *   alpha  : [B][H][d_k] fp32             beta: [B][H] fp32          (read)
 *   S      : [B][H][d_k][d_v] fp32, read and overwritten with S_t    (in place)
 *   o      : [B][H][d_v] o_dtype (KDA_F32 or KDA_BF16), o_t         (written)
 *
 * Each state is streamed once from HBM and written back once.  o must not
 * overlap S or any input (KDA_ERR_ALIAS).
 */
kda_status kda_decode_step(const void* q, const void* k, const void* v, kda_dtype qkv_dtype,
                           const float* alpha, const float* beta, float* S, void* o, kda_dtype o_dtype,
                           int B, int H, int d_k, int d_v, hipStream_t stream);

/*
 * kda_chunk_fwd over a packed batch of N sequences of different lengths (for
 * serving: prompts of a batch are concatenated along the token axis).  Sequence
 * b covers token rows [cu_seqlens[b], cu_seqlens[b+1]) and is an independent
 * recurrence with its own initial and final state.
 *
 *   q, k, alpha: [total_T][H][d_k]   v, o: [total_T][H][d_v]   beta: [total_T][H]
 *                (dtypes as in kda_chunk_fwd)
 *   S0, S_T    : [N][H][d_k][d_v] fp32 (S0 may be NULL; S_T may be NULL or S0)
 *   cu_seqlens : [N + 1] int32, DEVICE memory, non-decreasing from 0 to total_T.
 *                The kernels clamp each offset to [0, total_T] and each length
 *                to >= 0, so no offset can make them access memory out of
 *                range; o rows not covered by any sequence are not written.
 *   N          : >= 1 sequences;  total_T >= 0.
 *
 * Validation and errors as kda_chunk_fwd (cu_seqlens must be non-NULL and
 * 16-byte aligned, and may not overlap an output).  A sequence's results equal
 * kda_chunk_fwd run on that sequence alone up to rounding.
 */
kda_status kda_chunk_fwd_varlen(const void* q, const void* k, const void* v, kda_dtype qkv_dtype,
                                const float* alpha, const float* beta, const float* S0,
                                void* o, kda_dtype o_dtype, float* S_T,
                                const int* cu_seqlens, int N, int total_T,
                                int H, int d_k, int d_v, int chunk, hipStream_t stream);

/*
 * kda_chunk_fwd with the gate fused in: instead of alpha, the caller passes the
 * gate pre-activation z and a per-head log-scale A, and the kernels form the
 * lower-bounded retention of section 3.5 of the first page,
 *     alpha_t[i] = exp(-5 * sigmoid(exp(A_h) * z_t[i]))      (in (e^-5, 1)),
 * in fp32 as they read z, so no fp32 alpha tensor is stored or read: the
 * per-token-head input shrinks from 4*d_k to 2*d_k bytes with bf16 z.
 *
 *   z : [B][T][H][d_k] in qkv_dtype (read)        A : [H] fp32, device (read)
 * Every other argument as kda_chunk_fwd.  The result equals kda_chunk_fwd with
 * alpha = the formula above evaluated in fp32 (the exponentials and the
 * reciprocal use the hardware's approximations, within a few fp32 ulps).
 */
kda_status kda_chunk_fwd_gated(const void* q, const void* k, const void* v, kda_dtype qkv_dtype,
                               const void* z, const float* A, const float* beta, const float* S0,
                               void* o, kda_dtype o_dtype, float* S_T,
                               int B, int T, int H, int d_k, int d_v, int chunk, hipStream_t stream);

/*
 * Prefill with each sequence split into parts that run side by side: for few
 * long sequences (small B*H) the single-pass kernel has one workgroup per
 * (sequence, head, 32 state columns) and leaves most of the GPU idle.  Between
 * chunks only the state is carried (the second page, on putting the recurrence
 * on the GPU), and a run of tokens maps its incoming state S to M S + N with a
 * d_k x d_k transition M (section 3.3 of the first page: each token applies
 * (I - beta k k^T) Diag(alpha) to every state column and adds beta k v^T), so:
 * pass 1 computes N and M of every part but the last, in parallel; a combine
 * step chains S_in(j+1) = M_j S_in(j) + N_j in fp32 (from 9 parts on, as a tree
 * over the part maps: log2 levels of pairwise compositions, then one product
 * with S0); pass 2 reruns every part from its S_in and writes o and S_T.  Parts
 * are whole 32-token chunks.
 *
 *   parts     : 0 = the library's choice (a step-count model of the launches
 *               on num_cus compute units against the single pass the call would
 *               otherwise run; 1 part when splitting does not pay);
 *               1 = the single pass (kda_chunk_fwd); >= 2 = that many parts, or
 *               fewer when T has fewer 32-token chunks.
 *   num_cus   : compute units for the model; 0 = those of the current device.
 *   workspace : device memory of workspace_bytes bytes, 16-byte aligned, used
 *               for the transitions and incoming states; its contents on entry
 *               do not matter and are overwritten.  May be NULL when the
 *               resulting split has 1 part.  kda_chunk_fwd_split_plan gives the
 *               part count and the bytes needed:
 *               4 * B * H * d_k * (c * (P - 1) * (d_v + d_k) + P * d_v) for P
 *               parts, with c = 1 below 9 parts and c = 2 from 9 parts on.
 * Every other argument as kda_chunk_fwd.  Splitting is built for the pipelined
 * kernel's shapes (bf16 q/k/v, d_k in {64, 128}, d_v a multiple of 32, chunk 32
 * or 64); parts >= 2 for another shape returns KDA_ERR_UNSUPPORTED.  Errors:
 * as kda_chunk_fwd, plus KDA_ERR_NULL (workspace NULL when needed),
 * KDA_ERR_SHAPE (workspace_bytes too small, parts or num_cus < 0),
 * KDA_ERR_ALIAS (workspace overlaps an input or output), KDA_ERR_HIP (the
 * device's compute units could not be queried).  The result equals
 * kda_chunk_fwd up to rounding (the state entering each part goes through one
 * fp32 product with M instead of the chunk recurrence).  Three kernels are
 * enqueued on `stream` below 9 parts; from 9 parts on, 3 + ceil(log2(P - 1)).
 */
kda_status kda_chunk_fwd_split_plan(kda_dtype qkv_dtype, int B, int T, int H, int d_k, int d_v, int chunk,
                                    int parts, int num_cus, int* parts_out, size_t* workspace_bytes);
kda_status kda_chunk_fwd_split(const void* q, const void* k, const void* v, kda_dtype qkv_dtype,
                               const float* alpha, const float* beta, const float* S0,
                               void* o, kda_dtype o_dtype, float* S_T,
                               int B, int T, int H, int d_k, int d_v, int chunk,
                               int parts, int num_cus, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of device scratch kda_chunk_fwd_split_noalloc holds on each GPU (64 MiB). */
#define KDA_SPLIT_SCRATCH_BYTES ((size_t)64 << 20)

/*
 * kda_chunk_fwd_split for callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, harnesses that forbid allocation.  The
 * same split prefill, with its workspace in a fixed device array of
 * KDA_SPLIT_SCRATCH_BYTES that the library holds on each GPU it runs on (from
 * when the library's code is loaded on that GPU until the process ends).  The
 * call allocates nothing; the caller still passes every input and output.
 *
 *   parts : 0 = the library's choice among part counts whose workspace fits
 *           the scratch (1, the single pass, needs none); >= 2 = that many
 *           parts (or fewer, as kda_chunk_fwd_split), KDA_ERR_SHAPE when
 *           their workspace (kda_chunk_fwd_split_plan) exceeds
 *           KDA_SPLIT_SCRATCH_BYTES.
 * Every call on one GPU uses that GPU's one array and overwrites what the last
 * call left there: calls that overlap on one GPU (on other streams or from
 * other threads) race and must be ordered by the caller.  Every other argument
 * and error as kda_chunk_fwd_split; KDA_ERR_HIP also when the array's device
 * address cannot be obtained (kda_last_hip_error() holds the hipError_t).
 */
kda_status kda_chunk_fwd_split_noalloc(const void* q, const void* k, const void* v, kda_dtype qkv_dtype,
                                       const float* alpha, const float* beta, const float* S0,
                                       void* o, kda_dtype o_dtype, float* S_T,
                                       int B, int T, int H, int d_k, int d_v, int chunk,
                                       int parts, int num_cus, hipStream_t stream);

/*
 * kda_decode_step with the gate fused in (as kda_chunk_fwd_gated):
 *   z : [B][H][d_k] in qkv_dtype (read)           A : [H] fp32, device (read)
 */
kda_status kda_decode_step_gated(const void* q, const void* k, const void* v, kda_dtype qkv_dtype,
                                 const void* z, const float* A, const float* beta, float* S, void* o,
                                 kda_dtype o_dtype, int B, int H, int d_k, int d_v, hipStream_t stream);

/* Most draft tokens one speculative step may verify. */
#define KDA_MAX_DRAFT 16

/*
 * Speculative decoding, pass 1 of 2: verify K draft tokens of each of B
 * sequences without changing the state.  Each decode step overwrites the state
 * in place, so a rejected draft token could not be taken back afterwards (the
 * second page, "Kimi 모델 분석", serving section on speculative decoding; the
 * first page, section 13, on restoring the state after rejected draft tokens).
 * This call reads S once and gives what K kda_decode_step calls would (the
 * same recurrence, restated, in fp32): S is multiplied once by every draft's
 * key and query, each decayed to the draft's position, and the drafts' effect
 * on one another is resolved on those products with coefficients formed from
 * k, q and alpha alone.  It stores what the commit pass needs instead of the
 * state.
 *
 *   q, k   : [B][K][H][d_k] qkv_dtype     v: [B][K][H][d_v] qkv_dtype   (read)
 *   alpha  : [B][K][H][d_k] fp32          beta: [B][K][H] fp32          (read)
 *   S      : [B][H][d_k][d_v] fp32, the state before the drafts (read only)
 *   o      : [B][K][H][d_v] o_dtype: o_t as if tokens 1..t were accepted (written)
 *   u      : [B][H][K][d_v] fp32: the write vectors u_t = beta_t (v_t - Sbar^T k_t)
 *            of the K updates S_t = Diag(alpha_t) S_{t-1} + k_t u_t^T   (written)
 *   K      : 1 .. KDA_MAX_DRAFT
 *
 * o and u may overlap nothing else (KDA_ERR_ALIAS).  Other rules as for
 * kda_decode_step.
 */
kda_status kda_decode_verify(const void* q, const void* k, const void* v, kda_dtype qkv_dtype,
                             const float* alpha, const float* beta, const float* S,
                             void* o, kda_dtype o_dtype, float* u,
                             int B, int K, int H, int d_k, int d_v, hipStream_t stream);

/*
 * Speculative decoding, pass 2 of 2: advance the state over the accepted
 * prefix.  For sequence b, j = n_accept[b] (clamped to [0, K]) tokens were
 * accepted; S becomes the state after them,
 *     S_j = Diag(P_j) S + sum_{t<j} Diag(P_j / P_{t+1}) k_t u_t^T,
 *     P_m = prod_{s<m} alpha_s   (per key channel; products only, no division),
 * the closed form of j steps of the recurrence, in one read and one write of
 * each state (none when j = 0).  k, alpha and u are the arguments and output
 * of the kda_decode_verify call for the same drafts.
 *
 *   n_accept: [B] int32, DEVICE memory (read)
 *   S       : [B][H][d_k][d_v] fp32, updated in place
 *
 * S may overlap none of the inputs (KDA_ERR_ALIAS).
 */
kda_status kda_decode_commit(const void* k, kda_dtype qkv_dtype, const float* alpha, const float* u,
                             const int* n_accept, float* S,
                             int B, int K, int H, int d_k, int d_v, hipStream_t stream);

/* ---- norms of queries and keys ------------------------------------------------------- */

typedef enum {
  KDA_NORM_L2 = 0, /* x / sqrt(sum_i x_i^2 + eps) */
  KDA_NORM_RMS = 1 /* x / sqrt(mean_i x_i^2 + eps) */
} kda_norm;

typedef enum {
  KDA_PAIR_HALVES = 0, /* values i and i + rot/2 turn together */
  KDA_PAIR_ADJACENT = 1 /* values 2i and 2i + 1 turn together */
} kda_pairing;

/*
 * Normalises queries and keys for each token and head and, where asked, turns
 * their first `rot` values by the token's position, in one pass: what a layer
 * does to its projections before kda_chunk_fwd or kda_decode_step read them
 * (those calls take keys as they are given).  For a query or key x of one head,
 *     y = w . x / sqrt(sum_i x_i^2 + eps)           (KDA_NORM_RMS: the mean)
 *     (a, b) -> (a cos f - b sin f, b cos f + a sin f),  f = pos * inv_freq[i],
 *                                                    for the rot/2 pairs i
 * and queries are then multiplied by q_scale.  Norms, weights and rotation are
 * formed in fp32, the angle f and its reduction in fp64 (so far positions keep
 * their precision), and the result is rounded once to the output's type.
 *
 *   q          : n rows of H_q heads of d values, dtype; row t starts at q + t * q_stride
 *   k          : n rows of H_k heads of d values, dtype, k_stride apart (NULL when H_k = 0)
 *                (strides in elements: rows may be slices of a fused projection's rows;
 *                heads and values inside a row are dense)
 *   q_weight, k_weight: [d] fp32, or NULL for ones                     (read)
 *   eps        : finite and >= 0.  With eps = 0 a head of zeros gives NaN.
 *   positions  : [n] int32, any value; inv_freq: [rot / 2] fp32         (read)
 *                (both NULL when rot = 0)
 *   rot        : a multiple of 16 in [0, d]
 *   q_out, k_out: as q and k, with q_out_stride and k_out_stride, out_dtype (written)
 *   d          : a multiple of 8 in [8, 256];  H_q >= 1, H_k >= 0;  n >= 0 (0: nothing is done)
 *
 * Pointers are 16-byte aligned and row strides a multiple of 16 bytes
 * (KDA_ERR_MISALIGNED), at least H * d elements unless n <= 1 (KDA_ERR_SHAPE).
 * q_out may be q itself with the same stride and type, and so may k_out be k;
 * any other common byte of an output and another array is KDA_ERR_ALIAS (rows
 * that lie between each other's without touching, as in a fused projection, are
 * fine).  Unknown norm, pairing or dtype: KDA_ERR_DTYPE; d or rot as above:
 * KDA_ERR_UNSUPPORTED; eps: KDA_ERR_SHAPE.  The sum of squares is formed in
 * fp32: |x| should stay below 1e18.
 */
kda_status kda_qk_norm(const void* q, long long q_stride, const void* k, long long k_stride, kda_dtype dtype,
                       kda_norm norm, const float* q_weight, const float* k_weight, float eps, float q_scale,
                       const int* positions, const float* inv_freq, int rot, kda_pairing pairing,
                       void* q_out, long long q_out_stride, void* k_out, long long k_out_stride,
                       kda_dtype out_dtype, int n, int H_q, int H_k, int d, hipStream_t stream);

/* ---- a cache of state pages ------------------------------------------------------------
 *
 * A server keeps the states of its sequences in a pool of pages, one page per
 * state of a layer: pool [n_layers][n_pages][page_bytes], where a layer's part
 * is the [n_pages][H][d_k][d_v] fp32 array that kda_decode_step_paged reads.  A
 * page's number is the same on every layer.
 *   table : [n_rows][width] int32, one row per sequence slot of the server: the
 *           pages it holds.  A row's first n_private entries are states that
 *           its decode steps write (usually one, the running state); the others
 *           are recorded states (kda_chunk_fwd_snapshots) that rows may share.
 *           An entry outside [0, n_pages) holds no page; the calls write -1.
 *   ref   : [n_pages] int32, how many entries hold each page; a page with
 *           ref <= 0 is free.
 *   moves : [.][2] int32, (source page, destination page) pairs, and *n_moves,
 *           their number: what kda_cache_copy then carries out on a pool.  A
 *           source of -1 stands for zeros.
 * All of these are DEVICE arrays; entries out of range never make a kernel
 * access memory out of range.  The calls change only the arrays named as
 * written, in stream order, and can be captured into a graph and replayed.
 * Two calls that write the same table, ref or pool must be ordered by the
 * caller.  n_rows, width >= 1 and n_rows * width <= 2^26, else KDA_ERR_SHAPE.
 */

#define KDA_MAX_PAGES 65536       /* most pages of a pool */
#define KDA_MAX_FORKS 1024        /* most rows one kda_cache_fork call starts */
#define KDA_MAX_PAGED_SEQS 4096   /* most sequences of one call on pages that writes pages */

/*
 * Starts rows as copies of others (several samples of one prompt, a beam's
 * survivors) or anew.  For fork i, row children[i] of the table becomes a copy
 * of row parents[i] as it was before the call: each page in the parent's first
 * n_private entries is replaced by a free page, lowest first, and listed in
 * moves; the other pages are shared.  parents[i] = -1 starts an empty row: its
 * first n_private entries get free pages with a source of -1 in moves (zeros),
 * the others -1.  Every page's ref counts the entries that came to hold it.
 *
 *   table, ref       : as above                                   (updated in place)
 *   parents, children: [n] int32, 0 <= n <= KDA_MAX_FORKS         (read)
 *                      and n * width <= 2^26 (any n up to n_rows is)
 *   n_private        : 0 .. width, at most KDA_MAX_PAGES
 *   moves            : room for n * n_private pairs, n_moves: [1]  (written; what
 *                      moves holds past *n_moves is unspecified)
 *
 * Forks are served in order while free pages last: the first fork whose pages
 * are not there, and every later one, leaves its child's row as it was.  So
 * does a fork whose child's row holds a page (or lies out of range), whose
 * parent is neither -1 nor a row, or whose child an earlier fork names.
 */
kda_status kda_cache_fork(int* table, int* ref, const int* parents, const int* children, int* moves, int* n_moves,
                          int n, int n_private, int n_rows, int width, int n_pages, hipStream_t stream);

/*
 * Ends rows: each entry of the rows listed becomes -1 and its page's ref is
 * counted down (never below 0).  rows: [n] int32, n >= 0; a row out of range is
 * passed over, a row listed twice is freed once.  No page is touched.
 */
kda_status kda_cache_free(int* table, int* ref, const int* rows, int n, int n_rows, int width, int n_pages,
                          hipStream_t stream);

/*
 * Packs the pool: with n_live pages in use (ref > 0), each of them above n_live
 * moves to a free page below it, the lowest to the lowest, so that pages
 * [n_live, n_pages) are free and their memory can be handed back once
 * kda_cache_copy has carried out moves.
 *
 *   table, ref        : as above                                        (read)
 *   table_out, ref_out: the table and refs after the moves; each may be its input
 *                       (in place).  Entries that held a free page become -1.  Until
 *                       the moves run, and after, the old table's pages that moved
 *                       still hold their states.                        (written)
 *   moves             : room for n_pages / 2 pairs (at least one); n_moves, n_live: [1]
 *                       (written; moves past *n_moves is unspecified)
 */
kda_status kda_cache_compact(const int* table, const int* ref, int* table_out, int* ref_out, int* moves, int* n_moves,
                             int* n_live, int n_rows, int width, int n_pages, hipStream_t stream);

/*
 * Carries out the moves on every layer: page `destination` of dst becomes a copy
 * of page `source` of src, or zeros.  src and dst are pools of n_layers layers
 * with n_src_pages and n_dst_pages pages of page_bytes bytes (a multiple of 16)
 * each; they may be the same pool, or share no byte (KDA_ERR_ALIAS).
 *
 *   moves   : [max_moves][2] int32, 0 <= max_moves <= KDA_MAX_PAGES  (read)
 *   n_moves : [1] int32, clamped to [0, max_moves], or NULL for max_moves (read)
 *
 * The copies happen at once, in no order.  A move with a page out of range, or
 * onto its own source, is passed over, and so is every move that would race
 * with another one: two or more that name one destination, and in one pool a
 * move whose source is the destination of another one.  Lists written by
 * kda_cache_fork and kda_cache_compact hold no such move.
 */
kda_status kda_cache_copy(const void* src, void* dst, size_t page_bytes, int n_layers, int n_src_pages, int n_dst_pages,
                          const int* moves, const int* n_moves, int max_moves, hipStream_t stream);

/*
 * kda_decode_step on pages: one step of the recurrence for each of B sequences,
 * from the state on page pages_in[b] of the pool to page pages_out[b].
 *
 *   q, k, v, beta, o: as kda_decode_step
 *   alpha    : [B][H][d_k] fp32, or NULL with the gate inputs z ([B][H][d_k] in
 *              qkv_dtype) and A ([H] fp32) of kda_decode_step_gated; z and A are
 *              NULL when alpha is given (KDA_ERR_NULL when neither is)
 *   pool     : [n_pages][H][d_k][d_v] fp32                 (read and written)
 *   pages_in : [B] int32, DEVICE memory (read)
 *   pages_out: [B] int32, DEVICE memory (read), or NULL: each state is updated in
 *              place.  Another page keeps the state before the step as well (a
 *              fork without a copy of its own).
 *   B        : 1 .. KDA_MAX_PAGED_SEQS, n_pages: 1 .. KDA_MAX_PAGES;  B H <= 2^22
 *
 * A sequence with a page outside [0, n_pages) is passed over -- its row of o and
 * the pool are left as they were -- which is how a captured batch is padded; and
 * so is, rather than let them race, every sequence that reads or writes a page
 * that another sequence of the call (with both pages in range) writes.
 * Results equal kda_decode_step's on the same state bit for bit.
 */
kda_status kda_decode_step_paged(const void* q, const void* k, const void* v, kda_dtype qkv_dtype, const float* alpha,
                                 const void* z, const float* A, const float* beta, float* pool, int n_pages,
                                 const int* pages_in, const int* pages_out, void* o, kda_dtype o_dtype, int B, int H,
                                 int d_k, int d_v, hipStream_t stream);

/* ---- trees of drafted tokens ----------------------------------------------------------- */

/* Most nodes of one sequence's tree of drafted tokens. */
#define KDA_MAX_TREE 64

/*
 * kda_decode_verify for a tree of drafted tokens, over a cache of state pages:
 * node t of sequence b follows node parents[b][t], or the sequence's state when
 * that is -1, and its outputs are those of the recurrence run along its path
 * from the root.  The state is read once for the whole tree and not changed.
 *
 *   q, k   : [B][K][H][d_k] qkv_dtype     v: [B][K][H][d_v] qkv_dtype   (read)
 *   alpha  : [B][K][H][d_k] fp32          beta: [B][K][H] fp32          (read)
 *   pool   : [n_pages][H][d_k][d_v] fp32                                (read)
 *   pages  : [B] int32, DEVICE memory, the page of each sequence's state; NULL:
 *            page b (a dense [B][H][d_k][d_v] state; n_pages >= B)       (read)
 *   parents: [B][K] int32, DEVICE memory; -1 <= parents[b][t] < t, any other value
 *            is taken as -1                                             (read)
 *   n_nodes: [B] int32, DEVICE memory, the nodes of each tree, clamped to [0, K];
 *            NULL: K                                                    (read)
 *   o      : [B][K][H][d_v] o_dtype, o_t along the path to node t     (written)
 *   u      : [B][H][K][d_v] fp32, the write vectors kda_tree_commit needs (written)
 *   K      : 1 .. KDA_MAX_TREE;  n_pages: 1 .. KDA_MAX_PAGES;  B H <= 2^22 and
 *            K H max(d_k, d_v) < 2^30
 *
 * Rows of o and u behind a tree's last node, and every row of a sequence whose
 * page lies outside [0, n_pages), are left as they were.  o and u may overlap
 * nothing else (KDA_ERR_ALIAS).  All arithmetic is fp32; alpha may be any value
 * in [0, 1].
 */
kda_status kda_tree_verify(const void* q, const void* k, const void* v, kda_dtype qkv_dtype, const float* alpha,
                           const float* beta, const float* pool, int n_pages, const int* pages, const int* parents,
                           const int* n_nodes, void* o, kda_dtype o_dtype, float* u, int B, int K, int H, int d_k,
                           int d_v, hipStream_t stream);

/*
 * Commits the accepted path of each tree: page pages_out[b] receives the state
 * after the tokens on the path from the root to node last[b] (inclusive), from
 * the state on page pages_in[b], in one read and one write of it.
 *
 *   k, alpha, parents, n_nodes, u: the arguments and output of kda_tree_verify  (read)
 *   last     : [B] int32, DEVICE memory; a value outside [0, n_nodes[b]) accepts
 *              nothing (the state as it was)                             (read)
 *   pool, pages_in, pages_out, B: as kda_decode_step_paged, with its rules for pages
 *              out of range and shared pages; pages_in NULL: page b (n_pages >= B).  K: 1 ..
 *              KDA_MAX_TREE, B H <= 2^22
 */
kda_status kda_tree_commit(const void* k, kda_dtype qkv_dtype, const float* alpha, const float* u, const int* parents,
                           const int* n_nodes, const int* last, float* pool, int n_pages, const int* pages_in,
                           const int* pages_out, int B, int K, int H, int d_k, int d_v, hipStream_t stream);

/* ---- attention layers beside the recurrent ones ----------------------------------------
 *
 * A hybrid model has an attention layer after every few recurrent ones; these calls serve layers of plain
 * grouped heads (keys and values of each head are cached, no latent form of them).  Query head h
 * attends with the keys and values of head h / (H_q / H_kv) (grouped heads; H_q a multiple
 * of H_kv), and its output is
 *     o = sum_j p_j v_j,    p = softmax over the j it sees of  scale * q . k_j.
 * Maximum, sum and outputs are carried in fp32, for values below 1e30.  A query that sees
 * nothing (or only scores of minus infinity) gives zeros.  What a query does not see has no
 * influence on it, whatever it holds: infinities and NaN too.  An infinity or NaN in a value
 * that it does see makes that channel of its output NaN or infinite.
 *
 * Keys and values of earlier tokens lie in a pool of pages, page_tokens tokens of one layer
 * each, named by page tables like those of kda_cache_fork: entry j of a sequence's row is the
 * page of its tokens [j * page_tokens, (j + 1) * page_tokens).  kda_cache_fork with
 * n_private = 0 shares a prefix's pages (the one that is still being filled is then copied
 * with kda_cache_copy, whose page_bytes are these); kda_cache_free and kda_cache_compact
 * serve these tables as they serve those of states.  A page:
 *     keys   [H_kv][page_tokens][d_k], then values [H_kv][page_tokens][d_v], in kv_dtype;
 *     KDA_E4M3: then scales [2][H_kv] fp32, of each head's keys, then of its values, and
 *     zeros or anything up to a multiple of 16 bytes: what a code stands for is code * scale.
 * Arguments of the calls on pages:
 *   pool       : [n_pages][page_bytes] (kda_kv_page_bytes), 1 <= n_pages <= KDA_MAX_PAGES
 *   kv_dtype   : KDA_BF16 or KDA_E4M3
 *   page_tokens: 16, 32, 64 or 128
 *   table      : [n_rows][width] int32, DEVICE memory, n_rows * width <= 2^26 and
 *                width * page_tokens < 2^31 (KDA_ERR_SHAPE)
 *   rows       : [N] int32, DEVICE memory, the table row of each sequence of the call, or
 *                NULL: row b (N <= n_rows, KDA_ERR_SHAPE).  A row outside [0, n_rows) is padding.
 *   d_k, d_v   : 64 or 128 (KDA_ERR_UNSUPPORTED otherwise)
 * Lists in device memory that are wrong never make a kernel access memory out of range.
 * H_q, H_kv <= KDA_MAX_HEADS and tokens of a call <= KDA_MAX_CALL_TOKENS, else KDA_ERR_SHAPE.
 * No call of the library has a backward pass.
 */

#define KDA_MAX_HEADS 4096           /* most heads of one call of an attention layer */
#define KDA_MAX_CALL_TOKENS 4194304  /* most tokens of one call of an attention layer */

/*
 * Causal attention over whole prompts, with packed sequences of different lengths.
 * Query i of a sequence with n_q queries and n_k keys sees the keys j <= i + n_k - n_q: with
 * n_k = n_q the causal mask of a prompt, with more keys that of a prompt behind a cached
 * prefix (kda_kv_read), with fewer the first queries see nothing.
 *
 *   q      : total_q rows of H_q heads of d_k values, dtype, q_stride apart      (read)
 *   k, v   : total_k rows of H_kv heads of d_k and d_v values                    (read)
 *            (strides in elements, multiples of 16 bytes: rows may be slices of a fused
 *            projection's rows; heads and values inside a row are dense)
 *   cu_seqlens   : [N + 1] int32, DEVICE memory: sequence b's queries are the rows
 *            [cu[b], cu[b + 1]), clamped to [0, total_q]; NULL: N sequences of total_q / N
 *            queries and total_k / N keys (both have to divide, KDA_ERR_SHAPE)
 *   cu_seqlens_k : the same for keys and values, clamped to [0, total_k]; NULL: cu_seqlens,
 *            total_k = total_q (KDA_ERR_SHAPE).  NULL when cu_seqlens is (KDA_ERR_NULL).
 *   o      : total_q rows of H_q heads of d_v values, o_dtype, o_stride apart (written; rows
 *            outside every sequence are left as they were)
 *   scale  : finite (KDA_ERR_SHAPE)
 *   d_k, d_v: 16, 32, 64 or 128.  N >= 1; total_q, total_k >= 0 (no queries: nothing is done);
 *            (total_q / 64 + N + 2) * H_q <= 2^22 (KDA_ERR_SHAPE)
 *
 * cu_seqlens may not decrease.  o may share no byte with another array
 * (KDA_ERR_ALIAS).  fp32 inputs are multiplied in fp32; bf16 inputs on the bf16 matrix
 * cores with fp32 accumulation, the probabilities rounded to bf16, where d_k and d_v are each
 * 64 or 128 (and k_stride and v_stride below 2^24), and else in fp32 too.
 */
kda_status kda_attn_fwd(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                        long long v_stride, kda_dtype dtype, float scale, const int* cu_seqlens,
                        const int* cu_seqlens_k, int N, int total_q, int total_k, void* o, long long o_stride,
                        kda_dtype o_dtype, int H_q, int H_kv, int d_k, int d_v, hipStream_t stream);

/* Bytes of a page of keys and values, to *bytes.  Host only. */
kda_status kda_kv_page_bytes(kda_dtype kv_dtype, int page_tokens, int H_kv, int d_k, int d_v, size_t* bytes);

/*
 * Puts new tokens' keys and values on the pages of their sequences, the keys (and queries, where
 * given) turned by position on the way as kda_qk_norm does it:
 *     (a, b) -> (a cos f - b sin f, b cos f + a sin f),  f = pos * inv_freq[i].
 *
 *   k, v, q   : `total` rows of H_kv, H_kv and H_q heads, dtype, as kda_attn_fwd's    (read)
 *               (q NULL: no queries, q_out NULL, H_q is not looked at)
 *   cu_seqlens: [N + 1] int32, DEVICE memory, the new tokens of each sequence, clamped to
 *               [0, total]; it may not decrease.  NULL: one token a sequence, total = N (KDA_ERR_SHAPE)
 *   lens      : [N] int32, DEVICE memory, the tokens that each sequence has on its pages (below
 *               0: taken as 0).  Token i of sequence b goes to place lens[b] + i of its row.  (read)
 *   positions : [total] int32 positions for the rotation, or NULL: the token's place
 *   inv_freq  : [rot / 2] fp32;  rot: a multiple of 16 in [0, d_k]  (0: nothing is turned)
 *   q_out, k_out: the turned queries and keys as dense rows of `dtype`, with strides; k_out may be
 *               NULL.  q_out may be q itself with the same stride, and so may k_out be k.
 *               Rows outside every sequence are left as they were.     (written)
 *   pool      : the pages' entries for the new tokens                  (written)
 *   N         : 1 .. KDA_MAX_PAGED_SEQS
 *
 * Cosines and sines are formed in fp64, everything else is fp32; what goes to a bf16 page, q_out or k_out is
 * rounded once.  KDA_E4M3: each head's keys (values) on a page have the scale s, the smallest power
 * of two >= 2^-100 that brings the largest finite of them to 448 or below; codes are y / s rounded
 * to nearest even, values that are not finite become NaN.  A page that holds earlier tokens of the
 * sequence (its place in the row before lens[b]) keeps its scale, or, where the new tokens need a
 * larger one, has their codes rounded to that one -- exact, but for values below 2^-13 of the largest.
 * Tokens that are taken back (a smaller lens in the next call, as after rejected drafts) leave the scale and
 * that rounding behind on a page that still holds others.
 *
 * A token without a page (padding, an entry outside [0, n_pages), a place behind the row's end) is not
 * stored; its rows of q_out and k_out are written all the same.  Nor is, rather than let them
 * race, any token whose page another sequence's new tokens go to, or another place of its own row.
 */
kda_status kda_kv_append(const void* k, long long k_stride, const void* v, long long v_stride, const void* q,
                         long long q_stride, kda_dtype dtype, const int* positions, const float* inv_freq, int rot,
                         kda_pairing pairing, void* q_out, long long q_out_stride, void* k_out,
                         long long k_out_stride, void* pool, kda_dtype kv_dtype, int n_pages, int page_tokens,
                         const int* table, int n_rows, int width, const int* rows, const int* lens,
                         const int* cu_seqlens, int N, int total, int H_q, int H_kv, int d_k, int d_v,
                         hipStream_t stream);

/*
 * Cached keys and values back as dense rows: k_out [total][H_kv][d_k], v_out [total][H_kv][d_v], out_dtype
 * (bf16: exact).  Rows [cu[b], cu[b + 1]) are sequence b's tokens from place starts[b] on
 * (starts [N] int32, DEVICE memory; NULL or below 0: from 0 on).  A token without a page leaves its rows as they
 * were.  cu_seqlens as above, not NULL.  N: 1 .. KDA_MAX_PAGED_SEQS.
 */
kda_status kda_kv_read(const void* pool, kda_dtype kv_dtype, int n_pages, int page_tokens, const int* table, int n_rows,
                       int width, const int* rows, const int* starts, const int* cu_seqlens, void* k_out, void* v_out,
                       kda_dtype out_dtype, int N, int total, int H_kv, int d_k, int d_v, hipStream_t stream);

/*
 * Attention of the last K tokens of each sequence over its pages: K = 1 is a decode step behind
 * kda_kv_append, K > 1 a chain of drafted tokens, all of them appended.  Token t of sequence b sees its
 * first lens[b] - K + 1 + t tokens.
 *
 *   q   : [B][K][H_q][d_k] q_dtype (KDA_F32 or KDA_BF16)                    (read)
 *   pool: as above                                                        (read)
 *   lens: [B] int32, DEVICE memory, the tokens on each sequence's pages, these K among them;
 *         clamped to [0, width * page_tokens].  Tokens on a page out of range are not seen.   (read)
 *   o   : [B][K][H_q][d_v] o_dtype (written; the rows of padding are left as they were)
 *   workspace: device memory of workspace_bytes bytes (kda_attn_decode_plan), 16-byte aligned;
 *         its contents on entry do not matter.  NULL when the plan says 0.  Calls that may run
 *         at the same time need one each.                                   (written)
 *   B: 1 .. KDA_MAX_PAGED_SEQS, K: 1 .. KDA_MAX_ATTN_TOKENS, B * K * H_q <= 2^22,
 *   width * page_tokens <= 2^31 - 512 and B * (width * page_tokens / 128, rounded up) < 2^31
 *   (KDA_ERR_SHAPE).  The cache is read once for every 16 rows of queries that share a head
 *   (there are K * H_q / H_kv of them).
 *
 * fp32 queries are multiplied as three bf16 terms, and so are their probabilities: results
 * are fp32's.  With bf16 queries the probabilities are two bf16 terms (16 bits).  Errors: KDA_ERR_NULL (workspace needed),
 * KDA_ERR_SHAPE (workspace_bytes too small), KDA_ERR_ALIAS (o or workspace overlaps another array).
 */
#define KDA_MAX_ATTN_TOKENS 16 /* most tokens of a sequence in one kda_attn_decode call */
kda_status kda_attn_decode_plan(kda_dtype kv_dtype, int page_tokens, int width, int B, int K, int H_q, int H_kv, int d_k,
                                int d_v, size_t* workspace_bytes);
kda_status kda_attn_decode(const void* q, kda_dtype q_dtype, float scale, const void* pool, kda_dtype kv_dtype, int n_pages,
                           int page_tokens, const int* table, int n_rows, int width, const int* rows, const int* lens,
                           void* o, kda_dtype o_dtype, void* workspace, size_t workspace_bytes, int B, int K, int H_q,
                           int H_kv, int d_k, int d_v, hipStream_t stream);

/* Human-readable text for a status code (static storage; never NULL). */
const char* kda_status_string(kda_status s);

/* The hipError_t of the last failed launch on the calling thread (0 if none). */
int kda_last_hip_error(void);

/* Library version, major * 10000 + minor * 100 + patch. */
int kda_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
