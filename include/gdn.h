/*
 * gdn.h -- C ABI of libgdn.so: the Gated DeltaNet (GDN) recurrent state update for decode and for
 * multi-token-prediction (MTP) speculative verify, on one GB300 (sm_103a).
 *
 * The operation (the gated delta rule behind FlashInfer's gated_delta_rule_mtp, which sglang PR #23273
 * "[GDN] Enable FlashInfer MTP verify on SM100+ (Blackwell)" calls through its pool API, Summary):
 * for every request lane b whose pool index slot = state_indices[b] is not -1, and every value head h
 * (key/query head hk = h / (HV / HK): each group of HV/HK consecutive value heads shares one key head),
 *
 *     S = state_pool[slot, h]                                   (DV x DK, computed in fp32)
 *     for t in 0 .. T-1:
 *         qh = q[b,t,hk] / sqrt(|q[b,t,hk]|^2 + l2_eps)         (L2 normalisation)
 *         kh = k[b,t,hk] / sqrt(|k[b,t,hk]|^2 + l2_eps)
 *         g    = exp(-exp(A_log[h]) * softplus(a[b,t,h] + dt_bias[h]))
 *         beta = sigmoid(b[b,t,h])
 *         S = g * S
 *         S = S + beta * (v[b,t,h] - S kh) kh^T                 (delta rule)
 *         o[b,t,h] = scale * S qh
 *
 * Layouts: row-major, last index contiguous, no strides.
 *     q, k                    [B, T, HK, DK]          qkv_dtype
 *     v                       [B, T, HV, DV]          qkv_dtype
 *     a, b                    [B, T, HV]              qkv_dtype
 *     A_log, dt_bias          [HV]                    fp32 (A_log is fp32: same page, Summary)
 *     state_pool              [num_slots, HV, DV, DK] state_dtype (fp32, or bf16 as with
 *                                                     --mamba-ssm-dtype bfloat16, same page, Throughput)
 *     state_indices           [B]                     int32; -1 = padded lane
 *     o                       [B, T, HV, DV]          out_dtype
 *     intermediate_states     [B, T, HV, DV, DK]      state_dtype
 *     accept_len              [B]                     int32
 *
 * Common rules.
 *   - Every pointer is DEVICE memory owned by the caller, on the device that is current when the call is made
 *     (the one `stream` belongs to).  The library allocates nothing, keeps no state between calls besides
 *     launch-configuration caches (atomic, one entry per device, filled on first use), never synchronises,
 *     and enqueues its work asynchronously on `stream` (0 = legacy default stream).  Calls are thread-safe.
 *     A call with B == 0 (prefill: or no tokens; gated norm: rows == 0) enqueues nothing and returns GDN_OK.
 *   - Alignment: q, k, state_pool and intermediate_states start on 16 bytes; the other arrays on their
 *     element size.  Outputs must not overlap inputs (decode updates state_pool in place by design).
 *   - Errors the host can see are returned as a status before anything is enqueued.  Errors that depend on
 *     device data are defined, never a fault: a lane whose index is < -1 or >= num_slots, (commit) whose
 *     accept length is outside 0..T, or (prefill) whose token bounds are negative, decreasing or beyond the
 *     token count, is skipped and a bit is OR-ed into *err_word (if err_word is not NULL):
 *     GDN_ERRBIT_INDEX, GDN_ERRBIT_ACCEPT_LEN, GDN_ERRBIT_SEQLEN.  No kernel waits on another CTA or on a
 *     flag; the only waits are on the CTA's own bulk copies of state into shared memory, and they are
 *     bounded: one that runs out sets GDN_ERRBIT_TIMEOUT and that part of the state is left unprocessed.
 *     The caller zeroes *err_word and reads it when it wants.
 *   - Padded lanes (index -1, the padding index guard of FlashInfer #2810, same page, Requirements) are
 *     skipped: their o, intermediate states and pool slots are left untouched, bit for bit.
 *   - Distinct active lanes must use distinct slots in gdn_decode and gdn_commit (they write the pool);
 *     gdn_mtp_verify only reads the pool, so lanes may share a slot there.
 *   - GDN_ERR_CUDA: the launch failed; gdn_last_cuda_error() returns the cudaError_t of this thread's last
 *     failed launch.
 */
#ifndef GDN_H_
#define GDN_H_

#include <stdint.h>

/* The library exports these functions and nothing else (it is built with hidden default visibility). */
#if defined(__GNUC__)
#define GDN_API __attribute__((visibility("default")))
#else
#define GDN_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; declared here so that C callers need no CUDA header. */
typedef struct CUstream_st* gdn_stream_t;

typedef enum gdn_status {
    GDN_OK = 0,
    GDN_ERR_NULL = 1,        /* a required pointer is NULL */
    GDN_ERR_SHAPE = 2,       /* a size is out of range or inconsistent (HV % HK, T range, ...) */
    GDN_ERR_DTYPE = 3,       /* a dtype code is not a gdn_dtype */
    GDN_ERR_ALIGN = 4,       /* a pointer is misaligned */
    GDN_ERR_UNSUPPORTED = 5, /* a valid but unsupported configuration (DK not in {16,32,64,128,256}; D not in {64,128,256}) */
    GDN_ERR_CUDA = 6,        /* the kernel launch failed */
    GDN_ERR_VALUE = 7        /* a scalar is not finite, an epsilon < 0, or a cache scale no power of two */
} gdn_status;

typedef enum gdn_dtype { GDN_F32 = 0, GDN_BF16 = 1 } gdn_dtype;

enum { GDN_ERRBIT_INDEX = 1, GDN_ERRBIT_ACCEPT_LEN = 2, GDN_ERRBIT_TIMEOUT = 4, GDN_ERRBIT_SEQLEN = 8,
       GDN_ERRBIT_PAGES = 16, GDN_ERRBIT_NONFINITE = 32 };

enum { GDN_MAX_T = 16 }; /* tokens per call: decode (T >= 1), verify up to 16 (the page's MTP beyond T > 4) */

typedef struct gdn_dims {
    int32_t B;           /* request lanes, 0 .. 65535 */
    int32_t T;           /* tokens per lane, 1 .. GDN_MAX_T */
    int32_t HK;          /* query/key heads, >= 1 */
    int32_t HV;          /* value heads, multiple of HK, <= 65535 */
    int32_t DK;          /* key dimension: 16, 32, 64, 128 or 256 */
    int32_t DV;          /* value dimension (state rows), >= 1 */
    int32_t num_slots;   /* pool slots, >= 1 */
    int32_t qkv_dtype;   /* gdn_dtype of q, k, v, a, b */
    int32_t state_dtype; /* gdn_dtype of state_pool and intermediate_states */
    int32_t out_dtype;   /* gdn_dtype of o */
    float scale;         /* multiplies o (1.0 for o = S q) */
    float l2_eps;        /* added to |x|^2 inside the square root of the L2 normalisation (1e-6) */
} gdn_dims;

/*
 * gdn_decode -- T tokens (normally T = 1) from state_pool[state_indices[b]]; the final state is written
 * back into the same slot, rounded to state_dtype (round to nearest even for bf16).  The running state
 * stays fp32 between the tokens of one call.  Defines the SM100+ decode path of sglang PR #23273,
 * Summary, with the padding index guard of its Requirements.
 */
GDN_API gdn_status gdn_decode(const gdn_dims* dims, const void* q, const void* k, const void* v, const void* a,
                      const void* b, const float* A_log, const float* dt_bias, void* state_pool,
                      const int32_t* state_indices, void* o, int32_t* err_word, gdn_stream_t stream);

/*
 * gdn_mtp_verify -- T draft tokens from state_pool[state_indices[b]] (read only: the pool is never
 * written).  If intermediate_states is not NULL, the state after token t is stored, rounded to
 * state_dtype, in intermediate_states[b, t].  Without intermediate_states, bf16 state, T <= 8 and DK >= 64,
 * the outputs come from the chunked form of the same recurrence (S_0 [k q] on the tensor cores, k and q split
 * into bf16 hi + lo parts, about 16 significant bits), within fp32-level error of the token-by-token
 * outputs.  MTP verify through the pool API (initial_state_indices) of sglang PR #23273, Summary; bf16
 * state, T beyond 4 and intermediate caching from its Requirements (FlashInfer #2679).
 */
GDN_API gdn_status gdn_mtp_verify(const gdn_dims* dims, const void* q, const void* k, const void* v, const void* a,
                          const void* b, const float* A_log, const float* dt_bias, const void* state_pool,
                          const int32_t* state_indices, void* o, void* intermediate_states,
                          int32_t* err_word, gdn_stream_t stream);

/*
 * gdn_commit -- state_pool[state_indices[b], :] = intermediate_states[b, accept_len[b] - 1, :] (all heads),
 * bit for bit, for every active lane with accept_len[b] >= 1; accept_len 0 leaves the slot as it is.
 * Uses dims->B, T, HV, DK, DV, num_slots and state_dtype only.  The accepted-prefix checkpoint write of
 * the commit contract in TensorRT-LLM PR #20937 (GB300 Qwen3.8-Flash-Next NVFP4), "Moved out of this PR"
 * (the manager's all-layer commit) and its commit message, MTP > Verify (checkpoint-commit contract).
 */
GDN_API gdn_status gdn_commit(const gdn_dims* dims, void* state_pool, const int32_t* state_indices,
                      const void* intermediate_states, const int32_t* accept_len, int32_t* err_word,
                      gdn_stream_t stream);

/*
 * gdn_commit_replay -- the same pool update as gdn_commit, without intermediate states: for every active
 * lane with accept_len[b] >= 1, the first accept_len[b] tokens are run again from state_pool[slot] (which
 * gdn_mtp_verify left unchanged) and the final state is written back into that slot, rounded to
 * state_dtype.  fp32 state, or T > 8: the token-by-token arithmetic of gdn_mtp_verify, so the slot receives
 * exactly the bits gdn_commit would copy from intermediate_states[b, accept_len[b] - 1].  bf16 state with
 * T <= 8: the same state in chunked form (S_L = gamma S_0 + a sum of rank-1 terms, S_0 k on the tensor
 * cores with k split into bf16 hi + lo parts), within fp32-level error of that copy before the final bf16
 * rounding, so the two may differ in the last bf16 bit.  q, k, v, a, b, A_log, dt_bias, scale and l2_eps
 * must be those the verify call used; no outputs are written; accept_len 0 leaves the slot as it is,
 * lengths outside 0..T set GDN_ERRBIT_ACCEPT_LEN.  Verify then moves 1 state instead of 1 + T, at the cost
 * of reading each state once more here: the cached replay with in-kernel commit of TensorRT-LLM PR #20937
 * (GB300 Qwen3.8-Flash-Next NVFP4), "MTP > Verify" and "Moved out of this PR".
 */
GDN_API gdn_status gdn_commit_replay(const gdn_dims* dims, const void* q, const void* k, const void* v, const void* a,
                             const void* b, const float* A_log, const float* dt_bias, void* state_pool,
                             const int32_t* state_indices, const int32_t* accept_len, int32_t* err_word,
                             gdn_stream_t stream);

/* The gated RMSNorm applied to a verify's outputs (gdn_mtp_verify_gated, gdn_mtp_verify_commit): exactly
 * gdn_gated_rmsnorm of the o the call stores,
 *     y[b,t,h,i] = o[b,t,h,i] / sqrt(mean_i(o[b,t,h,:]^2) + eps) * norm_weight[i] * silu(z[b,t,h,i]),
 * computed in fp32 and stored in out_dtype; rows of padded lanes are left untouched.  Device memory. */
typedef struct gdn_gated_norm_out {
    const void* z;             /* [B, T, HV, DV] z_dtype: the gate projection */
    int32_t z_dtype;           /* gdn_dtype of z */
    const float* norm_weight;  /* [DV] fp32 */
    float eps;                 /* finite, >= 0 */
    void* y;                   /* [B, T, HV, DV] out_dtype; may be o itself (then o is replaced by y) */
} gdn_gated_norm_out;

/*
 * gdn_mtp_verify_gated -- gdn_mtp_verify (o and, if given, intermediate_states, as that call writes them)
 * followed by the gated RMSNorm of o into norm->y.  Where the verify runs on the chunked kernel (a bf16 pool
 * without intermediate states, T <= 8, DK >= 64), the norm runs inside it while DV <= 128 and the batch leaves
 * each of its item pipelines one item at most, else gdn_gated_rmsnorm runs after it.  Elsewhere the token-by-token
 * kernels apply it in the same launch: the CTAs that share a head run as one thread-block cluster (at most 8, i.e.
 * DV <= 256, or DV <= 1024 where one CTA holds 128 rows) and meet their sums of squares in distributed shared
 * memory.  A wider head, or a grid of more CTAs than the GPU holds at once (where the two launches measured faster),
 * gets the norm's own launch.  The decode-rows gated norm of TensorRT-LLM PR #20937 (GB300
 * Qwen3.8-Flash-Next NVFP4), Per-File QA Perspective, Source files, fused into the recurrence's output.
 */
GDN_API gdn_status gdn_mtp_verify_gated(const gdn_dims* dims, const void* q, const void* k, const void* v,
                                        const void* a, const void* b, const float* A_log, const float* dt_bias,
                                        const void* state_pool, const int32_t* state_indices, void* o,
                                        void* intermediate_states, const gdn_gated_norm_out* norm, int32_t* err_word,
                                        gdn_stream_t stream);

/*
 * gdn_decode_gated -- gdn_decode (the outputs and the write-back as that call stores them) with the gated RMSNorm of
 * o into norm->y, in the same launch where the head's CTAs fit one cluster and the grid one wave (as in
 * gdn_mtp_verify_gated above), else followed by the norm's own launch.  The decode-rows gated norm of TensorRT-LLM PR #20937, Per-File QA
 * Perspective, Source files (gdn_decode_rows_gated_norm).  Arguments, errors and ownership as gdn_decode and
 * gdn_gated_norm_out.
 */
GDN_API gdn_status gdn_decode_gated(const gdn_dims* dims, const void* q, const void* k, const void* v, const void* a,
                                    const void* b, const float* A_log, const float* dt_bias, void* state_pool,
                                    const int32_t* state_indices, void* o, const gdn_gated_norm_out* norm,
                                    int32_t* err_word, gdn_stream_t stream);

/* The tokens of an earlier gdn_mtp_verify call on the same lanes, whose accepted prefix gdn_mtp_verify_commit
 * commits before it verifies: the compact recovery record of a speculative step (its k, v, a, b and accept
 * lengths; q is not needed, the replay writes no outputs).  All device memory, layouts as in the header. */
typedef struct gdn_replay_tokens {
    int32_t T;                 /* tokens per lane of that call, 1 .. GDN_MAX_T */
    const void* k;             /* [B, T, HK, DK] qkv_dtype, 16-byte aligned */
    const void* v;             /* [B, T, HV, DV] qkv_dtype */
    const void* a;             /* [B, T, HV] qkv_dtype */
    const void* b;             /* [B, T, HV] qkv_dtype */
    const int32_t* accept_len; /* [B] int32: lane b commits its first accept_len[b] tokens (0: none) */
} gdn_replay_tokens;

/*
 * gdn_mtp_verify_commit -- one speculative step in one pass over the state pool: for every active lane, first
 * the commit of the earlier call's accepted prefix, exactly gdn_commit_replay(prev) (the state after
 * prev->accept_len[b] of prev's tokens written into state_pool[slot], rounded to state_dtype), then verify of
 * this call's T tokens from the slot as just written, exactly gdn_mtp_verify without intermediate states (o).
 * dims describes this call (dims->T tokens); prev->T may differ from it (the draft width may change between
 * steps).  With a bf16 pool, both token counts <= 4 and DK >= 64, one kernel reads each state once and writes it
 * once; otherwise the two calls run back to back (with more tokens they measured faster as two launches).  With
 * norm != NULL, the verify is gdn_mtp_verify_gated's (o and the gated norm into norm->y).  An accept length outside 0 .. prev->T sets
 * GDN_ERRBIT_ACCEPT_LEN and commits nothing for that lane (its verify still runs from the slot as it is).  The
 * in-kernel commit of TensorRT-LLM PR #20937 (GB300 Qwen3.8-Flash-Next NVFP4), "Moved out of this PR" (commits
 * in-kernel below 16 decode requests), fed by the compact GDN recovery records of the issue "Proposal: native
 * BF16 MTP speculative decoding for dense Qwen3.8-27B".
 */
GDN_API gdn_status gdn_mtp_verify_commit(const gdn_dims* dims, const gdn_replay_tokens* prev, const void* q,
                                         const void* k, const void* v, const void* a, const void* b,
                                         const float* A_log, const float* dt_bias, void* state_pool,
                                         const int32_t* state_indices, void* o, const gdn_gated_norm_out* norm,
                                         int32_t* err_word, gdn_stream_t stream);

/*
 * gdn_prefill -- prefill of B variable-length sequences packed along one token axis of N = dims->T tokens
 * (here T is the total token count, 0 .. 2^31 - 1, not bounded by GDN_MAX_T):
 *     q, k  [N, HK, DK]   v, o  [N, HV, DV]   a, b  [N, HV]   (qkv_dtype; o in out_dtype)
 *     cu_seqlens          [B + 1] int32, device: sequence b is tokens cu_seqlens[b] .. cu_seqlens[b+1]-1
 *     has_initial_state   [B] int32, device, nullable (NULL: every sequence has one)
 * Sequence b with slot = state_indices[b] != -1 starts from state_pool[slot, h] if has_initial_state[b]
 * is non-zero, else from the zero state (the slot is then not read: a fresh slot may hold anything), runs
 * its tokens with the recurrence above, writes o at their positions and the final state into
 * state_pool[slot, h], rounded to state_dtype once (the running state stays fp32).  An empty sequence
 * leaves its slot as it is.  Sequences must not overlap (their outputs would race); they may leave gaps
 * between them (o is not written there).  Bounds that are negative,
 * decreasing or beyond N skip the sequence and set GDN_ERRBIT_SEQLEN; a bad index sets GDN_ERRBIT_INDEX
 * (checked first).  Distinct active sequences must use distinct slots.  The chunked gated delta rule with
 * bf16 state pools and an initial-state mask ("fresh-state zeroing") of TensorRT-LLM PR #20937 (GB300
 * Qwen3.8-Flash-Next NVFP4), Per-File QA Perspective, Source files and Test-code files.  Alignment: q, k,
 * state_pool on 16 bytes, the rest on their element size.
 */
GDN_API gdn_status gdn_prefill(const gdn_dims* dims, const int32_t* cu_seqlens, const void* q, const void* k,
                               const void* v, const void* a, const void* b, const float* A_log,
                               const float* dt_bias, void* state_pool, const int32_t* state_indices,
                               const int32_t* has_initial_state, void* o, int32_t* err_word, gdn_stream_t stream);

/*
 * gdn_gated_rmsnorm -- gated RMSNorm of `rows` rows of DV outputs (one value head of one token per row):
 *     y[r, i] = o[r, i] / sqrt(mean_i(o[r, i]^2) + eps) * norm_weight[i] * silu(z[r, i]),
 *     silu(x) = x * sigmoid(x),
 * in fp32, y stored in o_dtype (round to nearest even for bf16).  o, y [rows, DV] o_dtype; z [rows, DV]
 * z_dtype (the gate projection); norm_weight [DV] fp32; all device memory.  y may be o itself (in place),
 * no other overlap.  rows == 0 enqueues nothing.  The decode-rows gated norm of TensorRT-LLM PR #20937,
 * Per-File QA Perspective, Source files (the page gives no formula: RMS over the value dimension, one
 * weight per column shared by all heads, SiLU gate after the norm, is the reading taken).  eps must be
 * finite and >= 0 (GDN_ERR_VALUE); o, z, y, norm_weight aligned to their element size.
 */
GDN_API gdn_status gdn_gated_rmsnorm(int64_t rows, int32_t DV, int32_t o_dtype, int32_t z_dtype, const void* o,
                                     const void* z, const float* norm_weight, float eps, void* y,
                                     gdn_stream_t stream);

/*
 * The in_proj projection of the decode / verify rows with its causal conv1d epilogue: TensorRT-LLM PR #20937
 * (GB300 Qwen3.8-Flash-Next NVFP4), What changes, Decode at small batch ("the in_proj GEMV with a fused conv1d
 * epilogue, for 2..16 verify rows and up to 8 decode rows").  The page gives no formula; the reading taken:
 *
 *   W [C, H] bf16 holds the C = 2*HK*DK + 2*HV*DV + 2*HV output channels in the order
 *     q (HK*DK) | k (HK*DK) | v (HV*DV) | z (HV*DV) | b (HV) | a (HV);
 *   the first Cc = 2*HK*DK + HV*DV channels (q, k, v) pass through a K-tap causal depthwise convolution whose
 *   state is the K-1 previous inputs of each channel, per pool slot:
 *     conv_state [num_slots, K-1, Cc] conv_dtype (oldest first),
 *   For lane b (rows b*T .. b*T+T-1 of x [B*T, H] bf16) with slot = state_indices[b] != -1, channel c, row t:
 *     p[t, c] = sum_h W[c, h] x[b*T + t, h]                      (fp32 accumulation)
 *     u[t, c] = p[t, c] rounded to conv_dtype                    (c < Cc: the value the state stores)
 *     seq     = conv_state[slot, 0 .. K-2, c], u[0 .. T-1, c]
 *     y[t, c] = conv_b[c] + sum_{j < K} conv_w[c, j] seq[t + j, c], then y * sigmoid(y) if dims->silu
 *   q, k [B, T, HK, DK], v [B, T, HV, DV] <- y of their channels; z [B, T, HV, DV], b, a [B, T, HV] <- p of theirs
 *   (all out_dtype).
 */
typedef struct gdn_conv_dims {
    int32_t B;          /* request lanes, 0 .. 65535 */
    int32_t T;          /* rows per lane, 1 .. GDN_MAX_T */
    int32_t H;          /* hidden size: a multiple of 8, 8 .. 65536 */
    int32_t HK;         /* query/key heads of the outputs, >= 1 */
    int32_t HV;         /* value heads, a multiple of HK */
    int32_t DK;         /* key dimension, >= 1 */
    int32_t DV;         /* value dimension, >= 1 */
    int32_t K;          /* convolution taps, 2 .. 4 */
    int32_t num_slots;  /* convolution-state slots, >= 1 */
    int32_t conv_dtype; /* gdn_dtype of conv_state and of the recovery records */
    int32_t out_dtype;  /* gdn_dtype of q, k, v, z, b, a */
    int32_t silu;       /* 1: SiLU after the convolution, 0: none */
} gdn_conv_dims;

/* Outputs of gdn_in_proj_conv: the inputs of gdn_decode / gdn_mtp_verify (q, k, v, a, b) and of the gated norm
 * (z); device memory, out_dtype, element-aligned, no overlap with anything else. */
typedef struct gdn_in_proj_out {
    void* q; /* [B, T, HK, DK] */
    void* k; /* [B, T, HK, DK] */
    void* v; /* [B, T, HV, DV] */
    void* z; /* [B, T, HV, DV] */
    void* b; /* [B, T, HV] */
    void* a; /* [B, T, HV] */
} gdn_in_proj_out;

/*
 * gdn_in_proj_conv -- the projection and convolution above for every lane whose index is not -1.
 * write_state = 1 (decode rows): conv_state[slot, j, c] = seq[T + j, c] for j < K-1 (the last K-1 entries).
 * write_state = 0 (verify rows): conv_state is only read; if records is not NULL it receives u:
 *     records [B, T, Cc] conv_dtype, the verify rows' recovery records for gdn_conv_commit.
 * conv_w [Cc, K] fp32, conv_b [Cc] fp32 or NULL (zero).  x and W start on 16 bytes; the rest on their element
 * size.  Lanes with index -1 are skipped (outputs, records and slot untouched); an index < -1 or >= num_slots
 * skips the lane and sets GDN_ERRBIT_INDEX.  Distinct active lanes must use distinct slots when write_state = 1.
 * The waits of the kernel on its own copies are bounded (GDN_ERRBIT_TIMEOUT, outputs of the tile left unwritten).
 */
GDN_API gdn_status gdn_in_proj_conv(const gdn_conv_dims* dims, const void* x, const void* W, const float* conv_w,
                                    const float* conv_b, void* conv_state, const int32_t* state_indices,
                                    int32_t write_state, const gdn_in_proj_out* out, void* records,
                                    int32_t* err_word, gdn_stream_t stream);

/*
 * gdn_conv_commit -- the convolution state after each lane's first L = accept_len[b] verify rows: with seq =
 * conv_state[slot, 0 .. K-2, c], records[b, 0 .. T-1, c], conv_state[slot, j, c] = seq[L + j, c] (bit copies).
 * L = 0 leaves the slot; L outside 0 .. T sets GDN_ERRBIT_ACCEPT_LEN, a bad index GDN_ERRBIT_INDEX (the lane is
 * skipped).  The commit of the convolution state with the accepted prefix (issue "Proposal: native BF16 MTP
 * speculative decoding for dense Qwen3.8-27B", What: the compact GDN recovery records and their commit).  Only
 * dims->B, T, HK, HV, DK, DV, K, num_slots and conv_dtype are read.
 */
GDN_API gdn_status gdn_conv_commit(const gdn_conv_dims* dims, void* conv_state, const int32_t* state_indices,
                                   const void* records, const int32_t* accept_len, int32_t* err_word,
                                   gdn_stream_t stream);

/*
 * The softmax-attention layers that a hybrid model runs between its Gated DeltaNet layers, over a paged 4-bit K/V cache
 * (the NVFP4 K/V cache of TensorRT-LLM PR #20937, GB300 Qwen3.8-Flash-Next NVFP4).  One step of such a layer:
 *     gdn_page_plan (once a step)  ->  gdn_qk_norm_rope with the cache  ->  gdn_kv4_attention
 * and gdn_kv4_read gives cached rows back as numbers.  The common rules above hold; a token whose slot is -1 is skipped.
 *
 * The cache of one layer: page_size tokens a page, keys (0) and values (1) of every key head,
 *     codes   [num_pages, 2, HK, page_size, D / 2]   bytes: dimensions 2j (lower half) and 2j + 1 of byte j, e2m1
 *     scales  [num_pages, 2, HK, page_size, D / 16]  bytes: one e4m3 scale for each 16 dimensions
 * and a number is code * scale * k_scale (v_scale).  A token's slot is page * page_size + its place in the page.
 */
typedef struct gdn_kv4_cache {
    void* codes;       /* 16-byte aligned */
    void* scales;      /* 16-byte aligned */
    int32_t num_pages; /* >= 1; num_pages * page_size < 2^31 */
    int32_t page_size; /* 16, 32, 64, 128 or 256 */
    int32_t HK;        /* key heads, 1 .. 1024 */
    int32_t D;         /* head dimension: 64, 128 or 256 */
    float k_scale;     /* a power of two, 2^-32 .. 2^32 (1.0) */
    float v_scale;
} gdn_kv4_cache;

/* What gdn_page_plan writes; device memory, int32. */
typedef struct gdn_page_plan_out {
    int32_t* cu_seqlens; /* [B + 1]: lane b's tokens are cu_seqlens[b] .. cu_seqlens[b + 1] - 1 of the step's */
    int32_t* positions;  /* [N]: 0 beyond the step's tokens */
    int32_t* slot_map;   /* [N]: -1 beyond them, and for lanes without pages */
    int32_t* total_lens; /* [B]: kv_lens + new_lens; kv_lens where the lane got no pages */
    int32_t* held;       /* [B]: pages of each lane after the step; may be the input */
    int32_t* taken;      /* [1]: pages taken from the free list after the step; may be the input */
} gdn_page_plan_out;

/*
 * gdn_page_plan -- block tables, slot map, positions and offsets of a step's tokens, from the lanes' lengths.
 *     need_b = max(0, ceil((kv_lens[b] + new_lens[b]) / page_size) - held[b]),  upto_b = need_0 + .. + need_b
 * Lane b gets pages free_pages[taken + upto_b - need_b ..] into block_tables[b, held[b] ..] while taken + upto_b <=
 * num_pages (a lane that needs none always goes on); the others keep their tables, their tokens get slot -1 and
 * GDN_ERRBIT_PAGES is set.  held may be more than the cached tokens fill (pages of rejected drafts).  A lane whose lengths
 * are negative, beyond max_pages pages or (cached) beyond its held pages is skipped likewise, with GDN_ERRBIT_SEQLEN; a
 * step of more than N tokens sets that bit too, and its tokens beyond N are not written.  A page outside
 * 0 .. num_pages - 1 gives slot -1 and GDN_ERRBIT_INDEX.  block_tables [B, max_pages], free_pages [num_pages].  ticket:
 * one int32, 0 before the first call and left 0, used by one call at a time.  B 0 .. 8192; with B 0 nothing is enqueued and
 * nothing written, so a caller that goes on to use the outputs of such a step sets them: cu_seqlens[0] = 0, slots -1.
 */
GDN_API gdn_status gdn_page_plan(int32_t B, int32_t N, int32_t page_size, int32_t max_pages, int32_t num_pages,
                                 const int32_t* kv_lens, const int32_t* new_lens, int32_t* block_tables,
                                 const int32_t* held, const int32_t* free_pages, const int32_t* taken,
                                 const gdn_page_plan_out* out, int32_t* ticket, int32_t* err_word,
                                 gdn_stream_t stream);

typedef struct gdn_qk_dims {
    int32_t N;           /* tokens */
    int32_t HQ;          /* query heads, 1 .. 1024 */
    int32_t HK;          /* key heads, 1 .. 1024 */
    int32_t D;           /* head dimension: 64, 128 or 256 */
    int32_t R;           /* rotated dimensions: the first R of D, a multiple of 16, 0 .. D */
    int32_t interleaved; /* pairs (2i, 2i + 1) if 1, (i, i + R / 2) if 0 */
    int32_t dtype;       /* gdn_dtype of q, k, v and of the outputs */
    int64_t q_stride;    /* elements from one token of q to the next: >= HQ * D, a multiple of 16 bytes */
    int64_t k_stride;    /* >= HK * D, likewise */
    int64_t v_stride;    /* >= HK * D, likewise */
    float eps;           /* finite, >= 0 */
} gdn_qk_dims;

/*
 * gdn_qk_norm_rope -- RMS norm of every query and key head and the position rotation, in one pass:
 *     y = x / sqrt(mean(x^2) + eps) * weight
 *     (y_a, y_b) = (y_a cos t - y_b sin t, y_b cos t + y_a sin t),  t = positions[n] * inv_freq[i]
 * q [N, HQ, D], k [N, HK, D] with their strides; q_weight, k_weight [D] fp32; positions [N] int32; inv_freq [R / 2] fp32
 * (read only if R > 0); q_out [N, HQ, D], k_out [N, HK, D] without gaps, which may be q and (without a cache) k themselves
 * where those have none.  With a cache, k (after norm and rotation, not rounded in between) and v [N, HK, D] are stored at slot_map[n]
 * ([N] int32; -1 stores nothing): for each 16 dimensions the scale e4m3(max|x| / 6 / k_scale), to nearest even and at
 * most 448, and the codes e2m1(x / (scale * k_scale)), to nearest even and at most 6.  The keys' codes are those of the
 * exact value whatever the rounding of the sums.  k_out may then be NULL.  NaN is stored as 0 and an infinity as the largest number,
 * and GDN_ERRBIT_NONFINITE is set; a slot below -1 or beyond the pages sets GDN_ERRBIT_INDEX and stores nothing.  Tokens of
 * one call have distinct slots.  v, slot_map and cache go together (all or none NULL).  All tensors on 16 bytes, positions
 * and slot_map on 4.
 */
GDN_API gdn_status gdn_qk_norm_rope(const gdn_qk_dims* dims, const void* q, const void* k, const float* q_weight,
                                    const float* k_weight, const int32_t* positions, const float* inv_freq,
                                    void* q_out, void* k_out, const void* v, const gdn_kv4_cache* cache,
                                    const int32_t* slot_map, int32_t* err_word, gdn_stream_t stream);

/* gdn_kv4_read -- the cached rows of N slots as bf16: k_out, v_out [N, HK, D] (exact while k_scale and v_scale leave the
 * numbers in bf16's range).  Rows of slot -1 stay as they are. */
GDN_API gdn_status gdn_kv4_read(const gdn_kv4_cache* cache, int32_t N, const int32_t* slot_map, void* k_out,
                                void* v_out, int32_t* err_word, gdn_stream_t stream);

typedef struct gdn_kv4_attention_dims {
    int32_t B;         /* lanes, 0 .. 65535 */
    int32_t N;         /* rows of q and o: tokens of all lanes; N * HQ < 2^31 */
    int32_t max_q;     /* most tokens of a lane, >= 1 */
    int32_t HQ;        /* query heads, a multiple of the cache's HK, HQ / HK <= 64 */
    int32_t max_pages; /* columns of block_tables, >= 1; max_pages * page_size < 2^31 */
    float scale;       /* multiplies q . k (1 / sqrt(D)) */
} gdn_kv4_attention_dims;

/*
 * gdn_kv4_attention -- causal attention of each lane's tokens over its cached pages: token t of lane b (of n_b) sees keys
 * 0 .. kv_lens[b] - n_b + t, its own key among them (the step's keys are stored before), query head h the key head
 * h / (HQ / HK).
 *     o = sum_j p_j v_j / sum_j p_j,  lse = log sum_j exp(scale q . k_j)
 * q, o [N, HQ, D] bf16 on 16 bytes; lse [N, HQ] fp32 or NULL; cu_seqlens [B + 1] or NULL (then N = B * max_q and lane b
 * holds rows b * max_q ..); kv_lens [B]: cached tokens, the step's included; block_tables [B, max_pages] (entries beyond a
 * lane's tokens are not read).  A token that sees no key gets o = 0 and lse = -inf.  A scale byte of NaN (no store writes one)
 * counts as 0 in the values, so that it does not reach tokens which do not see it; in the keys it makes NaN of the tokens
 * that see it.  Softmax statistics and sums are fp32.  Bounds that are negative, decreasing, longer than max_q or beyond N, and
 * a kv_len outside 0 .. max_pages * page_size, skip the lane (GDN_ERRBIT_SEQLEN; its rows stay as they are); the keys and
 * values of a page outside the cache count as zeros (GDN_ERRBIT_INDEX).  workspace: at least gdn_kv4_attention_workspace bytes
 * on 16 bytes, used by one call at a time; its contents need not be kept.
 */
GDN_API gdn_status gdn_kv4_attention(const gdn_kv4_attention_dims* dims, const gdn_kv4_cache* cache, const void* q,
                                     const int32_t* cu_seqlens, const int32_t* block_tables, const int32_t* kv_lens,
                                     void* o, float* lse, void* workspace, int64_t workspace_bytes, int32_t* err_word,
                                     gdn_stream_t stream);

/* Workspace bytes of gdn_kv4_attention on the current device for calls of up to B lanes and max_q tokens a lane; -1 if a
 * size is out of range. */
GDN_API int64_t gdn_kv4_attention_workspace(int32_t B, int32_t max_q, int32_t HQ, int32_t HK, int32_t D);

/*
 * Linear attention with a fixed decay for each head, on the state pools, lanes and drafts of the calls above (a hybrid model runs
 * such layers where it does not need the delta rule):
 *     S = g S + v k^T,   o = scale S q,   g = exp(log_decay[h])          (S [DV, DK] in fp32, q and k as they are)
 * log_decay [HV] fp32, at most 0 (-inf: no memory); HV / HK consecutive value heads share a query and key head.  dims, layouts,
 * alignment, padded lanes, errors and bf16 rounding are those of gdn_decode, gdn_mtp_verify, gdn_commit_replay and gdn_prefill
 * (l2_eps is not read).  out_indices [B], where a call takes it, names the slots that the final states go to, so that the
 * state read stays as it is (a cached prefix); NULL: state_indices.  There -1 writes no state, and anything else outside the
 * pool skips the lane (GDN_ERRBIT_INDEX).  Active lanes write distinct slots, and none that another lane reads.
 * What is not finite reaches what the recurrence lets it reach and nothing else: a q its own token, a k or v its token and those
 * behind it, a state its rows.  A state keeps infinities as the recurrence does, by whichever call it comes (but for an infinite k whose
 * v g^e underflows in a step or in 16 tokens: NaN); o is infinite or NaN there.
 *
 * gdn_linear_decode -- T tokens (1 .. GDN_MAX_T) from state_pool[state_indices[b]]: o, and the final state.
 */
GDN_API gdn_status gdn_linear_decode(const gdn_dims* dims, const void* q, const void* k, const void* v,
                                     const float* log_decay, void* state_pool, const int32_t* state_indices,
                                     const int32_t* out_indices, void* o, int32_t* err_word, gdn_stream_t stream);

/* gdn_linear_verify -- T draft tokens from states that are only read: o and, if intermediate_states [B, T, HV, DV, DK] is not
 * NULL, the state after every token (which gdn_commit takes).  Lanes may share a slot. */
GDN_API gdn_status gdn_linear_verify(const gdn_dims* dims, const void* q, const void* k, const void* v,
                                     const float* log_decay, const void* state_pool, const int32_t* state_indices, void* o,
                                     void* intermediate_states, int32_t* err_word, gdn_stream_t stream);

/* gdn_linear_commit -- the first accept_len[b] of a verify's T tokens again, without outputs: the final state.  accept_len 0
 * leaves the slot as it is (and copies the state where out_indices names another); outside 0 .. T the lane is skipped
 * (GDN_ERRBIT_ACCEPT_LEN). */
GDN_API gdn_status gdn_linear_commit(const gdn_dims* dims, const void* k, const void* v, const float* log_decay,
                                     void* state_pool, const int32_t* state_indices, const int32_t* out_indices,
                                     const int32_t* accept_len, int32_t* err_word, gdn_stream_t stream);

/* gdn_linear_prefill -- packed prompts as in gdn_prefill (dims->T = N tokens in all): o at their tokens and the final states.
 * A prompt of no tokens leaves its slot as it is (and copies its initial state where out_indices names another).  workspace: at
 * least gdn_linear_prefill_workspace bytes on 16 bytes (may be NULL if that is 0), used by one call at a time; its contents
 * need not be kept. */
GDN_API gdn_status gdn_linear_prefill(const gdn_dims* dims, const int32_t* cu_seqlens, const void* q, const void* k,
                                      const void* v, const float* log_decay, void* state_pool, const int32_t* state_indices,
                                      const int32_t* out_indices, const int32_t* has_initial_state, void* o,
                                      void* workspace, int64_t workspace_bytes, int32_t* err_word, gdn_stream_t stream);

/* Workspace bytes of gdn_linear_prefill on the current device for calls of exactly these sizes; -1 if one is out of range. */
GDN_API int64_t gdn_linear_prefill_workspace(int32_t B, int32_t N, int32_t HV, int32_t DK, int32_t DV);

/*
 * The sampling that ends a speculative step (the CTAs of a row or lane run as one thread-block cluster and meet at its hardware
 * barrier): the logits of its rows become probabilities (gdn_token_probs), drafts are accepted
 * against them and one more token is drawn (gdn_draft_accept), and accept_len goes to the commits above.  T is the step's: the
 * last token and T - 1 drafts; T = 1 is a decode step without drafts.
 */
typedef struct gdn_token_dims {
    int32_t B;             /* lanes, 0 .. 65535 */
    int32_t T;             /* rows per lane, >= 1; B * T < 2^31 */
    int32_t V;             /* tokens of the vocabulary, 1 .. 2^30 */
    int32_t dtype;         /* gdn_dtype of the logits */
    int64_t logits_stride; /* elements from one row to the next, >= V */
    int64_t probs_stride;  /* likewise */
} gdn_token_dims;

/*
 * gdn_token_probs -- probs[b, t, v] = exp((x_v - max x) / temperature[b]) / sum_u exp((x_u - max x) / temperature[b]) of the
 * row x = logits[b, t], in fp32.  A temperature of 0 (below the smallest normal number) puts 1 at the first of the largest
 * logits and 0 elsewhere.  Logits of -inf (forbidden tokens) get 0, and a row of nothing else is all 0.  A row with NaN or +inf,
 * or of a lane whose temperature is negative or not finite, is all 0 and sets GDN_ERRBIT_NONFINITE.  logits and probs on their
 * element size; the two must not overlap; room between rows is neither read nor written.
 */
GDN_API gdn_status gdn_token_probs(const gdn_token_dims* dims, const void* logits, const float* temperature, float* probs,
                                   int32_t* err_word, gdn_stream_t stream);

typedef struct gdn_accept_dims {
    int32_t B;             /* lanes, 0 .. 65535 */
    int32_t T;             /* rows per lane, 1 .. GDN_MAX_T: T - 1 drafts */
    int32_t V;             /* tokens of the vocabulary, 1 .. 2^30 */
    int64_t target_stride; /* elements from one row of target_probs to the next, >= V */
    int64_t draft_stride;  /* likewise (read only with draft_probs) */
} gdn_accept_dims;

/*
 * gdn_draft_accept -- target_probs [B, T] rows p_t of V fp32; draft_tokens [B, T - 1] x_t with the probabilities q_t they
 * were drawn from, draft_probs [B, T - 1] rows (NULL: 1 at the draft, as for drafts taken greedily); uniform [B, T] numbers
 * u_t in [0, 1).  Draft t is accepted while u_t q_t(x_t) < p_t(x_t).  With a drafts accepted the next token is drawn from
 * row a: r = max(p_a - q_a, 0) if draft a was refused, p_a after the last draft (and where r is all 0), and the token is the first v
 * with r_v > 0 and r_0 + .. + r_v > u_{T-1} (r_0 + .. + r_{V-1}).  Differences, products and sums are good to 2^-40 of the whole.
 *     accept_len[b] = a + 1 (the tokens to commit: the step's first and the accepted drafts)
 *     tokens[b]     = the a accepted drafts, the drawn token, then -1
 * A draft of -1 ends its lane's drafts there (lanes may have fewer), as does one outside the vocabulary, which sets
 * GDN_ERRBIT_INDEX.  Probabilities that are not finite count as 0 in r, and a row of which nothing is left draws -1: both set
 * GDN_ERRBIT_NONFINITE.  Lanes with state_indices[b] = -1 are skipped, their outputs left as they are (below -1:
 * GDN_ERRBIT_INDEX too); state_indices may be NULL.  Only the rows' needed parts are read.  All arrays on 4 bytes.
 */
GDN_API gdn_status gdn_draft_accept(const gdn_accept_dims* dims, const float* target_probs, const int32_t* draft_tokens,
                                    const float* draft_probs, const float* uniform, const int32_t* state_indices,
                                    int32_t* accept_len, int32_t* tokens, int32_t* err_word, gdn_stream_t stream);

/* Static string naming a status; never NULL. */
GDN_API const char* gdn_status_string(gdn_status status);

/* cudaError_t of the calling thread's last GDN_ERR_CUDA (0 if none). */
GDN_API int32_t gdn_last_cuda_error(void);

/* ABI version of this header: 1. */
GDN_API int32_t gdn_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H_ */
