/*
 * ssu.h -- libssu: the Mamba2 decode-step selective_state_update on AMD
 * Instinct MI355X (gfx950), as a C ABI.
 *
 * The operation (one decode token for a batch of requests; sglang PR #41223,
 * "[Perf] Mamba2 selective_state_update up to 2x faster on B200 via 8x1 launch
 * config for dstate 128", sections "Summary" and "Kernel measurement"): for
 * every request b and head h, with g = h / (H/G) the head's group,
 *
 *     slot    = idx[b]
 *     delta   = softplus(dt[b,h] + dt_bias[h])        (or dt + dt_bias when
 *                                                      dt_softplus == 0)
 *     a       = exp(A[h] * delta)
 *     S[p,n]  = state[slot,h,p,n] * a + delta * x[b,h,p] * B[b,g,n]
 *     state[slot,h,p,n] = S[p,n]                       (in place, fp32)
 *     out[b,h,p] = bf16( sum_n S[p,n] * C[b,g,n] + D[h] * x[b,h,p] )
 *
 * The page states the problem this way: an fp32 state pool [pool, H, P, N]
 * addressed through random state_batch_indices, x/B/C as views into one packed
 * bf16 tensor, and dt, A, D, dt_bias holding one value per head (zero strides
 * over the other axes). The
 * arguments below mirror that statement: every operand is a strided view.
 *
 * Numerics: fp32 arithmetic throughout; the sum over n is taken in one fixed
 * order that does not depend on the launch configuration (tile), so every tile
 * gives bitwise-identical state and out, and repeated runs are bitwise
 * reproducible. out is rounded to bf16 to nearest, ties to even.
 *
 * Ownership and threading: the caller owns every device buffer and the stream.
 * ssu_update is asynchronous on the stream: buffers must stay alive until the
 * stream's work completes. The library keeps no pointer after a call returns.
 * A handle is immutable after ssu_create, so calls on one handle from several
 * threads or streams are safe. ssu_update allocates nothing, never
 * synchronises and never reads device memory, so it may be captured into a
 * HIP graph.
 *
 * Errors: every function reports through ssu_status; nothing throws across the
 * ABI. ssu_last_error() gives a one-line description of the calling thread's
 * most recent failure.
 */
#ifndef SSU_H
#define SSU_H

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SSU_ABI_VERSION 1

typedef enum ssu_status {
    SSU_OK = 0,
    SSU_ERR_INVALID_ARGUMENT = 1, /* null pointer, negative size, wrong dtype tag, bad config */
    SSU_ERR_UNSUPPORTED = 2,      /* shape or layout the library does not run (see ssu_update) */
    SSU_ERR_MISALIGNED = 3,       /* state or B/C address not aligned for vector access */
    SSU_ERR_HIP = 4,              /* a HIP runtime call failed (launch, device query, copy) */
    SSU_ERR_NO_MEMORY = 5,        /* host allocation failed */
    SSU_ERR_BAD_INDEX = 6         /* ssu_check_indices: duplicate in-range slot ids */
} ssu_status;

typedef enum ssu_dtype {
    SSU_F32 = 0,
    SSU_BF16 = 1,
    SSU_I32 = 2,
    SSU_I64 = 3,
    SSU_F16 = 4, /* IEEE binary16 (ssu_scan activations) */
    SSU_E4M3 = 5 /* 8 bits, 4 of exponent, no infinities (ssu_add_rms_norm) */
} ssu_dtype;

/* Problem shape and options, fixed for the life of a handle. */
typedef struct ssu_config {
    int32_t nheads;      /* H >= 1 */
    int32_t headdim;     /* P: a multiple of 16, 16 <= P <= 256 */
    int32_t dstate;      /* N: 16, 32, 64, 128 or 256 */
    int32_t ngroups;     /* G >= 1, divides H; head h uses group h / (H/G) */
    int32_t dt_softplus; /* 1: delta = softplus(dt + dt_bias); 0: delta = dt + dt_bias */
    int32_t tile;        /* -1: launch configuration from the built-in table;
                            >= 0: always use tile #tile (for sweeps; see ssu_tile_info).
                            The environment variable SSU_TILE, read by ssu_create,
                            overrides a -1 here the same way. */
    int32_t device;      /* HIP device ordinal that launches run on (made
                            current for the call, then restored); -1: the
                            device current at each call */
    int32_t reserved;    /* must be 0 */
} ssu_config;

/* A strided view of device memory. Strides are in elements, outermost first;
 * unused trailing entries are ignored. */
typedef struct ssu_view {
    const void *ptr;
    int32_t dtype; /* ssu_dtype */
    int32_t reserved;
    int64_t stride[4];
} ssu_view;

/* One call's operands. Shapes are implied by the handle's config and `batch`;
 * the library cannot see buffer sizes, so the caller guarantees that every
 * view covers its shape.
 *
 *   state   [pool_slots, H, P, N] f32, read and written. stride[3] must be 1;
 *           the pointer and stride[0..2] must be 16-byte multiples.
 *   idx     [batch] i32 or i64 (state_batch_indices). stride[0] must be 1.
 *   x       [batch, H, P] bf16. stride[2] must be 1.
 *   B, C    [batch, G, N] bf16. stride[2] must be 1; the pointer and
 *           stride[0..1] must be 8-byte multiples.
 *   dt      [batch, H, P] bf16, one value per (request, head): stride[2] == 0.
 *   dt_bias [H, P] f32, stride[1] == 0. ptr may be NULL (no bias).
 *   A       [H, P, N] f32, stride[1] == stride[2] == 0.
 *   D       [H, P] f32, stride[1] == 0. ptr may be NULL (no skip term).
 *   out     [batch, H, P] bf16, written. stride[2] must be 1.
 *
 * x, B and C may be views into one packed tensor. Neither out nor the state
 * pool may overlap any input (the kernel reads inputs through the read-only
 * scalar cache), out must not overlap the state, and the state rows of
 * distinct requests must not overlap.
 *
 * dt is read as the aligned 32-bit words that hold its elements (the scalar
 * cache reads whole words), so reading the first or the last element of the
 * view may also read the 2 bytes beside it, just outside the view. An aligned
 * word never crosses a page, so such a read cannot fault wherever the element
 * itself is mapped, and the 2 extra bytes are never used; the caller need not
 * pad dt. A tool that tracks bytes (a sanitizer) may still report the read.
 */
typedef struct ssu_args {
    int32_t batch;      /* >= 0; 0 is a no-op */
    int32_t reserved;   /* must be 0 */
    int64_t pool_slots; /* number of slots in the state pool, >= 0 */
    ssu_view state, idx, x, B, C, dt, dt_bias, A, D, out;
} ssu_args;

/* Operands of a call that advances each request by `ntokens` tokens at once
 * (for example the draft tokens of speculative or multi-token-prediction
 * decoding). As ssu_args, but x, B, C, dt and out carry a token axis:
 *
 *   x    [batch, ntokens, H, P] bf16, stride[3] == 1
 *   B, C [batch, ntokens, G, N] bf16, stride[3] == 1
 *   dt   [batch, ntokens, H, P] bf16, stride[3] == 0
 *   out  [batch, ntokens, H, P] bf16, stride[3] == 1
 *
 * state, idx, dt_bias, A and D are as in ssu_args. Alignment rules extend to
 * the token stride (x: 4-byte multiples; B, C: 8-byte multiples). */
#define SSU_MAX_TOKENS 1024

typedef struct ssu_tokens_args {
    int32_t batch;      /* >= 0; 0 is a no-op */
    int32_t ntokens;    /* 1 .. SSU_MAX_TOKENS */
    int64_t pool_slots; /* number of slots in the state pool, >= 0 */
    ssu_view state, idx, x, B, C, dt, dt_bias, A, D, out;
} ssu_tokens_args;

typedef struct ssu_handle ssu_handle;

/* Description of one launch configuration. */
typedef struct ssu_tile_desc {
    int32_t dstate;          /* N this tile is compiled for */
    int32_t rows_per_wave;   /* state rows (p) each wave64 owns */
    int32_t waves;           /* waves per workgroup */
    int32_t rows_per_group;  /* rows_per_wave * waves */
    int32_t nontemporal;     /* 1: state loads/stores carry the non-temporal hint */
    int32_t xcd_remap;       /* 1: workgroups of neighbouring heads share an XCD */
    int32_t groups_per_cu;   /* residency cap: at most this many workgroups per CU
                                (enforced by reserving unused LDS); 0 = none */
    char name[48];
} ssu_tile_desc;

/* Validate `cfg` and create a handle. Does not touch the GPU.
 * Errors: SSU_ERR_INVALID_ARGUMENT (null, H/P/N/G out of range, G not dividing
 * H, tile index out of range), SSU_ERR_UNSUPPORTED (P or N the library has no
 * kernel for), SSU_ERR_NO_MEMORY. */
ssu_status ssu_create(const ssu_config *cfg, ssu_handle **out);

/* Enqueue one decode step on `stream` (NULL: the null stream).
 *
 * Preconditions the library cannot check without reading device memory (see
 * ssu_check_indices for a debug check): in-range entries of idx are distinct.
 * Entries outside [0, pool_slots) are padding: that request's state is neither
 * read nor written and its out rows are left untouched.
 *
 * Errors (nothing is launched): SSU_ERR_INVALID_ARGUMENT (null handle/args,
 * batch < 0, pool_slots < 0, null required pointer, wrong dtype tag, negative
 * stride, non-zero reserved field), SSU_ERR_UNSUPPORTED (an inner stride that
 * must be 1 is not, a broadcast stride that must be 0 is not),
 * SSU_ERR_MISALIGNED (state or B/C alignment), SSU_ERR_HIP (the launch
 * failed; the stream's state is the runtime's). batch == 0 returns SSU_OK
 * without launching and without reading any view. */
ssu_status ssu_update(const ssu_handle *h, const ssu_args *args, hipStream_t stream);

/* Enqueue `ntokens` decode steps per request in one launch: each request's
 * state is read once, advanced token by token (token t uses x, B, C, dt of
 * token t; out[:, t] is the output after token t) and written once. The
 * result is bitwise identical to `ntokens` successive ssu_update calls with
 * the per-token operands, at 1/ntokens of their state traffic. Same
 * preconditions, padding rule and errors as ssu_update, plus
 * SSU_ERR_INVALID_ARGUMENT for ntokens outside [1, SSU_MAX_TOKENS]. */
ssu_status ssu_update_tokens(const ssu_handle *h, const ssu_tokens_args *args, hipStream_t stream);

/* Release a handle. NULL is a no-op. */
void ssu_destroy(ssu_handle *h);

/* Debug check of idx, not for hot paths and not capturable: copies idx to the
 * host (synchronising `stream`) and returns SSU_ERR_BAD_INDEX if two in-range
 * entries are equal. Entries outside [0, pool_slots) are padding and allowed. */
ssu_status ssu_check_indices(const ssu_args *args, hipStream_t stream);

/* The launch configuration ssu_update would use for `batch` requests
 * (-1 if the handle's shape has none). */
int32_t ssu_select_tile(const ssu_handle *h, int32_t batch);

/* The launch configuration ssu_update_tokens would use for `batch` requests
 * of `ntokens` tokens (-1 if none). */
int32_t ssu_select_tile_tokens(const ssu_handle *h, int32_t batch, int32_t ntokens);

/* Number of compiled launch configurations, and their descriptions. */
int32_t ssu_tile_count(void);
ssu_status ssu_tile_info(int32_t tile, ssu_tile_desc *out);

/* Static string naming a status code. */
const char *ssu_status_string(ssu_status s);

/* The calling thread's most recent error description ("" if none). */
const char *ssu_last_error(void);

/* ---------------------------------------------------------- block copies --
 * Copy whole state blocks between slots, for prefix caching and multi-token
 * prediction in hybrid models (vLLM PR #48110, "[Perf][Hybrid] Vectorize
 * _copy_mamba_state_block to uint64 for temporal", section "Purpose"): for
 * every request r and every tensor k, block src_blocks[r] of tensor k is
 * copied to block dst_blocks[r] of tensor k.
 */

/* One state tensor (for example one layer's conv or temporal state). Block i
 * occupies bytes [base + i * block_stride, base + i * block_stride +
 * block_bytes). base, block_stride and block_bytes must be 16-byte multiples
 * (SSU_ERR_MISALIGNED otherwise: a guardrail, there is no narrow path). */
typedef struct ssu_block_tensor {
    void *base;
    int64_t block_stride; /* bytes, >= block_bytes unless nblocks <= 1 */
    int64_t block_bytes;  /* bytes copied per block (0: tensor skipped) */
    int64_t nblocks;      /* ids outside [0, nblocks) skip that request */
} ssu_block_tensor;

/* Enqueue the copies on `stream`. `tensors` is a host array read during the
 * call only; src_blocks and dst_blocks are device arrays [nreqs] int32.
 * src == dst is a no-op. Preconditions (not checked; the result would depend
 * on the order of the copies): destinations are distinct and no destination is
 * another request's source. tile = -1 uses the default launch configuration;
 * 0 .. ssu_copy_tile_count()-1 forces one (for sweeps). Asynchronous,
 * allocation-free and graph-capturable like ssu_update.
 * Errors: SSU_ERR_INVALID_ARGUMENT (negative sizes, null pointers, tile out of
 * range, overlapping blocks), SSU_ERR_MISALIGNED, SSU_ERR_UNSUPPORTED (more than
 * 2^31 workgroups in one launch), SSU_ERR_HIP. All of them but SSU_ERR_HIP are
 * found before anything is enqueued; more than 32 tensors take one launch per
 * 32, and SSU_ERR_HIP from a later launch leaves the earlier ones enqueued.
 * nreqs == 0 or ntensors == 0 is a no-op. */
ssu_status ssu_copy_blocks(const ssu_block_tensor *tensors, int32_t ntensors, const int32_t *src_blocks,
                           const int32_t *dst_blocks, int32_t nreqs, int32_t tile, hipStream_t stream);

/* Number of compiled copy configurations, and the name of one ("" if out of
 * range). */
int32_t ssu_copy_tile_count(void);
const char *ssu_copy_tile_name(int32_t tile);

/* ------------------------------------------------ selective scan (prefill) --
 * The selective scan over a whole sequence, as used to prefill a request
 * before decoding (COREY: Entropy-Guided Runtime Chunk Scheduling for
 * Selective Scan Kernels, Table 9, Table 17 and Table 18: selective_scan_fn
 * over dim channels with d_state states each, FP16 or BF16 activations, the
 * sequence cut into static chunks with one kernel call per chunk and the
 * state carried between calls). For every request b, channel d and token t in
 * order, with g = d / (dim / ngroups):
 *   Delta  = softplus(delta[b,d,t] + delta_bias[d])   (delta_softplus = 1)
 *          = delta[b,d,t] + delta_bias[d]             (delta_softplus = 0)
 *   h[n]   = h[n] * exp(A[d,n] * Delta) + (Delta * u[b,d,t]) * B[b,g,n,t]
 *   out[t] = sum_n h[n] * C[b,g,n,t] + D[d] * u[b,d,t]
 * h starts from state[b,d,:] and is written back there after the last token,
 * so a sequence may also be scanned piecewise over several calls. Arithmetic
 * is fp32; out is rounded to the activation type (nearest even).
 */
typedef struct ssu_scan_args {
    int32_t batch;          /* >= 0 (0: no-op) */
    int32_t dim;            /* channels, >= 1 */
    int32_t dstate;         /* states per channel, 1 .. 64 */
    int32_t ngroups;        /* B/C groups, divides dim */
    int64_t seqlen;         /* L >= 0 tokens (0: nothing to do) */
    int32_t delta_softplus; /* 1 or 0, see above */
    int32_t reserved;       /* must be 0 */
    ssu_view state;         /* [batch, dim, dstate] F32, read and written; stride[2] == 1 */
    ssu_view u;             /* [batch, dim, L] F16 or BF16; stride[2] == 1 */
    ssu_view delta;         /* [batch, dim, L], u's dtype; stride[2] == 1 */
    ssu_view B;             /* [batch, ngroups, dstate, L], u's dtype; stride[3] == 1 */
    ssu_view C;             /* [batch, ngroups, dstate, L], u's dtype; stride[3] == 1 */
    ssu_view A;             /* [dim, dstate] F32, finite */
    ssu_view D;             /* [dim] F32, contiguous; ptr may be NULL (no skip term) */
    ssu_view delta_bias;    /* [dim] F32, contiguous; ptr may be NULL (no bias) */
    ssu_view out;           /* [batch, dim, L], u's dtype, written; stride[2] == 1 */
} ssu_scan_args;

/* Enqueue the scan of `args` on `stream`, chunk after chunk of `chunk` tokens
 * (chunk = 0: the whole sequence), in order, the state carried between them
 * through `state`; a chunk is one kernel launch, or two when it ends in a
 * ragged or unaligned rest (its whole blocks, then the rest). Chunks whose
 * size is a multiple of 512 give bitwise the same results as one launch;
 * other chunk sizes agree within rounding. Every configuration with the same
 * token segment gives the same bits, so a request's results do not depend on
 * the batch it is scanned in. tile = -1 picks the launch configuration from
 * the chunk size and the number of channels; 0 .. ssu_scan_tile_count()-1
 * forces one.
 * Memory: the caller owns every buffer; the library allocates nothing and
 * keeps no pointer after the call. out and state must not overlap each other
 * or any input (the kernel reads inputs through the read-only cache).
 * Asynchronous and graph-capturable; nothing is checked on the device.
 * Errors (nothing is launched): SSU_ERR_INVALID_ARGUMENT (null pointers,
 * negative sizes or strides, wrong dtypes, non-zero reserved fields,
 * dim % ngroups != 0, tile out of range), SSU_ERR_UNSUPPORTED (non-contiguous
 * token or state axis, D or delta_bias, dstate > 64, batch * dim >= 2^31; a
 * forced staged or paired configuration when the channels of a group do not
 * split into its workgroups' 2, 4 or 8, or when B's or C's state stride is
 * 2^24 elements or more),
 * SSU_ERR_MISALIGNED (elements not aligned to their size), SSU_ERR_HIP
 * (launch failure; earlier chunks may have run). */
ssu_status ssu_scan(const ssu_scan_args *args, int64_t chunk, int32_t tile, hipStream_t stream);

/* Number of compiled scan configurations, and the name of one ("" if out of
 * range). */
int32_t ssu_scan_tile_count(void);
const char *ssu_scan_tile_name(int32_t tile);

/* The configuration ssu_scan(args, chunk, -1, ...) launches, from the tokens
 * one launch spans (chunk, or L if chunk is 0 or longer), the number of
 * channels (batch * dim), the channels of a group (dim / ngroups), dstate and
 * B's and C's state strides; only those fields of `args` are read (no
 * pointer is touched). Returns -1 if args is null or those sizes are invalid (negative
 * chunk, batch, seqlen or strides, dim or ngroups below 1, ngroups not
 * dividing dim). */
int32_t ssu_scan_select_tile(const ssu_scan_args *args, int64_t chunk);

/* ------------------------------------------------------- linear attention --
 * Linear attention with a decay for each head, over whole prompts and for
 * single tokens, on the decode step's state slots. For every sequence, head h
 * (group g = h / (nheads / ngroups)) and token t in order:
 *
 *   S[p,n]   = S[p,n] * exp(log_decay[t,h]) + beta[t,h] * v[t,h,p] * k[t,g,n]
 *   out[t,p] = bf16( scale * sum_n S[p,n] * q[t,g,n] )
 *
 * S starts from state[idx[b], h] and is written back there after the
 * sequence's last token. With q = C, k = B, v = x, beta = delta and
 * log_decay = A * delta this is the recurrence of ssu_update (without D), so a
 * prompt's state can be advanced by either step afterwards (by ssu_update for
 * Mamba2, which has softplus and D in the same pass); with log_decay constant in
 * t (stride 0) it is attention with fixed decay rates.
 *
 * Numerics: state, decays, sums and the recurrence in fp32 (the decays'
 * running sums in fp64, where a sum over many tokens would lose digits). Over
 * prompts the products run on bf16 matrix instructions with fp32 sums; the
 * state and a chunk's scores enter the output's as a bf16 pair (value and
 * remainder, 2^-17 relative), so that only the output's own rounding to bf16 is
 * seen, and decayed v enters the state's as three (2^-24). log_decay below -10000 counts as -10000 (exp is 0
 * from -104 on), so -inf is a reset of the state; NaN and infinite v reach
 * their own and later tokens of their channel p only, NaN and infinite k
 * their own and later tokens, NaN and infinite q their own token. Infinities go
 * through the recurrence as written, in fp32 (0 times one is NaN): a prompt
 * leaves the infinities and NaN in state and out that single steps leave. Where
 * a sequence's results are not finite they are computed again token by token,
 * 10 to 30 times as long. The sizes of a call set where its sequences are cut, and
 * so change its results within rounding; the same call gives the same bits.
 */
typedef struct ssu_linear_args {
    int32_t batch;      /* sequences, >= 0 (0: no-op) */
    int32_t nheads;     /* H >= 1 */
    int32_t headdim;    /* P: a multiple of 16, 16 <= P <= 256 */
    int32_t dstate;     /* N: 16, 32, 64, 128 or 256 */
    int32_t ngroups;    /* G >= 1, divides H */
    int32_t device;     /* HIP device ordinal that launches run on (made current
                           for the call, then restored); -1: the current one */
    int64_t ntokens;    /* T >= 0: rows of q, k, v, log_decay, beta and out */
    int64_t pool_slots; /* slots in the state pool, >= 0 */
    float scale;        /* finite */
    int32_t reserved;   /* must be 0 */
    ssu_view state;      /* [pool_slots, H, P, N] F32, read and written; stride[3] == 1;
                            pointer and stride[0..2] 16-byte multiples */
    ssu_view idx;        /* [batch] I32 or I64, stride[0] == 1; ids outside [0, pool_slots)
                            are padding: neither state nor out is touched */
    ssu_view cu_seqlens; /* [batch + 1] I32, stride[0] == 1: sequence b is rows
                            [cu_seqlens[b], cu_seqlens[b+1]), taken inside [0, T); an empty or
                            reversed range is an empty sequence. Rows of no sequence
                            are left untouched in out. ssu_linear_attention_step:
                            ptr NULL, token b belongs to request b */
    ssu_view q, k;       /* [T, G, N] BF16, stride[2] == 1 */
    ssu_view v;          /* [T, H, P] BF16, stride[2] == 1 */
    ssu_view log_decay;  /* [T, H] F32, any strides >= 0 (0: broadcast) */
    ssu_view beta;       /* [T, H] F32, any strides >= 0; ptr NULL: 1 */
    ssu_view out;        /* [T, H, P] BF16, written, stride[2] == 1 */
    void *workspace;     /* device memory, 16-byte aligned; its contents do not matter
                            before and after the call; NULL where none is needed */
    int64_t workspace_bytes;
} ssu_linear_args;

/* Bytes of workspace that ssu_linear_attention needs for `args` (only its sizes
 * are read; 0 where none is needed, -1 for sizes that it refuses). */
int64_t ssu_linear_attention_workspace(const ssu_linear_args *args);

/* Enqueue `args`' prompts on `stream`. In-range ids must be distinct and
 * cu_seqlens must not decrease (neither is checked on the device: with sequences
 * that share rows or slots the values there are unspecified, every access
 * stays inside the views). out, state and workspace must not overlap each
 * other or any input; calls that may run at the same time need workspaces of
 * their own. Asynchronous, allocation-free and graph-capturable like
 * ssu_update.
 * Errors (nothing is launched): SSU_ERR_INVALID_ARGUMENT (null pointers,
 * negative sizes or strides, wrong dtype tags, non-zero reserved fields, G not
 * dividing H, a scale that is not finite, a workspace too small),
 * SSU_ERR_UNSUPPORTED (P, N, inner strides, token strides of q, k, v and out of 2^24
 * elements or more, more than 2^31 tokens, 2^32 threads of a launch or more),
 * SSU_ERR_MISALIGNED, SSU_ERR_HIP. */
ssu_status ssu_linear_attention(const ssu_linear_args *args, hipStream_t stream);

/* The same for one token per request: ntokens == batch, token b advances
 * request b; cu_seqlens.ptr and workspace are NULL. Same errors, but token
 * strides of any size. */
ssu_status ssu_linear_attention_step(const ssu_linear_args *args, hipStream_t stream);

/* ------------------------------------------------------- gated delta rule --
 * The gated delta rule over whole prompts and for single tokens, on state slots
 * as ssu_linear_attention's: what a key already recalls is taken out of the
 * value before it is written. For every sequence, head h (group
 * g = h / (nheads / ngroups)) and token t in order:
 *
 *   S[p,n]   = S[p,n] * exp(log_decay[t,h])
 *   u[p]     = beta[t,h] * (v[t,h,p] - sum_n S[p,n] * k[t,g,n])
 *   S[p,n]   = S[p,n] + u[p] * k[t,g,n]
 *   out[t,p] = bf16( scale * sum_n S[p,n] * q[t,g,n] )
 *
 * With normalize, k and q stand for k / sqrt(sum_n k^2 + 1e-6) and
 * q / sqrt(sum_n q^2 + 1e-6). log_decay 0 (one zero, strides 0) is the delta rule
 * without a gate. The recurrence does not grow while beta |k|^2 <= 2 and
 * log_decay <= 0.
 *
 * Numerics as in ssu_linear_attention: state, decays, sums and the recurrence in
 * fp32; over prompts the products run on bf16 matrix instructions, fp32 operands
 * as three bf16 pieces where they enter the state (2^-24 relative), as two where
 * they enter only the output (2^-17). log_decay below -10000 counts as -10000. A chunk of tokens
 * with a value that is not finite, or whose state, keys, queries, gains and decays are so
 * large that a value might leave fp32 in it, goes through the recurrence token by
 * token, so that prompts leave the infinities and NaN that single steps leave: NaN and
 * infinite v reach their own and later tokens of their channel p only, NaN and
 * infinite k and beta their own and later tokens, NaN and infinite q their own
 * token. (Where finite terms of a sum over n leave fp32 on the way, it depends on their
 * order whether an infinity, NaN or a finite value comes of it, and prompts and steps
 * add up in orders of their own.) Such chunks take 20 to 100 times as long. The same call gives the same bits.
 */
typedef struct ssu_delta_args {
    int32_t batch;      /* sequences, >= 0 (0: no-op) */
    int32_t nheads;     /* H >= 1 */
    int32_t headdim;    /* P: a multiple of 16, 16 <= P <= 256 */
    int32_t dstate;     /* N: 16, 32, 64, 128 or 256 */
    int32_t ngroups;    /* G >= 1, divides H */
    int32_t device;     /* as in ssu_linear_args */
    int64_t ntokens;    /* T >= 0: rows of q, k, v, log_decay, beta and out */
    int64_t pool_slots; /* slots in the state pool, >= 0 */
    float scale;        /* finite */
    int32_t normalize;  /* 1 or 0 */
    ssu_view state;      /* [pool_slots, H, P, N] F32, this and the other views as in ssu_linear_args */
    ssu_view idx;        /* [batch] I32 or I64 */
    ssu_view cu_seqlens; /* [batch + 1] I32; ssu_gated_delta_rule_step: ptr NULL */
    ssu_view q, k;       /* [T, G, N] BF16 */
    ssu_view v;          /* [T, H, P] BF16 */
    ssu_view log_decay;  /* [T, H] F32, any strides >= 0 */
    ssu_view beta;       /* [T, H] F32, any strides >= 0; ptr NULL: 1 */
    ssu_view out;        /* [T, H, P] BF16, written */
    void *workspace;     /* as in ssu_linear_args */
    int64_t workspace_bytes;
} ssu_delta_args;

/* Bytes of workspace that ssu_gated_delta_rule needs for `args` (only its sizes
 * are read; -1 for sizes that it refuses): 8 KiB for each head and 32 tokens. */
int64_t ssu_gated_delta_rule_workspace(const ssu_delta_args *args);

/* Enqueue `args`' prompts on `stream`: conditions and errors of
 * ssu_linear_attention, and SSU_ERR_INVALID_ARGUMENT for another value of normalize. */
ssu_status ssu_gated_delta_rule(const ssu_delta_args *args, hipStream_t stream);

/* The same for one token per request: ntokens == batch, token b advances
 * request b; cu_seqlens.ptr and workspace are NULL. Same errors, but token
 * strides of any size. */
ssu_status ssu_gated_delta_rule_step(const ssu_delta_args *args, hipStream_t stream);

/* ------------------------------------------ queries and keys of attention --
 * Norms of queries and keys for each head with the position rotation, for the
 * attention layers of hybrid models. Each head row x of q and k [D] becomes
 *
 *   y = x / sqrt(mean(x^2) + eps) * weight        (no weight: factor 1)
 *   (y[a], y[b]) = (y[a] c_i - y[b] s_i, y[b] c_i + y[a] s_i),  i < rot / 2
 *
 * with (a, b) = (i, i + rot/2), or (2i, 2i + 1) when interleaved, and c_i, s_i
 * columns i and rot/2 + i of row positions[t] of cos_sin; values from rot on
 * are only normed. fp32 throughout, one rounding (to nearest even) at the end
 * (rows whose squares add up beyond fp32 become 0). Where rot is no multiple of 8,
 * calls of up to 2048 head rows and longer ones run in kernels of their own, whose
 * results differ within fp32's rounding before it.
 * With k_cache and v_cache, token t's keys and values also go into row
 * slots[t] of a paged cache (page slots[t] / page_size, row slots[t] %
 * page_size); slots outside the cache are skipped. A token whose position is
 * outside [0, max_pos) is padding: nothing of it is read or written.
 * (ssu_paged_attention reads caches of D = 64, 128 and 256.)
 */
typedef struct ssu_qk_args {
    int64_t ntokens;     /* T >= 0 (0: no-op) */
    int32_t nq, nk;      /* heads of q (>= 0) and of k (>= 0) */
    int32_t headdim;     /* D, 1 <= D <= 512 */
    int32_t rot;         /* even, 0 <= rot <= D (0: norm only) */
    int32_t interleaved; /* 1 or 0 */
    int32_t device;      /* as in ssu_linear_args */
    float eps;           /* >= 0, finite */
    int32_t page_size;   /* rows of a page, >= 1 (with k_cache) */
    int64_t max_pos;     /* rows of cos_sin, >= 0 */
    int64_t num_pages;   /* pages of the caches, >= 0 */
    ssu_view q, k;       /* [T, nq | nk, D] BF16 or F16, the same for all 16-bit views; stride[2] == 1 */
    ssu_view q_weight, k_weight; /* [D] F32 or the 16-bit type, stride[0] == 1; ptr NULL: 1 */
    ssu_view positions;  /* [T] I32 or I64, stride[0] == 1 */
    ssu_view cos_sin;    /* [max_pos, rot] F32, stride[1] == 1 */
    ssu_view q_out;      /* [T, nq, D] written, stride[2] == 1; may be q itself */
    ssu_view k_out;      /* [T, nk, D] written, stride[2] == 1; may be k itself; ptr NULL with
                            k_cache: keys go to the cache only */
    ssu_view v;          /* [T, nk, D], stride[2] == 1 (with k_cache) */
    ssu_view k_cache, v_cache; /* [num_pages, page_size, nk, D] written, stride[3] == 1; both
                            or neither (ptr NULL) */
    ssu_view slots;      /* [T] I32 or I64, stride[0] == 1 (with k_cache); in-range slots distinct */
} ssu_qk_args;

/* Enqueue it on `stream`. Outputs must not overlap inputs or each other, but
 * q_out may be q and k_out may be k (same pointer and strides). Asynchronous,
 * allocation-free, graph-capturable. Errors (nothing is launched):
 * SSU_ERR_INVALID_ARGUMENT (null pointers, sizes, strides, dtype tags),
 * SSU_ERR_UNSUPPORTED (D > 512, inner strides, 2^32 threads of a launch or more),
 * SSU_ERR_MISALIGNED (elements not aligned to their size), SSU_ERR_HIP. */
ssu_status ssu_qk_norm_rope(const ssu_qk_args *args, hipStream_t stream);

/* -------------------------------------------------------- paged attention --
 * Attention of one new token per request over a paged key-value cache, split
 * over the cache's length and joined. For request b and query head h, with
 * K_j, V_j row j % page_size of page block_table[b, j / page_size], head
 * h / (nq / nk), and n = min(seq_lens[b], max_pages * page_size):
 *
 *   w_j = exp(scale q[b,h] . K_j - m),  m = max_j (...)       j < n
 *   out[b,h] = sum_j w_j V_j / sum_j w_j
 *   lse[b,h] = m + log(sum_j w_j)
 *
 * No visible token, or only scores of -inf: out 0, lse -inf. A negative
 * seq_lens[b] marks a padding request, whose out and lse are left untouched.
 * Tokens of a page id outside [0, num_pages) are not visible. fp32 scores, statistics and sums; the
 * weights w_j enter the product with V as a 16-bit pair (value and
 * remainder), so that only the output's own rounding is seen. What the cache
 * holds in rows that no request sees, NaN and infinities too, does not matter;
 * infinities in rows of V that one sees give what the formula gives: an infinity,
 * or NaN where both signs meet or the score is -inf (a weight of 0). A wave that
 * meets one, or a NaN, reads its tokens again one by one, which takes longer.
 * The batch's other lengths and max_pages set where a request is split, and so
 * change its result within rounding; the same call gives the same bits.
 */
typedef struct ssu_attn_args {
    int32_t batch;       /* >= 0 (0: no-op) */
    int32_t nq, nk;      /* query and key/value heads, nk >= 1 divides nq */
    int32_t headdim;     /* D: 64, 128 or 256 */
    int32_t page_size;   /* >= 1 */
    int32_t device;      /* as in ssu_linear_args */
    int64_t num_pages;   /* pages of the caches, >= 0 */
    int64_t max_pages;   /* columns of block_table, >= 0 */
    float scale;         /* finite, also times log2(e) */
    int32_t reserved;    /* must be 0 */
    ssu_view q;          /* [batch, nq, D] BF16 or F16, stride[2] == 1 */
    ssu_view k_cache, v_cache; /* [num_pages, page_size, nk, D], q's type, stride[3] == 1 */
    ssu_view block_table; /* [batch, max_pages] I32, stride[1] == 1 */
    ssu_view seq_lens;   /* [batch] I32, stride[0] == 1 */
    ssu_view out;        /* [batch, nq, D] q's type, written, stride[2] == 1 */
    ssu_view lse;        /* [batch, nq] F32, written; ptr NULL: not wanted */
    void *workspace;     /* device memory, 16-byte aligned; contents do not matter;
                            NULL where none is needed */
    int64_t workspace_bytes;
} ssu_attn_args;

/* Bytes of workspace that ssu_paged_attention needs for `args` (only its sizes
 * are read; 0 where none is needed, -1 for sizes that it refuses). */
int64_t ssu_paged_attention_workspace(const ssu_attn_args *args);

/* Enqueue it on `stream`. Rows of 16-byte multiples (pointers and strides) are
 * read fastest; elements aligned to their size are enough. out, lse and
 * workspace must not overlap each other or any input; calls that may run at the
 * same time need workspaces of their own. Asynchronous, allocation-free,
 * graph-capturable. Errors (nothing is launched):
 * SSU_ERR_INVALID_ARGUMENT (null pointers, sizes, strides, dtype tags, a
 * workspace too small), SSU_ERR_UNSUPPORTED (D, inner strides, 2^32 threads
 * of a launch or more), SSU_ERR_MISALIGNED, SSU_ERR_HIP. */
ssu_status ssu_paged_attention(const ssu_attn_args *args, hipStream_t stream);

/* ----------------------------------------- attention over a shared prefix --
 * ssu_paged_attention for a batch whose requests all begin with the same tokens
 * (a system prompt, a document): request b attends to the n0 tokens of the
 * prefix, K_j, V_j row j % page_size of page prefix_table[j / page_size], and then
 * to its own seq_lens[b] of block_table, as one softmax over both:
 *
 *   n0 = min(max(prefix_len[0], 0), prefix_pages * page_size)
 *
 * The prefix is read once for the whole batch, and the products with it run on all
 * requests' query heads of a key head at once. seq_lens[b] = 0: the prefix alone; negative:
 * padding, of which neither q nor the prefix is used. Numerics as ssu_paged_attention, but
 * the weights of the prefix's V are rounded to 16 bits once, not kept as a pair: each is off by
 * half a step at most, out by 2^-8 (BF16; F16 2^-11) of the weighted mean of |V| beside its own
 * rounding, and with F16 each weight below 2^-28 of its row's largest by up to 2^-39 of that
 * one. (Whole weights: ssu_paged_attention with the prefix's pages in every request's table.)
 * Pieces of the prefix in which V holds infinities are read again token by token for rows that see
 * them, which takes 20 times as long or more. All that is said there of
 * visibility, infinities and repeated calls holds for the prefix.
 */
typedef struct ssu_shared_args {
    ssu_attn_args attn;    /* the requests' own tokens, and all other operands */
    ssu_view prefix_table; /* [prefix_pages] I32, stride[0] == 1 */
    ssu_view prefix_len;   /* [1] I32 */
    int64_t prefix_pages;  /* >= 0 */
} ssu_shared_args;

/* Bytes of workspace that ssu_shared_prefix_attention needs for `args` (only its
 * sizes are read; -1 for sizes that it refuses). */
int64_t ssu_shared_prefix_attention_workspace(const ssu_shared_args *args);

/* Enqueue it on `stream`: conditions and errors of ssu_paged_attention. */
ssu_status ssu_shared_prefix_attention(const ssu_shared_args *args, hipStream_t stream);

/* ------------------------------------------ norm with the residual added --
 * What stands between the layers: the residual stream takes a layer's output and
 * the next layer's input is its norm, in 16 bits or in 8 with scales. For every
 * row t of width D:
 *
 *   s = x[t] + residual[t]                      (no residual: s = x[t])
 *   residual[t] = s                             (rounded to its type)
 *   y = s / sqrt(mean(s^2) + eps) * weight      (no weight: factor 1)
 *   out[t] = y, or, in E4M3, for each `group` of consecutive values (0: all D)
 *   scales[t,i] = max(max|y| / 448, 2^-126),  out[t] = y / scales[t,i]
 *
 * fp32 throughout (the norm takes s before it is rounded into the residual),
 * each output rounded once, to nearest even. Rows whose squares add up beyond
 * fp32 become 0; with eps 0, rows whose squares add up below its least normal number lose
 * digits, and become infinities and NaN where that sum is 0. A NaN in a row's s makes its
 * y NaN, a NaN in y its group's scale and values.
 */
typedef struct ssu_norm_args {
    int64_t ntokens;    /* T >= 0 (0: no-op) */
    int32_t width;      /* D, 1 <= D <= 32768 */
    int32_t group;      /* E4M3: 0, or 32, 64, 128 or 256 dividing D; otherwise 0 */
    int32_t device;     /* as in ssu_linear_args */
    float eps;          /* >= 0, finite */
    ssu_view x;         /* [T, D] BF16 or F16, stride[1] == 1 */
    ssu_view residual;  /* [T, D] x's type or F32, read and written, stride[1] == 1; ptr NULL: none */
    ssu_view weight;    /* [D] x's type or F32, stride[0] == 1; ptr NULL: 1 */
    ssu_view out;       /* [T, D] x's type or E4M3, written, stride[1] == 1; may be x itself */
    ssu_view scales;    /* [T, group ? D / group : 1] F32, written (with E4M3; otherwise ptr NULL) */
} ssu_norm_args;

/* Enqueue it on `stream`. Outputs must not overlap inputs or each other, but out
 * may be x (same pointer and strides). Asynchronous, allocation-free,
 * graph-capturable, without workspace. Errors (nothing is launched):
 * SSU_ERR_INVALID_ARGUMENT (null pointers, sizes, strides, dtype tags, a group that
 * does not divide D, scales without E4M3), SSU_ERR_UNSUPPORTED (D > 32768, other
 * groups, inner strides, 2^32 threads of a launch or more), SSU_ERR_MISALIGNED
 * (elements not aligned to their size), SSU_ERR_HIP. */
ssu_status ssu_add_rms_norm(const ssu_norm_args *args, hipStream_t stream);

/* SSU_ABI_VERSION of the built library. */
int32_t ssu_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SSU_H */
