/*
 * iskv.h - C ABI of the iS-KV hot path on one B200 (sm_100a): block-incremental truncated SVD of
 * each (layer, sequence, kv-head) key and value stream, plus decode attention over the compressed
 * history and an exact recent window.
 *
 * Method: "iS-KV: Online Low-Rank KV Cache Compression via Block-Incremental SVD" (summary page).
 *   - "Architecture Overview": per K/V path an exact window of the most recent tokens and a
 *     low-rank history of rank at most r.
 *   - "Block-Incremental Decoding Updates": each fold takes the pending block F (b rows), forms the
 *     residual E = F - (F B) B^T and an orthonormal residual basis P, the core
 *     Z = [[Sigma, 0], [F B, F P]], its truncated SVD (G, Sigma+, H), and the updated factors
 *     U+ = diag(U, I_b) G, B+ = [B P] H. Old rows' coordinates move with the basis.
 *   - "Reconstruction and Storage": compressed row i is (U Sigma B^T)[i]; window rows are exact;
 *     storage k (n + d + 1) factor scalars per path plus d e exact scalars.
 *
 * Conventions shared by every entry point:
 *   - Return value: ISKV_OK (0) or a negative ISKV_ERR_* code; no C++ exception crosses the ABI.
 *     Argument errors are detected on the host before anything is enqueued.
 *   - Pointers named *_dev are device pointers owned by the caller; they must stay valid until
 *     the work enqueued on `stream` has completed. Pointers to host scalars are written before
 *     the call returns.
 *   - `stream` is a cudaStream_t (NULL = legacy default stream). All device work is enqueued on
 *     it asynchronously; nothing synchronises except iskv_sync_status().
 *   - The handle owns all persistent device state, allocated once by iskv_create() and sized by
 *     max_tokens; it is never reallocated. A handle is not thread-safe.
 *   - Each layer keeps its own token count t; layer = -1 addresses all layers at once (they must
 *     then hold the same t).
 *   - Device-side failures (a core SVD that did not converge, a non-finite singular value) set a
 *     sticky status word that iskv_sync_status() returns.
 */
#ifndef ISKV_H
#define ISKV_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct iskv_handle iskv_handle;
/* Layout-compatible with cudaStream_t. */
typedef struct CUstream_st *iskv_stream_t;

enum {
    ISKV_OK = 0,
    ISKV_ERR_INVALID_ARG = -1,  /* bad config, NULL pointer, layer out of range, ...        */
    ISKV_ERR_CAPACITY = -2,     /* t + m > max_tokens                                        */
    ISKV_ERR_CUDA = -3,         /* a CUDA runtime call failed (allocation, launch, copy)     */
    ISKV_ERR_NOT_CONVERGED = -4,/* a core SVD hit its sweep cap (sticky, device side)        */
    ISKV_ERR_NONFINITE = -5,    /* a non-finite singular value appeared (sticky, device side) */
    ISKV_ERR_UNSUPPORTED = -6,  /* valid request outside what this build implements          */
    ISKV_ERR_TIMEOUT = -7       /* a device-side wait hit its bound (sticky, device side)    */
};

enum { ISKV_BF16 = 0, ISKV_F32 = 1 };

typedef struct {
    int batch;            /* sequences decoded in lock-step                                  */
    int n_layers;
    int n_kv_heads;
    int n_q_heads;        /* multiple of n_kv_heads; q-head g reads kv-head g / (n_q/n_kv)    */
    int head_dim;         /* d; must be 128                                                  */
    int rank_k, rank_v;   /* rank budgets r_K, r_V (1 .. head_dim)                           */
    int block;            /* b: rows folded per update (1 .. 1024; blocks above 128 rows are  */
                          /*    folded through their 128-row triangular factor)              */
    int window;           /* w: exact rows kept before a fold may take them (>= 0)           */
    long long max_tokens; /* capacity per sequence and layer                                 */
    int kv_dtype;         /* ISKV_BF16 or ISKV_F32: dtype of appended rows and of the window  */
    int rope;             /* 1: rotate keys by RoPE (pairs j, j+d/2) after reconstruction     */
    double rope_theta;    /* RoPE base; angle of pair j at position i is i * theta^(-2j/d)    */
    int rotate_history;   /* 1: iS-KV (old coordinates rotate with the basis).               */
                          /* 0: stale-coordinate ablation (drift study only).                */
    int lookahead_folds;  /* 0: each fold runs on the caller's stream when the window releases  */
                          /*    its block.                                                     */
                          /* 1: each fold starts on an internal stream as soon as its block is */
                          /*    complete (up to window / block + 1 folds ahead) and is joined  */
                          /*    into the caller's stream when the window releases the block;   */
                          /*    every decode sees exactly the state of mode 0. Call            */
                          /*    iskv_join() before ending a stream capture that contains       */
                          /*    appends.                                                       */
    int fixed_basis;      /* 1: fixed-basis ablation ("Ablation Study", bases kept fixed): the   */
                          /*    regular update runs for the first ceil(min(r, d) / block) folds */
                          /*    of a path (they fill its rank budget); after that the path's   */
                          /*    basis and Sigma freeze and each later block is stored as its   */
                          /*    coordinates F B in the frozen basis (old coordinates untouched). */
                          /*    0: iS-KV. Cannot be combined with rotate_history = 0.           */
    int coord_bf16;       /* 1: store the coordinates C = U Sigma (the k n factor scalars that    */
                          /*    grow with the history) in bf16, rounded to nearest even after   */
                          /*    every fold and history rotation; arithmetic stays fp32 and B,    */
                          /*    Sigma stay fp32 ("Reconstruction and Storage": beta_f = 2 for C). */
                          /*    Needs rank_k <= 64, rank_k and rank_v multiples of 8 and a GQA   */
                          /*    group of 1, 2 or 4 (else ISKV_ERR_UNSUPPORTED). 0: fp32.         */
    int prot_cap;         /* 0: iskv_prefill() is not available. >= 1: it is, and the protected */
                          /*    stores hold up to prot_cap exact rows per unit and path        */
                          /*    ("Prefill Compression"; more set ISKV_ERR_CAPACITY, sticky).   */
    int joint_heads;      /* 1: joint per-layer factorisation ("Reconstruction and Storage",     */
                          /*    persistent storage per layer): the rows of all n_kv_heads of a   */
                          /*    (layer, sequence) at one position are concatenated, head by    */
                          /*    head, into one row of length d = n_kv_heads * head_dim, and one  */
                          /*    factorisation per (layer, sequence, path) folds them: one        */
                          /*    coordinate row of rank r per position, shared by the kv-heads,   */
                          /*    and a d x r basis whose rows h*128 .. h*128+127 reconstruct      */
                          /*    kv-head h. The exact window stays per kv-head. Needs            */
                          /*    rank + block <= 128 for both paths, fixed_basis = 0 and          */
                          /*    prot_cap = 0 (else ISKV_ERR_UNSUPPORTED). 0: one factorisation  */
                          /*    per (layer, sequence, kv-head, path).                           */
} iskv_config;

/* Key/value protection of iskv_prefill() ("Prefill Compression", steps 1-2). */
typedef struct {
    int chunk;            /* positions per key chunk (>= 1)                                   */
    int m;                /* outlier chunks protected per kv-head: the m lowest min-cosine     */
                          /*    scores (ties by chunk index) (>= 0)                            */
    int suffix;           /* positions just before the window that are protected too (>= 0)   */
    int rho;              /* value protection radius: P_V = positions within rho of P_K (>= 0) */
} iskv_protect;

/*
 * Creates a cache for `cfg` on the current CUDA device. Allocates every device buffer
 * (coordinates C = U Sigma [max compressed rows x r] in fp32, or bf16 with coord_bf16; bases
 * B [d x r], Sigma [r] and the
 * fold's H_top [r x r] in fp32, each in a ring of 2 buffers, or window / block + 3 with
 * lookahead_folds; the exact ring of window + block rows per path in kv_dtype; a RoPE table
 * [max_tokens x d/2] of (cos, sin); decode split partials; a status word) and, with
 * lookahead_folds, the internal streams and events of the early folds.
 * Errors: ISKV_ERR_INVALID_ARG (cfg out of range), ISKV_ERR_CUDA (allocation failed; nothing
 * leaks). On success *out owns the handle; release it with iskv_destroy().
 */
int iskv_create(const iskv_config *cfg, iskv_handle **out);

/* Frees every device buffer of the handle (synchronises the device first). NULL is a no-op. */
int iskv_destroy(iskv_handle *h);

/*
 * Appends m >= 1 new rows per (sequence, kv-head) to the key and value streams of `layer` and
 * folds every block that the window releases ("Block-Incremental Decoding Updates"): rows enter
 * the exact window one by one; whenever it holds window + block rows its oldest block is folded,
 * so after t tokens n_c(t) = block * floor(max(0, t - window) / block) rows are compressed.
 *   k_rows_dev, v_rows_dev: kv_dtype, row-major [batch][n_kv_heads][m][head_dim] for layer >= 0,
 *                           [n_layers][batch][n_kv_heads][m][head_dim] for layer == -1.
 *                           Keys are pre-RoPE.
 * Errors: ISKV_ERR_INVALID_ARG (NULL rows, m < 1, bad layer, layers with different t for -1),
 *         ISKV_ERR_CAPACITY (t + m > max_tokens), ISKV_ERR_CUDA (launch failed).
 */
int iskv_append_block(iskv_handle *h, int layer, const void *k_rows_dev, const void *v_rows_dev,
                      int m, iskv_stream_t stream);

/*
 * Prefill of an empty layer with T0 rows per (sequence, kv-head) ("Prefill Compression"): the
 * last `window` rows form the exact window; of the rows before it, the protected positions (keys:
 * P_K of step 1; values: P_V of step 2; none when protect is NULL) stay exact for good and the
 * others are factorised by one truncated SVD of rank r (step 3), computed from the rows'
 * triangular factor (Householder QR over 128-row chunks) and a one-sided Jacobi SVD of it; the
 * coordinates of protected positions are zero and decode reads their exact rows. Later appends
 * fold blocks from the window as usual. Chunk scores use keys rotated at their positions.
 *   k_rows_dev, v_rows_dev: kv_dtype [batch][n_kv_heads][T0][head_dim] (keys pre-RoPE).
 *   protect: host pointer or NULL.
 * Synchronises `stream` when protect is given (the largest protected count sizes the decode's
 * protected tiles). Needs cfg.prot_cap >= 1 (else ISKV_ERR_UNSUPPORTED); protection also needs
 * the persistent decode (rank_k <= 32 with fp32 coordinates, <= 64 with bf16; G of 1, 2 or 4).
 * Errors: ISKV_ERR_INVALID_ARG (layer not empty, bad protect values, T0 < 1),
 *         ISKV_ERR_CAPACITY (T0 > max_tokens), ISKV_ERR_UNSUPPORTED, ISKV_ERR_CUDA.
 */
int iskv_prefill(iskv_handle *h, int layer, const void *k_rows_dev, const void *v_rows_dev,
                 long long T0, const iskv_protect *protect, iskv_stream_t stream);

/*
 * Decode attention of `layer` over all t cached positions 0 .. t-1: compressed rows are
 * reconstructed as C B^T ("Reconstruction and Storage"), keys are then rotated by RoPE at their
 * position (when cfg.rope), scores use scale 1/sqrt(d), softmax is exact (fp32, log-sum-exp
 * merge of position splits). Two kernels (position splits, then their merge) on `stream`.
 *   q_dev:   fp32 [batch][n_q_heads][head_dim], already rotated for the query position,
 *            16-byte aligned (the kernels copy it in 16-byte units).
 *   out_dev: fp32 [batch][n_q_heads][head_dim].
 * Errors: ISKV_ERR_INVALID_ARG (NULL pointers, bad layer, t == 0, misaligned q_dev),
 *         ISKV_ERR_CUDA.
 */
int iskv_decode_attn(iskv_handle *h, int layer, const float *q_dev, float *out_dev,
                     iskv_stream_t stream);

/*
 * One decode step of `layer`: appends one new row per (sequence, kv-head) to the key and value
 * streams (with any fold the window releases, as iskv_append_block() with m = 1) and then runs
 * iskv_decode_attn() over positions 0 .. t (the new row included). Same results as those two
 * calls. With the tensor-core decode and window >= 1 the new rows are read by the decode kernel
 * itself, which also stores them in the exact ring, so the step needs no separate append launch;
 * otherwise the two calls are made in turn.
 *   k_row_dev, v_row_dev: kv_dtype [batch][n_kv_heads][1][head_dim] (keys pre-RoPE);
 *   q_dev, out_dev: as iskv_decode_attn().
 * Errors: those of iskv_append_block() and iskv_decode_attn().
 */
int iskv_append_decode(iskv_handle *h, int layer, const void *k_row_dev, const void *v_row_dev,
                       const float *q_dev, float *out_dev, iskv_stream_t stream);

/*
 * Writes the reconstructed cache of one path of `layer` ("Reconstruction and Storage"): row i is
 * (C B^T)[i] for i < n_c and the exact window row otherwise; keys are rotated by RoPE when
 * apply_rope != 0 (ignored for values).
 *   which:   0 = keys, 1 = values.
 *   out_dev: fp32 [batch][n_kv_heads][t][head_dim].
 * Errors: ISKV_ERR_INVALID_ARG, ISKV_ERR_CUDA.
 */
int iskv_reconstruct(iskv_handle *h, int layer, int which, int apply_rope, float *out_dev,
                     iskv_stream_t stream);

/*
 * Copies the factors of one unit (layer, seq, kv_head, path) into caller buffers (device to
 * device, on `stream`) and reports its current rank and compressed-row count.
 *   coords_dev: fp32 [n_c][rank] (row stride = rank budget of the path; bf16-stored coordinates
 *               are widened to fp32 exactly), may be NULL;
 *   basis_dev:  fp32 [head_dim][rank], may be NULL;
 *   sigma_dev:  fp32 [rank], may be NULL (entries >= *k_out are zero);
 *   k_out, n_c_out: host pointers, may be NULL.
 * Errors: ISKV_ERR_INVALID_ARG, ISKV_ERR_CUDA.
 */
int iskv_get_factors(iskv_handle *h, int layer, int seq, int kv_head, int which,
                     float *coords_dev, float *basis_dev, float *sigma_dev, int *k_out,
                     long long *n_c_out, iskv_stream_t stream);

/*
 * Empties every layer (t = n_c = 0, rank 0) and clears the sticky status, keeping all device
 * allocations, so a handle can serve a new batch of sequences. Joins pending early folds into
 * `stream` first (iskv_join); then host bookkeeping plus asynchronous device writes on `stream`;
 * later calls must be ordered after it on a stream.
 * Errors: ISKV_ERR_INVALID_ARG, ISKV_ERR_CUDA.
 */
int iskv_reset(iskv_handle *h, iskv_stream_t stream);

/*
 * Number of kernel launches this handle has enqueued since creation (host counter; launches
 * captured into a CUDA graph are counted once, at capture). Errors: ISKV_ERR_INVALID_ARG.
 */
int iskv_launch_count(const iskv_handle *h, long long *count_out);

/*
 * Statistics of the core SVDs run since creation or the last iskv_reset(): the largest number of
 * Jacobi sweeps one core needed, the total number of sweeps, and the number of cores solved.
 * Synchronises `stream` (a device-to-host copy). Any output pointer may be NULL.
 * Errors: ISKV_ERR_INVALID_ARG, ISKV_ERR_CUDA.
 */
int iskv_fold_stats(iskv_handle *h, iskv_stream_t stream, int *max_sweeps_out,
                    long long *total_sweeps_out, long long *cores_out);

/* Tokens cached in `layer` (host value). Errors: ISKV_ERR_INVALID_ARG. */
int iskv_num_tokens(const iskv_handle *h, int layer, long long *t_out);

/*
 * Persistent bytes of one layer per the storage formula of "Reconstruction and Storage":
 * sum_X [beta_c k_X n_X + 4 k_X (d + 1)] + beta_e * d * sum_X e_X, summed over sequences and
 * kv-heads, with beta_c = 2 (coord_bf16) or 4 bytes per coordinate, fp32 bases and Sigma, and
 * beta_e = bytes of kv_dtype. Host only.
 */
int iskv_storage_bytes(const iskv_handle *h, int layer, long long *bytes_out);

/*
 * Host-only schedule of the fold trigger ("Architecture Overview" window, read as: fold the
 * oldest block whenever window + block rows are exact). For a stream holding t tokens, appending
 * m rows leaves *n_c_out compressed rows and performs *folds_out folds. Needs no GPU.
 * Errors: ISKV_ERR_INVALID_ARG (block < 1, window < 0, t < 0, m < 0).
 */
int iskv_schedule(int block, int window, long long t, long long m, long long *n_c_out,
                  long long *folds_out);

/*
 * Makes `stream` wait for every fold that lookahead_folds started on an internal stream and that
 * no later call has joined yet (those whose blocks the window has not released). Required before
 * ending a stream capture that contains iskv_append_block() calls, so that the capture holds no
 * unjoined work; a no-op without lookahead_folds. Enqueues only event waits.
 * Errors: ISKV_ERR_INVALID_ARG, ISKV_ERR_CUDA.
 */
int iskv_join(iskv_handle *h, iskv_stream_t stream);

/*
 * Joins pending early folds (iskv_join), synchronises `stream` and returns the sticky status: ISKV_OK, ISKV_ERR_NOT_CONVERGED,
 * ISKV_ERR_NONFINITE or ISKV_ERR_TIMEOUT (the first error seen since creation or the last
 * iskv_reset()), or ISKV_ERR_CUDA if the synchronisation itself failed.
 */
int iskv_sync_status(iskv_handle *h, iskv_stream_t stream);

/*
 * Decode attention over caller-owned buffers that allocates nothing (no cudaMalloc, cudaFree or
 * allocating library routine, no handle). The paper has no counterpart: this entry point exists
 * for callers that cannot allocate device memory on their decode path - code running inside CUDA
 * stream capture (cudaMalloc is not capturable), engines whose device memory is entirely owned by
 * their own pool allocator, and latency-critical loops where cudaMalloc's implicit device
 * synchronisation is not acceptable.
 *
 * The computation is that of iskv_decode_attn() for one layer, on the CUDA-core decode kernels,
 * with the cache described by `view` instead of a handle. The split partials that
 * iskv_decode_attn() keeps in handle-owned memory live here in a file-scope device array of
 * ISKV_NOALLOC_SCRATCH_FLOATS floats (4 MiB) that every GPU which loads the library holds until the
 * process exits. Required scratch: batch * n_kv_heads * splits * (n_q_heads / n_kv_heads) *
 * (head_dim + 2) floats, with splits = ceil(n_c / 128) + ceil((t - n_c) / 128) at most; larger
 * requests return ISKV_ERR_CAPACITY before anything is enqueued.
 *
 * All calls share that array and it keeps the last call's contents; nothing in it has to start at
 * zero (every split writes its partials before the merge reads them). Calls whose work overlaps
 * on the GPU (different streams, or different host threads) race on the array: order them on one
 * stream. The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current) and keeps it; make that first call before any
 * stream capture.
 *   view:    cache description (layouts below), all pointers device pointers owned by the caller
 *            (one coordinate array per kv-head unit: a joint-factorisation cache, whose kv-heads
 *            share their coordinates, is decoded through iskv_decode_attn instead);
 *   q_dev:   fp32 [batch][n_q_heads][head_dim], already rotated for the query position;
 *   out_dev: fp32 [batch][n_q_heads][head_dim].
 * Errors: ISKV_ERR_INVALID_ARG (NULL pointer, inconsistent sizes), ISKV_ERR_CAPACITY (scratch
 * too small), ISKV_ERR_CUDA (address lookup or launch failed).
 */
#define ISKV_NOALLOC_SCRATCH_FLOATS (1 << 20)

typedef struct {
    long long n_c;        /* compressed rows per unit (positions 0 .. n_c-1)                   */
    long long t;          /* tokens: positions 0 .. t-1 are attended (t >= 1)                  */
    long long n_max;      /* coordinate rows per unit in coords_k / coords_v (>= n_c)          */
    int batch, n_kv_heads, n_q_heads, head_dim;    /* head_dim must be 128                  */
    int rank_k, rank_v;   /* row stride of the coordinate arrays = columns of the bases        */
    int k_k, k_v;         /* ranks in use (1 .. rank) when n_c > 0                             */
    int ring_rows;        /* R: exact row of position i (n_c <= i < t) sits at slot i mod R   */
    int kv_dtype;         /* ISKV_BF16 or ISKV_F32 (exact rows)                                */
    const float *coords_k, *coords_v;  /* [batch*n_kv_heads][n_max][rank] fp32                */
    const float *basis_k, *basis_v;    /* [batch*n_kv_heads][head_dim][rank] fp32             */
    const void *ring_k, *ring_v;       /* [batch*n_kv_heads][R][head_dim] kv_dtype, pre-RoPE */
    const float *rope_cs;              /* [t][head_dim/2] (cos, sin) pairs, or NULL: no RoPE */
} iskv_decode_view;

int iskv_decode_attn_noalloc(const iskv_decode_view *view, const float *q_dev, float *out_dev,
                             iskv_stream_t stream);

/*
 * ---- Exact caches --------------------------------------------------------------------------
 * Attention over rows that are kept as they are (the prompt before it is compressed, a cache that
 * is bounded by a window or by eviction instead of by its rank, samples that share a prompt), in
 * caller-owned memory. These calls keep no state and allocate nothing: the caller passes a
 * workspace of at least the size that the *_workspace() call of the same arguments gives (16-byte
 * aligned, contents irrelevant before and after). Calls whose work can overlap on the GPU need
 * workspaces of their own; that goes for two captured graphs that are replayed at the same time.
 * They run on the current CUDA device, which has to own all the pointers, and are capturable.
 *
 * Keys are as attended (already rotated), scores have the scale 1/sqrt(128), q-head g reads kv-head
 * g / (n_q/n_kv), and a query that sees no row gives zeros. The softmax is over all rows that a query
 * sees; maxima, sums and accumulators are float32. With float32 queries, products keep 22 bits and more.
 * With bf16 queries, a call that has more than 8 query rows (tokens or sequences, times q-heads) for a
 * kv-head's rows may round each softmax weight to bf16 before its product with the value (the sum of the
 * weights takes them unrounded): outputs are then off by up to 1.41 times what rounding them to bf16
 * alone gives. Others keep two bf16 terms of each weight. Rows that no
 * query of their sequence sees are not used: they may hold anything, NaN included. Device arrays
 * of lengths are read on the device: values below 0 count as 0, values above the capacity as the
 * capacity. Strides count elements and have to be multiples of 16 bytes; those of sequences, heads
 * and query tokens may be 0 where they share one place (never in outputs); a stride over an extent
 * of 1 is not read.
 */
typedef struct {
    const void *k, *v;       /* element (b, h, j, c) at b seq + h head + j row + c; 16-byte aligned */
    long long seq_stride, head_stride, row_stride;
    int batch, n_kv_heads;   /* batch * n_kv_heads <= 65535                                      */
    int rows;                /* capacity per sequence (0 .. 2^24; 0: k and v are not read)         */
    int dtype;               /* ISKV_BF16 or ISKV_F32                                             */
    const int *lens;         /* device, [batch]: rows held by each sequence; NULL: `rows`          */
} iskv_exact_rows;

typedef struct {
    const void *q;           /* element (b, g, i, c) at b seq + g head + i tok + c; 16-byte aligned */
    void *out;               /* the same with the o_ strides; must not overlap anything that is read */
    long long q_seq_stride, q_head_stride, q_tok_stride;
    long long o_seq_stride, o_head_stride, o_tok_stride;
    int n_q_heads;           /* n_kv_heads times 1 .. 8                                           */
    int m;                   /* query tokens per sequence (capacity)                              */
    int dtype;               /* of q and out: ISKV_BF16 or ISKV_F32 (float32 rows: ISKV_F32 only,  */
                             /* else ISKV_ERR_UNSUPPORTED)                                       */
    const int *q_lens;       /* device, [batch]: tokens of each sequence; NULL: m                 */
} iskv_exact_queries;

typedef struct {
    const void *k, *v;       /* element (h, j, c) at h head + j row + c; the rows' dtype           */
    long long head_stride, row_stride;
    int rows;                /* 0 .. 2^24                                                        */
} iskv_exact_prefix;

/*
 * Attention with a sliding window and a few first tokens that stay visible. The last q_lens[b] of a
 * sequence's lens[b] rows are the call's tokens: token i sits at p = lens[b] - q_lens[b] + i and
 * sees the rows j <= p with j < sinks or j > p - window (window >= lens: causal attention). From
 * a whole prompt (m = rows) to single tokens (m = 1). Outputs of tokens i >= q_lens[b] are not
 * written. A token's own row has to be in the cache before the call.
 * Where tokens see different rows of a call, a value that is not finite may reach every token
 * within 256 positions of one that sees it; it reaches no other.
 * Errors: ISKV_ERR_INVALID_ARG, ISKV_ERR_UNSUPPORTED, ISKV_ERR_CAPACITY (workspace too small),
 *         ISKV_ERR_CUDA.
 */
int iskv_window_attn(const iskv_exact_rows *rows, const iskv_exact_queries *q, int window,
                     int sinks, void *ws, size_t ws_bytes, iskv_stream_t stream);
int iskv_window_attn_workspace(const iskv_exact_rows *rows, const iskv_exact_queries *q,
                               int window, int sinks, size_t *bytes_out);

/*
 * Decode attention of one token per sequence (m = 1, q_lens = NULL) over all rows of its sequence,
 * which also accumulates the rows' attention weights:
 *   mass_out[b][h][j] = mass[b][h][j] + sum over the q-heads g of kv-head h of softmax_j(s_g)
 * for j < lens[b]; the other entries are not written. mass, mass_out: fp32 [batch][n_kv][rows];
 * they may be the same array, or not overlap.
 * Errors: as iskv_window_attn().
 */
int iskv_mass_decode(const iskv_exact_rows *rows, const iskv_exact_queries *q, const float *mass,
                     float *mass_out, void *ws, size_t ws_bytes, iskv_stream_t stream);
int iskv_mass_decode_workspace(const iskv_exact_rows *rows, const iskv_exact_queries *q,
                               size_t *bytes_out);

/*
 * Eviction: every (sequence, kv-head) that holds more than `budget` rows keeps that many, in its
 * slots 0 .. budget - 1. It keeps the rows of positions < sinks, the rows whose position is among
 * the `recent` last up to its largest one, and the heaviest of the others (ties: the lowest slot;
 * a NaN counts as heaviest). Kept rows of slots >= budget move into the freed slots below it, both
 * in ascending order; the other rows stay where they are, so slots are in no order of positions.
 * k and v are moved in place. mass fp32 and pos int32, [batch][n_kv][rows], hold each row's weight
 * and position (distinct within a kv-head); mass_out, pos_out and lens_out (device, [batch]) get
 * what the kept rows have, entries behind them are not written. Each may be its input (in place)
 * or not overlap it. sinks + recent <= budget.
 * Errors: as iskv_window_attn().
 */
int iskv_evict(const iskv_exact_rows *rows, const float *mass, float *mass_out, const int *pos,
               int *pos_out, int *lens_out, int budget, int recent, int sinks, void *ws,
               size_t ws_bytes, iskv_stream_t stream);
int iskv_evict_workspace(const iskv_exact_rows *rows, int budget, size_t *bytes_out);

/*
 * Decode attention of one token per sequence (m = 1, q_lens = NULL) over a prefix that the whole
 * batch shares, and then its sequence's own rows (capacity 0 allowed). The prefix's keys and values
 * are read once for a group of sequences, not once per sequence.
 * Errors: as iskv_window_attn().
 */
int iskv_prefix_decode(const iskv_exact_rows *rows, const iskv_exact_queries *q,
                       const iskv_exact_prefix *prefix, void *ws, size_t ws_bytes,
                       iskv_stream_t stream);
int iskv_prefix_decode_workspace(const iskv_exact_rows *rows, const iskv_exact_queries *q,
                                 const iskv_exact_prefix *prefix, size_t *bytes_out);

/*
 * Synchronises `stream` and returns the sticky status of the calls on exact caches on the current
 * device since the last such query: ISKV_OK, or ISKV_ERR_TIMEOUT when a device-side wait of one of
 * them hit its bound (its outputs are then incomplete), or ISKV_ERR_CUDA.
 */
int iskv_exact_status(iskv_stream_t stream);

/*
 * Polls, of up to 20 us each, after which a device-side wait of the calls on exact caches gives up: for
 * all calls of the process from now on, on all devices. ISKV_EXACT_POLLS (5 s) until it is called; 0: a wait
 * gives up at once, which shows what a program does with the status. A call whose waits give up returns
 * when its copies and products in flight have ended; what it has written is within its outputs.
 * Errors: ISKV_ERR_INVALID_ARG (negative).
 */
#define ISKV_EXACT_POLLS (1 << 18)
int iskv_exact_wait_limit(int polls);

/* Static description of an error code. */
const char *iskv_strerror(int code);

#ifdef __cplusplus
}
#endif

#endif /* ISKV_H */
