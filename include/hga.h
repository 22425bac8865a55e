/*
 * hga.h — C ABI of the B200 (sm_100a) library for Hierarchical Global
 * Attention (HGA): routed exact-token causal attention.
 *
 * Sources.  The operations follow the HGA paper-review page ("HGA:
 * Hierarchical Global Attention — Drop-In Exact-Token Routing for Pretrained
 * Long-Context Transformers", xllm-io), section 3 (技术架构): the mixed-RoPE
 * summary formula, the routing policy (deterministic visibility, middle
 * routing, the selection equation M_sel = topK_c, G_sel = topK_g), exact
 * token output attention (eq. (1) restricted to the routed set) and the
 * store's four operations (append closed chunk, read chunk summaries, fetch
 * group summaries, gather token K/V, section "三层 K/V 存储").  The
 * gist.science page "Hierarchical Global Attention (HGA)", technical summary,
 * "Core Mechanism", restates the same mechanism.
 *
 * Conventions for every call.
 *  - Pointers are DEVICE pointers (cudaMalloc / PyTorch CUDA memory) unless a
 *    comment says host.  The caller owns every buffer; the library allocates
 *    nothing and keeps no pointer after a call returns.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  Work is enqueued asynchronously; no call synchronises the host
 *    except where stated.
 *  - Layouts are dense row-major with the last index fastest:
 *      Q, O      [B, T, Hq,  D]      query head hq uses KV head hq / (Hq/Hkv)
 *      K, V, K_rot [B, T, Hkv, D]    K is the RAW (pre-RoPE) key projection
 *      pos       [B, T] int32        RoPE positions (any values; causality
 *                                    follows the token index, not pos)
 *      s_chunk   [B, Hkv, NC, D] f32 NC = T / C closed chunks (a partial last
 *                                    chunk is open and has no summary)
 *      s_group   [B, Hkv, NC*C/g_s, D] f32, group j of chunk m at m*C/g_s + j
 *      sel_chunk [B, NB, Hkv, K_c] int32, NB = ceil(T / C) query blocks
 *      sel_group [B, NB, Hkv, K_g] int32 global group ids
 *      lse       [B, Hq, T] f32      natural-log softmax denominators
 *    Selected ids are ascending and padded with -1.
 *  - dtype (hga_dims.dtype) is the element type of Q, K, V, K_rot and O:
 *    HGA_F32 or HGA_BF16.  Summaries, scores and accumulation are fp32 or
 *    wider.
 *  - Every tensor pointer (inputs, outputs, caches, summaries) must be
 *    16-byte aligned; another base is HGA_ERR_INVALID_ARG.
 *  - Errors: arguments are checked on the host first; a failing check
 *    returns HGA_ERR_INVALID_ARG or HGA_ERR_UNSUPPORTED and launches nothing.
 *    Size limits of this build (HGA_ERR_UNSUPPORTED beyond them): B <= 65535,
 *    Hkv <= 65535, and B * T (B * capacity for a K/V cache) below 2^31.
 *    A launch failure returns HGA_ERR_CUDA (the CUDA error is not cleared by
 *    the library; hga_last_cuda_error() gives its code).
 */
#ifndef HGA_H
#define HGA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum hga_status {
    HGA_OK = 0,
    HGA_ERR_INVALID_ARG = 1,   /* a null pointer, a bad size or a bad layout */
    HGA_ERR_UNSUPPORTED = 2,   /* valid, but not a shape this build handles  */
    HGA_ERR_CUDA = 3,          /* a CUDA launch or copy failed               */
    HGA_ERR_TIMEOUT = 4,       /* a bounded device wait gave up              */
    HGA_ERR_BOUNDS = 5,        /* a device-side index check failed           */
    HGA_ERR_WORKSPACE = 6      /* workspace missing or smaller than required */
} hga_status;

typedef enum hga_dtype { HGA_F32 = 0, HGA_BF16 = 1 } hga_dtype;

typedef enum hga_mode {
    HGA_PREFILL = 0, HGA_DECODE = 1, HGA_PREFILL_HOSTKV = 2,
    HGA_ATTEND_BACKWARD = 3     /* hga_workspace_size only: hga_attend_backward */
} hga_mode;

/* Method parameters (page section 3 and its setup table in section 6). */
typedef struct hga_params {
    int32_t C;            /* chunk length in tokens; this build needs C == 64,
                             which is also the prefill query block            */
    int32_t g_s;          /* group length; divides C                          */
    int32_t F;            /* sink chunks 0..F-1, always visible               */
    int32_t L;            /* recent closed chunks, always visible; with L == 0
                             the previous chunk is still forced visible       */
    int32_t K_c;          /* middle chunks routed per block and KV head (>=0) */
    int32_t K_g;          /* groups opened inside those chunks (>= 0)         */
    double rope_theta;    /* RoPE base: omega_i = theta^(-2i/D), pair (i, i+D/2) */
    double hf_wavelength; /* pair i is high-frequency iff 2*pi/omega_i is below
                             this; <= 0 selects C; +inf makes every pair high */
} hga_params;

/* Problem shape. */
typedef struct hga_dims {
    int32_t B;      /* sequences                                              */
    int32_t T;      /* prefill: tokens per sequence; decode: cache capacity   */
    int32_t Hq;     /* query heads, a multiple of Hkv                         */
    int32_t Hkv;    /* key/value heads                                        */
    int32_t D;      /* head dimension: 64 or 128                              */
    int32_t dtype;  /* hga_dtype                                              */
} hga_dims;

/* Decode state, all device memory owned by the caller, for `capacity` tokens
 * per sequence (Tc below; a multiple of C).  hga_forward(HGA_PREFILL) fills
 * it when io.cache.k_rot is non-NULL; every hga_forward(HGA_DECODE) appends
 * one token per sequence and increments lens. */
typedef struct hga_kv_cache {
    int32_t capacity;  /* Tc                                                  */
    void *k_rot;       /* [B, Tc, Hkv, D] rotated keys                        */
    void *v;           /* [B, Tc, Hkv, D] values                              */
    int32_t *pos;      /* [B, Tc] positions of the cached tokens              */
    void *k_open;      /* [B, Hkv, C, D] raw keys of each sequence's open chunk
                          (needed for the low-frequency pairs when it closes) */
    float *s_chunk;    /* [B, Hkv, Tc/C, D]                                   */
    float *s_group;    /* [B, Hkv, Tc/g_s, D]                                 */
    int32_t *lens;     /* [B] tokens already cached                           */
} hga_kv_cache;

/* Inputs and outputs of hga_forward.  Unused members must be NULL. */
typedef struct hga_io {
    /* HGA_PREFILL */
    const void *q;             /* [B, T, Hq, D]                                */
    const void *k;             /* [B, T, Hkv, D] raw keys                      */
    const void *v;             /* [B, T, Hkv, D]                               */
    const int32_t *pos;        /* [B, T]                                       */
    /* HGA_DECODE: one new token per sequence, at index lens[b]               */
    const void *q_new;         /* [B, Hq, D]                                   */
    const void *k_new;         /* [B, Hkv, D] raw key                          */
    const void *v_new;         /* [B, Hkv, D]                                  */
    const int32_t *pos_new;    /* [B]                                          */
    /* outputs */
    void *out;                 /* prefill [B, T, Hq, D]; decode [B, Hq, D]     */
    float *lse;                /* optional: prefill [B, Hq, T]; decode [B, Hq] */
    int32_t *sel_chunk;        /* optional: prefill [B, NB, Hkv, K_c];
                                  decode [B, Hkv, K_c]                         */
    int32_t *sel_group;        /* optional: prefill [B, NB, Hkv, K_g];
                                  decode [B, Hkv, K_g]                         */
    hga_kv_cache cache;        /* decode: required; prefill: optional output   */
    /* HGA_PREFILL_HOSTKV only, optional: a HOST pointer to pinned, mapped
     * memory [B, Hkv, NC*C/g_s, D] f32 that holds the group summaries in the
     * cold tier (page section 3's store table puts them in host RAM beside
     * the token K/V).  Stage 1 writes them there over the link and stage 2
     * reads only the groups of each block's routed chunks over the link
     * (store operation "fetch group summaries"); NULL keeps them in the
     * workspace on the GPU. */
    float *s_group_host;
} hga_io;

/* Stage 1 — rotate keys and build mixed-RoPE summaries ("append closed
 * chunk").  Page section 3, "Mixed-RoPE Routing Summaries": for each closed
 * chunk and each g_s-token group, high-frequency pairs are the mean of the
 * per-token rotated keys; low-frequency pairs are the mean raw key rotated at
 * the set's mean position.  Also writes K_rot = RoPE(K) for attention.
 * k_rot may be NULL (summaries only).  Shapes as in the header comment. */
hga_status hga_build_summaries(const hga_dims *dims, const hga_params *prm,
                               const void *k_raw, const int32_t *pos,
                               void *k_rot, float *s_chunk, float *s_group,
                               void *stream);

/* Stage 2 — two-level routing per 64-token query block and KV head.  Page
 * section 3, "路由策略" (routing policy) and the selection equation: the
 * routing query is the block's RoPE-rotated queries summed over its tokens and
 * over the KV head's query heads; middle chunks F..b-L-1 (minus the forced
 * previous chunk when L == 0) are scored by q.c_m, the top K_c kept, their
 * groups scored by q.g_{m,g} and the top K_g kept.  Ties in score go to the
 * lower index.  Outputs sel_chunk / sel_group as in the header comment.
 * q_rot (bf16 only, may be NULL; HGA_ERR_UNSUPPORTED for fp32): when given,
 * [B, T, Hq, D] bf16 receives every query rotated at its position, rounded
 * as hga_attend rounds its own rotation, for hga_attend's q_rot. */
hga_status hga_route(const hga_dims *dims, const hga_params *prm,
                     const void *q, const int32_t *pos,
                     const float *s_chunk, const float *s_group,
                     int32_t *sel_chunk, int32_t *sel_group, void *q_rot, void *stream);

/* Stage 3 — exact softmax attention over the routed token set.  Page section
 * 3, "精确 Token 输出注意力" (exact token output attention) with eq. (1): each
 * query token i of block b attends, with scale 1/sqrt(D), to the union of
 * sink chunks 0..F-1, recent chunks b-L..b-1, chunk b-1, the tokens of
 * sel_group, and tokens b*C..i of its own chunk.  q is raw (pre-RoPE) and is
 * rotated inside; k_rot comes from hga_build_summaries.  lse may be NULL.
 * q_rot (bf16 only, may be NULL): the rotated queries hga_route wrote; the
 * tensor-core kernel then loads them as they are instead of rotating q (the
 * result is bit-identical), q is still required for the CUDA-core kernel.
 * Which kernel runs: bf16 with Hq/Hkv a power of two <= 16, g_s a multiple
 * of 8 and a visible set of at most 2048 8-token segments runs on the tensor
 * cores (tcgen05): with q_rot given, Hq/Hkv >= 4 and at most 1024 segments
 * as one persistent CTA per SM walking the (block, KV head, 256-row) units,
 * else one CTA per unit; fp32, and bf16 outside those limits, run on the
 * CUDA cores in fp32 arithmetic.  Both give the same result within rounding (bf16
 * outputs are rounded from fp32 accumulators). */
hga_status hga_attend(const hga_dims *dims, const hga_params *prm,
                      const void *q, const int32_t *pos,
                      const void *k_rot, const void *v,
                      const int32_t *sel_group, void *out, float *lse,
                      const void *q_rot, void *stream);

/* Backward of stage 3 (training through the routed attention).  Page
 * section 6, Tab. 8 (a training step through HGA attention) and Sec. 5.9
 * (QK fine-tuning through it in the exact-token mode).  The page prints no
 * formula; this is the derivative of eq. (1) restricted to each query's
 * visible set, the routed groups held fixed (routing is a discrete choice, so
 * no gradient reaches the summaries):
 *   P_ij = exp(q~_i . k~_j / sqrt(D) - LSE_i) over j in V(i) (q~, k~ rotated)
 *   dv_j = sum_i P_ij dO_i
 *   dS_ij = P_ij (dO_i . v_j - Delta_i),  Delta_i = sum_j P_ij dO_i . v_j
 *   dq_i = R_{p_i}^T sum_j dS_ij k~_j / sqrt(D)
 *   dk_j = R_{p_j}^T sum_i dS_ij q~_i / sqrt(D)
 * with i over the query rows of every query head of k_j's KV head.  Delta_i
 * equals dO_i . O_i; the library forms it from its own P and dO . v, so the
 * forward output is not an input (with a rounded output, the cancellation in
 * dO . v_j - Delta_i on rows whose weight sits on few keys would magnify its
 * rounding error).
 * Inputs: q (raw), pos, k_rot, v and sel_group as given to hga_attend; lse as
 * hga_attend returned it (required); d_out [B, T, Hq, D] in the dtype of q;
 * q_rot (bf16, may be NULL) the rotated queries hga_route wrote for the
 * forward, which spares the backward rotating q again (same results).  Outputs, fp32: dq [B, T, Hq, D] with respect to the raw
 * q, dk [B, T, Hkv, D] with respect to the RAW k (the rotation undone at each
 * key's position), dv [B, T, Hkv, D]; every element is written.  workspace:
 * hga_workspace_size(HGA_ATTEND_BACKWARD) bytes, 256-byte aligned.  bf16 with
 * the tensor-core forward's shape limits runs on the tensor cores (tcgen05),
 * everything else on the CUDA cores.  dk and dv are sums over units formed by
 * atomic additions, so their low bits may differ between runs. */
hga_status hga_attend_backward(const hga_dims *dims, const hga_params *prm,
                               const void *q, const int32_t *pos, const void *k_rot,
                               const void *v, const int32_t *sel_group, const float *lse,
                               const void *d_out, const void *q_rot, float *dq, float *dk,
                               float *dv, void *workspace, size_t workspace_bytes,
                               void *stream);

/* Bytes of device workspace hga_forward (or, for HGA_ATTEND_BACKWARD,
 * hga_attend_backward) needs for `mode` (0 if none).  For HGA_PREFILL this
 * includes room for the rotated queries stage 2 hands to stage 3 (bf16
 * shapes of the tensor-core attention); hga_forward(HGA_PREFILL) also accepts
 * a workspace of hga_prefill_workspace_min bytes and then rotates the
 * queries inside stage 3 instead (same results). */
size_t hga_workspace_size(int mode, const hga_dims *dims, const hga_params *prm);

/* The smallest workspace hga_forward(HGA_PREFILL) accepts (0 if the
 * arguments are malformed): rotated keys, summaries and routed ids only. */
size_t hga_prefill_workspace_min(const hga_dims *dims, const hga_params *prm);

/* The whole path in one call.
 * HGA_PREFILL: stages 1-3 over the T prompt tokens (K_rot, summaries and
 *   selections live in the workspace unless io.cache / io.sel_* are given).
 *   With io.cache.k_rot set (capacity >= T), the cache is filled for decoding:
 *   K_rot, V, pos, summaries, the open chunk's raw keys, and lens = T.  With
 *   the cache set and io.q and io.out both NULL, only the cache is filled
 *   (stage 1; no routing or attention is computed).
 * HGA_DECODE: dims.T must equal io.cache.capacity.  For each sequence b, appends the new token at t = lens[b]
 *   (rotated key, value, position, raw key of the open chunk), builds the
 *   summaries of chunk t/C if t closes it (page section 3, store operation
 *   "append closed chunk"), routes with the token's own query (summed over the
 *   KV head's query heads), attends over the visible set of token t and
 *   increments lens[b].  Requires lens[b] < dims.T.  The attention over the
 *   keys routing does not choose (sinks, recent and current chunks) runs on
 *   a library-owned side stream (one per device, created on the first decode
 *   call) forked from and joined back into `stream` inside the call, so the
 *   caller sees ordinary stream order and can capture steps in a CUDA graph.
 * HGA_PREFILL_HOSTKV: the prefill of HGA_PREFILL with the token K/V history
 *   in host RAM (page section 3, the three-tier K/V store: the summaries stay
 *   on the GPU and only routed groups are fetched).  io.k and io.v are HOST
 *   pointers to pinned, mapped memory (cudaHostAlloc / cudaMallocHost /
 *   cudaHostRegister with mapping) holding raw K and V [B, T, Hkv, D]; q,
 *   pos and out (and lse, sel_chunk, sel_group when given) are device
 *   pointers; io.cache must be empty.  bf16 only, shapes the tensor-core
 *   attention takes (g_s a multiple of 8, Hq/Hkv a power of two <= 16).
 *   Stage 1 reads K over the host link once (with io.s_group_host set, it
 *   also writes the group summaries there, and stage 2 reads the routed
 *   chunks' group rows from there); stage 3 runs in waves of 32
 *   query blocks whose sink, recent and current K/V rows are fetched by the
 *   GPU over the link into two HBM staging buffers in the workspace, and
 *   whose routed groups go through a warm tier: a cache of routed groups in
 *   the workspace (page section 3's warm VRAM tier; CLOCK replacement) from
 *   which hits are read and into which misses are fetched.  The wave size
 *   and the cache's slots follow the workspace size (hga_hostkv_plan_for):
 *   by default 32 blocks and two waves' worth of groups per sequence and KV
 *   head (or all of them when fewer).
 *   This runs on a library-owned side stream (one per device, created on
 *   the first such call), the next wave's fetch overlapping this wave's
 *   attention; the call joins that stream back into `stream` before
 *   returning, so the caller sees ordinary stream order.  The cache lives
 *   for one call.  Host memory that is not pinned and
 *   mapped returns HGA_ERR_INVALID_ARG.  The outputs equal HGA_PREFILL's.
 * workspace: hga_workspace_size(mode) bytes of device memory, 256-byte
 * aligned (HGA_PREFILL_HOSTKV: any size from the plan's min_bytes up; see
 * hga_hostkv_plan_for).  For HGA_DECODE it must be zero-filled before its first use; the
 * library leaves it zeroed between calls.  Calls that share a workspace must
 * not overlap on the GPU. */
hga_status hga_forward(int mode, const hga_dims *dims, const hga_params *prm,
                       const hga_io *io, void *workspace, size_t workspace_bytes,
                       void *stream);

/* hga_forward(HGA_PREFILL) for callers that cannot allocate device memory.
 * The paper has no counterpart to this call: it is a convenience of this
 * library.  It is meant for code that only holds its inputs and outputs at
 * call time and may not call cudaMalloc then, for example a serving step
 * whose device memory belongs to another allocator or to a fixed arena
 * (a cudaMalloc there can fail, or stall the device mid-step), or a plug-in
 * that a host runtime hands nothing but tensors.
 *
 * Arguments are those of hga_forward(HGA_PREFILL) without a workspace: q, k,
 * v, pos and out as in the header comment, lse optional (NULL to skip).  The
 * scratch (rotated keys, summaries, routed ids) lives in one fixed 16 MiB
 * array inside the library's device image, which every GPU that loads the
 * library keeps until the process exits.  A shape whose scratch
 * (hga_prefill_workspace_min) exceeds 16 MiB is rejected with
 * HGA_ERR_WORKSPACE before anything is launched; about 14K tokens fit at
 * Hkv=4, D=128, bf16.  Nothing in the scratch needs to start at zero.
 *
 * The first call on a device, with that device current, looks up the
 * array's device address (cudaGetSymbolAddress) and caches it; make that
 * first call before any stream capture.  The cached address belongs to the
 * device's primary context as it was then: after cudaDeviceReset on that
 * device the address is stale, so do not call this entry point on a device
 * after resetting it (load the library in a fresh process instead).  All
 * calls share the one array:
 * calls that overlap on the GPU (other streams, other threads, without
 * ordering between them) race on it and give wrong results. */
hga_status hga_forward_prefill_noalloc(const hga_dims *dims, const hga_params *prm,
                                       const void *q, const void *k, const void *v,
                                       const int32_t *pos, void *out, float *lse, void *stream);

/* How HGA_PREFILL_HOSTKV uses a workspace of a given size: the warm tier
 * (page section 3's bounded VRAM cache of routed groups, which shrinks to
 * leave a configurable VRAM headroom) takes whatever the caller's workspace
 * holds.  hga_workspace_size(HGA_PREFILL_HOSTKV) is the default: waves of 32
 * query blocks and a cache of two waves' worth of routed groups per
 * (sequence, KV head).  A larger workspace keeps more groups cached (fewer
 * link bytes), up to every group of the sequence (max_bytes); a smaller one
 * shrinks the wave, and with it the staging buffers and the cache's floor of
 * two waves' worth, down to one query block per wave (min_bytes).  Outputs
 * are the same for every plan.  A caller that wants a headroom sizes the
 * workspace as the free device memory minus the headroom, clamped to
 * [min_bytes, max_bytes]. */
typedef struct hga_hostkv_plan {
    int32_t wave_blocks;   /* query blocks per wave                            */
    int32_t cache_slots;   /* warm-cache slots (one routed group each) per
                              (sequence, KV head)                              */
    size_t bytes;          /* workspace bytes this plan uses (0 if none fits)  */
    size_t min_bytes;      /* the smallest workspace any plan fits in          */
    size_t max_bytes;      /* the workspace that caches every group            */
} hga_hostkv_plan;

/* The plan hga_forward(HGA_PREFILL_HOSTKV) follows for workspace_bytes.
 * Host only.  Returns HGA_ERR_WORKSPACE (with min_bytes filled in) when the
 * workspace is below min_bytes; *plan must be a host pointer. */
hga_status hga_hostkv_plan_for(const hga_dims *dims, const hga_params *prm,
                               size_t workspace_bytes, hga_hostkv_plan *plan);

/* ---------------------------------------------------------- paged cache --
 *
 * Layers that attend over every cached token, or over a token window, keep
 * their keys and values in pages: a pool of num_pages pages of page_size
 * tokens, [num_pages, page_size, Hkv, D] for the rotated keys and the same for
 * the values, and a block table [B, max_pages] whose entry j is the page that
 * holds the tokens j*page_size .. of sequence b.  The slot of a token is its
 * page * page_size + its place in the page.  hga_paged_plan builds the table
 * and the slots of a step, hga_qk_norm_rope writes keys and values through the
 * slots, hga_paged_decode attends over the table.  Nothing here reads a length
 * on the host, so a serving step can be captured in a CUDA graph.
 *
 * Limits: B at least 1 (an empty batch is the caller's to skip); page_size a
 * power of two; num_pages * page_size, max_pages * page_size and B * max_pages
 * below 2^31; B and Hq at most 65535; D 64 or 128; for hga_paged_decode also B * Hkv * max_pages * page_size (max_pages * page_size
 * at most window + sinks with a window) below 2^36.
 * eps, magnitude and scale are taken in fp32: 0 or a normal number there (about
 * 1.2e-38 to 3.4e38; scale times log2 e).
 * int32 buffers need 4-byte alignment, rows of q, k, v, pages and gradients
 * 16-byte alignment.  Outputs must not overlap inputs except where stated, and
 * calls that share a workspace must not overlap on the GPU. */
typedef struct hga_paged_dims {
    int32_t B;          /* sequences: rows of the block table, of lens and of q */
    int32_t Hq, Hkv, D; /* as in hga_dims                                       */
    int32_t dtype;      /* hga_dtype of q, pages and out                        */
    int32_t num_pages;  /* pages in the pool                                    */
    int32_t page_size;  /* tokens per page                                      */
    int32_t max_pages;  /* columns of the block table                           */
} hga_paged_dims;

/* One step's plan.  All device pointers. */
typedef struct hga_paged_plan_io {
    const int32_t *lens;        /* [B] tokens each sequence holds               */
    const int32_t *new_tokens;  /* [B] tokens this step adds, >= 0              */
    const int32_t *release;     /* [B] or NULL: nonzero empties the row first   */
    int32_t *free_pages;        /* [num_pages] stack of free page ids           */
    const int32_t *free_count;  /* [1] entries on the stack; the top is the last */
    int32_t *block_table;       /* [B, max_pages], new pages written in place   */
    int32_t *lens_out;          /* [B] lens + granted; may be lens              */
    int32_t *free_count_out;    /* [1]; may be free_count                       */
    int32_t *cu_tokens;         /* [B + 1] exclusive sums of new_tokens         */
    int32_t *granted;           /* [B] new_tokens[b], or 0 if refused           */
    int32_t *slot;              /* [n_slots] slot of every packed new token     */
    int32_t *pos;               /* [n_slots] its index in its sequence          */
} hga_paged_plan_io;

/* Block table, slot map and positions of one step, from the lengths alone.
 * Rows with release[b] != 0 give their pages back first (rows in order, their
 * pages in order) and count as empty.  Sequence b then needs
 * ceil((lens+new)/page_size) - ceil(lens/page_size) pages; sequences are served
 * in order, and page i of b's is the i-th from the top of what the sequences
 * before it left.  A sequence is refused (granted 0, its length and row left as
 * they are, its tokens' slots -1) when lens+new exceeds max_pages * page_size,
 * when its packed tokens end beyond n_slots, or when it needs pages and the
 * demand up to and including it exceeds the stack; one that needs no page is
 * never refused for want of pages.  Packed token t of sequence b
 * (cu_tokens[b] <= t < cu_tokens[b+1]) has position lens + t - cu_tokens[b];
 * entries from cu_tokens[B] to n_slots get slot -1 and position 0, so a step of
 * fewer tokens can replay a graph of n_slots.  Pages are not counted: a page that
 * several rows hold (a shared prefix may be read so) must not be given back by more
 * than one of them, nor be one that a row still writes to.  Of dims, B, num_pages, page_size
 * and max_pages are read.
 * A negative length or count, a length beyond the row, a stack size outside
 * [0, num_pages], a page id outside [0, num_pages) and a release that would
 * overfill the stack are refused by the kernel: the row or the entry is left
 * out and hga_device_status reports HGA_ERR_BOUNDS.
 * workspace: hga_paged_plan_workspace(B, n_slots) bytes, 256-byte aligned; it
 * needs no initial value. */
hga_status hga_paged_plan(const hga_paged_dims *dims, const hga_paged_plan_io *io, int32_t n_slots,
                          void *workspace, size_t workspace_bytes, void *stream);
size_t hga_paged_plan_workspace(int32_t B, int32_t n_slots);

typedef enum hga_rope_layout { HGA_ROPE_HALF = 0, HGA_ROPE_INTERLEAVED = 1 } hga_rope_layout;
typedef enum hga_rope_scaling {
    HGA_ROPE_UNSCALED = 0, HGA_ROPE_LINEAR = 1, HGA_ROPE_YARN = 2
} hga_rope_scaling;

/* A position rotation.  Pair i < R/2 of the first R = rotary_dim dimensions is
 * (i, i + R/2) in the half layout and (2i, 2i + 1) in the interleaved one, and
 * turns by p * w_i; dimensions R.. pass through.  w_i = theta^(-2i/R), and
 *  LINEAR: w_i / factor;
 *  YARN:   w_i (1 - g_i) + w_i / factor * g_i with g_i = clamp((i - lo) /
 *          (hi - lo), 0, 1), lo = max(0, floor(d(beta_fast))), hi =
 *          min(R - 1, ceil(d(beta_slow))) (hi = lo + 0.001 if equal), d(t) =
 *          R ln(original_len / (2 pi t)) / (2 ln theta): pairs that turn more
 *          than beta_fast times over the original length keep their rate.
 *          hi < lo (all pairs on one side of the ramp) is refused.
 * The rotated part is multiplied by `magnitude`; 0 selects 1, for YARN
 * 0.1 ln(factor) + 1. */
typedef struct hga_rope {
    int32_t layout;        /* hga_rope_layout                                    */
    int32_t rotary_dim;    /* R: a multiple of 16 up to D; 0 = no rotation       */
    int32_t scaling;       /* hga_rope_scaling                                   */
    int32_t original_len;  /* YARN: the trained length                           */
    double theta, factor, beta_fast, beta_slow, magnitude;
} hga_rope;

/* Inputs and outputs of hga_qk_norm_rope.  q, k, v are [tokens, H, D] with the
 * heads of a token D apart and tokens *_stride elements apart (a multiple of 16
 * bytes, at least H*D), so views of a fused QKV buffer are read as they are. */
typedef struct hga_qk_io {
    const void *q, *k, *v;             /* raw projections; v may be NULL          */
    int64_t q_stride, k_stride, v_stride;
    const void *q_weight, *k_weight;   /* [D] norm weights; NULL: not normalised  */
    double eps;                        /* of the norms, >= 0                      */
    const int32_t *pos;                /* [tokens]; may be NULL if rotary_dim == 0 */
    void *q_out, *k_out, *v_out;       /* dense [tokens, H, D]; each may be NULL   */
    const int32_t *slot;               /* [tokens], with k_pages and v_pages       */
    void *k_pages, *v_pages;           /* [num_pages, page_size, Hkv, D] or NULL   */
    int64_t num_slots;                 /* num_pages * page_size                    */
} hga_qk_io;

/* Per-head RMS norms of queries and keys and the position rotation, in one pass
 * over the projections: y = R_p (x (mean x^2 + eps)^(-1/2) weight), computed in
 * fp32 and rounded once (a normed row of values above about 1e19, whose squares
 * pass fp32, comes out as zeros).  dims.B * dims.T tokens, below 2^31 (dims.T may
 * be any count, 0 included).
 * With rotary_dim == 0 the outputs are what hga_forward takes as raw q, k and v;
 * rotated keys and values go to k_pages and v_pages at slot[t] for
 * hga_paged_decode.  A slot of -1 writes no page row; any other slot outside
 * [0, num_slots) writes none and hga_device_status reports HGA_ERR_BOUNDS.  The
 * slots of one call must differ from one another.  Rows of the dense outputs are
 * written for every token. */
hga_status hga_qk_norm_rope(const hga_dims *dims, const hga_rope *rope, const hga_qk_io *io,
                            void *stream);

/* Inputs and outputs of hga_qk_norm_rope_backward. */
typedef struct hga_qk_grad_io {
    const void *q, *k;                 /* the forward's raw inputs (unused rows
                                          may be NULL with weights NULL)         */
    int64_t q_stride, k_stride;
    const void *q_weight, *k_weight;   /* as in the forward                       */
    double eps;
    const int32_t *pos;
    const void *d_q, *d_k, *d_v;       /* dense gradients of the dense outputs;
                                          d_v may be NULL                         */
    int32_t grad_dtype;                /* of d_q, d_k, d_v: HGA_F32 or dims.dtype */
    void *dq, *dk, *dv;                /* [tokens, H, D] in dims.dtype, strided;
                                          dv NULL exactly when d_v is             */
    int64_t dq_stride, dk_stride, dv_stride;
    float *d_q_weight, *d_k_weight;    /* [D], required exactly with the weights  */
} hga_qk_grad_io;

/* Gradients of hga_qk_norm_rope.  With g = R_p^T dy, r = (mean x^2 + eps)^(-1/2):
 *   d_weight_d = sum over tokens and heads of g_d x_d r
 *   dx = r (g w - x r^2 mean_d(g w x))      (g itself where not normalised)
 * and dv = d_v.  d_q, d_k, d_v may be the fp32 gradients of hga_attend_backward.
 * Sums are formed in a fixed order: the same inputs give the same bits.
 * workspace: hga_qk_norm_rope_backward_workspace(dims) bytes, 256-byte aligned;
 * it needs no initial value. */
hga_status hga_qk_norm_rope_backward(const hga_dims *dims, const hga_rope *rope,
                                     const hga_qk_grad_io *io, void *workspace,
                                     size_t workspace_bytes, void *stream);
size_t hga_qk_norm_rope_backward_workspace(const hga_dims *dims);

/* Attention of one new token per sequence over its pages.  q [B, Hq, D] is
 * rotated; sequence b attends, with `scale` (0 selects 1/sqrt(D)), to its tokens
 * j < lens[b], its own included; with window > 0 only to those with
 * j >= lens[b] - window or j < sinks.  out [B, Hq, D]; lse [B, Hq] f32 may be
 * NULL.  A sequence of length 0 gives zeros and an lse of -inf.  Pages that hold
 * no attended token are not read, and neither is what a last page holds behind
 * the length.  A length outside [0, max_pages * page_size] counts as 0, the keys
 * of a page id outside [0, num_pages) are left out, and hga_device_status
 * reports HGA_ERR_BOUNDS.
 * The work is split over sequences, heads and length by the lengths on the
 * device; partial results are joined in a fixed order, so the same inputs give
 * the same bits.  fp32 softmax statistics and sums; for bf16 a softmax weight
 * enters its product with the values as two bf16, good to 2^-15 of it.
 * workspace: hga_paged_decode_workspace(dims) bytes, 256-byte aligned; it needs
 * no initial value. */
hga_status hga_paged_decode(const hga_paged_dims *dims, const void *q, const void *k_pages,
                            const void *v_pages, const int32_t *block_table, const int32_t *lens,
                            int32_t window, int32_t sinks, double scale, void *out, float *lse,
                            void *workspace, size_t workspace_bytes, void *stream);
size_t hga_paged_decode_workspace(const hga_paged_dims *dims);

/* Status recorded by the kernels themselves since the last reset: a bounded
 * wait that gave up (HGA_ERR_TIMEOUT: the kernel recorded it, released what
 * it held and returned without finishing its tile) or a device-side index
 * check that refused an access (HGA_ERR_BOUNDS, e.g. a decode step for a
 * sequence whose lens[b] is outside [0, capacity); that sequence is skipped,
 * the others proceed).  Kernels never trap: a launch that met such a
 * condition still completes, and only this call reports it.  Waits for the
 * work already queued on `stream`, then reads the library's error words;
 * clear != 0 resets them.  Returns HGA_OK when none is set, the first set
 * status otherwise, or HGA_ERR_CUDA if the copies fail. */
hga_status hga_device_status(void *stream, int clear);

/* Bytes the host tier (HGA_PREFILL_HOSTKV) has moved over the host link
 * since the last reset: for stage 3 the K and V rows of sinks, windows and
 * the routed groups its warm cache did not hold; with the group summaries in
 * host memory also the summaries stage 1 wrote there and the group rows
 * stage 2 read (stage 1's single pass over K is not counted).  Waits for the work queued on `stream`; clear != 0 resets the
 * count.  *bytes must be a host pointer (HGA_ERR_INVALID_ARG if NULL). */
hga_status hga_hostkv_link_bytes(void *stream, unsigned long long *bytes, int clear);

/* Test hook, not for production use: exercises the bounded-wait timeout
 * path of a real kernel without a GPU fault.  With skip_summaries_copy != 0
 * the summaries kernel (stage 1, device-memory keys) does not issue the bulk
 * copy of its keys, so its wait for them runs out after summaries_wait_ns
 * (0 = the default limit of 2 s); the kernel then records HGA_ERR_TIMEOUT
 * (read by hga_device_status) and returns with nothing in flight, and its
 * outputs are left unwritten.  hga_set_test_hooks(0, 0, stream) restores
 * normal operation.  The settings are per device and apply to every call
 * that follows; the call waits for `stream`. */
hga_status hga_set_test_hooks(int skip_summaries_copy, unsigned long long summaries_wait_ns,
                              void *stream);

/* Static description of a status code. */
const char *hga_status_string(hga_status s);

/* The last CUDA error code seen by a failing call on this thread (0 = none). */
int hga_last_cuda_error(void);

#ifdef __cplusplus
}
#endif
#endif /* HGA_H */
