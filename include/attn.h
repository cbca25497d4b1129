/*
 * attn.h — C ABI of the GB300 (sm_103a) exact-attention library.
 *
 * Exact scaled-dot-product attention computed tile by tile with an online
 * softmax: per query row the kernels carry a running max m, a denominator l
 * and an output accumulator o, rescaled by exp(m_old - m_new) whenever a new
 * key tile raises the max, so the N x N score and probability matrices never
 * reach device memory ("Explain FlashAttention and why it is IO-aware",
 * "Keep only the state needed for the final weighted average"; "What is
 * FlashAttention?", Steps 2-3). The backward pass recomputes the score and
 * probability tiles from Q, K, V, O and the saved per-row log-sum-exp
 * ("What is FlashAttention?", Step 4; "FlashAttention", "What it does not do").
 *
 * Conventions shared by every entry point:
 *  - Tensors Q, K, V, O (and dO, dQ, dK, dV) are logically [B, H, N, d] with
 *    the last dimension contiguous; the three strides given for (b, h, n) are
 *    in ELEMENTS and may describe any permutation of B/H/N (e.g. BHND or
 *    BNHD). Base pointers and every stride in bytes must be multiples of 16.
 *  - LSE is float32 [B, H, N], contiguous (row-major).
 *  - The caller owns all memory. The library allocates no device memory; the
 *    backward pass uses a caller-provided workspace whose size
 *    attn_bwd_workspace_size() reports.
 *  - Calls are asynchronous on the given stream (a cudaStream_t passed as
 *    void*; NULL is the legacy default stream). Argument errors are found on
 *    the host before anything is launched and are returned directly, with a
 *    message from attn_last_error(). Errors inside a kernel (a bounded wait
 *    that ran out) are recorded in a device error word and reported by the
 *    next attn_status() on that device.
 *  - Launch chaining: the tensor-core kernels and the backward's and decode's
 *    helper kernels are launched with programmatic stream serialization.
 *    Such a kernel may start its on-chip set-up while the kernel before it
 *    on the stream is still finishing. Before it touches device memory it
 *    waits until that kernel has completed and its writes are visible. Stream
 *    order is therefore kept exactly; only the launch gap shrinks.
 *  - Values: Q, K, V and the mask must be finite, except that mask entries
 *    may be -inf ("masked"). NaN or +inf inputs give undefined results (the
 *    pages' row recurrence rejects them up front: "Explain FlashAttention and
 *    why it is IO-aware", "Executable recurrence, with an empty-state
 *    policy"). A query row whose every score is -inf (fully masked) returns
 *    O = 0 and LSE = -inf, and contributes nothing to the gradients (same
 *    section's empty-row policy).
 *  - Empty problems (B, H or N equal to 0) are accepted and do nothing.
 */
#ifndef ATTN_GB300_ATTN_H
#define ATTN_GB300_ATTN_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define ATTN_API __attribute__((visibility("default")))
#else
#define ATTN_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum attn_status_t {
    ATTN_OK = 0,
    ATTN_ERR_INVALID = -1,     /* null pointer, negative size, bad flag or stride */
    ATTN_ERR_UNSUPPORTED = -2, /* well-formed but not built: head dim, dtype pairing, size limit */
    ATTN_ERR_ALIGN = -3,       /* a base pointer or byte stride is not a multiple of 16 */
    ATTN_ERR_CUDA = -4,        /* a CUDA runtime or driver call failed */
    ATTN_ERR_TIMEOUT = -5,     /* a kernel's bounded wait ran out (reported by attn_status) */
    ATTN_ERR_WORKSPACE = -6    /* backward workspace missing or smaller than required */
} attn_status_t;

typedef enum attn_dtype_t {
    ATTN_BF16 = 0, /* bfloat16 storage, fp32 accumulation (tcgen05 tensor cores) */
    ATTN_F32 = 1,  /* float32 storage and arithmetic (CUDA cores; forward only)   */
    ATTN_F16 = 2,  /* IEEE half storage, fp32 accumulation (tcgen05 tensor cores);
                      P, dS and O are rounded to half as bf16 rounds them for bf16 */
    ATTN_E4M3 = 3  /* 8-bit E4M3 Q, K, V with per-tensor descale factors; the FP8
                      forward (attn_fwd_fp8) only, whose O is bf16 */
} attn_dtype_t;

/*
 * Forward problem. O = softmax(scale * Q K^T + mask, causal) V and
 * LSE = log(sum_j exp(s_ij)) over the scaled, masked scores of each row
 * ("Explain FlashAttention and why it is IO-aware", "Keep only the state
 * needed for the final weighted average").
 */
typedef struct attn_fwd_params {
    int32_t B, H, N, d;      /* batch, heads, sequence length, head dim: 64 or 128;
                                256 for bf16 / fp16 (forward and attn_bwd) */
    int32_t dtype;           /* attn_dtype_t of Q, K, V, O (and the mask) */
    int32_t causal;          /* 1: key j is masked for query i iff j > i (absolute
                                positions, 0-based; same N for queries and keys) */
    float scale;             /* softmax scale, > 0; 1/sqrt(d) is the usual choice */
    int32_t reserved0;       /* must be 0 */
    const void *q, *k, *v;   /* inputs, device memory */
    void *o;                 /* output, device memory, same dtype as q */
    float *lse;              /* output, device memory, float32 [B, H, N] */
    int64_t q_stride[3];     /* element strides of (b, h, n) */
    int64_t k_stride[3];
    int64_t v_stride[3];
    int64_t o_stride[3];
    const void *mask;        /* optional additive mask, same dtype as q, logically
                                [B, H, N, N] (query row, key column); NULL = none */
    int64_t mask_stride[3];  /* element strides of (b, h, row); 0 broadcasts over
                                that index; the key column is contiguous */
} attn_fwd_params;

/*
 * Backward problem: dQ, dK, dV of sum(dO * O) for the forward described by
 * `fwd`, whose o and lse (as written by attn_fwd) are READ here. Recomputes
 * S and P tile by tile; no gradient flows to the mask. bf16 and fp16 at
 * head dim 64, 128 or 256 (ATTN_F32 returns ATTN_ERR_UNSUPPORTED). At head
 * dim 256 the fp32 dK and dV of one key tile would fill tensor memory, so
 * each key tile is handled by two CTAs, one per half of the head dimension,
 * each recomputing the scores over the whole head dimension: 7/5 of the
 * minimal tensor-core work. ("What is FlashAttention?", "Trade-offs and edge
 * cases": FlashAttention-2 covers head dims up to 256.)
 */
typedef struct attn_bwd_params {
    attn_fwd_params fwd;
    const void *dout;        /* dO, device memory, same dtype as q */
    int64_t do_stride[3];
    void *dq, *dk, *dv;      /* outputs, device memory, same dtype as q */
    int64_t dq_stride[3];
    int64_t dk_stride[3];
    int64_t dv_stride[3];
    void *workspace;         /* device memory, >= attn_bwd_workspace_size(&fwd)
                                bytes, 256-byte aligned; contents need not be
                                initialised and are scratch after the call */
    size_t workspace_bytes;
} attn_bwd_params;

/* Forward pass (every dtype; head dim 256 with bf16 or fp16). */
ATTN_API attn_status_t attn_fwd(const attn_fwd_params *p, void *stream);

/*
 * FP8 forward problem ("What is FlashAttention?", FAQ: FlashAttention-3 has
 * an FP8 forward pass). Q, K and V hold E4M3 codes, one byte per element
 * (sign, 4 exponent bits with bias 7, 3 fraction bits, no infinities), and
 * stand for code value x descale. The result is the attention of those
 * values, as attn_fwd defines it, with the products on the 8-bit tensor
 * cores and P rounded to E4M3 before it multiplies V.
 *  - f.dtype = ATTN_E4M3; f.d = 128 or 256. q, k, v strides count bytes (elements)
 *    and must be multiples of 16. f.o is bf16 [B, H, N, d] (strides in bf16
 *    elements); f.mask, when given, is bf16 as for attn_fwd; f.lse as attn_fwd.
 *  - Accuracy: each probability carries up to 2^-4 relative rounding, so O
 *    differs from the exact attention of the decoded inputs by at most
 *    2^-4 x max|v| per element (plus bf16 output rounding), and typically by
 *    1-3 % in relative L2 norm.
 */
typedef struct attn_fwd_fp8_params {
    attn_fwd_params f;
    float q_descale, k_descale, v_descale;  /* finite and > 0 */
    int32_t reserved1;                      /* must be 0 */
} attn_fwd_fp8_params;

/* FP8 forward pass (tcgen05 kind::f8f6f4). Same conventions and errors as
 * attn_fwd; a 16-bit dtype here, or E4M3 given to attn_fwd, is rejected. */
ATTN_API attn_status_t attn_fwd_fp8(const attn_fwd_fp8_params *p, void *stream);

/* Bytes of workspace attn_bwd needs for this problem (0 for an empty one):
 * per (b, h) and 128-row query tile 1 KiB of fp32 row statistics
 * (-LSE * log2(e) and D = rowsum(dO * O), padded to whole tiles), then the
 * fp32 dQ accumulator [B, H, N, d]. */
ATTN_API size_t attn_bwd_workspace_size(const attn_fwd_params *p);

/* Backward pass: D pre-pass, recompute-and-accumulate kernel, dQ finalize.
 * Head dims 64, 128 and 256 (see attn_bwd_params). */
ATTN_API attn_status_t attn_bwd(const attn_bwd_params *p, void *stream);

/* The same backward pass without a caller workspace: the scratch (row
 * statistics and the fp32 dQ accumulator) lives in a 40 MiB array the
 * library keeps in device memory, so this call allocates nothing. It is for
 * callers that cannot call cudaMalloc or their framework's allocator where
 * they run the backward (inside an allocator callback, in a plug-in whose
 * host owns all memory, under a fixed memory budget). The source pages have
 * no counterpart; it is a convenience of this library.
 *  - Inputs and outputs are passed exactly as for attn_bwd; p->workspace and
 *    p->workspace_bytes are ignored.
 *  - Problems whose attn_bwd_workspace_size() exceeds 40 MiB are rejected
 *    with ATTN_ERR_WORKSPACE before anything is launched.
 *  - Every GPU that loads the library holds the 40 MiB until the process
 *    exits. The first call on a device looks up the array's device address
 *    (cudaGetSymbolAddress); make that first call before any stream capture.
 *  - All calls share the one array: calls that overlap on the GPU (other
 *    streams, other threads) race and give wrong gradients. Each call
 *    re-initialises everything it reads, so results do not depend on
 *    earlier calls. Calls queued back to back on one stream do not overlap:
 *    each call's first kernel waits for the previous kernel in the stream.
 *  - The array's address is looked up once per device and kept. The
 *    library must not be used on a device after cudaDeviceReset() (or any
 *    other teardown of its primary context) in the same process: the kept
 *    address would then point at memory the runtime has released. */
ATTN_API attn_status_t attn_bwd_noalloc(const attn_bwd_params *p, void *stream);

/* The backward pass with every gradient reproducible bit for bit: the same
 * inputs give the same dQ, dK and dV on every call and every run on a given
 * GPU model. attn_bwd adds each key tile's share of a dQ row into an fp32
 * accumulator as the tiles finish, so its dQ can differ in the last bits
 * between runs. Here dQ comes from a second tensor-core kernel that keeps a
 * query tile on chip, recomputes the scores and dP against every key tile
 * in order ("What is FlashAttention?", Step 3 loop order, Step 4 recompute)
 * and writes dQ once; dK and dV come from attn_bwd's key-stationary kernel,
 * whose sums over query tiles already run in a fixed order.
 *  - Arguments, workspace and errors exactly as attn_bwd, except that head
 *    dim 256 returns ATTN_ERR_UNSUPPORTED (built for 64 and 128).
 *  - It does about 1.4 times the tensor-core work of attn_bwd (the scores
 *    and dP are computed twice). Results agree with attn_bwd's to rounding. */
ATTN_API attn_status_t attn_bwd_deterministic(const attn_bwd_params *p, void *stream);

/*
 * Decode problem ("FlashAttention", "What it does not do": a decode step reads
 * the whole key/value cache for a few query rows, and what helps is splitting
 * that read across the sequence; "Explain FlashAttention and why it is
 * IO-aware": partial (m, l, o) states merge with the same rescaling as tiles).
 * nq query rows attend to nk >= 1 keys: O = softmax(scale * Q K^T + causal) V
 * per (b, h), with O and LSE as attn_fwd defines them. With causal = 1 the
 * queries are the LAST nq positions: query i sits at position nk - nq + i and
 * sees keys j <= nk - nq + i (a query with none, when nq > nk, gets O = 0 and
 * LSE = -inf). Layouts, alignment and dtypes (bf16 or fp16) as in
 * attn_fwd_params, with separate query and key row counts.
 */
typedef struct attn_decode_params {
    int32_t B, H;
    int32_t nq;              /* query rows per (b, h), 1 .. 128 (from 3 rows up the
                                per-split pass runs on the tensor cores) */
    int32_t nk;              /* keys per (b, h), >= 1 */
    int32_t d;               /* 64 or 128 */
    int32_t dtype;           /* ATTN_BF16 or ATTN_F16 */
    int32_t causal;          /* 0 or 1 (bottom-right aligned, see above) */
    float scale;             /* > 0 */
    const void *q;           /* [B, H, nq, d] */
    const void *k, *v;       /* [B, H, nk, d] */
    void *o;                 /* [B, H, nq, d], dtype of q */
    float *lse;              /* [B, H, nq] fp32, contiguous */
    int64_t q_stride[3], k_stride[3], v_stride[3], o_stride[3]; /* elements, (b, h, row) */
    int32_t num_splits;      /* key ranges per (b, h); 0 = chosen by the library */
    int32_t reserved0;       /* must be 0 */
    void *workspace;         /* >= attn_decode_workspace_size(p) bytes, 256-byte
                                aligned; scratch after the call */
    size_t workspace_bytes;
} attn_decode_params;

/* Bytes of workspace attn_decode needs (the per-split partial states), for
 * the split count it will use (p->num_splits, or its own choice when 0). */
ATTN_API size_t attn_decode_workspace_size(const attn_decode_params *p);

/* Split-KV decode: one kernel computes each split's partial (m, l, o) over
 * its key range, a second merges the splits into O and LSE. Errors as for
 * attn_fwd; nq outside 1 .. 128 returns ATTN_ERR_UNSUPPORTED. */
ATTN_API attn_status_t attn_decode(const attn_decode_params *p, void *stream);

/*
 * Paged key/value cache. Serving keeps the keys and values of many sequences
 * in pages of `page_size` tokens; a block table names each sequence's pages in
 * order, so key j of sequence b is slot j % page_size of page
 * block_table[b][j / page_size]. Four entry points work on it: attn_paged
 * attends to it, attn_pages_write stores new keys and values in it,
 * attn_pages_plan takes pages for a step's new tokens and says where each token
 * goes, attn_pages_release gives the pages of ended sequences back. A step is
 * plan, then (per layer) write and paged.
 *
 * Lengths, tables and slots are int32 arrays in DEVICE memory that the kernels
 * read when they run: nothing is copied to the host, and a captured graph of
 * these calls follows the lengths it finds at each replay. The kernels check
 * what they read (lengths against the table, pages against num_pages, slots
 * against the cache): an entry out of range is skipped or read as zeros, never
 * followed, and the next attn_status() reports ATTN_ERR_INVALID. Results of
 * such a call are unspecified for the sequence concerned.
 *
 * The cache tensors are logically [num_pages, num_kv_heads, page_size, d] with
 * element strides for (page, head, slot) and d contiguous, so pages may hold
 * [page_size, heads, d] or [heads, page_size, d]. page_size is a power of two,
 * 16 or more. Strides over an extent of 1 are ignored; the others must be
 * positive. bf16 and fp16, head dims 64 and 128.
 */

/*
 * Attention of new tokens over a paged cache. Sequence b of num_seqs brings
 * n = cu_q[b + 1] - cu_q[b] query rows, rows cu_q[b] .. cu_q[b + 1] - 1 of q, and
 * has L = kv_len[b] keys (the new tokens' own among them). Query head h attends
 * with key/value head h / (num_q_heads / num_kv_heads):
 *   O = softmax(scale * Q K^T + causal) V, LSE = log(sum exp(s)), per row.
 * causal = 1: the rows are the LAST n positions; row i sees keys
 * j <= L - n + i. causal = 0: every row sees all L keys (a decoder's rows
 * against an encoder's states of another length, kept in the same pages).
 * A row that sees no key (L = 0, or i < n - L) gets O = 0 and LSE = -inf.
 * n = 0 is allowed. Rows of q from cu_q[num_seqs] to total_q (padding) may be
 * read but reach no result (they may hold anything, NaN too), and their O and LSE
 * are left as they were. cu_q[0] must be 0 and cu_q must not decrease. Slots of
 * the last page beyond L are not used: they may hold anything, NaN too. o may be
 * q itself, with the same strides.
 * A row with a NaN among the scores it sees gets NaN in O and LSE. A V row that
 * is not finite may reach O of every row of its sequence, those too that causal
 * keeps from seeing it (a probability of 0 times it); LSE does not depend on V.
 *
 * The same call gives the same bits on a given GPU model. Lengths, max_q and the
 * table's width (one tile shape is for tables of up to 384 keys) choose the order
 * of the fp32 sums, and so may change the last bits.
 */
typedef struct attn_paged_params {
    int32_t num_seqs;        /* at most 2^31 - 1024 */
    int32_t num_q_heads;     /* a multiple of num_kv_heads, at most 128 times as many */
    int32_t num_kv_heads;
    int32_t d;               /* 64 or 128 */
    int32_t total_q;         /* rows of q and o, columns of lse; at most 2^31 - 1024 */
    int32_t max_q;           /* the most query rows a sequence is expected to bring, >= 1: chooses
                                the tile shape. More rows than this are still right, only slower */
    int32_t num_pages, page_size;
    int32_t max_pages;       /* columns of the block table, >= 1; max_pages * page_size <= 2^31 - 1024 */
    int32_t dtype;           /* ATTN_BF16 or ATTN_F16 (q, caches and o alike) */
    int32_t causal;          /* 0 or 1 */
    float scale;             /* > 0 */
    int32_t reserved0[2];    /* must be 0 */
    const void *q;           /* [total_q, num_q_heads, d] */
    const void *k_cache, *v_cache;
    void *o;                 /* [total_q, num_q_heads, d] */
    float *lse;              /* [num_q_heads, total_q] fp32, contiguous */
    const int32_t *cu_q;     /* [num_seqs + 1] */
    const int32_t *kv_len;   /* [num_seqs] */
    const int32_t *block_table; /* [num_seqs, max_pages]; entries beyond a sequence's pages are not read */
    int64_t table_stride;    /* elements from one sequence's row to the next; 0 = one row for all */
    int64_t q_stride[2], o_stride[2];  /* elements, (row, head) */
    int64_t k_stride[3], v_stride[3];  /* elements, (page, head, slot) */
    void *workspace;         /* >= attn_paged_workspace_size(p) bytes, 256-byte aligned; scratch after the
                                call. Calls that may overlap on the GPU need one each; calls on one
                                stream may share it, from several host threads too */
    size_t workspace_bytes;
} attn_paged_params;

/* Bytes of workspace attn_paged needs: a bound that depends on the head dim, the
 * head group, max_q and the GPU, not on the lengths. 0 for a call it would refuse. */
ATTN_API size_t attn_paged_workspace_size(const attn_paged_params *p);

ATTN_API attn_status_t attn_paged(const attn_paged_params *p, void *stream);

/*
 * Stores keys and values of new tokens: row t of k and v goes to slot
 * slots[t] % page_size of page slots[t] / page_size, for every head. Rows whose
 * slot is negative are skipped. Slots named twice in one call end up holding
 * either row's values, piece by piece: name each once. k and v may lie in the
 * caches, but not in a slot that the call writes.
 */
typedef struct attn_pages_write_params {
    int32_t rows;            /* rows of k and v */
    int32_t num_kv_heads;
    int32_t d;               /* 64 or 128 */
    int32_t num_pages, page_size;  /* num_pages * page_size < 2^31 */
    int32_t dtype;           /* ATTN_BF16 or ATTN_F16 */
    int32_t reserved0[2];    /* must be 0 */
    const void *k, *v;       /* [rows, num_kv_heads, d] */
    const int32_t *slots;    /* [rows] */
    void *k_cache, *v_cache;
    int64_t k_row_stride[2], v_row_stride[2];  /* elements, (row, head) */
    int64_t k_stride[3], v_stride[3];          /* elements, (page, head, slot) */
} attn_pages_write_params;

ATTN_API attn_status_t attn_pages_write(const attn_pages_write_params *p, void *stream);

/*
 * Block tables and slot map of one step. Sequence b has kv_len[b] tokens in the
 * cache and brings q_len[b] more. Pages for the blocks that the new tokens open
 * are popped from the stack free_pages[0 .. free_count): sequence by sequence, in
 * order of position, the k-th page taken is free_pages[free_count - 1 - k].
 * Written: the new entries of block_table; cu_q (exclusive prefix sums of q_len);
 * new_len = kv_len + q_len; for each new token, in order, its slot
 * (page * page_size + offset) and its position in its sequence; free_left =
 * free_count less the pages taken. Rows from cu_q[num_seqs] to total_q get slot
 * and position -1. The inputs other than the table stay as they are, so the same
 * call again gives the same answer; a step is taken by using new_len and
 * free_left as the next kv_len and free_count.
 * When the stack runs out free_left is negative by the pages that were missing,
 * and the table entries and slots that got none are -1 (a page below 0 on the stack
 * gives -1 too, and is reported). Such a step is not taken:
 * kv_len and free_count stay as they were, and it is planned again once pages
 * were released (by lengths before the step) or with fewer sequences.
 * The arrays that are written (block_table, cu_q, new_len, slots, positions,
 * free_left) share no element with one another or with the others
 * (ATTN_ERR_INVALID): kv_len cannot be updated in place.
 */
typedef struct attn_pages_plan_params {
    int32_t num_seqs;        /* at most 2^31 - 1024 */
    int32_t total_q;         /* entries of slots and positions, >= the sum of q_len */
    int32_t page_size;
    int32_t max_pages;       /* columns of the block table, >= 1; max_pages * page_size <= 2^31 - 1024 */
    int32_t free_capacity;   /* entries of free_pages */
    int32_t reserved0;       /* must be 0 */
    const int32_t *q_len, *kv_len;   /* [num_seqs] */
    int32_t *block_table;    /* [num_seqs, max_pages], updated */
    int64_t table_stride;    /* elements, >= max_pages */
    const int32_t *free_pages, *free_count;  /* [free_capacity], [1] */
    int32_t *cu_q;           /* [num_seqs + 1] */
    int32_t *new_len;        /* [num_seqs] */
    int32_t *slots, *positions;  /* [total_q] */
    int32_t *free_left;      /* [1] */
} attn_pages_plan_params;

ATTN_API attn_status_t attn_pages_plan(const attn_pages_plan_params *p, void *stream);

/*
 * Gives the pages of ended sequences back: for each b with done[b] != 0, in order,
 * the pages of its kv_len[b] tokens are pushed onto free_pages, the first of them
 * at free_pages[free_count]; new_len[b] becomes 0 (kv_len[b] for the others), and
 * free_left = free_count plus the pages given back. The block table is only read.
 * Entries below 0 among a sequence's pages are reported (ATTN_ERR_INVALID). A
 * page that several sequences name is pushed once for each of them that ended.
 * The arrays that are written (free_pages, new_len, free_left) share no element
 * with one another or with the others (ATTN_ERR_INVALID).
 */
typedef struct attn_pages_release_params {
    int32_t num_seqs;        /* at most 2^31 - 1024 */
    int32_t page_size;
    int32_t max_pages;       /* columns of the block table, >= 1; max_pages * page_size <= 2^31 - 1024 */
    int32_t free_capacity;   /* entries of free_pages */
    const int32_t *done, *kv_len;    /* [num_seqs] */
    const int32_t *block_table;      /* [num_seqs, max_pages] */
    int64_t table_stride;    /* elements, >= max_pages */
    int32_t *free_pages;     /* [free_capacity], updated from free_count on */
    const int32_t *free_count;       /* [1] */
    int32_t *new_len;        /* [num_seqs] */
    int32_t *free_left;      /* [1] */
} attn_pages_release_params;

ATTN_API attn_status_t attn_pages_release(const attn_pages_release_params *p, void *stream);

/*
 * The paged cache in 8 bits. A row of d values (one token and head, keys and values
 * apart) is held as E4M3 codes and one power of two, its scale: the smallest
 * 2^e, e in [-119, 119], with max|x| <= 448 * 2^e; code = x / 2^e rounded to nearest
 * even. A power of two keeps the quotient exact (the only rounding is the code's, at most
 * 2^-4 of the value, or 2^-10 * 2^e below 2^-6 * 2^e), and code * 2^e is a bf16 number, so
 * attention works on exactly the values that the cache stands for. The codes' caches are
 * laid out as those of 16 bits, one byte per element; scales are one byte each, e + 127 (the
 * E8M0 format), in [num_pages, num_kv_heads, page_size] with the slots contiguous. bf16
 * and fp16 rows, head dims 64 and 128.
 * A NaN is held as NaN, and does not count for the scale; values beyond 448 * 2^119,
 * infinities among them, are held as that.
 */

/*
 * Stores keys and values of new tokens in 8 bits, as attn_pages_write stores them in 16.
 * Rows whose slot is negative are skipped; slots named twice in one call end up
 * holding either row, piece by piece.
 */
typedef struct attn_pages_write_fp8_params {
    int32_t rows, num_kv_heads;
    int32_t d;               /* 64 or 128 */
    int32_t num_pages, page_size;  /* num_pages * page_size < 2^31 */
    int32_t dtype;           /* ATTN_BF16 or ATTN_F16: type of k and v */
    int32_t reserved0[2];    /* must be 0 */
    const void *k, *v;       /* [rows, num_kv_heads, d] */
    const int32_t *slots;    /* [rows] */
    void *k_cache, *v_cache; /* E4M3 codes, [num_pages, num_kv_heads, page_size, d] */
    void *k_scale, *v_scale; /* E8M0 bytes, [num_pages, num_kv_heads, page_size] */
    int64_t k_row_stride[2], v_row_stride[2];  /* elements, (row, head) */
    int64_t k_stride[3], v_stride[3];          /* bytes, (page, head, slot): multiples of 16 */
    int64_t k_scale_stride[2], v_scale_stride[2];  /* bytes, (page, head): multiples of 16 */
} attn_pages_write_fp8_params;

ATTN_API attn_status_t attn_pages_write_fp8(const attn_pages_write_fp8_params *p, void *stream);

/*
 * Reads keys and values of an 8-bit cache back into 16-bit rows, by the same struct: row t of
 * k and v (written here) becomes code * scale of slot slots[t], rounded to the rows' type
 * (exact in bf16; values beyond fp16's range become infinities). Rows whose slot is
 * negative are left as they were. The same slot may be named any number of times.
 */
ATTN_API attn_status_t attn_pages_read_fp8(const attn_pages_write_fp8_params *p, void *stream);

/*
 * Trees of drafted tokens. A sequence may bring the nodes of a tree in place of a run
 * of tokens: node i (its i-th new row) follows node parents[i] < i, or the context where
 * that is -1. Its keys are the context, its ancestors and itself. attn_tree_plan turns the
 * parents into what attention and rotary positions need: for each row its visible nodes
 * as bits (bit c % 32 of word c / 32: node c) and its position, the context's length plus
 * its depth.
 * A sequence of more than 32 * words rows is a chunk of a prompt that shares the
 * step: its parents are not read, its words are 0 and its positions consecutive; the
 * attention calls treat it as causal.
 * Rows from cu_q[num_seqs] to total_q get words 0 and position -1. Parents that are
 * not below their node or below -1 are taken as -1 and reported (ATTN_ERR_INVALID), and so
 * are fewer keys than rows.
 */
typedef struct attn_tree_plan_params {
    int32_t num_seqs;        /* at most 2^31 - 1024 */
    int32_t total_q;         /* at most 2^31 - 1024 */
    int32_t words;           /* of a row, 1 to 32 */
    int32_t reserved0;       /* must be 0 */
    const int32_t *parents;  /* [total_q] */
    const int32_t *cu_q;     /* [num_seqs + 1] */
    const int32_t *kv_len;   /* [num_seqs]: keys with the new rows' own */
    int32_t *mask;           /* [total_q, words] */
    int64_t mask_stride;     /* elements from one row to the next, >= words */
    int32_t *positions;      /* [total_q] */
} attn_tree_plan_params;

ATTN_API attn_status_t attn_tree_plan(const attn_tree_plan_params *p, void *stream);

/*
 * attn_paged for trees: row i of a sequence of up to 32 * words rows sees its context (keys
 * j < L - n) and, of its new rows' keys, L - n + c for every c < n whose bit is set in
 * the row's words. Any bits are allowed, below or above the row's own; a row that
 * sees no key gets O = 0 and LSE = -inf. Sequences with more rows than the mask has bits are
 * causal, as attn_paged has it. `f.causal` must be 0. Workspace and everything else as
 * attn_paged (attn_paged_workspace_size(&f)).
 */
typedef struct attn_paged_tree_params {
    attn_paged_params f;
    const int32_t *mask;     /* [total_q, words] */
    int64_t mask_stride;     /* elements from one row to the next; 0 = one row for all */
    int32_t words;           /* 1 to 32 */
    int32_t reserved1;       /* must be 0 */
} attn_paged_tree_params;

ATTN_API attn_status_t attn_paged_tree(const attn_paged_tree_params *p, void *stream);

/*
 * Attention over a paged cache in 8 bits, of a run of tokens (t.mask NULL; t.words, t.mask_stride
 * 0) or of trees (t.mask and t.words given; a batch without rows or sequences needs no mask). t.f as
 * for attn_paged, with f.dtype the type of q and o, the caches E4M3 codes and k_stride, v_stride in
 * bytes. Keys and values are code * scale, with the scales of attn_pages_write_fp8, 2^-119 to 2^119.
 * Values are taken in f.dtype: exact in bf16; in fp16 they have to be within its range, and are
 * rounded below 2^-14. The products, the softmax and their accuracy are attn_paged's, but that entries of
 * a row of q below 2^-16 of its largest are rounded, by at most 2^-24 of that (fp16: 2^-27). A row of q with
 * an infinity gets NaN in O and LSE, if it sees a key. Scores that q's rows leave ordinary may overflow,
 * to NaN, where keys reach 2^120 (with a scale above 1/8, 2^117; above 1, 2^117 / scale). Slots beyond a
 * sequence's length may hold any codes and scales.
 */
typedef struct attn_paged_fp8_params {
    attn_paged_tree_params t;
    const void *k_scale, *v_scale;  /* E8M0 bytes, [num_pages, num_kv_heads, page_size], 16-byte aligned */
    int64_t k_scale_stride[2], v_scale_stride[2];  /* bytes, (page, head): multiples of 16 */
} attn_paged_fp8_params;

/* Bytes of workspace attn_paged_fp8 needs: a bound of the same kind as attn_paged's. */
ATTN_API size_t attn_paged_fp8_workspace_size(const attn_paged_fp8_params *p);

ATTN_API attn_status_t attn_paged_fp8(const attn_paged_fp8_params *p, void *stream);

/*
 * Rotary positions of queries and keys, in one launch. Pair i < rotary_dim / 2 of a row at
 * position x is turned by the angle t = x * inv_freq[i]:
 *   y0 = magnitude * (x0 cos t - x1 sin t),  y1 = magnitude * (x1 cos t + x0 sin t),
 * where the pair is columns (i, i + rotary_dim / 2) or, interleaved, (2 i, 2 i + 1). Columns from
 * rotary_dim on are copied. Angles are taken modulo a turn in 64-bit integers, to 2^-32 of a
 * turn for any 32-bit position and |inv_freq| < 2^32, and sums in fp32, rounded once.
 * Tensors are [B, H, N, d] as for attn_fwd (a ragged batch of rows [N, H, d] is B = 1); bf16, fp16
 * and fp32. Rows whose position is negative (the padding of attn_pages_plan and
 * attn_tree_plan) are left as they were in the outputs. An output may be its input, with the
 * same strides; otherwise the two share no memory.
 */
typedef struct attn_rotary_params {
    int32_t B, N;
    int32_t Hq, Hk;          /* heads of q and of k; either may be 0, and its pointers are not read then */
    int32_t d;               /* a multiple of 16, up to 256 */
    int32_t rotary_dim;      /* a multiple of 16, up to d */
    int32_t dtype;           /* ATTN_BF16, ATTN_F16 or ATTN_F32 */
    int32_t interleaved;     /* 0 or 1 */
    float magnitude;         /* > 0 */
    int32_t reserved0;       /* must be 0 */
    const int32_t *positions;
    int64_t position_stride[2];  /* elements, (b, n); 0 broadcasts */
    const float *inv_freq;   /* [rotary_dim / 2] */
    const void *q, *k;
    void *q_out, *k_out;
    int64_t q_stride[3], k_stride[3], q_out_stride[3], k_out_stride[3];  /* elements, (b, h, n) */
} attn_rotary_params;

ATTN_API attn_status_t attn_rotary(const attn_rotary_params *p, void *stream);

/* The backward pass of attn_rotary: q and k hold the gradients of its outputs, q_out and k_out
 * receive those of its inputs (the transpose: the same turn, backwards; columns from rotary_dim on
 * are copied). Rows whose position is negative are left as they were. */
ATTN_API attn_status_t attn_rotary_bwd(const attn_rotary_params *p, void *stream);

/* Synchronizes `stream`, then reports (and clears) the current device's
 * error word: ATTN_ERR_TIMEOUT if a kernel gave up on a bounded wait since
 * the last call (outputs of calls since then are unspecified; their inputs and
 * workspaces can be used again), ATTN_ERR_INVALID if a paged-cache kernel met a
 * length, page or slot out of range, ATTN_ERR_CUDA for an asynchronous CUDA
 * error, else ATTN_OK. */
ATTN_API attn_status_t attn_status(void *stream);

/* Message for the last non-OK status returned on this host thread ("" if none). */
ATTN_API const char *attn_last_error(void);

/* Upper bound, in nanoseconds, on any single in-kernel wait (mbarrier or
 * pipeline slot) before the kernel records ATTN_ERR_TIMEOUT and returns.
 * Default 2e9 (2 s); values below 1e6 are raised to 1e6. Process-wide. A wait may
 * last while one CTA walks a sequence's keys, 1 to 1.6 us per 128 of them in
 * attn_paged: beyond 100 million keys a sequence, raise it. */
ATTN_API void attn_set_wait_timeout_ns(uint64_t ns);

/* Test hook for failure detection: when > 0, the next forward and paged
 * attention launches on this host thread have their load warps stop after this
 * many key/value tiles (of a CTA), so the consumers' bounded waits run out and report
 * ATTN_ERR_TIMEOUT. 0 (the default) disables it. */
ATTN_API void attn_debug_set_producer_stall(int32_t kv_tiles);

/* Profiling hook: while `events` is non-NULL, every attn_bwd call on this
 * host thread records events[0] before its pre-pass kernel, events[1] after
 * it, events[2] after the recompute kernel and events[3] after the dQ
 * finalize, on the call's stream, so a caller can time each of the three
 * launches with CUDA events. The four cudaEvent_t handles are passed as
 * void* and stay owned by the caller; the array is copied. NULL turns the
 * hook off. */
ATTN_API void attn_debug_set_bwd_events(void *const events[4]);

/* Launch log, for checking on a real system that each call runs as fused
 * kernels ("FlashAttention", "Checking it on a real system": the profiler
 * should show one fused attention kernel, not separate matmul, softmax and
 * matmul launches). attn_debug_launch_count() is the number of kernels this
 * library has launched from the calling host thread since the process
 * started; attn_debug_launch_name(back) is the symbol name of one of the
 * last 16 of them (back = 0 is the most recent), or NULL when `back` is out
 * of that range. The names are the CUDA runtime's (mangled C++ names) and
 * stay valid until the process exits. Every launch is counted once it has
 * been issued without a launch error. */
ATTN_API uint64_t attn_debug_launch_count(void);
ATTN_API const char *attn_debug_launch_name(uint32_t back);

/* Library version, major * 10000 + minor * 100 + patch. */
ATTN_API int32_t attn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_GB300_ATTN_H */
