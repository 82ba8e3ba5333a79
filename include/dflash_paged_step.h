/*
 * dflash_paged_step.h -- C ABI of a decoding step around the paged E4M3 attention
 * (dflash_verify_attn.h): the tables of the paged cache, rotary positions with the cache write,
 * and the attention of a batch over a shared prefix. One step of a serving loop calls them in this
 * order, then the attention of dflash_verify_attn.h or the shared-prefix one below, all from
 * device memory, so that one captured graph serves growing contexts.
 *
 * The conventions are those of dflash_verify_attn.h: every call returns a dflash_status; nothing
 * allocates, throws or synchronises; everything that runs on the GPU is stream-ordered and
 * capturable; host-checkable preconditions (null pointers, alignment, ranges) are refused before
 * anything is launched; device-only conditions never fault but set a bit of a sticky status word.
 * `status` is that word: 4 bytes of device memory zeroed once by the caller, the head of an
 * attention workspace if the step is to have a single word (dflash_verify_attn_read_flags reads
 * and clears either). Kernels run on the device that is current at the call; buffers and stream
 * belong to it. A buffer that a call writes overlaps no other buffer of the call unless the text
 * below says so (what starts at the same address is refused).
 */
#ifndef DFLASH_PAGED_STEP_H
#define DFLASH_PAGED_STEP_H

#include "dflash_verify_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DFLASH_PAGED_STEP_VERSION 1

/* Further bits of the device status word (beside DFLASH_FLAG_*). */
#define DFLASH_FLAG_PAGES_EXHAUSTED 0x10 /* the free list ended before every page was handed out */
#define DFLASH_FLAG_TOKENS_DROPPED 0x20  /* more new tokens than max_tokens: the rest have no entry */
#define DFLASH_FLAG_SLOT_RANGE 0x40      /* a cache slot past the pool: its token was not written  */

/* ------------------------------------------------------------------------------------------------
 * Tables of the paged cache, from request lengths.
 *
 * Request b has cached_lens[b] tokens in the cache, holds the first held_pages[b] pages of its
 * block-table row and gets new_lens[b] tokens more. With P = page_size and
 *   ctx_b   = cached_b + new_b                        (lengths below 0 count as 0; ctx_b above
 *                                                      max_context is cut to it, and new_b with it)
 *   need_b  = max(held_b, ceil(ctx_b / P))
 *   first_b = clamp(shared, held_b, need_b)           shared = prefix_pages, or 0 without a prefix
 *   take_b  = need_b - first_b,  at_b = free_head + sum of take over the requests before b
 * the row's entries change as follows: pages [held_b, first_b) become the shared prefix's,
 * prefix_table[p], and pages [first_b, need_b) come off the free list, free_pages[at_b + p -
 * first_b]. No other entry of the table is written. held_pages may exceed what the lengths need (a
 * verification that rejected drafted tokens leaves pages behind); they are used before new ones.
 * Token i of request b has position cached_b + i and the cache slot page * P + position % P, page
 * being its row's entry at position / P. The tokens of all requests lie one after the other.
 *   context_lens   ctx_b, as the attention takes it
 *   held_out       pages that the row holds now (need_b unless the free list ended)
 *   free_head_out  free_head + pages taken
 *   token_starts   [batch + 1] first token of each request, then their number
 *   positions      int32 [max_tokens]; 0 past the last token
 *   slots          int64 [max_tokens]; -1 past the last token, for a token without a page of its
 *                  own, and for a token inside the shared pages (those are read only; its query is
 *                  needed all the same: dflash_rope_kv_write_live with token_starts + batch)
 * Tokens past max_tokens have no position or slot (DFLASH_FLAG_TOKENS_DROPPED; their pages are
 * handed out all the same, and token_starts stops at max_tokens). Once the free list ends, the
 * requests' remaining pages in request order become -1 in the table, their tokens' slots -1, and
 * held_out counts the pages up to the first missing one (DFLASH_FLAG_PAGES_EXHAUSTED). A page
 * outside [0, num_pages) gives its tokens slot -1 (DFLASH_FLAG_PAGE_CLAMPED); context_lens above
 * max_context sets DFLASH_FLAG_CONTEXT_CLAMPED. held_pages outside [0, max_pages_per_seq] are cut
 * to that range, free_head below 0 counts as 0 and prefix_pages is cut to prefix_capacity.
 * Inputs and outputs are separate buffers (the same address twice is refused), so a step can be
 * repeated; a loop swaps them. prefix_table may be the first row of block_table whose request holds
 * the shared pages: entries below held_b are not written.
 */
typedef struct {
    int32_t version;           /* DFLASH_PAGED_STEP_VERSION */
    int32_t batch;             /* requests, 1 .. 4096 */
    int32_t page_size;         /* P >= 1 */
    int32_t max_pages_per_seq; /* block-table row stride */
    int32_t num_pages;         /* pages in the pool */
    int32_t max_context;       /* <= max_pages_per_seq * page_size */
    int32_t max_tokens;        /* entries of positions and slots, >= 1 */
    int32_t num_free;          /* entries of free_pages, >= 0 */
    int32_t prefix_capacity;   /* entries of prefix_table, 0 .. max_pages_per_seq (0: no prefix) */
} dflash_paged_tables_problem;

/*
 * All pointers device memory, int32 unless stated. prefix_table and prefix_pages (one int32) are
 * both NULL when prefix_capacity is 0. slots: 8-byte aligned.
 */
int dflash_paged_tables(const dflash_paged_tables_problem* problem, const int32_t* cached_lens,
                        const int32_t* new_lens, const int32_t* held_pages,
                        const int32_t* free_pages, const int32_t* free_head,
                        const int32_t* prefix_table, const int32_t* prefix_pages,
                        int32_t* block_table, int32_t* context_lens, int32_t* held_out,
                        int32_t* free_head_out, int32_t* token_starts, int32_t* positions,
                        int64_t* slots, int32_t* status, void* cuda_stream);

/* ------------------------------------------------------------------------------------------------
 * Rotary positions.
 *
 * The first rotary_dim elements of a head are rotary_dim / 2 pairs (x, y): elements i and
 * i + rotary_dim / 2 (DFLASH_ROPE_HALF) or 2i and 2i + 1 (DFLASH_ROPE_INTERLEAVED). At position t
 * pair i becomes
 *   (x cos a - y sin a, y cos a + x sin a) * amplitude,  a = t * theta_i;
 * the other elements stay as they are. theta_i = base^(-2i / rotary_dim), amplitude 1, unless
 * the frequencies are scaled for contexts longer than the trained one (s = factor >= 1):
 *   LINEAR      theta_i / s
 *   NTK         base * s^(d / (d - 2)) in place of base, d = rotary_dim
 *   YARN        (Peng et al. 2023) theta_i (1 - r_i + r_i / s), r_i = clamp((i - lo) / (hi - lo)),
 *               lo = max(0, floor(c(beta_fast))), hi = min(d - 1, ceil(c(beta_slow))) (hi - lo at
 *               least 0.001), c(n) = d ln(trained / (2 pi n)) / (2 ln base) the pair that turns n
 *               times over the trained context; amplitude 0.1 ln(s) + 1
 *   WAVELENGTH  theta_i (g_i + (1 - g_i) / s), g_i = clamp((n_i - low_turns) / (high_turns -
 *               low_turns)), n_i = trained * theta_i / (2 pi)   (clamp: to [0, 1])
 * Cosine, sine and the rotation are FP32; q_out and k_out are rounded once.
 */
#define DFLASH_ROPE_HALF 0
#define DFLASH_ROPE_INTERLEAVED 1

#define DFLASH_ROPE_SCALE_NONE 0
#define DFLASH_ROPE_SCALE_LINEAR 1
#define DFLASH_ROPE_SCALE_NTK 2
#define DFLASH_ROPE_SCALE_YARN 3
#define DFLASH_ROPE_SCALE_WAVELENGTH 4

#define DFLASH_FP16 0
#define DFLASH_BF16 1

typedef struct {
    int32_t version;         /* DFLASH_PAGED_STEP_VERSION */
    int32_t num_q_heads;     /* Hq, 1 .. 256 */
    int32_t num_kv_heads;    /* Hkv, 1 .. 256 */
    int32_t head_dim;        /* 256 */
    int32_t rotary_dim;      /* a multiple of 16, 16 .. head_dim */
    int32_t layout;          /* DFLASH_ROPE_HALF or DFLASH_ROPE_INTERLEAVED */
    int32_t dtype;           /* DFLASH_FP16 or DFLASH_BF16: type of q, k, v, q_out, k_out */
    int32_t scaling;         /* DFLASH_ROPE_SCALE_* */
    int32_t trained_context; /* YARN, WAVELENGTH: context of the training, >= 1 */
    int32_t page_size;       /* kv_write: tokens per page, >= 1 */
    int32_t num_pages;       /* kv_write: pages in each pool, >= 1 */
    int32_t reserved;        /* 0 */
    double base;             /* > 1 */
    double factor;           /* s >= 1 */
    double beta_fast, beta_slow;   /* YARN: > 0 */
    double low_turns, high_turns;  /* WAVELENGTH: low < high */
} dflash_rope_problem;

/* Written by dflash_rope_plan, read-only afterwards. */
typedef struct {
    int32_t version;
    float amplitude;
    dflash_rope_problem problem;
} dflash_rope_plan_t;

/*
 * Check the problem and compute its frequencies: phases (host memory, rotary_dim / 2 entries)
 * receives theta_i / (2 pi) as a 64-bit fraction of a turn. The caller keeps a copy on the device
 * for the calls below. t * phases[i] modulo 2^64 is then the exact fraction of a turn that
 * position t stands at, whatever the distance (theta_i carries 53 bits: at position 2^20 the angle
 * is within 2^-33 of a turn).
 */
int dflash_rope_plan(const dflash_rope_problem* problem, dflash_rope_plan_t* plan,
                     uint64_t* phases);

/*
 * Rotate Q and, unless k is NULL, K.
 *   q       [num_tokens, Hq, head_dim], token t at q + t * q_stride elements (strides are multiples
 *           of 8 elements, at least Hq * head_dim; heads lie one after the other)
 *   k       [num_tokens, Hkv, head_dim], stride k_stride; NULL with k_out NULL for Q alone
 *   positions  int32 [num_tokens]
 *   phases  as written by dflash_rope_plan, device memory, 8-byte aligned
 *   q_out, k_out  token strides q_out_stride, k_out_stride. q_out may be q with the same stride
 *           (k_out likewise k): the rotation is then done in place.
 * q, k, q_out, k_out 16-byte aligned. num_tokens 0 .. 2^31 - 1; 0 launches nothing.
 */
int dflash_rope_apply(const dflash_rope_plan_t* plan, int64_t num_tokens, const void* q,
                      int64_t q_stride, const void* k, int64_t k_stride, const int32_t* positions,
                      const uint64_t* phases, void* q_out, int64_t q_out_stride, void* k_out,
                      int64_t k_out_stride, void* cuda_stream);

/*
 * Rotate Q, and write the rotated K and V of each token into the paged E4M3 pools at its slot
 * (page * page_size + offset in the page, as dflash_paged_tables gives it).
 *   k, v    [num_tokens, Hkv, head_dim], strides k_stride, v_stride
 *   slots   int64 [num_tokens]. A token with a negative slot is padding: nothing of it is written,
 *           q_out neither (dflash_rope_kv_write_live tells padding from tokens that have a query
 *           but no slot of their own). A slot past the pool writes q_out alone
 *           (DFLASH_FLAG_SLOT_RANGE).
 *   k_pool, v_pool  as in dflash_verify_attn.h, 8-byte aligned
 *   k_scale, v_scale  one FP32 each (device)
 * Each element becomes the E4M3FN code of x / scale by the rule of dflash_verify_attn_kv_write (one
 * FP32 division, round to nearest even, saturated to +-448, NaN to a NaN code); K is quantised from
 * its rotated FP32 value, with no rounding to dtype between. Two tokens with the same slot leave
 * bytes of one or the other. q_out may be q with the same stride.
 */
int dflash_rope_kv_write(const dflash_rope_plan_t* plan, int64_t num_tokens, const void* q,
                         int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                         int64_t v_stride, const int32_t* positions, const int64_t* slots,
                         const uint64_t* phases, const float* k_scale, const float* v_scale,
                         void* q_out, int64_t q_out_stride, void* k_pool, void* v_pool,
                         int32_t* status, void* cuda_stream);

/*
 * The same with the number of tokens that are not padding: num_live, one int32 (device), what
 * dflash_paged_tables leaves in token_starts[batch]. A token below it with a negative slot has its
 * query rotated and nothing written to the pools. Such tokens are ordinary: a request whose whole
 * prompt is in the shared pages computes its last token's query again, at a position inside them.
 * From num_live on, counted from this call's first token, a negative slot is padding, as above
 * (num_live NULL: everywhere, as above).
 */
int dflash_rope_kv_write_live(const dflash_rope_plan_t* plan, int64_t num_tokens, const void* q,
                              int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                              int64_t v_stride, const int32_t* positions, const int64_t* slots,
                              const int32_t* num_live, const uint64_t* phases,
                              const float* k_scale, const float* v_scale, void* q_out,
                              int64_t q_out_stride, void* k_pool, void* v_pool, int32_t* status,
                              void* cuda_stream);

/* ------------------------------------------------------------------------------------------------
 * Head norms in the same pass.
 *
 * Each head x of Q (and of K) is first normed over its head_dim elements,
 *   x_i * (weight_offset + w_i) / sqrt(mean of x^2 + eps),
 * then rotated as above; V is not normed. Sum and division are FP32, nothing is rounded between norm and
 * rotation. (The squares' sum must stay below 2^128: bf16 elements below 2^60. With an eps below 2^-126 their
 * mean must be above that: of bf16 elements that are all below 2^-63 the squares are lost.)
 */
typedef struct {
    const void* q_weight; /* device, head_dim elements of the plan's dtype, 16-byte aligned; NULL: Q
                             is not normed */
    const void* k_weight; /* the same for K */
    float eps;            /* >= 0, finite */
    float weight_offset;  /* finite; 1 for weights that are kept about zero, else 0 */
} dflash_head_norm;       /* host struct; its fields are taken at the call */

/* dflash_rope_apply and dflash_rope_kv_write_live with norms (norm NULL: without). */
int dflash_norm_rope_apply(const dflash_rope_plan_t* plan, const dflash_head_norm* norm,
                           int64_t num_tokens, const void* q, int64_t q_stride, const void* k,
                           int64_t k_stride, const int32_t* positions, const uint64_t* phases,
                           void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                           void* cuda_stream);
int dflash_norm_rope_kv_write(const dflash_rope_plan_t* plan, const dflash_head_norm* norm,
                              int64_t num_tokens, const void* q, int64_t q_stride, const void* k,
                              int64_t k_stride, const void* v, int64_t v_stride,
                              const int32_t* positions, const int64_t* slots,
                              const int32_t* num_live, const uint64_t* phases,
                              const float* k_scale, const float* v_scale, void* q_out,
                              int64_t q_out_stride, void* k_pool, void* v_pool, int32_t* status,
                              void* cuda_stream);

/* ------------------------------------------------------------------------------------------------
 * Attention of a batch over a shared prefix.
 *
 * The result is dflash_verify_attn_forward's on the same q, pools, block_table and context_lens
 * (same causal rule, same empty rows). The caller adds that the first *prefix_len tokens of every
 * sequence are the same, and where their pages are. The prefix's whole pages, S = floor(*prefix_len
 * / page_size) * page_size keys, are then read once through prefix_table for the query rows of
 * the whole batch, and only keys S .. N - 1 of each sequence through its block-table row (entries
 * from S / page_size on; the ones before are not read). Maxima, sums and numerators of both parts
 * are FP32 and merged by a combine pass. Probabilities are three E4M3 terms (ROWS, and the sequences'
 * own keys) or FP16 (PAIRS): the output errs by 2.1e-4 to 2.2e-4 or 2.2e-4 to 3.0e-4 of its norm, of which
 * its own rounding to FP16 is 2.1e-4. Probabilities far below a row's largest have a fixed step of 2^-23 of
 * it, offset key by key so that the mean of many is right, or of 2^-28. AUTO takes the kernel that is
 * estimated to be faster.
 *   prefix_table  int32 [floor(max_prefix / page_size)]; a row of block_table may serve. NULL if
 *                 that is 0
 *   prefix_len    one int32 (device), cut to [0, max_prefix] (DFLASH_FLAG_CONTEXT_CLAMPED)
 * A sequence that ends inside the prefix, or is empty (a padded batch slot, N = 0), sees the keys
 * that the causal rule gives it. A row of q with a NaN or an infinity gives NaN, in its own row of
 * out and lse alone, if it sees a key. Codes at or past a length are never used, whatever they hold; a NaN
 * code of V below the prefix length may make NaN of every row, those that do not see its key included
 * (kv_write makes one of a NaN element only).
 */
#define DFLASH_PREFIX_KERNEL_AUTO 0
#define DFLASH_PREFIX_KERNEL_ROWS 1  /* blocks of 48 rows on the split kernel: E4M3 products     */
#define DFLASH_PREFIX_KERNEL_PAIRS 2 /* blocks of 256 rows on a pair of SMs: FP16 products        */

typedef struct {
    int32_t version;           /* DFLASH_PAGED_STEP_VERSION */
    int32_t batch;             /* sequences, 1 .. 4096 */
    int32_t q_len;             /* drafted tokens per sequence, >= 1 */
    int32_t num_q_heads;       /* Hq % Hkv == 0, q_len * Hq / Hkv <= 256 */
    int32_t num_kv_heads;
    int32_t head_dim;          /* 256 */
    int32_t page_size;         /* a multiple of 16 */
    int32_t max_pages_per_seq; /* block-table row stride; >= ceil(max_context / page_size) */
    int32_t num_pages;
    int32_t max_context;       /* largest N any call sees, 1 .. 2^30 */
    int32_t max_prefix;        /* largest *prefix_len, 0 .. max_context */
    int32_t device;            /* CUDA ordinal whose SM count sizes the plan; < 0: 152 SMs */
    int32_t kernel;            /* DFLASH_PREFIX_KERNEL_* of the prefix part */
    int32_t flags;             /* 0 */
} dflash_prefix_attn_problem;

typedef struct {
    int32_t version;
    int32_t prefix_kernel;     /* DFLASH_PREFIX_KERNEL_ROWS or _PAIRS */
    int32_t prefix_rows;       /* batch * q_len * Hq / Hkv rows per KV head over the prefix */
    int32_t prefix_row_blocks; /* blocks that they are dealt into */
    int32_t prefix_splits;     /* ROWS: key splits per KV head; PAIRS: SM pairs launched */
    int32_t prefix_slots;      /* split states of the prefix in the workspace */
    int32_t prefix_slot_rows;  /* rows of one such state */
    int32_t sm_count;
    dflash_verify_attn_plan_t suffix; /* the sequences' own keys: its workspace part comes first */
    size_t ws_prefix_state_offset;    /* float2 (m, l) [prefix_slots, prefix_slot_rows] */
    size_t ws_prefix_acc_offset;      /* float [prefix_slots, prefix_slot_rows, head_dim] */
    size_t ws_unit_offset;            /* int4 [batch, Hkv]: split slots of the own keys */
    size_t workspace_bytes;
    dflash_prefix_attn_problem problem;
} dflash_prefix_attn_plan_t;

/* Check the problem and choose kernels and splits (host only). */
int dflash_prefix_attn_plan(const dflash_prefix_attn_problem* problem,
                            dflash_prefix_attn_plan_t* plan);

/*
 * The whole operator on one stream. Buffers, alignments and workspace rules as for
 * dflash_verify_attn_forward (the caller zeroes the workspace's first 16 bytes once; calls that may
 * overlap on the GPU need a workspace each, captured graphs that replay at the same time included).
 */
int dflash_prefix_attn_forward(const dflash_prefix_attn_plan_t* plan, const void* q,
                               const void* k_pool, const void* v_pool, const int32_t* prefix_table,
                               const int32_t* prefix_len, const int32_t* block_table,
                               const int32_t* context_lens, const float* k_scale,
                               const float* v_scale, void* workspace, size_t workspace_bytes,
                               void* out, float* lse, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* DFLASH_PAGED_STEP_H */
