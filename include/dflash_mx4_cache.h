/*
 * dflash_mx4_cache.h -- C ABI of a paged KV cache held in 4 bits: keys and values appended to it,
 * cached tokens read back as numbers, and the attention of drafted tokens over it. It stands beside
 * the E4M3 cache of dflash_verify_attn.h at 53 % of its bytes: the same page tables, slots, causal
 * rule, splits and workspace; dflash_paged_tables (dflash_paged_step.h) serves both.
 *
 * The conventions are those of dflash_paged_step.h: every call returns a dflash_status; nothing
 * allocates, throws or synchronises; everything that runs on the GPU is stream-ordered and
 * capturable; what the host can check is refused before a launch; device-only conditions never fault
 * but set a bit of a sticky status word. A buffer that a call writes overlaps no other buffer of the
 * call unless the text says so (what starts at the same address is refused).
 *
 * The numbers (OCP microscaling, E2M1 elements with E8M0 scales). A head of 256 elements is 8 blocks
 * of 32. A block has a power of two 2^e, kept as the byte e + 127, and each element is one of 0, 0.5,
 * 1, 1.5, 2, 3, 4, 6 times it, with a sign: 4 bits, sign first, codes in the order of the sizes.
 * Writing takes the smallest e with max |x| <= 7 * 2^e and rounds x / 2^e to the nearest, ties to the
 * even code: it is off by 2^e at most, half of the grid's last step, above 6 * 2^e as well. A block of
 * zeros has byte 0. A block with a NaN or an infinity gets the byte 255, NaN; its codes are 0.
 *
 * The pools, one of K and one of V, are uint8 [num_pages, page_size / 16, Hkv, 2176]: a chunk of 16
 * tokens of one head is 2048 bytes of codes and 128 of scales. Slot s (page * page_size + offset, as
 * dflash_paged_tables gives it) is token s % 16 of chunk s / 16. In its chunk token t has
 *   K: elements 32 j + 2 i and 32 j + 2 i + 1 in the low and high half of byte 256 j + 16 t + i
 *   V: elements i and i + 128 in the low and high half of byte 16 i + t
 *   both: the scale of block j in byte 2048 + 8 t + j
 * so that a chunk is one copy, a key's codes are 16-byte pieces, and a lane of the attention that
 * holds an element of V finds its 16 tokens in one. Every byte of a pool has a meaning: a new pool
 * is zeroed, and holds zeros.
 */
#ifndef DFLASH_MX4_CACHE_H
#define DFLASH_MX4_CACHE_H

#include "dflash_paged_step.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DFLASH_MX4_CHUNK_TOKENS 16
#define DFLASH_MX4_CHUNK_BYTES 2176

/* plan.kernel of dflash_mx4_attn_plan */
#define DFLASH_KERNEL_MX4 3

/*
 * dflash_norm_rope_kv_write for the 4-bit pools: Q normed and rotated, the normed and rotated K and
 * V of each token written at its slot. All arguments as there, without scales; norm may be NULL.
 *   k_pool, v_pool  as above, 16-byte aligned; the plan's page_size is a multiple of 16
 * K is quantised from its rotated FP32 value, with no rounding to dtype between. Two tokens with the same
 * slot leave a mixture of both in it (the slot's bytes alone).
 */
int dflash_mx4_kv_write(const dflash_rope_plan_t* plan, const dflash_head_norm* norm,
                        int64_t num_tokens, const void* q, int64_t q_stride, const void* k,
                        int64_t k_stride, const void* v, int64_t v_stride,
                        const int32_t* positions, const int64_t* slots, const int32_t* num_live,
                        const uint64_t* phases, void* q_out, int64_t q_out_stride, void* k_pool,
                        void* v_pool, int32_t* status, void* cuda_stream);

/* Types of the numbers that dflash_mx4_read writes. */
#define DFLASH_E5M2 2 /* holds every number of the format from 2^-15 to 57344, and 2^-16 */

/*
 * The numbers of cached tokens: row i of k_out and v_out gets the token at slots[i].
 *   slots   int64 [num_tokens] (device). A negative slot leaves its rows as they are, and so does one
 *           past the pool (DFLASH_FLAG_SLOT_RANGE)
 *   k_out, v_out  [num_tokens, Hkv, 256] of dtype (DFLASH_FP16, DFLASH_BF16, DFLASH_E5M2), 16-byte
 *           aligned, token strides in elements (a multiple of 16, at least Hkv * 256); either
 *           is NULL with its pool if it is not wanted
 * Numbers past a type's range become its infinity (E5M2: its largest number), those below its
 * smallest are rounded, a block with byte 255 is NaN. num_tokens 0 .. 2^31 - 1; 0 launches nothing.
 */
int dflash_mx4_read(int32_t num_kv_heads, int32_t head_dim, int32_t page_size, int32_t num_pages,
                    const void* k_pool, const void* v_pool, int64_t num_tokens,
                    const int64_t* slots, int32_t dtype, void* k_out, int64_t k_out_stride,
                    void* v_out, int64_t v_out_stride, int32_t* status, void* cuda_stream);

/*
 * Attention over the 4-bit pools: dflash_verify_attn_plan and _forward with these pools and without
 * scales (the numbers carry their own). problem.kernel is DFLASH_KERNEL_AUTO; of the flags
 * DFLASH_PROBLEM_PDL is taken, DFLASH_PROBLEM_FUSED_COMBINE is not (DFLASH_ERR_UNSUPPORTED). Sequences times
 * KV heads are at most 65535.
 * Buffers, alignments and workspace as for dflash_verify_attn_forward. A batch of more units (sequences times
 * KV heads) than half the SMs gets several SMs' worths of slots, and a call shares out one of them (or a slot a
 * unit) or all, by its lengths; dflash_verify_attn_split_slots says what, for these plans too.
 *
 * Q stays FP16, K and V are exact in FP16 up to the limits below, all sums are FP32. The output's weights
 * are FP16: a probability times the largest power among its key's blocks of V, rounded by 2^-11 of
 * itself or 2^-33 of the row's largest such product, whichever is more (so a key whose V is 2^20 times
 * the others' in one block costs the others' weights precision in all blocks; lse is not affected). A key whose K or V has a NaN scale makes NaN of
 * every row that sees it, in out and lse, and of no other; so does a row of q with a NaN or an
 * infinity of itself, if it sees a key. Codes at or past a length are never used, whatever they hold.
 * Of a key's blocks, one whose scale is more than 2^26 below the key's largest counts as zeros; so do
 * V's below 2^-66. V's scales above 2^41 count as 2^41. A key whose largest scale of K is above 2^100 counts
 * with that one at 2^100 and its others as far below it as they are.
 */
int dflash_mx4_attn_plan(const dflash_verify_attn_problem* problem,
                         dflash_verify_attn_plan_t* plan);
int dflash_mx4_attn_forward(const dflash_verify_attn_plan_t* plan, const void* q,
                            const void* k_pool, const void* v_pool, const int32_t* block_table,
                            const int32_t* context_lens, void* workspace, size_t workspace_bytes,
                            void* out, float* lse, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* DFLASH_MX4_CACHE_H */
