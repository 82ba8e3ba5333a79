// common.cuh -- device-side parameter blocks and helpers shared by the partial and combine kernels.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "dflash_verify_attn.h"

namespace dflash {

constexpr int kHeadDim = 256;  // the only head dim the kernels are built for
constexpr int kMaxRows = 256;  // q_len * Hq / Hkv rows per KV head (split over row blocks)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct PartialParams {
    const __half* q;
    const uint8_t* k_pool;
    const uint8_t* v_pool;
    const int32_t* block_table;
    const int32_t* context_lens;
    const float* k_scale;
    const float* v_scale;
    int32_t* status;   // workspace status word
    float2* ws_state;  // (m, l) [B, Hkv, S, R]
    float* ws_acc;     // [B, Hkv, S, R, D]
    int batch, q_len, num_q_heads, num_kv_heads, group, rows;
    int page_size, max_pages_per_seq, num_pages, max_context;
    int num_splits, tile_keys, min_split_keys;
    int num_slots;  // workspace split slots: Hkv * num_splits for one sequence, else the plan's
    int round_slots;  // slots that run at once, where a batch may take more (0: it takes num_slots)
    // Row blocks: the grid's x extent is num_splits * row_blocks; CTA x = split * row_blocks + k
    // carries rows [k * block_rows, min(rows, (k + 1) * block_rows)) of that split's slot.
    int row_blocks, block_rows;
    // keys per split of a max_context-long context (the split size the kernels guess while the
    // context length is in flight), and log2 of page_size when it is a power of two (else -1)
    int per_max, page_shift;
    // merge of the splits inside the same launch (every CTA resident): grid barrier words in the
    // workspace header, then FP16 output and FP32 log-sum-exp; null out when not fused
    unsigned long long* grid_bar;  // ticket counter of the grid barrier (workspace header)
    __half* out;
    float* lse;
    int pdl;  // host side: launch as a programmatic dependent of the preceding kernel
    // Which keys of which rows a launch covers. View::kWhole: every sequence's rows over its own
    // context. Shared-prefix attention cuts each context at `shared_keys` (below):
    // View::kSuffix covers the keys from there on, sequence by sequence; View::kPrefix the keys
    // before it, once for the rows of the whole batch (one sequence of batch * q_len tokens whose
    // block table is the prefix's; batch_q_len below is then each sequence's q_len).
    const int32_t* prefix_len;  // device scalar; null for View::kWhole
    int max_prefix;             // bound of *prefix_len
    int batch_q_len;            // View::kPrefix: tokens per sequence (q_len is the batch's total)
    int batch_max_context;      // View::kPrefix: bound of context_lens (max_context: max_prefix)
    int4* unit_slots;           // View::kSuffix: each unit's (first slot, slots, keys) for the combine
};

enum class View { kWhole, kSuffix, kPrefix };

struct CombineParams {
    const float2* ws_state;
    const float* ws_acc;
    const int32_t* context_lens;
    __half* out;
    float* lse;
    int batch, q_len, num_q_heads, num_kv_heads, group, rows;
    int max_context, num_splits, tile_keys, min_split_keys;
    int num_slots, round_slots;
    int pdl;  // host side: launch as a programmatic dependent of the preceding kernel
};

// This CTA's place in a row-blocked grid: the split position x / row_blocks (the workspace slot
// is that position plus one grid row's worth per (y, z) grid row: a single sequence launches
// (num_splits, Hkv, 1) slots, a batch (num_slots, 1, 1)) and its row range.
struct RowBlock {
    int xs;      // split position within the grid row
    int slot;    // workspace slot
    int row_lo;  // first row (of R) this CTA carries
    int rows;    // rows it carries, >= 1
};

// Host check of a launch's row blocks: every block carries 1..capacity rows and together they
// cover the R rows exactly once.
inline bool row_blocks_valid(const PartialParams& p, int capacity) {
    return p.row_blocks >= 1 && p.block_rows >= 1 && p.block_rows <= capacity &&
           (int64_t)p.row_blocks * p.block_rows >= p.rows &&
           (int64_t)(p.row_blocks - 1) * p.block_rows < p.rows;
}

__device__ __forceinline__ RowBlock row_block(const PartialParams& p) {
    RowBlock rb;
    if (p.row_blocks == 1) {  // one CTA per split: no division
        rb.xs = blockIdx.x;
        rb.row_lo = 0;
        rb.rows = p.rows;
        rb.slot = blockIdx.x + gridDim.x * (blockIdx.y + gridDim.y * blockIdx.z);
        return rb;
    }
    rb.xs = blockIdx.x / p.row_blocks;
    rb.row_lo = (blockIdx.x - rb.xs * p.row_blocks) * p.block_rows;
    rb.rows = min(p.block_rows, p.rows - rb.row_lo);
    rb.slot = rb.xs + (gridDim.x / p.row_blocks) * (blockIdx.y + gridDim.y * blockIdx.z);
    return rb;
}

// ---- programmatic dependent launch -------------------------------------------------------------
// Let the next kernel on the stream, if it was launched as this one's programmatic dependent,
// start launching its CTAs (it still waits for this grid's completion where it calls
// griddep_wait). Issued by every thread of a CTA; idempotent.
__device__ __forceinline__ void griddep_launch_dependents() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// Wait until the grid this one depends on programmatically (the preceding kernel on the stream)
// has completed and its memory writes are visible; returns at once when this grid was launched
// without the programmatic attribute. The wait ends because that grid's CTAs are all resident
// or done by the time this grid starts.
__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// For a CTA that needs nothing of the grid before it. Who waits for this grid must find that one complete
// too (its outputs may be written again): the grid's last CTA stays until it is. (Every CTA doing so would
// hold its SM for nothing.)
__device__ __forceinline__ void griddep_end() {
    if (blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1) griddep_wait();
}

// Context length of sequence b as the kernels see it: clamped into [0, max_context].
__device__ __forceinline__ int clamped_context(const int32_t* context_lens, int b, int max_context,
                                              int* flags) {
    int n = context_lens[b];
    int f = 0;
    if (n > max_context) {
        n = max_context;
        f |= DFLASH_FLAG_CONTEXT_CLAMPED;
    }
    if (n < 0) {
        n = 0;
    }
    *flags = f;
    return n;
}

// Keys that a batch takes from its shared prefix: the prefix's whole pages (a page that the prefix
// ends in is in every sequence's own row). Sets DFLASH_FLAG_CONTEXT_CLAMPED for a length above the
// plan's.
__device__ __forceinline__ int shared_keys(const int32_t* prefix_len, int max_prefix,
                                           int page_size, int* flags) {
    int n = *prefix_len;
    if (n > max_prefix) {
        n = max_prefix;
        *flags |= DFLASH_FLAG_CONTEXT_CLAMPED;
    }
    return n <= 0 ? 0 : n / page_size * page_size;
}

// Keys per split for context n (the rule dflash_verify_attn_split_bounds restates on the host).
__device__ __forceinline__ int keys_per_split(int n, int num_splits, int tile_keys,
                                              int min_split_keys) {
    int per = (n + num_splits - 1) / num_splits;
    per = per > min_split_keys ? per : min_split_keys;
    return (per + tile_keys - 1) / tile_keys * tile_keys;
}

// A block-table entry clamped into the pool of num_pages pages.
__device__ __forceinline__ int clamp_page(int phys, int num_pages, bool* clamped) {
    if (phys < 0 || phys >= num_pages) {
        *clamped = true;
        phys = phys < 0 ? 0 : num_pages - 1;
    }
    return phys;
}

// Physical page of logical page lp of sequence b, clamped into the pool.
__device__ __forceinline__ int physical_page(const int32_t* block_table, int b,
                                             int max_pages_per_seq, int lp, int num_pages,
                                             bool* clamped) {
    return clamp_page(block_table[(int64_t)b * max_pages_per_seq + lp], num_pages, clamped);
}

// ---- split slots of a batch -------------------------------------------------------------------
// The plan's C split slots (one CTA each; as many as the GPU runs at once unless the split
// count is forced, then batch * Hkv * S) are shared out among the (sequence, KV head) units so
// that the busiest slot has as few 128-key tiles as possible. With w_b = ceil(n_b / 128) tiles
// in sequence b, T is the smallest tile count with
//   Hkv * sum_b ceil(w_b / T) <= C,
// and each KV head of sequence b owns c_b = ceil(w_b / T) contiguous slots, unit u = b * Hkv + h
// from slot Hkv * (c of the sequences before b) + h * c_b; the slots past all units stay idle.
// A unit's splits then hold at most T tiles each (the least any split of the units into
// contiguous pieces achieves), an empty unit owns no slot. A single sequence keeps num_splits
// slots per KV head (the same splits: its units are equal). dflash_verify_attn_split_slots does
// the same integer arithmetic on the host.
//
// With as many units as SMs, or more, one slot each would leave a long sequence to a single CTA. A plan of
// several rounds (round_slots of its slots run at once) has slots to spare for every unit, and how many of them
// a batch takes goes by its lengths: those of one round (or one a unit), or all, whichever
// is expected to be done sooner. A slot costs kSlotStart tiles beside its own; the slots of one round take the
// longest's time, those of several the mean work of an SM and 0.4 (a slot a unit) or 0.3 (all slots) of the longest's. The longest is
// not searched for twice: c slots a KV head for E sequences of w tiles in all leave about w / (c - E / 2)
// tiles a split, half a split a sequence being lost, and the longest sequence c - E + 1 of them at most. Measured
// for the 4-bit attention, us with one round (or a slot a unit) and with all of the plan's slots, contexts of
// L / 3 to L tokens, what is chosen in brackets. 24/4 heads, one token a sequence:
//   units    L = 1024        L = 4096          L = 16384         one of 262144 among units of 1000 tokens
//     96     [18.5] 23.3     [29.6] 35.2       102.9 [88.7]
//    128     [18.6] 25.4     [40.7] 43.1       122.9 [105.3]
//    152     [20.8] 29.3     [44.6] 49.9       143.0 [136.4]     2063 [139]
//    156     [24.2] 29.2     48.4 [51.4]       141.9 [144.6]     2062 [102]
//    192     [30.3] 32.8     65.1 [56.8]       206.4 [149.8]
//    256     [33.8] 44.1     [75.6] 78.8       216.0 [202.7]
//    384     [51.2] 64.9     [112.2] 116.9     321.8 [317.2]     2108 [150] (400 units)
// and of 48 rows: 24/4 heads 96 units L = 4096 [45] 52, 16384 141 [123], 156 units 4096 77 [83], 16384 202
// [208]; 6/1 heads L = 4096, 80 units [48] 55, 152 [83] 98, 160 108 [102], 256 [161] 179.
// The choice costs 1 us, slots left idle 2.
constexpr int kSlotStart = 8;
__host__ __device__ __forceinline__ int slots_of_lengths(long long w, int longest, int E, int Hkv, int slots,
                                                         int round) {
    const int units = E * Hkv, first = units > round ? units : round;
    if (slots <= first) return slots;
    auto split = [&](int C) {  // tiles of the longest split
        const int c = C / Hkv, one = longest / (c - E + 1) + 1;
        const long long even = 2 * w / (2ll * c - E) + 1, T = even > one ? even : one;
        return T < longest ? T : longest;
    };
    // ten times `round` times the tiles' time of n slots, T tiles the longest
    auto slots_time = [&](int n, long long T, int tenths) {
        const long long last = (T + kSlotStart) * round;
        return n <= round ? 10 * last : 10 * (w * Hkv + (long long)n * kSlotStart) + tenths * last;
    };
    return slots_time(slots, split(slots), 3) < slots_time(first, split(first), 4) ? slots : first;
}

struct UnitSlots {
    int b, h;    // the unit (b = -1: no unit owns the slot)
    int first;   // its first slot
    int count;   // its slot count (its split count)
    int n;       // context length of sequence b, clamped to [0, max_context]
    int flags;   // DFLASH_FLAG_CONTEXT_* of the whole batch
};

__device__ __forceinline__ int slot_granules(int n) { return (n + 127) >> 7; }

// The clamped length of sequence b past its first `base` keys; sets the batch's context flags.
__device__ __forceinline__ int slot_length(const int32_t* context_lens, int b, int max_context,
                                           int q_len, int* flags, int base = 0) {
    int n = context_lens[b];
    if (n > max_context) {
        n = max_context;
        *flags |= DFLASH_FLAG_CONTEXT_CLAMPED;
    }
    n = n < 0 ? 0 : n;
    if (n < q_len) *flags |= DFLASH_FLAG_CONTEXT_SHORT;
    return max(n - base, 0);
}

// Slots of a single sequence: its units are equal, S slots each.
__device__ __forceinline__ UnitSlots locate_slots_single(const int32_t* context_lens, int Hkv,
                                                         int S, int max_context, int q_len,
                                                         int key, bool by_slot,
                                                         int base = 0) {
    UnitSlots r = {-1, 0, 0, 0, 0, 0};
    int flags = 0;
    const int n = slot_length(context_lens, 0, max_context, q_len, &flags, base);
    const int u = by_slot ? key / S : key;
    r.flags = flags;
    if (n == 0 || u >= Hkv) return r;
    r.b = 0;
    r.h = u;
    r.first = u * S;
    r.count = S;
    r.n = n;
    return r;
}

// Slots of a batch of several sequences. Warp-cooperative: every lane of the warp calls it with
// the same arguments and gets the same result. by_slot: the unit owning slot key; else the slots
// of unit key. kRounds: with round_slots.
template <bool kRounds>
__device__ __forceinline__ UnitSlots locate_slots_batch_body(const int32_t* context_lens,
                                                             int B, int Hkv, int num_slots,
                                                             int round_slots, int max_context,
                                                             int q_len, int key, bool by_slot,
                                                             int base) {
    const int lane = threadIdx.x & 31;
    UnitSlots r = {-1, 0, 0, 0, 0, 0};
    int unused = 0;
    auto tiles = [&](int b) {  // w_b (0 past the batch)
        return b < B ? slot_granules(slot_length(context_lens, b, max_context, q_len, &unused, base))
                     : 0;
    };
    // tiles in all (W), the longest sequence, non-empty sequences, the batch's context flags
    long long W = 0;
    int wmax = 0, E = 0, flags = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
        const int b = b0 + lane;
        const int w =
            b < B ? slot_granules(slot_length(context_lens, b, max_context, q_len, &flags, base))
                  : 0;
        W += w;
        wmax = max(wmax, w);
        E += w > 0;
    }
    for (int o = 16; o > 0; o >>= 1) {
        W += __shfl_xor_sync(0xffffffffu, W, o);
        wmax = max(wmax, __shfl_xor_sync(0xffffffffu, wmax, o));
        E += __shfl_xor_sync(0xffffffffu, E, o);
        flags |= __shfl_xor_sync(0xffffffffu, flags, o);
    }
    r.flags = flags;
    if (W == 0) return r;
    const long long U = (long long)Hkv * E;
    // slots that splits of T tiles need (counts of tiles stay below 2^24)
    auto need = [&](int T) {
        long long sum = 0;
        for (int b0 = 0; b0 < B; b0 += 32)
            sum += (unsigned)(tiles(b0 + lane) + T - 1) / (unsigned)T;
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        return sum * Hkv;
    };
    // T: binary search between W Hkv / C (no split can do better) and the first count that is
    // surely enough, W Hkv / (C - U) (U = Hkv E: each unit's last split may be short), or wmax
    long long C = num_slots;
    if constexpr (kRounds) {
        C = slots_of_lengths(W, wmax, E, Hkv, num_slots, round_slots);
        if (by_slot && key >= C) return r;  // a slot of the rounds that this batch leaves out
    }
    int hi = wmax;
    if (C > U) hi = (int)min((long long)hi, (W * Hkv + (C - U) - 1) / (C - U));
    int lo = (int)max(1ll, min((W * Hkv + C - 1) / C, (long long)hi));
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (need(mid) <= C)
            hi = mid;
        else
            lo = mid + 1;
    }
    const int T = lo;
    // slots per KV head of each sequence, scanned over the batch
    int c_carry = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
        const int b = b0 + lane;
        const int n = b < B ? slot_length(context_lens, b, max_context, q_len, &unused, base) : 0;
        const int c = (slot_granules(n) + T - 1) / T;
        int sc = c;  // inclusive scan over the chunk
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, sc, o);
            if (lane >= o) sc += t;
        }
        const int c_before = c_carry + sc - c;  // per KV head, sequences before b
        const bool mine = by_slot ? (b < B && c > 0 && key >= Hkv * c_before &&
                                     key < Hkv * (c_before + c))
                                  : b == key / Hkv;
        const unsigned m = __ballot_sync(0xffffffffu, mine);
        if (m) {
            const int src = __ffs(m) - 1;
            const int cb0 = __shfl_sync(0xffffffffu, c_before, src);
            const int cb = __shfl_sync(0xffffffffu, c, src);
            const int nb = __shfl_sync(0xffffffffu, n, src);
            const int hh = by_slot ? (key - Hkv * cb0) / cb : key % Hkv;
            r.b = b0 + src;
            r.h = hh;
            r.first = Hkv * cb0 + hh * cb;
            r.count = cb;
            r.n = nb;
            return r;
        }
        c_carry += __shfl_sync(0xffffffffu, sc, 31);
    }
    return r;
}

template <bool kRounds>
static __device__ __noinline__ UnitSlots locate_slots_batch(const int32_t* context_lens, int B,
                                                            int Hkv, int num_slots,
                                                            int round_slots, int max_context,
                                                            int q_len, int key, bool by_slot,
                                                            int base) {
    return locate_slots_batch_body<kRounds>(context_lens, B, Hkv, num_slots, round_slots, max_context,
                                            q_len, key, by_slot, base);
}

// The slots of a unit or the unit of a slot (see above). Warp-cooperative. The several-sequence
// search is called out of line: it runs once per CTA, and the kernels' hot code stays compact.
__device__ __forceinline__ UnitSlots locate_slots(const int32_t* context_lens, int B, int Hkv,
                                                  int S, int num_slots, int max_context,
                                                  int q_len, int key, bool by_slot,
                                                  int base = 0, int round_slots = 0) {
    if (B == 1)
        return locate_slots_single(context_lens, Hkv, S, max_context, q_len, key, by_slot, base);
    if (round_slots)
        return locate_slots_batch<true>(context_lens, B, Hkv, num_slots, round_slots, max_context,
                                        q_len, key, by_slot, base);
    return locate_slots_batch<false>(context_lens, B, Hkv, num_slots, 0, max_context, q_len, key,
                                     by_slot, base);
}

// Grid of a partial launch: (splits x row blocks, Hkv, 1) for a single sequence, (slots x row
// blocks, 1, 1) for a batch.
inline dim3 partial_grid(const PartialParams& p) {
    return p.batch == 1 ? dim3(p.num_splits * p.row_blocks, p.num_kv_heads, 1)
                        : dim3(p.num_slots * p.row_blocks, 1, 1);
}

}  // namespace dflash
