// mx4_attn.cu -- attention of drafted tokens over the 4-bit cache (dflash_mx4_attn_*): the tensor-core partial
// kernel and its entry points. Splits, slots, split state and combine are those of the E4M3 attention.
//
// One CTA per (split, KV head, sequence) and block of up to 48 query rows. Both products have FP16 operands
// (every number of the cache times a power of two is exact, Q is FP16, P is rounded to it) and FP32 sums, keys or
// head-dim elements on the 128 lanes: S^T = K Q^T and O^T = V^T P^T. What bounds such a kernel is shared
// memory: stored there as FP16, a tile of 128 keys would be written (128 KB) and read by the tensor core
// (128 KB), 2048 clocks of 128 bytes, while its codes come from HBM in 1500. So neither K nor V goes there
// decoded: both are the products' first operand, which may lie in tensor memory, and warps write it from
// registers, a lane a key of K, or two elements of the head, i and i + 128, of V. The cache's layout
// is made for that (dflash_mx4_cache.h): a thread reads its codes in 16-byte pieces without bank
// conflicts, and a chunk of 16 tokens comes by one bulk copy.
//
//  * Scales. A key of K is brought to 2^12 of its largest block's power and the rest, one power of two a
//    key, goes into the factor of its scores. V's rest goes into the weights: with ev = the key's largest
//    exponent (cut to +-40) the kernel takes p = 2^(s + ev - m), m the reference of s + ev, sums p 2^-ev
//    for the denominator and multiplies p by v 2^-ev. A weight is so large only if its value is.
//  * Probabilities are p 2^8 of a row's first maximum and move their reference past 2^15: below 2^-14
//    FP16 has a fixed step, 2^-24, 2^-32 of the largest at least. Their rounding to FP16 (2^-11, as the output's)
//    takes the error against 64 bits from 2.1e-4 to 2.9e-4 of the output; a second term of P would double
//    the output's products. The denominator sums them unrounded.
//  * NaN. A key with a NaN scale in K or V gets a NaN factor or exponent: its probability is NaN in
//    every row that sees it and 0, selected, in the others. V's own factors are finite.
//  * Warps: 0 copies the codes (four tiles ahead), 1 and 2 issue the products of the scores and of the
//    output, 3 works out the factors of a tile's keys, 4-7 decode K, 8-11 V, the others are the softmax, four
//    for 16 rows.
//  * Every wait on another warp or on a copy is bounded: on a timeout the CTA sets
//    DFLASH_FLAG_KERNEL_TIMEOUT, sees its copies and products through (bounded too) and returns.
//
// Measured with the combine, in a graph: 24/4 heads, 8 drafted tokens over 261888 tokens 84 us, 50 % of the copy
// rate; 32 sequences of one token up to 16384 long, 24/4 heads, 106 us, 56 %; one rank, 8 tokens over 261888
// tokens 30.4 us. What bounds it is the warps: 7810 warp instructions a tile for 48 rows in 3150 clocks, 5430
// for 16 in 2450, 68 and 61 % of the issue slots, with no role ahead of the others by more than a
// few hundred clocks. They share the instruction caches, so that fewer instructions in a loop count
// for more than their number, and unrolling costs: hence the rolled loops (two chunks of V at a time 104 us
// for 99, two blocks of K 135 for 130 us of the single tokens).
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "dflash_mx4_cache.h"
#include "mx4.cuh"
#include "tc_ptx.cuh"

namespace dflash {
int check_attn_plan(const dflash_verify_attn_plan_t* plan);
PartialParams attn_params(const dflash_verify_attn_plan_t* plan, const void* q, const void* k_pool,
                          const void* v_pool, const int32_t* block_table,
                          const int32_t* context_lens, const float* k_scale, const float* v_scale,
                          void* workspace);
CombineParams combine_params(const dflash_verify_attn_plan_t* plan, const void* workspace,
                             const int32_t* context_lens, void* out, float* lse);
cudaError_t launch_combine(const CombineParams& p, cudaStream_t stream);
int round_slots(const dflash_verify_attn_plan_t& plan);

namespace mx4 {

using namespace ptx;

constexpr int kTile = 128;       // keys per tile = MMA M
constexpr int kChunks = kTile / kTokens;
constexpr int kMaxRP = 48;       // padded rows a CTA carries
constexpr int kGroupRows = 16;
constexpr int kStages = 4;       // tiles of codes of K, and of V, on their way
constexpr int kInfos = 4;        // tiles of factors
constexpr uint32_t kStageBytes = kChunks * kChunkBytes;
constexpr uint64_t kWaitLimitNs = 200ull * 1000 * 1000;
constexpr uint32_t kSuspendNs = 20000;
constexpr float kShift = 8.f;          // probabilities are 2^8 at the reference
constexpr float kLazyThreshold = 15.f; // largest exponent of one
constexpr int kFactorTop = 12;         // a key's largest block is brought to 2^12
constexpr int kMaxEv = 40;
// Largest scale byte of a key of K, 2^100: a score is below 2^38.6 (256 products of 65504 and 6 2^12) times the
// factor 2^84.6, so that it stays a number. An infinite one could not be told from that of a key not seen.
constexpr int kMaxKe = 127 + 100;
constexpr int kKWarp = 4, kVWarp = 8, kSoftWarp = 12;

// Shared memory: Q | P | codes of K | codes of V | factors | Small. Tensor memory: K [two head-dim
// halves][64] | V [two halves of the keys][64] | S [two tiles][RP] | O [two halves of
// the head dim][RP].
template <int RP>
struct Cfg {
    static constexpr int kGroups = RP / kGroupRows;
    static constexpr int kSoftWarps = 4 * kGroups;
    static constexpr int kThreads = 32 * (kSoftWarp + kSoftWarps);
    static constexpr uint32_t kOffP = RP * kHeadDim * 2;
    static constexpr uint32_t kPBytes = 2 * RP * 2 * kTile * 2;
    static constexpr uint32_t kOffK = kOffP + kPBytes;
    static constexpr uint32_t kOffV = kOffK + kStages * kStageBytes;
    static constexpr uint32_t kOffInfo = kOffV + kStages * kStageBytes;
    static constexpr uint32_t kColK = 0, kColV = 128, kColS = 256, kColO = kColS + 2 * RP;
    static constexpr uint32_t kTmemCols = 512;
    static_assert(RP % kGroupRows == 0 && RP <= kMaxRP, "rows per CTA");
    static_assert(kColO + 2 * RP <= kTmemCols, "tensor memory");
    static_assert(kOffP % 1024 == 0 && kOffK % 128 == 0 && kOffInfo % 16 == 0, "alignment");
};

// Factors of a tile's keys: of their scores (in log2 units), V's exponent, and of V's blocks (FP16).
struct Info {
    float2 c[kTile];  // (score factor, V's exponent)
    uint32_t f[kBlocks / 2][kTile];  // blocks j and j + 4
};

struct Small {
    uint64_t full[kStages], empty[kStages];  // of codes
    uint64_t infofull[kInfos], infofree[kInfos];
    uint64_t kafull[2], kafree[2], vafull[2], vafree[2];  // halves of the operands in tensor memory
    uint64_t sfull[2], sfree[2], pfull, pfree, odone, qready;
    uint32_t tmem_base;
    int abort;
    int never;  // stays 0: for a wait that goes on when the CTA gives up
    float rmax[kMaxRP / kGroupRows][4][kGroupRows];   // per-group, per-warp row maxima of a tile
    float rsum[kMaxRP / kGroupRows][4][kGroupRows];   // per-group, per-warp row sums of the split
    float mref[kMaxRP / kGroupRows][kGroupRows];      // the split state's max of each row
    float nmcur[kMaxRP / kGroupRows][4][kGroupRows];  // each warp's copy of the shift minus the reference
};

template <int RP>
constexpr uint32_t smem_bytes() {
    return Cfg<RP>::kOffInfo + kInfos * sizeof(Info) + sizeof(Small);
}
static_assert(smem_bytes<kMaxRP>() <= 227 * 1024, "shared memory budget");
static_assert(sizeof(Info) % 16 == 0, "factors are read in 16-byte pieces");

// Byte offset of (row, 16-byte piece u of its 512 bytes) of Q: K-major with the 128-byte swizzle, 8-row groups
// 1 KB apart, blocks of 64 elements rows * 128 bytes apart.
__device__ __forceinline__ uint32_t q_off(int row, int u, int rows) {
    return (u >> 3) * rows * 128 + (row >> 3) * 1024 + (row & 7) * 128 + (((u & 7) ^ (row & 7)) << 4);
}
// P, the output's second operand. A byte of V's codes holds elements e and e + 128 of a key, and decoded as they
// lie they are neighbours in the contraction, which so runs over 2 x 128 places: place 2 key has the key's
// weights in columns row, place 2 key + 1 in columns RP + row, and zeros are in the others. That doubles the
// products' work, of which there is room for, and spares V's decoder the sorting of half bytes into pairs of
// keys, a third of its operations (24/4 heads over 261888 tokens 105 -> 99 us).
// MN-major without swizzle, core matrices of 8 rows x 8 places (of 16 bytes each): groups of places 128
// bytes apart (the descriptor's leading offset), blocks of 8 rows 4 KB (its stride offset).
__device__ __forceinline__ uint32_t p_off(int row_block, int k) {
    return row_block * 4096 + (k >> 3) * 128 + (k & 7) * 16;
}

__device__ __forceinline__ float f32(uint32_t x) { return __uint_as_float(x); }

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a),
                              *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// 2^e twice as FP16x2 bits, for e <= 13; 0 below 2^-14 (an exponent field of 0).
__device__ __forceinline__ uint32_t f16x2_power(int e) { return (uint32_t)max(e + 15, 0) * 0x04000400u; }

// D += A B^T over 16 elements of K, FP16: A in tensor memory (a lane a row, two elements a column).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// One lane of a whole warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// kChunkBytes from global to shared memory (both 16-byte aligned).
__device__ __forceinline__ void copy_chunk(uint32_t dst, const uint8_t* src, uint32_t bar,
                                           uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1], %2, [%3], %4;" ::"r"(dst),
        "l"(src), "r"((uint32_t)kChunkBytes), "r"(bar), "l"(policy)
        : "memory");
}

// One try, for which the hardware may suspend the thread up to the hinted time.
__device__ __forceinline__ bool try_wait_hint(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kSuspendNs)
        : "memory");
    return ok != 0;
}

// The rest of a wait whose first try failed. Not inlined: the warps' loops compete for the instruction caches, and
// with this code at each of twenty waits 32 sequences of one token took 158 us for 155. (Reading the clock
// between the tries keeps them apart: without, the waiting warps took the others' time, 131 us for 109.)
__device__ __noinline__ bool wait_on(uint32_t addr, uint32_t parity, volatile int* abort,
                                     int32_t* status) {
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        if (try_wait_hint(addr, parity)) return true;
        if (*abort) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) break;
    }
    *abort = 1;
    atomicOr(status, DFLASH_FLAG_KERNEL_TIMEOUT);
    return false;
}

struct Ctx {
    Small* sm;
    int32_t* status;
    __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) const {
        const uint32_t addr = smem_u32(bar);
        return try_wait_hint(addr, parity) || wait_on(addr, parity, &sm->abort, status);
    }
    // by a whole warp, whose lanes agree on the result. What follows (tcgen05.ld and st, group barriers) wants
    // them together: a first try may succeed for some lanes only, and the vote alone does not promise it.
    __device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) const {
        const bool ok = __all_sync(0xffffffffu, wait(bar, parity));
        __syncwarp();
        return ok;
    }
    __device__ bool aborted() const { return *reinterpret_cast<volatile int*>(&sm->abort) != 0; }
};

// Place of a tile in a ring of kN, and the parity of its phase there.
template <int kN>
struct Ring {
    int i = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++i == kN) {
            i = 0;
            parity ^= 1;
        }
    }
};

// This warp has done with what `bar` counts.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(bar));
}
// ... and its stores to tensor memory are complete.
__device__ __forceinline__ void warp_arrive_tmem(uint64_t* bar) {
    tmem_st_wait();
    tc_fence_before();
    warp_arrive(bar);
}

// Named barrier of one softmax group's 128 threads, optionally OR-reducing a vote. After a failed wait a warp goes
// on to the next vote, which takes all four out of the loop (what it computes until then is not stored:
// the launch has failed), so each barrier is reached by all of them.
__device__ __forceinline__ bool group_vote(int g, bool v) {
    uint32_t r;
    __syncwarp();  // (lanes may come from a branch of their own)
    asm volatile(
        "{\n\t.reg .pred pv, pr;\n\t"
        "setp.ne.u32 pv, %1, 0;\n\t"
        "bar.red.or.pred pr, %2, 128, pv;\n\t"
        "selp.u32 %0, 1, 0, pr;\n\t}"
        : "=r"(r)
        : "r"(v ? 1u : 0u), "r"(1 + g)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void group_bar(int g) {
    __syncwarp();
    asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory");
}

// A transposed butterfly over the warp: each step trades half of the rows with the lane `off` away, so that
// lane l ends with op over the lanes of row (l >> 1) & 15.
template <typename Op>
__device__ __forceinline__ float rows_reduce(float (&v)[kGroupRows], int lane, Op op) {
#pragma unroll
    for (int half = kGroupRows / 2, off = 16; half >= 1; half >>= 1, off >>= 1) {
        const bool upper = (lane & off) != 0;
#pragma unroll
        for (int j = 0; j < half; ++j) {
            const float keep = upper ? v[j + half] : v[j];
            const float send = upper ? v[j] : v[j + half];
            v[j] = op(keep, __shfl_xor_sync(0xffffffffu, send, off));
        }
    }
    return op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

__device__ __forceinline__ int largest_byte(uint2 s) {
    // halves of 16 bits, whose upper bytes decide
    const uint32_t m = __vmaxu2(__vimax3_u16x2(s.x, s.y, s.x << 8), s.y << 8);
    return (int)(__vmaxu2(m, m << 16) >> 24);
}

// One warp's copies of both pools, tile after tile into their rings: lane c < 8 copies chunk c of K, lane 8 + c
// of V. All lanes look up the block table, for four tiles at a time and ahead.
__device__ __forceinline__ void copy_tiles(const PartialParams& p, const Ctx& ctx, uint8_t* k_ring,
                                           uint8_t* v_ring, int b, int h, int start, int end,
                                           int ntiles, int drafted) {
    const int lane = threadIdx.x & 31;
    Small& sm = *ctx.sm;
    const uint64_t policy = l2_evict_first_policy();  // every page is read once
    bool clamped = false;
    // pool chunk that this lane's place among four tiles from tile t on has (-1 past the end)
    auto ahead = [&](int t) -> int64_t {
        const int j = start + t * kTile + lane * kTokens;
        if (j >= end) return -1;
        const int lp = p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size;
        const int phys = physical_page(p.block_table, b, p.max_pages_per_seq, lp, p.num_pages,
                                       &clamped);
        return (int64_t)phys * (p.page_size / kTokens) + (j - lp * p.page_size) / kTokens;
    };
    const bool is_v = lane >= kChunks;
    const int c = lane & (kChunks - 1);
    const uint8_t* pool = is_v ? p.v_pool : p.k_pool;
    const uint32_t ring = smem_u32((is_v ? v_ring : k_ring) + c * kChunkBytes);
    int64_t next = ahead(0), now = -1;
    bool dep_done = false;
    int t = 0;
    Ring<kStages> ring_at;
#pragma unroll 1
    for (; t < ntiles; ++t, ring_at.next()) {
        if ((t & 3) == 0) {
            now = next;
            next = ahead(t + 4);
        }
        const int s = ring_at.i;
        const uint32_t parity = ring_at.parity ^ 1;
        if (!ctx.wait_warp(&sm.empty[s], parity)) break;
        // keys from `drafted` on may be written by the kernel just before this one
        if (!dep_done && start + (t + 1) * kTile > drafted) {
            griddep_wait();
            dep_done = true;
        }
        const int64_t chunk = __shfl_sync(0xffffffffu, now, (t & 3) * kChunks + c);
        const int n = min(kChunks, (end - start - t * kTile + kTokens - 1) / kTokens);
        if (lane == 0) mbar_arrive_expect_tx(smem_u32(&sm.full[s]), 2 * n * kChunkBytes);
        __syncwarp();
        if (lane < 2 * kChunks && c < n)
            copy_chunk(ring + s * kStageBytes, pool + (chunk * p.num_kv_heads + h) * kChunkBytes,
                       smem_u32(&sm.full[s]), policy);
    }
    if (clamped) atomicOr(p.status, DFLASH_FLAG_PAGE_CLAMPED);
    // no copy may still be writing shared memory when the CTA retires
    __syncwarp();
    if (lane == 0)
#pragma unroll 1
        for (int u = t - kStages < 0 ? 0 : t - kStages; u < t; ++u)
            mbar_wait(smem_u32(&sm.full[u % kStages]), (u / kStages) & 1, &sm.never, kWaitLimitNs);
}

template <int RP>
__global__ void __launch_bounds__(Cfg<RP>::kThreads, 1)
    mx4_partial_kernel(const PartialParams p) {
    using C = Cfg<RP>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Info* const infos = reinterpret_cast<Info*>(smem + C::kOffInfo);
    Small& sm = *reinterpret_cast<Small*>(smem + C::kOffInfo + kInfos * sizeof(Info));
    // (the shuffle tells the compiler that a warp's roles, loops and addresses are the same in all its lanes)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const RowBlock rblk = row_block(p);
    const int R = rblk.rows, row_lo = rblk.row_lo, G = p.group, slot = rblk.slot;
    griddep_launch_dependents();
    const UnitSlots us =
        p.batch == 1 ? locate_slots_single(p.context_lens, p.num_kv_heads, p.num_splits,
                                           p.max_context, p.q_len, blockIdx.y, false)
                     : locate_slots(p.context_lens, p.batch, p.num_kv_heads, p.num_splits,
                                    p.num_slots, p.max_context, p.q_len, slot, true, 0, p.round_slots);
    if (slot == 0 && tid == 0 && us.flags) atomicOr(p.status, us.flags);
    const int b = us.b, h = us.h, split = slot - us.first, n = us.n;
    const int per = b < 0 ? 1 : keys_per_split(n, us.count, kTile, p.min_split_keys);
    const int start = split * per;
    if (b < 0 || start >= n) {  // idle slot: the combine never reads it
        griddep_end();
        return;
    }
    const int end = min(n, start + per);
    const int ntiles = (end - start + kTile - 1) / kTile;
    if (smem_u32(smem) & 1023u) {  // the swizzled layouts need a 1 KB aligned base
        if (tid == 0) atomicOr(p.status, DFLASH_FLAG_KERNEL_TIMEOUT);
        return;
    }
    const Ctx ctx{&sm, p.status};
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&sm.full[i]), 1);
            mbar_init(smem_u32(&sm.empty[i]), 9);  // eight decoders and the factors' warp
        }
        for (int i = 0; i < kInfos; ++i) {
            mbar_init(smem_u32(&sm.infofull[i]), 1);
            mbar_init(smem_u32(&sm.infofree[i]), 4 + C::kSoftWarps);  // V's decoders, softmax
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sm.kafull[i]), 4);
            mbar_init(smem_u32(&sm.kafree[i]), 1);
            mbar_init(smem_u32(&sm.vafull[i]), 4);
            mbar_init(smem_u32(&sm.vafree[i]), 1);
            mbar_init(smem_u32(&sm.sfull[i]), 2);  // the products, and the tile's factors
            mbar_init(smem_u32(&sm.sfree[i]), C::kSoftWarps);
        }
        mbar_init(smem_u32(&sm.pfull), C::kSoftWarps);
        mbar_init(smem_u32(&sm.pfree), 1);
        mbar_init(smem_u32(&sm.odone), 2);  // both threads that issue products
        mbar_init(smem_u32(&sm.qready), C::kSoftWarps);
        sm.abort = sm.never = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&sm.tmem_base), C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);

    if (warp == 0) {
        copy_tiles(p, ctx, smem + C::kOffK, smem + C::kOffV, b, h, start, end, ntiles, n - p.q_len);
    } else if (warp == 1 || warp == 2) {
        // ---------------------------------------------------------------- products
        // One thread issues the scores, another the output: a product takes its thread some 50 clocks, the
        // tensor core half of that for the scores (N 48: 24 with two threads, 46 with one) and as long for
        // the output (N 96), a commit or a wait 50 to 80. Each product's addresses are a base and a constant:
        // worked out from the indices they took 145 clocks a product. Both operands come in halves (of the
        // head dim, of the keys), so that one is decoded while the other is read.
        const bool issuer = elect_one();
        bool ok = issuer && ctx.wait(&sm.qready, 0);
        if (warp == 1 && issuer) {
            constexpr uint32_t idesc = idesc_f32acc(128, RP, 0, 0, 0, 0);
            const uint32_t qb = smem_u32(smem);
            auto tile = [&](int kS, int t) {
                ok = ctx.wait(&sm.sfree[kS], ((t >> 1) & 1) ^ 1);
#pragma unroll 1
                for (int hd = 0; hd < 2; ++hd) {
                    ok = ok && ctx.wait(&sm.kafull[hd], kS);
                    if (!ok) return;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_ts(C::kColS + kS * RP, C::kColK + hd * 64 + kk * 8,
                               smem_desc(qb + (2 * hd + (kk >> 2)) * (RP * 128) + (kk & 3) * 32, 16, 1024,
                                         kSwizzle128B),
                               idesc, hd || kk);
                    mma_commit(smem_u32(&sm.kafree[hd]));
                }
                mma_commit(smem_u32(&sm.sfull[kS]));
                // the softmax reads the factors of a tile's keys with its scores: one wait for both
                ok = ctx.wait(&sm.infofull[t % kInfos], (t / kInfos) & 1);
                if (ok) mbar_arrive(smem_u32(&sm.sfull[kS]));
            };
#pragma unroll 1
            for (int t = 0; ok && t < ntiles; ++t) tile(t & 1, t);
        } else if (issuer) {
            constexpr uint32_t idesc = idesc_f32acc(128, 2 * RP, 0, 0, 0, 1);
            const uint32_t pb = smem_u32(smem + C::kOffP);
#pragma unroll 1
            for (int t = 0; ok && t < ntiles; ++t) {
                ok = ctx.wait(&sm.pfull, t & 1);
#pragma unroll
                for (int hv = 0; hv < 2; ++hv) {
                    ok = ok && ctx.wait(&sm.vafull[hv], t & 1);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_ts(C::kColO, C::kColV + hv * 64 + kk * 8,
                               smem_desc(pb + (8 * hv + kk) * 256, 128, 4096, kSwizzleNone), idesc,
                               hv || kk || t != 0);
                    mma_commit(smem_u32(&sm.vafree[hv]));
                }
                if (ok) mma_commit(smem_u32(&sm.pfree));
            }
        }
        if (issuer) mma_commit(smem_u32(&sm.odone));  // tracks every product this thread issued
        __syncwarp();
    } else if (warp == 3) {
        // ---------------------------------------------------------------- factors of a tile's keys
        constexpr float kScore = 0.0625f * kLog2e / (1 << kFactorTop);  // D^-1/2 = 1/16
        Ring<kStages> ring;
        Ring<kInfos> iring;
#pragma unroll 1
        for (int t = 0; t < ntiles; ++t, ring.next(), iring.next()) {
            const int s = ring.i, is = iring.i;
            if (!ctx.wait_warp(&sm.infofree[is], iring.parity ^ 1) ||
                !ctx.wait_warp(&sm.full[s], ring.parity))
                break;
            Info& info = infos[is];
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                const int key = lane + 32 * i;
                const uint32_t at = (key / kTokens) * kChunkBytes + kCodeBytes + (key % kTokens) * kBlocks;
                const uint2 ks = *reinterpret_cast<const uint2*>(smem + C::kOffK + s * kStageBytes + at);
                const uint2 vs = *reinterpret_cast<const uint2*>(smem + C::kOffV + s * kStageBytes + at);
                const int ke = largest_byte(ks), ve = largest_byte(vs);
                const int ev = max(-kMaxEv, min(kMaxEv, ve - 127));
                info.c[key] = make_float2(ke == kNanScale ? NAN : __int_as_float(min(ke, kMaxKe) << 23) * kScore,
                                          ve == kNanScale ? NAN : (float)ev);
                // block j's factor is 2^(s - 127 - ev + 12), at most 2^13 (finite for a NaN block and for
                // whatever lies past the split's end: those weights are NaN and 0), and 0 for blocks
                // 2^26 below the key's largest
                const uint32_t shift = ((uint32_t)(kFactorTop + 15 - 127 - ev) & 0xFFFFu) * 0x00010001u;
#pragma unroll
                for (int j = 0; j < kBlocks / 2; ++j) {
                    const uint32_t two = __byte_perm(vs.x, vs.y, j | (4 + j) << 8) & 0x00FF00FFu;
                    info.f[j][key] = __viaddmin_s16x2_relu(two, shift, (kFactorTop + 16) * 0x00010001u)
                                     << 10;
                }
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&sm.empty[s]));
                mbar_arrive(smem_u32(&sm.infofull[is]));
            }
        }
    } else if (warp < kVWarp) {
        // ---------------------------------------------------------------- K: lane = key
        const int key = (warp - kKWarp) * 32 + lane;
        const uint32_t at = (key / kTokens) * kChunkBytes + (key % kTokens) * 16;
        const uint32_t scales = (key / kTokens) * kChunkBytes + kCodeBytes + (key % kTokens) * kBlocks;
        Ring<kStages> ring;
#pragma unroll 1
        for (int t = 0; t < ntiles; ++t, ring.next()) {
            const int s = ring.i;
            if (!ctx.wait_warp(&sm.full[s], ring.parity)) break;
            const uint8_t* stage = smem + C::kOffK + s * kStageBytes;
            const uint2 sc = *reinterpret_cast<const uint2*>(stage + scales);
            const int top = largest_byte(sc) - kFactorTop;
            bool ok = true;
#pragma unroll 1
            for (int hd = 0; hd < 2; ++hd) {
                const uint8_t* codes = stage + at + 4 * hd * 256;
                uint32_t scale = hd ? sc.y : sc.x;
                ok = ctx.wait_warp(&sm.kafree[hd], (t & 1) ^ 1);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int j = 0; j < 4; ++j) {
                    const uint32_t f = f16x2_power((int)(scale & 255u) - top);
                    const uint4 next = *reinterpret_cast<const uint4*>(codes + j * 256);
                    const uint32_t u[4] = {next.x, next.y, next.z, next.w};
                    scale >>= 8;
                    uint32_t o[16];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        o[4 * i] = mul_f16x2(codes_to_f16x2<0>(u[i]), f);
                        o[4 * i + 1] = mul_f16x2(codes_to_f16x2<1>(u[i]), f);
                        o[4 * i + 2] = mul_f16x2(codes_to_f16x2<2>(u[i]), f);
                        o[4 * i + 3] = mul_f16x2(codes_to_f16x2<3>(u[i]), f);
                    }
                    tmem_st16(lane_base + C::kColK + hd * 64 + j * 16, o);
                }
                warp_arrive_tmem(&sm.kafull[hd]);
            }
            if (!ok) break;
            warp_arrive(&sm.empty[s]);
        }
    } else if (warp < kSoftWarp) {
        // ---------------------------------------------------------------- V: lane = element (and + 128)
        const int quad = warp & 3, e = quad * 32 + lane;
        Ring<kStages> ring;
        Ring<kInfos> iring;
#pragma unroll 1
        for (int t = 0; t < ntiles; ++t, ring.next(), iring.next()) {
            const int s = ring.i, is = iring.i;
            // the factors' warp has waited for the codes
            if (!ctx.wait_warp(&sm.infofull[is], iring.parity)) break;
            const uint8_t* stage = smem + C::kOffV + s * kStageBytes + e * kTokens;
            const uint32_t* f = infos[is].f[quad];
            bool ok = true;
#pragma unroll 1
            for (int hv = 0; hv < 2; ++hv) {
                ok = ctx.wait_warp(&sm.vafree[hv], (t & 1) ^ 1);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 4 * hv; c < 4 * hv + 4; ++c) {  // a chunk: 16 keys, a column each
                    const uint4 w = *reinterpret_cast<const uint4*>(stage + c * kChunkBytes);
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
                    uint32_t o[16];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 x = *reinterpret_cast<const uint4*>(f + c * kTokens + 4 * i);
                        o[4 * i] = mul_f16x2(codes_to_f16x2<0>(u[i]), x.x);
                        o[4 * i + 1] = mul_f16x2(codes_to_f16x2<1>(u[i]), x.y);
                        o[4 * i + 2] = mul_f16x2(codes_to_f16x2<2>(u[i]), x.z);
                        o[4 * i + 3] = mul_f16x2(codes_to_f16x2<3>(u[i]), x.w);
                    }
                    tmem_st16(lane_base + C::kColV + c * 16, o);
                }
                warp_arrive_tmem(&sm.vafull[hv]);
            }
            if (!ok) break;
            warp_arrive(&sm.empty[s]);
            warp_arrive(&sm.infofree[is]);
        }
    } else {
        // ---------------------------------------------------------------- softmax
        const int sw = warp - kSoftWarp;
        const int g = sw >> 2;            // rows [16 g, 16 g + 16)
        const int wq = warp & 3;          // tensor-memory lane quadrant
        const int st = (wq << 5) | lane;  // key of the tile
        const int row0 = kGroupRows * g;
        const int qoff = n - p.q_len;  // row r of the slot sees keys j <= qoff + r / G
        griddep_wait();
        {
            constexpr int kRowsPerWarp = RP / C::kSoftWarps;  // 4
            uint4 qraw[kRowsPerWarp];
#pragma unroll
            for (int k = 0; k < kRowsPerWarp; ++k) {
                const int r = sw + C::kSoftWarps * k;
                qraw[k] = make_uint4(0, 0, 0, 0);
                if (r < R) {
                    const int i = (row_lo + r) / G, gg = (row_lo + r) % G;
                    const int64_t qrow = ((int64_t)b * p.q_len + i) * p.num_q_heads + h * G + gg;
                    qraw[k] = *reinterpret_cast<const uint4*>(p.q + qrow * kHeadDim + lane * 8);
                }
            }
#pragma unroll
            for (int k = 0; k < kRowsPerWarp; ++k) {
                // a row with an infinity is a row of NaN (its scores could all be -inf, as if it saw
                // no key): exponent field all ones in any of its halves
                auto inf_in = [&](uint32_t x) {
                    return (x & 0x7C00u) == 0x7C00u || (x & 0x7C000000u) == 0x7C000000u;
                };
                const bool bad = inf_in(qraw[k].x) || inf_in(qraw[k].y) || inf_in(qraw[k].z) ||
                                 inf_in(qraw[k].w);
                if (__any_sync(0xffffffffu, bad)) qraw[k].x = 0x7E007E00u;
                *reinterpret_cast<uint4*>(smem + q_off(sw + C::kSoftWarps * k, lane, RP)) = qraw[k];
            }
            for (uint32_t i = (sw * 32 + lane) * 16; i < C::kPBytes; i += C::kSoftWarps * 32 * 16)
                *reinterpret_cast<uint4*>(smem + C::kOffP + i) = make_uint4(0, 0, 0, 0);
            fence_async_smem();
            warp_arrive(&sm.qready);
        }
        uint64_t lsum[kGroupRows / 2];
        uint64_t nm[kGroupRows / 2];  // the shift minus each row's reference (+inf: none yet), in pairs
#pragma unroll
        for (int q = 0; q < kGroupRows / 2; ++q) {
            lsum[q] = 0;
            nm[q] = pk2(INFINITY, INFINITY);
        }
        if (lane < kGroupRows) sm.nmcur[g][wq][lane] = INFINITY;
        __syncwarp();
        bool alive = true;
#pragma unroll 1
        for (int t = 0; t < ntiles; ++t) {
            const int tile0 = start + t * kTile, j = tile0 + st, is = t % kInfos;
            alive = alive & ctx.wait_warp(&sm.sfull[t & 1], (t >> 1) & 1);
            const float2 cev = infos[is].c[st];
            const float c = cev.x, ev = cev.y;
            tc_fence_after();
            auto scores = [&](uint64_t (&y)[kGroupRows / 2]) {
                uint32_t a[16];
                tmem_ld16(lane_base + C::kColS + (t & 1) * RP + row0, a);
                tmem_ld_wait(a);
#pragma unroll
                for (int q = 0; q < kGroupRows / 2; ++q) y[q] = pk2(f32(a[2 * q]), f32(a[2 * q + 1]));
            };
            uint64_t e[kGroupRows / 2];
            scores(e);
            // bit i: key j visible to row row0 + i (rows past the slot's count: zeros of Q, not stored)
            uint32_t validm = 0xFFFFu;
            if (!((tile0 + kTile <= end) && (tile0 + kTile - 1 <= qoff))) {
                // row r of the slot sees key j iff r >= (j - qoff) G: the group's rows from `first` on
                const int first = (j - qoff) * G - row_lo - row0;
                if (j >= end)
                    validm = 0;
                else if (first > 0)
                    validm = first >= kGroupRows ? 0u : (0xFFFFu << first) & 0xFFFFu;
            }
            // exponents of the shifted weights: s c + ev + (shift - reference)
            const uint64_t c2 = pk2(c, c), ev2 = pk2(ev, ev);
#pragma unroll
            for (int q = 0; q < kGroupRows / 2; ++q) e[q] = fma2(e[q], c2, add2(nm[q], ev2));
            if (validm != 0xFFFFu) {
#pragma unroll
                for (int q = 0; q < kGroupRows / 2; ++q)
                    e[q] = pk2(((validm >> (2 * q)) & 1u) ? lo2(e[q]) : -INFINITY,
                               ((validm >> (2 * q + 1)) & 1u) ? hi2(e[q]) : -INFINITY);
            }
            float m = lo2(e[0]);
#pragma unroll
            for (int q = 0; q < kGroupRows / 2; ++q) m = fmaxf(m, fmaxf(lo2(e[q]), hi2(e[q])));
            const bool need = m > kLazyThreshold;
            bool need_any = true;  // tile 0 sets the reference
            if (t > 0) need_any = group_vote(g, need || !alive);
            if (need_any) {
                if (group_vote(g, !alive)) break;  // all four warps together
                // exact tile maximum per row -> new reference; row sums and O rescaled. Lanes 2i and
                // 2i + 1 derive row i's, the shuffles hand it to every lane. (The next tile's vote stands
                // between these reads of the maxima and their next writing.)
                float v[kGroupRows];
                uint64_t y[kGroupRows / 2];
                scores(y);
#pragma unroll
                for (int q = 0; q < kGroupRows / 2; ++q) {
                    y[q] = fma2(y[q], c2, ev2);
                    v[2 * q] = ((validm >> (2 * q)) & 1u) ? lo2(y[q]) : -INFINITY;
                    v[2 * q + 1] = ((validm >> (2 * q + 1)) & 1u) ? hi2(y[q]) : -INFINITY;
                }
                const float vm = rows_reduce(v, lane, [](float a, float b2) { return fmaxf(a, b2); });
                if ((lane & 1) == 0) sm.rmax[g][wq][lane >> 1] = vm;
                group_bar(g);
                const int ri = (lane >> 1) & (kGroupRows - 1);
                const float mo = kShift - sm.nmcur[g][wq][ri];
                const float tm = fmaxf(fmaxf(sm.rmax[g][0][ri], sm.rmax[g][1][ri]),
                                       fmaxf(sm.rmax[g][2][ri], sm.rmax[g][3][ri]));
                const float mn = fmaxf(mo, tm);
                const float alpha_r = (mn == -INFINITY) ? 1.f : ex2(mo - mn);
                const float nm_r = (mn == -INFINITY) ? INFINITY : kShift - mn;
                __syncwarp();
                if ((lane & 1) == 0) sm.nmcur[g][wq][ri] = nm_r;
                float alpha[kGroupRows];
#pragma unroll
                for (int q = 0; q < kGroupRows / 2; ++q) {
                    alpha[2 * q] = __shfl_sync(0xffffffffu, alpha_r, 4 * q);
                    alpha[2 * q + 1] = __shfl_sync(0xffffffffu, alpha_r, 4 * q + 2);
                    nm[q] = pk2(__shfl_sync(0xffffffffu, nm_r, 4 * q),
                                __shfl_sync(0xffffffffu, nm_r, 4 * q + 2));
                    lsum[q] = mul2(lsum[q], pk2(alpha[2 * q], alpha[2 * q + 1]));
                    e[q] = add2(y[q], nm[q]);
                    if (!((validm >> (2 * q)) & 1u)) e[q] = pk2(-INFINITY, hi2(e[q]));
                    if (!((validm >> (2 * q + 1)) & 1u)) e[q] = pk2(lo2(e[q]), -INFINITY);
                }
                if (t > 0) {
                    alive = ctx.wait_warp(&sm.pfree, (t - 1) & 1);  // O holds the tiles before
                    tc_fence_after();
#pragma unroll 1
                    for (int mh = 0; mh < 2; ++mh) {
                        const uint32_t addr = lane_base + C::kColO + mh * RP + row0;
                        uint32_t o[16];
                        tmem_ld16(addr, o);
                        tmem_ld_wait(o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(f32(o[i]) * alpha[i]);
                        tmem_st16(addr, o);
                    }
                    tmem_st_wait();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&sm.sfree[t & 1]));
                mbar_arrive(smem_u32(&sm.infofree[is]));
            }
            // weights, their sum without V's exponent, and their FP16 rounding
            const float iev = ev == ev ? ex2(-ev) : 1.f;
            const uint64_t iev2 = pk2(iev, iev);
            uint32_t ph[kGroupRows / 2];
#pragma unroll
            for (int q = 0; q < kGroupRows / 2; ++q) {
                const float p0 = ex2(lo2(e[q])), p1 = ex2(hi2(e[q]));
                lsum[q] = fma2(pk2(p0, p1), iev2, lsum[q]);
                const __half2 r = __floats2half2_rn(p0, p1);
                ph[q] = *reinterpret_cast<const uint32_t*>(&r);
            }
            // (passes before the first product: the phase before the barrier's first)
            alive = alive & ctx.wait_warp(&sm.pfree, (t - 1) & 1);
#pragma unroll
            for (int k = 0; k < 2; ++k) {  // half the lanes begin with the other place: other banks
                const int mh = k ^ ((lane >> 2) & 1);
                uint8_t* at = smem + C::kOffP + p_off(mh * (RP / 8) + 2 * g, 2 * st + mh);
                *reinterpret_cast<uint4*>(at) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
                *reinterpret_cast<uint4*>(at + 4096) = make_uint4(ph[4], ph[5], ph[6], ph[7]);
            }
            fence_async_smem();
            tc_fence_before();
            warp_arrive(&sm.pfull);
        }
        // split state: the reference minus the shift, shifted sums and numerators
        {
            float v[kGroupRows];
#pragma unroll
            for (int q = 0; q < kGroupRows / 2; ++q) {
                v[2 * q] = lo2(lsum[q]);
                v[2 * q + 1] = hi2(lsum[q]);
            }
            const float sum = rows_reduce(v, lane, [](float a, float b2) { return a + b2; });
            if ((lane & 1) == 0) sm.rsum[g][wq][lane >> 1] = sum;
            if (lane == 0 && wq == 0) {
#pragma unroll
                for (int q = 0; q < kGroupRows / 2; ++q) {
                    sm.mref[g][2 * q] = -lo2(nm[q]);
                    sm.mref[g][2 * q + 1] = -hi2(nm[q]);
                }
            }
        }
        group_bar(g);
        if (alive && !ctx.aborted() && wq == 0 && lane < kGroupRows && row0 + lane < R) {
            const float L = sm.rsum[g][0][lane] + sm.rsum[g][1][lane] + sm.rsum[g][2][lane] +
                            sm.rsum[g][3][lane];
            // (a row of NaN may have no maximum; it is not an empty one)
            const float m = L != L ? INFINITY : sm.mref[g][lane];
            p.ws_state[(int64_t)slot * p.rows + row_lo + row0 + lane] = make_float2(m, L);
        }
        const bool ok = ctx.wait_warp(&sm.odone, 0);
        tc_fence_after();
        if (__all_sync(0xffffffffu, ok && !ctx.aborted())) {
            constexpr float kBack = 1.f / (1 << kFactorTop);
#pragma unroll 1
            for (int mh = 0; mh < 2; ++mh) {
                uint32_t o[16];
                tmem_ld16(lane_base + C::kColO + mh * RP + row0, o);
                tmem_ld_wait(o);
                const int d = mh * 128 + st;
#pragma unroll
                for (int i = 0; i < kGroupRows; ++i) {
                    const int r = row0 + i;
                    if (r < R)
                        p.ws_acc[((int64_t)slot * p.rows + row_lo + r) * kHeadDim + d] = f32(o[i]) * kBack;
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        // (of a CTA that gave up products may still be on their way: no wait above saw them through)
        mbar_wait(smem_u32(&sm.odone), 0, &sm.never, kWaitLimitNs);
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

template <int RP>
cudaError_t launch_rp(const PartialParams& p, cudaStream_t stream) {
    constexpr uint32_t smem = smem_bytes<RP>();
    cudaError_t e = cudaFuncSetAttribute(mx4_partial_kernel<RP>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = partial_grid(p);
    cfg.blockDim = dim3(Cfg<RP>::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    if (p.pdl) {  // a programmatic dependent of the preceding kernel on the stream
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, mx4_partial_kernel<RP>, p);
}

// Plans for contexts up to here have one round of slots: with more units than that has slots cutting them up costs
// what it gains (16 tiles, common.cuh, slots_of_lengths); with fewer the longest split is 32 tiles, and slots
// left idle cost 2.4 us (96 units up to 4096 tokens 29.6 and 32.0).
constexpr int kRoundsFrom = 2048, kRoundsFromOne = 4096;

int rows_pad(int rows) { return (rows + kGroupRows - 1) / kGroupRows * kGroupRows; }

cudaError_t launch_partial(const PartialParams& p, cudaStream_t stream) {
    if (!row_blocks_valid(p, kMaxRP)) return cudaErrorInvalidValue;
    switch (rows_pad(p.block_rows)) {
        case 16: return launch_rp<16>(p, stream);
        case 32: return launch_rp<32>(p, stream);
        default: return launch_rp<48>(p, stream);
    }
}

static bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The plan as the split and combine rules of the E4M3 kernel see it (the same tile and row blocks).
static dflash_verify_attn_plan_t as_split_plan(const dflash_verify_attn_plan_t& plan) {
    dflash_verify_attn_plan_t p = plan;
    p.kernel = DFLASH_KERNEL_TCGEN05;
    return p;
}

}  // namespace mx4
}  // namespace dflash

using namespace dflash;

extern "C" {

int dflash_mx4_attn_plan(const dflash_verify_attn_problem* problem,
                         dflash_verify_attn_plan_t* plan) {
    if (!problem || !plan) return DFLASH_ERR_INVALID_ARGUMENT;
    dflash_verify_attn_problem pr = *problem;
    if (pr.kernel < DFLASH_KERNEL_AUTO || pr.kernel > DFLASH_KERNEL_TCGEN05)
        return DFLASH_ERR_INVALID_ARGUMENT;
    if (pr.kernel != DFLASH_KERNEL_AUTO || (pr.flags & ~DFLASH_PROBLEM_PDL))
        return DFLASH_ERR_UNSUPPORTED;
    pr.kernel = DFLASH_KERNEL_TCGEN05;
    const int rc = dflash_verify_attn_plan(&pr, plan);
    if (rc != DFLASH_OK) return rc;
    plan->kernel = DFLASH_KERNEL_MX4;
    // A batch has an SM's worth of slots, shared out by length, or one a unit. With more than half as many units
    // as a round has slots that leaves little to share, or nothing: it gets rounds with about half a
    // round to spare or more, of which a call takes what its lengths want (common.cuh, slots_of_lengths). Fewer units
    // gain nothing: 64 of 24/4 heads, one token each, up to 4096 tokens 24 us with one round and 32 with two,
    // up to 16384 tokens 67 and 66.
    const int64_t units = (int64_t)pr.batch * pr.num_kv_heads, round = plan->sm_count / plan->row_blocks;
    if (units > 65535) return DFLASH_ERR_UNSUPPORTED;  // the combine's grid: found out here, not behind the products
    const int64_t cap = units * ((pr.max_context + plan->min_split_keys - 1) / plan->min_split_keys);
    const int64_t slots = std::min(((units + (round - 1) / 2) / round + 1) * round, cap);
    if (pr.batch > 1 && pr.num_splits == 0 && slots > plan->num_slots &&
        pr.max_context > (units > round ? mx4::kRoundsFrom : mx4::kRoundsFromOne)) {
        if (slots * plan->row_blocks > 0x7FFFFFFF) return DFLASH_ERR_UNSUPPORTED;
        plan->num_slots = (int32_t)slots;
        const size_t rows = (size_t)plan->num_slots * plan->rows;
        plan->ws_acc_offset = plan->ws_state_offset + (rows * sizeof(float2) + 255) / 256 * 256;
        plan->workspace_bytes = plan->ws_acc_offset + rows * kHeadDim * sizeof(float);
    }
    const int block_rows = (plan->rows + plan->row_blocks - 1) / plan->row_blocks;
    switch (mx4::rows_pad(block_rows)) {
        case 16:
            plan->threads = mx4::Cfg<16>::kThreads;
            plan->smem_bytes = (int32_t)mx4::smem_bytes<16>();
            break;
        case 32:
            plan->threads = mx4::Cfg<32>::kThreads;
            plan->smem_bytes = (int32_t)mx4::smem_bytes<32>();
            break;
        default:
            plan->threads = mx4::Cfg<48>::kThreads;
            plan->smem_bytes = (int32_t)mx4::smem_bytes<48>();
    }
    plan->problem = *problem;
    return DFLASH_OK;
}

int dflash_mx4_attn_forward(const dflash_verify_attn_plan_t* plan, const void* q,
                            const void* k_pool, const void* v_pool, const int32_t* block_table,
                            const int32_t* context_lens, void* workspace, size_t workspace_bytes,
                            void* out, float* lse, void* cuda_stream) {
    if (!plan || plan->kernel != DFLASH_KERNEL_MX4) return DFLASH_ERR_INVALID_ARGUMENT;
    const dflash_verify_attn_plan_t split = mx4::as_split_plan(*plan);
    const int rc = check_attn_plan(&split);
    if (rc != DFLASH_OK) return rc;
    if (!q || !k_pool || !v_pool || !block_table || !context_lens || !workspace || !out || !lse)
        return DFLASH_ERR_INVALID_ARGUMENT;
    if (!mx4::aligned(q, 16) || !mx4::aligned(k_pool, 16) || !mx4::aligned(v_pool, 16) ||
        !mx4::aligned(workspace, 256) || !mx4::aligned(block_table, 4) || !mx4::aligned(context_lens, 4) ||
        !mx4::aligned(out, 8) || !mx4::aligned(lse, 4))
        return DFLASH_ERR_INVALID_ARGUMENT;
    const void* const outs[] = {workspace, out, lse};
    const void* const others[] = {q, k_pool, v_pool, block_table, context_lens};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 5; ++j)
            if (outs[i] == others[j]) return DFLASH_ERR_INVALID_ARGUMENT;
        for (int j = 0; j < i; ++j)
            if (outs[i] == outs[j]) return DFLASH_ERR_INVALID_ARGUMENT;
    }
    if (workspace_bytes < plan->workspace_bytes) return DFLASH_ERR_WORKSPACE_TOO_SMALL;
    PartialParams p = attn_params(&split, q, k_pool, v_pool, block_table, context_lens, nullptr, nullptr,
                                  workspace);
    CombineParams c = combine_params(&split, workspace, context_lens, out, lse);
    p.round_slots = c.round_slots = round_slots(*plan);
    c.pdl = 1;  // it waits for the partial kernel where it reads the split state
    cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    if (mx4::launch_partial(p, stream) != cudaSuccess || launch_combine(c, stream) != cudaSuccess) {
        cudaGetLastError();
        return DFLASH_ERR_CUDA;
    }
    return DFLASH_OK;
}

}  // extern "C"
