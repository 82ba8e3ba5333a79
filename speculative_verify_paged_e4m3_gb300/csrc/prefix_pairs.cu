// prefix_pairs.cu -- attention over a shared prefix for many query rows: FP16 tensor-core products
// on pairs of SMs (tcgen05, cta_group::2).
//
// With batch * q_len * Hq / Hkv rows per KV head the prefix is no longer bound by HBM but by the
// products, 4 D flops per row and key. The split kernel's three E4M3 terms cost 1.5 times the
// tensor work of FP16 operands, and its accumulators (one per term) leave room for 48 rows. Here Q
// stays FP16, K and V are decoded to FP16 (exact) on their way into shared memory, P is rounded
// to FP16 (2^-11 of each probability), all sums are FP32.
//
//  * A pair of SMs carries 256 rows: 128 on each (tensor-memory lane = row), accumulator O [128,
//    256] FP32 in each SM's tensor memory. One SM's 128 rows alone would need each decoded K and V
//    byte written and read by that SM only: by count 3500 clocks of shared-memory traffic per 2048 of
//    tensor work. With cta_group::2 the pair's second operand is split between the two SMs, so that
//    each decodes and stores half of it (half of the tile's keys of K, half of the head dim of V).
//  * Tiles of 96 keys: two score buffers of 96 columns and P (48 columns, two FP16 each) fit beside O
//    in the 512 columns of tensor memory, and P needs no buffer of its own in shared memory. P does not
//    share its columns with scores, so that no product overwrites what another one may still read; it
//    is handed over in two halves of 48 keys, so that the softmax writes the next tile's first half
//    while the products still read this one's second (in one piece a tile took 2020 clocks even with
//    the decoders' and the softmax's work left out).
//  * Warps: 0-7 softmax (thread = row, warps 0-3 the tile's first 48 keys, 4-7 the others), 8-9 decode
//    K, 10-11 decode V, 12 issues the score products of the pair and 13 its PV (one thread each, in
//    the leader SM alone), 14 and 15 copy the codes of K and of V (TMA, three and two tiles
//    ahead).
//  * Probabilities are p = 2^(score - m) for a reference m that is set 2^4 below the first tile's
//    maximum, and moves only when a row's probabilities of 48 keys sum to more than 2^15 (so that all
//    are inside FP16): scores, exponentials and sums are one pass with no maximum in front of it. When
//    one row's moves, those of the SM's other rows go up to 2^4 below what they have in that tile too
//    (one after the other they made 16 x 8 tokens with scores of spread 4 on 5 % of 32768 keys 117 us, so
//    109). The rows' O columns are rescaled in place and the tile is done again, which stalls the pair
//    for more than a tile. Below 2^-14 FP16 has a fixed step of 2^-24, half of which each of N keys may
//    lose, all the same way, beside a sum of at least 2^4: N 2^-29, 2^-12 of 2^17 keys. (With m 2^4 above the
//    first maximum that case takes 100 us, but a strong key in front of 65536 others lost 2^-5: 0.060 for
//    0.042, 21 bits below it. At its maximum plain scores cost the same, and 17 bits lost too much.)
//  * Pairs take equal shares of all (KV head, row block) units' tiles (prefix_pairs.cuh); a share may
//    end in the middle of a unit, the combine puts the parts together.
//  * Bound by the tensor pipe and by what feeds it: a tile takes 1.07 us (0.99, 1912 clocks, before the two
//    SMs' hand-overs were ordered over the cluster), its products by themselves 1565 clocks. 40 x 8 tokens
//    of 24/4 heads over 131000 keys: 699 us, 1.47 PFLOP/s, 77 % of the bf16 library product's burst rate; 16 x 8
//    tokens over 32768 keys 95 us, 106 with peaked scores.
//  * Every wait is bounded (200 ms, then DFLASH_FLAG_KERNEL_TIMEOUT and a clean exit); both SMs of
//    a pair leave together.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "e4m3.cuh"
#include "prefix_pairs.cuh"
#include "tc_ptx.cuh"

namespace dflash {
namespace pairs {

using namespace ptx;

constexpr int kRows = kPairRows / 2;  // per SM
constexpr int kTile = kPairTile;
constexpr int kHalfKeys = kTile / 2;
constexpr int kStages = 2;      // decoded tiles of K, and of V
constexpr int kRawK = 3, kRawV = 2;  // tiles of codes on their way
constexpr int kSoftWarps = 8, kDecodeWarps = 2;  // decoders per operand
constexpr int kQkWarp = kSoftWarps + 2 * kDecodeWarps, kPvWarp = kQkWarp + 1;
constexpr int kCopyWarp = kPvWarp + 1;  // and the next one
constexpr int kThreads = 32 * (kCopyWarp + 2);  // 16 warps: 128 registers a thread
constexpr uint64_t kWaitLimitNs = 200ull * 1000 * 1000;
constexpr float kMaxExp = 4.f;      // a reference is set 2^4 below the maximum that moves it
constexpr float kMaxSum = 32768.f;  // a row's probabilities of a half tile sum to this at most

// Shared memory: Q | K stages | V stages | codes of K | codes of V | Small. All operands are 128-byte swizzled: Q and K
// [head-dim block of 64][row][64 FP16], V [head-dim block of 64][key][64 FP16].
constexpr uint32_t kQBytes = kRows * kHeadDim * 2;
constexpr uint32_t kKStage = kHalfKeys * kHeadDim * 2;       // this SM's 48 keys
constexpr uint32_t kVStage = kTile * (kHeadDim / 2) * 2;     // this SM's 128 elements of 96 keys
constexpr uint32_t kOffK = kQBytes;
constexpr uint32_t kOffV = kOffK + kStages * kKStage;
constexpr uint32_t kRawStage = kHalfKeys * kHeadDim;         // codes of either: 12 KB
constexpr uint32_t kOffRawK = kOffV + kStages * kVStage;     // [key][256]
constexpr uint32_t kOffRawV = kOffRawK + kRawK * kRawStage;  // [key][128]
constexpr uint32_t kOffSmall = kOffRawV + kRawV * kRawStage;
static_assert(kRawStage == kTile * kHeadDim / 2, "either operand");
// Tensor memory columns
constexpr uint32_t kColO = 0, kColS = kHeadDim, kColP = kColS + 2 * kTile;
static_assert(kColP + kTile / 2 <= 512, "tensor memory");
static_assert(kOffK % 1024 == 0 && kOffV % 1024 == 0 && kKStage % 1024 == 0 &&
                  kVStage % 1024 == 0,
              "swizzled operands are 1 KB aligned");

struct Small {
    // in the leader: operands and P ready, scores read
    uint64_t kfull[kStages], vfull[kStages], qfull, pfull[2], sfree[2];
    // in both, by the pair's commits: scores complete (and their K stage free), P's first half read,
    // V stage (and P's second half) free, everything complete
    uint64_t sfull[kStages], pdone, vempty[kStages], done;
    uint64_t rkfull[kRawK], rkempty[kRawK], rvfull[kRawV], rvempty[kRawV];  // this SM's copies
    uint32_t tmem_base;
    int abort;
    float part[2][kRows];  // row maxima, then row sums, of the two halves of a tile's keys
};
constexpr uint32_t kSmemBytes = kOffSmall + sizeof(Small);
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");

// ---- cluster and pair instructions -------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// Arrive on the barrier at the same place in the leader's shared memory. For tensor memory: what it holds is
// ordered by the tcgen05 fences around the arrival and the leader's wait, and the arrival has nothing to
// release.
__device__ __forceinline__ void arrive_leader(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .b32 remote;\n\t"
        "mapa.shared::cluster.u32 remote, %0, 0;\n\t"
        "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [remote];\n\t}" ::"r"(bar)
        : "memory");
}
// The same behind stores to this SM's shared memory (already fenced for the async proxy). The release is
// over the cluster, of shared memory alone, about 110 clocks a tile: 40 x 8 tokens over 131000 keys 735 us.
// With a release of all memory on the arrival 809; with one of the CTA's scope, which promises the other SM
// nothing, 692; passed on by an idle warp of the other SM 738.
__device__ __forceinline__ void release_to_leader(uint32_t bar) {
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
    arrive_leader(bar);
}
// Look-ups of barriers that either SM, or the leader's commits, arrive on.
__device__ __forceinline__ bool pair_test_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool pair_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// D += A B^T over 16 elements of K, FP16 operands: A from shared memory, or from tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive on the barrier of both SMs once every product issued so far has completed.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
    const uint16_t both = 3;
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(bar),
        "h"(both)
        : "memory");
}
// 2-D tiled copy global -> this SM's shared memory; coordinates innermost first.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* map, int x, int y,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(
                     taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                 "r"(r[7])
                 : "memory");
}
// OR of a predicate over the softmax threads (named barrier 1), and a plain barrier of theirs.
__device__ __forceinline__ bool soft_vote(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred pv, pr;\n\tsetp.ne.u32 pv, %1, 0;\n\t"
        "bar.red.or.pred pr, 1, %2, pv;\n\tselp.u32 %0, 1, 0, pr;\n\t}"
        : "=r"(r)
        : "r"(v ? 1u : 0u), "n"(32 * kSoftWarps)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void soft_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kSoftWarps) : "memory");
}

struct Ctx {
    Small* sm;
    int32_t* status;
    __device__ bool aborted() const { return *reinterpret_cast<volatile int*>(&sm->abort) != 0; }
    __device__ void give_up() const {
        *reinterpret_cast<volatile int*>(&sm->abort) = 1;
        atomicOr(status, DFLASH_FLAG_KERNEL_TIMEOUT);
    }
    __device__ bool wait(uint64_t* bar, uint32_t parity) const {
        const uint32_t a = smem_u32(bar);
        if (pair_try_wait(a, parity)) return true;
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t it = 1;; ++it) {
            if (pair_try_wait(a, parity)) return true;
            if ((it & 7) == 0) {
                if (aborted()) return false;
                if (globaltimer_ns() - t0 > kWaitLimitNs) {
                    give_up();
                    return false;
                }
            }
        }
    }
    // Two barriers at once: their look-ups overlap.
    __device__ bool wait2(uint64_t* bar_a, uint32_t parity_a, uint64_t* bar_b,
                          uint32_t parity_b) const {
        const uint32_t a = smem_u32(bar_a), b = smem_u32(bar_b);
        const bool ra = pair_test_wait(a, parity_a), rb = pair_test_wait(b, parity_b);
        if (ra & rb) return true;
        return wait(bar_a, parity_a) && wait(bar_b, parity_b);
    }
    // every lane waits and the warp agrees on the result
    __device__ bool wait_warp(uint64_t* bar, uint32_t parity) const {
        return __all_sync(0xffffffffu, wait(bar, parity));
    }
};

// Wait (bounded, whatever became of the other warps) for a copy in flight.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(smem_u32(bar), parity) && globaltimer_ns() - t0 < kWaitLimitNs) {
    }
}

// Keys [0, limit) of the prefix are visible to row rr of the batch.
__device__ __forceinline__ int row_limit(const PrefixPairsParams& p, int rr, int keys) {
    const int i = rr / p.group, b = i / p.q_len;
    const int ctx_len = min(p.context_lens[b], p.max_context);
    return min(keys, ctx_len - p.q_len + (i - b * p.q_len) + 1);
}

// The segments of a pair, in order: every role walks the same list.
struct Segments {
    int64_t at, end;  // tiles of the line still to do
    int64_t pitch;
    int tiles;  // per unit
    int unit, first, count;  // the current segment: its unit, first tile, tile count
    __device__ Segments(const PairShare& s, int pair, int units) {
        const int64_t total = units * s.pitch;
        pitch = s.pitch;
        tiles = s.tiles;
        at = pair * s.per_pair;
        end = at + s.per_pair < total ? at + s.per_pair : total;
    }
    __device__ bool next() {
        if (at >= end) return false;
        unit = (int)(at / pitch);
        first = (int)(at - unit * pitch);  // < tiles: a unit's empty end is shorter than a share
        const int64_t left = end - at;
        count = left < tiles - first ? (int)left : tiles - first;
        at = unit * pitch + first + count == unit * pitch + tiles ? (unit + 1) * pitch : at + count;
        return true;
    }
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    prefix_pairs_kernel(const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap, const PrefixPairsParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Small& sm = *reinterpret_cast<Small*>(smem + kOffSmall);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1;
    int flags = 0;
    const int keys = shared_keys(p.prefix_len, p.max_prefix, p.page_size, &flags);
    if (flags && blockIdx.x == 0 && tid == 0) atomicOr(p.status, flags);
    const PairShare share = pair_share(keys, p.units, p.pairs);
    // the next kernel on the stream may be launched beside this one's last CTAs
    griddep_launch_dependents();
    if (pair * share.per_pair >= p.units * share.pitch) return;  // both SMs agree
    if (smem_u32(smem) & 1023u) {  // the swizzled layouts need a 1 KB aligned base
        if (tid == 0) atomicOr(p.status, DFLASH_FLAG_KERNEL_TIMEOUT);
        return;
    }
    Segments seg(share, pair, p.units);
    const Ctx ctx{&sm, p.status};

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&sm.kfull[i]), 2 * kDecodeWarps);
            mbar_init(smem_u32(&sm.vfull[i]), 2 * kDecodeWarps);
            mbar_init(smem_u32(&sm.sfull[i]), 1);
            mbar_init(smem_u32(&sm.vempty[i]), 1);
        }
        mbar_init(smem_u32(&sm.qfull), 2 * kSoftWarps);
        mbar_init(smem_u32(&sm.pfull[0]), kSoftWarps);  // half of the warps, on both SMs
        mbar_init(smem_u32(&sm.pfull[1]), kSoftWarps);
        mbar_init(smem_u32(&sm.pdone), 1);
        mbar_init(smem_u32(&sm.sfree[0]), 2 * kSoftWarps);
        mbar_init(smem_u32(&sm.sfree[1]), 2 * kSoftWarps);
        mbar_init(smem_u32(&sm.done), 2);  // one commit of each issuing warp
        sm.abort = 0;
        fence_mbar_init();
    }
    // The two copying warps (K, V): lane c < 6 looks up the page of the tile's 16-key chunk c, a tile
    // ahead (the entry is not looked at before its tile's turn, so its load waits for nobody); lane 0
    // issues. They touch this SM alone, and fill their rings before the pair has met.
    const bool copies_k = warp == kCopyWarp;
    bool clamped = false;
    int copied = 0, copy_tile = 0, copy_page = 0;  // tiles issued; tile of the segment, its entry
    bool copy_live = false;
    auto logical = [&](int j) { return p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size; };
    auto lookup = [&](int tile) {
        const int j = tile * kTile + 16 * lane;
        return lane < kTile / 16 && j < keys ? p.prefix_table[logical(j)] : 0;
    };
    auto copy_step = [&]() {  // the next tile of the pair's line; false: none left, or gave up
        if (!copy_live) return false;
        const int page = copy_page;
        copy_page = lookup(seg.first + copy_tile + 1);
        const int tile0 = (seg.first + copy_tile) * kTile, j = tile0 + 16 * lane;
        const int chunks = min((keys - tile0) / 16, kTile / 16);  // of this tile
        int row = 0;                                              // the chunk's row of the pool
        if (lane < chunks)
            row = clamp_page(page, p.num_pages, &clamped) * p.page_size +
                  (j - logical(j) * p.page_size);
        const int ring = copies_k ? kRawK : kRawV, st = copied % ring;
        if (!ctx.wait_warp(&(copies_k ? sm.rkempty : sm.rvempty)[st], ((copied / ring) & 1) ^ 1))
            return false;
        const uint32_t bar = smem_u32(&(copies_k ? sm.rkfull : sm.rvfull)[st]);
        const uint32_t dst =
            smem_u32(smem + (copies_k ? kOffRawK : kOffRawV) + st * kRawStage);
        // K: this SM's three chunks, whole rows; V: all six, this SM's half of the head dim
        const int c0 = copies_k ? 3 * (int)rank : 0, most = copies_k ? 3 : kTile / 16;
        const int n = min(max(chunks - c0, 0), most);
        const uint32_t box = kRawStage / most;
        const int x = seg.unit / p.blocks * kHeadDim + (copies_k ? 0 : (int)rank * (kHeadDim / 2));
        if (lane == 0) mbar_arrive_expect_tx(bar, n * box);
        for (int c = 0; c < n; ++c) {
            const int y = __shfl_sync(0xffffffffu, row, c0 + c);
            if (lane == 0) tma_load_2d(dst + c * box, copies_k ? &kmap : &vmap, x, y, bar);
        }
        ++copied;
        if (++copy_tile == seg.count) {
            copy_live = seg.next();
            copy_tile = 0;
            if (copy_live) copy_page = lookup(seg.first);
        }
        return true;
    };
    if (warp >= kCopyWarp) {
        const int ring = copies_k ? kRawK : kRawV;
        if (lane == 0) {
            prefetch_tensormap(copies_k ? &kmap : &vmap);
            for (int i = 0; i < ring; ++i) {
                mbar_init(smem_u32(&(copies_k ? sm.rkfull : sm.rvfull)[i]), 1);
                mbar_init(smem_u32(&(copies_k ? sm.rkempty : sm.rvempty)[i]), kDecodeWarps);
            }
            fence_mbar_init();
        }
        __syncwarp();
        copy_live = seg.next();
        if (copy_live) copy_page = lookup(seg.first);
        for (int i = 0; i < ring; ++i) copy_step();  // (the ring is empty: none of them waits)
    }
    if (warp == kQkWarp) {
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_u32(&sm.tmem_base))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    tc_fence_after();
    // All 512 columns were allocated, so they start at column 0, lane 0: the addresses below are
    // constants. (Both SMs of the pair must agree, and always do: an allocation elsewhere would be
    // a smaller one.)
    constexpr uint32_t tmem = 0;

    if (warp >= kSoftWarps && warp < kQkWarp) {
        // ------------------------------------------------------------------ decoders
        // A lane takes 8 codes (8 bytes) at a time and stores them as one 16-byte unit: loads of a warp
        // are whole rows of codes and the 8 lanes of a store phase fill one 128-byte row, so neither
        // meets a bank twice. K warp w has keys 24 w + n of this SM's 48, V warp w keys 48 w + 2 n and
        // 48 w + 2 n + 1 of the tile's 96 (n < 24).
        const bool is_k = warp < kSoftWarps + kDecodeWarps;
        const int w = warp - kSoftWarps - (is_k ? 0 : kDecodeWarps);
        uint64_t* full = is_k ? sm.kfull : sm.vfull;
        uint64_t* empty = is_k ? sm.sfull : sm.vempty;  // the scores of a tile free its K
        uint64_t* raw_full = is_k ? sm.rkfull : sm.rvfull;
        uint64_t* raw_empty = is_k ? sm.rkempty : sm.rvempty;
        const int raw_stages = is_k ? kRawK : kRawV;
        const int own_keys = (is_k ? kHalfKeys : kTile) / kDecodeWarps;  // of a tile
        const uint8_t* src0 = smem + (is_k ? kOffRawK : kOffRawV) + w * (kRawStage / kDecodeWarps) + 8 * lane;
        const int b = is_k ? 0 : lane >> 4;  // which of a V lane's two keys
        const int group = is_k ? lane : lane & 15;
        uint8_t* dst0 = smem + (is_k ? kOffK : kOffV) +
                        (group >> 3) * ((is_k ? kHalfKeys : kTile) * 128) +
                        (w * own_keys + b) * 128;
        const uint32_t unit = (uint32_t)((group & 7) ^ b) << 4;  // swizzled by the key's low bits
        const uint32_t stage_bytes = is_k ? kKStage : kVStage;
        const int key_shift = is_k ? 0 : 1;
        constexpr int kRounds = kHalfKeys / kDecodeWarps;  // keys of K, pairs of keys of V
        static_assert(kRounds % 8 == 0 && kRounds * kDecodeWarps == kHalfKeys, "decoders");
        uint32_t place[8];  // of a round's keys (less the lane's own bit), from the round's first
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t r = k << key_shift;
            place[k] = r * 128 + (unit ^ ((r & 7) << 4));
        }
        int rs = 0, rphase = 0;
        bool live = true;
        for (int g = 0; live && seg.next();) {
            for (int i = 0; i < seg.count; ++i, ++g) {
                const int s = g % kStages;
                const int j0 = (seg.first + i) * kTile +
                               (is_k ? (int)rank * kHalfKeys : 0) + w * own_keys;
                live = ctx.wait_warp(&raw_full[rs], rphase) &&
                       ctx.wait_warp(&empty[s], ((g / kStages) & 1) ^ 1);
                if (!live) break;
                const uint8_t* src = src0 + rs * kRawStage;
                uint8_t* dst = dst0 + s * stage_bytes;
                // Keys past the prefix were not copied and become zeros. Eight keys (pairs of V) a round,
                // and the same code for both operands: the roles share the instruction cache, and
                // straight-line code for each of them was slower.
                const int live_n = (keys - j0) >> key_shift;
                auto decode = [&](auto whole_) {
                    constexpr bool kWhole = decltype(whole_)::value;
#pragma unroll 1
                    for (int n0 = 0; n0 < kRounds; n0 += 8) {
                        uint2 v[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            v[k] = *reinterpret_cast<const uint2*>(src + (n0 + k) * 256);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            uint4 f;
                            e4m3x4_to_f16x4(v[k].x, f.x, f.y);
                            e4m3x4_to_f16x4(v[k].y, f.z, f.w);
                            if (!kWhole && n0 >= live_n) f = make_uint4(0, 0, 0, 0);
                            *reinterpret_cast<uint4*>(dst + (n0 << key_shift) * 128 + place[k]) = f;
                        }
                    }
                };
                if (live_n >= kRounds)
                    decode(std::true_type{});
                else
                    decode(std::false_type{});
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    release_to_leader(smem_u32(&full[s]));
                    mbar_arrive(smem_u32(&raw_empty[rs]));
                }
                if (++rs == raw_stages) {
                    rs = 0;
                    rphase ^= 1;
                }
            }
        }
    } else if (warp >= kCopyWarp) {
        // ------------------------------------------------------------------ copies
        while (copy_step()) {
        }
        if (clamped) atomicOr(p.status, DFLASH_FLAG_PAGE_CLAMPED);
        // no copy may still be writing this SM's shared memory when it leaves
        const int ring = copies_k ? kRawK : kRawV;
        for (int t = max(copied - ring, 0); t < copied; ++t)
            drain(&(copies_k ? sm.rkfull : sm.rvfull)[t % ring], (t / ring) & 1);
    } else if (warp == kQkWarp || warp == kPvWarp) {
        // ------------------------------------------------------------------ products
        // Issuing a product takes its thread about 50 clocks, a commit as long and a wait that is
        // already over some 80. With the decoders' and the softmax's work left out a tile took 2040
        // clocks with one issuing thread, 1796 with one for the scores and one for PV (and P in halves,
        // eight softmax warps); its products alone run in 1565. The tensor core takes from both. Stages and score buffers go by the tile's parity, a compile-time
        // constant below: every descriptor is then a constant from the shared-memory base.
        static_assert(kStages == 2, "a tile's stage is its parity");
        using Even = std::integral_constant<int, 0>;
        using Odd = std::integral_constant<int, 1>;
        if (rank == 0 && lane == 0 && warp == kQkWarp) {
            constexpr uint32_t idesc = idesc_f32acc(256, kTile, 0, 0, 0, 0);
            const uint32_t qb = smem_u32(smem), kb = smem_u32(smem + kOffK);
            int sidx = 0;
            bool ok = true;
            auto tile = [&](auto parity, int t) {
                constexpr int kS = decltype(parity)::value;
                // the softmax has read the scores of tile t - 2 out of this buffer
                ok = ctx.wait2(&sm.kfull[kS], (t >> 1) & 1, &sm.sfree[kS], ((t >> 1) & 1) ^ 1);
                if (!ok) return;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < kHeadDim / 16; ++k)
                    mma_ss(kColS + kS * kTile,
                           smem_desc(qb + (k >> 2) * (kRows * 128) + (k & 3) * 32, 16, 1024,
                                     kSwizzle128B),
                           smem_desc(kb + kS * kKStage + (k >> 2) * (kHalfKeys * 128) + (k & 3) * 32,
                                     16, 1024, kSwizzle128B),
                           idesc, k > 0);
                commit_pair(smem_u32(&sm.sfull[kS]));
            };
            for (int t = 0; ok && seg.next(); ++sidx) {
                ok = ctx.wait(&sm.qfull, sidx & 1);
                for (int i = 0; ok && i < seg.count; ++i, ++t) {
                    if (t & 1)
                        tile(Odd{}, t);
                    else
                        tile(Even{}, t);
                }
            }
            commit_pair(smem_u32(&sm.done));  // every product issued above
        } else if (rank == 0 && lane == 0) {
            constexpr uint32_t idesc = idesc_f32acc(256, kHeadDim, 0, 0, 0, 1);
            const uint32_t vb = smem_u32(smem + kOffV);
            bool ok = true;
            auto tile = [&](auto parity, int t, bool first) {
                constexpr int kS = decltype(parity)::value;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {  // the two halves of P
                    ok = hf ? ctx.wait(&sm.pfull[1], t & 1)
                            : ctx.wait2(&sm.vfull[kS], (t >> 1) & 1, &sm.pfull[0], t & 1);
                    if (!ok) return;
                    tc_fence_after();
#pragma unroll
                    for (int k = 3 * hf; k < 3 * hf + 3; ++k)
                        mma_ts(kColO, kColP + 8 * k,
                               smem_desc(vb + kS * kVStage + k * 2048, kTile * 128, 1024,
                                         kSwizzle128B),
                               idesc, k > 0 || !first);
                    commit_pair(smem_u32(hf ? &sm.vempty[kS] : &sm.pdone));
                }
            };
            for (int t = 0; ok && seg.next();) {
                for (int i = 0; ok && i < seg.count; ++i, ++t) {
                    if (t & 1)
                        tile(Odd{}, t, i == 0);
                    else
                        tile(Even{}, t, i == 0);
                }
            }
            commit_pair(smem_u32(&sm.done));
        }
    } else {
        // ------------------------------------------------------------------ softmax
        // Warps 0-3 have the first 48 keys of every tile, warps 4-7 the others; both halves of a row
        // keep the same reference.
        const int hf = warp >> 2, row = tid & (kRows - 1);  // row of this SM's = tensor-memory lane
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        // D^-1/2 = 1/16, log2 units. Row maxima below are taken before this factor, so it has to be
        // positive: a negative scale's sign goes into Q, a scale of zero becomes a tiny one (and one that
        // is not a number stays so).
        const float c_signed = __ldg(p.k_scale) * 0.0625f * kLog2e;
        const float c = fabsf(c_signed) < 1e-30f ? 1e-30f : fabsf(c_signed);
        const uint32_t q_sign = c_signed < 0.f ? 0x80008000u : 0u;
        const float vs = __ldg(p.v_scale);
        const uint64_t c2 = pk2(c, c);
        int g = 0;  // tile of the pair's line
        bool alive = true;
        while (seg.next()) {
            const int head = seg.unit / p.blocks, blk = seg.unit - head * p.blocks;
            const int row0 = blk * kPairRows + (int)rank * kRows;  // this SM's first row
            const int slot = pair + seg.unit;
            // Q rows -> swizzled shared memory, 16 rows a warp, all loads in flight. The loads are
            // not conditional (rows past the last read it again): a branch around each would make
            // them wait for one another.
            {
                constexpr int kOwn = kRows / kSoftWarps;
                // row of Q that this lane's row of the warp is; a row that sees no key (a padded
                // slot of the batch may hold anything) becomes zeros, like those past the last
                int at;
                bool live;
                {
                    const int rr = row0 + warp * kOwn + (lane & (kOwn - 1));
                    const int rc = min(rr, p.rows - 1), i = rc / p.group;
                    at = i * p.num_q_heads + head * p.group + (rc - i * p.group);
                    live = rr < p.rows && row_limit(p, rc, keys) > 0;
                }
                const uint32_t live_rows = __ballot_sync(0xffffffffu, live);
                uint4 w[kOwn];
#pragma unroll
                for (int k = 0; k < kOwn; ++k) {
                    const int qrow = __shfl_sync(0xffffffffu, at, k);
                    w[k] = reinterpret_cast<const uint4*>(p.q + (int64_t)qrow * kHeadDim)[lane];
                }
#pragma unroll
                for (int k = 0; k < kOwn; ++k) {
                    const int r = warp * kOwn + k;
                    const uint32_t keep = (live_rows >> k) & 1 ? 0xffffffffu : 0u;
                    *reinterpret_cast<uint4*>(smem + (lane >> 3) * (kRows * 128) + r * 128 +
                                              (((lane & 7) ^ (r & 7)) << 4)) =
                        make_uint4((w[k].x ^ q_sign) & keep, (w[k].y ^ q_sign) & keep,
                                   (w[k].z ^ q_sign) & keep, (w[k].w ^ q_sign) & keep);
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) release_to_leader(smem_u32(&sm.qfull));
            // keys [0, limit) are visible to this thread's row
            const int limit = row0 + row < p.rows ? row_limit(p, row0 + row, keys) : keys;
            float nm = INFINITY;  // minus the reference maximum (log2 units); +inf: no key yet
            float lsum = 0.f;
#pragma unroll 1
            for (int i = 0; i < seg.count; ++i) {
                const int t = g + i;
                const int j0 = (seg.first + i) * kTile + hf * kHalfKeys;
                const uint32_t s_col = lanes + kColS + (t & 1) * kTile + hf * kHalfKeys;
                if (alive) alive = ctx.wait_warp(&sm.sfull[t & 1], (t >> 1) & 1);
                tc_fence_after();
                uint32_t code[kHalfKeys / 2];
                // p = 2^(s c + nm) as FP16 pairs and their FP32 sum, of the unrounded values, in one
                // pass over the scores
                auto probabilities = [&](auto whole_) {
                    // whole: the row sees all of these keys, or none (then all are 2^-inf)
                    constexpr bool kWhole = decltype(whole_)::value;
                    const float nmr = kWhole && j0 >= limit ? -INFINITY : nm;
                    const uint64_t nm2 = pk2(nmr, nmr);
                    uint64_t sum[2] = {0, 0};
                    uint32_t a[3][16];
#pragma unroll
                    for (int k = 0; k < 3; ++k) tmem_ld16(s_col + 16 * k, a[k]);
#pragma unroll
                    for (int k = 0; k < 3; ++k) tmem_ld_wait(a[k]);
#pragma unroll
                    for (int k = 0; k < 3; ++k)
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const uint64_t e = fma2(pk2(__uint_as_float(a[k][2 * q]),
                                                        __uint_as_float(a[k][2 * q + 1])),
                                                    c2, nm2);
                            const int j = j0 + 16 * k + 2 * q;
                            const float p0 = kWhole || j < limit ? ex2(lo2(e)) : 0.f;
                            const float p1 = kWhole || j + 1 < limit ? ex2(hi2(e)) : 0.f;
                            sum[q & 1] = add2(sum[q & 1], pk2(p0, p1));
                            const __half2 x = __floats2half2_rn(p0, p1);
                            code[8 * k + q] = *reinterpret_cast<const uint32_t*>(&x);
                        }
                    sum[0] = add2(sum[0], sum[1]);
                    return lo2(sum[0]) + hi2(sum[0]);
                };
                float psum = INFINITY;
                if (i > 0 && __all_sync(0xffffffffu, j0 + kHalfKeys <= limit || j0 >= limit))
                    psum = probabilities(std::true_type{});
                // A sum that is too large (or infinite, or not a number) moves the reference: no
                // probability is above its half tile's sum, so smaller sums are inside FP16. The first
                // tile of a segment and those with keys that some row does not see come here too. All
                // 256 threads agree (and reach the barriers whatever became of their waits).
                if (soft_vote(!(psum <= kMaxSum))) {
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int k = 0; k < 3; ++k) {
                        uint32_t a[16];
                        tmem_ld16(s_col + 16 * k, a);
                        tmem_ld_wait(a);
#pragma unroll
                        for (int q = 0; q < 16; ++q)
                            if (j0 + 16 * k + q < limit) mx = fmaxf(mx, __uint_as_float(a[q]));
                    }
                    sm.part[hf][row] = mx;
                    soft_sync();
                    mx = fmaxf(mx, sm.part[hf ^ 1][row]);
                    mx *= c;
                    // (48 keys that sum to over 2^15 have one above 2^9: that row's reference rises)
                    const float mo = -nm, mn = fmaxf(mo, mx - kMaxExp);
                    const float alpha = mn == -INFINITY ? 1.f : ex2(mo - mn);
                    nm = -mn;
                    lsum *= alpha;
                    if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                        // O holds the tiles before this one, once their products are done: this
                        // half's columns
                        if (alive)
                            alive = ctx.wait_warp(&sm.vempty[(t - 1) & 1], ((t - 1) >> 1) & 1);
                        tc_fence_after();
                        if (alive) {
#pragma unroll 1
                            for (int k = 0; k < 8; ++k) {
                                const uint32_t col = lanes + kColO + hf * 128 + 16 * k;
                                uint32_t o[16];
                                tmem_ld16(col, o);
                                tmem_ld_wait(o);
#pragma unroll
                                for (int q = 0; q < 16; ++q)
                                    o[q] = __float_as_uint(__uint_as_float(o[q]) * alpha);
                                tmem_st16(col, o);
                            }
                            tmem_st_wait();
                        }
                    }
                    psum = probabilities(std::false_type{});
                    // O is rescaled as a whole, and part read, before P of either half is handed over
                    tc_fence_before();
                    soft_sync();
                    tc_fence_after();
                }
                lsum += psum;
                if (!alive) continue;
                // the scores are read: their buffer is free before P is written
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_leader(smem_u32(&sm.sfree[t & 1]));
                // this half of P is free once the products that read it in tile t - 1 are done
                if (i > 0)
                    alive = hf ? ctx.wait_warp(&sm.vempty[(t - 1) & 1], ((t - 1) >> 1) & 1)
                               : ctx.wait_warp(&sm.pdone, (t - 1) & 1);
                if (!alive) continue;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    tmem_st8(lanes + kColP + hf * (kHalfKeys / 2) + 8 * k, code + 8 * k);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_leader(smem_u32(&sm.pfull[hf]));
            }
            g += seg.count;
            // ---- the segment's split state: (m, l), then the numerator through this warp's 8 KB of
            // the Q area (no product reads Q any more), so that rows are stored whole
            if (alive) alive = ctx.wait_warp(&sm.vempty[(g - 1) & 1], ((g - 1) >> 1) & 1);
            sm.part[hf][row] = lsum;
            soft_sync();  // (also: the last scores are complete for every warp, the Q area is free)
            if (alive) {
                tc_fence_after();
                if (hf == 0 && row0 + row < p.rows)
                    p.ws_state[(int64_t)slot * kPairRows + rank * kRows + row] =
                        make_float2(-nm, lsum + sm.part[1][row]);
                float4* stage = reinterpret_cast<float4*>(smem + warp * 8192);
#pragma unroll 1
                for (int part = 0; part < 2; ++part) {  // 64 of this half's 128 columns each
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t o[16];
                        tmem_ld16(lanes + kColO + hf * 128 + part * 64 + 16 * k, o);
                        tmem_ld_wait(o);
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            stage[lane * 16 + ((4 * k + q) ^ (lane & 15))] =
                                make_float4(__uint_as_float(o[4 * q]) * vs,
                                            __uint_as_float(o[4 * q + 1]) * vs,
                                            __uint_as_float(o[4 * q + 2]) * vs,
                                            __uint_as_float(o[4 * q + 3]) * vs);
                    }
                    __syncwarp();
#pragma unroll 8
                    for (int r2 = 0; r2 < 16; ++r2) {
                        const int r = 2 * r2 + (lane >> 4), cc = lane & 15;
                        const int rr = (warp & 3) * 32 + r;
                        if (row0 + rr < p.rows)
                            reinterpret_cast<float4*>(
                                p.ws_acc + ((int64_t)slot * kPairRows + rank * kRows + rr) *
                                               kHeadDim)[hf * 32 + part * 16 + cc] =
                                stage[r * 16 + (cc ^ (r & 15))];
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
            soft_sync();  // every warp is through with the Q area and part
        }
        if (alive) ctx.wait_warp(&sm.done, 0);
    }
    tc_fence_before();
    __syncthreads();
    cluster_arrive();
    cluster_wait();  // neither SM leaves while the other may still arrive here or read here
    if (warp == kQkWarp) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem)
                     : "memory");
    }
}

}  // namespace pairs

// (tc_partial.cu)
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

cudaError_t launch_prefix_pairs(const PrefixPairsParams& p, cudaStream_t stream) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    // A pool as rows (tokens) of Hkv * 256 codes; boxes of one 16-token chunk of one head: whole rows
    // of K (4 KB), this SM's half of the head dim of V (2 KB).
    CUtensorMap kmap, vmap;
    const cuuint64_t row = (cuuint64_t)p.num_kv_heads * kHeadDim;
    const cuuint64_t dims[2] = {row, (cuuint64_t)p.num_pages * p.page_size};
    const cuuint64_t strides[1] = {row};
    const cuuint32_t kbox[2] = {kHeadDim, 16}, vbox[2] = {kHeadDim / 2, 16}, unit[2] = {1, 1};
    const CUresult r1 = encode(&kmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                               const_cast<uint8_t*>(p.k_pool), dims, strides, kbox, unit,
                               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    const CUresult r2 = encode(&vmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                               const_cast<uint8_t*>(p.v_pool), dims, strides, vbox, unit,
                               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r1 != CUDA_SUCCESS || r2 != CUDA_SUCCESS) return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(pairs::prefix_pairs_kernel,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               pairs::kSmemBytes);
    if (e != cudaSuccess) return e;
    pairs::prefix_pairs_kernel<<<2 * p.pairs, pairs::kThreads, pairs::kSmemBytes, stream>>>(
        kmap, vmap, p);
    return cudaGetLastError();
}

}  // namespace dflash
