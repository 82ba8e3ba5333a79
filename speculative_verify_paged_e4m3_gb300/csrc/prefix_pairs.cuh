// prefix_pairs.cuh -- how the pair kernel deals the shared prefix out to pairs of SMs, for the
// kernel, the combine and the planner.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace dflash {

constexpr int kPairRows = 256;     // query rows of a block: 128 on each SM of a pair
constexpr int kPairTile = 96;      // keys per tile
constexpr int kPairMinTiles = 4;   // least tiles worth a pair of their own

// The work is units (KV head, row block), tiles of keys inside a unit, in one line, `pitch` tiles
// of it to a unit: pair p takes tiles [p * per_pair, (p + 1) * per_pair). A pair's share of one unit
// is a segment with a split state of its own in workspace slot p + unit: along the line either p or
// the unit moves on at each new segment, so the sum names it, and pairs + units slots are enough.
// Equal shares of everything (pitch = tiles) let a pair's share run over a unit's end, which costs a
// second epilogue, Q and pipeline fill, about kPairSwitch tiles. Where whole pairs for each unit
// (pitch = a multiple of per_pair, the end of it empty) cost no more than that, they are taken: 32
// single tokens over 65536 keys 82 -> 79 us, 16 x 8 tokens over 32768 keys 118 -> 111 (24/4 heads, the
// whole call, without and with).
constexpr int kPairSwitch = 7;

struct PairShare {
    int tiles;         // per unit
    int64_t pitch;     // tiles of the line per unit, >= tiles
    int64_t per_pair;  // tiles per pair
};

__host__ __device__ inline PairShare pair_share(int keys, int units, int pairs) {
    PairShare s;
    s.tiles = (keys + kPairTile - 1) / kPairTile;
    s.pitch = s.tiles;
    const int64_t total = (int64_t)units * s.tiles;
    s.per_pair = (total + pairs - 1) / pairs;
    if (s.per_pair < kPairMinTiles) s.per_pair = kPairMinTiles;
    const int own = pairs / units;  // whole pairs a unit
    if (own > 0) {
        int per = (s.tiles + own - 1) / own;
        if (per < kPairMinTiles) per = kPairMinTiles;
        if (per <= s.per_pair + kPairSwitch) {
            s.per_pair = per;
            s.pitch = (int64_t)((s.tiles + per - 1) / per) * per;
        }
    }
    return s;
}

struct PrefixPairsParams {
    const __half* q;
    const uint8_t *k_pool, *v_pool;
    const int32_t *prefix_table, *prefix_len, *context_lens;
    const float *k_scale, *v_scale;
    int32_t* status;
    float2* ws_state;  // [slots, 256]
    float* ws_acc;     // [slots, 256, D]
    int rows, blocks, units, pairs;
    int q_len, group, num_q_heads, num_kv_heads;
    int page_size, page_shift, num_pages, max_prefix, max_context;
};

cudaError_t launch_prefix_pairs(const PrefixPairsParams& p, cudaStream_t stream);

}  // namespace dflash
