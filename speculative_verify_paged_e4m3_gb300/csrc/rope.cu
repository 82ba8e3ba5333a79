// rope.cu -- rotary positions of Q and K, alone or with the write into the E4M3 or the 4-bit cache, head
// norms in the same pass (dflash_paged_step.h and dflash_mx4_cache.h have the definitions).
//
// Angles. Position t turns pair i by t * theta_i. With the frequency held as a 64-bit fraction of a
// turn, f_i = theta_i / (2 pi) * 2^64, the low 64 bits of t * f_i are the fraction of a turn left
// after all whole ones: the range reduction is one integer product, exact at any distance (an FP32
// product would be 2^-6 rad off at position 2^18). The top 32 bits, signed, are within 2^-32 of the
// fraction and become an angle in half turns for sincospi.
//
// One CTA per token, a warp per head row; several tokens a CTA where a token has no more rows than a CTA
// warps (one rank's heads: a CTA's latency for 4 KB). The loads of the rows go out first, up to four a warp;
// while they are in flight the threads compute the token's rotary_dim / 2 cosines and sines, once for all
// heads, into shared memory. A lane has four pairs, whole: in the half layout 4 elements of each half
// (two 8-byte pieces), interleaved 8 in a row; lanes past the rotated part pass 8 elements through.
// Bound by HBM for many tokens, by latency for few: 24571 tokens of 24 + 4 heads in bf16, 112 us, 6.3 TB/s
// (93 % of the copy rate); with the cache write 16381 tokens of 24 + 4 + 4 heads, 87 us, 5.8 TB/s; 8 tokens
// of one rank 2.2 us. With norms 24571 tokens 149 us, 4.7 TB/s: the sum of a row's squares is five exchanges
// between its loads and its stores, of up to four rows at a time; with norms and the write of 16381 tokens into
// the E4M3 cache 116 us, into the 4-bit one 129 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "dflash_mx4_cache.h"
#include "mx4.cuh"
#include "tc_ptx.cuh"

namespace dflash {
namespace {

// Where the rows of K (and V) go: k_out, or the pools of either cache.
enum class To { kRows, kE4m3, kMx4 };

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 5;  // registers cut to fit: 24571 tokens 121 us with 4, 112 with 5, 114 with 6
// With norms, or into the 4-bit cache: 24571 normed tokens 161 us with 3, 149 with 4, 178 with 5 (spills).
constexpr int kCtasMore = 4;
template <To kTo, bool kNorm>
constexpr int ctas_per_sm() {
    return kNorm || kTo == To::kMx4 ? kCtasMore : kCtasPerSm;
}
constexpr int kRows = 4;       // rows of a token that a warp has in flight
// Tokens a CTA for at most 8 rows a token: one up to a wave of CTAs on 152 SMs, two up to three waves, then
// four. One rank's 6 + 1 heads, 256 rotated elements, us with 1 / 2 / 4 tokens a CTA, rotary alone and with
// the cache write: 600 tokens 2.3 / 2.3 / 2.4 and 2.7 / 2.9 / 3.9, 1500 tokens 3.5 / 3.2 / 3.4 and 4.3 /
// 3.8 / 4.6, 16000 tokens 21.9 / 20.7 / 17.5 and 30.9 / 27.1 / 26.1.
constexpr int64_t kTokensOne = 760, kTokensTwo = 4560;
constexpr int64_t kMaxTokens = 0x7FFFFFFF;  // CTAs of a launch
// Rows of V (tokens x KV heads) from which they go to the 4-bit cache by groups of 64 tokens, and tokens up to
// which its CTAs and the tokens' are launched together (256 heads: 5 CTAs a token). With norms, us by groups
// and row by row, slots in runs of 1 (single tokens of as many sequences), of 8 (drafted blocks), in one run
// (a prompt); 24 + 4 heads, then 6 + 1 heads:
//   rows    runs of 1    of 8         one run        runs of 1    of 8         one run
//   1536    7.7   6.3    7.7   7.2    6.2   7.2      7.7   7.2    8.2   7.2    6.2   7.2
//   2048    8.4   7.7    8.7   8.2    6.7   8.2      8.7   7.8    8.2   7.7    7.1   7.7
//   4096   10.8  11.8   10.8  12.1   10.3  12.3     12.7  13.3   12.3  12.8   11.8  12.8
//   8192   19.5  21.1   19.3  21.0   17.4  20.6     21.8  23.6   21.5  22.6   19.5  22.6
//  32768   86.8  80.2   73.8  75.0   65.4  73.7
// (Single tokens of 8192 and more sequences lose 8 %: each token's 128 bytes are sectors of their own either way.)
constexpr int64_t kVGroupFrom = 2048, kVGroupTo = 1 << 28;

struct RopeParams {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const int32_t* positions;
    const int64_t* slots;
    const int32_t* num_live;  // null: every token with a negative slot is padding
    const uint64_t* phases;
    const float *k_scale, *v_scale;
    void *q_out, *k_out;
    int64_t q_out_stride, k_out_stride;
    uint8_t *k_pool, *v_pool;
    int32_t* status;
    int64_t num_tokens, num_slots;
    int num_q_heads, num_kv_heads, rotary_dim;
    float amplitude;
    int64_t v_ctas;                   // To::kMx4: first CTAs, which write V by groups of tokens (0: rows do)
    const void *q_weight, *k_weight;  // head norms; null: that operand is not normed
    float eps, weight_offset;
};

// Four elements of a row (8 bytes).
template <typename T>
__device__ __forceinline__ void unpack(const uint2& w, float (&x)[4]) {
    const uint32_t u[2] = {w.x, w.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float2 f;
        if constexpr (std::is_same_v<T, __half>)
            f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
        else
            f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <typename T>
__device__ __forceinline__ uint2 pack(const float (&x)[4]) {
    uint32_t u[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (std::is_same_v<T, __half>) {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return make_uint2(u[0], u[1]);
}

__device__ __forceinline__ uint32_t e4m3x4(const float (&x)[4], float scale) {
    return ptx::f32x2_to_e4m3x2(__fdiv_rn(x[0], scale), __fdiv_rn(x[1], scale)) |
           (uint32_t)ptx::f32x2_to_e4m3x2(__fdiv_rn(x[2], scale), __fdiv_rn(x[3], scale)) << 16;
}

// Four pairs turned in FP32: of the pieces (a, b) in the half layout, inside each of them interleaved.
template <bool kHalf>
__device__ __forceinline__ void rotate(float (&a)[4], float (&b)[4], const float (&c)[4],
                                       const float (&s)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float& x = kHalf ? a[i] : (i < 2 ? a[2 * i] : b[2 * i - 4]);
        float& y = kHalf ? b[i] : (i < 2 ? a[2 * i + 1] : b[2 * i - 3]);
        const float x0 = x;
        x = fmaf(x0, c[i], -y * s[i]);
        y = fmaf(y, c[i], x0 * s[i]);
    }
}

// Cosine and sine of pair i at position pos, times the amplitude.
__device__ __forceinline__ float2 turn_of(const RopeParams& p, int pos, int i) {
    const uint64_t turn = (uint64_t)(int64_t)pos * p.phases[i];
    float s, c;
    // signed 2^-32 turns -> half turns
    sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &c);
    return make_float2(c * p.amplitude, s * p.amplitude);
}

// The cosines and sines of this lane's four pairs.
__device__ __forceinline__ void lane_turns(const float2* cs, int lane, float (&c)[4], float (&s)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 f = reinterpret_cast<const float4*>(cs)[2 * lane + i];
        c[2 * i] = f.x;
        s[2 * i] = f.y;
        c[2 * i + 1] = f.z;
        s[2 * i + 1] = f.w;
    }
}

// Tokens from here on are padding if their slot is negative.
template <To kTo>
__device__ __forceinline__ int64_t live_tokens(const RopeParams& p) {
    return kTo != To::kRows && p.num_live ? *p.num_live : 0;
}

// The scale of a row's codes (1 for a row of Q).
template <To kTo>
__device__ __forceinline__ float scale_of(const RopeParams& p, int h) {
    return kTo != To::kE4m3 || h < 0 ? 1.f : (h < p.num_kv_heads ? *p.k_scale : *p.v_scale);
}

// Head norms. A head's 256 elements lie in the warp, eight a lane.
__device__ __forceinline__ const void* norm_weight(const RopeParams& p, int h) {
    return h < 0 ? p.q_weight : (h < p.num_kv_heads ? p.k_weight : nullptr);
}
// 1 / sqrt(mean of squares + eps) of several heads, their sums over the warp side by side.
template <typename T, int kHeads>
__device__ __forceinline__ void norm_factors(const RopeParams& p, const uint2 (&wa)[kHeads],
                                             const uint2 (&wb)[kHeads], float (&r)[kHeads]) {
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
        float a[4], b[4];
        unpack<T>(wa[k], a);
        unpack<T>(wb[k], b);
        r[k] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) r[k] = fmaf(a[i], a[i], fmaf(b[i], b[i], r[k]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < kHeads; ++k) r[k] += __shfl_xor_sync(0xffffffffu, r[k], o);
#pragma unroll
    for (int k = 0; k < kHeads; ++k) r[k] = rsqrtf(fmaf(r[k], 1.f / kHeadDim, p.eps));
}
// The lane's pieces (elements from `at` and from at + gap on) times the factor and the weights. (Weights kept
// in registers over the rows of Q cost more in warps than their loads: 24571 tokens 154 us, so 149.)
template <typename T>
__device__ __forceinline__ void norm_row(const RopeParams& p, const void* weight, float r, int at, int gap,
                                         float (&a)[4], float (&b)[4]) {
    float wa[4], wb[4];
    const T* w = static_cast<const T*>(weight) + at;
    unpack<T>(__ldg(reinterpret_cast<const uint2*>(w)), wa);
    unpack<T>(__ldg(reinterpret_cast<const uint2*>(w + gap)), wb);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] = a[i] * r * (p.weight_offset + wa[i]);
        b[i] = b[i] * r * (p.weight_offset + wb[i]);
    }
}

// The largest size of 2^kLog neighbouring lanes' elements, as bits.
template <int kLog>
__device__ __forceinline__ uint32_t lanes_max(uint32_t m) {
#pragma unroll
    for (int o = 1; o < 1 << kLog; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}
__device__ __forceinline__ uint32_t size_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// A row of K into its chunk: the warp brings it in order through its 256 floats of shared memory, so that
// a lane has 8 elements in a row and four lanes a block, whatever the rotary layout.
__device__ __forceinline__ void put_mx4_k(uint8_t* chunk, int tok, int lane, int at, int gap,
                                          const float (&a)[4], const float (&b)[4], float* row) {
    __syncwarp();  // the row before this one has been read
    *reinterpret_cast<float4*>(row + at) = make_float4(a[0], a[1], a[2], a[3]);
    *reinterpret_cast<float4*>(row + at + gap) = make_float4(b[0], b[1], b[2], b[3]);
    __syncwarp();
    const float4 u = reinterpret_cast<const float4*>(row)[2 * lane];
    const float4 v = reinterpret_cast<const float4*>(row)[2 * lane + 1];
    float x[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, size_bits(x[i]));
    const int s = mx4::scale_of_max(lanes_max<2>(m));
    const float inv = mx4::inverse_of_scale(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= inv;
    const uint32_t codes = s == mx4::kNanScale ? 0u : mx4::codes_of(x);
    const int block = lane >> 2;
    *reinterpret_cast<uint32_t*>(chunk + block * 256 + tok * 16 + (lane & 3) * 4) = codes;
    if ((lane & 3) == 0)
        chunk[mx4::kCodeBytes + tok * mx4::kBlocks + block] = (uint8_t)s;
}

// A lane's elements 4 lane + i and 4 lane + 128 + i of a row of V: their codes (byte i), and the scale bytes of
// the two blocks.
struct VCodes {
    uint32_t codes;
    int sa, sb;
};
__device__ __forceinline__ VCodes v_codes(const float (&a)[4], const float (&b)[4]) {
    uint32_t ma = 0, mb = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        ma = max(ma, size_bits(a[i]));
        mb = max(mb, size_bits(b[i]));
    }
    VCodes v;
    v.sa = mx4::scale_of_max(lanes_max<3>(ma));
    v.sb = mx4::scale_of_max(lanes_max<3>(mb));
    const float ia = mx4::inverse_of_scale(v.sa), ib = mx4::inverse_of_scale(v.sb);
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = v.sa == mx4::kNanScale ? 0.f : a[i] * ia;
        x[2 * i + 1] = v.sb == mx4::kNanScale ? 0.f : b[i] * ib;
    }
    v.codes = mx4::codes_of(x);
    return v;
}
__device__ __forceinline__ void put_v_scales(uint8_t* chunk, int tok, int lane, const VCodes& v) {
    if ((lane & 7) == 0) {
        uint8_t* scales = chunk + mx4::kCodeBytes + tok * mx4::kBlocks + (lane >> 3);
        scales[0] = (uint8_t)v.sa;
        scales[4] = (uint8_t)v.sb;
    }
}

// A row of V into its chunk: eight lanes have a block of each half, a lane four bytes, 16 apart.
__device__ __forceinline__ void put_mx4_v(uint8_t* chunk, int tok, int lane, const float (&a)[4],
                                          const float (&b)[4]) {
    const VCodes v = v_codes(a, b);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        chunk[(4 * lane + i) * mx4::kTokens + tok] = (uint8_t)(v.codes >> (8 * i));
    put_v_scales(chunk, tok, lane, v);
}

// V of many tokens: a CTA takes 64 tokens of one head, has their codes in shared memory by words of four
// tokens ([group of four][byte of the row]), and writes what is a whole chunk (16 slots in a row, as tokens of
// a prompt have) in 16-byte pieces, the other tokens byte by byte. Row by row, a token's bytes are 128 stores of
// one, and the L2 takes a sector for each.
constexpr int kVGroup = 64;
template <typename T>
__device__ __forceinline__ void put_v_group(const RopeParams& p, int64_t group, uint32_t* words,
                                            int64_t* places, uint64_t* masks) {
    static_assert(mx4::kTokens == 16 && mx4::kChunkBytes % 16 == 0, "a token's place tells its chunk");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = (int)(group % p.num_kv_heads);
    const int64_t t0 = group / p.num_kv_heads * kVGroup;
    const int n = (int)min((int64_t)kVGroup, p.num_tokens - t0);
    // each token's first byte in the pool (-1: no slot), and as bits which have a slot, and which follow the
    // token before them inside a chunk
    uint32_t* const bits = reinterpret_cast<uint32_t*>(masks);
    if (tid < kVGroup) {
        auto slot_of = [&](int i) -> int64_t {
            const int64_t s = i >= 0 && i < n ? p.slots[t0 + i] : -1;
            return s < p.num_slots ? s : -1;
        };
        const int64_t s = slot_of(tid);
        places[tid] = s < 0 ? -1 : mx4::chunk_offset(s, p.num_kv_heads, h) + s % mx4::kTokens;
        const uint32_t has = __ballot_sync(0xffffffffu, s >= 0);
        const uint32_t follows = __ballot_sync(
            0xffffffffu, s >= 0 && s % mx4::kTokens != 0 && tid > 0 && slot_of(tid - 1) == s - 1);
        if (lane == 0) {
            bits[warp] = has;
            bits[2 + warp] = follows;
        }
    }
    __syncthreads();
    const T* v = static_cast<const T*>(p.v) + h * kHeadDim + 4 * lane;
#pragma unroll
    for (int g = 0; g < kVGroup / 4 / kWarps; ++g) {
        const int tg = warp * (kVGroup / 4 / kWarps) + g;
        uint2 wa[4], wb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const T* row = v + (t0 + min(4 * tg + i, n - 1)) * p.v_stride;
            wa[i] = __ldcs(reinterpret_cast<const uint2*>(row));
            wb[i] = __ldcs(reinterpret_cast<const uint2*>(row + kHeadDim / 2));
        }
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a[4], b[4];
            unpack<T>(wa[i], a);
            unpack<T>(wb[i], b);
            const VCodes c = v_codes(a, b);
            u[i] = c.codes;
            const int64_t at = places[4 * tg + i];
            if (at >= 0) put_v_scales(p.v_pool + (at & ~15ll), (int)(at & 15), lane, c);
        }
        uint32_t w[4];  // four tokens' bytes of elements 4 lane + k
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t two = k | (4 + k) << 4;
            w[k] = __byte_perm(__byte_perm(u[0], u[1], two), __byte_perm(u[2], u[3], two), 0x5410);
        }
        *reinterpret_cast<uint4*>(words + tg * 128 + 4 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncthreads();
    // a thread has one byte of the row; half of the CTA each second whole chunk, and half of the other tokens
    const int e = tid & 127, half = tid >> 7;
    uint64_t whole = masks[1] >> 1;  // first tokens of whole chunks: 15 that follow
    whole &= whole >> 1;
    whole &= whole >> 2;
    whole &= whole >> 4;
    whole &= whole >> 7;
    uint64_t rest = masks[0];
    for (int run = 0; whole; ++run, whole &= whole - 1) {
        const int i = __ffsll((long long)whole) - 1;
        rest &= ~(0xFFFFull << i);
        if ((run & 1) != half) continue;
        const uint32_t* src = words + (i >> 2) * 128 + e;
        const int shift = 8 * (i & 3);
        uint32_t w[5];  // (i <= 47 if it is shifted: the fifth word is there)
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = src[k * 128];
        w[4] = shift ? src[4 * 128] : 0;
        *reinterpret_cast<uint4*>(p.v_pool + places[i] + e * mx4::kTokens) =
            make_uint4(__funnelshift_r(w[0], w[1], shift), __funnelshift_r(w[1], w[2], shift),
                       __funnelshift_r(w[2], w[3], shift), __funnelshift_r(w[3], w[4], shift));
    }
    uint8_t* const pool = p.v_pool + e * mx4::kTokens;
#pragma unroll 4
    for (uint32_t left = (uint32_t)(rest >> (32 * half)); left; left &= left - 1) {
        const int i = 32 * half + __ffs((int)left) - 1;
        pool[places[i]] = (uint8_t)(words[(i >> 2) * 128 + e] >> (8 * (i & 3)));
    }
}

// This lane's two pieces (at, at + gap) of a row: whole pairs, or what makes whole bytes of V's chunk.
struct Pieces {
    int at, gap;
};
template <bool kHalf, To kTo>
__device__ __forceinline__ Pieces pieces_of(int lane, bool turned, int rotary_dim, bool is_v) {
    if (kTo == To::kMx4 && is_v) return {4 * lane, kHeadDim / 2};
    return kHalf && turned ? Pieces{4 * lane, rotary_dim / 2} : Pieces{8 * lane, 4};
}

// Row r of token t: Q rows, then K's, then V's. Its two pieces (at, at + gap) normed and turned, then rounded
// and stored, by the scale that scale_now(its head past Q's) gives. norm: its norm's factor (kNorm); row:
// the warp's shared memory (To::kMx4).
template <typename T, bool kHalf, To kTo, bool kNorm, typename Scale>
__device__ __forceinline__ void put_row(const RopeParams& p, int64_t t, int64_t slot, int r, int at,
                                        int gap, bool turned, const uint2& wa, const uint2& wb,
                                        const float (&c)[4], const float (&s)[4], Scale scale_now,
                                        float norm, float* row) {
    constexpr bool kWrite = kTo != To::kRows;
    const int h = r - p.num_q_heads;
    const bool is_q = h < 0, is_v = h >= p.num_kv_heads;
    const int hk = is_v ? h - p.num_kv_heads : h;
    float a[4], b[4];
    unpack<T>(wa, a);
    unpack<T>(wb, b);
    if constexpr (kNorm) {
        const void* weight = norm_weight(p, h);
        if (weight) norm_row<T>(p, weight, norm, at, gap, a, b);
    }
    // (elements past the rotated part are not multiplied: an infinity times a zero sine
    // would be NaN)
    if (!is_v && turned) rotate<kHalf>(a, b, c, s);
    if (is_q || !kWrite) {
        T* dst = (is_q ? static_cast<T*>(p.q_out) + t * p.q_out_stride + r * kHeadDim
                       : static_cast<T*>(p.k_out) + t * p.k_out_stride + hk * kHeadDim) +
                 at;
        *reinterpret_cast<uint2*>(dst) = pack<T>(a);
        *reinterpret_cast<uint2*>(dst + gap) = pack<T>(b);
    } else if (slot >= 0 && slot < p.num_slots) {
        if constexpr (kTo == To::kMx4) {
            const int tok = (int)(slot % mx4::kTokens), lane = threadIdx.x & 31;
            uint8_t* chunk = (is_v ? p.v_pool : p.k_pool) +
                             mx4::chunk_offset(slot, p.num_kv_heads, hk);
            if (is_v)
                put_mx4_v(chunk, tok, lane, a, b);
            else
                put_mx4_k(chunk, tok, lane, at, gap, a, b, row);
            return;
        }
        const float scale = scale_now(h);
        uint8_t* dst = (is_v ? p.v_pool : p.k_pool) +
                       (slot * p.num_kv_heads + hk) * kHeadDim + at;
        *reinterpret_cast<uint32_t*>(dst) = e4m3x4(a, scale);
        *reinterpret_cast<uint32_t*>(dst + gap) = e4m3x4(b, scale);
    }
}

// Rows of a token that its CTA has: Q's, K's and V's.
template <To kTo>
__host__ __device__ inline int rows_of(const RopeParams& p) {
    return p.num_q_heads + p.num_kv_heads * (kTo != To::kRows ? (p.v_ctas ? 1 : 2) : (p.k ? 1 : 0));
}

// One token a CTA, up to kRows rows of it a warp at a time. K and V rows go to the pools;
// To::kRows: K (if any) to k_out.
template <typename T, bool kHalf, To kTo, bool kNorm>
__global__ void __launch_bounds__(kThreads, (ctas_per_sm<kTo, kNorm>())) rope_kernel(const RopeParams p) {
    constexpr bool kWrite = kTo != To::kRows;
    __shared__ __align__(16) float2 cs[kHeadDim / 2];
    __shared__ __align__(16) float staged[kTo == To::kMx4 ? kWarps : 1][kTo == To::kMx4 ? kHeadDim : 4];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rows = rows_of<kTo>(p);
    int64_t t = blockIdx.x;
    if constexpr (kTo == To::kMx4) {
        __shared__ int64_t v_places[kVGroup];
        __shared__ uint64_t v_masks[2];
        if (t < p.v_ctas) {
            put_v_group<T>(p, t, reinterpret_cast<uint32_t*>(staged), v_places, v_masks);
            return;
        }
        t -= p.v_ctas;
    }
    const int64_t slot = kWrite ? p.slots[t] : 0, live = live_tokens<kTo>(p);
    const int pos = p.positions[t];
    const T* q = static_cast<const T*>(p.q) + t * p.q_stride;
    const T* k = static_cast<const T*>(p.k) + t * p.k_stride;
    const T* v = static_cast<const T*>(p.v) + t * p.v_stride;
    const bool turned = lane < p.rotary_dim / 8;
    auto piece = [&](int h) {
        return pieces_of<kHalf, kTo>(lane, turned, p.rotary_dim, h >= p.num_kv_heads);
    };
    for (int r0 = 0; r0 < rows; r0 += kRows * kWarps) {
        uint2 wa[kRows], wb[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {  // (rows past the last read it again)
            const int r = min(r0 + i * kWarps + warp, rows - 1), h = r - p.num_q_heads;
            const T* src = h < 0 ? q + r * kHeadDim
                                 : (h < p.num_kv_heads ? k + h * kHeadDim
                                                       : v + (h - p.num_kv_heads) * kHeadDim);
            const Pieces pc = piece(h);
            wa[i] = __ldcs(reinterpret_cast<const uint2*>(src + pc.at));
            wb[i] = __ldcs(reinterpret_cast<const uint2*>(src + pc.at + pc.gap));
        }
        if (r0 == 0) {
            if (tid < p.rotary_dim / 2) cs[tid] = turn_of(p, pos, tid);
            __syncthreads();
            if (slot < 0 && t >= live) return;  // padding (the whole CTA agrees)
            if (kWrite && slot >= p.num_slots && tid == 0)
                atomicOr(p.status, DFLASH_FLAG_SLOT_RANGE);
        }
        float c[4], s[4], norm[kRows];
        if constexpr (kNorm) norm_factors<T>(p, wa, wb, norm);
        if (turned) lane_turns(cs, lane, c, s);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i * kWarps + warp;
            if (r >= rows) break;
            const Pieces pc = piece(r - p.num_q_heads);
            put_row<T, kHalf, kTo, kNorm>(p, t, slot, r, pc.at, pc.gap, turned, wa[i], wb[i], c, s,
                                          [&](int hs) { return scale_of<kTo>(p, hs); },
                                          kNorm ? norm[i] : 1.f, staged[kTo == To::kMx4 ? warp : 0]);
        }
    }
}

// kTokens tokens a CTA, for at most kWarps rows a token: warp w has row w of each of them.
template <typename T, bool kHalf, To kTo, bool kNorm, int kTokens>
__global__ void __launch_bounds__(kThreads, (ctas_per_sm<kTo, kNorm>())) rope_tokens_kernel(const RopeParams p) {
    constexpr bool kWrite = kTo != To::kRows;
    __shared__ __align__(16) float2 cs[kTokens][kHeadDim / 2];
    __shared__ __align__(16) float staged[kTo == To::kMx4 ? kWarps : 1][kTo == To::kMx4 ? kHeadDim : 4];
    __shared__ int64_t slots[kTokens];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rows = rows_of<kTo>(p);
    int64_t block = blockIdx.x;
    if constexpr (kTo == To::kMx4) {
        __shared__ int64_t v_places[kVGroup];
        __shared__ uint64_t v_masks[2];
        if (block < p.v_ctas) {
            put_v_group<T>(p, block, reinterpret_cast<uint32_t*>(staged), v_places, v_masks);
            return;
        }
        block -= p.v_ctas;
    }
    const int64_t t0 = block * kTokens, last = p.num_tokens - 1;
    const bool turned = lane < p.rotary_dim / 8;
    // (what is past the last row or token is read again and not stored)
    const int r = min(warp, rows - 1), h = r - p.num_q_heads;
    const Pieces pc = pieces_of<kHalf, kTo>(lane, turned, p.rotary_dim, h >= p.num_kv_heads);
    const int at = pc.at, gap = pc.gap;
    const T* src;
    int64_t stride;
    if (h < 0) {
        src = static_cast<const T*>(p.q) + r * kHeadDim;
        stride = p.q_stride;
    } else if (h < p.num_kv_heads) {
        src = static_cast<const T*>(p.k) + h * kHeadDim;
        stride = p.k_stride;
    } else {
        src = static_cast<const T*>(p.v) + (h - p.num_kv_heads) * kHeadDim;
        stride = p.v_stride;
    }
    uint2 wa[kTokens], wb[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const T* row = src + min(t0 + i, last) * stride;
        wa[i] = __ldcs(reinterpret_cast<const uint2*>(row + at));
        wb[i] = __ldcs(reinterpret_cast<const uint2*>(row + at + gap));
    }
    float norm[kTokens];
    if constexpr (kNorm) norm_factors<T>(p, wa, wb, norm);
    const float scale = scale_of<kTo>(p, h);
    const int64_t live = live_tokens<kTo>(p);
    if (kWrite && tid < kTokens) {
        const int64_t slot = p.slots[min(t0 + tid, last)];
        if (slot >= p.num_slots) atomicOr(p.status, DFLASH_FLAG_SLOT_RANGE);
        slots[tid] = slot;
    }
    constexpr int kPairs = kHeadDim / 2, kEach = kThreads / kPairs;
    if (tid % kPairs < p.rotary_dim / 2) {
#pragma unroll
        for (int i = tid / kPairs; i < kTokens; i += kEach)
            cs[i][tid % kPairs] = turn_of(p, p.positions[min(t0 + i, last)], tid % kPairs);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const int64_t t = t0 + i;
        if (t > last || warp >= rows) return;
        const int64_t slot = kWrite ? slots[i] : 0;
        if (slot < 0 && t >= live) continue;  // padding
        float c[4], s[4];
        if (turned) lane_turns(cs[i], lane, c, s);
        put_row<T, kHalf, kTo, kNorm>(p, t, slot, r, at, gap, turned, wa[i], wb[i], c, s,
                                      [&](int) { return scale; }, kNorm ? norm[i] : 1.f,
                                      staged[kTo == To::kMx4 ? warp : 0]);
    }
}

template <typename T, bool kHalf, To kTo, bool kNorm>
cudaError_t launch_as(const RopeParams& p, cudaStream_t stream) {
    const int rows = rows_of<kTo>(p);
    auto ctas = [&](int tokens) {
        return (unsigned)((p.num_tokens + tokens - 1) / tokens + p.v_ctas);
    };
    if (rows > kWarps)
        rope_kernel<T, kHalf, kTo, kNorm><<<ctas(1), kThreads, 0, stream>>>(p);
    else if (p.num_tokens <= kTokensOne)
        rope_tokens_kernel<T, kHalf, kTo, kNorm, 1><<<ctas(1), kThreads, 0, stream>>>(p);
    else if (p.num_tokens <= kTokensTwo)
        rope_tokens_kernel<T, kHalf, kTo, kNorm, 2><<<ctas(2), kThreads, 0, stream>>>(p);
    else
        rope_tokens_kernel<T, kHalf, kTo, kNorm, 4><<<ctas(4), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <To kTo, bool kNorm>
cudaError_t launch_typed(const dflash_rope_plan_t* plan, const RopeParams& p, cudaStream_t stream) {
    const bool half = plan->problem.layout == DFLASH_ROPE_HALF;
    if (plan->problem.dtype == DFLASH_FP16)
        return half ? launch_as<__half, true, kTo, kNorm>(p, stream)
                    : launch_as<__half, false, kTo, kNorm>(p, stream);
    return half ? launch_as<__nv_bfloat16, true, kTo, kNorm>(p, stream)
                : launch_as<__nv_bfloat16, false, kTo, kNorm>(p, stream);
}

// One launch; without a norm, by kernels that have none.
template <To kTo>
int launch(const dflash_rope_plan_t* plan, RopeParams& p, const dflash_head_norm* norm,
           void* cuda_stream) {
    cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    cudaError_t e;
    if (norm && (norm->q_weight || norm->k_weight)) {
        p.q_weight = norm->q_weight;
        p.k_weight = norm->k_weight;
        p.eps = norm->eps;
        p.weight_offset = norm->weight_offset;
        e = launch_typed<kTo, true>(plan, p, stream);
    } else {
        e = launch_typed<kTo, false>(plan, p, stream);
    }
    return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A strided [tokens, heads, 256] operand: 16-byte rows, token stride of whole 8-element groups.
bool rows_ok(const void* x, int64_t stride, int heads) {
    return x && aligned(x, 16) && stride % 8 == 0 && stride >= (int64_t)heads * kHeadDim &&
           stride <= (int64_t)1 << 40;
}

// An output at the address of another buffer (in place, q_out = q or k_out = k, is the caller's to
// check) would be read, or written twice, while it is written.
template <int kOuts, int kOthers>
bool distinct(const void* const (&outs)[kOuts], const void* const (&others)[kOthers]) {
    for (int i = 0; i < kOuts; ++i) {
        for (int j = 0; j < kOthers; ++j)
            if (outs[i] && outs[i] == others[j]) return false;
        for (int j = 0; j < i; ++j)
            if (outs[i] && outs[i] == outs[j]) return false;
    }
    return true;
}

bool finite(double x) { return x - x == 0.0; }

int check_problem(const dflash_rope_problem* pr) {
    if (!pr || pr->version != DFLASH_PAGED_STEP_VERSION) return DFLASH_ERR_INVALID_ARGUMENT;
    if (pr->num_q_heads < 1 || pr->num_q_heads > 256 || pr->num_kv_heads < 1 ||
        pr->num_kv_heads > 256 || pr->page_size < 1 || pr->num_pages < 1 || pr->reserved != 0 ||
        pr->layout < DFLASH_ROPE_HALF || pr->layout > DFLASH_ROPE_INTERLEAVED ||
        pr->dtype < DFLASH_FP16 || pr->dtype > DFLASH_BF16 ||
        pr->scaling < DFLASH_ROPE_SCALE_NONE || pr->scaling > DFLASH_ROPE_SCALE_WAVELENGTH)
        return DFLASH_ERR_INVALID_ARGUMENT;
    if (pr->head_dim < 1 || pr->rotary_dim < 1 || pr->rotary_dim > pr->head_dim)
        return DFLASH_ERR_INVALID_ARGUMENT;
    if (!finite(pr->base) || pr->base <= 1.0) return DFLASH_ERR_INVALID_ARGUMENT;
    if (pr->scaling != DFLASH_ROPE_SCALE_NONE && (!finite(pr->factor) || pr->factor < 1.0))
        return DFLASH_ERR_INVALID_ARGUMENT;
    if (pr->scaling >= DFLASH_ROPE_SCALE_YARN && pr->trained_context < 1)
        return DFLASH_ERR_INVALID_ARGUMENT;
    if (pr->scaling == DFLASH_ROPE_SCALE_YARN &&
        (!finite(pr->beta_fast) || !finite(pr->beta_slow) || pr->beta_fast <= 0.0 ||
         pr->beta_slow <= 0.0))
        return DFLASH_ERR_INVALID_ARGUMENT;
    if (pr->scaling == DFLASH_ROPE_SCALE_WAVELENGTH &&
        (!finite(pr->low_turns) || !finite(pr->high_turns) || pr->low_turns >= pr->high_turns))
        return DFLASH_ERR_INVALID_ARGUMENT;
    if (pr->head_dim != kHeadDim || pr->rotary_dim % 16 != 0) return DFLASH_ERR_UNSUPPORTED;
    return DFLASH_OK;
}

int check_plan(const dflash_rope_plan_t* plan) {
    if (!plan || plan->version != DFLASH_PAGED_STEP_VERSION) return DFLASH_ERR_INVALID_ARGUMENT;
    return check_problem(&plan->problem);
}

// A norm's own fields, and its weights apart from what the call writes.
template <int kOuts>
bool norm_ok(const dflash_head_norm* norm, const void* const (&outs)[kOuts]) {
    if (!norm) return true;
    if (!finite(norm->eps) || norm->eps < 0.f || !finite(norm->weight_offset) ||
        !aligned(norm->q_weight, 16) || !aligned(norm->k_weight, 16))
        return false;
    for (int i = 0; i < kOuts; ++i)
        if (outs[i] && (outs[i] == norm->q_weight || outs[i] == norm->k_weight)) return false;
    return true;
}

double clamp01(double x) { return x < 0.0 ? 0.0 : (x > 1.0 ? 1.0 : x); }

// The cache writes: checks and launch. k_scale and v_scale are To::kE4m3's.
template <To kTo>
int write(const dflash_rope_plan_t* plan, const dflash_head_norm* norm, int64_t num_tokens,
          const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
          int64_t v_stride, const int32_t* positions, const int64_t* slots,
          const int32_t* num_live, const uint64_t* phases, const float* k_scale,
          const float* v_scale, void* q_out, int64_t q_out_stride, void* k_pool, void* v_pool,
          int32_t* status, void* cuda_stream) {
    constexpr bool kScaled = kTo == To::kE4m3;
    constexpr size_t kPoolAlign = kScaled ? 8 : 16;
    const int rc = check_plan(plan);
    if (rc != DFLASH_OK) return rc;
    const dflash_rope_problem& pr = plan->problem;
    if (!kScaled && pr.page_size % mx4::kTokens != 0) return DFLASH_ERR_UNSUPPORTED;
    if (num_tokens < 0 || num_tokens > kMaxTokens) return DFLASH_ERR_INVALID_ARGUMENT;
    if (num_tokens == 0) return DFLASH_OK;
    if (!rows_ok(q, q_stride, pr.num_q_heads) || !rows_ok(k, k_stride, pr.num_kv_heads) ||
        !rows_ok(v, v_stride, pr.num_kv_heads) || !rows_ok(q_out, q_out_stride, pr.num_q_heads) ||
        !positions || !aligned(positions, 4) || !slots || !aligned(slots, 8) || !phases ||
        !aligned(phases, 8) ||
        (kScaled &&
         (!k_scale || !aligned(k_scale, 4) || !v_scale || !aligned(v_scale, 4))) ||
        !k_pool || !aligned(k_pool, kPoolAlign) || !v_pool || !aligned(v_pool, kPoolAlign) ||
        !status || !aligned(status, 4) || !aligned(num_live, 4) ||
        (q == q_out && q_stride != q_out_stride))
        return DFLASH_ERR_INVALID_ARGUMENT;
    const void* const outs[] = {q_out, k_pool, v_pool, status};
    const void* const others[] = {k, v, positions, slots, phases, k_scale, v_scale, num_live};
    if (!distinct(outs, others) || k_pool == q || v_pool == q || status == q ||
        !norm_ok(norm, outs))
        return DFLASH_ERR_INVALID_ARGUMENT;
    RopeParams p = {};
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.positions = positions;
    p.slots = slots;
    p.num_live = num_live;
    p.phases = phases;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.q_out = q_out;
    p.q_out_stride = q_out_stride;
    p.k_pool = static_cast<uint8_t*>(k_pool);
    p.v_pool = static_cast<uint8_t*>(v_pool);
    p.status = status;
    p.num_tokens = num_tokens;
    p.num_slots = (int64_t)pr.num_pages * pr.page_size;
    p.num_q_heads = pr.num_q_heads;
    p.num_kv_heads = pr.num_kv_heads;
    p.rotary_dim = pr.rotary_dim;
    p.amplitude = plan->amplitude;
    if (!kScaled && num_tokens * pr.num_kv_heads >= kVGroupFrom && num_tokens <= kVGroupTo)
        p.v_ctas = (num_tokens + kVGroup - 1) / kVGroup * pr.num_kv_heads;
    return launch<kTo>(plan, p, norm, cuda_stream);
}

}  // namespace
}  // namespace dflash

using namespace dflash;

extern "C" {

int dflash_rope_plan(const dflash_rope_problem* pr, dflash_rope_plan_t* plan, uint64_t* phases) {
    const int rc = check_problem(pr);
    if (rc != DFLASH_OK) return rc;
    if (!plan || !phases) return DFLASH_ERR_INVALID_ARGUMENT;
    const double kTwoPi = 6.283185307179586476925;
    const int d = pr->rotary_dim;
    const double s = pr->factor;
    double base = pr->base;
    if (pr->scaling == DFLASH_ROPE_SCALE_NTK) base *= pow(s, (double)d / (d - 2));
    double lo = 0, hi = 0;
    if (pr->scaling == DFLASH_ROPE_SCALE_YARN) {
        const double per = d / (2.0 * log(base));
        lo = floor(per * log(pr->trained_context / (pr->beta_fast * kTwoPi)));
        hi = ceil(per * log(pr->trained_context / (pr->beta_slow * kTwoPi)));
        if (lo < 0) lo = 0;
        if (hi > d - 1) hi = d - 1;
    }
    for (int i = 0; i < d / 2; ++i) {
        double theta = pow(base, -2.0 * i / d);
        if (pr->scaling == DFLASH_ROPE_SCALE_LINEAR) {
            theta /= s;
        } else if (pr->scaling == DFLASH_ROPE_SCALE_YARN) {
            const double r = clamp01((i - lo) / (hi - lo < 0.001 ? 0.001 : hi - lo));
            theta = theta / s * r + theta * (1.0 - r);
        } else if (pr->scaling == DFLASH_ROPE_SCALE_WAVELENGTH) {
            const double turns = pr->trained_context * theta / kTwoPi;
            const double g = clamp01((turns - pr->low_turns) / (pr->high_turns - pr->low_turns));
            theta = theta / s * (1.0 - g) + theta * g;
        }
        phases[i] = (uint64_t)ldexp(theta / kTwoPi, 64);  // theta <= 1: below 2^62
    }
    plan->version = DFLASH_PAGED_STEP_VERSION;
    plan->amplitude =
        pr->scaling == DFLASH_ROPE_SCALE_YARN ? (float)(0.1 * log(s) + 1.0) : 1.0f;
    plan->problem = *pr;
    return DFLASH_OK;
}

int dflash_rope_apply(const dflash_rope_plan_t* plan, int64_t num_tokens, const void* q,
                      int64_t q_stride, const void* k, int64_t k_stride, const int32_t* positions,
                      const uint64_t* phases, void* q_out, int64_t q_out_stride, void* k_out,
                      int64_t k_out_stride, void* cuda_stream) {
    return dflash_norm_rope_apply(plan, nullptr, num_tokens, q, q_stride, k, k_stride, positions,
                                  phases, q_out, q_out_stride, k_out, k_out_stride, cuda_stream);
}

int dflash_norm_rope_apply(const dflash_rope_plan_t* plan, const dflash_head_norm* norm,
                           int64_t num_tokens, const void* q, int64_t q_stride, const void* k,
                           int64_t k_stride, const int32_t* positions, const uint64_t* phases,
                           void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                           void* cuda_stream) {
    const int rc = check_plan(plan);
    if (rc != DFLASH_OK) return rc;
    const dflash_rope_problem& pr = plan->problem;
    if (num_tokens < 0 || num_tokens > kMaxTokens || (k == nullptr) != (k_out == nullptr))
        return DFLASH_ERR_INVALID_ARGUMENT;
    if (num_tokens == 0) return DFLASH_OK;
    if (!rows_ok(q, q_stride, pr.num_q_heads) || !rows_ok(q_out, q_out_stride, pr.num_q_heads) ||
        (k && (!rows_ok(k, k_stride, pr.num_kv_heads) ||
               !rows_ok(k_out, k_out_stride, pr.num_kv_heads))) ||
        !positions || !aligned(positions, 4) || !phases || !aligned(phases, 8) ||
        (q == q_out && q_stride != q_out_stride) || (k && k == k_out && k_stride != k_out_stride))
        return DFLASH_ERR_INVALID_ARGUMENT;
    const void* const outs[] = {q_out, k_out};
    const void* const others[] = {positions, phases};
    if (!distinct(outs, others) || q_out == k || (k && k_out == q) || !norm_ok(norm, outs))
        return DFLASH_ERR_INVALID_ARGUMENT;
    RopeParams p = {};
    p.q = q;
    p.k = k;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.positions = positions;
    p.phases = phases;
    p.q_out = q_out;
    p.k_out = k_out;
    p.q_out_stride = q_out_stride;
    p.k_out_stride = k_out_stride;
    p.num_tokens = num_tokens;
    p.num_q_heads = pr.num_q_heads;
    p.num_kv_heads = pr.num_kv_heads;
    p.rotary_dim = pr.rotary_dim;
    p.amplitude = plan->amplitude;
    return launch<To::kRows>(plan, p, norm, cuda_stream);
}

int dflash_rope_kv_write(const dflash_rope_plan_t* plan, int64_t num_tokens, const void* q,
                         int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                         int64_t v_stride, const int32_t* positions, const int64_t* slots,
                         const uint64_t* phases, const float* k_scale, const float* v_scale,
                         void* q_out, int64_t q_out_stride, void* k_pool, void* v_pool,
                         int32_t* status, void* cuda_stream) {
    return dflash_rope_kv_write_live(plan, num_tokens, q, q_stride, k, k_stride, v, v_stride,
                                     positions, slots, nullptr, phases, k_scale, v_scale, q_out,
                                     q_out_stride, k_pool, v_pool, status, cuda_stream);
}

int dflash_rope_kv_write_live(const dflash_rope_plan_t* plan, int64_t num_tokens, const void* q,
                              int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                              int64_t v_stride, const int32_t* positions, const int64_t* slots,
                              const int32_t* num_live, const uint64_t* phases,
                              const float* k_scale, const float* v_scale, void* q_out,
                              int64_t q_out_stride, void* k_pool, void* v_pool, int32_t* status,
                              void* cuda_stream) {
    return dflash_norm_rope_kv_write(plan, nullptr, num_tokens, q, q_stride, k, k_stride, v,
                                     v_stride, positions, slots, num_live, phases, k_scale,
                                     v_scale, q_out, q_out_stride, k_pool, v_pool, status,
                                     cuda_stream);
}

int dflash_norm_rope_kv_write(const dflash_rope_plan_t* plan, const dflash_head_norm* norm,
                              int64_t num_tokens, const void* q, int64_t q_stride, const void* k,
                              int64_t k_stride, const void* v, int64_t v_stride,
                              const int32_t* positions, const int64_t* slots,
                              const int32_t* num_live, const uint64_t* phases,
                              const float* k_scale, const float* v_scale, void* q_out,
                              int64_t q_out_stride, void* k_pool, void* v_pool, int32_t* status,
                              void* cuda_stream) {
    return write<To::kE4m3>(plan, norm, num_tokens, q, q_stride, k, k_stride, v, v_stride,
                            positions, slots, num_live, phases, k_scale, v_scale, q_out,
                            q_out_stride, k_pool, v_pool, status, cuda_stream);
}

int dflash_mx4_kv_write(const dflash_rope_plan_t* plan, const dflash_head_norm* norm,
                        int64_t num_tokens, const void* q, int64_t q_stride, const void* k,
                        int64_t k_stride, const void* v, int64_t v_stride,
                        const int32_t* positions, const int64_t* slots, const int32_t* num_live,
                        const uint64_t* phases, void* q_out, int64_t q_out_stride, void* k_pool,
                        void* v_pool, int32_t* status, void* cuda_stream) {
    return write<To::kMx4>(plan, norm, num_tokens, q, q_stride, k, k_stride, v, v_stride,
                           positions, slots, num_live, phases, nullptr, nullptr, q_out,
                           q_out_stride, k_pool, v_pool, status, cuda_stream);
}

}  // extern "C"
