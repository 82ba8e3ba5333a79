// mx4_read.cu -- tokens of the 4-bit cache as numbers (dflash_mx4_read; dflash_mx4_cache.h has the
// format).
//
// A CTA takes 16 tokens of one head, half of its warps K, half V. K's rows go a warp each, 8 elements a lane. V's
// chunk has a token's bytes 16 apart, so that a thread takes four of them (elements 4j .. 4j + 3 and 128
// more) for four tokens: a word each, if the four lie one after the other in a chunk, as tokens of a context
// do, or two words shifted; else bytes. Bound by HBM: 65536 tokens of 4 heads as FP16, 69 us, 4.9 TB/s (72 % of
// the copy rate); few tokens by latency, 64 tokens of one head 3.1 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "dflash_mx4_cache.h"
#include "mx4.cuh"

namespace dflash {
namespace {

constexpr int kReadThreads = 256;
constexpr int kReadWarps = kReadThreads / 32;
constexpr int kReadTokens = 16;
// CTAs an SM, registers cut to fit: 262144 tokens of 4 heads 300 us with 4 to 6, 271 with 8.
constexpr int kReadCtas = 8;
constexpr int64_t kMaxTokens = 0x7FFFFFFF;

struct E5m2 {
    uint8_t code;
};

struct ReadParams {
    const uint8_t *k_pool, *v_pool;
    const int64_t* slots;
    void *k_out, *v_out;
    int64_t k_stride, v_stride, num_tokens, num_slots;
    int32_t* status;
    int num_kv_heads;
};

// Numbers, stored in one piece.
template <typename T, int kN>
__device__ __forceinline__ void store(T* dst, const float (&x)[kN]) {
    static_assert(kN == 4 || kN == 8, "four or eight");
    if constexpr (std::is_same_v<T, E5m2>) {
        uint32_t w[kN / 4];
#pragma unroll
        for (int i = 0; i < kN / 4; ++i)
            asm("{\n\t.reg .b16 lo, hi;\n\t"
                "cvt.rn.satfinite.e5m2x2.f32 lo, %2, %1;\n\t"
                "cvt.rn.satfinite.e5m2x2.f32 hi, %4, %3;\n\t"
                "mov.b32 %0, {lo, hi};\n\t}"
                : "=r"(w[i])
                : "f"(x[4 * i]), "f"(x[4 * i + 1]), "f"(x[4 * i + 2]), "f"(x[4 * i + 3]));
        if constexpr (kN == 4)
            *reinterpret_cast<uint32_t*>(dst) = w[0];
        else
            *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    } else {
        uint32_t w[kN / 2];
#pragma unroll
        for (int i = 0; i < kN / 2; ++i) {
            if constexpr (std::is_same_v<T, __half>) {
                const __half2 r = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&r);
            } else {
                const __nv_bfloat162 r = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&r);
            }
        }
        if constexpr (kN == 4)
            *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// The four bytes of codes w as numbers, low halves to lo and high halves to hi.
__device__ __forceinline__ void numbers(uint32_t w, float (&lo)[4], float (&hi)[4]) {
    const uint32_t h[4] = {mx4::codes_to_f16x2<0>(w), mx4::codes_to_f16x2<1>(w),
                           mx4::codes_to_f16x2<2>(w), mx4::codes_to_f16x2<3>(w)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        lo[i] = f.x;
        hi[i] = f.y;
    }
}

template <typename T>
__global__ void __launch_bounds__(kReadThreads, kReadCtas) mx4_read_kernel(const ReadParams p) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = blockIdx.y;
    const int64_t t0 = (int64_t)blockIdx.x * kReadTokens;
    __shared__ int64_t slots[kReadTokens];
    if (tid < kReadTokens) {
        int64_t s = t0 + tid < p.num_tokens ? p.slots[t0 + tid] : -1;
        if (s >= p.num_slots) {
            if (h == 0) atomicOr(p.status, DFLASH_FLAG_SLOT_RANGE);
            s = -1;
        }
        slots[tid] = s;
    }
    __syncthreads();
    constexpr int kHalf = kReadWarps / 2;
    if (warp < kHalf) {
        if (!p.k_pool) return;
#pragma unroll
        for (int i = 0; i < kReadTokens / kHalf; ++i) {
            const int r = warp + kHalf * i;
            const int64_t slot = slots[r];
            if (slot < 0) continue;
            const int tok = (int)(slot % mx4::kTokens), block = lane >> 2;
            const uint8_t* chunk = p.k_pool + mx4::chunk_offset(slot, p.num_kv_heads, h);
            const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(
                chunk + block * 256 + tok * 16 + (lane & 3) * 4));
            const float power = mx4::power_of_scale(
                __ldg(chunk + mx4::kCodeBytes + tok * mx4::kBlocks + block));
            float lo[4], hi[4];
            numbers(w, lo, hi);
            float x[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[2 * k] = lo[k] * power;
                x[2 * k + 1] = hi[k] * power;
            }
            store(static_cast<T*>(p.k_out) + (t0 + r) * p.k_stride + h * kHeadDim + 8 * lane, x);
        }
        return;
    }
    if (!p.v_pool) return;
    constexpr int kEach = 4;  // tokens, and elements of each half of the head, a thread
    static_assert(kHalf * kEach == kReadTokens && kEach * 32 == kHeadDim / 2, "threads of a CTA");
    const int e = kEach * lane, first = kEach * (warp - kHalf);
    const int64_t* s = slots + first;
    const bool run = s[0] >= 0 && s[1] == s[0] + 1 && s[2] == s[0] + 2 && s[3] == s[0] + 3 &&
                     s[0] % mx4::kTokens <= mx4::kTokens - kEach;
    uint32_t w[kEach] = {};  // the four tokens' bytes of element e + k
    if (run) {
        const int tok = (int)(s[0] % mx4::kTokens);
        const uint8_t* at =
            p.v_pool + mx4::chunk_offset(s[0], p.num_kv_heads, h) + e * mx4::kTokens + (tok & ~3);
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const uint32_t* q = reinterpret_cast<const uint32_t*>(at + k * mx4::kTokens);
            w[k] = __ldg(q);
            if (tok & 3) w[k] = __funnelshift_r(w[k], __ldg(q + 1), 8 * (tok & 3));
        }
    } else {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (s[i] < 0) continue;
            const uint8_t* at = p.v_pool + mx4::chunk_offset(s[i], p.num_kv_heads, h) + e * mx4::kTokens +
                                s[i] % mx4::kTokens;
#pragma unroll
            for (int k = 0; k < kEach; ++k) w[k] |= (uint32_t)__ldg(at + k * mx4::kTokens) << (8 * i);
        }
    }
    // token first + i, byte i of the words
    auto put = [&](auto byte) {
        constexpr int i = decltype(byte)::value;
        if (s[i] < 0) return;
        const uint8_t* scales = p.v_pool + mx4::chunk_offset(s[i], p.num_kv_heads, h) + mx4::kCodeBytes +
                                s[i] % mx4::kTokens * mx4::kBlocks + e / mx4::kBlock;
        const float pl = mx4::power_of_scale(__ldg(scales)), ph = mx4::power_of_scale(__ldg(scales + 4));
        T* dst = static_cast<T*>(p.v_out) + (t0 + first + i) * p.v_stride + h * kHeadDim + e;
        float a[kEach], b[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const uint32_t x = mx4::codes_to_f16x2<i>(w[k]);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
            a[k] = f.x * pl;
            b[k] = f.y * ph;
        }
        store(dst, a);
        store(dst + kHeadDim / 2, b);
    };
    put(std::integral_constant<int, 0>{});
    put(std::integral_constant<int, 1>{});
    put(std::integral_constant<int, 2>{});
    put(std::integral_constant<int, 3>{});
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A pool with its output: both there and well formed, or neither.
bool operand_ok(const void* pool, const void* out, int64_t stride, int heads) {
    if (!pool && !out) return true;
    return pool && out && aligned(pool, 16) && aligned(out, 16) && stride % 16 == 0 &&
           stride >= (int64_t)heads * kHeadDim && stride <= (int64_t)1 << 40;
}

}  // namespace
}  // namespace dflash

using namespace dflash;

extern "C" int dflash_mx4_read(int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                               int32_t num_pages, const void* k_pool, const void* v_pool,
                               int64_t num_tokens, const int64_t* slots, int32_t dtype,
                               void* k_out, int64_t k_out_stride, void* v_out,
                               int64_t v_out_stride, int32_t* status, void* cuda_stream) {
    if (num_kv_heads < 1 || num_kv_heads > 256 || head_dim < 1 || page_size < 1 || num_pages < 1 ||
        dtype < DFLASH_FP16 || dtype > DFLASH_E5M2 || num_tokens < 0 || num_tokens > kMaxTokens)
        return DFLASH_ERR_INVALID_ARGUMENT;
    if (head_dim != kHeadDim || page_size % mx4::kTokens != 0) return DFLASH_ERR_UNSUPPORTED;
    if (num_tokens == 0) return DFLASH_OK;
    if ((!k_pool && !v_pool) || !operand_ok(k_pool, k_out, k_out_stride, num_kv_heads) ||
        !operand_ok(v_pool, v_out, v_out_stride, num_kv_heads) || !slots || !aligned(slots, 8) ||
        !status || !aligned(status, 4))
        return DFLASH_ERR_INVALID_ARGUMENT;
    const void* const outs[] = {k_out, v_out, status};
    const void* const others[] = {k_pool, v_pool, slots};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 3; ++j)
            if (outs[i] && outs[i] == others[j]) return DFLASH_ERR_INVALID_ARGUMENT;
        for (int j = 0; j < i; ++j)
            if (outs[i] && outs[i] == outs[j]) return DFLASH_ERR_INVALID_ARGUMENT;
    }
    ReadParams p = {};
    p.k_pool = static_cast<const uint8_t*>(k_pool);
    p.v_pool = static_cast<const uint8_t*>(v_pool);
    p.slots = slots;
    p.k_out = k_out;
    p.v_out = v_out;
    p.k_stride = k_out_stride;
    p.v_stride = v_out_stride;
    p.num_tokens = num_tokens;
    p.num_slots = (int64_t)num_pages * page_size;
    p.status = status;
    p.num_kv_heads = num_kv_heads;
    const dim3 ctas((unsigned)((num_tokens + kReadTokens - 1) / kReadTokens), num_kv_heads);
    cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    if (dtype == DFLASH_FP16)
        mx4_read_kernel<__half><<<ctas, kReadThreads, 0, stream>>>(p);
    else if (dtype == DFLASH_BF16)
        mx4_read_kernel<__nv_bfloat16><<<ctas, kReadThreads, 0, stream>>>(p);
    else
        mx4_read_kernel<E5m2><<<ctas, kReadThreads, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}
