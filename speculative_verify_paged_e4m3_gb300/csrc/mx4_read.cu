// mx4_read.cu -- tokens of the 4-bit cache as numbers (dflash_mx4_read; dflash_mx4_cache.h has the
// format).
//
// A CTA takes 16 tokens, a warp a row (token, head) of one pool at a time. Tokens that follow one another in
// the cache share V's 16-byte pieces (a byte of each), which the L1 then holds for the CTA.
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

// Four numbers, stored.
template <typename T>
__device__ __forceinline__ void store4(T* dst, const float (&x)[4]) {
    if constexpr (std::is_same_v<T, E5m2>) {
        uint32_t r;
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "cvt.rn.satfinite.e5m2x2.f32 lo, %2, %1;\n\t"
            "cvt.rn.satfinite.e5m2x2.f32 hi, %4, %3;\n\t"
            "mov.b32 %0, {lo, hi};\n\t}"
            : "=r"(r)
            : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]));
        *reinterpret_cast<uint32_t*>(dst) = r;
    } else {
        uint2 w;
        if constexpr (std::is_same_v<T, __half>) {
            const __half2 a = __floats2half2_rn(x[0], x[1]), b = __floats2half2_rn(x[2], x[3]);
            w.x = *reinterpret_cast<const uint32_t*>(&a);
            w.y = *reinterpret_cast<const uint32_t*>(&b);
        } else {
            const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]),
                                 b = __floats2bfloat162_rn(x[2], x[3]);
            w.x = *reinterpret_cast<const uint32_t*>(&a);
            w.y = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint2*>(dst) = w;
    }
}

// The four bytes of codes w as numbers, low halves to lo and high halves to hi.
__device__ __forceinline__ void numbers(uint32_t w, float lo_power, float hi_power, float (&lo)[4],
                                        float (&hi)[4]) {
    const uint32_t h[4] = {mx4::codes_to_f16x2<0>(w), mx4::codes_to_f16x2<1>(w),
                           mx4::codes_to_f16x2<2>(w), mx4::codes_to_f16x2<3>(w)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        lo[i] = f.x * lo_power;
        hi[i] = f.y * hi_power;
    }
}

template <typename T>
__global__ void __launch_bounds__(kReadThreads) mx4_read_kernel(const ReadParams p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t0 = (int64_t)blockIdx.x * kReadTokens;
    const int rows = kReadTokens * p.num_kv_heads;
    // (row r: token r % 16, so that the CTA's warps are in one head's chunk at a time)
    for (int r = warp; r < rows; r += kReadWarps) {
        const int64_t t = t0 + r % kReadTokens;
        const int h = r / kReadTokens;
        if (t >= p.num_tokens) continue;
        const int64_t slot = p.slots[t];
        if (slot < 0 || slot >= p.num_slots) {
            if (slot >= 0 && h == 0 && lane == 0) atomicOr(p.status, DFLASH_FLAG_SLOT_RANGE);
            continue;
        }
        const int tok = (int)(slot % mx4::kTokens);
        const int64_t at = mx4::chunk_offset(slot, p.num_kv_heads, h);
        if (p.k_pool) {
            const uint8_t* chunk = p.k_pool + at;
            const int block = lane >> 2;
            const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(
                chunk + block * 256 + tok * 16 + (lane & 3) * 4));
            const float power = mx4::power_of_scale(
                __ldg(chunk + mx4::kCodeBytes + tok * mx4::kBlocks + block));
            float lo[4], hi[4];
            numbers(w, power, power, lo, hi);
            const float a[4] = {lo[0], hi[0], lo[1], hi[1]}, b[4] = {lo[2], hi[2], lo[3], hi[3]};
            T* dst = static_cast<T*>(p.k_out) + t * p.k_stride + h * kHeadDim + 8 * lane;
            store4(dst, a);
            store4(dst + 4, b);
        }
        if (p.v_pool) {
            const uint8_t* chunk = p.v_pool + at;
            uint32_t w = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w |= (uint32_t)__ldg(chunk + (4 * lane + i) * mx4::kTokens + tok) << (8 * i);
            const uint8_t* scales = chunk + mx4::kCodeBytes + tok * mx4::kBlocks + (lane >> 3);
            float lo[4], hi[4];
            numbers(w, mx4::power_of_scale(__ldg(scales)), mx4::power_of_scale(__ldg(scales + 4)), lo,
                    hi);
            T* dst = static_cast<T*>(p.v_out) + t * p.v_stride + h * kHeadDim + 4 * lane;
            store4(dst, lo);
            store4(dst + kHeadDim / 2, hi);
        }
    }
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
    const unsigned ctas = (unsigned)((num_tokens + kReadTokens - 1) / kReadTokens);
    cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    if (dtype == DFLASH_FP16)
        mx4_read_kernel<__half><<<ctas, kReadThreads, 0, stream>>>(p);
    else if (dtype == DFLASH_BF16)
        mx4_read_kernel<__nv_bfloat16><<<ctas, kReadThreads, 0, stream>>>(p);
    else
        mx4_read_kernel<E5m2><<<ctas, kReadThreads, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}
