// rope.cu -- rotary positions of Q and K, alone or with the E4M3 cache write
// (dflash_paged_step.h has the definition).
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
// of one rank 2.2 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "dflash_paged_step.h"
#include "tc_ptx.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 5;  // registers cut to fit: 24571 tokens 121 us with 4, 112 with 5, 114 with 6
constexpr int kRows = 4;       // rows of a token that a warp has in flight
// Tokens a CTA for at most 8 rows a token: one up to a wave of CTAs on 152 SMs, two up to three waves, then
// four. One rank's 6 + 1 heads, 256 rotated elements, us with 1 / 2 / 4 tokens a CTA, rotary alone and with
// the cache write: 600 tokens 2.3 / 2.3 / 2.4 and 2.7 / 2.9 / 3.9, 1500 tokens 3.5 / 3.2 / 3.4 and 4.3 /
// 3.8 / 4.6, 16000 tokens 21.9 / 20.7 / 17.5 and 30.9 / 27.1 / 26.1.
constexpr int64_t kTokensOne = 760, kTokensTwo = 4560;
constexpr int64_t kMaxTokens = 0x7FFFFFFF;  // CTAs of a launch

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
template <bool kWrite>
__device__ __forceinline__ int64_t live_tokens(const RopeParams& p) {
    return kWrite && p.num_live ? *p.num_live : 0;
}

// The scale of a row's codes (1 for a row of Q).
template <bool kWrite>
__device__ __forceinline__ float scale_of(const RopeParams& p, int h) {
    return !kWrite || h < 0 ? 1.f : (h < p.num_kv_heads ? *p.k_scale : *p.v_scale);
}

// Row r of token t: Q rows, then K's, then V's. Its two pieces (at, at + gap) turned, then rounded and
// stored, by the scale that scale_now(its head past Q's) gives.
template <typename T, bool kHalf, bool kWrite, typename Scale>
__device__ __forceinline__ void put_row(const RopeParams& p, int64_t t, int64_t slot, int r, int at,
                                        int gap, bool turned, const uint2& wa, const uint2& wb,
                                        const float (&c)[4], const float (&s)[4], Scale scale_now) {
    const int h = r - p.num_q_heads;
    const bool is_q = h < 0, is_v = h >= p.num_kv_heads;
    const int hk = is_v ? h - p.num_kv_heads : h;
    float a[4], b[4];
    unpack<T>(wa, a);
    unpack<T>(wb, b);
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
        const float scale = scale_now(h);
        uint8_t* dst = (is_v ? p.v_pool : p.k_pool) +
                       (slot * p.num_kv_heads + hk) * kHeadDim + at;
        *reinterpret_cast<uint32_t*>(dst) = e4m3x4(a, scale);
        *reinterpret_cast<uint32_t*>(dst + gap) = e4m3x4(b, scale);
    }
}

// One token a CTA, up to kRows rows of it a warp at a time. kWrite: K and V rows go to the pools as E4M3;
// else K (if any) to k_out.
template <typename T, bool kHalf, bool kWrite>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) rope_kernel(const RopeParams p) {
    __shared__ __align__(16) float2 cs[kHeadDim / 2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rows = p.num_q_heads + p.num_kv_heads * (kWrite ? 2 : (p.k ? 1 : 0));
    const int64_t t = blockIdx.x;
    const int64_t slot = kWrite ? p.slots[t] : 0, live = live_tokens<kWrite>(p);
    const int pos = p.positions[t];
    const T* q = static_cast<const T*>(p.q) + t * p.q_stride;
    const T* k = static_cast<const T*>(p.k) + t * p.k_stride;
    const T* v = static_cast<const T*>(p.v) + t * p.v_stride;
    // this lane's two pieces of a row
    const bool turned = lane < p.rotary_dim / 8;
    const int at = kHalf && turned ? 4 * lane : 8 * lane;
    const int gap = kHalf && turned ? p.rotary_dim / 2 : 4;
    for (int r0 = 0; r0 < rows; r0 += kRows * kWarps) {
        uint2 wa[kRows], wb[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {  // (rows past the last read it again)
            const int r = min(r0 + i * kWarps + warp, rows - 1), h = r - p.num_q_heads;
            const T* src = h < 0 ? q + r * kHeadDim
                                 : (h < p.num_kv_heads ? k + h * kHeadDim
                                                       : v + (h - p.num_kv_heads) * kHeadDim);
            wa[i] = __ldcs(reinterpret_cast<const uint2*>(src + at));
            wb[i] = __ldcs(reinterpret_cast<const uint2*>(src + at + gap));
        }
        if (r0 == 0) {
            if (tid < p.rotary_dim / 2) cs[tid] = turn_of(p, pos, tid);
            __syncthreads();
            if (slot < 0 && t >= live) return;  // padding (the whole CTA agrees)
            if (kWrite && slot >= p.num_slots && tid == 0)
                atomicOr(p.status, DFLASH_FLAG_SLOT_RANGE);
        }
        float c[4], s[4];
        if (turned) lane_turns(cs, lane, c, s);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i * kWarps + warp;
            if (r >= rows) break;
            put_row<T, kHalf, kWrite>(p, t, slot, r, at, gap, turned, wa[i], wb[i], c, s,
                                      [&](int hs) { return scale_of<kWrite>(p, hs); });
        }
    }
}

// kTokens tokens a CTA, for at most kWarps rows a token: warp w has row w of each of them.
template <typename T, bool kHalf, bool kWrite, int kTokens>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) rope_tokens_kernel(const RopeParams p) {
    __shared__ __align__(16) float2 cs[kTokens][kHeadDim / 2];
    __shared__ int64_t slots[kTokens];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rows = p.num_q_heads + p.num_kv_heads * (kWrite ? 2 : (p.k ? 1 : 0));
    const int64_t t0 = (int64_t)blockIdx.x * kTokens, last = p.num_tokens - 1;
    const bool turned = lane < p.rotary_dim / 8;
    const int at = kHalf && turned ? 4 * lane : 8 * lane;
    const int gap = kHalf && turned ? p.rotary_dim / 2 : 4;
    // (what is past the last row or token is read again and not stored)
    const int r = min(warp, rows - 1), h = r - p.num_q_heads;
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
    const float scale = scale_of<kWrite>(p, h);
    const int64_t live = live_tokens<kWrite>(p);
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
        put_row<T, kHalf, kWrite>(p, t, slot, r, at, gap, turned, wa[i], wb[i], c, s,
                                  [&](int) { return scale; });
    }
}

template <typename T, bool kHalf, bool kWrite>
cudaError_t launch_as(const RopeParams& p, cudaStream_t stream) {
    const int rows = p.num_q_heads + p.num_kv_heads * (kWrite ? 2 : (p.k ? 1 : 0));
    auto ctas = [&](int tokens) { return (unsigned)((p.num_tokens + tokens - 1) / tokens); };
    if (rows > kWarps)
        rope_kernel<T, kHalf, kWrite><<<ctas(1), kThreads, 0, stream>>>(p);
    else if (p.num_tokens <= kTokensOne)
        rope_tokens_kernel<T, kHalf, kWrite, 1><<<ctas(1), kThreads, 0, stream>>>(p);
    else if (p.num_tokens <= kTokensTwo)
        rope_tokens_kernel<T, kHalf, kWrite, 2><<<ctas(2), kThreads, 0, stream>>>(p);
    else
        rope_tokens_kernel<T, kHalf, kWrite, 4><<<ctas(4), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <bool kWrite>
cudaError_t launch(const dflash_rope_plan_t* plan, const RopeParams& p, cudaStream_t stream) {
    const bool half = plan->problem.layout == DFLASH_ROPE_HALF;
    if (plan->problem.dtype == DFLASH_FP16)
        return half ? launch_as<__half, true, kWrite>(p, stream)
                    : launch_as<__half, false, kWrite>(p, stream);
    return half ? launch_as<__nv_bfloat16, true, kWrite>(p, stream)
                : launch_as<__nv_bfloat16, false, kWrite>(p, stream);
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

double clamp01(double x) { return x < 0.0 ? 0.0 : (x > 1.0 ? 1.0 : x); }

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
    if (!distinct(outs, others) || q_out == k || (k && k_out == q))
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
    return launch<false>(plan, p, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess
               ? DFLASH_OK
               : DFLASH_ERR_CUDA;
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
    const int rc = check_plan(plan);
    if (rc != DFLASH_OK) return rc;
    const dflash_rope_problem& pr = plan->problem;
    if (num_tokens < 0 || num_tokens > kMaxTokens) return DFLASH_ERR_INVALID_ARGUMENT;
    if (num_tokens == 0) return DFLASH_OK;
    if (!rows_ok(q, q_stride, pr.num_q_heads) || !rows_ok(k, k_stride, pr.num_kv_heads) ||
        !rows_ok(v, v_stride, pr.num_kv_heads) || !rows_ok(q_out, q_out_stride, pr.num_q_heads) ||
        !positions || !aligned(positions, 4) || !slots || !aligned(slots, 8) || !phases ||
        !aligned(phases, 8) || !k_scale || !aligned(k_scale, 4) || !v_scale ||
        !aligned(v_scale, 4) || !k_pool || !aligned(k_pool, 8) || !v_pool ||
        !aligned(v_pool, 8) || !status || !aligned(status, 4) || !aligned(num_live, 4) ||
        (q == q_out && q_stride != q_out_stride))
        return DFLASH_ERR_INVALID_ARGUMENT;
    const void* const outs[] = {q_out, k_pool, v_pool, status};
    const void* const others[] = {k, v, positions, slots, phases, k_scale, v_scale, num_live};
    if (!distinct(outs, others) || k_pool == q || v_pool == q || status == q)
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
    return launch<true>(plan, p, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess
               ? DFLASH_OK
               : DFLASH_ERR_CUDA;
}

}  // extern "C"
