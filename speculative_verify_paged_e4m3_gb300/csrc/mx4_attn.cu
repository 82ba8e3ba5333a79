// mx4_attn.cu -- attention of drafted tokens over the 4-bit cache (dflash_mx4_attn_*): the partial kernel and
// its entry points. Splits, slots, split state and combine are those of the E4M3 attention.
//
// CUDA-core kernel: one CTA per (split, KV head, sequence) and block of up to 48 rows, 32 keys at a time, all in
// FP32.
#include <cuda_runtime.h>
#include <math.h>

#include "common.cuh"
#include "dflash_mx4_cache.h"
#include "mx4.cuh"

namespace dflash {
int check_attn_plan(const dflash_verify_attn_plan_t* plan);
PartialParams attn_params(const dflash_verify_attn_plan_t* plan, const void* q, const void* k_pool,
                          const void* v_pool, const int32_t* block_table,
                          const int32_t* context_lens, const float* k_scale, const float* v_scale,
                          void* workspace);
CombineParams combine_params(const dflash_verify_attn_plan_t* plan, const void* workspace,
                             const int32_t* context_lens, void* out, float* lse);
cudaError_t launch_combine(const CombineParams& p, cudaStream_t stream);

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 48;
constexpr int kTile = 32;
constexpr int kKStride = kHeadDim + 1;
constexpr int kPStride = kTile + 1;
constexpr size_t kSmem =
    sizeof(float) * (kRows * kHeadDim + kTile * kKStride + kTile * kHeadDim + kRows * kPStride + kRows);

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float code_number(uint32_t code) {
    const uint32_t h = mx4::codes_to_f16x2<0>(code & 15u);
    return __half2float(__ushort_as_half((unsigned short)(h & 0xFFFFu)));
}

__global__ void __launch_bounds__(kThreads, 1) mx4_partial_kernel(PartialParams p) {
    extern __shared__ float smem[];
    float* Qs = smem;
    float* Ks = Qs + kRows * kHeadDim;
    float* Vs = Ks + kTile * kKStride;
    float* Ps = Vs + kTile * kHeadDim;
    float* alpha_s = Ps + kRows * kPStride;
    __shared__ float key_nan[kTile];  // NaN where a scale of V is
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_launch_dependents();
    const RowBlock rb = row_block(p);
    const int G = p.group, R = rb.rows, row_lo = rb.row_lo, slot = rb.slot;
    const UnitSlots us = locate_slots(p.context_lens, p.batch, p.num_kv_heads, p.num_splits,
                                      p.num_slots, p.max_context, p.q_len, slot, true);
    if (slot == 0 && tid == 0 && us.flags) atomicOr(p.status, us.flags);
    const int b = us.b, h = us.h, split = slot - us.first, n = us.n;
    if (b < 0) return;
    const int per = keys_per_split(n, us.count, p.tile_keys, p.min_split_keys);
    const int start = split * per;
    if (start >= n) return;
    const int end = min(n, start + per);
    griddep_wait();
    for (int idx = tid; idx < kRows * kHeadDim; idx += kThreads) {
        const int r = idx / kHeadDim, d = idx % kHeadDim;
        float v = 0.f;
        if (r < R) {
            const int i = (row_lo + r) / G, g = (row_lo + r) % G;
            const int64_t qrow = ((int64_t)b * p.q_len + i) * p.num_q_heads + h * G + g;
            v = __half2float(p.q[qrow * kHeadDim + d]) * (0.0625f * kLog2e);
            if (fabsf(v) == INFINITY) v = NAN;
        }
        Qs[idx] = v;
    }
    float m_run[kRows / 8], l_run[kRows / 8], acc[kRows];
#pragma unroll
    for (int m = 0; m < kRows / 8; ++m) {
        m_run[m] = -INFINITY;
        l_run[m] = 0.f;
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) acc[r] = 0.f;
    bool page_clamped = false;
    for (int t0 = start; t0 < end; t0 += kTile) {
        __syncthreads();
        {
            const int kk = tid >> 3, part = tid & 7, j = t0 + kk;
            if (part == 0) key_nan[kk] = 0.f;
            __syncwarp();
            if (j < end) {
                const int phys = physical_page(p.block_table, b, p.max_pages_per_seq,
                                               j / p.page_size, p.num_pages, &page_clamped);
                const int64_t s = (int64_t)phys * p.page_size + j % p.page_size;
                const int64_t at = mx4::chunk_offset(s, p.num_kv_heads, h);
                const int tok = (int)(s % mx4::kTokens);
                const int scale = mx4::kCodeBytes + tok * mx4::kBlocks + part;
                const float kp = mx4::power_of_scale(p.k_pool[at + scale]);
                float vp = mx4::power_of_scale(p.v_pool[at + scale]);
                if (vp != vp) {
                    key_nan[kk] = NAN;
                    vp = 0.f;
                }
                for (int e = 0; e < 32; ++e) {
                    const int d = part * 32 + e;
                    const uint32_t kc = p.k_pool[at + part * 256 + tok * 16 + e / 2];
                    const uint32_t vc = p.v_pool[at + (d % 128) * 16 + tok];
                    Ks[kk * kKStride + d] = code_number(kc >> (4 * (e & 1))) * kp;
                    Vs[kk * kHeadDim + d] = code_number(vc >> (4 * (d / 128))) * vp;
                }
            } else {
                for (int e = 0; e < 32; ++e)
                    Ks[kk * kKStride + part * 32 + e] = Vs[kk * kHeadDim + part * 32 + e] = 0.f;
            }
        }
        __syncthreads();
        float s[kRows / 8];
#pragma unroll
        for (int m = 0; m < kRows / 8; ++m) s[m] = key_nan[lane];
        for (int d = 0; d < kHeadDim; ++d) {
            const float kv = Ks[lane * kKStride + d];
#pragma unroll
            for (int m = 0; m < kRows / 8; ++m)
                s[m] = fmaf(Qs[(warp + 8 * m) * kHeadDim + d], kv, s[m]);
        }
        const int j = t0 + lane;
#pragma unroll
        for (int m = 0; m < kRows / 8; ++m) {
            const int r = warp + 8 * m;
            const bool valid = r < R && j < end && j <= n - p.q_len + (row_lo + r) / G;
            const float sv = valid ? s[m] : -INFINITY;
            const float mn = fmaxf(m_run[m], warp_max(sv));
            float pj = 0.f, alpha = 1.f;
            if (mn != -INFINITY) {
                pj = valid ? exp2f(sv - mn) : 0.f;
                alpha = exp2f(m_run[m] - mn);
            } else if (valid && sv != sv) {
                pj = NAN;
            }
            l_run[m] = l_run[m] * alpha + warp_sum(pj);
            m_run[m] = mn;
            Ps[r * kPStride + lane] = pj;
            if (lane == 0) alpha_s[r] = alpha;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kRows; ++r) acc[r] *= alpha_s[r];
        for (int kk = 0; kk < kTile; ++kk) {
            const float v = Vs[kk * kHeadDim + tid];
#pragma unroll
            for (int r = 0; r < kRows; ++r) acc[r] = fmaf(Ps[r * kPStride + kk], v, acc[r]);
        }
    }
    if (page_clamped) atomicOr(p.status, DFLASH_FLAG_PAGE_CLAMPED);
#pragma unroll
    for (int m = 0; m < kRows / 8; ++m) {
        const int r = warp + 8 * m;
        // (a row of NaN is not an empty one)
        const float mx = l_run[m] != l_run[m] ? INFINITY : m_run[m];
        if (r < R && lane == 0)
            p.ws_state[(int64_t)slot * p.rows + row_lo + r] = make_float2(mx, l_run[m]);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
        if (r < R) p.ws_acc[((int64_t)slot * p.rows + row_lo + r) * kHeadDim + tid] = acc[r];
}

cudaError_t launch_partial(const PartialParams& p, cudaStream_t stream) {
    if (!row_blocks_valid(p, kRows)) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(mx4_partial_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = partial_grid(p);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    if (p.pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, mx4_partial_kernel, p);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The plan as the split and combine rules of the E4M3 kernel see it (the same tile and row blocks).
dflash_verify_attn_plan_t as_split_plan(const dflash_verify_attn_plan_t& plan) {
    dflash_verify_attn_plan_t p = plan;
    p.kernel = DFLASH_KERNEL_TCGEN05;
    return p;
}

}  // namespace
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
    plan->threads = kThreads;
    plan->smem_bytes = (int32_t)kSmem;
    plan->problem = *problem;
    return DFLASH_OK;
}

int dflash_mx4_attn_forward(const dflash_verify_attn_plan_t* plan, const void* q,
                            const void* k_pool, const void* v_pool, const int32_t* block_table,
                            const int32_t* context_lens, void* workspace, size_t workspace_bytes,
                            void* out, float* lse, void* cuda_stream) {
    if (!plan || plan->kernel != DFLASH_KERNEL_MX4) return DFLASH_ERR_INVALID_ARGUMENT;
    const dflash_verify_attn_plan_t split = as_split_plan(*plan);
    const int rc = check_attn_plan(&split);
    if (rc != DFLASH_OK) return rc;
    if (!q || !k_pool || !v_pool || !block_table || !context_lens || !workspace || !out || !lse)
        return DFLASH_ERR_INVALID_ARGUMENT;
    if (!aligned(q, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) ||
        !aligned(workspace, 256) || !aligned(block_table, 4) || !aligned(context_lens, 4) ||
        !aligned(out, 8) || !aligned(lse, 4))
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
    const PartialParams p = attn_params(&split, q, k_pool, v_pool, block_table, context_lens,
                                        nullptr, nullptr, workspace);
    CombineParams c = combine_params(&split, workspace, context_lens, out, lse);
    c.pdl = 1;  // it waits for the partial kernel where it reads the split state
    cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    if (launch_partial(p, stream) != cudaSuccess || launch_combine(c, stream) != cudaSuccess) {
        cudaGetLastError();
        return DFLASH_ERR_CUDA;
    }
    return DFLASH_OK;
}

}  // extern "C"
