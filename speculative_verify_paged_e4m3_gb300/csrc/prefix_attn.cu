// prefix_attn.cu -- attention of a batch over a shared prefix: planner, launches and combine
// (dflash_paged_step.h has the definition).
//
// Softmax attention over a set of keys splits into any disjoint parts that keep a maximum m, a sum
// l and a numerator per row: M = max m, w = 2^(m - M), out = sum w acc / sum w l. The two parts
// here are the prefix's whole pages, read once for the rows of the whole batch, and each sequence's
// own keys, for which the split kernel of the plain attention runs on the tail of its table row.
// The prefix's rows are batch * q_len * Hq / Hkv per KV head: in memory [batch, q_len, Hq, D] is
// one sequence of batch * q_len tokens, so the split kernel takes the prefix as that one sequence,
// its rows in blocks of 48 (View::kPrefix).
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include "combine_impl.cuh"
#include "common.cuh"
#include "dflash_paged_step.h"
#include "prefix_pairs.cuh"

namespace dflash {

cudaError_t launch_tc_partial(const PartialParams& p, cudaStream_t stream, View view);
int tc_max_rows();

namespace {

constexpr int kMaxBatch = 4096;
constexpr int kMinSplitKeys = 256;
constexpr int kPairsFromRows = 400;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct PrefixCombineParams {
    const float2 *own_state, *pre_state;
    const float *own_acc, *pre_acc;
    const int32_t *context_lens, *prefix_len;
    __half* out;
    float* lse;
    int batch, q_len, num_q_heads, num_kv_heads, group, rows, page_size;
    int max_context, max_prefix;
    int own_splits, own_slots;   // the suffix plan's num_splits and num_slots
    int pre_splits, pre_rows;    // prefix: splits per KV head, rows of the whole batch
    int pre_blocks, pre_pairs;   // pair kernel: row blocks per KV head, pairs of SMs (else 0)
};

constexpr int kRowCols = kHeadDim / 4;                   // 64 float4 columns per row
constexpr int kRowsPerCta = kCombineThreads / kRowCols;  // 4

// One CTA per four rows of a (sequence, KV head) unit, a thread per float4 column of a row: the
// maximum over both parts' splits, then one weighted sum, as combine_rows_kernel does it.
__global__ void __launch_bounds__(kCombineThreads)
    prefix_combine_kernel(const PrefixCombineParams p) {
    const int unit = blockIdx.x, b = unit / p.num_kv_heads, h = unit % p.num_kv_heads;
    const int r = blockIdx.y * kRowsPerCta + threadIdx.x / kRowCols;
    const int col = threadIdx.x % kRowCols;
    int unused = 0;
    const int base = p.max_prefix > 0
                         ? shared_keys(p.prefix_len, p.max_prefix, p.page_size, &unused)
                         : 0;
    const UnitSlots us = locate_slots(p.context_lens, p.batch, p.num_kv_heads, p.own_splits,
                                      p.own_slots, p.max_context, p.q_len, unit, false, base);
    if (r >= p.rows) return;  // whole warps: a row is two warps
    // own keys: slots [us.first, + own_active) of p.rows rows, this row at r
    const int own_n = us.count > 0 ? us.n : 0;
    const int own_per = own_n > 0 ? keys_per_split(own_n, us.count, 128, kMinSplitKeys) : 1;
    const int own_active = own_n > 0 ? (own_n + own_per - 1) / own_per : 0;
    // prefix: pre_active states, pre_step rows apart from pre0 on
    const int prow = b * p.rows + r;  // row of the whole batch
    int pre_active = 0, pre_step = p.pre_rows;
    int64_t pre0 = 0;
    if (base > 0 && p.pre_pairs > 0) {  // the segments of this row's block, in slots pair + unit
        const PairShare share = pair_share(base, p.pre_blocks * p.num_kv_heads, p.pre_pairs);
        const int pu = h * p.pre_blocks + prow / kPairRows;
        const int64_t t0 = (int64_t)pu * share.tiles;
        const int first = (int)(t0 / share.per_pair);
        pre_active = (int)((t0 + share.tiles - 1) / share.per_pair) - first + 1;
        pre_step = kPairRows;
        pre0 = (int64_t)(first + pu) * kPairRows + prow % kPairRows;
    } else if (base > 0) {  // slots [h * pre_splits, + pre_active) of pre_rows rows
        const int per = keys_per_split(base, p.pre_splits, 128, kMinSplitKeys);
        pre_active = (base + per - 1) / per;
        pre0 = (int64_t)h * p.pre_splits * p.pre_rows + prow;
    }
    const int64_t own0 = (int64_t)us.first * p.rows + r;
    const int total = pre_active + own_active;
    auto state_at = [&](int s) {
        return s < pre_active ? p.pre_state + pre0 + (int64_t)s * pre_step
                              : p.own_state + own0 + (int64_t)(s - pre_active) * p.rows;
    };
    auto acc_at = [&](int s) {
        const float* a = s < pre_active
                             ? p.pre_acc + (pre0 + (int64_t)s * pre_step) * kHeadDim
                             : p.own_acc + (own0 + (int64_t)(s - pre_active) * p.rows) * kHeadDim;
        return reinterpret_cast<const float4*>(a) + col;
    };
    float M = -INFINITY;
    for (int s = 0; s < total; ++s) M = fmaxf(M, __ldcg(state_at(s)).x);
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
    if (M != -INFINITY) {
        constexpr int kLoads = 8;  // splits whose loads are in flight together
        for (int s0 = 0; s0 < total; s0 += kLoads) {
            float2 st[kLoads];
            float4 a[kLoads];
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const int s = min(s0 + k, total - 1);
                st[k] = __ldcg(state_at(s));
                a[k] = __ldcg(acc_at(s));
            }
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                if (s0 + k >= total) break;
                const float w = st[k].x == -INFINITY ? 0.f : merge_ex2(st[k].x - M);
                t.x = fmaf(w, a[k].x, t.x);
                t.y = fmaf(w, a[k].y, t.y);
                t.z = fmaf(w, a[k].z, t.z);
                t.w = fmaf(w, a[k].w, t.w);
                L = fmaf(w, st[k].y, L);
            }
        }
        const float inv = 1.f / L;
        t.x *= inv;
        t.y *= inv;
        t.z *= inv;
        t.w *= inv;
    }
    const int i = r / p.group, g = r % p.group;
    const int64_t orow = ((int64_t)b * p.q_len + i) * p.num_q_heads + h * p.group + g;
    __half2* out2 = reinterpret_cast<__half2*>(p.out + orow * kHeadDim + col * 4);
    out2[0] = __floats2half2_rn(t.x, t.y);
    out2[1] = __floats2half2_rn(t.z, t.w);
    if (col == 0) p.lse[orow] = (M == -INFINITY) ? -INFINITY : (M + log2f(L)) * kLn2;
}

// The plan that a problem has; a plan handed to forward must be the same bytes.
int make_plan(const dflash_prefix_attn_problem* pr, dflash_prefix_attn_plan_t* plan) {
    if (!pr || pr->version != DFLASH_PAGED_STEP_VERSION) return DFLASH_ERR_INVALID_ARGUMENT;
    if (pr->batch < 1 || pr->max_prefix < 0 || pr->max_prefix > pr->max_context ||
        pr->flags != 0 || pr->kernel < DFLASH_PREFIX_KERNEL_AUTO ||
        pr->kernel > DFLASH_PREFIX_KERNEL_PAIRS)
        return DFLASH_ERR_INVALID_ARGUMENT;
    memset(plan, 0, sizeof(*plan));
    // the sequences' own keys: the plain attention's plan on the tensor-core kernel
    dflash_verify_attn_problem own;
    memset(&own, 0, sizeof(own));
    own.version = DFLASH_VERIFY_ATTN_VERSION;
    own.batch = pr->batch;
    own.q_len = pr->q_len;
    own.num_q_heads = pr->num_q_heads;
    own.num_kv_heads = pr->num_kv_heads;
    own.head_dim = pr->head_dim;
    own.page_size = pr->page_size;
    own.max_pages_per_seq = pr->max_pages_per_seq;
    own.num_pages = pr->num_pages;
    own.max_context = pr->max_context;
    own.device = pr->device;
    own.kernel = DFLASH_KERNEL_TCGEN05;
    const int rc = dflash_verify_attn_plan(&own, &plan->suffix);
    if (rc != DFLASH_OK) return rc;
    if (pr->batch > kMaxBatch) return DFLASH_ERR_UNSUPPORTED;
    plan->version = DFLASH_PAGED_STEP_VERSION;
    plan->sm_count = plan->suffix.sm_count;
    const int64_t rows = (int64_t)pr->batch * plan->suffix.rows;
    plan->prefix_rows = (int32_t)rows;
    const bool use_pairs = pr->kernel == DFLASH_PREFIX_KERNEL_PAIRS ||
                           (pr->kernel == DFLASH_PREFIX_KERNEL_AUTO && rows >= kPairsFromRows);
    int64_t slots;
    if (use_pairs) {
        plan->prefix_kernel = DFLASH_PREFIX_KERNEL_PAIRS;
        const int64_t blocks = ceil_div(rows, kPairRows);
        plan->prefix_row_blocks = (int32_t)blocks;
        plan->prefix_splits = plan->sm_count / 2;
        if (plan->prefix_splits < 1) return DFLASH_ERR_UNSUPPORTED;
        slots = plan->prefix_splits + blocks * pr->num_kv_heads;  // a segment's slot: pair + unit
        plan->prefix_slot_rows = kPairRows;
    } else {
        plan->prefix_kernel = DFLASH_PREFIX_KERNEL_ROWS;
        const int64_t blocks = ceil_div(rows, tc_max_rows());
        int64_t S = plan->sm_count / (blocks * pr->num_kv_heads);  // one wave
        const int64_t cap = ceil_div(pr->max_prefix, kMinSplitKeys);
        if (S > cap) S = cap;
        if (S < 1) S = 1;
        plan->prefix_row_blocks = (int32_t)blocks;
        plan->prefix_splits = (int32_t)S;
        slots = S * pr->num_kv_heads;
        plan->prefix_slot_rows = (int32_t)rows;
        if (S * blocks > 0x7FFFFFFF || pr->num_kv_heads > 65535) return DFLASH_ERR_UNSUPPORTED;
    }
    if (slots > 0x7FFFFFFF) return DFLASH_ERR_UNSUPPORTED;
    plan->prefix_slots = pr->max_prefix > 0 ? (int32_t)slots : 0;
    const size_t states = (size_t)plan->prefix_slots * plan->prefix_slot_rows;
    plan->ws_prefix_state_offset = align_up(plan->suffix.workspace_bytes, 256);
    plan->ws_prefix_acc_offset =
        plan->ws_prefix_state_offset + align_up(states * sizeof(float2), 256);
    plan->workspace_bytes = plan->ws_prefix_acc_offset + states * kHeadDim * sizeof(float);
    plan->problem = *pr;
    return DFLASH_OK;
}

}  // namespace
}  // namespace dflash

using namespace dflash;

extern "C" {

int dflash_prefix_attn_plan(const dflash_prefix_attn_problem* problem,
                            dflash_prefix_attn_plan_t* plan) {
    if (!problem || !plan) return DFLASH_ERR_INVALID_ARGUMENT;
    return make_plan(problem, plan);
}

int dflash_prefix_attn_forward(const dflash_prefix_attn_plan_t* plan, const void* q,
                               const void* k_pool, const void* v_pool, const int32_t* prefix_table,
                               const int32_t* prefix_len, const int32_t* block_table,
                               const int32_t* context_lens, const float* k_scale,
                               const float* v_scale, void* workspace, size_t workspace_bytes,
                               void* out, float* lse, void* cuda_stream) {
    if (!plan || plan->version != DFLASH_PAGED_STEP_VERSION) return DFLASH_ERR_INVALID_ARGUMENT;
    dflash_prefix_attn_plan_t made;
    const dflash_prefix_attn_problem pr = plan->problem;
    const int rc = make_plan(&pr, &made);
    if (rc != DFLASH_OK) return rc;
    if (memcmp(&made, plan, sizeof(made)) != 0) return DFLASH_ERR_INVALID_ARGUMENT;
    const bool prefix = pr.max_prefix > 0;
    if (!q || !k_pool || !v_pool || !block_table || !context_lens || !k_scale || !v_scale ||
        !workspace || !out || !lse || (prefix && (!prefix_table || !prefix_len)))
        return DFLASH_ERR_INVALID_ARGUMENT;
    if (!aligned(q, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) ||
        !aligned(workspace, 256) || !aligned(block_table, 4) || !aligned(context_lens, 4) ||
        !aligned(out, 8) || !aligned(lse, 4) || !aligned(prefix_table, 4) ||
        !aligned(prefix_len, 4) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
        return DFLASH_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < plan->workspace_bytes) return DFLASH_ERR_WORKSPACE_TOO_SMALL;
    cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    const dflash_verify_attn_plan_t& own = plan->suffix;
    char* ws = static_cast<char*>(workspace);

    PartialParams p;
    memset(&p, 0, sizeof(p));
    p.q = static_cast<const __half*>(q);
    p.k_pool = static_cast<const uint8_t*>(k_pool);
    p.v_pool = static_cast<const uint8_t*>(v_pool);
    p.context_lens = context_lens;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.status = reinterpret_cast<int32_t*>(ws);
    p.num_q_heads = pr.num_q_heads;
    p.num_kv_heads = pr.num_kv_heads;
    p.group = pr.num_q_heads / pr.num_kv_heads;
    p.page_size = pr.page_size;
    p.max_pages_per_seq = pr.max_pages_per_seq;
    p.num_pages = pr.num_pages;
    p.tile_keys = own.tile_keys;
    p.min_split_keys = own.min_split_keys;
    p.per_max = 1;  // no lookup ahead of the lengths
    p.page_shift = -1;
    for (int s = 0; s < 31; ++s)
        if (pr.page_size == (1 << s)) p.page_shift = s;
    p.max_prefix = pr.max_prefix;
    p.prefix_len = prefix_len;
    cudaError_t e = cudaSuccess;
    const bool by_pairs = plan->prefix_kernel == DFLASH_PREFIX_KERNEL_PAIRS;
    if (prefix && by_pairs) {
        PrefixPairsParams a;
        a.q = p.q;
        a.k_pool = p.k_pool;
        a.v_pool = p.v_pool;
        a.prefix_table = prefix_table;
        a.prefix_len = prefix_len;
        a.context_lens = context_lens;
        a.k_scale = k_scale;
        a.v_scale = v_scale;
        a.status = p.status;
        a.ws_state = reinterpret_cast<float2*>(ws + plan->ws_prefix_state_offset);
        a.ws_acc = reinterpret_cast<float*>(ws + plan->ws_prefix_acc_offset);
        a.rows = plan->prefix_rows;
        a.blocks = plan->prefix_row_blocks;
        a.units = a.blocks * pr.num_kv_heads;
        a.pairs = plan->prefix_splits;
        a.q_len = pr.q_len;
        a.group = p.group;
        a.num_q_heads = pr.num_q_heads;
        a.num_kv_heads = pr.num_kv_heads;
        a.page_size = pr.page_size;
        a.page_shift = p.page_shift;
        a.num_pages = pr.num_pages;
        a.max_prefix = pr.max_prefix;
        a.max_context = pr.max_context;
        e = launch_prefix_pairs(a, stream);
    } else if (prefix) {
        PartialParams a = p;
        a.block_table = prefix_table;
        a.ws_state = reinterpret_cast<float2*>(ws + plan->ws_prefix_state_offset);
        a.ws_acc = reinterpret_cast<float*>(ws + plan->ws_prefix_acc_offset);
        a.batch = 1;
        a.q_len = pr.batch * pr.q_len;
        a.batch_q_len = pr.q_len;
        a.batch_max_context = pr.max_context;
        a.rows = plan->prefix_rows;
        a.row_blocks = plan->prefix_row_blocks;
        a.block_rows = (int)ceil_div(a.rows, a.row_blocks);
        a.max_context = pr.max_prefix;
        a.num_splits = plan->prefix_splits;
        a.num_slots = plan->prefix_slots;
        e = launch_tc_partial(a, stream, View::kPrefix);
    }
    if (e == cudaSuccess) {
        p.block_table = block_table;
        p.ws_state = reinterpret_cast<float2*>(ws + own.ws_state_offset);
        p.ws_acc = reinterpret_cast<float*>(ws + own.ws_acc_offset);
        p.batch = pr.batch;
        p.q_len = pr.q_len;
        p.rows = own.rows;
        p.row_blocks = own.row_blocks;
        p.block_rows = (int)ceil_div(own.rows, own.row_blocks);
        p.max_context = pr.max_context;
        p.num_splits = own.num_splits;
        p.num_slots = own.num_slots;
        e = launch_tc_partial(p, stream, prefix ? View::kSuffix : View::kWhole);
    }
    if (e == cudaSuccess) {
        PrefixCombineParams c;
        c.own_state = reinterpret_cast<const float2*>(ws + own.ws_state_offset);
        c.own_acc = reinterpret_cast<const float*>(ws + own.ws_acc_offset);
        c.pre_state = reinterpret_cast<const float2*>(ws + plan->ws_prefix_state_offset);
        c.pre_acc = reinterpret_cast<const float*>(ws + plan->ws_prefix_acc_offset);
        c.context_lens = context_lens;
        c.prefix_len = prefix_len;
        c.out = static_cast<__half*>(out);
        c.lse = lse;
        c.batch = pr.batch;
        c.q_len = pr.q_len;
        c.num_q_heads = pr.num_q_heads;
        c.num_kv_heads = pr.num_kv_heads;
        c.group = p.group;
        c.rows = own.rows;
        c.page_size = pr.page_size;
        c.max_context = pr.max_context;
        c.max_prefix = pr.max_prefix;
        c.own_splits = own.num_splits;
        c.own_slots = own.num_slots;
        c.pre_splits = plan->prefix_splits;
        c.pre_rows = plan->prefix_rows;
        c.pre_blocks = plan->prefix_row_blocks;
        c.pre_pairs = by_pairs ? plan->prefix_splits : 0;
        const dim3 grid(pr.batch * pr.num_kv_heads, (own.rows + kRowsPerCta - 1) / kRowsPerCta);
        prefix_combine_kernel<<<grid, kCombineThreads, 0, stream>>>(c);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return DFLASH_ERR_CUDA;
    }
    return DFLASH_OK;
}

}  // extern "C"
