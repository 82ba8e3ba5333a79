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
constexpr int kLongOwn = 2048;
// The combine takes a CTA a row for at most so many rows of at least so many splits (768 rows of two
// splits: 15.1 us a call so, 12.6 us with a warp a row).
constexpr int kCtaPerRow = 2048, kCtaSplits = 12;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct PrefixCombineParams {
    const float2 *own_state, *pre_state;
    const float *own_acc, *pre_acc;
    const int4* unit_slots;  // of the own keys, by the split kernel (tc_partial.cu)
    const int32_t *context_lens, *prefix_len;
    __half* out;
    float* lse;
    int total_rows;  // batch * q_len * num_q_heads
    int q_len, num_q_heads, num_kv_heads, group, rows, page_size;
    int max_context, max_prefix;
    int pre_splits, pre_rows;   // prefix: splits per KV head, rows of the whole batch
    int pre_blocks, pre_pairs;  // pair kernel: row blocks per KV head, pairs of SMs (else 0)
};

constexpr int kMergeWarps = 8;

// kRowWarps warps per query row, 8 columns a lane. The row's split states are read a lane each (so that
// their loads overlap, whatever their number), the maximum and the weights follow by shuffles, and each
// warp adds its splits' numerators in split order, prefix first; the warps of a row add up in order.
// One warp a row where there are rows enough for the GPU (bound by L2, 1 KB a row and split), eight for
// few rows, which often have many splits (a warp alone took 30 us for 128 of them).
template <int kRowWarps>
__global__ void __launch_bounds__(32 * kMergeWarps)
    prefix_combine_kernel(const PrefixCombineParams p) {
    constexpr int kRowsPerCta = kMergeWarps / kRowWarps;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int orow = blockIdx.x * kRowsPerCta + warp / kRowWarps, part = warp % kRowWarps;
    if (orow >= p.total_rows) return;  // (whole rows)
    const int token = orow / p.num_q_heads, hq = orow - token * p.num_q_heads;
    const int b = token / p.q_len, h = hq / p.group;
    const int r = (token - b * p.q_len) * p.group + (hq - h * p.group);  // of its (sequence, KV head)
    int unused = 0;
    const int base = p.max_prefix > 0
                         ? shared_keys(p.prefix_len, p.max_prefix, p.page_size, &unused)
                         : 0;
    const int ctx = min(p.context_lens[b], p.max_context);
    // prefix: pre_active states, pre_step rows apart from pre0 on
    const int prow = b * p.rows + r;  // row of the whole batch
    int pre_active = 0, pre_step = p.pre_rows;
    int64_t pre0 = 0;
    if (base > 0 && p.pre_pairs > 0) {  // the segments of this row's block, in slots pair + unit
        const PairShare share = pair_share(base, p.pre_blocks * p.num_kv_heads, p.pre_pairs);
        const int pu = h * p.pre_blocks + prow / kPairRows;
        const int64_t t0 = pu * share.pitch;
        const int first = (int)(t0 / share.per_pair);
        pre_active = (int)((t0 + share.tiles - 1) / share.per_pair) - first + 1;
        pre_step = kPairRows;
        pre0 = (int64_t)(first + pu) * kPairRows + prow % kPairRows;
    } else if (base > 0) {  // slots [h * pre_splits, + pre_active) of pre_rows rows
        const int per = keys_per_split(base, p.pre_splits, 128, kMinSplitKeys);
        pre_active = (base + per - 1) / per;
        pre0 = (int64_t)h * p.pre_splits * p.pre_rows + prow;
    }
    // From here on what both kernels before this one wrote: they are complete (the split kernel waited
    // for the other). Own keys: own_active states, rows apart from own0 on.
    griddep_wait();
    int own_active = 0;
    int64_t own0 = 0;
    if (ctx > base) {
        const int4 us = __ldcg(&p.unit_slots[b * p.num_kv_heads + h]);
        const int per = keys_per_split(us.z, us.y, 128, kMinSplitKeys);
        own_active = (us.z + per - 1) / per;
        own0 = (int64_t)us.x * p.rows + r;
    }
    const int total = pre_active + own_active;
    auto state_of = [&](int s) {  // split s: past the end, no weight
        if (s >= total) return make_float2(-INFINITY, 0.f);
        return __ldcg(s < pre_active ? p.pre_state + pre0 + (int64_t)s * pre_step
                                     : p.own_state + own0 + (int64_t)(s - pre_active) * p.rows);
    };
    const float2 st0 = state_of(lane);
    float M = st0.x;
    bool lost = isnan(st0.y);
    for (int s = 32 + lane; s < total; s += 32) {
        const float2 st = state_of(s);
        M = fmaxf(M, st.x);
        lost |= isnan(st.y);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    // scores that are not numbers leave no maximum but a sum that is not one either: such a row is not
    // an empty one
    if (__any_sync(0xffffffffu, lost)) M = NAN;
    float4 t0 = make_float4(0.f, 0.f, 0.f, 0.f), t1 = t0;
    float L = 0.f;
    if (M != -INFINITY) {
        for (int s0 = 0; s0 < total; s0 += 32) {
            const float2 st = s0 == 0 ? st0 : state_of(s0 + lane);
            const float w = st.x == -INFINITY ? 0.f : merge_ex2(st.x - M);
            L = fmaf(w, st.y, L);
            const int n = min(total - s0, 32);
#pragma unroll 4
            for (int k = part; k < n; k += kRowWarps) {  // (32 is a multiple of kRowWarps)
                const int s = s0 + k;
                const float wk = __shfl_sync(0xffffffffu, w, k);
                const float* a = s < pre_active
                                     ? p.pre_acc + (pre0 + (int64_t)s * pre_step) * kHeadDim
                                     : p.own_acc +
                                           (own0 + (int64_t)(s - pre_active) * p.rows) * kHeadDim;
                const float4 a0 = __ldcg(reinterpret_cast<const float4*>(a) + lane);
                const float4 a1 = __ldcg(reinterpret_cast<const float4*>(a) + 32 + lane);
                t0.x = fmaf(wk, a0.x, t0.x);
                t0.y = fmaf(wk, a0.y, t0.y);
                t0.z = fmaf(wk, a0.z, t0.z);
                t0.w = fmaf(wk, a0.w, t0.w);
                t1.x = fmaf(wk, a1.x, t1.x);
                t1.y = fmaf(wk, a1.y, t1.y);
                t1.z = fmaf(wk, a1.z, t1.z);
                t1.w = fmaf(wk, a1.w, t1.w);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    }
    const float inv = M == -INFINITY ? 0.f : 1.f / L;
    __half2* out2 = reinterpret_cast<__half2*>(p.out + (int64_t)orow * kHeadDim);
    if constexpr (kRowWarps > 1) {
        static_assert(kRowWarps == 1 || kRowWarps == kMergeWarps, "a row is a warp or the CTA");
        __shared__ float4 sums[kMergeWarps][kHeadDim / 4];
        sums[part][lane] = t0;
        sums[part][32 + lane] = t1;
        __syncthreads();
        if (part < 2) {  // half a row each
            float4 t = sums[0][32 * part + lane];
#pragma unroll
            for (int w = 1; w < kRowWarps; ++w) {
                const float4 u = sums[w][32 * part + lane];
                t = make_float4(t.x + u.x, t.y + u.y, t.z + u.z, t.w + u.w);
            }
            out2[64 * part + 2 * lane] = __floats2half2_rn(t.x * inv, t.y * inv);
            out2[64 * part + 2 * lane + 1] = __floats2half2_rn(t.z * inv, t.w * inv);
        }
    } else {
        out2[2 * lane] = __floats2half2_rn(t0.x * inv, t0.y * inv);
        out2[2 * lane + 1] = __floats2half2_rn(t0.z * inv, t0.w * inv);
        out2[64 + 2 * lane] = __floats2half2_rn(t1.x * inv, t1.y * inv);
        out2[64 + 2 * lane + 1] = __floats2half2_rn(t1.z * inv, t1.w * inv);
    }
    if (part == 0 && lane == 0)
        p.lse[orow] = (M == -INFINITY) ? -INFINITY : (M + log2f(L)) * kLn2;
}

// Estimated times in us, over the longest prefix, for own keys half as many as the plan allows. A CTA of
// the split kernel takes 9 us and 1.3 us a 128-key tile, a pair 10 us and 1.0 us a 96-key tile (1.07 by
// itself; with 1.05 here, 32 single tokens over 65536 keys have a pair more, too few SMs are left to their own
// keys, and 79 us are 85).
constexpr double kRowsCtaUs = 9.0, kRowsTileUs = 1.3, kPairCtaUs = 10.0, kPairTileUs = 1.0;

// SM time of all sequences' own keys.
double own_sm_us(const dflash_prefix_attn_problem* pr) {
    const int64_t keys = (pr->max_context - pr->max_prefix) / 2 + pr->q_len;
    return (double)pr->batch * pr->num_kv_heads *
           (kRowsCtaUs + kRowsTileUs * (double)ceil_div(keys, 128));
}

// Key splits of the prefix in blocks of 48 rows: one wave of CTAs.
int64_t rows_splits(int64_t blocks, int sm_count, const dflash_prefix_attn_problem* pr) {
    int64_t S = sm_count / (blocks * pr->num_kv_heads);
    const int64_t cap = ceil_div(pr->max_prefix, kMinSplitKeys);
    if (S > cap) S = cap;
    return S < 1 ? 1 : S;
}

// Prefix and own keys in blocks of 48 rows. Own keys that the SMs left over have no time for start after
// the prefix, another CTA's 9 us.
double rows_us(int64_t blocks, int sm_count, const dflash_prefix_attn_problem* pr) {
    const int64_t S = rows_splits(blocks, sm_count, pr);
    int64_t per = ceil_div(pr->max_prefix, S);
    if (per < kMinSplitKeys) per = kMinSplitKeys;
    per = ceil_div(per, 128) * 128;
    const int64_t ctas = blocks * pr->num_kv_heads * ceil_div(pr->max_prefix, per);
    const int64_t keys = per < pr->max_prefix ? per : pr->max_prefix;
    double us = kRowsCtaUs + kRowsTileUs * (double)ceil_div(keys, 128);
    if (ctas > sm_count) us *= (double)ctas / sm_count;
    const double hbm = kRowsCtaUs + 0.076e-3 * pr->max_prefix * pr->num_kv_heads;
    if (us < hbm) us = hbm;
    const int64_t spare = ctas < sm_count ? sm_count - ctas : 0;
    const double left = own_sm_us(pr) - (double)spare * us;
    return left > 0 ? us + left / sm_count + kRowsCtaUs : us;
}

// SM pairs for the prefix, and the time of prefix and own keys with them. The sequences' own keys run on
// the SMs left over, from the start, and on all of them once the prefix is done, so that on an idle GPU at
// the end most of its SMs wait for the longest. The count is the one that lets both end soonest (fewer
// leave those SMs idle for a part, more run on after the prefix). The rate matters: with 1.2 us a tile in place
// of 1.0, 32 single tokens over 65536 keys take 85 us, not 79, and 16 x 8 tokens over 32768 keys 117, not
// 111.
int64_t pairs_for(int64_t blocks, int sm_count, const dflash_prefix_attn_problem* pr,
                  double* pairs_us) {
    const int64_t all = sm_count / 2;
    const int units = (int)(blocks * pr->num_kv_heads);
    const double own = own_sm_us(pr);
    int64_t best = all;
    double best_us = 0;
    for (int64_t pairs = all; pairs > 0 && pairs >= all / 2; --pairs) {
        const PairShare share = pair_share(pr->max_prefix, units, (int)pairs);
        double us = kPairCtaUs + kPairTileUs * (double)share.per_pair;
        // a share over a unit's end has a second start and epilogue
        if (share.pitch == share.tiles && share.pitch % share.per_pair != 0)
            us += kPairTileUs * kPairSwitch;
        const double left = own - (double)(sm_count - 2 * pairs) * us;
        if (left > 0) us += left / sm_count + 15.0;
        if (pairs == all || us < best_us) {
            best = pairs;
            best_us = us;
        }
    }
    if (pairs_us) *pairs_us = best_us;
    return best;
}

// Which kernel takes less time. Measured, 24/4 heads over 120000 keys: 96 rows 91 against 100 us, 144 rows
// 138 against 105, 384 rows 496 against 196; 6/1 heads over 32768 keys: 144 rows 25 against 27 us, 192 rows
// 35 against 28. Over 520 random problems the choice costs 1.4 % over the better kernel's time in the mean,
// 37 % at worst.
bool pairs_win(int64_t rows, int sm_count, const dflash_prefix_attn_problem* pr) {
    if (pr->max_prefix == 0 || sm_count < 2) return false;
    double pairs_us;
    pairs_for(ceil_div(rows, kPairRows), sm_count, pr, &pairs_us);
    return rows_us(ceil_div(rows, tc_max_rows()), sm_count, pr) > pairs_us + 1.0;
}

// The plan that a problem has; a plan handed to forward must be the same bytes. There `made` is that
// plan: its kernel and pair count, which the estimates chose (2 us of host time), are taken from it once
// they are in range, and everything else follows from them.
int make_plan(const dflash_prefix_attn_problem* pr, const dflash_prefix_attn_plan_t* made,
              dflash_prefix_attn_plan_t* plan) {
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
    // rows of the batch are counted in 32 bits from here on
    if (pr->batch > kMaxBatch ||
        (int64_t)pr->batch * pr->q_len * pr->num_q_heads > 0x7FFFFFFF / kPairRows)
        return DFLASH_ERR_UNSUPPORTED;
    // With about as many units as SMs a slot per SM leaves the longest sequences unsplit: two of
    // them per SM instead, where they may be long (40 sequences of up to 4000 keys and 4 KV heads on
    // 152 SMs: the longest 32 tiles, then 12, and 13 us less in all; for up to 1000 keys a second
    // CTA's start costs more than that, 4 us).
    if (pr->batch > 1 && pr->max_context - pr->max_prefix >= kLongOwn &&
        2 * (int64_t)pr->batch * pr->num_kv_heads > plan->suffix.sm_count) {
        dflash_verify_attn_plan_t& sp = plan->suffix;
        const int64_t most =
            (int64_t)pr->batch * pr->num_kv_heads * ceil_div(pr->max_context, kMinSplitKeys);
        int64_t slots = 2 * (int64_t)sp.sm_count / sp.row_blocks;
        if (slots > most) slots = most;
        if (slots > sp.num_slots) sp.num_slots = (int32_t)slots;
        sp.ws_acc_offset =
            sp.ws_state_offset + align_up((size_t)sp.num_slots * sp.rows * sizeof(float2), 256);
        sp.workspace_bytes =
            sp.ws_acc_offset + (size_t)sp.num_slots * sp.rows * kHeadDim * sizeof(float);
    }
    plan->version = DFLASH_PAGED_STEP_VERSION;
    plan->sm_count = plan->suffix.sm_count;
    const int64_t rows = (int64_t)pr->batch * plan->suffix.rows;
    plan->prefix_rows = (int32_t)rows;
    if (made && ((made->prefix_kernel != DFLASH_PREFIX_KERNEL_ROWS &&
                  made->prefix_kernel != DFLASH_PREFIX_KERNEL_PAIRS) ||
                 (pr->kernel != DFLASH_PREFIX_KERNEL_AUTO && made->prefix_kernel != pr->kernel) ||
                 made->prefix_splits < 1 ||
                 (made->prefix_kernel == DFLASH_PREFIX_KERNEL_PAIRS &&
                  made->prefix_splits > plan->sm_count / 2)))
        return DFLASH_ERR_INVALID_ARGUMENT;
    const bool use_pairs = made ? made->prefix_kernel == DFLASH_PREFIX_KERNEL_PAIRS
                                : pr->kernel == DFLASH_PREFIX_KERNEL_PAIRS ||
                                      (pr->kernel == DFLASH_PREFIX_KERNEL_AUTO &&
                                       pairs_win(rows, plan->sm_count, pr));
    int64_t slots;
    if (use_pairs) {
        plan->prefix_kernel = DFLASH_PREFIX_KERNEL_PAIRS;
        const int64_t blocks = ceil_div(rows, kPairRows);
        plan->prefix_row_blocks = (int32_t)blocks;
        plan->prefix_splits =
            made ? made->prefix_splits
                 : (int32_t)pairs_for(blocks, plan->sm_count, pr, nullptr);
        if (plan->prefix_splits < 1) return DFLASH_ERR_UNSUPPORTED;
        slots = plan->prefix_splits + blocks * pr->num_kv_heads;  // a segment's slot: pair + unit
        plan->prefix_slot_rows = kPairRows;
    } else {
        plan->prefix_kernel = DFLASH_PREFIX_KERNEL_ROWS;
        const int64_t blocks = ceil_div(rows, tc_max_rows());
        const int64_t S = rows_splits(blocks, plan->sm_count, pr);
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
    plan->ws_unit_offset = plan->ws_prefix_acc_offset + states * kHeadDim * sizeof(float);
    plan->workspace_bytes =
        plan->ws_unit_offset + (size_t)pr->batch * pr->num_kv_heads * sizeof(int4);
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
    return make_plan(problem, nullptr, plan);
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
    const int rc = make_plan(&pr, plan, &made);
    if (rc != DFLASH_OK) return rc;
    if (memcmp(&made, plan, sizeof(made)) != 0) return DFLASH_ERR_INVALID_ARGUMENT;
    const bool prefix = pr.max_prefix > 0;
    if (!q || !k_pool || !v_pool || !block_table || !context_lens || !k_scale || !v_scale ||
        !workspace || !out || !lse || (prefix && !prefix_len) ||
        (!prefix_table && pr.max_prefix >= pr.page_size))  // (a shorter prefix has no whole page)
        return DFLASH_ERR_INVALID_ARGUMENT;
    if (!aligned(q, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) ||
        !aligned(workspace, 256) || !aligned(block_table, 4) || !aligned(context_lens, 4) ||
        !aligned(out, 8) || !aligned(lse, 4) || !aligned(prefix_table, 4) ||
        !aligned(prefix_len, 4) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
        return DFLASH_ERR_INVALID_ARGUMENT;
    // an output or the workspace that is another buffer would be read while it is written
    const void* ins[] = {q,          k_pool,      v_pool,       prefix_table, prefix_len,
                         block_table, context_lens, k_scale,    v_scale};
    const void* outs[] = {out, lse, workspace};
    for (const void* o : outs)
        for (const void* i : ins)
            if (o == i) return DFLASH_ERR_INVALID_ARGUMENT;
    if (out == lse || out == workspace || lse == workspace) return DFLASH_ERR_INVALID_ARGUMENT;
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
    p.prefix_len = prefix ? prefix_len : nullptr;
    p.unit_slots = reinterpret_cast<int4*>(ws + plan->ws_unit_offset);
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
        // It needs nothing of the prefix kernel and so may start beside its last CTAs (that kernel, an
        // ordinary launch, has itself waited for everything before this call).
        p.pdl = prefix ? 1 : 0;
        e = launch_tc_partial(p, stream, View::kSuffix);
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
        c.unit_slots = p.unit_slots;
        c.total_rows = pr.batch * pr.q_len * pr.num_q_heads;
        c.q_len = pr.q_len;
        c.num_q_heads = pr.num_q_heads;
        c.num_kv_heads = pr.num_kv_heads;
        c.group = p.group;
        c.rows = own.rows;
        c.page_size = pr.page_size;
        c.max_context = pr.max_context;
        c.max_prefix = pr.max_prefix;
        c.pre_splits = plan->prefix_splits;
        c.pre_rows = plan->prefix_rows;
        c.pre_blocks = plan->prefix_row_blocks;
        c.pre_pairs = by_pairs ? plan->prefix_splits : 0;
        cudaLaunchConfig_t cfg = {};
        // a CTA a row where a row has many splits and there are few rows
        const int units = pr.batch * pr.num_kv_heads;
        const int pre_each = !prefix    ? 0
                             : by_pairs ? plan->prefix_splits / (c.pre_blocks * pr.num_kv_heads) + 1
                                        : plan->prefix_splits;
        const bool few = c.total_rows <= kCtaPerRow &&
                         pre_each + (own.num_slots + units - 1) / units >= kCtaSplits;
        cfg.gridDim = dim3(few ? c.total_rows : (c.total_rows + kMergeWarps - 1) / kMergeWarps);
        cfg.blockDim = dim3(32 * kMergeWarps);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(
            &cfg, few ? prefix_combine_kernel<kMergeWarps> : prefix_combine_kernel<1>, c);
    }
    if (e == cudaSuccess) {
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return DFLASH_ERR_CUDA;
    }
    return DFLASH_OK;
}

}  // extern "C"
