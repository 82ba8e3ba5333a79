// paged_tables.cu -- block-table entries, positions and cache slots of a step's new tokens, from
// request lengths (dflash_paged_step.h has the definition).
//
// One launch, no CTA waiting for another. Everything follows from two exclusive sums over the
// requests (tokens before request b, free pages taken before it); every CTA forms both in shared
// memory for itself, a few thousand lengths out of L2, and then does its share of the tokens and of
// the rows. A token's page is worked out from the inputs (held entry, prefix entry or free-list
// entry), never from an entry that another CTA may be writing. Bound by latency: the sums and two
// dependent loads, about 3 us of device time at a few requests.
#include <cuda_runtime.h>

#include "dflash_paged_step.h"

namespace dflash {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxBatch = 4096;

struct TablesParams {
    dflash_paged_tables_problem pr;
    const int32_t *cached_lens, *new_lens, *held_pages, *free_pages, *free_head, *prefix_table,
        *prefix_pages;
    int32_t *block_table, *context_lens, *held_out, *free_head_out, *token_starts, *positions;
    int64_t* slots;
    int32_t* status;
};

// One request's lengths, cut to the problem's ranges.
struct Request {
    int cached, fresh, held, need, first;  // fresh: new tokens; pages [held, first) are shared
};

__device__ Request load_request(const TablesParams& p, int b, int shared, int* flags) {
    Request r;
    const int P = p.pr.page_size, top = p.pr.max_context;
    r.cached = max(p.cached_lens[b], 0);
    const int64_t ctx = (int64_t)r.cached + max(p.new_lens[b], 0);
    if (ctx > top) *flags |= DFLASH_FLAG_CONTEXT_CLAMPED;
    r.cached = min(r.cached, top);
    r.fresh = (int)min(ctx, (int64_t)top) - r.cached;
    r.held = min(max(p.held_pages[b], 0), p.pr.max_pages_per_seq);
    const int n = r.cached + r.fresh;
    r.need = max(r.held, n / P + (n % P != 0));
    r.first = min(max(shared, r.held), r.need);
    return r;
}

__global__ void __launch_bounds__(kThreads) paged_tables_kernel(const TablesParams p) {
    // tokens and taken pages before request b (entry B: all of them)
    extern __shared__ long long sums[];
    long long* tok = sums;
    long long* take = sums + p.pr.batch + 1;
    __shared__ long long warp_tok[kThreads / 32], warp_take[kThreads / 32];
    const int B = p.pr.batch, P = p.pr.page_size, tid = threadIdx.x, lane = tid & 31;
    const int shared =
        p.prefix_pages ? min(max(*p.prefix_pages, 0), p.pr.prefix_capacity) : 0;
    const int head = max(*p.free_head, 0);
    int flags = 0;
    // thread t sums the requests [t * per, (t + 1) * per)
    const int per = (B + kThreads - 1) / kThreads, b0 = min(tid * per, B),
              b1 = min(b0 + per, B);
    long long my_tok = 0, my_take = 0;
    for (int b = b0; b < b1; ++b) {
        const Request r = load_request(p, b, shared, &flags);
        tok[b] = my_tok;
        take[b] = my_take;
        my_tok += r.fresh;
        my_take += r.need - r.first;
    }
    long long in_tok = my_tok, in_take = my_take;
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, in_tok, o),
                        c = __shfl_up_sync(0xffffffffu, in_take, o);
        if (lane >= o) {
            in_tok += a;
            in_take += c;
        }
    }
    if (lane == 31) {
        warp_tok[tid >> 5] = in_tok;
        warp_take[tid >> 5] = in_take;
    }
    __syncthreads();
    long long base_tok = in_tok - my_tok, base_take = in_take - my_take;
    for (int w = 0; w < (tid >> 5); ++w) {
        base_tok += warp_tok[w];
        base_take += warp_take[w];
    }
    for (int b = b0; b < b1; ++b) {
        tok[b] += base_tok;
        take[b] += base_take;
    }
    if (tid == kThreads - 1) {
        tok[B] = base_tok + my_tok;
        take[B] = base_take + my_take;
    }
    __syncthreads();
    const long long T = tok[B], cap = p.pr.max_tokens;
    const long long left = (long long)p.pr.num_free - head;  // pages on the free list

    // rows: a warp per request writes its outputs and its row's new entries
    const int warp = (blockIdx.x * kThreads + tid) >> 5, warps = gridDim.x * (kThreads / 32);
    for (int b = warp; b < B; b += warps) {
        const Request r = load_request(p, b, shared, &flags);
        int32_t* row = p.block_table + (int64_t)b * p.pr.max_pages_per_seq;
        for (int q = r.held + lane; q < r.need; q += 32) {
            int page;
            if (q < r.first) {
                page = p.prefix_table[q];
            } else {
                const long long k = take[b] + q - r.first;
                page = k < left ? p.free_pages[head + k] : -1;
            }
            row[q] = page;
        }
        if (lane == 0) {
            const long long got = min(max(left - take[b], 0ll), (long long)(r.need - r.first));
            p.context_lens[b] = r.cached + r.fresh;
            p.held_out[b] = r.first + (int)got;
            p.token_starts[b] = (int)min(tok[b], cap);
        }
    }
    if (blockIdx.x == 0 && tid == 0) {
        p.token_starts[B] = (int)min(T, cap);
        p.free_head_out[0] = head + (int)min(take[B], max(left, 0ll));
        if (take[B] > left) flags |= DFLASH_FLAG_PAGES_EXHAUSTED;
        if (T > cap) flags |= DFLASH_FLAG_TOKENS_DROPPED;
    }

    // tokens: the request is the last one that starts at or before the token
    for (long long t = (long long)blockIdx.x * kThreads + tid; t < cap;
         t += (long long)gridDim.x * kThreads) {
        int pos = 0;
        int64_t slot = -1;
        if (t < T) {
            int lo = 0, hi = B;  // tok[lo] <= t < tok[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (tok[mid] <= t)
                    lo = mid;
                else
                    hi = mid;
            }
            const Request r = load_request(p, lo, shared, &flags);
            pos = r.cached + (int)(t - tok[lo]);
            const int q = pos / P;
            int page = -1;
            bool missing = false;  // the free list ended before it
            if (q >= shared) {  // the shared pages are read only
                if (q < r.held) {
                    page = p.block_table[(int64_t)lo * p.pr.max_pages_per_seq + q];
                } else {  // q >= first: not held, not shared
                    const long long k = take[lo] + q - r.first;
                    missing = k >= left;
                    if (!missing) page = p.free_pages[head + k];
                }
                if (!missing && (page < 0 || page >= p.pr.num_pages)) {
                    flags |= DFLASH_FLAG_PAGE_CLAMPED;
                    page = -1;
                }
            }
            if (page >= 0) slot = (int64_t)page * P + (pos - q * P);
        }
        p.positions[t] = pos;
        p.slots[t] = slot;
    }
    if (flags) atomicOr(p.status, flags);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace
}  // namespace dflash

using namespace dflash;

extern "C" int dflash_paged_tables(const dflash_paged_tables_problem* pr,
                                   const int32_t* cached_lens, const int32_t* new_lens,
                                   const int32_t* held_pages, const int32_t* free_pages,
                                   const int32_t* free_head, const int32_t* prefix_table,
                                   const int32_t* prefix_pages, int32_t* block_table,
                                   int32_t* context_lens, int32_t* held_out,
                                   int32_t* free_head_out, int32_t* token_starts,
                                   int32_t* positions, int64_t* slots, int32_t* status,
                                   void* cuda_stream) {
    if (!pr || pr->version != DFLASH_PAGED_STEP_VERSION) return DFLASH_ERR_INVALID_ARGUMENT;
    if (pr->batch < 1 || pr->page_size < 1 || pr->max_pages_per_seq < 1 || pr->num_pages < 1 ||
        pr->max_context < 1 || pr->max_tokens < 1 || pr->num_free < 0 ||
        pr->prefix_capacity < 0 || pr->prefix_capacity > pr->max_pages_per_seq ||
        (int64_t)pr->max_pages_per_seq * pr->page_size < pr->max_context)
        return DFLASH_ERR_INVALID_ARGUMENT;
    if (pr->batch > kMaxBatch) return DFLASH_ERR_UNSUPPORTED;
    if (!cached_lens || !new_lens || !held_pages || !free_head || !block_table ||
        !context_lens || !held_out || !free_head_out || !token_starts || !positions || !slots ||
        !status || (pr->num_free > 0 && !free_pages))
        return DFLASH_ERR_INVALID_ARGUMENT;
    if ((pr->prefix_capacity > 0) != (prefix_table != nullptr) ||
        (prefix_table != nullptr) != (prefix_pages != nullptr))
        return DFLASH_ERR_INVALID_ARGUMENT;
    const void* words[] = {cached_lens, new_lens,     held_pages,   free_pages,
                           free_head,   prefix_table, prefix_pages, block_table,
                           context_lens, held_out,    free_head_out, token_starts,
                           positions,   status};
    for (const void* w : words)
        if (!aligned(w, 4)) return DFLASH_ERR_INVALID_ARGUMENT;
    if (!aligned(slots, 8)) return DFLASH_ERR_INVALID_ARGUMENT;
    // an output that is another buffer would be read, or written twice, while it is written (but the
    // table's first row may be the prefix's owner, whose entries are only read)
    const void* ins[] = {cached_lens, new_lens,     held_pages,  free_pages,
                         free_head,   prefix_table, prefix_pages};
    const void* outs[] = {context_lens, held_out, free_head_out, token_starts,
                          positions,    slots,    status,        block_table};
    for (const void*& o : outs) {
        for (const void* i : ins)
            if (o == i && !(o == block_table && i == prefix_table))
                return DFLASH_ERR_INVALID_ARGUMENT;
        for (const void** before = outs; before != &o; ++before)
            if (o == *before) return DFLASH_ERR_INVALID_ARGUMENT;
    }
    TablesParams p = {*pr,          cached_lens,  new_lens,      held_pages,   free_pages,
                      free_head,    prefix_table, prefix_pages,  block_table,  context_lens,
                      held_out,     free_head_out, token_starts, positions,    slots,
                      status};
    // a CTA per 512 tokens or 16 rows, two per SM at most
    const int64_t by_tokens = ((int64_t)pr->max_tokens + kThreads - 1) / kThreads;
    const int64_t by_rows = ((int64_t)pr->batch + kThreads / 32 - 1) / (kThreads / 32);
    int64_t grid = by_tokens > by_rows ? by_tokens : by_rows;
    if (grid > 304) grid = 304;
    const size_t smem = 2 * (size_t)(pr->batch + 1) * sizeof(long long);
    // 48 KB a launch gets without asking, the kernel's own arrays included. What is asked for is the most
    // that any batch takes: a smaller amount would be one less for a call on another thread.
    constexpr size_t kMostSmem = 2 * (size_t)(kMaxBatch + 1) * sizeof(long long);
    if (smem > 32 * 1024 &&
        cudaFuncSetAttribute(paged_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)kMostSmem) != cudaSuccess) {
        cudaGetLastError();
        return DFLASH_ERR_CUDA;
    }
    paged_tables_kernel<<<(unsigned)grid, kThreads, smem,
                          static_cast<cudaStream_t>(cuda_stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}
