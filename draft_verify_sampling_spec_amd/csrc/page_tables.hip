// page_tables.hip -- page tables and slot maps built from the requests'
// lengths, for MI355X (gfx950).
//
// What is computed: page i of request b is needed if it holds a position of
// [0, ctx + len) that is a sink (below `sinks`) or not in front of the first
// row's window (at or behind ctx - window + 1). A page that a row holds and
// does not need is given back (one reference less); a needed page that the row
// does not hold is taken from the same place of its parent's row (a shared
// prefix, one reference more) or is new: new pages are the lowest-numbered
// free ones (no references), dealt out in the order of requests and, within
// one, of positions. A request whose new pages, with those of all requests
// before it, are more than there are free gets none. Everything is whole
// numbers, and every sum is taken in a fixed order or is one of integers, so
// the result is a function of the arguments alone.
//
// Three launches: the rows' own part (counts given back and shared, new pages
// counted), one workgroup that sums the counts and lists the free pages that are
// wanted, and the rows again (new pages, slots). A row's classification is
// cheaper to repeat than to keep.
#include <algorithm>
#include <initializer_list>

#include "cache_tile.h"

namespace {

using namespace svcache;

struct PlanArgs {
    int32_t* table;
    int32_t* refs;
    const int32_t* ctx_lens;
    const int32_t* budgets;
    const int32_t* parents;
    const int32_t* prefix_lens;
    int32_t* starts;
    int32_t* slots;
    int32_t* positions;
    int32_t* status;
    int32_t* news;      // [2 B + 1]: new pages of each request, those of all before it, free pages found
    int32_t* free_list; // the wanted free pages
    Pages pages;
    int B, T, window, sinks;
};

// What a request's row needs: pages [0, sink_end) and [first, end).
struct Row {
    int ctx, len;           // len 0: no tokens
    int sink_end, first, end;
    bool keep;              // it does not fit: the row stays as it is
    __device__ __forceinline__ bool need(int i) const { return i < end && (i >= first || i < sink_end); }
};

__device__ __forceinline__ Row row_of(const PlanArgs& a, int b, bool report) {
    const int ctx = a.ctx_lens[b];
    const Block blk = block_of(a.ctx_lens, a.budgets, b, a.T, a.pages, a.status, report);
    Row r{blk.ctx, blk.len, 0, 0, 0, ctx >= 0 && blk.len == 0};
    if (blk.len > 0) {
        const int size = 1 << a.pages.shift;
        r.end = (blk.ctx + blk.len + size - 1) >> a.pages.shift;
        if (a.window > 0) {
            r.first = max(0, blk.ctx - a.window + 1) >> a.pages.shift;
            r.sink_end = (int)(((long long)a.sinks + size - 1) >> a.pages.shift);
        }
    }
    return r;
}

// The row's parent, or -1. A parent's row must not change in this call other
// than by losing pages, so a parent has none itself.
__device__ __forceinline__ int parent_of(const PlanArgs& a, int b, bool report) {
    if (!a.parents) return -1;
    const int p = a.parents[b];
    if (p < 0) return -1;
    if (p >= a.B || p == b || a.parents[p] >= 0) {
        if (report) flag(a.status, SV_FLAG_BAD_PARENT);
        return -1;
    }
    return p;
}

__device__ __forceinline__ bool in_pool(const PlanArgs& a, int page) {
    return (unsigned)page < (unsigned)a.pages.num_pages;
}

// Sum over a workgroup of 256 threads, known to all.
__device__ __forceinline__ int block_sum(int v, int* sh) {
    #pragma unroll
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    return sh[0] + sh[1] + sh[2] + sh[3];
}

// A workgroup per request: pages given back and shared, new ones counted.
__global__ __launch_bounds__(256) void plan_rows_kernel(PlanArgs a) {
    __shared__ int sh[4];
    const int b = blockIdx.x;
    const Row r = row_of(a, b, threadIdx.x == 0);
    int news = 0;
    if (!r.keep) {
        const int parent = parent_of(a, b, threadIdx.x == 0);
        const int common = parent >= 0 && r.len > 0 ? max(a.prefix_lens[b], 0) >> a.pages.shift : 0;
        int32_t* row = a.table + (size_t)b * a.pages.max_pages;
        const int32_t* other = a.table + (size_t)max(parent, 0) * a.pages.max_pages;
        for (int i = threadIdx.x; i < a.pages.max_pages; i += 256) {
            const int page = row[i];
            const bool has = in_pool(a, page), need = r.need(i);
            if (page >= 0 && !has) flag(a.status, SV_FLAG_BAD_PAGE);
            if (has && !need) atomicSub(a.refs + page, 1);
            if (need && !has) {
                const int shared = i < common ? other[i] : -1;
                if (in_pool(a, shared)) {
                    atomicAdd(a.refs + shared, 1);
                    row[i] = shared;
                } else {
                    ++news;
                }
            }
        }
    }
    news = block_sum(news, sh);
    if (threadIdx.x == 0) a.news[b] = news;
}

// One workgroup: the first new page of every request, and the free pages.
__global__ __launch_bounds__(1024) void plan_free_kernel(PlanArgs a) {
    __shared__ int sums[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // Exclusive sum over the workgroup; total: over all of it. 1,024 counts of at
    // most SV_MAX_CONTEXT / 32 pages stay below 2^30.
    auto exclusive = [&](int v, int& total) {
        int upto = v;
        #pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int u = __shfl_up(upto, o);
            if (lane >= o) upto += u;
        }
        __syncthreads();
        if (lane == 63) sums[wave] = upto;
        __syncthreads();
        int before = 0;
        total = 0;
        #pragma unroll
        for (int w = 0; w < 16; ++w) {
            if (w < wave) before += sums[w];
            total += sums[w];
        }
        return before + upto - v;
    };
    // More than the pool holds is as good as one more than that.
    const int most = a.pages.num_pages;
    int wanted = 0;
    for (int b0 = 0; b0 < a.B; b0 += 1024) {
        const int b = b0 + threadIdx.x;
        int total;
        const int at = exclusive(b < a.B ? a.news[b] : 0, total);
        if (b < a.B) a.news[a.B + b] = min(wanted + at, most + 1);
        wanted = min(wanted + total, most + 1);
    }
    const int list = min(wanted, most);
    int found = 0;
    for (int p0 = 0; p0 < most && found < list; p0 += 1024) {
        const int p = p0 + threadIdx.x;
        const bool free = p < most && a.refs[p] <= 0;
        int total;
        const int at = found + exclusive(free ? 1 : 0, total);
        if (free && at < list) a.free_list[at] = p;
        found += total;
    }
    if (threadIdx.x == 0) a.news[2 * a.B] = min(found, list);
}

__global__ __launch_bounds__(256) void plan_slots_kernel(PlanArgs a) {
    __shared__ int sums[4];
    const int b = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Row r = row_of(a, b, false);
    const int news = a.news[b], first = a.news[a.B + b];
    const bool granted = news == 0 || (long long)first + news <= a.news[2 * a.B];
    if (!granted && threadIdx.x == 0) flag(a.status, SV_FLAG_NO_PAGES);
    int32_t* row = a.table + (size_t)b * a.pages.max_pages;
    if (!r.keep) {
        int at = first;
        for (int i0 = 0; i0 < a.pages.max_pages; i0 += 256) {
            const int i = i0 + threadIdx.x;
            const int page = i < a.pages.max_pages ? row[i] : -1;
            const bool has = in_pool(a, page), need = i < a.pages.max_pages && r.need(i);
            const bool want = need && !has && granted;
            const unsigned long long who = __ballot(want);
            __syncthreads();
            if (lane == 0) sums[wave] = __popcll(who);
            __syncthreads();
            int mine = at + __popcll(who & ((1ull << lane) - 1));
            #pragma unroll
            for (int w = 0; w < 4; ++w) {
                if (w < wave) mine += sums[w];
                at += sums[w];
            }
            if (want) {
                const int fresh = a.free_list[mine];
                row[i] = fresh;
                a.refs[fresh] = 1;
            } else if (i < a.pages.max_pages && page != -1 && !(has && need)) {
                row[i] = -1;
            }
        }
    }
    __syncthreads();
    const bool live = granted && r.len > 0;
    if (threadIdx.x == 0) a.starts[b] = live ? r.ctx : -1;
    for (int t = threadIdx.x; t < a.T; t += 256) {
        int slot = -1, pos = -1;
        if (live && t < r.len) {
            pos = r.ctx + t;
            slot = (row[pos >> a.pages.shift] << a.pages.shift) + (pos & ((1 << a.pages.shift) - 1));
        }
        a.slots[(size_t)b * a.T + t] = slot;
        a.positions[(size_t)b * a.T + t] = pos;
    }
}

}  // namespace

extern "C" size_t spec_verify_pages_plan_workspace_bytes(int B, int max_pages, int num_pages) {
    if (B < 1 || B > SV_MAX_BATCH || max_pages < 1 || max_pages > SV_MAX_CONTEXT / kTile || num_pages < 1) return 0;
    const size_t list = std::min((size_t)num_pages, (size_t)B * max_pages);
    return ((2 * (size_t)B + 1 + list) * sizeof(int32_t) + 255) / 256 * 256;
}

extern "C" int spec_verify_pages_plan(int32_t* page_table, int32_t* page_refs, const int32_t* ctx_lens,
                                      const int32_t* budgets, const int32_t* parents,
                                      const int32_t* prefix_lens, int B, int T, int page_size,
                                      int max_pages, int num_pages, int window, int sinks,
                                      int32_t* out_starts, int32_t* out_slots,
                                      int32_t* out_positions, int32_t* out_status, void* workspace,
                                      size_t workspace_bytes, void* stream) {
    if (B < 0 || B > SV_MAX_BATCH || T < 1 || T > SV_MAX_CONTEXT || window < 0 || sinks < 0 ||
        !geometry_ok(1, 64, page_size, max_pages, num_pages) ||
        (long long)num_pages * page_size > 0x7fffffffll) {
        return SV_ERR_ARG;
    }
    if (B == 0) return SV_OK;
    if (!page_table || !page_refs || !ctx_lens || !out_starts || !out_slots || !out_positions ||
        !workspace || (parents && !prefix_lens)) {
        return SV_ERR_NULL;
    }
    for (const void* p : {(const void*)page_table, (const void*)page_refs, (const void*)ctx_lens,
                          (const void*)budgets, (const void*)parents, (const void*)prefix_lens,
                          (const void*)out_starts, (const void*)out_slots,
                          (const void*)out_positions, (const void*)out_status}) {
        if (!aligned(p, 4)) return SV_ERR_ALIGN;
    }
    if (!aligned(workspace, 256)) return SV_ERR_ALIGN;
    if (workspace_bytes < spec_verify_pages_plan_workspace_bytes(B, max_pages, num_pages)) {
        return SV_ERR_ARG;
    }
    PlanArgs a{};
    a.table = page_table;
    a.refs = page_refs;
    a.ctx_lens = ctx_lens;
    a.budgets = budgets;
    a.parents = parents;
    a.prefix_lens = prefix_lens;
    a.starts = out_starts;
    a.slots = out_slots;
    a.positions = out_positions;
    a.status = out_status;
    a.news = static_cast<int32_t*>(workspace);
    a.free_list = a.news + 2 * (size_t)B + 1;
    a.pages = make_pages(page_table, 1, page_size, max_pages, num_pages);
    a.B = B;
    a.T = T;
    a.window = window;
    a.sinks = sinks;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipLaunchKernelGGL(plan_rows_kernel, dim3((unsigned)B), dim3(256), 0, s, a);
    hipLaunchKernelGGL(plan_free_kernel, dim3(1), dim3(1024), 0, s, a);
    hipLaunchKernelGGL(plan_slots_kernel, dim3((unsigned)B), dim3(256), 0, s, a);
    return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}
