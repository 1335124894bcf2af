// page_tables.hip -- page tables and slot maps built from the requests'
// lengths, for MI355X (gfx950).
//
// What is computed: page i of request b is needed if it holds a position of
// [0, ctx + len) that is a sink (below `sinks`) or not in front of the first
// row's window (at or behind ctx - window + 1). A page that a row holds and
// does not need is given back (one reference less); a needed page that the row
// does not hold is taken from the same place of its parent's row (a shared
// prefix, one reference more; only pages in front of the row's new tokens, whose
// slots so never lie in another row's page; flagged if the parent lacks one) or
// is new: new pages are the lowest-numbered
// free ones (no references), dealt out in the order of requests and, within
// one, of positions. A request whose new pages, with those of all requests
// before it, are more than there are free gets none. Everything is whole
// numbers, and every sum is taken in a fixed order or is one of integers, so
// the result is a function of the arguments alone.
//
// Small tables and pools (kSmall entries each) are one workgroup's work, in one
// launch: every thread holds consecutive entries, whose places among the new pages
// and among the free ones come from two prefix sums. Others take three launches: a
// workgroup a row (pages given back and shared, new ones counted), a workgroup per
// chunk of the pool (its free pages listed) and one that sums the rows' counts,
// then the rows again (new pages, slots); a row's classification is cheaper to
// repeat than to keep. Tokens that are many for a row's workgroup take one more.
//
// What bounds them is the latency of a few trips to memory one after another: the
// small kernel 7.4 us (8 requests of 64 pages), the three others 5.5 + 4.2 + 7.5 for
// 512 requests of 1,024 pages out of 524,288, where reading table and counts once
// takes 0.7.
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
    int32_t* news;      // [B]: new pages of each request
    int32_t* before;    // [B]: of all before it
    int32_t* free;      // [chunks]: free pages of a chunk
    int32_t* list;      // [chunk][chunk_pages]: which
    Pages pages;
    int B, T, window, sinks;
    int chunks, chunk_pages;
    bool tokens_apart;  // slots and positions by a kernel of their own
};

constexpr int kSmall = 16384;       // 16 entries of each of 1,024 threads
constexpr int kEach = kSmall / 1024;
constexpr int kChunk = 4096;        // pages that a workgroup of 1,024 threads lists at a time
constexpr int kMostChunks = 1024;
constexpr int kWide = 2048;         // tokens of a request that its workgroup still writes by itself

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

// How many of its first pages the row may take from the parent's: whole pages of
// the prefix, in front of its own new tokens.
__device__ __forceinline__ int common_of(const PlanArgs& a, const Row& r, int b, int parent) {
    if (parent < 0 || r.len == 0) return 0;
    return min(max(a.prefix_lens[b], 0), r.ctx) >> a.pages.shift;
}

__device__ __forceinline__ bool in_pool(const PlanArgs& a, int page) {
    return (unsigned)page < (unsigned)a.pages.num_pages;
}

// What becomes of an entry: the page it holds, or takes from the parent's row;
// `want`: it needs a new one.
struct Entry {
    int page;
    bool want;
};

// First look at entry i of row b: pages given back and shared are counted, and what
// is shared is entered (a parent's row, which has no parent, is not).
__device__ __forceinline__ Entry classify(const PlanArgs& a, const Row& r, int32_t* row, int i, const int32_t* parent,
                                          int common) {
    const int page = row[i];
    const bool has = in_pool(a, page), need = r.need(i);
    if (page >= 0 && !has) flag(a.status, SV_FLAG_BAD_PAGE);
    if (has && !need) atomicSub(a.refs + page, 1);
    if (!need) return Entry{-1, false};
    if (has) return Entry{page, false};
    if (i >= common) return Entry{-1, true};
    const int shared = parent[i];
    if (!in_pool(a, shared)) {
        flag(a.status, SV_FLAG_NO_PREFIX);
        return Entry{-1, true};
    }
    atomicAdd(a.refs + shared, 1);
    row[i] = shared;
    return Entry{shared, false};
}

// Slot and position of token t of a request whose tokens start at `start`.
__device__ __forceinline__ void put_token(const PlanArgs& a, int b, int t, int start, int len) {
    int slot = -1, pos = -1;
    if (start >= 0 && t < len) {
        pos = start + t;
        slot = (a.pages.page(b, pos) << a.pages.shift) + (pos & ((1 << a.pages.shift) - 1));
    }
    a.slots[(size_t)b * a.T + t] = slot;
    a.positions[(size_t)b * a.T + t] = pos;
}

// Exclusive prefix sum over a workgroup of kWaves wavefronts; total: over all of it.
template <int kWaves>
__device__ __forceinline__ int exclusive(int v, int& total, int (&sums)[kWaves]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before += sums[w];
        total += sums[w];
    }
    return before + upto - v;
}

// All of a small call: B <= 1024, B max_pages and num_pages at most kSmall.
__global__ __launch_bounds__(1024) void plan_small_kernel(PlanArgs a) {
    __shared__ Row rows[1024];
    __shared__ int parents[1024], commons[1024], ends[1024];    // ends: new pages up to the end of each row
    __shared__ int sums[16];
    __shared__ uint16_t list[kSmall];               // free pages
    const int tid = threadIdx.x, width = a.pages.max_pages, all = a.B * width;
    if (tid < a.B) {
        const Row r = row_of(a, tid, true);
        rows[tid] = r;
        const int p = r.keep ? -1 : parent_of(a, tid, true);
        parents[tid] = p;
        commons[tid] = common_of(a, r, tid, p);
    }
    __syncthreads();
    // Consecutive entries of a thread.
    const int each = (all + 1023) / 1024, e0 = min(tid * each, all), n = min(each, all - e0);
    int pages[kEach], wants = 0;
    unsigned want = 0;
    {
        int b = n > 0 ? e0 / width : 0, i = e0 - b * width;
        #pragma unroll
        for (int k = 0; k < kEach; ++k) {
            if (k >= n) continue;
            const Row r = rows[b];
            int32_t* row = a.table + (size_t)b * width;
            Entry e{0, false};
            if (r.keep) {
                e.page = row[i];
            } else {
                e = classify(a, r, row, i, a.table + (size_t)max(parents[b], 0) * width, commons[b]);
            }
            pages[k] = e.page;
            want |= (unsigned)e.want << k;
            if (++i == width) {
                i = 0;
                ++b;
            }
        }
        wants = __popc(want);
    }
    __threadfence();                // the counts, before they are read
    int wanted, found;
    const int first = exclusive(wants, wanted, sums);
    {
        int at = first, b = n > 0 ? e0 / width : 0, i = e0 - b * width;
        for (int k = 0; k < n; ++k) {
            at += want >> k & 1;
            if (++i == width) {
                ends[b++] = at;
                i = 0;
            }
        }
    }
    // Free pages, consecutive ones of a thread.
    const int some = (a.pages.num_pages + 1023) / 1024, p0 = min(tid * some, a.pages.num_pages);
    unsigned free = 0;
    #pragma unroll
    for (int k = 0; k < kEach; ++k) {
        if (k < some && p0 + k < a.pages.num_pages && __hip_atomic_load(a.refs + p0 + k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) <= 0) {
            free |= 1u << k;
        }
    }
    int at = exclusive(__popc(free), found, sums);
    while (free != 0) {
        list[at++] = (uint16_t)(p0 + __builtin_ctz(free));
        free &= free - 1;
    }
    __syncthreads();
    // A request gets all of its new pages or none.
    {
        int rank = first, b = n > 0 ? e0 / width : 0, i = e0 - b * width;
        #pragma unroll
        for (int k = 0; k < kEach; ++k) {
            if (k >= n) continue;
            if (!rows[b].keep) {
                int page = pages[k];
                if (want >> k & 1) {
                    if (ends[b] <= found) {
                        page = list[rank];
                        a.refs[page] = 1;
                    }
                    ++rank;
                }
                a.table[e0 + k] = page;
            }
            if (++i == width) {
                i = 0;
                ++b;
            }
        }
    }
    __syncthreads();
    if (tid < a.B) {
        const Row r = rows[tid];
        const int news = ends[tid] - (tid > 0 ? ends[tid - 1] : 0);
        const bool granted = news == 0 || ends[tid] <= found;
        if (!granted) flag(a.status, SV_FLAG_NO_PAGES);
        a.starts[tid] = parents[tid] = granted && r.len > 0 ? r.ctx : -1;
    }
    if (a.tokens_apart) return;
    __syncthreads();
    for (int x = tid; x < a.B * a.T; x += 1024) {
        const int b = x / a.T;
        put_token(a, b, x - b * a.T, parents[b], rows[b].len);
    }
}

// A workgroup per request: pages given back and shared, new ones counted.
__global__ __launch_bounds__(256) void plan_rows_kernel(PlanArgs a) {
    __shared__ int sums[4];
    const int b = blockIdx.x;
    const Row r = row_of(a, b, threadIdx.x == 0);
    int news = 0;
    if (!r.keep) {
        const int parent = parent_of(a, b, threadIdx.x == 0), common = common_of(a, r, b, parent);
        int32_t* row = a.table + (size_t)b * a.pages.max_pages;
        const int32_t* other = a.table + (size_t)max(parent, 0) * a.pages.max_pages;
        for (int i = threadIdx.x; i < a.pages.max_pages; i += 256) news += classify(a, r, row, i, other, common).want;
    }
    int total;
    exclusive(news, total, sums);
    if (threadIdx.x == 0) a.news[b] = total;
}

// A workgroup per chunk of the pool: its free pages in order. The last one: new
// pages of all requests before each.
__global__ __launch_bounds__(1024) void plan_free_kernel(PlanArgs a) {
    __shared__ int sums[16];
    if ((int)blockIdx.x == a.chunks) {
        // More than the pool holds is as good as one more than that, and 1,024
        // counts of at most SV_MAX_CONTEXT / 32 pages stay below 2^30.
        int wanted = 0;
        for (int b0 = 0; b0 < a.B; b0 += 1024) {
            const int b = b0 + threadIdx.x;
            int total;
            const int at = exclusive(b < a.B ? a.news[b] : 0, total, sums);
            if (b < a.B) a.before[b] = min(wanted + at, a.pages.num_pages + 1);
            wanted = min(wanted + total, a.pages.num_pages + 1);
        }
        return;
    }
    const int p0 = blockIdx.x * a.chunk_pages, p1 = min(p0 + a.chunk_pages, a.pages.num_pages);
    int found = 0;
    for (int p = p0; p < p1; p += kChunk) {
        const int mine = p + 4 * threadIdx.x;
        unsigned free = 0;
        #pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (mine + k < p1 && a.refs[mine + k] <= 0) free |= 1u << k;
        }
        int total, at = exclusive(__popc(free), total, sums) + found;
        while (free != 0) {
            a.list[p0 + at++] = mine + __builtin_ctz(free);
            free &= free - 1;
        }
        found += total;
    }
    if (threadIdx.x == 0) a.free[blockIdx.x] = found;
}

// A workgroup per request: its new pages, slots and positions.
__global__ __launch_bounds__(256) void plan_slots_kernel(PlanArgs a) {
    __shared__ int sums[4], upto[kMostChunks];
    const int b = blockIdx.x;
    const Row r = row_of(a, b, false);
    const int news = a.news[b], first = a.before[b];
    bool granted = true;
    if (news > 0) {
        // Free pages up to the end of every chunk.
        int c[kMostChunks / 256], mine = 0, total;
        #pragma unroll
        for (int k = 0; k < kMostChunks / 256; ++k) {
            const int i = threadIdx.x * (kMostChunks / 256) + k;
            mine += i < a.chunks ? a.free[i] : 0;
            c[k] = mine;
        }
        const int at = exclusive(mine, total, sums);
        #pragma unroll
        for (int k = 0; k < kMostChunks / 256; ++k) upto[threadIdx.x * (kMostChunks / 256) + k] = at + c[k];
        granted = (long long)first + news <= total;
        if (!granted && threadIdx.x == 0) flag(a.status, SV_FLAG_NO_PAGES);
        __syncthreads();
    }
    int32_t* row = a.table + (size_t)b * a.pages.max_pages;
    if (!r.keep) {
        int at = first;
        for (int i0 = 0; i0 < a.pages.max_pages; i0 += 256) {
            const int i = i0 + threadIdx.x;
            const int page = i < a.pages.max_pages ? row[i] : -1;
            const bool has = in_pool(a, page), need = i < a.pages.max_pages && r.need(i);
            const bool want = need && !has && granted;
            int rank = 0;
            if (news > 0) {
                int total;
                rank = at + exclusive((int)want, total, sums);
                at += total;
            }
            if (want) {
                // The first chunk that reaches beyond this place.
                int lo = 0, hi = a.chunks - 1;
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (upto[mid] > rank) hi = mid;
                    else lo = mid + 1;
                }
                const int fresh = a.list[lo * a.chunk_pages + rank - (lo > 0 ? upto[lo - 1] : 0)];
                row[i] = fresh;
                a.refs[fresh] = 1;
            } else if (i < a.pages.max_pages && page != -1 && !(has && need)) {
                row[i] = -1;
            }
        }
    }
    const int start = granted && r.len > 0 ? r.ctx : -1;
    if (threadIdx.x == 0) a.starts[b] = start;
    if (a.tokens_apart) return;
    __syncthreads();
    for (int t = threadIdx.x; t < a.T; t += 256) put_token(a, b, t, start, r.len);
}

// 1,024 tokens of a request a workgroup.
__global__ __launch_bounds__(256) void plan_tokens_kernel(PlanArgs a) {
    const int b = blockIdx.y, start = a.starts[b];
    const Row r = row_of(a, b, false);
    #pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int t = blockIdx.x * 1024 + 256 * k + threadIdx.x;
        if (t < a.T) put_token(a, b, t, start, r.len);
    }
}

bool is_small(int B, int max_pages, int num_pages) {
    return B <= 1024 && (long long)B * max_pages <= kSmall && num_pages <= kSmall;
}

// Pages of a chunk: a multiple of what a workgroup lists at a time, few enough chunks.
int chunk_of(int num_pages) {
    const int parts = (num_pages + kChunk - 1) / kChunk;
    return (parts + kMostChunks - 1) / kMostChunks * kChunk;
}

}  // namespace

extern "C" size_t spec_verify_pages_plan_workspace_bytes(int B, int max_pages, int num_pages) {
    if (B < 1 || B > SV_MAX_BATCH || max_pages < 1 || max_pages > SV_MAX_CONTEXT / kTile || num_pages < 1) return 0;
    if (is_small(B, max_pages, num_pages)) return 256;
    return ((2 * (size_t)B + kMostChunks + num_pages) * sizeof(int32_t) + 255) / 256 * 256;
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
    a.before = a.news + B;
    a.free = a.before + B;
    a.list = a.free + kMostChunks;
    a.chunk_pages = chunk_of(num_pages);
    a.chunks = (num_pages + a.chunk_pages - 1) / a.chunk_pages;
    a.pages = make_pages(page_table, 1, page_size, max_pages, num_pages);
    a.B = B;
    a.T = T;
    a.window = window;
    a.sinks = sinks;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (is_small(B, max_pages, num_pages)) {
        a.tokens_apart = (long long)B * T > kSmall;
        hipLaunchKernelGGL(plan_small_kernel, dim3(1), dim3(1024), 0, s, a);
    } else {
        a.tokens_apart = T > kWide;
        hipLaunchKernelGGL(plan_rows_kernel, dim3((unsigned)B), dim3(256), 0, s, a);
        hipLaunchKernelGGL(plan_free_kernel, dim3((unsigned)a.chunks + 1), dim3(1024), 0, s, a);
        hipLaunchKernelGGL(plan_slots_kernel, dim3((unsigned)B), dim3(256), 0, s, a);
    }
    if (a.tokens_apart) {
        hipLaunchKernelGGL(plan_tokens_kernel, dim3((unsigned)((T + 1023) / 1024), (unsigned)B), dim3(256), 0, s, a);
    }
    return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}
