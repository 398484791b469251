// Page tables, slot map and positions of a batch built on the GPU from its request lengths.
#include <cstdint>

#include <cuda_runtime.h>

#include "nanoflow.h"
#include "nf_internal.h"
#include "nf_kv4.h"

namespace nf {
namespace {

constexpr int kMapThreads = 1024;
constexpr size_t kMapScratch = sizeof(int64_t) * kMapThreads / 32;  // static shared memory

struct PageMapArgs {
    const int *ctx_len, *new_len;
    int R;
    int* table;
    int stride;
    const int* free_pages;
    int free_cap;
    const int* free_count;
    int num_pages;
    int *kv_len, *indptr, *indices;
    int page_cap;
    int *slots, *positions;
    int token_cap;
    int* free_left;
    int* status;
};

struct Span {  // n words from p
    const int* p;
    int64_t n;
    bool meets(const Span& b) const {
        return n > 0 && b.n > 0 && reinterpret_cast<uintptr_t>(p) < reinterpret_cast<uintptr_t>(b.p) + 4 * b.n &&
               reinterpret_cast<uintptr_t>(b.p) < reinterpret_cast<uintptr_t>(p) + 4 * n;
    }
};

struct Need {
    int ctx, fresh;  // cached tokens, new tokens
    int before;      // pages of the cached tokens
    int take;        // pages the new tokens add (0 when refused)
    bool dead, wide; // cached tokens do not fit the table row; the new ones do not
    bool bad;        // a negative length
};

__device__ __forceinline__ Need need_of(const PageMapArgs& a, int r) {
    Need n;
    const int c = a.ctx_len[r], f = a.new_len ? a.new_len[r] : 1;
    n.bad = c < 0 || f < 0;
    n.ctx = n.bad ? 0 : c;
    n.fresh = n.bad ? 0 : f;
    n.before = (int)(((int64_t)n.ctx + kKv4Slots - 1) / kKv4Slots);
    const int after = (int)(((int64_t)n.ctx + n.fresh + kKv4Slots - 1) / kKv4Slots);
    n.dead = n.before > a.stride;
    n.wide = after > a.stride || (int64_t)n.ctx + n.fresh > 0x7fffffff;
    n.take = n.dead || n.wide ? 0 : after - n.before;
    return n;
}

// Exclusive prefix over the block of one int64 per thread; *total gets the sum.
__device__ __forceinline__ int64_t block_prefix(int64_t x, int64_t* scratch, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    if (lane == 31) scratch[warp] = s;
    __syncthreads();
    if (warp == 0) {
        int64_t w = scratch[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        scratch[lane] = w;
    }
    __syncthreads();
    const int64_t before = (warp ? scratch[warp - 1] : 0) + s - x;
    *total = scratch[31];
    __syncthreads();
    return before;
}

// Largest r with off[r] <= e (off ascending, off[0] = 0, e < off[R]).
__device__ __forceinline__ int row_of(const int* off, int R, int e) {
    int lo = 0, hi = R;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= e) lo = mid; else hi = mid;
    }
    return lo;
}

// With b = ceil(ctx / 16) and a = ceil((ctx + new) / 16) pages of a request before and after, the k-th new
// page of the batch, in request order, is free_pages[count - 1 - k]. Every CTA scans all R lengths itself
// (a thread takes R / 1024 consecutive requests; four block scans of three barriers each, of the pages asked for and,
// once it is known who gets them, of pages, tokens and pages taken) and keeps the offsets in shared memory, so no CTA
// waits for another; the output entries, one per page and one per token, are dealt evenly over all CTAs, each finding its
// request by bisection. The kernel is bound by latency, not by its few hundred KB: 512 requests of one new token take 6.4
// us, 1024, every eighth with a prompt chunk of up to 1024, 7.6.
__global__ void __launch_bounds__(kMapThreads) page_map_kernel(const PageMapArgs a) {
    extern __shared__ int sm[];
    int* page_off = sm;                    // [R + 1]
    int* tok_off = page_off + a.R + 1;     // [R + 1]
    int* take_off = tok_off + a.R + 1;     // [R]: first new page's place in the order; -1: refused
    __shared__ int64_t scratch[kMapScratch / sizeof(int64_t)];
    const int tid = threadIdx.x;
    const bool first = blockIdx.x == 0;
    const int per = (a.R + kMapThreads - 1) / kMapThreads;
    const int r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
    int count = *a.free_count;
    if (count < 0 || count > a.free_cap) {
        if (first && tid == 0) set_status(a.status, NF_ERR_DEVICE_BOUNDS);
        count = count < 0 ? 0 : a.free_cap;
    }
    int64_t asked = 0;
    for (int r = r0; r < r1; ++r) asked += need_of(a, r).take;
    int64_t total_asked, total_pages, total_tokens, total_taken;
    int64_t at = block_prefix(asked, scratch, &total_asked);
    int64_t pages = 0, tokens = 0, taken = 0;
    for (int r = r0; r < r1; ++r) {
        const Need n = need_of(a, r);
        if (first && (n.bad || n.dead || n.wide)) set_status(a.status, NF_ERR_DEVICE_BOUNDS);
        const bool fits = !n.dead && !n.wide && (n.take == 0 || at + n.take <= count);
        if (first && !fits && !n.dead && !n.wide) set_status(a.status, NF_ERR_OUT_OF_MEMORY);
        take_off[r] = fits ? (int)min(at, (int64_t)0x7fffffff) : -1;  // used where pages are taken: < count
        if (fits) taken += n.take;
        pages += n.dead ? 0 : n.before + (fits ? n.take : 0);
        tokens += n.fresh;
        at += n.take;
    }
    int64_t page_at = block_prefix(pages, scratch, &total_pages);
    int64_t tok_at = block_prefix(tokens, scratch, &total_tokens);
    block_prefix(taken, scratch, &total_taken);
    // a batch larger than the arrays is refused whole: empty requests, no page taken
    const bool refused = total_pages > a.page_cap || total_tokens > a.token_cap;
    if (refused && first && tid == 0) set_status(a.status, NF_ERR_DEVICE_BOUNDS);
    if (refused) {
        const int64_t T = min(total_tokens, (int64_t)a.token_cap);
        for (int64_t t = (int64_t)blockIdx.x * kMapThreads + tid; t < T; t += (int64_t)gridDim.x * kMapThreads)
            a.slots[t] = -1;
        for (int r = blockIdx.x * kMapThreads + tid; r < a.R; r += gridDim.x * kMapThreads) {
            a.kv_len[r] = 0;
            a.indptr[r + 1] = 0;
        }
        if (first && tid == 0) {
            a.indptr[0] = 0;
            *a.free_left = count;
        }
        return;
    }
    for (int r = r0; r < r1; ++r) {
        const Need n = need_of(a, r);
        page_off[r] = (int)page_at;
        tok_off[r] = (int)tok_at;
        page_at += n.dead ? 0 : n.before + (take_off[r] >= 0 ? n.take : 0);
        tok_at += n.fresh;
    }
    if (tid == 0) {
        page_off[a.R] = (int)total_pages;
        tok_off[a.R] = (int)total_tokens;
    }
    __syncthreads();

    const int step = gridDim.x * kMapThreads, me = blockIdx.x * kMapThreads + tid;
    if (first && tid == 0) {
        a.indptr[0] = 0;
        *a.free_left = count - (int)total_taken;
    }
    for (int r = me; r < a.R; r += step) {
        const Need n = need_of(a, r);
        a.kv_len[r] = n.dead ? 0 : n.ctx + (take_off[r] >= 0 ? n.fresh : 0);
        a.indptr[r + 1] = page_off[r + 1];
    }
    // page i of request r: an old entry of its table row, or one of the new pages
    auto page_of = [&](int r, int before, int i) {
        return i < before ? a.table[(int64_t)r * a.stride + i] : a.free_pages[count - 1 - (take_off[r] + i - before)];
    };
    for (int64_t e = me; e < total_pages; e += step) {
        const int r = row_of(page_off, a.R, (int)e), i = (int)e - page_off[r];
        const int before = need_of(a, r).before;
        const int page = page_of(r, before, i);
        if ((unsigned)page >= (unsigned)a.num_pages) set_status(a.status, NF_ERR_DEVICE_BOUNDS);
        if (i >= before) a.table[(int64_t)r * a.stride + i] = page;
        a.indices[e] = page;
    }
    for (int64_t e = me; e < total_tokens; e += step) {
        const int r = row_of(tok_off, a.R, (int)e);
        const Need n = need_of(a, r);
        const int64_t pos = (int64_t)n.ctx + ((int)e - tok_off[r]);
        int slot = -1;
        if (take_off[r] >= 0) {
            const int page = page_of(r, n.before, (int)(pos / kKv4Slots));
            if ((unsigned)page < (unsigned)a.num_pages) slot = page * kKv4Slots + (int)(pos % kKv4Slots);
        }
        a.slots[e] = slot;
        a.positions[e] = (int)min(pos, (int64_t)0x7fffffff);
    }
}

}  // namespace
}  // namespace nf

extern "C" nf_status nf_op_page_map(const int32_t* ctx_len, const int32_t* new_len, int32_t num_requests,
                                    int32_t* block_table, int32_t table_stride, const int32_t* free_pages,
                                    int32_t free_cap, const int32_t* free_count, int32_t num_pages, int32_t* kv_len,
                                    int32_t* page_indptr, int32_t* page_indices, int32_t page_cap, int32_t* slots,
                                    int32_t* positions, int32_t token_cap, int32_t* free_left,
                                    int32_t* status_device, void* stream) try {
    if (!ctx_len || !block_table || !free_pages || !free_count || !kv_len || !page_indptr || !page_indices || !slots ||
        !positions || !free_left || !status_device)
        return NF_ERR_INVALID_ARGUMENT;
    if (num_requests < 0 || num_requests > NF_KV4_MAX_REQUESTS || table_stride < 1 || free_cap < 0 || page_cap < 0 ||
        token_cap < 0 || num_pages < 1 || num_pages > NF_KV4_MAX_PAGES)
        return NF_ERR_INVALID_ARGUMENT;
    // every CTA reads all of the inputs while others write: an array that is written is a memory of its own
    const nf::Span read[] = {{ctx_len, num_requests}, {new_len, new_len ? num_requests : 0}, {free_pages, free_cap},
                             {free_count, 1}};
    const nf::Span written[] = {{block_table, (int64_t)num_requests * table_stride}, {kv_len, num_requests},
                                {page_indptr, (int64_t)num_requests + 1}, {page_indices, page_cap}, {slots, token_cap},
                                {positions, token_cap}, {free_left, 1}};
    for (const nf::Span& w : written) {
        for (const nf::Span& r : read)
            if (w.meets(r)) return NF_ERR_INVALID_ARGUMENT;
        for (const nf::Span& other : written)
            if (&other != &w && w.meets(other)) return NF_ERR_INVALID_ARGUMENT;
    }
    const nf_status st = nf::check_on_device(ctx_len, new_len, block_table, free_pages, free_count, kv_len, page_indptr,
                                             page_indices, slots, positions, free_left, status_device);
    if (st != NF_OK) return st;
    const int sms = nf::device_sm_count();
    if (sms <= 0) return NF_ERR_CUDA;
    const int64_t entries = (int64_t)page_cap + token_cap;
    int64_t grid = (entries + nf::kMapThreads - 1) / nf::kMapThreads;
    grid = grid < 1 ? 1 : grid > sms ? sms : grid;
    const size_t smem = sizeof(int) * ((size_t)3 * num_requests + 2);
    constexpr int kMost = sizeof(int) * (3 * NF_KV4_MAX_REQUESTS + 2);
    static_assert(kMost + nf::kMapScratch <= 227 * 1024, "offsets fit shared memory");
    // 48 KB without opting in, those of `scratch` among them. The limit is the kernel's, whichever thread sets it and for
    // captured calls too: always the largest, so that no call lowers what another one needs.
    if (smem + nf::kMapScratch > 48 * 1024 &&
        cudaFuncSetAttribute(nf::page_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost) != cudaSuccess)
        return NF_ERR_CUDA;
    const nf::PageMapArgs a{ctx_len, new_len, num_requests, block_table, table_stride, free_pages, free_cap, free_count,
                            num_pages, kv_len, page_indptr, page_indices, page_cap, slots, positions, token_cap,
                            free_left, status_device};
    nf::page_map_kernel<<<(int)grid, nf::kMapThreads, smem, static_cast<cudaStream_t>(stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? NF_OK : NF_ERR_CUDA;
} catch (...) {
    return NF_ERR_INVALID_ARGUMENT;
}
