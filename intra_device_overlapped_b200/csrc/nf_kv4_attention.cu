// Paged GQA decode attention over the 4-bit cache (format: nf_kv4.h).
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "nanoflow.h"
#include "nf_internal.h"
#include "nf_kv4.h"

namespace nf {
namespace {

constexpr int kMaxGroup = 8;               // query heads per KV head: the N = 8 columns of the tensor instruction
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kCtasPerSm = 4;              // 16 warps of 128 registers
constexpr int kStages = 2;                 // pairs of tiles in flight per warp
constexpr int kItemSlots = 3;
constexpr int kMaxCtas = kCtasPerSm * 160; // sizes the workspace (a B200 has 148 SMs)
constexpr int kItemsPerCta = 4;            // work items that a batch of many (request, head) pairs is cut into, per CTA
constexpr int kMinChunk = 16;              // pages
constexpr int kMaxParts = 2 * kItemsPerCta * kMaxCtas;

struct Kv4AttnArgs {
    const uint16_t* q;
    uint16_t* out;
    int64_t q_stride, out_stride;
    const uint8_t* pool;
    int num_pages;
    const int *kv_len, *indptr, *indices;
    int R, nkv, G;
    float scale_log2;
    uint32_t one;        // 0x3C003C00 (unpack4)
    int *claim, *done;   // work items taken beyond the first of each CTA; CTAs finished. Both 0 between calls
    int* arrived;        // [kMaxParts] chunks of a split (request, head) written so far, at its first part. 0 between calls
    float2* part_ml;     // [kMaxParts][kMaxGroup] maximum and sum
    float* part_o;       // [kMaxParts][G][D]
    int* status;
};

struct Item {
    int r, h;
    int first;      // place of its first page in page_indices
    int pages, keys;
    int chunks, c;  // of the request, this one
    int part;       // part of the request's chunk 0 of head h (chunks > 1)
};

template <int D>
struct Smem {
    static constexpr int kHead = 18 * D;            // K and V tile of a head
    static constexpr int kRow = D + 4;              // merge rows, padded against bank conflicts
    static constexpr int kHeads = 4 * kThreads / D; // heads joined at a time: a thread has 4 columns of one
    alignas(128) uint8_t ring[kWarps][kStages][2 * kHead];
    alignas(16) uint16_t q[kItemSlots][kMaxGroup * D];
    float merge[kWarps][kHeads][kRow];
    uint64_t item_full[kItemSlots];
    Item item[kItemSlots];
    float2 ml[kWarps][kMaxGroup];
    int64_t scan[kWarps];
    int item_start[kThreads + 1], part_start[kThreads + 1];
    int abort, last;
};

// Pages that request r reads: its keys, cut to what its row of the page table holds.
__device__ __forceinline__ int pages_of(const Kv4AttnArgs& a, int r, int* keys, bool report) {
    const int p0 = a.indptr[r];
    int64_t np = (int64_t)a.indptr[r + 1] - p0;
    int n = a.kv_len[r];
    bool bad = n < 0 || p0 < 0 || np < 0;
    if (n < 0 || p0 < 0 || np < 0) n = 0;
    if (np < 0) np = 0;
    if ((int64_t)n > np * kKv4Slots) {
        bad = true;
        n = (int)(np * kKv4Slots);
    }
    if (report && bad) set_status(a.status, NF_ERR_DEVICE_BOUNDS);
    *keys = n;
    return (int)(((int64_t)n + kKv4Slots - 1) / kKv4Slots);
}

__device__ __forceinline__ int chunks_of(int pages, int chunk) { return pages <= chunk ? 1 : (pages + chunk - 1) / chunk; }

__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ int warp_prefix(int x, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// Every lane of the warp learns that the phase has completed, or (false) that the wait gave up.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
    if (__all_sync(0xffffffffu, mbar_try_wait(smem_u32(bar), parity))) return true;
    int ok = 0;
    if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, abort_flag, status) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    return ok && __all_sync(0xffffffffu, mbar_test_wait(smem_u32(bar), parity));
}

// D = A B + C of 16 x 16 by 16 x 8, fp16 in, fp32 out
__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1, const float* c) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Codes of four pairs as fp16: nibble p of both halves of w, put under the exponent of 1 and freed of the bias
// again, exactly: (code - 8) / 1024 for the even nibbles, which spare a shift, (code - 8) / 64 for the odd ones.
// `one`, 0x3C003C00, comes as a value that the compiler does not know: with two constants it makes two logic
// operations of each (64 more instructions a tile).
__device__ __forceinline__ void unpack4(uint32_t w, uint32_t one, uint32_t* e) {
    constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u;
    const uint32_t t = w >> 8;
    e[0] = sub_f16x2((w & kLow) | one, 0x3C083C08u);
    e[1] = sub_f16x2((w & kHigh) | one, 0x3C803C80u);
    e[2] = sub_f16x2((t & kLow) | one, 0x3C083C08u);
    e[3] = sub_f16x2((t & kHigh) | one, 0x3C803C80u);
}

// Transpose of an 8 x 8 matrix of 16-bit values (two of a row to a lane)
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// 2^n / f for a power of two f that a bf16 holds
__device__ __forceinline__ float over_pow2(int n, uint32_t f_bits) {
    return __int_as_float((n + 254 - (int)(f_bits >> 7)) << 23);
}

template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void cp_async_16_hint(uint32_t dst, const void* src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy)
                 : "memory");
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Words of NG / 2 scales pairs (one slot)
template <int NG>
__device__ __forceinline__ void load_scales(const uint8_t* at, uint32_t* w) {
    if constexpr (NG == 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(at);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(at);
    }
}

template <int NG>
__device__ __forceinline__ void load_words(const uint8_t* at, uint32_t* w) {
    if constexpr (NG == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(at);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(at);
        w[0] = v.x; w[1] = v.y;
    }
}

// 2^(m - M) for partial sums: a part without keys (m = -inf) holds zeros, or the NaN of a NaN score
__device__ __forceinline__ float part_factor(float m, float M) { return m == -INFINITY ? 1.f : ex2_approx(m - M); }

// Warp 0: looks up the CTA's next item (`claimed`, in lane 0), publishes it as number `n` of the CTA with its q on
// the way, and claims another, which it returns (lane 0). The items go through a ring of three: number n's slot
// was that of n - 3, which every warp has read before it reached the barrier at that item's end; warp 0 publishes n
// when it works on n - 2 or later. Kept out of line: it runs once an item and would cost the tile loop registers.
template <int D>
__device__ __noinline__ int publish_item(const Kv4AttnArgs& a, Smem<D>& s, int claimed, int n_item, int per, int chunk) {
    const int lane = threadIdx.x & 31;
    Item it;
    it.r = -1;
    const int item = __shfl_sync(0xffffffffu, claimed, 0);
    if (item < s.item_start[kThreads]) {
        if (lane == 0) claimed = atomicAdd(a.claim, 1) + (int)gridDim.x;
        // the thread's share of requests that holds the item, by 32 and 4 of their starts; then the request
        constexpr int kSub = kThreads / 32;
        int span = (__popc(__ballot_sync(0xffffffffu, s.item_start[lane * kSub] <= item)) - 1) * kSub;
        span += __popc(__ballot_sync(0xffffffffu, lane < kSub && s.item_start[span + (lane & (kSub - 1))] <= item)) - 1;
        int at = s.item_start[span], part = s.part_start[span];
        const int end = min(a.R, (span + 1) * per);
        for (int r = span * per; r < end; r += 32) {
            const int mine = r + lane;
            int n = 0, kk = 0, pages = 0;
            if (mine < end) {
                pages = pages_of(a, mine, &kk, false);
                n = chunks_of(pages, chunk) * a.nkv;
            }
            const int pi = at + warp_prefix(n, lane);
            const int pp = part + warp_prefix(n > a.nkv ? n : 0, lane);
            const uint32_t past = __ballot_sync(0xffffffffu, pi > item);
            if (past) {
                const int src = __ffs(past) - 1;
                pages = __shfl_sync(0xffffffffu, pages, src);
                kk = __shfl_sync(0xffffffffu, kk, src);
                n = __shfl_sync(0xffffffffu, n, src);
                const int local = item - (__shfl_sync(0xffffffffu, pi, src) - n);
                it.r = r + src;
                it.c = local / a.nkv;
                it.h = local - it.c * a.nkv;
                it.chunks = n / a.nkv;
                it.part = __shfl_sync(0xffffffffu, pp, src) - n + it.h;
                const int b = (int)((int64_t)pages * it.c / it.chunks);
                const int e = (int)((int64_t)pages * (it.c + 1) / it.chunks);
                it.first = a.indptr[it.r] + b;
                it.pages = e - b;
                it.keys = min(kk - b * kKv4Slots, it.pages * kKv4Slots);
                break;
            }
            at = __shfl_sync(0xffffffffu, pi, 31);
            part = __shfl_sync(0xffffffffu, pp, 31);
        }
    }
    if (lane == 0) {
        const int slot = n_item % kItemSlots;
        s.item[slot] = it;
        if (it.r >= 0) {
            const uint32_t bytes = a.G * D * 2;
            mbar_arrive_expect_tx(&s.item_full[slot], bytes);
            bulk_load(s.q[slot], a.q + it.r * a.q_stride + (int64_t)it.h * a.G * D, bytes, &s.item_full[slot]);
        } else {
            mbar_arrive(&s.item_full[slot]);
        }
    }
    __syncwarp();
    return claimed;
}

// o = softmax(q K^T) V per (request, KV head), G query heads at a time, in one pass over the cache.
//
// The cache is read once, 144 bytes a key and head (d = 128), and the kernel has to turn codes into operands as
// fast as the HBM brings them: per SM one 16-key tile of K and V (2304 bytes) every 100 cycles, 400 issue slots.
// Codes become fp16 in registers, right in the operand layout of the warp-level mma (that is the order they
// are stored in): no shared-memory round trip, which tcgen05 operands would need.
//   Scores. S[key, head] = sum over groups j of s_k[key, j] * sum over d in j of code q. A = K's codes (unpack4),
//   B = q as fp16 times a power of two per head (exact but below 2^-24 of the row's largest; columns of the even
//   nibbles times 16 for their codes' 1 / 1024). The scale is applied to the 16 x 8 accumulator of each group, 32
//   columns, in fp32.
//   Output. O^T[d, head] += V^T[d, key] P^T[key, head], P = 2^(x - M) s_v[key, j] f_j in fp16 (2^-11), V's
//   codes exact. f_j, a power of two that follows the largest scale of the group so far, and M, the integral
//   running maximum of the head, keep P within 2^15; both move only when a value has outgrown them (2^5 and 2^2
//   of slack), which one vote per two tiles detects. P goes from accumulator to operand layout by movmatrix.
// Sums and statistics are fp32. M0, M1 etc. belong to the two head columns 2 t, 2 t + 1 of a lane.
//
// Work. A request's pages are cut into chunks of at most `chunk` pages. With few (request, head) pairs, at most
// half the CTAs, chunk = pages in all / (CTAs - pairs): no more chunks than CTAs, one round of equal ones; with many,
// a quarter of a CTA's share, so that lengths even out and few requests are split. Each CTA scans the lengths
// itself (no second launch, nothing on the host depends on them). An item is one chunk of one KV head; its pages
// go round the 4 warps by twos. CTAs take their first item by number, further ones from a counter. Every warp keeps
// its own ring of tiles full (cp.async: per-thread groups, no barriers) and runs up to one item ahead of the one it
// works on, so that item ends do not drain the loads; warp 0 also claims items and copies q, two items ahead. Chunks
// of one (request, head) meet in the workspace; the CTA that brings the last one joins them, in chunk order.
template <int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) kv4_attention_kernel(const __grid_constant__ Kv4AttnArgs a) {
    constexpr int NG = D / 32, NW = NG / 2;
    using S = Smem<D>;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    S& s = *reinterpret_cast<S*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    volatile int* abort_flag = &s.abort;

    if (tid == 0) {
        s.abort = 0;
        for (int i = 0; i < kItemSlots; ++i) mbar_init(&s.item_full[i], 1);
        fence_mbar_init();
    }
    // --- the batch: pages in all, chunk size, items and parts before each thread's requests
    const int per = (a.R + kThreads - 1) / kThreads;
    const int r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
    int chunk;
    {
        int keys;
        int64_t sum = 0;
        for (int r = r0; r < r1; ++r) sum += pages_of(a, r, &keys, blockIdx.x == 0);
        sum = warp_sum(sum);
        if (lane == 0) s.scan[warp] = sum;
        __syncthreads();
        int64_t total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) total += s.scan[w];
        total *= a.nkv;
        const int pairs = a.R * a.nkv, ctas = gridDim.x;
        const int64_t share = 2 * pairs <= ctas ? ctas - pairs : kItemsPerCta * ctas;
        chunk = (int)max((int64_t)kMinChunk, min((total + share - 1) / share, (int64_t)0x7fffffff));
        int items = 0, parts = 0;
        for (int r = r0; r < r1; ++r) {
            const int n = chunks_of(pages_of(a, r, &keys, false), chunk) * a.nkv;
            items += n;
            if (n > a.nkv) parts += n;
        }
        const int pi = warp_prefix(items, lane), pp = warp_prefix(parts, lane);
        __syncthreads();
        if (lane == 31) s.scan[warp] = (int64_t)pi << 32 | (uint32_t)pp;
        __syncthreads();
        int bi = 0, bp = 0;
        for (int w = 0; w < warp; ++w) {
            bi += (int)(s.scan[w] >> 32);
            bp += (int)s.scan[w];
        }
        s.item_start[tid + 1] = bi + pi;
        s.part_start[tid + 1] = bp + pp;
        if (tid == 0) s.item_start[0] = s.part_start[0] = 0;
        __syncthreads();
    }

    int claimed = blockIdx.x, published = 0;
    if (warp == 0) claimed = publish_item<D>(a, s, claimed, published++, per, chunk);

    // --- every warp: its ring of tile pairs. Pair i of the warp is pages 8 i + 2 warp and the next one of an item.
    int flying = 0;                // pairs on their way or waiting, the number of cp.async groups in flight at most
    uint32_t absent = 0;           // two bits per stage: no such page, or one outside the pool
    int in_st = 0, out_st = 0;     // stages of the next pair issued, used
    int ahead = 0, left = 0, at_pair = 0, ids = 0;  // items begun to load; the last of them
    bool ok = true, ended = false;
    const uint32_t my_ring = smem_u32(s.ring[warp]) + lane * 16;
    const uint8_t* const my_pool = a.pool + lane * 16;
    auto fill = [&](int working) {  // `working`: the item that the warp works on
        while (flying < kStages) {
            if (left == 0) {
                if (ended || ahead > working + 1) return;
                if (warp == 0 && published == ahead + 1)
                    claimed = publish_item<D>(a, s, claimed, published++, per, chunk);
                const int slot = ahead % kItemSlots;
                ok = wait_warp(&s.item_full[slot], (ahead / kItemSlots) & 1, abort_flag, a.status);
                if (!ok || s.item[slot].r < 0) {
                    ended = true;
                    return;
                }
                left = max(0, (s.item[slot].pages - 2 * warp + 2 * kWarps - 1) / (2 * kWarps));
                at_pair = 0;
                ++ahead;
                if (left == 0) continue;
            }
            if ((at_pair & 15) == 0) {  // lane l: tile of the l-th page of the next 16 pairs; -1: none, or outside
                const Item& it = s.item[(ahead - 1) % kItemSlots];
                const int p = 2 * kWarps * (at_pair + (lane >> 1)) + 2 * warp + (lane & 1);
                ids = -1;
                if (p < it.pages) {
                    const int page = __ldg(a.indices + it.first + p);
                    if ((unsigned)page < (unsigned)a.num_pages)
                        ids = page * a.nkv + it.h;
                    else
                        set_status(a.status, NF_ERR_DEVICE_BOUNDS);
                }
            }
            const int t0 = __shfl_sync(0xffffffffu, ids, 2 * (at_pair & 15));
            const int t1 = __shfl_sync(0xffffffffu, ids, 2 * (at_pair & 15) + 1);
            const uint32_t dst = my_ring + in_st * 2 * S::kHead;
            const uint8_t* src0 = my_pool + (int64_t)t0 * S::kHead;
            const uint8_t* src1 = my_pool + (int64_t)t1 * S::kHead - S::kHead;
            const uint64_t policy = l2_policy_evict_first();
            constexpr int kPieces = (2 * S::kHead + 511) / 512;  // piece lane + 32 i of the two tiles, 16 bytes
            absent &= ~(3u << 2 * in_st);
            if ((t0 | t1) >= 0) {
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const bool second = 512 * i >= S::kHead || (512 * i + 512 > S::kHead && 512 * i + lane * 16 >= S::kHead);
                    if (512 * i + 512 <= 2 * S::kHead || 512 * i + lane * 16 < 2 * S::kHead)
                        cp_async_16_hint(dst + 512 * i, (second ? src1 : src0) + 512 * i, policy);
                }
            } else {
                absent |= ((uint32_t)(t0 < 0) | (uint32_t)(t1 < 0) << 1) << 2 * in_st;
#pragma unroll 1
                for (int i = 0; i < kPieces; ++i) {
                    const int at = 512 * i + lane * 16;
                    if (at < S::kHead ? t0 >= 0 : at < 2 * S::kHead && t1 >= 0)
                        cp_async_16_hint(dst + 512 * i, (at < S::kHead ? src0 : src1) + 512 * i, policy);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            ++flying;
            ++at_pair;
            --left;
            if (++in_st == kStages) in_st = 0;
        }
    };

    const int gid = lane >> 2, tig = lane & 3;
    const uint32_t one = a.one;
    for (int k = 0;; ++k) {
        const int slot = k % kItemSlots;
        if (ok) fill(k);
        ok = ok && wait_warp(&s.item_full[slot], (k / kItemSlots) & 1, abort_flag, a.status);
        const bool live = ok && s.item[slot].r >= 0;
        const int pages = live ? s.item[slot].pages : 0, keys = s.item[slot].keys;
        float O[NG][2][4], M0 = -INFINITY, M1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        uint32_t f[NW];
#pragma unroll
        for (int u = 0; u < NG; ++u) {
            f[u / 2] = 0x71807180u;  // 2^100: the first scale outgrows it
#pragma unroll
            for (int i = 0; i < 4; ++i) O[u][0][i] = O[u][1][i] = 0.f;
        }
        if (pages > 2 * warp) {
            // q of head gid, columns 32 j + 8 t .. + 7, as fp16 times 2^(10 - e), 2^e the row's largest; pairs of even
            // nibbles times 16 more
            uint32_t qf[NG][4];
            float hs0, hs1;
            {
                uint4 raw[NG];
                uint32_t top = 0;
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    raw[j] = gid < a.G ? *reinterpret_cast<const uint4*>(&s.q[slot][gid * D + 32 * j + 8 * tig])
                                       : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7FFFu, w[i] >> 16 & 0x7FFFu));
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // exponent field; rows of zeros or subnormals count as 1, infinities and NaN as 254
                const int ex = min(max((int)(top >> 7), 1), 254);
                // 2^(10 - (ex - 127)) in two steps, either a normal number
                const int up = 10 + 127 - ex, up0 = up / 2, up1 = up - up0;
                const float m0 = __int_as_float((127 + up0) << 23), m1 = __int_as_float((127 + up1) << 23);
                // (not 0, so that minus infinity times it stays that)
                const float hs = fmaxf(a.scale_log2 * 64.f * __int_as_float((127 - up0) << 23) *
                                           __int_as_float((127 - up1) << 23), 0x1p-140f);
                hs0 = __shfl_sync(0xffffffffu, hs, 8 * tig);
                hs1 = __shfl_sync(0xffffffffu, hs, 8 * tig + 4);
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float m = i % 2 ? m1 : m1 * 16.f;
                        qf[j][i] = pack_f16x2(lo_bf16(w[i]) * m0 * m, hi_bf16(w[i]) * m0 * m);
                    }
                }
            }
            for (int p = 2 * warp; p < pages; p += 2 * kWarps) {
                if (flying == kStages)
                    cp_async_wait<kStages - 1>();
                else
                    cp_async_wait<0>();
                __syncwarp();
                const uint8_t* tile = s.ring[warp][out_st];
                const uint32_t none = absent >> 2 * out_st & 3u;
                float x[2][4];
                uint32_t va[2][NG], vb[2][NG], ta[2][NW], tb[2][NW];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint8_t* kt = tile + i * S::kHead;
                    uint32_t ka[NG], kb[NG], sa[NW], sb[NW];
                    load_words<NG>(kt + lane * (D / 8), ka);            // slot gid
                    load_words<NG>(kt + 4 * D + lane * (D / 8), kb);    // slot gid + 8
                    load_scales<NG>(kt + 8 * D + gid * (2 * NG), sa);
                    load_scales<NG>(kt + 8 * D + (gid + 8) * (2 * NG), sb);
#pragma unroll
                    for (int j = 0; j < NG; ++j) {
                        uint32_t ea[4], eb[4];
                        unpack4(ka[j], one, ea);
                        unpack4(kb[j], one, eb);
                        const uint32_t a0[4] = {ea[0], eb[0], ea[1], eb[1]}, a1[4] = {ea[2], eb[2], ea[3], eb[3]};
                        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
                        float acc[4];
                        mma_f16(acc, a0, qf[j][0], qf[j][1], zero);
                        mma_f16(acc, a1, qf[j][2], qf[j][3], acc);
                        const float ga = j % 2 ? hi_bf16(sa[j / 2]) : lo_bf16(sa[j / 2]);
                        const float gb = j % 2 ? hi_bf16(sb[j / 2]) : lo_bf16(sb[j / 2]);
                        x[i][0] = j ? fmaf(ga, acc[0], x[i][0]) : ga * acc[0];
                        x[i][1] = j ? fmaf(ga, acc[1], x[i][1]) : ga * acc[1];
                        x[i][2] = j ? fmaf(gb, acc[2], x[i][2]) : gb * acc[2];
                        x[i][3] = j ? fmaf(gb, acc[3], x[i][3]) : gb * acc[3];
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint8_t* vt = tile + i * S::kHead + 9 * D;
                    load_words<NG>(vt + (tig * 8 + gid) * (D / 8), va[i]);          // slots 2 t, 2 t + 1
                    load_words<NG>(vt + 4 * D + (tig * 8 + gid) * (D / 8), vb[i]);  // slots 2 t + 8, 2 t + 9
                    load_scales<NG>(vt + 8 * D + gid * (2 * NG), ta[i]);
                    load_scales<NG>(vt + 8 * D + (gid + 8) * (2 * NG), tb[i]);
                }
                __syncwarp();
                --flying;
                if (++out_st == kStages) out_st = 0;
                fill(k);
                if (none == 3u) continue;
                const int valid = keys - p * kKv4Slots;
                if (none || valid < 2 * kKv4Slots) {
                    // slots behind the request's length, and of pages that are not there, hold anything
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int n = none >> i & 1u ? 0 : valid - i * kKv4Slots;
                        if (gid >= n) {
                            x[i][0] = x[i][1] = -INFINITY;
#pragma unroll
                            for (int u = 0; u < NW; ++u) ta[i][u] = 0;
                        }
                        if (gid + 8 >= n) {
                            x[i][2] = x[i][3] = -INFINITY;
#pragma unroll
                            for (int u = 0; u < NW; ++u) tb[i][u] = 0;
                        }
                    }
                }
                uint32_t grown = 0;
#pragma unroll
                for (int u = 0; u < NW; ++u)
                    grown = max_bf16x2(grown, mul_bf16x2(max_bf16x2(max_bf16x2(ta[0][u], tb[0][u]),
                                                                    max_bf16x2(ta[1][u], tb[1][u])), f[u]));
                float y[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    y[i][0] = fmaf(x[i][0], hs0, -M0);
                    y[i][1] = fmaf(x[i][1], hs1, -M1);
                    y[i][2] = fmaf(x[i][2], hs0, -M0);
                    y[i][3] = fmaf(x[i][3], hs1, -M1);
                }
                const float most = fmaxf(fmaxf(fmaxf(y[0][0], y[0][1]), fmaxf(y[0][2], y[0][3])),
                                         fmaxf(fmaxf(y[1][0], y[1][1]), fmaxf(y[1][2], y[1][3])));
                const bool over = most > 5.f || lo_bf16(grown) >= 1024.f || hi_bf16(grown) >= 1024.f;
                if (__any_sync(0xffffffffu, over)) {
                    // columns of heads beyond G are zeros throughout
                    float n0 = fmaxf(fmaxf(x[0][0], x[0][2]), fmaxf(x[1][0], x[1][2])) * hs0;
                    float n1 = fmaxf(fmaxf(x[0][1], x[0][3]), fmaxf(x[1][1], x[1][3])) * hs1;
                    uint32_t top[NW];
#pragma unroll
                    for (int u = 0; u < NW; ++u)
                        top[u] = max_bf16x2(max_bf16x2(ta[0][u], tb[0][u]), max_bf16x2(ta[1][u], tb[1][u]));
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) {
                        n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, o));
                        n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, o));
#pragma unroll
                        for (int u = 0; u < NW; ++u)
                            top[u] = max_bf16x2(top[u], __shfl_xor_sync(0xffffffffu, top[u], o));
                    }
                    n0 = softmax_max_update(M0, n0);
                    n1 = softmax_max_update(M1, n1);
                    const float c0 = M0 == n0 ? 1.f : ex2_approx(M0 - n0), c1 = M1 == n1 ? 1.f : ex2_approx(M1 - n1);
                    M0 = n0;
                    M1 = n1;
                    l0 *= c0;
                    l1 *= c1;
#pragma unroll
                    for (int u = 0; u < NG; ++u) {
                        const uint32_t was = u % 2 ? f[u / 2] >> 16 : f[u / 2] & 0xFFFFu;
                        const float t = u % 2 ? hi_bf16(top[u / 2]) : lo_bf16(top[u / 2]);
                        float g = 1.f;
                        if (t * __uint_as_float(was << 16) >= 1024.f) {  // the new largest scale comes to [2^8, 2^9)
                            const int e = (int)(__float_as_uint(t) >> 23);
                            const uint32_t now = (uint32_t)min(max(254 + 8 - e, 1), 254) << 7;
                            f[u / 2] = u % 2 ? (f[u / 2] & 0xFFFFu) | now << 16 : (f[u / 2] & 0xFFFF0000u) | now;
                            g = __int_as_float(max(0, 127 + (int)(now >> 7) - (int)(was >> 7)) << 23);
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            O[u][i][0] *= c0 * g;
                            O[u][i][1] *= c1 * g;
                            O[u][i][2] *= c0 * g;
                            O[u][i][3] *= c1 * g;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        y[i][0] = fmaf(x[i][0], hs0, -M0);
                        y[i][1] = fmaf(x[i][1], hs1, -M1);
                        y[i][2] = fmaf(x[i][2], hs0, -M0);
                        y[i][3] = fmaf(x[i][3], hs1, -M1);
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[i][e] = ex2_approx(y[i][e]);
                    l0 += y[i][0] + y[i][2];
                    l1 += y[i][1] + y[i][3];
#pragma unroll
                    for (int u = 0; u < NW; ++u) {
                        const uint32_t pa = mul_bf16x2(ta[i][u], f[u]), pb = mul_bf16x2(tb[i][u], f[u]);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float ga = e ? hi_bf16(pa) : lo_bf16(pa), gb = e ? hi_bf16(pb) : lo_bf16(pb);
                            const uint32_t b0 = transpose8(pack_f16x2(y[i][0] * ga, y[i][1] * ga));
                            const uint32_t b1 = transpose8(pack_f16x2(y[i][2] * gb, y[i][3] * gb));
                            uint32_t ea[4], eb[4];
                            unpack4(va[i][2 * u + e], one, ea);
                            unpack4(vb[i][2 * u + e], one, eb);
                            const uint32_t a0[4] = {ea[0], ea[1], eb[0], eb[1]}, a1[4] = {ea[2], ea[3], eb[2], eb[3]};
                            mma_f16(O[2 * u + e][0], a0, b0, b1, O[2 * u + e][0]);
                            mma_f16(O[2 * u + e][1], a1, b0, b1, O[2 * u + e][1]);
                        }
                    }
                }
            }
        }
        // --- join the warps. One barrier per round for every warp, whatever happened: a wait that gave up (in any
        // warp) ends all of them here. It also tells that the previous item's sums have been read.
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, o);
            l1 += __shfl_xor_sync(0xffffffffu, l1, o);
        }
        const Item it = s.item[slot];  // read before the barrier: the slot may be written anew after it
        if (bar_red_or(1, kThreads, !ok)) break;
        if (!live) break;
        if (gid == 0) {
            s.ml[warp][2 * tig] = make_float2(M0, l0);
            s.ml[warp][2 * tig + 1] = make_float2(M1, l1);
        }
        const int col = tid % (D / 4) * 4;
        const int64_t part = (int64_t)it.part + (int64_t)it.c * a.nkv;
        auto store = [&](int h, float4 o, float L) {
            const float inv = L == 0.f ? 0.f : 1.f / L;
            *reinterpret_cast<uint2*>(a.out + it.r * a.out_stride + (int64_t)(it.h * a.G + h) * D + col) =
                make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        };
        for (int h0 = 0; h0 < a.G; h0 += S::kHeads) {
            if (h0) bar_sync_n(1, kThreads);
            const int mine = 2 * tig - h0;
            if (mine >= 0 && mine < S::kHeads) {
#pragma unroll
                for (int u = 0; u < NG; ++u) {
                    const uint32_t fu = u % 2 ? f[u / 2] >> 16 : f[u / 2] & 0xFFFFu;
                    const float g = over_pow2(6, fu), ge = over_pow2(10, fu);
                    float* row = &s.merge[warp][mine][32 * u + 4 * gid];
                    *reinterpret_cast<float4*>(row) =
                        make_float4(O[u][0][0] * ge, O[u][0][2] * g, O[u][1][0] * ge, O[u][1][2] * g);
                    *reinterpret_cast<float4*>(row + S::kRow) =
                        make_float4(O[u][0][1] * ge, O[u][0][3] * g, O[u][1][1] * ge, O[u][1][3] * g);
                }
            }
            bar_sync_n(1, kThreads);
            const int row = tid / (D / 4), h = h0 + row;
            if (h >= a.G) continue;
            float M = -INFINITY, L = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s.ml[w][h].x);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 ml = s.ml[w][h];
                const float c = part_factor(ml.x, M);
                const float4 v = *reinterpret_cast<const float4*>(&s.merge[w][row][col]);
                L += c * ml.y;
                o.x += c * v.x;
                o.y += c * v.y;
                o.z += c * v.z;
                o.w += c * v.w;
            }
            if (it.chunks == 1) {
                store(h, o, L);
            } else {
                __stcg(reinterpret_cast<float4*>(a.part_o + (part * a.G + h) * D + col), o);
                if (col == 0) __stcg(a.part_ml + part * kMaxGroup + h, make_float2(M, L));
            }
        }
        if (it.chunks == 1) continue;
        __threadfence();
        bar_sync_n(1, kThreads);
        if (tid == 0) {
            const int n = atomicAdd(a.arrived + it.part, 1);
            s.last = n == it.chunks - 1;
            if (s.last) a.arrived[it.part] = 0;
        }
        bar_sync_n(1, kThreads);
        if (!s.last) continue;
        __threadfence();
        for (int h = tid / (D / 4); h < a.G; h += S::kHeads) {
            const float2* ml = a.part_ml + (int64_t)it.part * kMaxGroup + h;
            const float* po = a.part_o + ((int64_t)it.part * a.G + h) * D + col;
            const int64_t step = (int64_t)a.nkv * a.G * D;
            float M = -INFINITY, L = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int c = 0; c < it.chunks; ++c) M = fmaxf(M, __ldcg(ml + (int64_t)c * a.nkv * kMaxGroup).x);
#pragma unroll 8
            for (int c = 0; c < it.chunks; ++c) {
                const float2 m = __ldcg(ml + (int64_t)c * a.nkv * kMaxGroup);
                const float4 v = __ldcg(reinterpret_cast<const float4*>(po + c * step));
                const float w = part_factor(m.x, M);
                L += w * m.y;
                o.x += w * v.x;
                o.y += w * v.y;
                o.z += w * v.z;
                o.w += w * v.w;
            }
            store(h, o, L);
        }
    }
    cp_async_wait<0>();
    if (*abort_flag && tid == 0) {  // the copies in flight land before the memory is given up
        int none = 0;
        for (int i = max(0, published - kItemSlots); i < published; ++i)
            mbar_wait(&s.item_full[i % kItemSlots], (i / kItemSlots) & 1, &none, a.status);
    }
    __syncthreads();
    if (tid == 0) {
        const int n = atomicAdd(a.done, 1);
        if (n == (int)gridDim.x - 1) {  // every CTA has made its claims
            *a.claim = 0;
            *a.done = 0;
        }
    }
}

// Workspace: claim and done counters (256 bytes), arrived, part_ml, part_o.
struct Workspace {
    int64_t arrived, ml, o, bytes;
    Workspace(int G, int d) {
        arrived = 256;
        ml = arrived + (int64_t)sizeof(int) * kMaxParts;
        o = ml + (int64_t)sizeof(float2) * kMaxGroup * kMaxParts;
        bytes = o + (int64_t)sizeof(float) * G * d * kMaxParts;
    }
};

template <int D>
cudaError_t launch(const Kv4AttnArgs& a, int grid, cudaStream_t s) {
    static_assert(kCtasPerSm * (sizeof(Smem<D>) + 1024) <= 228 * 1024, "CTAs of an SM share its memory");
    const cudaError_t e = cudaFuncSetAttribute(kv4_attention_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)sizeof(Smem<D>));
    if (e != cudaSuccess) return e;
    kv4_attention_kernel<D><<<grid, kThreads, sizeof(Smem<D>), s>>>(a);
    return cudaGetLastError();
}

nf_status check_shape(int32_t nq, int32_t nkv, int32_t d) {
    if (nq < 1) return NF_ERR_INVALID_ARGUMENT;
    const nf_status st = kv4_check_heads(nkv, d);
    if (st != NF_OK) return st;
    return nq % nkv ? NF_ERR_INVALID_ARGUMENT : nq / nkv > kMaxGroup ? NF_ERR_UNSUPPORTED : NF_OK;
}

}  // namespace
}  // namespace nf

extern "C" int64_t nf_kv4_workspace_bytes(int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim) {
    const nf_status st = nf::check_shape(n_q_heads, n_kv_heads, head_dim);
    return st == NF_OK ? nf::Workspace(n_q_heads / n_kv_heads, head_dim).bytes : -(int64_t)st;
}

extern "C" nf_status nf_op_kv4_decode_attention(const void* q, int64_t q_stride, void* out, int64_t out_stride,
                                                const void* pool, int32_t num_pages, const int32_t* kv_len,
                                                const int32_t* page_indptr, const int32_t* page_indices,
                                                int32_t num_requests, int32_t n_q_heads, int32_t n_kv_heads,
                                                int32_t head_dim, float softmax_scale, void* workspace,
                                                int64_t workspace_bytes, int32_t* status_device, int32_t sm_count,
                                                void* stream) try {
    if (!q || !out || !pool || !kv_len || !page_indptr || !page_indices || !workspace || !status_device)
        return NF_ERR_INVALID_ARGUMENT;
    nf_status st = nf::check_shape(n_q_heads, n_kv_heads, head_dim);
    if (st != NF_OK) return st;
    const int64_t row = (int64_t)n_q_heads * head_dim;
    // (tiles are numbered page * n_kv_heads + head in 32 bits: a pool of 2^31 tiles would not fit any device)
    if (num_pages < 1 || num_pages > NF_KV4_MAX_PAGES || (int64_t)num_pages * n_kv_heads > 0x7fffffff || num_requests < 0 || num_requests > NF_KV4_MAX_REQUESTS ||
        sm_count < 0 || !(softmax_scale >= 0.f) || !std::isfinite(softmax_scale))
        return NF_ERR_INVALID_ARGUMENT;
    if (q_stride < row || out_stride < row || q_stride % 8 || out_stride % 8 || !nf::aligned(q, 16) ||
        !nf::aligned(out, 16) || !nf::aligned(pool, 16) || !nf::aligned(workspace, 256) ||
        workspace_bytes < nf_kv4_workspace_bytes(n_q_heads, n_kv_heads, head_dim))
        return NF_ERR_INVALID_ARGUMENT;
    if (num_requests == 0) return NF_OK;
    if ((st = nf::check_on_device(q, (const void*)out, pool, (const void*)kv_len, (const void*)page_indptr,
                                  (const void*)page_indices, (const void*)workspace, (const void*)status_device)) !=
        NF_OK)
        return st;
    int sms = nf::device_sm_count();
    if (sms <= 0) return NF_ERR_CUDA;
    if (sm_count > 0 && sm_count < sms) sms = sm_count;
    const int grid = std::min(sms * nf::kCtasPerSm, nf::kMaxCtas);
    const double scale = softmax_scale > 0.f ? (double)softmax_scale : 1.0 / std::sqrt((double)head_dim);
    const int G = n_q_heads / n_kv_heads;
    const nf::Workspace at(G, head_dim);
    uint8_t* w = static_cast<uint8_t*>(workspace);
    const nf::Kv4AttnArgs a{static_cast<const uint16_t*>(q), static_cast<uint16_t*>(out), q_stride, out_stride,
                            static_cast<const uint8_t*>(pool), num_pages, kv_len, page_indptr, page_indices,
                            num_requests, n_kv_heads, G, (float)(scale * 1.4426950408889634), 0x3C003C00u,
                            reinterpret_cast<int*>(w), reinterpret_cast<int*>(w) + 32,
                            reinterpret_cast<int*>(w + at.arrived), reinterpret_cast<float2*>(w + at.ml),
                            reinterpret_cast<float*>(w + at.o), status_device};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = head_dim == 64 ? nf::launch<64>(a, grid, s) : nf::launch<128>(a, grid, s);
    return e == cudaSuccess ? NF_OK : NF_ERR_CUDA;
} catch (...) {
    return NF_ERR_INVALID_ARGUMENT;
}
