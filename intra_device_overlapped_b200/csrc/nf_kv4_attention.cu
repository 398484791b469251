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
constexpr int kWarps = 8;                  // consumer warps; one more loads
constexpr int kConsumers = kWarps * 32;
constexpr int kThreads = kConsumers + 32;
constexpr int kStages = 4;                 // tiles in flight per consumer warp
constexpr int kItemSlots = 2;
constexpr int kSpans = kConsumers;         // the scan deals the requests to this many threads
constexpr int kCtasPerSm = 2;
constexpr int kMaxCtas = kCtasPerSm * 160; // sizes the workspace (a B200 has 148 SMs)
constexpr int kItemsPerCta = 4;            // work items that a long batch is cut into, per CTA
constexpr int kMinChunk = 32;              // pages: one ring of every warp
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
    static constexpr int kHead = 18 * D;          // K and V tile of a head
    static constexpr int kRow = D + 4;            // merge rows, padded against bank conflicts
    alignas(128) uint8_t ring[kWarps][kStages][kHead];
    alignas(16) uint16_t q[kItemSlots][kMaxGroup * D];
    float merge[kWarps][kMaxGroup][kRow];
    float2 ml[kWarps][kMaxGroup];
    uint64_t full[kWarps][kStages], empty[kWarps][kStages], item_full[kItemSlots], item_empty[kItemSlots];
    Item item[kItemSlots];
    int skip[kWarps][kStages];                    // the page of this stage lies outside the pool
    int64_t scan[kSpans / 32];
    int item_start[kSpans + 1], part_start[kSpans + 1];
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
    asm volatile(
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

// Codes of four pairs as fp16: nibble p of both halves of w under the exponent of 1, 1 + code / 64.
__device__ __forceinline__ void unpack4(uint32_t w, uint32_t* e) {
    constexpr uint32_t kMask = 0x00F000F0u, kOne = 0x3C003C00u;
    e[0] = (w << 4 & kMask) | kOne;
    e[1] = (w & kMask) | kOne;
    e[2] = (w >> 4 & kMask) | kOne;
    e[3] = (w >> 8 & kMask) | kOne;
}

__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// bf16 scales of NG groups (one slot) as fp32
template <int NG>
__device__ __forceinline__ void load_scales(const uint8_t* at, float* s) {
    if constexpr (NG == 4) {
        const uint2 w = *reinterpret_cast<const uint2*>(at);
        s[0] = __uint_as_float(w.x << 16);
        s[1] = __uint_as_float(w.x & 0xFFFF0000u);
        s[2] = __uint_as_float(w.y << 16);
        s[3] = __uint_as_float(w.y & 0xFFFF0000u);
    } else {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(at);
        s[0] = __uint_as_float(w << 16);
        s[1] = __uint_as_float(w & 0xFFFF0000u);
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
__device__ __forceinline__ float part_factor(float m, float M) { return m == -INFINITY ? 1.f : exp2f(m - M); }

// o = softmax(q K^T) V per (request, KV head), G query heads at a time, in one pass over the cache.
//
// The cache is read once, 144 bytes a key and head (d = 128) against 2.7 KB of fp32 multiplications' worth of
// arithmetic, so the kernel has to stream at the HBM's rate while it turns codes into operands: per SM one
// 16-key tile of K and V (2304 bytes) every 100 cycles, 400 issue slots. Codes become fp16 in registers, right
// in the operand layout of the warp-level mma (that is the order they are stored in): one logic operation per
// two codes, no shared-memory round trip, which tcgen05 operands would need.
//   Scores. S[key, head] = sum over groups j of s_k[key, j] * sum over d in j of code q. A = K's codes as
//   1 + (code + 8) / 64, B = q as fp16 times a power of two per head (exact but below 2^-29 of the row's
//   largest); the bias leaves through the accumulator's start, -1.125 sum q. The scale is applied to the
//   16 x 8 accumulator of each group, 32 columns, in fp32.
//   Output. O^T[d, head] += V^T[d, key] P^T[key, head], P = 2^(x - M) s_v[key, j] f_j in fp16 (2^-11), V's
//   codes exact ((code) / 64: the bias is subtracted, since P's rounding must not meet it). f_j, a
//   power of two that follows the largest scale of the group so far, and M, the integral running maximum of
//   the head, keep P within 2^15; both move only when a value has outgrown them (2^5 and 2^2 of slack), which
//   one vote per tile detects. P goes from accumulator to operand layout by movmatrix.
// Sums and statistics are fp32. M0, M1 etc. belong to the two head columns 2 t, 2 t + 1 of a lane.
//
// Work. A request's pages are cut into chunks of at most `chunk` = max(32, total pages x heads / (4 CTAs))
// pages: long batches get four items per CTA and are rarely split, small ones spread over the SMs. Each CTA scans
// the lengths itself (no second launch, nothing on the host depends on them). An item is one chunk of one KV head;
// its pages go round the 8 consumer warps. CTAs take their first item by number, further ones from a counter. The
// ninth warp runs ahead: it claims items, copies q, and keeps 4 tiles in flight for each warp (one bulk copy a
// tile), so that item ends do not drain the loads. Chunks of one (request, head) meet in the workspace; the
// CTA that brings the last one joins them, in chunk order.
template <int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) kv4_attention_kernel(const Kv4AttnArgs a) {
    constexpr int NG = D / 32;
    using S = Smem<D>;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    S& s = *reinterpret_cast<S*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    volatile int* abort_flag = &s.abort;

    if (tid == 0) {
        s.abort = 0;
        for (int w = 0; w < kWarps; ++w)
            for (int i = 0; i < kStages; ++i) {
                mbar_init(&s.full[w][i], 1);
                mbar_init(&s.empty[w][i], 1);
            }
        for (int i = 0; i < kItemSlots; ++i) {
            mbar_init(&s.item_full[i], 1);
            mbar_init(&s.item_empty[i], kWarps);
        }
        fence_mbar_init();
    }
    // --- the batch: pages in all, chunk size, items and parts before each span of requests
    const int per = (a.R + kSpans - 1) / kSpans;
    const int r0 = min(a.R, tid * per), r1 = tid < kSpans ? min(a.R, r0 + per) : r0;
    int keys;
    int64_t sum = 0;
    for (int r = r0; r < r1; ++r) sum += pages_of(a, r, &keys, blockIdx.x == 0);
    sum = warp_sum(sum);
    if (lane == 0 && warp < kWarps) s.scan[warp] = sum;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += s.scan[w];
    const int64_t cut = (total * a.nkv + kItemsPerCta * gridDim.x - 1) / (kItemsPerCta * gridDim.x);
    const int chunk = (int)max((int64_t)kMinChunk, min(cut, (int64_t)0x7fffffff));
    int items = 0, parts = 0;
    for (int r = r0; r < r1; ++r) {
        const int n = chunks_of(pages_of(a, r, &keys, false), chunk) * a.nkv;
        items += n;
        if (n > a.nkv) parts += n;
    }
    {
        const int pi = warp_prefix(items, lane), pp = warp_prefix(parts, lane);
        __syncthreads();
        if (lane == 31 && warp < kWarps) s.scan[warp] = (int64_t)pi << 32 | (uint32_t)pp;
        __syncthreads();
        int bi = 0, bp = 0;
        for (int w = 0; w < min(warp, kWarps); ++w) {
            bi += (int)(s.scan[w] >> 32);
            bp += (int)s.scan[w];
        }
        if (tid < kSpans) {
            s.item_start[tid + 1] = bi + pi;
            s.part_start[tid + 1] = bp + pp;
        }
        if (tid == 0) s.item_start[0] = s.part_start[0] = 0;
        __syncthreads();
    }
    const int all_items = s.item_start[kSpans];

    if (warp == kWarps) {
        // ------------------------------------------------------------ loader
        const uint64_t policy = l2_policy_evict_first();
        uint32_t issued = 0;  // tiles issued to consumer warp `lane` (lane < kWarps)
        int item = blockIdx.x, k = 0;
        bool ok = true;
        for (;; ++k) {
            const int slot = k % kItemSlots;
            if (k >= kItemSlots) ok = wait_warp(&s.item_empty[slot], (k / kItemSlots - 1) & 1, abort_flag, a.status);
            if (!ok) break;
            Item it;
            it.r = -1;
            int next = 0;
            if (item < all_items) {
                if (lane == 0) next = atomicAdd(a.claim, 1) + (int)gridDim.x;
                // the span, by 32 and 8 of its starts; then its requests, 32 at a time
                int span = __popc(__ballot_sync(0xffffffffu, s.item_start[lane * (kSpans / 32)] <= item)) - 1;
                span *= kSpans / 32;
                span += __popc(__ballot_sync(0xffffffffu, lane < kSpans / 32 && s.item_start[span + lane] <= item)) - 1;
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
            if (it.r < 0) break;
            int ids = lane < it.pages ? a.indices[it.first + lane] : 0, ids_next = 0;
            for (int j = 0; j * kWarps < it.pages; ++j) {
                const int sub = (j * kWarps) & 31;
                if (sub == 0) {
                    if (j) ids = ids_next;
                    const int p = j * kWarps + 32 + lane;
                    ids_next = p < it.pages ? a.indices[it.first + p] : 0;
                }
                const int page = __shfl_sync(0xffffffffu, ids, sub + (lane & (kWarps - 1)));
                bool fine = true;
                if (lane < kWarps && j * kWarps + lane < it.pages) {
                    const int st = issued % kStages;
                    if (issued >= kStages)
                        fine = mbar_wait(&s.empty[lane][st], (issued / kStages - 1) & 1, abort_flag, a.status);
                    if (fine) {
                        const bool in = (unsigned)page < (unsigned)a.num_pages;
                        s.skip[lane][st] = !in;
                        if (in) {
                            mbar_arrive_expect_tx(&s.full[lane][st], S::kHead);
                            bulk_load_hint(s.ring[lane][st], a.pool + ((int64_t)page * a.nkv + it.h) * S::kHead, S::kHead,
                                           &s.full[lane][st], policy);
                        } else {
                            set_status(a.status, NF_ERR_DEVICE_BOUNDS);
                            mbar_arrive(&s.full[lane][st]);
                        }
                        ++issued;
                    }
                }
                ok = __all_sync(0xffffffffu, fine);
                if (!ok) break;
            }
            if (!ok) {
                ++k;
                break;
            }
            item = __shfl_sync(0xffffffffu, next, 0);
        }
        if (*abort_flag) {  // the copies in flight land before the memory is given up
            int none = 0;
            if (lane < kWarps)
                for (uint32_t i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
                    mbar_wait(&s.full[lane][i % kStages], (i / kStages) & 1, &none, a.status);
            if (lane == 0)
                for (int i = k > kItemSlots ? k - kItemSlots : 0; i < k; ++i)
                    mbar_wait(&s.item_full[i % kItemSlots], (i / kItemSlots) & 1, &none, a.status);
        }
    } else {
        // ------------------------------------------------------------ consumers
        const int gid = lane >> 2, tig = lane & 3;
        uint32_t used = 0;  // tiles of this warp so far
        for (int k = 0;; ++k) {
            const int slot = k % kItemSlots;
            bool ok = wait_warp(&s.item_full[slot], (k / kItemSlots) & 1, abort_flag, a.status);
            Item it;
            it.r = -1;
            if (ok) it = s.item[slot];
            float O[NG][2][4], M0 = -INFINITY, M1 = -INFINITY, l0 = 0.f, l1 = 0.f, f[NG];
#pragma unroll
            for (int u = 0; u < NG; ++u) {
                f[u] = 0x1p100f;
#pragma unroll
                for (int i = 0; i < 4; ++i) O[u][0][i] = O[u][1][i] = 0.f;
            }
            if (ok && it.r >= 0) {
                // q of head gid, columns 32 j + 8 t .. + 7, as fp16 times 2^(14 - e), 2^e the row's largest
                uint32_t qf[NG][4];
                float start[NG][2], hs0, hs1;
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
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.item_empty[slot]);
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // exponent field; rows of zeros or subnormals count as 1, infinities and NaN as 254
                    const int ex = min(max((int)(top >> 7), 1), 254);
                    // 2^(14 - (ex - 127)) in two steps, either a normal number
                    const int up = 14 + 127 - ex, up0 = up / 2, up1 = up - up0;
                    const float m0 = __int_as_float((127 + up0) << 23), m1 = __int_as_float((127 + up1) << 23);
                    const float hs = a.scale_log2 * 64.f * __int_as_float((127 - up0) << 23) *
                                     __int_as_float((127 - up1) << 23);
                    hs0 = __shfl_sync(0xffffffffu, hs, 8 * tig);
                    hs1 = __shfl_sync(0xffffffffu, hs, 8 * tig + 4);
#pragma unroll
                    for (int j = 0; j < NG; ++j) {
                        const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
                        float sum_q = 0.f;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float lo = __uint_as_float(w[i] << 16) * m0 * m1;
                            const float hi = __uint_as_float(w[i] & 0xFFFF0000u) * m0 * m1;
                            qf[j][i] = pack_f16x2(lo, hi);
                            const __half2 back = *reinterpret_cast<__half2*>(&qf[j][i]);
                            sum_q += __low2float(back) + __high2float(back);
                        }
                        sum_q += __shfl_xor_sync(0xffffffffu, sum_q, 1);
                        sum_q += __shfl_xor_sync(0xffffffffu, sum_q, 2);
                        start[j][0] = -1.125f * __shfl_sync(0xffffffffu, sum_q, 8 * tig);
                        start[j][1] = -1.125f * __shfl_sync(0xffffffffu, sum_q, 8 * tig + 4);
                    }
                }
                for (int p = warp; p < it.pages; p += kWarps, ++used) {
                    const int st = used % kStages;
                    ok = wait_warp(&s.full[warp][st], (used / kStages) & 1, abort_flag, a.status);
                    if (!ok) break;
                    const bool skip = s.skip[warp][st] != 0;
                    const uint8_t* tile = s.ring[warp][st];
                    float x[4] = {0.f, 0.f, 0.f, 0.f};
                    if (!skip) {
                        uint32_t ka[NG], kb[NG];
                        float sa[NG], sb[NG];
                        load_words<NG>(tile + lane * (D / 8), ka);            // slot gid
                        load_words<NG>(tile + 4 * D + lane * (D / 8), kb);    // slot gid + 8
                        load_scales<NG>(tile + 8 * D + gid * (2 * NG), sa);
                        load_scales<NG>(tile + 8 * D + (gid + 8) * (2 * NG), sb);
#pragma unroll
                        for (int j = 0; j < NG; ++j) {
                            uint32_t ea[4], eb[4];
                            unpack4(ka[j], ea);
                            unpack4(kb[j], eb);
                            const uint32_t a0[4] = {ea[0], eb[0], ea[1], eb[1]}, a1[4] = {ea[2], eb[2], ea[3], eb[3]};
                            const float c[4] = {start[j][0], start[j][1], start[j][0], start[j][1]};
                            float acc[4];
                            mma_f16(acc, a0, qf[j][0], qf[j][1], c);
                            mma_f16(acc, a1, qf[j][2], qf[j][3], acc);
                            x[0] = fmaf(sa[j], acc[0], x[0]);
                            x[1] = fmaf(sa[j], acc[1], x[1]);
                            x[2] = fmaf(sb[j], acc[2], x[2]);
                            x[3] = fmaf(sb[j], acc[3], x[3]);
                        }
                        x[0] *= hs0;
                        x[1] *= hs1;
                        x[2] *= hs0;
                        x[3] *= hs1;
                    }
                    uint32_t va[NG], vb[NG];
                    float ta[NG], tb[NG];
                    if (!skip) {
                        const uint8_t* v = tile + 9 * D;
                        load_words<NG>(v + (tig * 8 + gid) * (D / 8), va);          // slots 2 t, 2 t + 1
                        load_words<NG>(v + 4 * D + (tig * 8 + gid) * (D / 8), vb);  // slots 2 t + 8, 2 t + 9
                        load_scales<NG>(v + 8 * D + gid * (2 * NG), ta);
                        load_scales<NG>(v + 8 * D + (gid + 8) * (2 * NG), tb);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.empty[warp][st]);
                    if (skip) continue;
                    const int valid = it.keys - p * kKv4Slots;
                    if (valid < kKv4Slots) {  // the request's last page: slots behind its length hold anything
                        if (gid >= valid) {
                            x[0] = x[1] = -INFINITY;
#pragma unroll
                            for (int u = 0; u < NG; ++u) ta[u] = 0.f;
                        }
                        if (gid + 8 >= valid) {
                            x[2] = x[3] = -INFINITY;
#pragma unroll
                            for (int u = 0; u < NG; ++u) tb[u] = 0.f;
                        }
                    }
                    float grown = 0.f;
#pragma unroll
                    for (int u = 0; u < NG; ++u) grown = fmaxf(grown, fmaxf(fabsf(ta[u]), fabsf(tb[u])) * f[u]);
                    const bool over = grown >= 1024.f || fmaxf(x[0], x[2]) - M0 > 5.f || fmaxf(x[1], x[3]) - M1 > 5.f;
                    if (__any_sync(0xffffffffu, over)) {
                        float n0 = fmaxf(x[0], x[2]), n1 = fmaxf(x[1], x[3]), top[NG];
#pragma unroll
                        for (int u = 0; u < NG; ++u) top[u] = fmaxf(fabsf(ta[u]), fabsf(tb[u]));
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) {
                            n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, o));
                            n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, o));
#pragma unroll
                            for (int u = 0; u < NG; ++u)
                                top[u] = fmaxf(top[u], __shfl_xor_sync(0xffffffffu, top[u], o));
                        }
                        n0 = softmax_max_update(M0, n0);
                        n1 = softmax_max_update(M1, n1);
                        const float c0 = M0 == n0 ? 1.f : exp2f(M0 - n0), c1 = M1 == n1 ? 1.f : exp2f(M1 - n1);
                        M0 = n0;
                        M1 = n1;
                        l0 *= c0;
                        l1 *= c1;
#pragma unroll
                        for (int u = 0; u < NG; ++u) {
                            float g = 1.f;
                            if (top[u] * f[u] >= 1024.f) {  // the new largest scale comes to [2^8, 2^9)
                                const int e = (int)(__float_as_uint(top[u]) >> 23);
                                const float fn = __int_as_float(min(max(254 + 8 - e, 1), 254) << 23);
                                g = fn / f[u];
                                f[u] = fn;
                            }
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                O[u][i][0] *= c0 * g;
                                O[u][i][1] *= c1 * g;
                                O[u][i][2] *= c0 * g;
                                O[u][i][3] *= c1 * g;
                            }
                        }
                    }
                    x[0] = ex2_approx(x[0] - M0);
                    x[1] = ex2_approx(x[1] - M1);
                    x[2] = ex2_approx(x[2] - M0);
                    x[3] = ex2_approx(x[3] - M1);
                    l0 += x[0] + x[2];
                    l1 += x[1] + x[3];
#pragma unroll
                    for (int u = 0; u < NG; ++u) {
                        const float pa = ta[u] * f[u], pb = tb[u] * f[u];
                        const uint32_t b0 = movmatrix_trans(pack_f16x2(x[0] * pa, x[1] * pa));
                        const uint32_t b1 = movmatrix_trans(pack_f16x2(x[2] * pb, x[3] * pb));
                        uint32_t ea[4], eb[4];
                        unpack4(va[u], ea);
                        unpack4(vb[u], eb);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            ea[i] = sub_f16x2(ea[i], 0x3C803C80u);  // 1.125: (code - 8) / 64, exact
                            eb[i] = sub_f16x2(eb[i], 0x3C803C80u);
                        }
                        const uint32_t a0[4] = {ea[0], ea[1], eb[0], eb[1]}, a1[4] = {ea[2], ea[3], eb[2], eb[3]};
                        mma_f16(O[u][0], a0, b0, b1, O[u][0]);
                        mma_f16(O[u][1], a1, b0, b1, O[u][1]);
                    }
                }
            }
            // --- join the warps. One barrier per round for every consumer, whatever happened: a wait that gave up
            // (in any warp) ends all of them here. It also tells that the previous item's sums have been read.
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                l0 += __shfl_xor_sync(0xffffffffu, l0, o);
                l1 += __shfl_xor_sync(0xffffffffu, l1, o);
            }
            if (bar_red_or(1, kConsumers, !ok)) break;
            if (it.r < 0) break;
            if (gid == 0) {
                s.ml[warp][2 * tig] = make_float2(M0, l0);
                s.ml[warp][2 * tig + 1] = make_float2(M1, l1);
            }
#pragma unroll
            for (int u = 0; u < NG; ++u) {
                const float g = 64.f / f[u];
                const int col = 32 * u + 4 * gid;
                if (2 * tig < a.G)
                    *reinterpret_cast<float4*>(&s.merge[warp][2 * tig][col]) =
                        make_float4(O[u][0][0] * g, O[u][0][2] * g, O[u][1][0] * g, O[u][1][2] * g);
                if (2 * tig + 1 < a.G)
                    *reinterpret_cast<float4*>(&s.merge[warp][2 * tig + 1][col]) =
                        make_float4(O[u][0][1] * g, O[u][0][3] * g, O[u][1][1] * g, O[u][1][3] * g);
            }
            bar_sync_n(2, kConsumers);
            // thread -> 4 columns of one head
            const int head = tid / (D / 4), col = tid % (D / 4) * 4;
            const bool mine = head < a.G;
            float M = -INFINITY, L = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            if (mine) {
#pragma unroll
                for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s.ml[w][head].x);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float2 ml = s.ml[w][head];
                    const float c = part_factor(ml.x, M);
                    const float4 v = *reinterpret_cast<const float4*>(&s.merge[w][head][col]);
                    L += c * ml.y;
                    o.x += c * v.x;
                    o.y += c * v.y;
                    o.z += c * v.z;
                    o.w += c * v.w;
                }
            }
            if (it.chunks > 1) {
                const int64_t part = (int64_t)it.part + (int64_t)it.c * a.nkv;
                if (mine) {
                    __stcg(reinterpret_cast<float4*>(a.part_o + (part * a.G + head) * D + col), o);
                    if (col == 0) __stcg(a.part_ml + part * kMaxGroup + head, make_float2(M, L));
                }
                __threadfence();
                bar_sync_n(2, kConsumers);
                if (tid == 0) {
                    const int n = atomicAdd(a.arrived + it.part, 1);
                    s.last = n == it.chunks - 1;
                    if (s.last) a.arrived[it.part] = 0;
                }
                bar_sync_n(2, kConsumers);
                if (!s.last) continue;
                __threadfence();
                if (mine) {
                    const float2* ml = a.part_ml + (int64_t)it.part * kMaxGroup + head;
                    const float* po = a.part_o + ((int64_t)it.part * a.G + head) * D + col;
                    const int64_t step = (int64_t)a.nkv * a.G * D;
                    M = -INFINITY;
                    for (int c = 0; c < it.chunks; ++c) M = fmaxf(M, __ldcg(ml + (int64_t)c * a.nkv * kMaxGroup).x);
                    L = 0.f;
                    o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
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
                }
            }
            if (mine) {
                const float inv = L == 0.f ? 0.f : 1.f / L;
                *reinterpret_cast<uint2*>(a.out + it.r * a.out_stride + (int64_t)(it.h * a.G + head) * D + col) =
                    make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
            }
        }
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
    if (num_pages < 1 || num_pages > NF_KV4_MAX_PAGES || num_requests < 0 || num_requests > NF_KV4_MAX_REQUESTS ||
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
                            num_requests, n_kv_heads, G, (float)(scale * 1.4426950408889634),
                            reinterpret_cast<int*>(w), reinterpret_cast<int*>(w) + 32,
                            reinterpret_cast<int*>(w + at.arrived), reinterpret_cast<float2*>(w + at.ml),
                            reinterpret_cast<float*>(w + at.o), status_device};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = head_dim == 64 ? nf::launch<64>(a, grid, s) : nf::launch<128>(a, grid, s);
    return e == cudaSuccess ? NF_OK : NF_ERR_CUDA;
} catch (...) {
    return NF_ERR_INVALID_ARGUMENT;
}
