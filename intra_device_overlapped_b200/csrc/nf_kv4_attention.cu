// Paged GQA decode attention over the 4-bit cache (format: nf_kv4.h).
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "nanoflow.h"
#include "nf_internal.h"
#include "nf_kv4.h"

namespace nf {
namespace {

constexpr int kMaxGroup = 8;               // query heads per KV head: the N = 8 columns of the tensor instruction
constexpr int kWarps = 16;                 // one CTA per SM, 128 registers a thread
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 2;                 // pairs of tiles in flight per warp
constexpr int kMaxCtas = 160;              // sizes the workspace (a B200 has 148 SMs)
constexpr int kMinShare = 4;               // places of a worker at least (Deal)
constexpr int kOverhead = 8;              // what beginning and ending a (request, head) costs, in pages
constexpr int kJoin = 64, kJoinPart = 6;   // what a join by a warp costs, and each of its parts, in pages of a CTA
constexpr uint32_t kNoScale = 0x7180;     // (Output, below) f = 2^100: any scale outgrows it
constexpr int kMaxParts = 2 * kWarps * kMaxCtas;

struct Kv4AttnArgs {
    const uint16_t* q;
    uint16_t* out;
    int64_t q_stride, out_stride;
    const uint8_t* pool;
    int num_pages;
    const int *kv_len, *indptr, *indices;
    int R, nkv, G;
    float scale_log2;
    int* arrived;        // [kMaxParts] parts of a (request, head) written so far, at its first part. 0 between calls
    float2* part_ml;     // [kMaxParts][kMaxGroup] maximum and sum
    float* part_o;       // [kMaxParts][G][D]
    int* status;
};

// A worker's stretch of one (request, KV head)
struct Item {
    int r, h;       // r = -1: none
    int first;      // place of its first page in page_indices
    int pages, keys;
    int parts, c;   // stretches of this (request, head), which of them this is
    int slot;       // of its part 0; part c > 0 has slot + 2 c - 1
};

__device__ __forceinline__ int part_slot(const Item& it, int c) { return c ? it.slot + 2 * c - 1 : it.slot; }

// a / b of numbers from 0 on (the division of 64 bits takes about as long as a load from L2)
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
    return (a | b) >> 32 ? a / b : (uint32_t)a / (uint32_t)b;
}

// How the pages are dealt: every (request, KV head) takes a number of places in one long order, worker w places
// [w share, (w + 1) share). Warps as workers: a pair takes kOverhead places and one a page. CTAs ("team"): one place for
// each `chunk` pages or less, and a share is one place.
struct Deal {
    int64_t total, share;
    int chunk;  // 0: warps
    __device__ __forceinline__ int64_t places(int pages) const {
        return pages == 0 ? 0 : chunk ? (pages + chunk - 1) / chunk : (int64_t)pages + kOverhead;
    }
    __device__ __forceinline__ int worker_of(int64_t pos) const {
        return (int)divide(pos, share);
    }
};

template <int D>
struct Smem {
    static constexpr int kHead = 18 * D;            // K and V tile of a head
    static constexpr int kRow = D + 4;              // merge rows, padded against bank conflicts
    alignas(128) uint8_t ring[kWarps][kStages][2 * kHead];
    // rows of a team's warp: in the memory of its ring, which has done by then
    __device__ __forceinline__ float* merge(int warp, int h) { return reinterpret_cast<float*>(ring[warp][0]) + h * kRow; }
    alignas(16) uint16_t q[kWarps][2][kMaxGroup * D];
    uint4 bias[kWarps][32];  // a lane's two bias operands, its heads' factors of scores
    Item item[kWarps][2], pending[kWarps][2];
    float2 ml[kWarps][kMaxGroup];
    int64_t scan[kWarps], start[kThreads + 1];
    int64_t pos[kWarps];  // the place where the warp's next stretch begins
    Deal deal;
    int last[2];
    int4 rest[kWarps];  // what exact_rest goes on from: k, ahead, more, pending
};

// Pages that request r reads: its keys, cut to what its row of the page table holds; *at: where the row begins.
__device__ __forceinline__ int pages_of(const Kv4AttnArgs& a, int r, int* keys, int* at, bool report) {
    const int p0 = *at = a.indptr[r];
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

__device__ __forceinline__ int64_t warp_prefix(int64_t x, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// D = A B + C of 16 x 16 by 16 x 8, fp16 in, fp32 out
__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1, const float* c) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// the same in bf16, C = 0
__device__ __forceinline__ void mma_bf16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    const float z = 0.f;
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z));
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

// Codes of four pairs as fp16, nibble p of both halves of w as the last bits of a subnormal number: 2^-24 code for the
// even nibbles, which spare a shift, 2^-20 code for the odd ones. kExact takes the bias off: 2^-24 (code - 8) and
// 2^-20 (code - 8), exactly. (Under the exponent of 1 the bias would be 1032 and 72 codes, not 8.)
template <bool kExact>
__device__ __forceinline__ void unpack4(uint32_t w, uint32_t* e) {
    constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u;
    const uint32_t t = w >> 8;
    e[0] = w & kLow;
    e[1] = w & kHigh;
    e[2] = t & kLow;
    e[3] = t & kHigh;
    if constexpr (kExact) {
        e[0] = sub_f16x2(e[0], 0x00080008u);
        e[1] = sub_f16x2(e[1], 0x00800080u);
        e[2] = sub_f16x2(e[2], 0x00080008u);
        e[3] = sub_f16x2(e[3], 0x00800080u);
    }
}

// Transpose of an 8 x 8 matrix of 16-bit values (two of a row to a lane)
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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

// The whole warp: its next stretch, from s.pos to the end of a (request, head) or of the worker's share. r = -1: without
// pages (s.pos in the overhead before the end of the share). Returns whether the share goes on behind it. Kept out of line
// and its state in shared memory: it runs once a stretch and would cost the tile loop registers.
template <int D>
__device__ __noinline__ bool find_item(const Kv4AttnArgs& a, Smem<D>& s, Item* out) {
    const Deal& deal = s.deal;
    const int warp = threadIdx.x >> 5, worker = deal.chunk ? blockIdx.x : blockIdx.x * kWarps + warp;
    const int per = (a.R + kThreads - 1) / kThreads;
    const int64_t pos = s.pos[warp], stop = min(deal.total, (worker + 1) * deal.share);
    const int lane = threadIdx.x & 31;
    Item it;
    it.r = -1;
    int64_t next = stop;
    // the thread's stretch of requests that holds the place, by 32 and then kSub of their starts; then the request
    constexpr int kSub = kThreads / 32;
    int span = (__popc(__ballot_sync(0xffffffffu, s.start[lane * kSub] <= pos)) - 1) * kSub;
    span += __popc(__ballot_sync(0xffffffffu, lane < kSub && s.start[span + min(lane, kSub - 1)] <= pos)) - 1;
    int64_t at = s.start[span];
    const int end = min(a.R, (span + 1) * per);
    for (int r = span * per; r < end; r += 32) {
        int keys = 0, pages = 0, row = 0;
        if (r + lane < end) pages = pages_of(a, r + lane, &keys, &row, false);
        int64_t places = deal.places(pages);
        const int64_t upto = at + warp_prefix(places * a.nkv, lane);
        const uint32_t past = __ballot_sync(0xffffffffu, upto > pos);
        if (past) {
            const int src = __ffs(past) - 1;
            pages = __shfl_sync(0xffffffffu, pages, src);
            keys = __shfl_sync(0xffffffffu, keys, src);
            row = __shfl_sync(0xffffffffu, row, src);
            places = __shfl_sync(0xffffffffu, places, src);
            const int64_t begin = __shfl_sync(0xffffffffu, upto, src) - places * a.nkv;
            int h = -1;  // the last head that begins at or before pos
            for (int h0 = 0; h0 < a.nkv; h0 += 32)
                h += __popc(__ballot_sync(0xffffffffu, h0 + lane < a.nkv && begin + (h0 + lane) * places <= pos));
            const int64_t u0 = begin + h * places;
            int b, e;  // pages of the stretch
            if (deal.chunk) {
                it.parts = (int)places;
                it.c = (int)(pos - u0);
                b = (int)((int64_t)pages * it.c / it.parts);
                e = (int)((int64_t)pages * (it.c + 1) / it.parts);
                next = pos + 1;
            } else {
                const int64_t p0 = u0 + kOverhead, p1 = p0 + pages;
                b = (int)max(pos - p0, (int64_t)0);
                e = (int)(min(p1, stop) - p0);  // negative where stop lies in the overhead
                next = min(p1, stop);
                const int w0 = pos <= p0 ? worker : deal.worker_of(p0);
                it.c = worker - w0;
                it.parts = (p1 <= stop ? worker : deal.worker_of(p1 - 1)) - w0 + 1;
            }
            if (b < e) {
                it.r = r + src;
                it.h = h;
                it.first = row + b;
                it.pages = e - b;
                it.keys = min(keys - b * kKv4Slots, it.pages * kKv4Slots);
                it.slot = 2 * (worker - it.c) + 1;
            }
            break;
        }
        at = __shfl_sync(0xffffffffu, upto, 31);
    }
    __syncwarp();  // (all have read s.pos)
    if (lane == 0) {
        *out = it;
        s.pos[warp] = next;
    }
    __syncwarp();
    return next < stop;
}

// 4 columns of a head's output row from its sums
__device__ __forceinline__ void store_out(const Kv4AttnArgs& a, const Item& it, int d, int h, int col, float4 o, float L) {
    const float inv = L == 0.f ? 0.f : 1.f / L;
    *reinterpret_cast<uint2*>(a.out + it.r * a.out_stride + (int64_t)(it.h * a.G + h) * d + col) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}

// A number 0..15 less 8 (no conversion instruction)
__device__ __forceinline__ float code_of(uint32_t nibble) {
    return __uint_as_float((nibble & 15u) | 0x4B000000u) - 8388616.f;
}

// The sums of a stretch (its pages `offset` and `offset` + 1 of every `step`) in fp32 throughout, to the team's memory,
// the output or the workspace. A key at a time, read from the pool again: lane (g, t) takes columns 4 g .. 4 g + 3 of
// each group for heads 2 t and 2 t + 1, in scores and output alike. About 300 instructions a key, where the tensor
// instructions' loop takes 19.
template <int D>
__device__ __forceinline__ void exact_sums(const Kv4AttnArgs& a, Smem<D>& sm, const Item& it, int offset, int step) {
    constexpr int NG = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, h0 = 2 * (lane & 3);
    uint2 q[2][NG];
    float m[2], hs[2], M[2], l[2], sum[2][NG][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint16_t* const row = a.q + it.r * a.q_stride + (int64_t)(it.h * a.G + min(h0 + i, a.G - 1)) * D + 4 * gid;
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            q[i][j] = *reinterpret_cast<const uint2*>(row + 32 * j);
            top = max(top, max(max(q[i][j].x & 0x7FFFu, q[i][j].x >> 16 & 0x7FFFu),
                               max(q[i][j].y & 0x7FFFu, q[i][j].y >> 16 & 0x7FFFu)));
            sum[i][j][0] = sum[i][j][1] = sum[i][j][2] = sum[i][j][3] = 0.f;
        }
#pragma unroll
        for (int of = 4; of < 32; of <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, of));
        // q over 2^e, its row's largest or nearly so, as at the kernel
        const int ex = min(max((int)(top >> 7), 1), 253);
        m[i] = __int_as_float((254 - ex) << 23);
        hs[i] = fminf(fmaxf(a.scale_log2 * __int_as_float(ex << 23), 0x1p-140f), 0x1p127f);
        M[i] = -INFINITY;
        l[i] = 0.f;
    }
#pragma unroll 1
    for (int p = offset; p < it.pages; p += p & 1 ? step - 1 : 1) {  // (offset is even)
        const int id = __ldg(a.indices + it.first + p);
        if ((unsigned)id >= (unsigned)a.num_pages) continue;
        const uint8_t* const kt = a.pool + ((int64_t)id * a.nkv + it.h) * (18 * D);
        const uint8_t* const vt = kt + 9 * D;
        const int n = min(it.keys - p * kKv4Slots, kKv4Slots);
#pragma unroll 1
        for (int s = 0; s < n; ++s) {
            uint32_t kw[NG], ks[NG / 2], vw[NG], vs[NG / 2];
            load_words<NG>(kt + s * (D / 2) + (gid >> 1) * (D / 8), kw);
            load_scales<NG>(kt + 8 * D + s * (2 * NG), ks);
            load_words<NG>(vt + (s >> 3) * 4 * D + ((s & 7) >> 1) * D + gid * (D / 8), vw);
            load_scales<NG>(vt + 8 * D + s * (2 * NG), vs);
            float x[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const uint32_t v = kw[j] >> 8 * (gid & 1);
                const float c0 = code_of(v), c1 = code_of(v >> 16), c2 = code_of(v >> 4), c3 = code_of(v >> 20);
                const float g = j % 2 ? hi_bf16(ks[j / 2]) : lo_bf16(ks[j / 2]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float dot = lo_bf16(q[i][j].x) * m[i] * c0;
                    dot = fmaf(hi_bf16(q[i][j].x) * m[i], c1, dot);
                    dot = fmaf(lo_bf16(q[i][j].y) * m[i], c2, dot);
                    dot = fmaf(hi_bf16(q[i][j].y) * m[i], c3, dot);
                    x[i] = fmaf(g, dot, x[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int of = 4; of < 32; of <<= 1) x[i] += __shfl_xor_sync(0xffffffffu, x[i], of);
                x[i] = __fmul_rn(x[i], hs[i]);
                const float now = softmax_max_update(M[i], x[i]);
                if (now != M[i]) {
                    const float c = ex2_approx(M[i] - now);
                    M[i] = now;
                    l[i] *= c;
#pragma unroll
                    for (int j = 0; j < NG; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sum[i][j][e] *= c;
                }
                x[i] = x[i] == -INFINITY ? 0.f : ex2_approx(x[i] - M[i]);
                l[i] += x[i];
            }
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const uint32_t v = vw[j] >> 16 * (s & 1);
                const float g = j % 2 ? hi_bf16(vs[j / 2]) : lo_bf16(vs[j / 2]);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[i][j][e] = fmaf(x[i] * g, code_of(v >> 4 * e), sum[i][j][e]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int h = h0 + i;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const int col = 32 * j + 4 * gid;
            const float4 o = make_float4(sum[i][j][0], sum[i][j][1], sum[i][j][2], sum[i][j][3]);
            if (sm.deal.chunk)
                *reinterpret_cast<float4*>(sm.merge(warp, h) + col) = o;
            else if (h < a.G && it.parts == 1)
                store_out(a, it, D, h, col, o, l[i]);
            else if (h < a.G)
                __stcg(reinterpret_cast<float4*>(a.part_o + ((int64_t)part_slot(it, it.c) * a.G + h) * D + col), o);
        }
        if (gid == 0 && sm.deal.chunk)
            sm.ml[warp][h] = make_float2(M[i], l[i]);
        else if (gid == 0 && it.parts > 1)
            __stcg(a.part_ml + (int64_t)part_slot(it, it.c) * kMaxGroup + h, make_float2(M[i], l[i]));
    }
}

// The rest of the warp's share by exact_sums, from a stretch on whose fp16 weights or q may have lost something (Scores
// and Output, at the kernel). Returns the parts to be reported. The warp does not come back to the tensor instructions:
// kept alive across this call, the state of their loop cost registers, and 512 requests of 1280 keys 6 % of their time.
template <int D>
__device__ __noinline__ int exact_rest(const Kv4AttnArgs& a, Smem<D>& s) {
    const int warp = threadIdx.x >> 5;
    int k = s.rest[warp].x, ahead = s.rest[warp].y, pending = s.rest[warp].w;
    bool more = s.rest[warp].z;
    const int offset = s.deal.chunk ? 2 * warp : 0, step = s.deal.chunk ? 2 * kWarps : 2;
#pragma unroll 1
    for (;; ++k) {
        Item& it = s.item[warp][k & 1];
        if (k == ahead) {
            do {
                if (!more) return pending;
                more = find_item<D>(a, s, &it);
            } while (it.r < 0);
            ++ahead;
        }
        exact_sums<D>(a, s, it, offset, step);
        if (it.parts > 1) {
            if ((threadIdx.x & 31) == 0) s.pending[warp][pending] = it;
            ++pending;
        }
        __syncwarp();
    }
}

// Parts of a (request, head), joined in order into the output by one warp: heads h0 .. h0 + H - 1, 4 columns of a head
// to a lane. The weights of 32 / H parts are formed by a lane each; rows of 4 parts are loaded at a time, the first before
// the maximum is known. One body for any number of parts (the last is loaded again, with weight 0, for those that are
// missing): what a join costs is mostly code that no cache holds yet.
template <int D, int H>
__device__ __noinline__ void join_parts(const Kv4AttnArgs& a, const Item& it, int h0) {
    constexpr int kRows = 128 / D, kAtOnce = 32 / H;  // heads that the lanes cover at a time; parts a round
    static_assert(kAtOnce % 4 == 0, "rows of 4 parts at a time");
    const int lane = threadIdx.x & 31, col = lane % (D / 4) * 4, row = lane / (D / 4), parts = it.parts;
    const float2* const ml = a.part_ml + h0 + lane % H;
    const float* const po = a.part_o + (int64_t)h0 * D + col;
    const int last = a.G - 1 - h0;
    auto weight_of = [&](int c) {
        return c < parts ? __ldcg(ml + (int64_t)part_slot(it, c) * kMaxGroup) : make_float2(-INFINITY, 0.f);
    };
    float4 v[4][H / kRows], o[H / kRows];
    auto load = [&](int c) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const float* at = po + (int64_t)part_slot(it, min(c + p, parts - 1)) * a.G * D;
#pragma unroll
            for (int i = 0; i < H / kRows; ++i)
                v[p][i] = __ldcg(reinterpret_cast<const float4*>(at + min(i * kRows + row, last) * D));
        }
    };
    float2 m = weight_of(lane / H);
    load(0);
    float M = m.x, L = 0.f;
#pragma unroll 1
    for (int c = kAtOnce + lane / H; c < parts; c += kAtOnce) M = fmaxf(M, weight_of(c).x);
#pragma unroll
    for (int of = H; of < 32; of <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, of));
#pragma unroll
    for (int i = 0; i < H / kRows; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    float w = 0.f;
#pragma unroll 1
    for (int c = 0; c < parts; c += 4) {
        if (c % kAtOnce == 0) {
            if (c) m = weight_of(c + lane / H);
            w = c + lane / H < parts ? part_factor(m.x, M) : 0.f;
            L += w * m.y;
        }
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
            for (int i = 0; i < H / kRows; ++i) {
                const float f = __shfl_sync(0xffffffffu, w, H * (c % kAtOnce + p) + i * kRows + row);
                o[i].x += f * v[p][i].x;
                o[i].y += f * v[p][i].y;
                o[i].z += f * v[p][i].z;
                o[i].w += f * v[p][i].w;
            }
        if (c + 4 < parts) load(c + 4);
    }
#pragma unroll
    for (int of = H; of < 32; of <<= 1) L += __shfl_xor_sync(0xffffffffu, L, of);
#pragma unroll
    for (int i = 0; i < H / kRows; ++i) {
        const int h = i * kRows + row;
        const float sum = __shfl_sync(0xffffffffu, L, h);
        if (h <= last) store_out(a, it, D, h0 + h, col, o[i], sum);
    }
}

// o = softmax(q K^T) V per (request, KV head), G query heads at a time, in one pass over the cache.
//
// The cache is read once, 144 bytes a key and head (d = 128), and the kernel has to turn codes into operands as
// fast as the HBM brings them: per SM one 16-key tile of K and V (2304 bytes) every 100 cycles, 400 issue slots.
// Codes become fp16 in registers, right in the operand layout of the warp-level mma (that is the order they
// are stored in): no shared-memory round trip, which tcgen05 operands would need.
//   Scores. S[key, head] = sum over groups j of s_k[key, j] * (sum over d in j of t q - b_j), t the codes as unpack4
//   leaves them, q in fp16 times a power of two per head (exact but below 2^-24 of the row's largest; columns of the
//   even nibbles times 16 for their codes' 2^-24), b_j = sum of bias times q. The scale is applied to the 16 x 8
//   accumulator of each group, 32 columns, in fp32; -sum s_k b_j for all keys and heads is one more tensor
//   instruction, the scales as stored times b_j in three bf16 terms (24 bits), and starts the sum. (Codes with their
//   bias are at most 15 where the values reach 7: the sums lose one bit to it.) A column of q is off by 2^-35 of its row's
//   largest at most. Where that is more than 2^-24 of the largest in its group, whose K may be as much larger, the stretch
//   goes to exact_rest.
//   Output. O^T[d, head] += V^T[d, key] P^T[key, head], P = 2^(x - M) s_v[key, j] f_j, a product in fp32 that is rounded
//   to fp16 once (2^-11; rounded before the product too, to form it in packed halves, 512 requests of 1280 keys take 153
//   us instead of 157), V's codes exact (their bias would meet the sum of all weights, which grows with the length while
//   the result does not). f_j, a power of two that follows the largest scale of the group so far, and M, the integral
//   running maximum of the head, keep P below 2^15; both move only when a value has outgrown them (2^5 and 2^2 of slack),
//   which one vote per two tiles detects. P goes from accumulator to operand layout by movmatrix.
//   P is 2^-25 off at most where it is below fp16's normal numbers, and counts for nothing below that: with scales far
//   from one another, or zeros, at the keys that weigh most, this may be all that a head gets from a group. So a stretch
//   of n keys is taken for good where, for each head and group with any scale, the largest of the 32 sums is n 2^-10 in P's
//   units or more (2^6 from 2^16 keys on): what is lost, at most n 2^-25 times 7, is then 2^-12 of it (n 2^-28). In a head
//   whose heaviest key has the largest scale P reaches 2^7 and its sums 7 times that. Otherwise the warp takes this stretch,
//   and the rest of its share, in fp32 (exact_rest): 15 times the time. The comparison costs 0.6 us of 165.
// Sums and statistics are fp32. M0, M1 etc. belong to the two head columns 2 t, 2 t + 1 of a lane.
//
// Work. Each CTA scans the lengths itself (no second launch, nothing on the host depends on them). With many (request,
// KV head) pairs a worker is a warp: the pages of all pairs, in order, are dealt to the warps (Deal), so that a share
// covers some pairs whole and one at either end in part; no barrier, nothing shared. With fewer pairs
// than CTAs a worker may be a CTA ("team"): a pair is cut into equal chunks of at most pages / (CTAs - pairs), no more than
// there are CTAs, whose pages go round the warps by twos and whose sums meet in shared memory. That costs balance and
// saves joins of many parts by one warp: 64 query heads on 8 KV heads, 8193 keys each, 1 request 16 us (warps as workers:
// 68), 4 19.5 (37), 9 27 (37), 18 39.6 (49.7). A team is taken where its largest chunk is less than an equal share and
// what the joins cost. Every warp keeps its own ring of
// tiles full with cp.async (waits are for its own copies only) and runs up to one stretch ahead of the one it works on.
// Parts of one pair meet in the workspace; a worker reports its parts, two at most, when its share is done, and whoever
// brings the last one joins them, in order.
//
// Measured, calls back to back: 512 requests of 1024 to 1536 keys, 32 query and 8 KV heads of 128: 157-165 us on different
// B200s, 0.70-0.74 of a copy of the 761 MB; of 1 to 2048 keys 101 us (0.67); 2 of 131072 keys with 64 query heads 69 us
// (0.64). What bounds it is the turning of codes into operands: about 320 instructions a tile, 66 % of the issue slots and
// 52 % of the logic pipe in use, with 4 warps a scheduler to cover latencies. To fit 128 registers (12 bytes are spilled)
// q's operands are read from shared memory again for every tile; 12 warps of 168 registers hold them and took 3 % more.
template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_attention_kernel(const __grid_constant__ Kv4AttnArgs a) {
    constexpr int NG = D / 32, NW = NG / 2;
    using S = Smem<D>;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    S& s = *reinterpret_cast<S*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    // --- the batch: how its pages are dealt, and the places before each thread's requests
    const int per = (a.R + kThreads - 1) / kThreads;
    {
        int workers = gridDim.x * kWarps;
        const int r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
        Deal d;
        d.chunk = 0;
        int keys, at;
        int64_t sum = 0, upto, before;
        auto scan = [&]() {
            upto = warp_prefix(sum * a.nkv, lane);
            if (lane == 31) s.scan[warp] = upto;
            __syncthreads();
            before = d.total = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) before += s.scan[w];
                d.total += s.scan[w];
            }
            __syncthreads();
        };
        const int64_t pairs = (int64_t)a.R * a.nkv;
        if (pairs < gridDim.x) {  // (one request to a thread at most)
            const int pages = r0 < r1 ? pages_of(a, r0, &keys, &at, blockIdx.x == 0) : 0;
            sum = pages;
            scan();
            const int n = (int)pairs, others = gridDim.x - n;
            d.chunk = (int)min(max(divide(d.total + others - 1, others), (int64_t)(2 * kWarps)), (int64_t)0x7fffffff);
            // a team as long as its largest share is no more work than an equal one with the warps' joins
            const int64_t most = divide(d.total, gridDim.x) + kJoin + kJoinPart * (workers / n);
            if (__syncthreads_and(pages <= most * d.places(pages)))
                workers = gridDim.x;
            else
                d.chunk = 0;
            sum = d.places(pages);
        } else {
            for (int r = r0; r < r1; ++r) sum += d.places(pages_of(a, r, &keys, &at, blockIdx.x == 0));
        }
        scan();
        d.share = d.chunk ? 1 : max(divide(d.total + workers - 1, workers), (int64_t)kMinShare);
        s.start[tid + 1] = before + upto;
        if (tid == 0) {
            s.start[0] = 0;
            s.deal = d;
        }
        __syncthreads();
    }
    // (read again where it is used: the loop has no register for it)
    auto team = [&]() { return s.deal.chunk != 0; };
    bool more;  // of the worker's share
    {
        const int worker = team() ? blockIdx.x : blockIdx.x * kWarps + warp;
        const int64_t pos = worker * s.deal.share;
        more = pos < s.deal.total;
        if (lane == 0) s.pos[warp] = pos;
        __syncwarp();
    }

    // --- this warp's stretches and its ring of tile pairs. Pair i is pages step i + offset and the next one.
    const int step = team() ? 2 * kWarps : 2;
    auto offset = [&]() { return team() ? 2 * warp : 0; };
    static_assert(kStages == 2, "stages are told apart by one bit");
    constexpr int kStage = 2 * S::kHead;
    int flying = 0;                // pairs on their way or waiting: cp.async groups in flight at most
    uint32_t absent = 0;           // two bits a pair on its way, the next one lowest: no such page, or not of the pool
    int out_st = 0;                // offset of the stage of the next pair used
    int ahead = 0;                 // stretches begun to load; of the last of them:
    int rem = 0;                   // pages from the next pair on
    const int* idp = a.indices;    // their places in the page table
    int id = -1;                   // the page that the lane copies, fetched while the pair before is worked on
    // half a warp copies a tile: 16 bytes a lane at a time
    const int half = lane >> 4;
    const uint32_t my_ring = smem_u32(s.ring[warp]) + half * S::kHead + (lane & 15) * 16;
    const uint8_t* from = a.pool;  // the lane's first 16 bytes of the head's tile of page 0
    const int page = a.nkv * S::kHead;
    auto fetch_id = [&]() { id = rem > half ? __ldg(idp) : -1; };
    auto issue = [&]() {  // the next pair's tiles (rem > 0)
        const bool bad = (unsigned)id >= (unsigned)a.num_pages;
        const uint32_t dst = my_ring + (flying ? out_st ^ kStage : out_st);
        const uint8_t* src = from + (int64_t)id * page;
        if (!bad) {
            constexpr int kPieces = (S::kHead + 255) / 256;
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
                if (256 * i + 256 <= S::kHead || 256 * i + (lane & 15) * 16 < S::kHead)
                    cp_async(dst + 256 * i, src + 256 * i);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        const uint32_t lost = __ballot_sync(0xffffffffu, bad);
        if (lost) {
            absent |= ((lost & 1) | (lost >> 31) << 1) << 2 * flying;
            if ((lost & 1) || rem > 1) set_status(a.status, NF_ERR_DEVICE_BOUNDS);
        }
        ++flying;
        rem -= step;
        idp += step;
        fetch_id();
    };
    auto fill = [&](int working) {  // `working`: the stretch that the warp works on
        while (flying < kStages) {
            if (rem <= 0) {
                if (!more || ahead > working + 1) return;
                Item& it = s.item[warp][ahead & 1];
                more = find_item<D>(a, s, &it);
                if (it.r < 0) continue;
                ++ahead;
                rem = it.pages - offset();
                if (rem <= 0) continue;
                from = a.pool + (int64_t)it.h * S::kHead + (lane & 15) * 16;
                idp = a.indices + it.first + offset() + half;
                fetch_id();
                // q of the stretch, in one group with its first tiles
                const uint8_t* q = reinterpret_cast<const uint8_t*>(a.q + it.r * a.q_stride + (int64_t)it.h * a.G * D);
                const uint32_t dst = smem_u32(s.q[warp][(ahead - 1) & 1]);
                for (int i = lane * 16; i < a.G * D * 2; i += 512) cp_async(dst + i, q + i);
            }
            issue();
        }
    };

    const int gid = lane >> 2, tig = lane & 3;
    int pending = 0;  // parts written, to be reported
    fill(0);
    // requests without keys: zeros
    for (int r = blockIdx.x; r < a.R; r += gridDim.x) {
        int keys, at;
        if (pages_of(a, r, &keys, &at, false) == 0)
            for (int i = tid * 8; i < a.nkv * a.G * D; i += kThreads * 8)
                *reinterpret_cast<uint4*>(a.out + r * a.out_stride + i) = make_uint4(0, 0, 0, 0);
    }
    for (int k = 0;; ++k) {
        if (flying < kStages) fill(k);
        if (k >= ahead) break;
        const int keys = s.item[warp][k & 1].keys;
        float O[NG][2][4], M0 = -INFINITY, M1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        uint32_t f[NW];  // of the groups, as bf16
#pragma unroll
        for (int u = 0; u < NG; ++u) {
            f[u / 2] = kNoScale * 0x10001u;
#pragma unroll
            for (int i = 0; i < 4; ++i) O[u][0][i] = O[u][1][i] = 0.f;
        }
        bool lost = false;
        if (keys > offset() * kKv4Slots) {
            if (flying == kStages)  // the first pair, and q with it
                cp_async_wait<kStages - 1>();
            else
                cp_async_wait<0>();
            __syncwarp();
            // q of head gid, columns 32 j + 8 t .. + 7, as fp16 times 2^(10 - e), 2^e the row's largest; pairs of even
            // nibbles times 16 more
            uint4* const qf = reinterpret_cast<uint4*>(s.q[warp][k & 1]) + lane;  // in the memory of q
            {
                float sum[NG];
#pragma unroll
                for (int j = 0; j < NG; ++j) sum[j] = 0.f;
                uint4 raw[NG];
                uint32_t tops[NW] = {};  // the largest of each group
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    raw[j] = gid < a.G ? *reinterpret_cast<const uint4*>(&s.q[warp][k & 1][gid * D + 32 * j + 8 * tig])
                                       : make_uint4(0, 0, 0, 0);
                    const uint32_t both = __vmaxu2(__vmaxu2(raw[j].x & 0x7FFF7FFFu, raw[j].y & 0x7FFF7FFFu),
                                                   __vmaxu2(raw[j].z & 0x7FFF7FFFu, raw[j].w & 0x7FFF7FFFu));
                    tops[j / 2] |= max(both & 0xFFFFu, both >> 16) << 16 * (j % 2);
                }
                __syncwarp();  // all have read their q
                uint32_t top = 0;
#pragma unroll
                for (int u = 0; u < NW; ++u) {
                    tops[u] = __vmaxu2(tops[u], __shfl_xor_sync(0xffffffffu, tops[u], 1));
                    tops[u] = __vmaxu2(tops[u], __shfl_xor_sync(0xffffffffu, tops[u], 2));
                    top = max(top, max(tops[u] & 0xFFFFu, tops[u] >> 16));
                }
                // exponent field; rows of zeros or subnormals count as 1, infinities and NaN as 254
                const int ex = min(max((int)(top >> 7), 1), 254);
#pragma unroll
                for (int u = 0; u < NW; ++u) {
                    // (Scores, above) a group of small q, 2^-11 of the row's or less
                    const int lo = tops[u] & 0xFFFFu, hi = tops[u] >> 16;
                    lost |= (lo && (lo >> 7) + 11 < ex) || (hi && (hi >> 7) + 11 < ex);
                }
                lost = __any_sync(0xffffffffu, lost);
                // 2^(10 - (ex - 127)) in two steps, either a normal number
                const int up = 10 + 127 - ex, up0 = up / 2, up1 = up - up0;
                const float m0 = __int_as_float((127 + up0) << 23), m1 = __int_as_float((127 + up1) << 23);
                // Not 0, so that minus infinity times it stays that, and finite: where the upper limit is met (|q| scale of
                // 2^107 and more) scores that differ do so by 2^20 and more, with the limit as without.
                const float hs = fminf(fmaxf(a.scale_log2 * __int_as_float((127 - up0) << 23) *
                                                 __int_as_float((127 - up1) << 23) * 0x1p20f, 0x1p-140f), 0x1p127f);
                const float hs0 = __shfl_sync(0xffffffffu, hs, 8 * tig), hs1 = __shfl_sync(0xffffffffu, hs, 8 * tig + 4);
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
                    uint32_t v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float m = i % 2 ? m1 : m1 * 16.f;
                        v[i] = pack_f16x2(lo_bf16(w[i]) * m0 * m, hi_bf16(w[i]) * m0 * m);
                        const __half2 back = *reinterpret_cast<__half2*>(&v[i]);
                        sum[j] -= (__low2float(back) + __high2float(back)) * (i % 2 ? 0x1p-17f : 0x1p-21f);
                    }
                    qf[32 * j] = make_uint4(v[0], v[1], v[2], v[3]);
                    sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 1);
                    sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 2);
                }
                // -b_j of head gid in three bf16 terms, term t in rows 2 t, 2 t + 1 of the operand (groups 0, 1) and
                // 8 + 2 t, 9 + 2 t (groups 2, 3)
                auto term = [&](float lo, float hi) {
                    uint32_t w = 0;
#pragma unroll
                    for (int i = 0; i < 3; ++i) {
                        const uint32_t v = pack_bf16x2(lo, hi);
                        lo -= lo_bf16(v);
                        hi -= hi_bf16(v);
                        if (i == tig) w = v;
                    }
                    return w;
                };
                s.bias[warp][lane] = make_uint4(term(sum[0], sum[1]), NW == 2 ? term(sum[NG - 2], sum[NG - 1]) : 0,
                                                __float_as_uint(hs0), __float_as_uint(hs1));
            }
            // `left`: keys from the pair on
            for (int left = lost ? 0 : keys - offset() * kKv4Slots; left > 0; left -= step * kKv4Slots) {
                if (flying < kStages) fill(k);  // (a new stretch to begin)
                if (flying == kStages)
                    cp_async_wait<kStages - 1>();
                else
                    cp_async_wait<0>();
                __syncwarp();
                const uint8_t* tile = s.ring[warp][0] + out_st;
                const uint32_t none = absent & 3u;
                uint32_t ta[2][NW], tb[2][NW], va[NG], vb[NG];
                float y[2][4];
                auto load_v = [&](int i) {
                    const uint8_t* vt = tile + i * S::kHead + 9 * D;
                    load_words<NG>(vt + (tig * 8 + gid) * (D / 8), va);          // slots 2 t, 2 t + 1
                    load_words<NG>(vt + 4 * D + (tig * 8 + gid) * (D / 8), vb);  // slots 2 t + 8, 2 t + 9
                };
                auto add_tile = [&](float* yy, const uint32_t* tta, const uint32_t* ttb) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) yy[e] = ex2_approx(yy[e]);
                    l0 += yy[0] + yy[2];
                    l1 += yy[1] + yy[3];
#pragma unroll
                    for (int u = 0; u < NW; ++u) {
                        const uint32_t pa = mul_bf16x2(tta[u], f[u]), pb = mul_bf16x2(ttb[u], f[u]);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float ga = e ? hi_bf16(pa) : lo_bf16(pa), gb = e ? hi_bf16(pb) : lo_bf16(pb);
                            const uint32_t b0 = transpose8(pack_f16x2(yy[0] * ga, yy[1] * ga));
                            const uint32_t b1 = transpose8(pack_f16x2(yy[2] * gb, yy[3] * gb));
                            uint32_t ea[4], eb[4];
                            unpack4<true>(va[2 * u + e], ea);
                            unpack4<true>(vb[2 * u + e], eb);
                            const uint32_t a0[4] = {ea[0], ea[1], eb[0], eb[1]}, a1[4] = {ea[2], ea[3], eb[2], eb[3]};
                            mma_f16(O[2 * u + e][0], a0, b0, b1, O[2 * u + e][0]);
                            mma_f16(O[2 * u + e][1], a1, b0, b1, O[2 * u + e][1]);
                        }
                    }
                };
                if (none != 3u) {
                    float x[2][4];
                    const uint2 bias = *reinterpret_cast<const uint2*>(&s.bias[warp][lane]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint8_t* kt = tile + i * S::kHead;
                        uint32_t ka[NG], kb[NG], sa[NW], sb[NW];
                        load_words<NG>(kt + lane * (D / 8), ka);            // slot gid
                        load_words<NG>(kt + 4 * D + lane * (D / 8), kb);    // slot gid + 8
                        load_scales<NG>(kt + 8 * D + gid * (2 * NG), sa);
                        load_scales<NG>(kt + 8 * D + (gid + 8) * (2 * NG), sb);
                        mma_bf16(x[i], sa[0], sb[0], sa[NW - 1], sb[NW - 1], bias.x, bias.y);
#pragma unroll
                        for (int j = 0; j < NG; ++j) {
                            uint32_t ea[4], eb[4];
                            unpack4<false>(ka[j], ea);
                            unpack4<false>(kb[j], eb);
                            const uint32_t a0[4] = {ea[0], eb[0], ea[1], eb[1]}, a1[4] = {ea[2], eb[2], ea[3], eb[3]};
                            const float zero[4] = {0.f, 0.f, 0.f, 0.f};
                            float acc[4];
                            const uint4 qv = qf[32 * j];
                            mma_f16(acc, a0, qv.x, qv.y, zero);
                            mma_f16(acc, a1, qv.z, qv.w, acc);
                            const float ga = j % 2 ? hi_bf16(sa[j / 2]) : lo_bf16(sa[j / 2]);
                            const float gb = j % 2 ? hi_bf16(sb[j / 2]) : lo_bf16(sb[j / 2]);
                            x[i][0] = fmaf(ga, acc[0], x[i][0]);
                            x[i][1] = fmaf(ga, acc[1], x[i][1]);
                            x[i][2] = fmaf(gb, acc[2], x[i][2]);
                            x[i][3] = fmaf(gb, acc[3], x[i][3]);
                        }
                    }
                    const float2 hs = *reinterpret_cast<const float2*>(&s.bias[warp][lane].z);
                    const float hs0 = hs.x, hs1 = hs.y;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint8_t* vt = tile + i * S::kHead + 17 * D;
                        load_scales<NG>(vt + gid * (2 * NG), ta[i]);
                        load_scales<NG>(vt + (gid + 8) * (2 * NG), tb[i]);
                    }
                    if (none || left < 2 * kKv4Slots) {
                        // slots behind the request's length, and of pages that are not there, hold anything
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int n = none >> i & 1u ? 0 : left - i * kKv4Slots;
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
                    constexpr uint32_t kFull = (2 * 127 + 10) << 7;  // of the bits of a scale and of f: s f reaches 2^10
                    uint32_t grown = 0;
#pragma unroll
                    for (int u = 0; u < NW; ++u)
                        grown |= __viaddmax_u16x2(max_bf16x2(max_bf16x2(ta[0][u], tb[0][u]), max_bf16x2(ta[1][u], tb[1][u])),
                                                  f[u], (kFull - 1) * 0x10001u) ^ (kFull - 1) * 0x10001u;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        y[i][0] = fmaf(x[i][0], hs0, -M0);
                        y[i][1] = fmaf(x[i][1], hs1, -M1);
                        y[i][2] = fmaf(x[i][2], hs0, -M0);
                        y[i][3] = fmaf(x[i][3], hs1, -M1);
                    }
                    const float most = fmaxf(fmaxf(fmaxf(y[0][0], y[0][1]), fmaxf(y[0][2], y[0][3])),
                                             fmaxf(fmaxf(y[1][0], y[1][1]), fmaxf(y[1][2], y[1][3])));
                    const bool over = most > 5.f || grown;
                    if (__any_sync(0xffffffffu, over)) {
                        // columns of heads beyond G are zeros throughout
                        float n0 = __fmul_rn(fmaxf(fmaxf(x[0][0], x[0][2]), fmaxf(x[1][0], x[1][2])), hs0);
                        float n1 = __fmul_rn(fmaxf(fmaxf(x[0][1], x[0][3]), fmaxf(x[1][1], x[1][3])), hs1);
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
                            const uint32_t t = u % 2 ? top[u / 2] >> 16 : top[u / 2] & 0xFFFFu;
                            float g = 1.f;
                            if (t + was >= kFull) {  // the new largest scale comes to [2^8, 2^9)
                                const uint32_t now = (uint32_t)min(max(2 * 127 + 8 - (int)(t >> 7), 24), 254) << 7;
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
                        // rounded like the maximum: of a score beyond 2^27 the exact product may lie far above it
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            y[i][0] = __fmul_rn(x[i][0], hs0) - M0;
                            y[i][1] = __fmul_rn(x[i][1], hs1) - M1;
                            y[i][2] = __fmul_rn(x[i][2], hs0) - M0;
                            y[i][3] = __fmul_rn(x[i][3], hs1) - M1;
                        }
                    }
                    load_v(0);
                    add_tile(y[0], ta[0], tb[0]);
                    load_v(1);
                }
                __syncwarp();  // all read: the stage may be filled again
                --flying;
                out_st ^= kStage;
                absent >>= 2;
                if (rem > 0) issue();
                if (none != 3u) add_tile(y[1], ta[1], tb[1]);
            }
        }
        // --- the item's sums
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, o);
            l1 += __shfl_xor_sync(0xffffffffu, l1, o);
        }
        const int seen = s.item[warp][k & 1].keys;
        if (!lost && seen > offset() * kKv4Slots) {
            // (Output, above) the least that the largest sum of a group has to be, in the accumulators' units
            const float least = 0x1p-20f * fminf(0x1p-10f * (team() ? seen / kWarps + 2 * kKv4Slots : seen), 64.f);
#pragma unroll
            for (int u = 0; u < NG; ++u) {
                const bool any = (u % 2 ? f[u / 2] >> 16 : f[u / 2] & 0xFFFFu) != kNoScale;  // else all zeros
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float most = fmaxf(fmaxf(fabsf(O[u][0][e]), fabsf(O[u][1][e])) * 16.f,
                                             fmaxf(fabsf(O[u][0][2 + e]), fabsf(O[u][1][2 + e])));
                    const uint32_t enough = __ballot_sync(0xffffffffu, !(most < least));
                    lost |= any && 2 * tig + e < a.G && !(enough & 0x11111111u << tig);
                }
            }
            lost = __any_sync(0xffffffffu, lost);
        }
        if (lost) {
            if (lane == 0) s.rest[warp] = make_int4(k, ahead, more, pending);
            pending = -1;
            break;
        }
        const Item it = s.item[warp][k & 1];
        const int64_t part = part_slot(it, it.c);
        if (gid == 0 && team()) {  // (one stretch: the sums have their memory for themselves)
            s.ml[warp][2 * tig] = make_float2(M0, l0);
            s.ml[warp][2 * tig + 1] = make_float2(M1, l1);
        }
        // rows of heads 2 t, 2 t + 1: columns 32 u + 4 g .. + 3
#pragma unroll
        for (int u = 0; u < NG; ++u) {
            // 2^20 and, for the even nibbles, 2^24, over f
            const float g = __uint_as_float(((2 * 127 + 20) << 23) - ((u % 2 ? f[u / 2] >> 16 : f[u / 2] & 0xFFFFu) << 16));
            const float ge = g * 16.f;
            const float4 o0 = make_float4(O[u][0][0] * ge, O[u][0][2] * g, O[u][1][0] * ge, O[u][1][2] * g);
            const float4 o1 = make_float4(O[u][0][1] * ge, O[u][0][3] * g, O[u][1][1] * ge, O[u][1][3] * g);
            const int col = 32 * u + 4 * gid;
            if (team()) {
                *reinterpret_cast<float4*>(s.merge(warp, 2 * tig) + col) = o0;
                *reinterpret_cast<float4*>(s.merge(warp, 2 * tig + 1) + col) = o1;
            } else if (it.parts == 1) {
                if (2 * tig < a.G) store_out(a, it, D, 2 * tig, col, o0, l0);
                if (2 * tig + 1 < a.G) store_out(a, it, D, 2 * tig + 1, col, o1, l1);
            } else {
                float* po = a.part_o + (part * a.G + 2 * tig) * D + col;
                if (2 * tig < a.G) __stcg(reinterpret_cast<float4*>(po), o0);
                if (2 * tig + 1 < a.G) __stcg(reinterpret_cast<float4*>(po + D), o1);
            }
        }
        if (it.parts > 1) {
            if (!team() && gid == 0) {
                __stcg(a.part_ml + part * kMaxGroup + 2 * tig, make_float2(M0, l0));
                __stcg(a.part_ml + part * kMaxGroup + 2 * tig + 1, make_float2(M1, l1));
            }
            if (lane == 0) s.pending[warp][pending] = it;
            ++pending;
        }
    }
    if (pending < 0) {
        cp_async_wait<0>();  // (nothing more is taken from the ring)
        __syncwarp();
        pending = exact_rest<D>(a, s);
    }
    if (team() && blockIdx.x < s.deal.total) {  // its one stretch
        __syncthreads();
        const Item& it = s.item[warp][0];
        const int col = tid % (D / 4) * 4, h = tid / (D / 4);  // thread -> 4 columns of one head
        if (h < a.G) {
            float M = -INFINITY, L = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s.ml[w][h].x);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 ml = s.ml[w][h];
                const float c = part_factor(ml.x, M);
                const float4 v = *reinterpret_cast<const float4*>(s.merge(w, h) + col);
                L += c * ml.y;
                o.x += c * v.x;
                o.y += c * v.y;
                o.z += c * v.z;
                o.w += c * v.w;
            }
            if (it.parts == 1) {
                store_out(a, it, D, h, col, o, L);
            } else {
                const int64_t part = part_slot(it, it.c);
                __stcg(reinterpret_cast<float4*>(a.part_o + (part * a.G + h) * D + col), o);
                if (col == 0) __stcg(a.part_ml + part * kMaxGroup + h, make_float2(M, L));
            }
        }
    }
    if (pending) {  // (all warps of a team have the same)
        __threadfence();
        if (team()) __syncthreads(); else __syncwarp();
        int last = 0;
        if ((team() ? tid : lane) < pending) {
            const Item& it = s.pending[warp][lane];
            last = atomicAdd(a.arrived + it.slot, 1) == it.parts - 1;
            if (last) a.arrived[it.slot] = 0;
            if (team()) s.last[lane] = last;
        }
        if (team()) __syncthreads();
        __threadfence();
        for (int i = 0; i < pending; ++i)
            if (team() ? s.last[i] : __shfl_sync(0xffffffffu, last, i)) {
                const Item& it = s.pending[warp][i];
                if (team()) {
                    if (2 * warp < a.G) join_parts<D, 2>(a, it, 2 * warp);
                } else {
                    for (int h0 = 0; h0 < a.G; h0 += 4) join_parts<D, 4>(a, it, h0);
                }
            }
    }
}

// Workspace: arrived, part_ml, part_o.
struct Workspace {
    int64_t arrived, ml, o, bytes;
    Workspace(int G, int d) {
        arrived = 0;
        ml = arrived + (int64_t)sizeof(int) * kMaxParts;
        o = ml + (int64_t)sizeof(float2) * kMaxGroup * kMaxParts;
        bytes = o + (int64_t)sizeof(float) * G * d * kMaxParts;
    }
};

template <int D>
cudaError_t launch(const Kv4AttnArgs& a, int grid, cudaStream_t s) {
    static_assert(sizeof(Smem<D>) <= 227 * 1024, "shared memory of a CTA");
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
    if (num_pages < 1 || num_pages > NF_KV4_MAX_PAGES || (int64_t)num_pages * n_kv_heads > 0x7fffffff ||
        num_requests < 0 || num_requests > NF_KV4_MAX_REQUESTS || sm_count < 0)
        return NF_ERR_INVALID_ARGUMENT;
    const double scale = softmax_scale != 0.f ? (double)softmax_scale : 1.0 / std::sqrt((double)head_dim);
    const float scale_log2 = (float)(scale * 1.4426950408889634);
    if (!(scale > 0.0) || !std::isfinite(scale_log2)) return NF_ERR_INVALID_ARGUMENT;
    if (q == out && q_stride != out_stride) return NF_ERR_INVALID_ARGUMENT;
    if (q_stride < row || out_stride < row || q_stride % 8 || out_stride % 8 || !nf::aligned(q, 16) ||
        !nf::aligned(out, 16) || !nf::aligned(pool, 16) || !nf::aligned(workspace, 256) ||
        workspace_bytes < nf_kv4_workspace_bytes(n_q_heads, n_kv_heads, head_dim))
        return NF_ERR_INVALID_ARGUMENT;
    if (num_requests == 0) return NF_OK;
    if ((st = nf::check_on_device(q, out, pool, kv_len, page_indptr, page_indices, workspace, status_device)) != NF_OK)
        return st;
    int sms = nf::device_sm_count();
    if (sms <= 0) return NF_ERR_CUDA;
    if (sm_count > 0 && sm_count < sms) sms = sm_count;
    const int grid = std::min(sms, nf::kMaxCtas);
    const int G = n_q_heads / n_kv_heads;
    const nf::Workspace at(G, head_dim);
    uint8_t* w = static_cast<uint8_t*>(workspace);
    const nf::Kv4AttnArgs a{static_cast<const uint16_t*>(q), static_cast<uint16_t*>(out), q_stride, out_stride,
                            static_cast<const uint8_t*>(pool), num_pages, kv_len, page_indptr, page_indices,
                            num_requests, n_kv_heads, G, scale_log2,
                            reinterpret_cast<int*>(w + at.arrived), reinterpret_cast<float2*>(w + at.ml),
                            reinterpret_cast<float*>(w + at.o), status_device};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = head_dim == 64 ? nf::launch<64>(a, grid, s) : nf::launch<128>(a, grid, s);
    return e == cudaSuccess ? NF_OK : NF_ERR_CUDA;
} catch (...) {
    return NF_ERR_INVALID_ARGUMENT;
}
