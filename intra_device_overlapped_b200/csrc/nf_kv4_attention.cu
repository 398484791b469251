// Paged GQA decode attention over the 4-bit cache (format: nf_kv4.h).
#include <cmath>
#include <cstdint>
#include <new>

#include <cuda_runtime.h>

#include "nanoflow.h"
#include "nf_internal.h"
#include "nf_kv4.h"

namespace nf {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxGroup = 8;  // query heads per KV head

struct Kv4AttnArgs {
    const uint16_t* q;
    uint16_t* out;
    int64_t q_stride, out_stride;
    const uint8_t* pool;
    int num_pages;
    const int *kv_len, *indptr, *indices;
    int R, nkv, G;
    float scale_log2;
    int* status;
};

// One CTA per (request, KV head); each pass takes 128 keys: a thread forms the scores of one key, then
// the weights of all keys for one column of the output. fp32 throughout.
template <int D>
__global__ void __launch_bounds__(kThreads) kv4_attention_kernel(const Kv4AttnArgs a) {
    __shared__ float qs[kMaxGroup][D], w[kMaxGroup][kThreads], red[kMaxGroup][4];
    __shared__ int page_s[kThreads / 16];
    const int tid = threadIdx.x, G = a.G;
    const int r = blockIdx.x / a.nkv, h = blockIdx.x - r * a.nkv;
    for (int i = tid; i < G * D; i += kThreads)
        qs[i / D][i % D] = bf2f(a.q[(int64_t)r * a.q_stride + (int64_t)h * G * D + i]) * a.scale_log2;
    const int p0 = a.indptr[r], np = a.indptr[r + 1] - p0;
    int n = a.kv_len[r];
    if (n < 0 || n > np * 16) {
        if (tid == 0) set_status(a.status, NF_ERR_DEVICE_BOUNDS);
        n = n < 0 ? 0 : max(0, np * 16);
    }
    float m[kMaxGroup], l[kMaxGroup], o[kMaxGroup];
#pragma unroll
    for (int g = 0; g < kMaxGroup; ++g) { m[g] = -INFINITY; l[g] = 0.f; o[g] = 0.f; }
    for (int k0 = 0; k0 < n; k0 += kThreads) {
        __syncthreads();
        if (tid < kThreads / 16) {
            int page = -1;
            if (k0 + tid * 16 < n) {
                page = a.indices[p0 + k0 / 16 + tid];
                if ((unsigned)page >= (unsigned)a.num_pages) {
                    set_status(a.status, NF_ERR_DEVICE_BOUNDS);
                    page = -1;
                }
            }
            page_s[tid] = page;
        }
        __syncthreads();
        const int slot = tid & 15, page = page_s[tid >> 4];
        const bool seen = page >= 0 && k0 + tid < n;
        float x[kMaxGroup];
#pragma unroll
        for (int g = 0; g < kMaxGroup; ++g) x[g] = 0.f;
        if (seen) {
            const uint8_t* tile = a.pool + ((int64_t)page * a.nkv + h) * (2 * kv4_tile_bytes(D));
            for (int j = 0; j < D / 32; ++j) {
                const float s = bf2f(*reinterpret_cast<const uint16_t*>(tile + 8 * D + (slot * (D / 32) + j) * 2));
                for (int t = 0; t < 4; ++t) {
                    const uint32_t c =
                        *reinterpret_cast<const uint32_t*>(tile + slot * (D / 2) + t * (D / 8) + 4 * j);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {  // column 8 t + 2 p + h: byte 2 h + p / 2, nibble p % 2
                        const int p = i >> 1, hh = i & 1;
                        const float v = s * (float)((int)(c >> (8 * (2 * hh + p / 2) + 4 * (p & 1)) & 15u) - 8);
#pragma unroll
                        for (int g = 0; g < kMaxGroup; ++g)
                            if (g < G) x[g] = fmaf(qs[g][32 * j + 8 * t + i], v, x[g]);
                    }
                }
            }
        }
#pragma unroll
        for (int g = 0; g < kMaxGroup; ++g) {
            if (g >= G) break;
            float top = seen ? x[g] : -INFINITY;
            for (int of = 16; of; of >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, of));
            if ((tid & 31) == 0) red[g][tid >> 5] = top;
        }
        __syncthreads();
#pragma unroll
        for (int g = 0; g < kMaxGroup; ++g) {
            if (g >= G) break;
            const float mn = fmaxf(fmaxf(fmaxf(red[g][0], red[g][1]), fmaxf(red[g][2], red[g][3])), m[g]);
            const float c = mn == -INFINITY ? 1.f : exp2f(m[g] - mn);
            l[g] *= c;
            o[g] *= c;
            m[g] = mn;
            w[g][tid] = seen ? exp2f(x[g] - mn) : 0.f;
        }
        __syncthreads();
        const int keys = min(kThreads, n - k0);
        const int col = tid & (D - 1), j = col / 32, gg = col % 32 / 4, p = col & 3;
        for (int k = 0; k < keys; ++k) {
            const int pg = page_s[k >> 4], sl = k & 15;
            if (pg < 0) continue;
            const uint8_t* tile =
                a.pool + ((int64_t)pg * a.nkv + h) * (2 * kv4_tile_bytes(D)) + kv4_tile_bytes(D);
            const int at = (sl >> 3) * 4 * D + ((sl & 7) >> 1) * D + gg * (D / 8) + 4 * j + 2 * (sl & 1) + p / 2;
            const float s = bf2f(*reinterpret_cast<const uint16_t*>(tile + 8 * D + (sl * (D / 32) + j) * 2));
            const float v = s * (float)((int)(tile[at] >> (4 * (p & 1)) & 15u) - 8);
#pragma unroll
            for (int g = 0; g < kMaxGroup; ++g) {
                if (g < G) {
                    l[g] += w[g][k];
                    o[g] = fmaf(w[g][k], v, o[g]);
                }
            }
        }
    }
    if (tid < D) {
#pragma unroll
        for (int g = 0; g < kMaxGroup; ++g)
            if (g < G)
                a.out[(int64_t)r * a.out_stride + (int64_t)(h * G + g) * D + tid] = f2bf(l[g] == 0.f ? 0.f : o[g] / l[g]);
    }
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
    return st == NF_OK ? 256 : -(int64_t)st;
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
    const double scale = softmax_scale > 0.f ? (double)softmax_scale : 1.0 / std::sqrt((double)head_dim);
    const nf::Kv4AttnArgs a{static_cast<const uint16_t*>(q), static_cast<uint16_t*>(out), q_stride, out_stride,
                            static_cast<const uint8_t*>(pool), num_pages, kv_len, page_indptr, page_indices,
                            num_requests, n_kv_heads, n_q_heads / n_kv_heads,
                            (float)(scale * 1.4426950408889634), status_device};
    const int grid = num_requests * n_kv_heads;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (head_dim == 64)
        nf::kv4_attention_kernel<64><<<grid, nf::kThreads, 0, s>>>(a);
    else
        nf::kv4_attention_kernel<128><<<grid, nf::kThreads, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? NF_OK : NF_ERR_CUDA;
} catch (...) {
    return NF_ERR_INVALID_ARGUMENT;
}
