// Rows of K and V written to and read from the 4-bit paged cache (format: nf_kv4.h).
#include <cstdint>
#include <new>

#include <cuda_runtime.h>

#include "nanoflow.h"
#include "nf_kv4.h"

namespace nf {
namespace {

constexpr int kRowThreads = 256;
constexpr float kLargest = 0x1p60f, kSmallest = 0x1p-60f;

struct Kv4RowArgs {
    const void *k, *v;      // rows in (append)
    void *k_out, *v_out;    // rows out (read)
    int64_t k_stride, v_stride;
    const int* slots;
    int T, num_pages, nkv;
    uint8_t* pool;
    int* status;
};

// Work is dealt in lines: line 2 (t nkv + h) + w is head h of token t's K (w = 0) or V (w = 1) row, d / 4
// lanes of 4 columns each. `lane4` is this lane's place in its line.
template <int D>
struct Line {
    int t, h, which, lane4;
    __device__ __forceinline__ Line(int64_t line, int nkv) {
        which = (int)(line & 1);
        const int64_t th = line >> 1;
        t = (int)(th / nkv);
        h = (int)(th - (int64_t)t * nkv);
        lane4 = threadIdx.x & (D / 4 - 1);
    }
    // where this lane's 4 codes stand in its tile: V, the 2-byte unit; K, the 4-byte word that lanes 2 i and
    // 2 i + 1 share (p = 0, 1 and p = 2, 3: the low and the high byte of each half)
    __device__ __forceinline__ int v_unit(int slot) const {
        return (slot >> 3) * 4 * D + ((slot & 7) >> 1) * D + (lane4 & 7) * (D / 8) + 4 * (lane4 >> 3) + 2 * (slot & 1);
    }
    __device__ __forceinline__ int k_word(int slot) const {
        return slot * (D / 2) + ((lane4 & 7) >> 1) * (D / 8) + 4 * (lane4 >> 3);
    }
    __device__ __forceinline__ int scale_at(int slot) const { return 8 * D + (slot * (D / 32) + (lane4 >> 3)) * 2; }
};

// Code of x in units of s: the exact quotient x / s rounded half to even. x * (1 / s) is off by under 2^-22 of
// it, so k is the right integer or, next to a border, its neighbour; x - k s has at most 24 bits there
// (|x - k s| <= s and x is no finer than 2^-24 s where k != 0), so the fma gives it exactly and tells the
// side. |x| <= 7.04 s: no code leaves -7..7.
__device__ __forceinline__ int code_of(float x, float s, float inv) {
    float k = rintf(x * inv);
    const float r = fmaf(-k, s, x), half = 0.5f * s;
    const bool odd = ((int)k & 1) != 0;
    if (fabsf(r) > half || (fabsf(r) == half && odd)) k += r > 0.f ? 1.f : -1.f;
    return (int)k + 8;
}

template <int D, typename TK, typename TV>
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(const Kv4RowArgs a) {
    constexpr int kPerBlock = kRowThreads / (D / 4);
    const int64_t lines = (int64_t)a.T * a.nkv * 2;
    // every lane of a warp stays in the loop (the shuffles need all of them)
    for (int64_t base = (int64_t)blockIdx.x * kPerBlock; base < lines; base += (int64_t)gridDim.x * kPerBlock) {
        const int64_t line = base + threadIdx.x / (D / 4);
        const bool live = line < lines;
        const Line<D> l(live ? line : 0, a.nkv);
        const int slot_id = live ? __ldg(a.slots + l.t) : -1;
        const bool ok = slot_id >= 0 && (slot_id >> 4) < a.num_pages;
        if (!ok && slot_id != -1) set_status(a.status, NF_ERR_DEVICE_BOUNDS);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ok) {
            const int64_t col = l.h * D + 4 * l.lane4;
            x = l.which ? load_row4<TV>(a.v, l.t * a.v_stride + col) : load_row4<TK>(a.k, l.t * a.k_stride + col);
        }
        // largest magnitude of the group by its bits: ordered like the values, NaN above infinity
        uint32_t top = max(max(__float_as_uint(x.x) & 0x7fffffffu, __float_as_uint(x.y) & 0x7fffffffu),
                           max(__float_as_uint(x.z) & 0x7fffffffu, __float_as_uint(x.w) & 0x7fffffffu));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float big = __uint_as_float(top);
        const float ab = big <= kLargest * 2.f ? bf2f(f2bf(big)) : big;
        uint16_t sbits = 0;
        uint32_t codes = 0x8888;
        if (!(ab <= kLargest)) {
            sbits = 0x7FC0;
        } else if (ab >= kSmallest) {
            // two roundings to bf16 (of the magnitude and of its seventh): the scale is stored in 16 bits, and the
            // codes are taken against the stored value
            sbits = f2bf(__fdiv_rn(ab, 7.f));
            const float s = bf2f(sbits), inv = __frcp_rn(s);
            codes = code_of(x.x, s, inv) | code_of(x.y, s, inv) << 4 | code_of(x.z, s, inv) << 8 |
                    code_of(x.w, s, inv) << 12;
        }
        // K: columns 4 m .. 4 m + 3 are (p, h) = (p0, 0), (p0, 1), (p0 + 1, 0), (p0 + 1, 1), p0 = 0 on even lanes
        // and 2 on odd ones: bytes h = 0, 1 of p0, p0 + 1
        const uint32_t b0 = (codes & 15u) | (codes >> 4 & 0xF0u), b1 = (codes >> 4 & 15u) | (codes >> 8 & 0xF0u);
        const uint32_t mine = b0 | b1 << 16;
        const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
        if (!ok) continue;
        const int slot = slot_id & 15;
        uint8_t* tile = a.pool + ((int64_t)(slot_id >> 4) * a.nkv + l.h) * (2 * kv4_tile_bytes(D)) +
                        l.which * kv4_tile_bytes(D);
        if (l.which) {
            *reinterpret_cast<uint16_t*>(tile + l.v_unit(slot)) = (uint16_t)codes;
        } else if ((l.lane4 & 1) == 0) {
            *reinterpret_cast<uint32_t*>(tile + l.k_word(slot)) = mine | other << 8;
        }
        if ((l.lane4 & 7) == 0) *reinterpret_cast<uint16_t*>(tile + l.scale_at(slot)) = sbits;
    }
}

template <int D, typename T>
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(const Kv4RowArgs a) {
    constexpr int kPerBlock = kRowThreads / (D / 4);
    const int64_t lines = (int64_t)a.T * a.nkv * 2;
    for (int64_t line = (int64_t)blockIdx.x * kPerBlock + threadIdx.x / (D / 4); line < lines;
         line += (int64_t)gridDim.x * kPerBlock) {
        const Line<D> l(line, a.nkv);
        const int slot_id = __ldg(a.slots + l.t);
        if (slot_id < 0 || (slot_id >> 4) >= a.num_pages) {
            if (slot_id != -1) set_status(a.status, NF_ERR_DEVICE_BOUNDS);
            continue;
        }
        const int slot = slot_id & 15;
        const uint8_t* tile = a.pool + ((int64_t)(slot_id >> 4) * a.nkv + l.h) * (2 * kv4_tile_bytes(D)) +
                              l.which * kv4_tile_bytes(D);
        uint32_t codes;
        if (l.which) {
            codes = *reinterpret_cast<const uint16_t*>(tile + l.v_unit(slot));
        } else {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(tile + l.k_word(slot)) >> ((l.lane4 & 1) * 8);
            codes = (w & 15u) | (w >> 16 & 15u) << 4 | (w >> 4 & 15u) << 8 | (w >> 20 & 15u) << 12;
        }
        const float s = bf2f(*reinterpret_cast<const uint16_t*>(tile + l.scale_at(slot)));
        auto value = [&](int i) { return s * (float)((int)(codes >> (4 * i) & 15u) - 8); };
        const int64_t at = (int64_t)l.t * (l.which ? a.v_stride : a.k_stride) + l.h * D + 4 * l.lane4;
        store_row4<T>(l.which ? a.v_out : a.k_out, at, make_float4(value(0), value(1), value(2), value(3)));
    }
}

template <int D>
int row_grid(const Kv4RowArgs& a) {
    constexpr int kPerBlock = kRowThreads / (D / 4);
    const int64_t blocks = ((int64_t)a.T * a.nkv * 2 + kPerBlock - 1) / kPerBlock;
    return (int)(blocks < 148 * 8 ? blocks : 148 * 8);
}

template <int D>
cudaError_t launch_append(const Kv4RowArgs& a, bool k32, bool v32, cudaStream_t s) {
    const int grid = row_grid<D>(a);
    if (k32)
        v32 ? kv4_append_kernel<D, float, float><<<grid, kRowThreads, 0, s>>>(a)
            : kv4_append_kernel<D, float, uint16_t><<<grid, kRowThreads, 0, s>>>(a);
    else
        v32 ? kv4_append_kernel<D, uint16_t, float><<<grid, kRowThreads, 0, s>>>(a)
            : kv4_append_kernel<D, uint16_t, uint16_t><<<grid, kRowThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_read(const Kv4RowArgs& a, bool out32, cudaStream_t s) {
    const int grid = row_grid<D>(a);
    out32 ? kv4_read_kernel<D, float><<<grid, kRowThreads, 0, s>>>(a)
          : kv4_read_kernel<D, uint16_t><<<grid, kRowThreads, 0, s>>>(a);
    return cudaGetLastError();
}

nf_status check_rows(const Kv4RowArgs& a, const void* k, const void* v, int32_t d, int32_t k_dtype, int32_t v_dtype) {
    if (!k || !v || !a.slots || !a.pool || !a.status) return NF_ERR_INVALID_ARGUMENT;
    if (a.T < 0 || a.num_pages < 1 || a.num_pages > NF_KV4_MAX_PAGES) return NF_ERR_INVALID_ARGUMENT;
    for (int32_t t : {k_dtype, v_dtype})
        if (t != NF_DTYPE_BF16 && t != NF_DTYPE_F32) return NF_ERR_INVALID_ARGUMENT;
    const nf_status st = kv4_check_heads(a.nkv, d);
    if (st != NF_OK) return st;
    const int64_t row = (int64_t)a.nkv * d;
    if (a.k_stride < row || a.v_stride < row || a.k_stride % 4 || a.v_stride % 4) return NF_ERR_INVALID_ARGUMENT;
    if (!aligned(k, k_dtype == NF_DTYPE_F32 ? 16 : 8) || !aligned(v, v_dtype == NF_DTYPE_F32 ? 16 : 8) ||
        !aligned(a.pool, 16))
        return NF_ERR_INVALID_ARGUMENT;
    if (a.T == 0) return NF_OK;
    return check_on_device(k, v, (const void*)a.slots, (const void*)a.pool, (const void*)a.status);
}

}  // namespace
}  // namespace nf

extern "C" int64_t nf_kv4_page_bytes(int32_t n_kv_heads, int32_t head_dim) {
    const nf_status st = nf::kv4_check_heads(n_kv_heads, head_dim);
    return st == NF_OK ? (int64_t)n_kv_heads * 2 * nf::kv4_tile_bytes(head_dim) : -(int64_t)st;
}

extern "C" nf_status nf_op_kv4_append(const void* k, int64_t k_stride, int32_t k_dtype, const void* v,
                                      int64_t v_stride, int32_t v_dtype, const int32_t* slots, int32_t num_tokens,
                                      void* pool, int32_t num_pages, int32_t n_kv_heads, int32_t head_dim,
                                      int32_t* status_device, void* stream) try {
    const nf::Kv4RowArgs a{k, v, nullptr, nullptr, k_stride, v_stride, slots, num_tokens, num_pages, n_kv_heads,
                           static_cast<uint8_t*>(pool), status_device};
    const nf_status st = nf::check_rows(a, k, v, head_dim, k_dtype, v_dtype);
    if (st != NF_OK || num_tokens == 0) return st;
    const bool k32 = k_dtype == NF_DTYPE_F32, v32 = v_dtype == NF_DTYPE_F32;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e =
        head_dim == 64 ? nf::launch_append<64>(a, k32, v32, s) : nf::launch_append<128>(a, k32, v32, s);
    return e == cudaSuccess ? NF_OK : NF_ERR_CUDA;
} catch (...) {
    return NF_ERR_INVALID_ARGUMENT;
}

extern "C" nf_status nf_op_kv4_read(const void* pool, int32_t num_pages, const int32_t* slots, int32_t num_tokens,
                                    int32_t n_kv_heads, int32_t head_dim, void* k_out, int64_t k_stride, void* v_out,
                                    int64_t v_stride, int32_t out_dtype, int32_t* status_device, void* stream) try {
    const nf::Kv4RowArgs a{nullptr, nullptr, k_out, v_out, k_stride, v_stride, slots, num_tokens, num_pages, n_kv_heads,
                           static_cast<uint8_t*>(const_cast<void*>(pool)), status_device};
    const nf_status st = nf::check_rows(a, k_out, v_out, head_dim, out_dtype, out_dtype);
    if (st != NF_OK || num_tokens == 0) return st;
    const bool out32 = out_dtype == NF_DTYPE_F32;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = head_dim == 64 ? nf::launch_read<64>(a, out32, s) : nf::launch_read<128>(a, out32, s);
    return e == cudaSuccess ? NF_OK : NF_ERR_CUDA;
} catch (...) {
    return NF_ERR_INVALID_ARGUMENT;
}
