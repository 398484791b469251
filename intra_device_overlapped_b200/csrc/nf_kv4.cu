// Rows of K and V written to and read from the 4-bit paged cache (format: nf_kv4.h).
#include <cstdint>

#include <cuda_runtime.h>

#include "nanoflow.h"
#include "nf_kv4.h"

namespace nf {
namespace {

constexpr int kRowThreads = 128;  // append of fp32 rows: with 256 6 % slower, with 512 18 %
constexpr int kUnroll = 4;  // heads of a lane, in flight together: append of 8192 rows is fastest so (with 2 6 % slower, with 8 26 %)
constexpr float kLargest = 0x1p60f, kSmallest = 0x1p-60f;

struct Kv4RowArgs {
    const void *k, *v;      // rows in (append)
    void *k_out, *v_out;    // rows out (read)
    int64_t k_stride, v_stride;
    const int* slots;
    int T, num_pages, nkv;
    uint8_t* pool;
    int* status;
    FastDiv tasks;          // warps per token
};

// A warp takes kUnroll (D = 64: twice as many) heads of one token: D / 8 lanes a head's K row and the next D / 8 its V
// row, 8 columns each. Lane m's codes (columns 8 m .. 8 m + 7, group m / 4) are one 4-byte word of a K tile and two 2-byte
// units, d / 8 bytes apart, of a V tile. All that depends on the token is found once for all heads: with a line of work
// for each (token, head) of its own the kernels were bound by address arithmetic (310 instructions a line).
template <int D>
struct Task {
    static constexpr int kLanes = D / 8, kAtOnce = 32 / (2 * kLanes), kHeads = kUnroll * kAtOnce;
    int t, h, which, m;  // token, the lane's first head (then every kAtOnce-th)
    int id;              // the token's slot
    int scale;           // of the group, from the codes
    uint8_t* codes;      // in head h's tile
    __device__ __forceinline__ Task(const Kv4RowArgs& a) {
        const uint32_t lane = threadIdx.x & 31, warp = blockIdx.x * (kRowThreads / 32) + threadIdx.x / 32;
        t = a.tasks(warp);
        h = (warp - t * a.tasks.d) * kHeads + lane / (2 * kLanes);
        which = lane / kLanes & 1;
        m = lane & (kLanes - 1);
        id = t < a.T ? __ldg(a.slots + t) : -1;
    }
    // false (for the whole warp): the token has no slot
    __device__ __forceinline__ bool find(const Kv4RowArgs& a) {
        if (id < 0 || (id >> 4) >= a.num_pages) {
            if (id != -1 && (threadIdx.x & 31) == 0) set_status(a.status, NF_ERR_DEVICE_BOUNDS);
            return false;
        }
        const int slot = id & 15;
        const int at = (m & 3) * (D / 8) * (which ? 2 : 1) + 4 * (m >> 2) +
                       (which ? (slot >> 3) * 4 * D + ((slot & 7) >> 1) * D + 2 * (slot & 1) : slot * (D / 2));
        scale = 8 * D + (slot * (D / 32) + (m >> 2)) * 2 - at;
        codes = a.pool + ((int64_t)(id >> 4) * a.nkv + h) * (2 * kv4_tile_bytes(D)) + which * kv4_tile_bytes(D) + at;
        return true;
    }
};

// Codes of 8 values in units of s, code + 8 of x[e] in nibble e: the exact quotients x / s rounded half to even.
// q = x inv, inv within 2^-23 of 1 / s, and its remainder x - q s, exact by the fma, give the quotient as nearest fp32
// number but for 2^-45. A quotient half way between integers is such a number. Another one is more than half a step of
// fp32 away from it (x lies on a grid no finer than its own steps, and s has 8 bits), so it is not taken for it. Adding
// 1.5 * 2^23 then rounds to an integer in the last bits (no conversion instruction: those run at a quarter of the rate).
// |x| <= 7.04 s: no code leaves -7..7.
__device__ __forceinline__ uint32_t codes_of(const float* x, float s, float inv) {
    constexpr float kMagic = 12582912.f;
    // the sum of 16^e (0x4B400000 + k_e), and what makes it the sum of 16^e (8 + k_e), in 32 bits
    uint32_t codes = 0x88888888u - 0x4B400000u * 0x11111111u;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float q = x[e] * inv;
        codes += __float_as_uint(fmaf(fmaf(-q, s, x[e]), inv, q) + kMagic) << (4 * e);
    }
    return codes;
}

// The larger, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Nibble 2 p + h of a word to nibble p of half h, and back
__device__ __forceinline__ uint32_t unshuffle_nibbles(uint32_t x) {
    uint32_t t = (x ^ (x >> 4)) & 0x00F000F0u;
    x ^= t ^ (t << 4);
    t = (x ^ (x >> 8)) & 0x0000FF00u;
    return x ^ t ^ (t << 8);
}
__device__ __forceinline__ uint32_t shuffle_nibbles(uint32_t x) {
    uint32_t t = (x ^ (x >> 8)) & 0x0000FF00u;
    x ^= t ^ (t << 8);
    t = (x ^ (x >> 4)) & 0x00F000F0u;
    return x ^ t ^ (t << 4);
}

// Append. A group's largest magnitude is found by 4 lanes, its scale by each of them; a K row's codes are written as 4-byte
// words of 64 (32) consecutive bytes, a V row's as 2-byte units of 4 (2) sectors that two neighbouring slots share and L2
// joins. All of a lane's rows are loaded before the first is quantised, and before its token's slot is known. 8192
// rows of 8 heads of 128 take 10.6 us in bf16 (34 MB read, 9.4 written: 6.6 at a copy's rate), 12.8 in fp32 (11.7), 32768
// in bf16 38 (26): bound by instruction issue, of which the rounding takes a third.
template <int D, typename TK, typename TV>
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(const Kv4RowArgs a) {
    using W = Task<D>;
    W w(a);
    if (w.t >= a.T) return;
    float x[kUnroll][8];
    auto load = [&](const auto* row) {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
            if (w.h + i * W::kAtOnce < a.nkv) load_row8(row + i * W::kAtOnce * D, x[i]);
        }
    };
    const int64_t col = (int64_t)w.h * D + 8 * w.m;
    if constexpr (sizeof(TK) == sizeof(TV)) {
        load(static_cast<const TK*>(w.which ? a.v : a.k) + w.t * (w.which ? a.v_stride : a.k_stride) + col);
    } else if (w.which) {
        load(static_cast<const TV*>(a.v) + w.t * a.v_stride + col);
    } else {
        load(static_cast<const TK*>(a.k) + w.t * a.k_stride + col);
    }
    if (!w.find(a)) return;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        // largest magnitude of the group, NaN above all
        float big = fabsf(x[i][0]);
#pragma unroll
        for (int e = 1; e < 8; ++e) big = max_nan(big, fabsf(x[i][e]));
        big = max_nan(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = max_nan(big, __shfl_xor_sync(0xffffffffu, big, 2));
        float ab = big;
        if constexpr (sizeof(TK) == 4 || sizeof(TV) == 4) ab = big <= kLargest * 2.f ? bf2f(f2bf(big)) : big;
        uint16_t sbits = 0;
        uint32_t codes = 0x88888888u;  // code of column 8 m + e in nibble e
        if (!(ab <= kLargest)) {
            sbits = 0x7FC0;
        } else if (ab >= kSmallest) {
            // Two roundings to bf16 (of the magnitude and of its seventh): the scale is stored in 16 bits, and the codes
            // are taken against the stored value. ab has 8 bits, so ab / 7 is at least 2^-11 of it away from every border
            // of bf16 and a product with 1 / 7, 2^-23 off, rounds like the quotient.
            sbits = f2bf(ab * (1.f / 7.f));
            const float s = bf2f(sbits);
            float inv;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
            codes = codes_of(x[i], s, inv);
        }
        if (w.h + i * W::kAtOnce >= a.nkv) continue;
        uint8_t* at = w.codes + i * W::kAtOnce * 2 * kv4_tile_bytes(D);
        if (w.which) {
            *reinterpret_cast<uint16_t*>(at) = (uint16_t)codes;
            *reinterpret_cast<uint16_t*>(at + D / 8) = (uint16_t)(codes >> 16);
        } else {
            *reinterpret_cast<uint32_t*>(at) = unshuffle_nibbles(codes);
        }
        if ((w.m & 3) == 0) *reinterpret_cast<uint16_t*>(at + w.scale) = sbits;
    }
}

// Read: the reverse. Bound by the rows written: 8192 rows of 8 heads of 128 in bf16 take 8.8 us (0.75 of a copy), 32768
// 33.4 (0.79).
template <int D, typename T>
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(const Kv4RowArgs a) {
    using W = Task<D>;
    W w(a);
    if (!w.find(a)) return;
    uint32_t codes[kUnroll];
    uint16_t scale[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        if (w.h + i * W::kAtOnce >= a.nkv) continue;
        const uint8_t* at = w.codes + i * W::kAtOnce * 2 * kv4_tile_bytes(D);
        if (w.which) {
            const uint32_t lo = *reinterpret_cast<const uint16_t*>(at);
            codes[i] = lo | *reinterpret_cast<const uint16_t*>(at + D / 8) << 16;
        } else {
            codes[i] = shuffle_nibbles(*reinterpret_cast<const uint32_t*>(at));
        }
        scale[i] = *reinterpret_cast<const uint16_t*>(at + w.scale);
    }
    T* out = static_cast<T*>(w.which ? a.v_out : a.k_out) + w.t * (w.which ? a.v_stride : a.k_stride) + (int64_t)w.h * D +
             8 * w.m;
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        if (w.h + i * W::kAtOnce >= a.nkv) continue;
        const float s = bf2f(scale[i]), bias = -8388616.f;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)  // the code under the exponent of 2^23 (no conversion instruction)
            x[e] = s * (__uint_as_float((codes[i] >> (4 * e) & 15u) | 0x4B000000u) + bias);
        store_row8(out + i * W::kAtOnce * D, x);
    }
}

// Blocks of a launch, and its warps per token
template <int D>
int row_grid(Kv4RowArgs& a) {
    a.tasks = FastDiv((a.nkv + Task<D>::kHeads - 1) / Task<D>::kHeads);
    return (int)(((int64_t)a.T * a.tasks.d + kRowThreads / 32 - 1) / (kRowThreads / 32));
}

template <int D>
cudaError_t launch_append(Kv4RowArgs a, bool k32, bool v32, cudaStream_t s) {
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
cudaError_t launch_read(Kv4RowArgs a, bool out32, cudaStream_t s) {
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
    const int k_unit = k_dtype == NF_DTYPE_F32 ? 4 : 8, v_unit = v_dtype == NF_DTYPE_F32 ? 4 : 8;  // 16 bytes
    if (a.k_stride < row || a.v_stride < row || a.k_stride % k_unit || a.v_stride % v_unit) return NF_ERR_INVALID_ARGUMENT;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(a.pool, 16)) return NF_ERR_INVALID_ARGUMENT;
    // (warps are counted in 32 bits)
    if ((int64_t)a.T * a.nkv > 0x40000000) return NF_ERR_INVALID_ARGUMENT;
    if (a.T == 0) return NF_OK;
    return check_on_device(k, v, a.slots, a.pool, a.status);
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
                           static_cast<uint8_t*>(pool), status_device, nf::FastDiv()};
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
                           static_cast<uint8_t*>(const_cast<void*>(pool)), status_device,
                           nf::FastDiv()};
    const nf_status st = nf::check_rows(a, k_out, v_out, head_dim, out_dtype, out_dtype);
    if (st != NF_OK || num_tokens == 0) return st;
    const bool out32 = out_dtype == NF_DTYPE_F32;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = head_dim == 64 ? nf::launch_read<64>(a, out32, s) : nf::launch_read<128>(a, out32, s);
    return e == cudaSuccess ? NF_OK : NF_ERR_CUDA;
} catch (...) {
    return NF_ERR_INVALID_ARGUMENT;
}
