// The 4-bit paged KV cache: its format, and checks shared by its entry points.
//
// A page holds 16 slots of every KV head; per head a K tile, then a V tile, each 9 d bytes: 8 d bytes
// of codes and 16 x d/32 bf16 scales (value = (code - 8) * scale, one scale per slot and 32 columns).
// The code order inside a tile is the operand order of the warp-level tensor instruction, so that a lane
// of the attention kernel finds its operand's codes in consecutive bytes:
//   K, slot s, column 32 j + 8 t + 2 p + h:       byte s d/2 + t d/8 + 4 j + 2 h + p / 2, nibble p % 2
//     (the A operand's row s; lane t of a quad holds the pairs h = 0, 1 of both half-steps of group j)
//   V, slot 8 e + 2 t + h, column 32 j + 4 g + p: byte e 4d + t d + g d/8 + 4 j + 2 h + p / 2, nibble p % 2
//     (the A operand's column pair t, half e of V^T; p = the rows g, g + 8 of two 16-row tiles)
// A slot's K codes are d/2 consecutive bytes and its V codes 2-byte units of their own, so that no two
// slots share a byte and rows can be written in parallel without read-modify-write.
#pragma once
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "nanoflow.h"
#include "nf_ptx.cuh"

namespace nf {

constexpr int kKv4Slots = 16;   // slots per page
constexpr int kKv4MaxHeads = 256;

__host__ __device__ constexpr int kv4_tile_bytes(int d) { return 9 * d; }

// nf_status of a head shape of the 4-bit cache.
inline nf_status kv4_check_heads(int32_t nkv, int32_t d) {
    if (nkv < 1 || d < 1) return NF_ERR_INVALID_ARGUMENT;
    if ((d != 64 && d != 128) || nkv > kKv4MaxHeads) return NF_ERR_UNSUPPORTED;
    return NF_OK;
}

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <typename T>
constexpr uintptr_t align_of() {
    if constexpr (std::is_void_v<T>) return 1; else return alignof(T);
}

// NF_OK when every (non-null) pointer is aligned to its type and memory of the current device (or managed),
// else NF_ERR_INVALID_ARGUMENT; NF_ERR_CUDA without a device. A host pointer, another device's or a misaligned
// one would fault in the kernel. No stream operation: allowed while a stream is being captured.
template <typename... P>
nf_status check_on_device(const P*... ptrs) {
    if (!(aligned(ptrs, align_of<P>()) && ...)) return NF_ERR_INVALID_ARGUMENT;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) { cudaGetLastError(); return NF_ERR_CUDA; }
    const void* list[] = {ptrs...};
    for (const void* p : list) {
        if (p == nullptr) continue;
        cudaPointerAttributes at;
        if (cudaPointerGetAttributes(&at, p) != cudaSuccess) { cudaGetLastError(); return NF_ERR_CUDA; }
        if (at.type == cudaMemoryTypeManaged) continue;
        if (at.type != cudaMemoryTypeDevice || at.device != dev) return NF_ERR_INVALID_ARGUMENT;
    }
    return NF_OK;
}

// n / d for 0 <= n < 2^31 and a divisor known on the host: with m = ceil(2^(31 + s) / d), 2^(s - 1) < d <= 2^s, the
// error of n m / 2^(31 + s) is below n / 2^31 / d, too little to reach the next integer.
struct FastDiv {
    uint32_t m, s, d;
    explicit FastDiv(uint32_t div = 1) : m(0), s(0), d(div) {
        while ((1u << s) < div) ++s;
        m = (uint32_t)(((uint64_t)(1ull << (31 + s)) + div - 1) / div);
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
        return (uint32_t)(((uint64_t)n * m) >> (31 + s));
    }
};

// Eight consecutive values of a bf16 or fp32 row as fp32, and back (16 and 32 bytes, 16-byte aligned). Rows are streamed:
// written evict-first, 32768 rows read back from the cache take 33 us, else 41.
template <typename T>
__device__ __forceinline__ void load_row8(const T* row, float* x) {
    if constexpr (sizeof(T) == 4) {
        const float4 a = __ldcs(reinterpret_cast<const float4*>(row)), b = __ldcs(reinterpret_cast<const float4*>(row) + 1);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        const uint4 w = __ldcs(reinterpret_cast<const uint4*>(row));
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(v[i] << 16);
            x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
        }
    }
}

template <typename T>
__device__ __forceinline__ void store_row8(T* row, const float* x) {
    if constexpr (sizeof(T) == 4) {
        __stcs(reinterpret_cast<float4*>(row), make_float4(x[0], x[1], x[2], x[3]));
        __stcs(reinterpret_cast<float4*>(row) + 1, make_float4(x[4], x[5], x[6], x[7]));
    } else {
        __stcs(reinterpret_cast<uint4*>(row), make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                    pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])));
    }
}

}  // namespace nf
