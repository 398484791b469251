// Rotary positions: frequencies (host) and the rotation of rows of q and k heads.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "nanoflow.h"
#include "nf_kv4.h"

namespace nf {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxDim = 512;

struct RopeSide {
    const void* in;
    void* out;
    int64_t in_stride, out_stride;
    int heads;
};

struct RopeArgs {
    RopeSide q, k;
    const int* positions;
    const double* freq;
    float scale;
    int T, d, rot, interleaved;
    int copy;  // columns behind `rot` have to be written (the output is another buffer or type)
};

// Cosines and sines of token t's positions, times `scale`, by `threads` threads.
__device__ __forceinline__ void form_turns(const RopeArgs& a, int t, float2* cs, int thread, int threads) {
    const double pos = (double)a.positions[t];
    for (int i = thread; i < a.rot / 2; i += threads) {
        // turns in 64 bits (131072 positions leave fp32 no bits of the fraction), then sin and cos of pi x
        const double turn = pos * a.freq[i] * 0.15915494309189533577;
        float s, c;
        sincospif((float)(2.0 * (turn - rint(turn))), &s, &c);
        cs[i] = make_float2(c * a.scale, s * a.scale);
    }
}

// (x, y) at angle p f: (x c - y s, y c + x s). A block takes a token, whose turns are formed once, in shared memory, for all
// its heads; a thread takes 8 pairs of a head at a time, two vectors of 8 columns in (16 bytes in bf16) and out. Every value
// is read and written once, so the kernel is bound by HBM: 8192 rows of 72 bf16 heads of 128 take 50.7 us, 0.91 of a copy,
// 8192 of 40 heads from fp32 to bf16 40.1, 0.96. Blocks of 256 threads end soonest where each has an SM nearly for itself,
// small ones keep more loads in flight and more tokens' turns beside them: with 256, 128 and 64 threads 32 such rows 3.2, 3.9
// and 5.6 us, 512 5.3, 5.3 and 6.6, 1024 8.5, 7.6 and 8.2, 2048 16, 14.8 and 13.2. Few heads, 2 of 64 to 9 of 128, change at
// the same numbers of tokens: 700 2.4, 2.3 and 2.4 us, 2000 4.3, 3.3 and 3.0 (2 of 64). (Two vectors a thread at a time: 10 %
// more time, for the registers that they hold.)
template <typename TI, typename TO>
__global__ void __launch_bounds__(kRopeThreads) rope_vec_kernel(const RopeArgs a, const FastDiv per_head) {
    __shared__ float2 cs[kRopeMaxDim / 2];
    const int64_t t = blockIdx.x;
    const int half = a.rot / 2, turned = a.rot / 16, units = (a.q.heads + a.k.heads) * per_head.d;
    form_turns(a, (int)t, cs, threadIdx.x, blockDim.x);
    __syncthreads();
#pragma unroll 1
    for (int e = threadIdx.x; e < units; e += blockDim.x) {
        int h = per_head(e);
        const int u = e - h * per_head.d;
        const bool isq = h < a.q.heads;
        const RopeSide& side = isq ? a.q : a.k;
        h -= isq ? 0 : a.q.heads;
        // columns i .. i + 7 and j .. j + 7
        int i = 16 * u, j = i + 8;
        if (u < turned && !a.interleaved) {
            i = 8 * u;
            j = i + half;
        }
        if (u >= turned && !a.copy) continue;
        const TI* x = static_cast<const TI*>(side.in) + t * side.in_stride + (int64_t)h * a.d;
        TO* y = static_cast<TO*>(side.out) + t * side.out_stride + (int64_t)h * a.d;
        float p[8], q[8];
        load_row8(x + i, p);
        load_row8(x + j, q);
        if (u < turned) {
            if (a.interleaved) {
#pragma unroll
                for (int n = 0; n < 8; n += 2) {
                    const float2 w = cs[8 * u + n / 2], z = cs[8 * u + 4 + n / 2];
                    const float p0 = p[n], q0 = q[n];
                    p[n] = p0 * w.x - p[n + 1] * w.y;
                    p[n + 1] = p[n + 1] * w.x + p0 * w.y;
                    q[n] = q0 * z.x - q[n + 1] * z.y;
                    q[n + 1] = q[n + 1] * z.x + q0 * z.y;
                }
            } else {
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const float2 w = cs[8 * u + n];
                    const float p0 = p[n];
                    p[n] = p0 * w.x - q[n] * w.y;
                    q[n] = q[n] * w.x + p0 * w.y;
                }
            }
        }
        store_row8(y + i, p);
        store_row8(y + j, q);
    }
}

// One pair per step, any sizes and alignment.
template <typename TI, typename TO>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
    __shared__ float2 cs[kRopeMaxDim / 2];
    const int half = a.rot / 2;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        form_turns(a, (int)t, cs, threadIdx.x, kRopeThreads);
        __syncthreads();
        const int units = a.d / 2, heads = a.q.heads + a.k.heads;
        for (int e = threadIdx.x; e < heads * units; e += kRopeThreads) {
            const int h = e / units, u = e - h * units;
            const bool isq = h < a.q.heads;
            const RopeSide& side = isq ? a.q : a.k;
            const int hh = isq ? h : h - a.q.heads;
            const TI* x = static_cast<const TI*>(side.in) + t * side.in_stride + (int64_t)hh * a.d;
            TO* y = static_cast<TO*>(side.out) + t * side.out_stride + (int64_t)hh * a.d;
            int i, j;
            if (u >= half) { i = 2 * u; j = i + 1; }
            else if (a.interleaved) { i = 2 * u; j = i + 1; }
            else { i = u; j = u + half; }
            float x0, x1;
            if constexpr (sizeof(TI) == 4) { x0 = x[i]; x1 = x[j]; }
            else { x0 = bf2f(x[i]); x1 = bf2f(x[j]); }
            if (u < half) {
                const float2 w = cs[u];
                const float y0 = x0 * w.x - x1 * w.y;
                x1 = x1 * w.x + x0 * w.y;
                x0 = y0;
            } else if (!a.copy) {
                continue;
            }
            if constexpr (sizeof(TO) == 4) { y[i] = x0; y[j] = x1; }
            else { y[i] = f2bf(x0); y[j] = f2bf(x1); }
        }
        __syncthreads();
    }
}

template <typename TI, typename TO>
bool side_vec(const RopeSide& s) {
    return s.heads == 0 || (aligned(s.in, 16) && aligned(s.out, 16) && s.in_stride * sizeof(TI) % 16 == 0 &&
                            s.out_stride * sizeof(TO) % 16 == 0);
}

template <typename TI, typename TO>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
    if (a.d % 16 == 0 && a.rot % 16 == 0 && side_vec<TI, TO>(a.q) && side_vec<TI, TO>(a.k)) {
        rope_vec_kernel<TI, TO><<<a.T, a.T < 768 ? 256 : a.T < 1536 ? 128 : 64, 0, s>>>(a, FastDiv(a.d / 16));
    } else {
        const int grid = a.T < 148 * 8 ? a.T : 148 * 8;
        rope_kernel<TI, TO><<<grid, kRopeThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

// A side may be rotated in place (same buffer, type and stride). NF_ERR_INVALID_ARGUMENT for a missing
// buffer, a row stride shorter than its heads, or one buffer used with two strides or types.
nf_status check_side(const RopeSide& s, int d, bool same_type) {
    if (s.heads == 0) return NF_OK;
    if (!s.in || !s.out || s.in_stride < (int64_t)s.heads * d || s.out_stride < (int64_t)s.heads * d)
        return NF_ERR_INVALID_ARGUMENT;
    if (s.in == s.out && (!same_type || s.in_stride != s.out_stride)) return NF_ERR_INVALID_ARGUMENT;
    return NF_OK;
}

}  // namespace
}  // namespace nf

extern "C" nf_status nf_rope_frequencies(const nf_rope_config* cfg, double* inv_freq, float* cos_sin_scale) try {
    if (!cfg || !inv_freq || !cos_sin_scale) return NF_ERR_INVALID_ARGUMENT;
    const int rot = cfg->rot_dim;
    const double theta = cfg->theta, factor = cfg->factor;
    if (rot < 2 || rot % 2 || rot > nf::kRopeMaxDim || !(theta > 0.0) || !std::isfinite(theta))
        return NF_ERR_INVALID_ARGUMENT;
    if (cfg->scaling != NF_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return NF_ERR_INVALID_ARGUMENT;
    const double pi = 3.14159265358979323846;
    const double span = (double)cfg->original_positions;
    const bool banded = cfg->scaling == NF_ROPE_WAVELENGTH || cfg->scaling == NF_ROPE_YARN;
    if (banded && (cfg->original_positions < 1 || !(cfg->low > 0.f) || !(cfg->high > cfg->low) ||
                   !std::isfinite(cfg->high)))
        return NF_ERR_INVALID_ARGUMENT;
    *cos_sin_scale = 1.f;
    double base = theta;
    switch (cfg->scaling) {
        case NF_ROPE_PLAIN:
        case NF_ROPE_LINEAR:
        case NF_ROPE_WAVELENGTH:
            break;
        case NF_ROPE_NTK:
            if (rot <= 2) return NF_ERR_INVALID_ARGUMENT;
            base = theta * std::pow(factor, (double)rot / (rot - 2));
            break;
        case NF_ROPE_YARN:
            if (!(theta > 1.0)) return NF_ERR_INVALID_ARGUMENT;
            *cos_sin_scale = (float)(0.1 * std::log(factor) + 1.0);
            break;
        default:
            return NF_ERR_INVALID_ARGUMENT;
    }
    // the pair index whose wave turns `turns` times over the original span
    auto index_of = [&](double turns) {
        return rot * std::log(span / (turns * 2.0 * pi)) / (2.0 * std::log(theta));
    };
    for (int i = 0; i < rot / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rot);
        double out = f;
        if (cfg->scaling == NF_ROPE_LINEAR) {
            out = f / factor;
        } else if (cfg->scaling == NF_ROPE_WAVELENGTH) {
            double keep = (span * f / (2.0 * pi) - cfg->low) / ((double)cfg->high - cfg->low);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            out = (1.0 - keep) * f / factor + keep * f;
        } else if (cfg->scaling == NF_ROPE_YARN) {
            double first = std::floor(index_of(cfg->high)), last = std::ceil(index_of(cfg->low));
            first = first < 0.0 ? 0.0 : first;
            last = last > rot - 1 ? rot - 1 : last;
            double blend = (i - first) / (last > first ? last - first : 1e-3);
            blend = blend < 0.0 ? 0.0 : blend > 1.0 ? 1.0 : blend;
            out = blend * f / factor + (1.0 - blend) * f;
        }
        inv_freq[i] = out;
    }
    return NF_OK;
} catch (...) {
    return NF_ERR_INVALID_ARGUMENT;
}

extern "C" nf_status nf_op_rope(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, int32_t n_q_heads,
                                const void* k, int64_t k_stride, void* k_out, int64_t k_out_stride, int32_t n_kv_heads,
                                int32_t in_dtype, int32_t out_dtype, const int32_t* positions, int32_t num_tokens,
                                int32_t head_dim, int32_t rot_dim, int32_t interleaved, const double* inv_freq,
                                float cos_sin_scale, void* stream) try {
    if (num_tokens < 0 || n_q_heads < 0 || n_kv_heads < 0 || head_dim < 2 || head_dim % 2 || rot_dim < 2 ||
        rot_dim % 2 || rot_dim > head_dim || (interleaved != 0 && interleaved != 1) || !std::isfinite(cos_sin_scale))
        return NF_ERR_INVALID_ARGUMENT;
    if ((in_dtype != NF_DTYPE_BF16 && in_dtype != NF_DTYPE_F32) ||
        (out_dtype != NF_DTYPE_BF16 && out_dtype != NF_DTYPE_F32))
        return NF_ERR_INVALID_ARGUMENT;
    if (head_dim > nf::kRopeMaxDim || n_q_heads > 65536 || n_kv_heads > 65536) return NF_ERR_UNSUPPORTED;
    if (!positions || !inv_freq) return NF_ERR_INVALID_ARGUMENT;
    nf::RopeArgs a;
    a.q = {q, q_out, q_stride, q_out_stride, n_q_heads};
    a.k = {k, k_out, k_stride, k_out_stride, n_kv_heads};
    nf_status st;
    const bool same = in_dtype == out_dtype;
    if ((st = nf::check_side(a.q, head_dim, same)) != NF_OK || (st = nf::check_side(a.k, head_dim, same)) != NF_OK)
        return st;
    const uintptr_t in_size = in_dtype == NF_DTYPE_F32 ? 4 : 2, out_size = out_dtype == NF_DTYPE_F32 ? 4 : 2;
    if (!nf::aligned(q, in_size) || !nf::aligned(k, in_size) || !nf::aligned(q_out, out_size) ||
        !nf::aligned(k_out, out_size))
        return NF_ERR_INVALID_ARGUMENT;
    if (num_tokens == 0 || n_q_heads + n_kv_heads == 0) return NF_OK;
    if ((st = nf::check_on_device(n_q_heads ? q : nullptr, n_q_heads ? q_out : nullptr, n_kv_heads ? k : nullptr,
                                  n_kv_heads ? k_out : nullptr, positions, inv_freq)) != NF_OK)
        return st;
    a.positions = positions;
    a.freq = inv_freq;
    a.scale = cos_sin_scale;
    a.T = num_tokens;
    a.d = head_dim;
    a.rot = rot_dim;
    a.interleaved = interleaved;
    a.copy = (n_q_heads && q != q_out) || (n_kv_heads && k != k_out);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e =
        in_dtype == NF_DTYPE_F32
            ? (out_dtype == NF_DTYPE_F32 ? nf::launch<float, float>(a, s) : nf::launch<float, uint16_t>(a, s))
            : (out_dtype == NF_DTYPE_F32 ? nf::launch<uint16_t, float>(a, s) : nf::launch<uint16_t, uint16_t>(a, s));
    return e == cudaSuccess ? NF_OK : NF_ERR_CUDA;
} catch (...) {
    return NF_ERR_INVALID_ARGUMENT;
}
