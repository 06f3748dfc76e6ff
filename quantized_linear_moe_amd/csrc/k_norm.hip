// Residual addition + RMS norm, with the normed row also written as the activation codes of the
// quantized linear that reads it (what stands between two linears of a decoder layer).
//
//   h  = rn(x + res)                              (res NULL: h = x)
//   r  = float32(1 / sqrt(sum_j h[j]^2 / d + eps))   sums, root and quotient in 64 bits
//   xn = rn((h * r) * w)                          float32 products, one rounding to the row's type
//   codes of xn / smooth: per-token integers (a_bits 6, 8: as qe_quant_act makes them from xn) or
//   microscaled 4-bit blocks (a_bits 4: as qe_mx4_quant makes them from xn)
//
// The sum is kept in 64 bits because the codes are decided at rounding borders: with it the factor
// r is the correctly rounded one, so xn and its codes do not depend on the order of the additions.
//
// One workgroup per token; every thread keeps its channels in registers from the load to the last
// store, so each tensor crosses memory once.

#include <algorithm>

#include "qe_act.h"
#include "qe_internal.h"
#include "qe_mx4.h"

namespace qe {

__device__ inline double wave_sum(double v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

// 8 consecutive float32 values to the row's type (bf16: round to nearest even), and the values the
// stored elements hold
template <bool kBf16>
__device__ inline void store8(void* p, size_t idx, float v[8]) {
    if constexpr (kBf16) {
        v4u o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = mx4_bf16_bits(v[2 * i]), hi = mx4_bf16_bits(v[2 * i + 1]);
            o[i] = lo | (hi << 16);
        }
        if (p) *reinterpret_cast<v4u*>(reinterpret_cast<uint16_t*>(p) + idx) = o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(o[i] << 16);
            v[2 * i + 1] = __uint_as_float(o[i] & 0xFFFF0000u);
        }
    } else if (p) {
        v4f* q = reinterpret_cast<v4f*>(reinterpret_cast<float*>(p) + idx);
        q[0] = v4f{v[0], v[1], v[2], v[3]};
        q[1] = v4f{v[4], v[5], v[6], v[7]};
    }
}

// kMode: 0 no codes, 4 microscaled blocks, 8 per-token integers (6 or 8 bits: qmax).
// IT: groups of 8 channels per thread.
template <bool kBf16, int kMode, int IT>
__global__ __launch_bounds__(1024) void add_rmsnorm_kernel(const void* x, const void* res, const void* __restrict__ w,
                                                           int w_dtype, float eps, int d, void* h, void* xn,
                                                           const float* __restrict__ smooth, int qmax,
                                                           uint8_t* __restrict__ codes, void* __restrict__ scales) {
    constexpr int kDt = kBf16 ? QE_BF16 : QE_F32;
    const size_t t = blockIdx.x, row = t * (size_t)d;
    const int nthr = blockDim.x, wid = threadIdx.x / kWave, lane = threadIdx.x % kWave, nw = nthr / kWave;
    __shared__ double red_s[16];
    __shared__ float red_m[16];

    float v[IT][8];
    double sum = 0.0;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
        const int j = (it * nthr + threadIdx.x) * 8;
        if (j >= d) continue;
        load8(x, kDt, row + j, v[it]);
        if (res) {
            float r[8];
            load8(res, kDt, row + j, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[it][i] += r[i];
            store8<kBf16>(h, row + j, v[it]);
        } else if (h) {
            store8<kBf16>(h, row + j, v[it]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += (double)v[it][i] * (double)v[it][i];
    }
    sum = wave_sum(sum);
    if (lane == 0) red_s[wid] = sum;
    __syncthreads();
    sum = red_s[0];
    for (int i = 1; i < nw; ++i) sum += red_s[i];
    const float r = (float)(1.0 / sqrt(sum / (double)d + (double)eps));

    float amax = 0.0f;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
        const int j = (it * nthr + threadIdx.x) * 8;
        if (j >= d) continue;
        float wv[8];
        load8(w, w_dtype, j, wv);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[it][i] = (v[it][i] * r) * wv[i];
        store8<kBf16>(xn, row + j, v[it]);
        if constexpr (kMode != 0) {
            if (smooth) smooth8<false>(smooth, nullptr, j, v[it]);
        }
        if constexpr (kMode == 4) {
            mx4_store8(v[it], codes + row / 2, reinterpret_cast<uint8_t*>(scales) + row / 32, j);
        } else if constexpr (kMode == 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, __builtin_fabsf(v[it][i]));
        }
    }
    if constexpr (kMode == 8) {
        amax = wave_max(amax);
        if (lane == 0) red_m[wid] = amax;
        __syncthreads();
        amax = red_m[0];
        for (int i = 1; i < nw; ++i) amax = fmaxf(amax, red_m[i]);
        const float sx = amax / (float)qmax;
        if (threadIdx.x == 0) reinterpret_cast<float*>(scales)[t] = sx;
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const int j = (it * nthr + threadIdx.x) * 8;
            if (j >= d) continue;
            *reinterpret_cast<v2u*>(codes + row + j) = quant8(v[it], sx, (float)qmax);
        }
    }
}

template <bool kBf16, int kMode>
static void launch_norm(int it, int threads, int T, const void* x, const void* res, const void* w, int w_dtype,
                        float eps, int d, void* h, void* xn, const float* smooth, int qmax, uint8_t* codes,
                        void* scales, hipStream_t st) {
#define QE_NORM(IT_)                                                                                                 \
    hipLaunchKernelGGL((add_rmsnorm_kernel<kBf16, kMode, IT_>), dim3(T), dim3(threads), 0, st, x, res, w, w_dtype,  \
                       eps, d, h, xn, smooth, qmax, codes, scales)
    if (it == 1) QE_NORM(1);
    else QE_NORM(4);
#undef QE_NORM
}

hipError_t launch_add_rmsnorm(const void* x, const void* res, int x_dtype, const void* w, int w_dtype, float eps,
                              int T, int d, void* h, void* xn, const float* smooth, int a_bits, uint8_t* codes,
                              void* scales, hipStream_t st) {
    const int groups = d / 8;
    const int it = groups <= 256 ? 1 : 4;
    const int threads = ((groups + it - 1) / it + kWave - 1) / kWave * kWave;
    if (threads > 1024) return hipErrorInvalidValue;  // d > 32768: rejected by the caller
    const int mode = a_bits == 0 ? 0 : a_bits == 4 ? 4 : 8;
    const int qmax = mode == 8 ? (1 << (a_bits - 1)) - 1 : 0;
    const bool bf = x_dtype == QE_BF16;
#define QE_NORM_MODE(M)                                                                                              \
    if (mode == M) {                                                                                                 \
        if (bf) launch_norm<true, M>(it, threads, T, x, res, w, w_dtype, eps, d, h, xn, smooth, qmax, codes, scales, st); \
        else launch_norm<false, M>(it, threads, T, x, res, w, w_dtype, eps, d, h, xn, smooth, qmax, codes, scales, st);  \
    }
    QE_NORM_MODE(0)
    QE_NORM_MODE(4)
    QE_NORM_MODE(8)
#undef QE_NORM_MODE
    return hipGetLastError();
}

}  // namespace qe
