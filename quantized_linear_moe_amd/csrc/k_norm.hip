// Residual addition + RMS norm, with the normed row also written as the activation codes of the
// quantized linear that reads it (what stands between two linears of a decoder layer).
//
//   h  = rn(x + res)                              (res NULL: h = x)
//   r  = float32(1 / sqrt(sum_j h[j]^2 / d + eps))   sums, root and quotient in 64 bits
//   xn = rn((h * r) * w)                          float32 products, one rounding to the row's type
//   codes of xn / smooth: per-token integers (a_bits 6, 8: as qe_quant_act makes them from xn) or
//   microscaled 4-bit blocks (a_bits 4: as qe_mx4_quant makes them from xn)
//
// The sum is kept in 64 bits because the codes are decided at rounding borders: of at most 32768 exact squares
// it is off by less than 2^-37 relative in any order of the additions, so r is the correctly rounded factor
// unless the exact one lies that close to a border between two float32 values.
//
// A workgroup takes rows in turn and its threads the same channels of each: the norm weight, the
// smoothing factors and their reciprocals stay in registers, the next row is requested before the current
// one is reduced, and each element crosses memory once: bound by memory when large.  4096 x 8192
// bf16 with residual: 54 us without codes (5.0 TB/s, a large copy's rate), 65 with microscaled ones (4.4),
// 67 with 8 bits (4.5; its second reduction); 2048 x 1536 with 6 bits 10; one row of 1536 3.
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
        for (int i = 0; i < 4; ++i) o[i] = mx4_bf16_bits(v[2 * i]) | (mx4_bf16_bits(v[2 * i + 1]) << 16);
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

// 8 consecutive elements as loaded, and their values
template <bool kBf16>
struct Raw8 {
    v4u w[kBf16 ? 1 : 2];
    __device__ inline void load(const void* p, size_t idx) {
        const v4u* q = reinterpret_cast<const v4u*>(reinterpret_cast<const uint8_t*>(p) + idx * (kBf16 ? 2 : 4));
#pragma unroll
        for (int i = 0; i < (kBf16 ? 1 : 2); ++i) w[i] = q[i];
    }
    __device__ inline float operator[](int i) const {
        if constexpr (kBf16) return __uint_as_float(i & 1 ? w[0][i >> 1] & 0xFFFF0000u : w[0][i >> 1] << 16);
        else return __uint_as_float(w[i >> 2][i & 3]);
    }
};

// kMode: 0 no codes, 4 microscaled blocks, 8 per-token integers (6 or 8 bits: qmax).
// IT: groups of 8 channels per thread; with 4 (rows over 16384 channels) the registers do not hold the
// weights and factors too, and they are loaded for every row.
template <bool kBf16, int kMode, int IT>
__global__ __launch_bounds__(1024) void add_rmsnorm_kernel(const void* x, const void* res, const void* __restrict__ w,
                                                           int w_dtype, float eps, int T, int d, void* h, void* xn,
                                                           const float* __restrict__ smooth, int qmax,
                                                           uint8_t* __restrict__ codes, void* __restrict__ scales) {
    const int nthr = blockDim.x, wid = threadIdx.x / kWave, lane = threadIdx.x % kWave, nw = nthr / kWave;
    // two sets, used in turn: a row's partial sums are read before the next row's barrier, so that one
    // barrier per reduction is enough
    __shared__ double red_s[2][16];
    __shared__ float red_m[2][16];

    constexpr bool kKeep = IT <= 2;
    float wv[kKeep ? IT : 1][8], s[kKeep && kMode ? IT : 1][8], is[kKeep && kMode ? IT : 1][8];
    bool s_ok = true;
    const bool smoothed = kMode != 0 && smooth != nullptr;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
        const int j = (it * nthr + threadIdx.x) * 8;
        if (j >= d || !kKeep) continue;
        load8(w, w_dtype, j, wv[it]);
        if constexpr (kMode != 0) {
            if (!smoothed) continue;
            load8(smooth, QE_F32, j, s[it]);
#pragma unroll
            for (int i = 0; i < 8; ++i) is[it][i] = 1.0f / s[it][i];
            s_ok = s_ok && code_div_ok(s[it]);
        }
    }
    Raw8<kBf16> px[IT], pr[IT];  // the next row
    auto request = [&](long t) {
        if (t >= T) return;
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const int j = (it * nthr + threadIdx.x) * 8;
            if (j >= d) continue;
            px[it].load(x, (size_t)t * d + j);
            if (res) pr[it].load(res, (size_t)t * d + j);
        }
    };
    request(blockIdx.x);
    int turn = 0;
    for (long t = blockIdx.x; t < T; t += gridDim.x, turn ^= 1) {
        const size_t row = (size_t)t * d;
        float v[IT][8];
        double sum = 0.0;
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const int j = (it * nthr + threadIdx.x) * 8;
            if (j >= d) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[it][i] = res ? px[it][i] + pr[it][i] : px[it][i];
            if (res || h) store8<kBf16>(h, row + j, v[it]);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += (double)v[it][i] * (double)v[it][i];
        }
        request(t + gridDim.x);
        sum = wave_sum(sum);
        if (lane == 0) red_s[turn][wid] = sum;
        __syncthreads();
        sum = red_s[turn][0];
        for (int i = 1; i < nw; ++i) sum += red_s[turn][i];
        const float r = (float)(1.0 / sqrt(sum / (double)d + (double)eps));

        float amax = 0.0f;
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const int j = (it * nthr + threadIdx.x) * 8;
            if (j >= d) continue;
            const int k = kKeep ? it : 0;
            if constexpr (!kKeep) load8(w, w_dtype, j, wv[0]);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[it][i] = (v[it][i] * r) * wv[k][i];
            store8<kBf16>(xn, row + j, v[it]);
            if constexpr (kMode != 0) {
                if (smoothed) {
                    if constexpr (!kKeep) {
                        load8(smooth, QE_F32, j, s[0]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) is[0][i] = 1.0f / s[0][i];
                        s_ok = code_div_ok(s[0]);
                    }
                    code_div8(v[it], s[k], is[k], s_ok);
                }
            }
            if constexpr (kMode == 4) {
                mx4_store8(v[it], codes + row / 2, reinterpret_cast<uint8_t*>(scales) + row / 32, j);
            } else if constexpr (kMode == 8) {
                amax = fmaxf(amax, absmax8(v[it]));
            }
        }
        if constexpr (kMode == 8) {
            amax = wave_max(amax);
            if (lane == 0) red_m[turn][wid] = amax;
            __syncthreads();
            amax = red_m[turn][0];
            for (int i = 1; i < nw; ++i) amax = fmaxf(amax, red_m[turn][i]);
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
}

// Threads per row and rows per workgroup.  One group of 8 channels per thread up to 4096 channels, two up to
// 16384 (4096 x 8192 with codes of 8 bits: 67 us; with one, in 1024 threads, 90; with four, whose kept
// factors spill, 170), else four without keeping factors.  About 1024 threads per CU take rows in turn:
// 2048 are as fast for long rows but give every workgroup half the rows to spread its factors over
// (2048 x 3584, 8 bits: 22.5 us against 20.1).
template <bool kBf16, int kMode>
static void launch_norm(int T, const void* x, const void* res, const void* w, int w_dtype, float eps, int d, void* h,
                        void* xn, const float* smooth, int qmax, uint8_t* codes, void* scales, hipStream_t st) {
    const int groups = d / 8, it = groups <= 512 ? 1 : groups <= 2048 ? 2 : 4;
    const int threads = ((groups + it - 1) / it + kWave - 1) / kWave * kWave;
    const dim3 grid(std::min(T, std::max(256, 256 * (1024 / threads)))), block(threads);
#define QE_NORM(IT_)                                                                                               \
    hipLaunchKernelGGL((add_rmsnorm_kernel<kBf16, kMode, IT_>), grid, block, 0, st, x, res, w, w_dtype, eps, T, d, \
                       h, xn, smooth, qmax, codes, scales)
    if (it == 1) QE_NORM(1);
    else if (it == 2) QE_NORM(2);
    else QE_NORM(4);
#undef QE_NORM
}

hipError_t launch_add_rmsnorm(const void* x, const void* res, int x_dtype, const void* w, int w_dtype, float eps,
                              int T, int d, void* h, void* xn, const float* smooth, int a_bits, uint8_t* codes,
                              void* scales, hipStream_t st) {
    if (T <= 0) return hipSuccess;
    if (d > 32768) return hipErrorInvalidValue;  // rejected by the caller
    const int qmax = a_bits >= 6 ? (1 << (a_bits - 1)) - 1 : 0;
#define QE_NORM_MODE(M)                                                                                          \
    if (x_dtype == QE_BF16)                                                                                      \
        launch_norm<true, M>(T, x, res, w, w_dtype, eps, d, h, xn, smooth, qmax, codes, scales, st);             \
    else                                                                                                         \
        launch_norm<false, M>(T, x, res, w, w_dtype, eps, d, h, xn, smooth, qmax, codes, scales, st)
    if (a_bits == 0) {
        QE_NORM_MODE(0);
    } else if (a_bits == 4) {
        QE_NORM_MODE(4);
    } else {
        QE_NORM_MODE(8);
    }
#undef QE_NORM_MODE
    return hipGetLastError();
}

}  // namespace qe
