// Microscaled 4-bit floating point: quantization, reading back, and the load-time layout of weights.
//
// Canonical form of a [T][d] tensor: uint8 codes [T][d/2] (channel 2m in the low nibble; sign, two
// exponent bits, one mantissa bit) and uint8 scales [T][d/32] (2^(byte - 127); 255 is NaN).
//
// All three kernels are bound by memory: each element crosses it once in either form.  (A large copy
// reaches 4.3 to 5.0 TB/s here, a large read 5.2.)

#include <algorithm>

#include "qe_act.h"
#include "qe_internal.h"
#include "qe_mx4.h"

namespace qe {

// ---------------------------------------------------------------- quantization
// A thread owns 8 channels (a block is 4 neighbouring lanes) and walks down the rows with them, so
// the smoothing factors and their reciprocals are loaded and divided once per column, not once per
// element.  Workgroup: `cc` chunks of 8 channels across, 256 / cc rows down; grid: column segments x
// row ranges of `rows` rows.  4093 x 14336 bf16 with factors 33 us (4.5 TB/s), 29568 x 8192 float32 228 us
// (4.8).  Loads past the caches were 8 % faster on cold bf16 rows, but 6 % slower on float32 and 15 % on
// rows that the kernel before had left in the caches; requesting a row ahead changed nothing.
template <bool kBf16, int kSmooth>  // kSmooth: 0 none, 1 divide, 2 multiply
__global__ __launch_bounds__(256) void mx4_quant_kernel(const void* __restrict__ x, const float* __restrict__ smooth,
                                                        int T, int d, int cc, int rows, uint8_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales) {
    const int rr = threadIdx.x / cc, c = threadIdx.x - rr * cc;
    const int step = blockDim.x / cc;
    const int j = (blockIdx.x * cc + c) * 8;
    if (j >= d || rr >= step) return;
    float s[8], is[8];
    bool s_ok = true;
    if constexpr (kSmooth != 0) {
        load8(smooth, QE_F32, j, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (kSmooth == 1) is[i] = 1.0f / s[i];
        }
        s_ok = code_div_ok(s);
    }
    const long t0 = (long)blockIdx.y * rows, t1 = min((long)T, t0 + rows);
    for (long t = t0 + rr; t < t1; t += step) {
        float v[8];
        load8(x, kBf16 ? QE_BF16 : QE_F32, (size_t)t * d + j, v);
        if constexpr (kSmooth == 1) {
            code_div8(v, s, is, s_ok);
        } else if constexpr (kSmooth == 2) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= s[i];
        }
        mx4_store8(v, codes + (size_t)t * (d / 2), scales + (size_t)t * (d / 32), j);
    }
}

hipError_t launch_mx4_quant(const void* x, int x_dtype, const float* smooth, bool multiply, int T, int d,
                            uint8_t* codes, uint8_t* scales, hipStream_t st) {
    if (T <= 0) return hipSuccess;
    // chunks across (a multiple of 4: whole blocks), rows down, and enough row ranges to fill the GPU
    const int cc = std::min(d / 8, 256), segs = (d / 8 + cc - 1) / cc, step = 256 / cc;
    const long want = std::max(1l, (long)T * segs / step / 4096);  // passes of a workgroup down its rows
    int rows = (int)std::min<long>(want * step, T);
    while ((T + (long)rows - 1) / rows > 65535) rows *= 2;
    const dim3 grid(segs, (unsigned)((T + (long)rows - 1) / rows)), block(256);
    const int sm = !smooth ? 0 : multiply ? 2 : 1;
#define QE_MXQ(BF, SM) \
    hipLaunchKernelGGL((mx4_quant_kernel<BF, SM>), grid, block, 0, st, x, smooth, T, d, cc, rows, codes, scales)
    if (x_dtype == QE_BF16) {
        if (sm == 0) QE_MXQ(true, 0);
        else if (sm == 1) QE_MXQ(true, 1);
        else QE_MXQ(true, 2);
    } else {
        if (sm == 0) QE_MXQ(false, 0);
        else if (sm == 1) QE_MXQ(false, 1);
        else QE_MXQ(false, 2);
    }
#undef QE_MXQ
    return hipGetLastError();
}

// ---------------------------------------------------------------- reading back
// A thread turns the 4 bytes of 8 codes into values; every value is exact in float32 and bf16
// (two significant bits; float32 also holds the products with scales down to 2^-127).
// 29568 x 8192 into bf16: 118 us, 5.2 TB/s.
__device__ inline float mx4_value(uint32_t code, float scale) {
    // magnitude bits: exponent e and mantissa m give (1 + m/2) 2^(e-1), or m/2 for e = 0
    const uint32_t e = (code >> 1) & 3u, m = code & 1u;
    const float mag = e ? __uint_as_float(((e + 126u) << 23) | (m << 22)) : 0.5f * (float)m;
    return (code & 8u) ? -(mag * scale) : mag * scale;
}

__device__ inline float mx4_scale(uint32_t byte) {  // 2^(byte - 127); 255: NaN
    return byte == 255u ? __uint_as_float(0x7FC00000u) : byte == 0u ? 0x1p-127f : __uint_as_float(byte << 23);
}

template <bool kBf16>
__global__ __launch_bounds__(256) void mx4_dequant_kernel(const uint32_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales, size_t n8,
                                                          void* __restrict__ x) {
    const size_t stride = (size_t)gridDim.x * 256;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += stride) {
        const uint32_t c = codes[i];
        const float s = mx4_scale(scales[i >> 2]);
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = mx4_value((c >> (4 * k)) & 15u, s);
        if constexpr (kBf16) {
            v4u o;
#pragma unroll
            for (int k = 0; k < 4; ++k)  // exact above bf16's smallest normal number; rounded to nearest below
                o[k] = mx4_bf16_bits(v[2 * k]) | (mx4_bf16_bits(v[2 * k + 1]) << 16);
            reinterpret_cast<v4u*>(x)[i] = o;
        } else {
            v4f* p = reinterpret_cast<v4f*>(x) + 2 * i;
            p[0] = v4f{v[0], v[1], v[2], v[3]};
            p[1] = v4f{v[4], v[5], v[6], v[7]};
        }
    }
}

hipError_t launch_mx4_dequant(const uint8_t* codes, const uint8_t* scales, int T, int d, void* x, int x_dtype,
                              hipStream_t st) {
    const size_t n8 = (size_t)T * d / 8;
    if (n8 == 0) return hipSuccess;
    const unsigned grid = (unsigned)std::min<size_t>((n8 + 255) / 256, 256 * 32);
    if (x_dtype == QE_BF16)
        hipLaunchKernelGGL(mx4_dequant_kernel<true>, dim3(grid), dim3(256), 0, st,
                           reinterpret_cast<const uint32_t*>(codes), scales, n8, x);
    else
        hipLaunchKernelGGL(mx4_dequant_kernel<false>, dim3(grid), dim3(256), 0, st,
                           reinterpret_cast<const uint32_t*>(codes), scales, n8, x);
    return hipGetLastError();
}

// ---------------------------------------------------------------- load-time layout
// Codes: tiles of 32 channels x 64 K, 1 KB each, ordered (channel block, 128-wide K step, half step,
// lane): lane l owns channel 32*nb + l%32 and the 32 codes k = 128*kb + 64*h + 32*(l/32) + [0, 32),
// one operand fragment of the 32x32x64 product and exactly one scale block.  Scales: one dword per
// channel and K step, byte i the scale of its block i, ordered (channel block, K step, channel).
// Channels past d_out (an odd number of 16-channel groups) hold zeros.
//
// The same layout holds a product's activations (rows: tokens, in the order of perm when it is given).  A wave
// reads two steps of 32 rows, 64 bytes per row and step, and writes them as 512-byte pieces.
// 29568 x 8192 46 us (5.6 TB/s of both), 4096 x 8192 out of the caches 9.
__global__ __launch_bounds__(256) void mx4_tile_kernel(const uint8_t* __restrict__ codes,
                                                       const uint8_t* __restrict__ scales,
                                                       const int32_t* __restrict__ perm, int rows, int d_in,
                                                       v4u* __restrict__ tiled, uint32_t* __restrict__ tiled_scale) {
    const int KB = d_in / 128, NB = (rows + 31) / 32;
    const size_t n = (size_t)NB * KB * 32, stride = (size_t)gridDim.x * 256;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += stride) {
        const int l = (int)(i & 31);
        const size_t q = i >> 5;  // (row block, K step)
        const int nb = (int)(q / KB), kb = (int)(q - (size_t)nb * KB);
        const int pos = nb * 32 + l;
        v4u c[4] = {v4u{0, 0, 0, 0}, v4u{0, 0, 0, 0}, v4u{0, 0, 0, 0}, v4u{0, 0, 0, 0}};
        uint32_t sc = 0;
        if (pos < rows) {
            const size_t r = perm ? perm[pos] : pos;
            const v4u* p = reinterpret_cast<const v4u*>(codes + r * (d_in / 2) + (size_t)kb * 64);
#pragma unroll
            for (int k = 0; k < 4; ++k) c[k] = p[k];
            sc = *reinterpret_cast<const uint32_t*>(scales + r * (d_in / 32) + kb * 4);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) tiled[q * 128 + k * 32 + l] = c[k];  // chunk k: half step k / 2, lanes 32 (k % 2) + l
        tiled_scale[q * 32 + l] = sc;
    }
}

hipError_t launch_mx4_tile(const uint8_t* codes, const uint8_t* scales, const int32_t* perm, int rows, int d_in,
                           uint8_t* tiled, uint32_t* tiled_scale, hipStream_t st) {
    const size_t n = (size_t)((rows + 31) / 32) * (d_in / 128) * 32;
    const unsigned grid = (unsigned)std::min<size_t>((n + 255) / 256, 256 * 16);
    hipLaunchKernelGGL(mx4_tile_kernel, dim3(grid), dim3(256), 0, st, codes, scales, perm, rows, d_in,
                       reinterpret_cast<v4u*>(tiled), tiled_scale);
    return hipGetLastError();
}

}  // namespace qe
