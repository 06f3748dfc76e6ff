// Microscaled 4-bit floating point (blocks of 32 along a row): the block format's device helpers and
// the launch wrappers of its kernels (k_mx4.hip, k_gemm_mx4.hip) and of the fused norm (k_norm.hip).
#pragma once

#include "qe_internal.h"

namespace qe {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef int v8i __attribute__((ext_vector_type(8)));

constexpr int kMxBlock = 32;         // elements that share a scale
constexpr int kMxMaxRows = 1 << 30;  // tokens and output channels of a product: tile ends stay below 2^31
constexpr int kMxMaxTStream = 64;    // token counts served by the weight-streaming product

// float32 -> bf16 bits, round to nearest even, NaN kept
__device__ inline uint32_t mx4_bf16_bits(float f) {
    const __bf16 b = (__bf16)f;
    return (uint32_t)__builtin_bit_cast(uint16_t, b);
}

// largest of a 32-bit unsigned value over the 4 lanes 4q..4q+3 (all active)
__device__ inline uint32_t quad_umax(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));  // lanes 1,0,3,2
    return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));  // lanes 2,3,0,1
}

// Codes of 8 values over the scale 2^(sc - 127); low: some lane of the wave has sc == 0
__device__ inline uint32_t mx4_pack8(const float v[8], uint32_t sc, bool low) {
    uint32_t c = 0;
    if (__builtin_expect(low, 0)) {
        // scale 2^-127 is not a normal float32: twice the values over 2^-126 (exact, all below 2^-123)
        const float f = sc == 0u ? 2.0f : 1.0f, s = __uint_as_float(max(sc, 1u) << 23);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0] * f, v[1] * f, s, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2] * f, v[3] * f, s, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4] * f, v[5] * f, s, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6] * f, v[7] * f, s, 3);
    } else {
        const float s = __uint_as_float(sc << 23);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
    }
    return c;
}

// The block form of 8 channels j..j+7 of one row, the other 24 of the block in the neighbouring
// lanes of the quad (lane 4q + i holds the block's channels 8i..8i+7): with E = floor(log2 amax)
// the block's scale is 2^(E - 2) (byte E - 2 + 127, at least 0), and the codes are the values
// over it rounded to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (ties to the even code), at most 6.
// amax is compared as bits, so a NaN or an infinity is the largest: such a block gets scale byte
// 255 (NaN) and zero codes.
__device__ inline uint32_t mx4_codes8(const float v[8], uint32_t* scale_byte) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    const uint32_t field = quad_umax(m) >> 23;
    const uint32_t sc = field == 255u ? 255u : field > 2u ? field - 2u : 0u;
    *scale_byte = sc;
    const uint32_t c = mx4_pack8(v, sc, __any(sc == 0u));
    return sc == 255u ? 0u : c;
}

// A whole block held by one lane: its 16 bytes of codes
__device__ inline v4u mx4_codes32(const float v[4][8], uint32_t* scale_byte) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) m = max(m, __float_as_uint(v[i >> 3][i & 7]) & 0x7FFFFFFFu);
    const uint32_t field = m >> 23;
    const uint32_t sc = field == 255u ? 255u : field > 2u ? field - 2u : 0u;
    *scale_byte = sc;
    const bool low = __any(sc == 0u);
    v4u out;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t c = mx4_pack8(v[q], sc, low);
        out[q] = sc == 255u ? 0u : c;
    }
    return out;
}

// mx4_codes8 into a row's codes and scales
__device__ inline void mx4_store8(const float v[8], uint8_t* codes_row, uint8_t* scales_row, int j) {
    uint32_t sc;
    const uint32_t c = mx4_codes8(v, &sc);
    *reinterpret_cast<uint32_t*>(codes_row + j / 2) = c;
    if ((j & 31) == 0) scales_row[j >> 5] = (uint8_t)sc;
}

// ------------------------------------------------------------------ launch wrappers
hipError_t launch_add_rmsnorm(const void* x, const void* res, int x_dtype, const void* w, int w_dtype, float eps,
                              int T, int d, void* h, void* xn, const float* smooth, int a_bits, uint8_t* codes,
                              void* scales, hipStream_t st);
hipError_t launch_mx4_quant(const void* x, int x_dtype, const float* smooth, bool multiply, int T, int d,
                            uint8_t* codes, uint8_t* scales, hipStream_t st);
hipError_t launch_mx4_dequant(const uint8_t* codes, const uint8_t* scales, int T, int d, void* x, int x_dtype,
                              hipStream_t st);
// canonical codes and scales of [rows][d_in] into the product's tiles (see k_mx4.hip), rows in the
// order of `perm` when it is given
hipError_t launch_mx4_tile(const uint8_t* codes, const uint8_t* scales, const int32_t* perm, int rows, int d_in,
                           uint8_t* tiled, uint32_t* tiled_scale, hipStream_t st);
// launch_expert_quant with microscaled codes: as rows, or (tiled) as the tiles of launch_mx4_tile in the
// order of perm, which it writes (no routes: token order)
hipError_t launch_expert_mx4(const uint16_t* x, int T, int d_in, const float* smooth, const float* inv_smooth,
                             const int32_t* expert, int n_r, const uint16_t* mt_re, int rr_pad, int r_r, int ksq,
                             int32_t* perm, float* vpart, uint8_t* codes, uint8_t* scales, bool tiled, uint16_t* v,
                             hipStream_t st);
// launch_xproj_finish of a forward (routes, u, v) and the codes and scales of x in one launch
hipError_t launch_xproj_finish_mx4(const float* part, int ksplit, int T, int ncols_pad, int col0, int se_col, int r_s,
                                   int rs_pad, int re_col, int n_r, int r_r, int rr_pad, int router_col,
                                   int32_t* expert, uint16_t* u, uint16_t* v, const void* x, int x_dtype, int d_in,
                                   const float* smooth, const float* inv_smooth, uint8_t* codes, uint8_t* scales,
                                   hipStream_t st);
// bytes of the tiles of [rows][d_in] (codes, scales)
inline size_t mx4_tile_codes(size_t rows, size_t d_in) { return (rows + 31) / 32 * 32 * d_in / 2; }
inline size_t mx4_tile_scales(size_t rows, size_t d_in) { return (rows + 31) / 32 * 32 * d_in / kMxBlock; }

// How the product runs for T tokens: which kernel and how many K splits (more than one: float32
// partials [ksplit][T][d_out] in the workspace, added by a finish kernel)
struct Mx4Plan {
    int bm, bn;  // tokens and channels of a tile; 0: weight streaming (T <= kMxMaxTStream)
    int ksplit;
};
Mx4Plan mx4_plan(int T, int d_in, int d_out);
// Whether its activations come as tiles.  Making them is a launch (3 us, 10 at 4096 x 8192), for 128-token
// tiles worth it on long sums: 512 x 29568 -> 8192 113 us from rows, 88 from tiles; 1024 x 8192 -> 8192 53, 49;
// 2048 x 4096 -> 4096 31.7, 32.3; 384 x 3584 -> 18944 32, 37.
inline bool mx4_tiled(const Mx4Plan& P, int d_in) { return P.bm == 256 || (P.bm == 128 && d_in >= 8192); }

struct Mx4Gemm {
    const uint8_t* codes;      // [T][d_in/2] or NULL
    const uint8_t* scales;     // [T][d_in/32] or NULL
    const uint8_t* w_tiled;
    const uint32_t* w_scale;
    const uint16_t* u;         // [T][rs_pad] or NULL
    const uint16_t* bt_s;      // [d_out][rs_pad]
    const uint16_t* v;         // [T][rr_pad] or NULL
    const int32_t* expert;     // [T]
    const uint16_t* bt_r;      // [n_r][d_out][rr_pad]
    const int32_t* perm;       // [T] or NULL
    float* y;                  // [T][d_out] (bf16 elements when y_bf16)
    float* part;               // [ksplit][T][d_out] when ksplit > 1
    uint8_t* a_tiled;          // the activations' tiles (128- and 256-token tiles), in the order of perm: made
    uint32_t* a_scale;         // from codes and scales when those are given, else already there
    int T, d_in, d_out, rs_pad, rr_pad, n_r;
    bool y_bf16;
};
hipError_t launch_mx4_gemm(const Mx4Gemm& G, const Mx4Plan& P, hipStream_t st);

}  // namespace qe
