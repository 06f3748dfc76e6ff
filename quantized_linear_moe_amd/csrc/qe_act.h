// Device helpers of the activation-side kernels: loading activations as float32, the exact
// smoothing division, and wave reductions.
#pragma once

#include "qe_internal.h"

namespace qe {

__device__ inline float bf16_bits_to_f32(uint32_t h) { return __uint_as_float(h << 16); }

// a / b correctly rounded, given inv_b = RN(1/b).  One multiply and two fused
// multiply-adds (Markstein's correction).  Exact for |a| in [2^-100, 2^100] and b
// in [2^-90, 2^90] with quotients of magnitude >= 2^-3; callers fall back to the
// IEEE division outside that domain.  The remainder is taken as b q0 - a: of a zero it is +0, and the last
// step, q0 - 0, keeps q0's sign (a - b q0 would turn -0 / b into +0).
__device__ inline float div_markstein(float a, float b, float inv_b) {
    float q0 = a * inv_b;
    float r = __builtin_fmaf(b, q0, -a);
    return __builtin_fmaf(-r, inv_b, q0);
}

__device__ inline bool in_markstein_range(float a) {
    float m = __builtin_fabsf(a);
    return (m >= 0x1p-100f && m <= 0x1p100f) || m == 0.0f;
}

// x / s exactly as IEEE float32 division
__device__ inline float smooth_div(float x, float s, float inv_s) {
    return in_markstein_range(x) ? div_markstein(x, s, inv_s) : x / s;
}

// load 8 consecutive activations as float
__device__ inline void load8(const void* x, int x_dtype, size_t idx, float out[8]) {
    if (x_dtype == QE_BF16) {
        v4u p = *reinterpret_cast<const v4u*>(reinterpret_cast<const uint16_t*>(x) + idx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            out[2 * i] = __uint_as_float(p[i] << 16);
            out[2 * i + 1] = __uint_as_float(p[i] & 0xFFFF0000u);
        }
    } else {
        const v4f* p = reinterpret_cast<const v4f*>(reinterpret_cast<const float*>(x) + idx);
        v4f a = p[0], b = p[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            out[i] = a[i];
            out[4 + i] = b[i];
        }
    }
}

__device__ inline float wave_max(float v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
    return v;
}

// x / s for 8 consecutive channels (exactly the IEEE division), with or without stored reciprocals
template <bool kHasInv>
__device__ inline void smooth8(const float* __restrict__ smooth, const float* __restrict__ inv_smooth, int j,
                               float v[8]) {
    const v4f s0 = *reinterpret_cast<const v4f*>(smooth + j), s1 = *reinterpret_cast<const v4f*>(smooth + j + 4);
    float s[8] = {s0[0], s0[1], s0[2], s0[3], s1[0], s1[1], s1[2], s1[3]};
    float is[8];
    if (kHasInv) {
        const v4f i0 = *reinterpret_cast<const v4f*>(inv_smooth + j), i1 = *reinterpret_cast<const v4f*>(inv_smooth + j + 4);
        is[0] = i0[0]; is[1] = i0[1]; is[2] = i0[2]; is[3] = i0[3];
        is[4] = i1[0]; is[5] = i1[1]; is[6] = i1[2]; is[7] = i1[3];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) is[i] = 1.0f / s[i];
    }
    bool ok = true;
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        r[i] = div_markstein(v[i], s[i], is[i]);
        ok = ok && in_markstein_range(v[i]);
    }
    if (__builtin_expect(__any(!ok), 0)) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!in_markstein_range(v[i])) r[i] = v[i] / s[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r[i];
}

// largest |v| of 8 values (NaN: ignored)
__device__ inline float absmax8(const float v[8]) {
    float m = __builtin_fabsf(v[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = fmaxf(m, __builtin_fabsf(v[i]));
    return m;
}

// v / s for 8 channels whose factors' reciprocals are kept, as codes need it: exactly the IEEE quotient,
// except that a quotient too small to get a code other than zero may be off.  One range check serves the 8
// values: with all s in [2^-20, 2^20] (s_ok) and their largest |v| in [2^-40, 2^100], the corrected quotient
// is exact for |v| >= 2^-100, and a smaller |v| gives less than 2^-80 beside a largest quotient of at
// least 2^-60, far below half a code.  Otherwise the division itself.
__device__ inline void code_div8(float v[8], const float s[8], const float is[8], bool s_ok) {
    const float m = absmax8(v);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = div_markstein(v[i], s[i], is[i]);
    if (__builtin_expect(__any(!(s_ok && (m == 0.0f || (m >= 0x1p-40f && m <= 0x1p100f)))), 0)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = v[i] / s[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = q[i];
}
__device__ inline bool code_div_ok(const float s[8]) {
    bool ok = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) ok = ok && s[i] >= 0x1p-20f && s[i] <= 0x1p20f;
    return ok;
}

// 8 per-token integer codes clamp(rint(v / sx), -fq, fq) (sx == 0: zeros; NaN: -fq), packed, for sx = max |v| / fq.
// A normal sx keeps every quotient within fq (1 + 2^-23), but a subnormal one is off by up to a third of itself,
// and a NaN gets its code from the clamp: one instruction per value (4096 x 8192, 8 bits: 65.0 us, without it 64.5;
// 2048 x 1536, 6 bits: 9.85, 9.77).  Adding 1.5 * 2^23 rounds to the nearest even integer, whose two's complement
// low byte is then the sum's.
__device__ inline v2u quant8(const float v[8], float sx, float fq) {
    const float inv = sx != 0.0f ? 1.0f / sx : 0.0f;
    const bool fast = sx >= 0x1p-90f && sx <= 0x1p90f;  // (the same in the whole row)
    uint32_t b[8];
    if (fast) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            b[i] = __float_as_uint(__builtin_amdgcn_fmed3f(div_markstein(v[i], sx, inv), -fq, fq) + 12582912.0f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            b[i] = sx != 0.0f ? __float_as_uint(__builtin_amdgcn_fmed3f(v[i] / sx, -fq, fq) + 12582912.0f) : 0u;
    }
    v2u out;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t lo = __builtin_amdgcn_perm(b[4 * k + 1], b[4 * k], 0x0C0C0400u);
        const uint32_t hi = __builtin_amdgcn_perm(b[4 * k + 3], b[4 * k + 2], 0x04000C0Cu);
        out[k] = lo | hi;
    }
    return out;
}

}  // namespace qe
