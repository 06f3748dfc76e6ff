// Rotary positions of query heads, and keys and values appended to the paged cache with the keys rotated on the way.
//
//   a = pos * inv_freq[i] (float64);  c = float32(scale cos a), s = float32(scale sin a)
//   (x1, x2) -> (x1 c - x2 s, x2 c + x1 s) in float32, one rounding to the output's type
//   8-bit cache: scale = max |x'| / 127 over the head, codes as qe_quant_act makes them
//
// Angles of far positions lose their fraction in 32 bits (10^6 radians: a step of 0.06), so the angle and its sine and
// cosine are taken in 64 bits, once per token and pair for all its heads, into LDS.  A workgroup takes one token (few
// heads: several); a lane takes 16 channels of a head as two vectors of 8, whose pairs both lie in the lane.
//
// Bound by memory where there are many tokens: x read once, y written once.  4093 tokens of 64 heads of 128 channels (bf16,
// three rows of positions): 23 us, 5.8 TB/s; 4096 tokens appended with 64 query and 8 key heads: 36 us, 4.7 TB/s; 777 with
// 32 and 8 heads to 8-bit codes: 8.8 us.  One token: 2.4 us, a launch and its trips to memory.
#include <algorithm>

#include "qe_act.h"
#include "qe_cache.h"
#include "qe_mx4.h"

namespace qe {

namespace {

constexpr int kRopeThreads = 256;  // at most
constexpr int kRopeTokens = 16;  // tokens of a workgroup at most

struct RopeArgs {
    const void* x[3];
    int64_t x_stride[3];
    int heads[3];
    int T, head_dim, tokens, parts;  // tokens of a workgroup, workgroups of a token
    int lanes, lane_shift;    // lanes of a head: the power of two at or above head_dim / 16
    int rot, n_pos, sec0, sec1;
    double scale;
    const double* inv_freq;
    const int32_t* pos;
    void* q_out;
    int64_t q_out_stride;
    int q_out_bf16;
    void* cache[2];
    float* cache_scale[2];
    int page_shift;
    uint32_t slots;
    const int32_t* slot;
};

// Sine and cosine of a (|a| < 2^33): a less the nearest multiple of pi / 2, which is taken off in two parts of 53 bits
// each with one rounding apiece (the rest of pi / 2, below 2^-108, times 2^33 does not count), then the Taylor sums of both
// functions on [-pi / 4, pi / 4], whose first terms left out are below 2^-54 and 2^-58: float64 values good to a few of
// their last places, of which float32 keeps 24 bits.  The math library's sincos, whose branch for huge arguments needs
// scratch memory, took the kernel for 4093 x 64 heads from 27 us to 160.
__device__ inline void sin_cos(double a, double* s, double* c) {
    constexpr double kHalfPiHi = 0x1.921fb54442d18p+0, kHalfPiLo = 0x1.1a62633145c07p-54;
    const double n = __builtin_rint(a * 0x1.45f306dc9c883p-1);
    const double r = __builtin_fma(-n, kHalfPiLo, __builtin_fma(-n, kHalfPiHi, a));
    const double z = r * r;
    double p = -1.0 / 1307674368000.0, q = 1.0 / 20922789888000.0;
    p = __builtin_fma(p, z, 1.0 / 6227020800.0);
    q = __builtin_fma(q, z, -1.0 / 87178291200.0);
    p = __builtin_fma(p, z, -1.0 / 39916800.0);
    q = __builtin_fma(q, z, 1.0 / 479001600.0);
    p = __builtin_fma(p, z, 1.0 / 362880.0);
    q = __builtin_fma(q, z, -1.0 / 3628800.0);
    p = __builtin_fma(p, z, -1.0 / 5040.0);
    q = __builtin_fma(q, z, 1.0 / 40320.0);
    p = __builtin_fma(p, z, 1.0 / 120.0);
    q = __builtin_fma(q, z, -1.0 / 720.0);
    p = __builtin_fma(p, z, -1.0 / 6.0);
    q = __builtin_fma(q, z, 1.0 / 24.0);
    q = __builtin_fma(q, z, -0.5);
    const double sr = __builtin_fma(r * z, p, r), cr = __builtin_fma(z, q, 1.0);
    const int k = (int)(long long)n & 3;  // quarter turns
    const double u = k & 1 ? cr : sr, w = k & 1 ? sr : cr;
    *s = k & 2 ? -u : u;
    *c = (k + 1) & 2 ? -w : w;
}

__device__ inline void store8_as(void* p, size_t idx, const float v[8], bool bf16) {
    if (bf16) {
        v4u o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = mx4_bf16_bits(v[2 * i]) | (mx4_bf16_bits(v[2 * i + 1]) << 16);
        *reinterpret_cast<v4u*>(reinterpret_cast<uint16_t*>(p) + idx) = o;
    } else {
        v4f* q = reinterpret_cast<v4f*>(reinterpret_cast<float*>(p) + idx);
        q[0] = v4f{v[0], v[1], v[2], v[3]};
        q[1] = v4f{v[4], v[5], v[6], v[7]};
    }
}

// A lane's 16 channels of one head: which they are, and their values
struct Item {
    int part, head, ch0, ch1;  // part 0 q, 1 k, 2 v; -1: none
    long t;
    bool turn;
    int pair0;
    float a[8], b[8];
};

template <bool kBf16, bool kPairs>
__device__ inline void load_item(const RopeArgs& A, int item, int n_items, long t0, Item& I) {
    const int per_token = (A.heads[0] + A.heads[1] + A.heads[2]) << A.lane_shift;
    const int tok = A.tokens == 1 ? 0 : item / per_token, rest = item - tok * per_token;
    int head = rest >> A.lane_shift;
    const int lane = rest & (A.lanes - 1);
    I.t = t0 + tok;
    I.part = -1;
#pragma unroll
    for (int i = 0; i < 8; ++i) I.a[i] = I.b[i] = 0.0f;
    if (item >= n_items || I.t >= A.T || lane * 16 >= A.head_dim) return;
    int part = 0;
    if (head >= A.heads[0]) {
        head -= A.heads[0];
        part = 1;
        if (head >= A.heads[1]) {
            head -= A.heads[1];
            part = 2;
        }
    }
    I.part = part;
    I.head = head;
    I.turn = part < 2 && lane * 16 < A.rot;
    I.pair0 = 8 * lane;
    const bool halves = I.turn && !kPairs;
    I.ch0 = halves ? 8 * lane : 16 * lane;
    I.ch1 = halves ? A.rot / 2 + 8 * lane : 16 * lane + 8;
    // (values, not members, on the arms: a choice between members would put the arguments into scratch memory)
    const void *xq = A.x[0], *xk = A.x[1], *xv = A.x[2];
    const int64_t sq = A.x_stride[0], sk = A.x_stride[1], sv = A.x_stride[2];
    const void* x = part == 0 ? xq : part == 1 ? xk : xv;
    const int64_t stride = part == 0 ? sq : part == 1 ? sk : sv;
    const size_t at = (size_t)I.t * stride + (size_t)head * A.head_dim;
    load8(x, kBf16 ? QE_BF16 : QE_F32, at + I.ch0, I.a);
    load8(x, kBf16 ? QE_BF16 : QE_F32, at + I.ch1, I.b);
}

// (the layout is a template's: with both in one kernel the compiler keeps the channels in scratch memory)
template <bool kPairs>
__device__ inline void turn_item(const RopeArgs& A, const float2 (*cs)[kMaxHeadDim / 2], long t0, Item& I) {
    const float2* p = cs[I.t - t0] + I.pair0;
    if constexpr (!kPairs) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float c = p[i].x, s = p[i].y, x1 = I.a[i], x2 = I.b[i];
            I.a[i] = x1 * c - x2 * s;
            I.b[i] = x2 * c + x1 * s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float c = p[i].x, s = p[i].y, x1 = I.a[2 * i], x2 = I.a[2 * i + 1];
            I.a[2 * i] = x1 * c - x2 * s;
            I.a[2 * i + 1] = x2 * c + x1 * s;
            const float c2 = p[4 + i].x, s2 = p[4 + i].y, y1 = I.b[2 * i], y2 = I.b[2 * i + 1];
            I.b[2 * i] = y1 * c2 - y2 * s2;
            I.b[2 * i + 1] = y2 * c2 + y1 * s2;
        }
    }
}

// (every lane of the wave calls it: the 8-bit form takes the largest value over a head's lanes)
template <bool kI8>
__device__ inline void store_item(const RopeArgs& A, const Item& I) {
    if (I.part == 0) {
        const size_t at = (size_t)I.t * A.q_out_stride + (size_t)I.head * A.head_dim;
        store8_as(A.q_out, at + I.ch0, I.a, A.q_out_bf16);
        store8_as(A.q_out, at + I.ch1, I.b, A.q_out_bf16);
    }
    float sx = 0.0f;
    if constexpr (kI8) {
        float m = fmaxf(absmax8(I.a), absmax8(I.b));
        for (int off = A.lanes >> 1; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, kWave));
        sx = m / 127.0f;
    }
    if (I.part < 1) return;
    const uint32_t slot = (uint32_t)A.slot[I.t];
    if (slot >= A.slots) return;  // (negative: padding)
    const bool val = I.part == 2;
    const int heads = A.heads[1];
    const size_t row = ((((size_t)(slot >> A.page_shift) * heads + I.head) << A.page_shift)) +
                       (slot & ((1u << A.page_shift) - 1));
    void *ck = A.cache[0], *cv = A.cache[1];
    float *ks = A.cache_scale[0], *vs = A.cache_scale[1];
    void* dst = val ? cv : ck;
    if constexpr (kI8) {
        uint8_t* o = reinterpret_cast<uint8_t*>(dst) + row * A.head_dim;
        *reinterpret_cast<v2u*>(o + I.ch0) = quant8(I.a, sx, 127.0f);
        *reinterpret_cast<v2u*>(o + I.ch1) = quant8(I.b, sx, 127.0f);
        if (I.pair0 == 0) (val ? vs : ks)[row] = sx;
    } else {
        store8_as(dst, row * A.head_dim + I.ch0, I.a, true);
        store8_as(dst, row * A.head_dim + I.ch1, I.b, true);
    }
}

template <bool kBf16, bool kPairs, bool kI8>
__global__ __launch_bounds__(kRopeThreads, 4) void rope_kernel(RopeArgs A) {
    __shared__ float2 cs[kRopeTokens][kMaxHeadDim / 2];
    const long t0 = (long)(blockIdx.x / A.parts) * A.tokens;
    const int n_items = A.tokens * ((A.heads[0] + A.heads[1] + A.heads[2]) << A.lane_shift);
    const int item = (int)(blockIdx.x % A.parts) * kRopeThreads + (int)threadIdx.x;
    Item now;
    load_item<kBf16, kPairs>(A, item, n_items, t0, now);  // (under way while the angles are worked out)
    const int pairs = A.rot / 2;
    for (int i = threadIdx.x; i < A.tokens * pairs; i += blockDim.x) {
        const int tok = A.tokens == 1 ? 0 : i / pairs, p = i - tok * pairs;
        if (t0 + tok >= A.T) break;
        const int row = A.n_pos == 1 ? 0 : p < A.sec0 ? 0 : p < A.sec0 + A.sec1 ? 1 : 2;
        double s, c;
        sin_cos((double)A.pos[(size_t)row * A.T + t0 + tok] * A.inv_freq[p], &s, &c);
        cs[tok][p] = make_float2((float)(c * A.scale), (float)(s * A.scale));
    }
    __syncthreads();
    if (now.part >= 0 && now.turn) turn_item<kPairs>(A, cs, t0, now);
    store_item<kI8>(A, now);
}

}  // namespace

hipError_t launch_rope(const RopeLaunch& R, hipStream_t st) {
    RopeArgs A = {};
    for (int i = 0; i < 3; ++i) {
        A.x[i] = R.x[i];
        A.x_stride[i] = R.x_stride[i];
        A.heads[i] = R.x[i] ? R.heads[i] : 0;
    }
    A.T = R.T;
    A.head_dim = R.head_dim;
    while (16 << A.lane_shift < R.head_dim) ++A.lane_shift;
    A.lanes = 1 << A.lane_shift;
    const long per_token = (long)(A.heads[0] + A.heads[1] + A.heads[2]) << A.lane_shift;
    A.tokens = (int)std::max<long>(1, std::min<long>(kRopeTokens, 256 / per_token));
    const long items = A.tokens * per_token;
    A.parts = (int)((items + kRopeThreads - 1) / kRopeThreads);
    const int threads = (int)std::min<long>(kRopeThreads, (items + kWave - 1) / kWave * kWave);
    if (R.rope) {
        A.rot = R.rope->rot_dim;
        A.n_pos = R.rope->n_pos;
        A.sec0 = R.rope->sections[0];
        A.sec1 = R.rope->sections[1];
        A.scale = R.rope->scale;
        A.inv_freq = R.rope->inv_freq;
    }
    A.pos = R.pos;
    A.q_out = R.q_out;
    A.q_out_stride = R.q_out_stride;
    A.q_out_bf16 = R.q_out_bf16;
    if (R.cache) {
        A.cache[0] = R.cache->k;
        A.cache[1] = R.cache->v;
        A.cache_scale[0] = R.cache->k_scale;
        A.cache_scale[1] = R.cache->v_scale;
        while (1 << A.page_shift < R.cache->page_size) ++A.page_shift;
        A.slots = (uint32_t)R.cache->n_pages * (uint32_t)R.cache->page_size;
        A.slot = R.slot;
    }
    const long groups = ((long)R.T + A.tokens - 1) / A.tokens * A.parts;
    const dim3 grid((unsigned)groups);
    const bool pairs = R.rope && R.rope->layout == QE_ROPE_PAIRS;
    const bool i8 = R.cache && R.cache->dtype == QE_I8;
#define QE_ROPE_LAUNCH(B, P)                                                                          \
    do {                                                                                              \
        if (i8) hipLaunchKernelGGL((rope_kernel<B, P, true>), grid, dim3(threads), 0, st, A);         \
        else hipLaunchKernelGGL((rope_kernel<B, P, false>), grid, dim3(threads), 0, st, A);           \
    } while (0)
    if (R.x_bf16 && pairs) QE_ROPE_LAUNCH(true, true);
    else if (R.x_bf16) QE_ROPE_LAUNCH(true, false);
    else if (pairs) QE_ROPE_LAUNCH(false, true);
    else QE_ROPE_LAUNCH(false, false);
#undef QE_ROPE_LAUNCH
    return hipGetLastError();
}

}  // namespace qe
