// Attention of new tokens over the paged cache: o = softmax(scale q K^T + mask) V, causal or along a tree of drafts.
//
// Transposed products keep a query in one lane of a half wave: S^T = K Q^T puts query l % 32 in lane l with 16 of the
// keys of a 32-key block, 8 (i / 4) + 4 (l / 32) + i % 4, so the softmax needs one exchange between the lane halves per
// tile (the maximum), its weights are the B operand of O^T = V^T P^T as they lie (V^T is read from LDS in the same key
// order by transposing reads), and the running factors of O^T are per lane.
//
//   m' = max(m, c + max_j s_j), taken over only when it exceeds m by 8 (in units of log2);
//   l' = l 2^(m - m') + sum_j 2^(s_j - m'), o' = o 2^(m - m') + sum_j 2^(s_j - m') v_j, all in float32
//
// with c = 8 + the bits of the number of keys, so that a weight is at most 2^(8 - c) and all of them at most 1 together:
// o stays within the values' own range, whatever it is.  The exponent s - m' is then off by up to c 2^-24 (1.3e-6 at 8192
// keys), little beside the weights' rounding to bf16 (2^-8).  At the other end, what lies below 2^-126 in the sums of o is
// kept to steps of 2^-149, but a weight times an 8-bit value's scale is lost there.
//
// The weights are rounded to bf16 for the matrix cores (at most 2^-8 relative each, as the values they multiply were); l
// is summed from the rounded weights, so that what is divided by is the sum of what was multiplied (8-bit cache: from the
// unrounded ones, as the values' scales go into the weights).
//
// Rows of a sequence and key head are its tokens times its group of query heads.  Two forms:
//   many rows: a wave has 32 rows, the waves of a workgroup share tiles of 64 keys
//   few rows (at most 32): every wave has them all, and its own tiles of 32 keys in turn; the waves' results join in LDS
// Long sequences of few workgroups are split into pieces of `chunk` keys whose unnormalised results join in a second
// kernel, in order.  Keys past the sequence or of a page outside the cache are never read: their rows come from a zero
// constant, so that whatever those places hold stays out of the products; of keys that only some rows see (later ones, other
// branches) neither scores nor values reach the other rows.
//
// Bounds (kernel times of runs of 0.25 s; after a pause the first 50 or so large launches take up to a quarter more, until the
// clock has settled).
// A prompt: 4096 tokens, 64 heads on 8 key heads of 128 channels: 276 to 280 us, 0.98 to 1.0 PFLOP/s (a large bf16
// product: 1.15 to 1.26).  The matrix cores are busy 46 % of the cycles at 2.14 GHz, where the single tokens below run
// at 2.46, and taking out a part of any of the loop's work (products, exponentials, LDS reads, copies) shortened it in
// proportion to that part: the readings of a part held by power, though power itself was not read.  Tiles of 64 keys
// in two buffers and 4 waves leave room for two workgroups per CU, of which one computes while the other waits (one
// per CU: 362 us; 8 waves: +3 %; scores a tile ahead in the same wave: +1 % or spills).  The form of 128 channels and
// bf16 has 256 registers and 8 bytes of scratch memory, outside its loops.  8-bit cache: 353 us, as every workgroup
// turns the codes of its tiles into bf16; heads of 64 channels: 158, as many exponentials for half the products; both:
// 242.
// Single tokens: memory.  64 sequences of 512 to 8192 keys: 210 us, 5.4 TB/s of the cache's bytes.
// Trees: rows that fill no tile of 128, the pieces' unlike ends and the join.  8 trees of 7 to 48 tokens over up to 4000
// keys, 28 heads on 4, 8-bit cache: 26 us and 5 to 6 of the join.
#include <algorithm>
#include <cmath>

#include "qe_cache.h"
#include "qe_dma.h"
#include "qe_mx4.h"

namespace qe {

namespace {

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef uint16_t v2us __attribute__((ext_vector_type(2)));

constexpr float kLowest = -3.402823466e38f;
constexpr float kLazy = 8.0f;
__device__ inline float lift_of(int keys) { return kLazy + (float)(32 - __builtin_clz(max(keys, 1))); }  // c above

__device__ __attribute__((aligned(16))) const uint32_t kZero16[4] = {0, 0, 0, 0};

struct AttnArgs {
    const uint16_t* q;
    int64_t q_stride;
    const uint8_t *k, *v;
    const float *ks, *vs;
    const int32_t *q_start, *kv_len, *pages;
    const uint32_t* tree;
    int tree_words;
    int T, n_heads, n_kv, group, n_seq, max_pages, n_pages, page_shift, max_q, max_kv;
    int row_tiles, splits, chunk;
    float sc;  // scale log2(e)
    uint16_t* out;
    int64_t out_stride;
    float* part_o;
    float2* part_ml;
};

// A sequence's new tokens [first, first + n) and keys (clamped to what the arguments allow).  Which keys the new tokens are
// goes by the length as given: what the bounds cut off is missing, and nothing else moves.
struct Seq {
    int first, n, len, ctx;  // ctx: keys before the new tokens, at most len (may be negative)
};
__device__ inline Seq seq_of(const AttnArgs& A, int s) {
    Seq q;
    q.first = min(max(A.q_start[s], 0), A.T);
    const int n = min(max(A.q_start[s + 1], q.first), A.T) - q.first;
    q.n = min(n, A.max_q);
    const long cap = min((long)A.max_kv, (long)A.max_pages << A.page_shift);
    const int given = max(A.kv_len[s], 0);
    q.len = (int)min((long)given, cap);
    q.ctx = min(given - n, q.len);  // (ctx + n is at most given: 31 bits)
    return q;
}

__device__ inline float half_max(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ inline float half_sum(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Order of the 16-byte pieces of a key's row in LDS, chosen so that the reads below touch every bank once:
// K's rows are read at one piece by lanes of consecutive keys, V's by 4 consecutive keys at 64 bytes
template <int HD>
__device__ inline int k_swizzle(int row) {
    return HD == 128 ? row & 15 : (row >> 1) & 7;
}
template <int HD>
__device__ inline int v_swizzle(int row) {
    return HD == 128 ? (row & 3) << 2 : ((row >> 1) & 1) << 2;
}

// 16 codes to bf16 (exact)
__device__ inline void codes_to_bf16(v4u c, v4u out[2]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int w = (int)c[i];
        const uint32_t f0 = __float_as_uint((float)(int8_t)w), f1 = __float_as_uint((float)(int8_t)(w >> 8));
        const uint32_t f2 = __float_as_uint((float)(int8_t)(w >> 16)), f3 = __float_as_uint((float)(int8_t)(w >> 24));
        out[i >> 1][2 * (i & 1)] = __builtin_amdgcn_perm(f1, f0, 0x07060302u);
        out[i >> 1][2 * (i & 1) + 1] = __builtin_amdgcn_perm(f3, f2, 0x07060302u);
    }
}

// A sequence's page numbers, 64 at a time in the lanes and the next 64 beside them (-1: no such page).  The first are
// requested before the sequence's length is known, to make one trip to memory of both; later ones are waited for as they
// are read (they are checked there), one trip to memory every 64 pages.
struct Pages {
    const int32_t* p;
    int width, n, n_pages, base, now, next;
    uint64_t ok;  // of the 64 at hand

    __device__ inline int read(int i) const { return (uint32_t)i < (uint32_t)width ? p[i] : -1; }
    __device__ inline int checked(int i, int v) const { return i < n && (uint32_t)v < (uint32_t)n_pages ? v : -1; }
    __device__ inline void early(const AttnArgs& A, int seq, int first) {
        p = A.pages + (size_t)seq * A.max_pages;
        width = A.max_pages;
        n_pages = A.n_pages;
        base = first;
        const int i = first + (int)(threadIdx.x % kWave);
        now = read(i);
        next = read(i + kWave);
    }
    __device__ inline void init(int len, int shift) {
        n = (len + (1 << shift) - 1) >> shift;
        const int i = base + (int)(threadIdx.x % kWave);
        now = checked(i, now);
        next = checked(i + kWave, next);
        ok = __ballot(now >= 0);
    }
    // the 64 with page i, which lies in them or behind
    __device__ inline void seek(int i) {
        while (i - base >= kWave) {
            base += kWave;
            now = next;
            const int j = base + kWave + (int)(threadIdx.x % kWave);
            next = checked(j, read(j));
            ok = __ballot(now >= 0);
        }
    }
    __device__ inline int page(int i) const { return __builtin_amdgcn_readlane(now, i - base); }
    __device__ inline bool whole(int k0, int n_keys, int shift, int len) const {
        const uint64_t need = (1 << shift) >= n_keys ? 1 : (1ull << (n_keys >> shift)) - 1;
        return (ok >> ((k0 >> shift) - base) & need) == need && k0 + n_keys <= len;
    }
    // which of the n <= 64 keys from k0 on (the first of a page, or all in one) there are
    __device__ inline uint64_t keys(int k0, int n_keys, int shift, int len) const {
        const int i = (k0 >> shift) - base;
        uint64_t m = ~0ull;
        if ((1 << shift) >= n_keys) {
            m = ok >> i & 1 ? ~0ull : 0;
        } else {
            const uint64_t run = (1ull << (1 << shift)) - 1;
            m = 0;
            for (int k = 0; k << shift < n_keys; ++k)
                if (ok >> (i + k) & 1) m |= run << (k << shift);
        }
        const int left = len - k0;
        if (left < 64) m &= left <= 0 ? 0 : (1ull << left) - 1;
        return n_keys < 64 ? m & ((1ull << (n_keys & 63)) - 1) : m;
    }
};

// Tiles of BK keys (or values: kV) brought to LDS by NT threads (whole waves), a wave's rows of a tile at a time: runs of
// 16 keys, of one page each where pages have 16 places or more (kRuns), else every lane's own key
template <int HD, int BK, int NT, bool I8, bool kV, bool kRuns>
struct Stage {
    static constexpr int kRow = I8 ? HD : HD * 2;                      // bytes of a key in memory
    static constexpr int kCount = BK * kRow / 1024 / (NT / kWave);     // 1 KB requests of a wave
    static constexpr int kLanes = kRow / 16, kRun = kWave / kLanes;    // lanes of a key, keys of a request
    static constexpr int kGroup = 16 / kRun;                           // requests of a run
    static_assert(kCount * kRun % 16 == 0, "");
    v4u codes[I8 ? kCount : 1];
    float scale;
    uint32_t off[kCount];  // of the lane's bytes from its run's address on
    int wave, lane;

    __device__ static inline int swizzle(int row) { return kV ? v_swizzle<HD>(row) : k_swizzle<HD>(row); }
    __device__ inline int row_of(int j) const { return (wave * kCount + j) * kRun + lane / kLanes; }

    __device__ inline void init(int tid) {
        wave = NT == kWave ? 0 : __builtin_amdgcn_readfirstlane(tid / kWave);
        lane = tid % kWave;
#pragma unroll
        for (int j = 0; j < kCount; ++j) {
            const int c = lane % kLanes;
            off[j] = (j % kGroup * kRun + lane / kLanes) * kRow + ((I8 ? c : c ^ swizzle(row_of(j))) << 4);
        }
    }
    // bytes from the cache's start to a run
    __device__ static inline uint64_t run_at(const AttnArgs& A, int head, uint32_t page, int key) {
        return ((((uint64_t)page * A.n_kv + head) << A.page_shift) + (key & ((1 << A.page_shift) - 1))) * kRow;
    }
    // from runs that are there; at[]: run_at of the wave's runs
    __device__ inline void request_runs(const AttnArgs& A, const uint64_t (&at)[kCount / kGroup], uint32_t buf) {
        const uint8_t* base = kV ? A.v : A.k;
#pragma unroll
        for (int j = 0; j < kCount; ++j) {
            if constexpr (I8) codes[j] = *reinterpret_cast<const v4u*>(base + at[j / kGroup] + off[j]);
            else dma16_at(base + at[j / kGroup], off[j], buf + (wave * kCount + j) * 1024);
        }
    }
    // pid: the page of key k0 + lane % BK, -1 where there is none (those keys' rows are zeros)
    __device__ inline void request_keys(const AttnArgs& A, int head, int k0, int pid, uint32_t buf) {
        const uint8_t* base = kV ? A.v : A.k;
#pragma unroll
        for (int j = 0; j < kCount; ++j) {
            const int row = row_of(j), c = lane % kLanes;
            const int pg = __shfl(pid, row % BK, kWave);
            const uint8_t* p = base + run_at(A, head, (uint32_t)pg, k0 + row) + ((I8 ? c : c ^ swizzle(row)) << 4);
            if (pg < 0) p = reinterpret_cast<const uint8_t*>(kZero16);
            if constexpr (I8) codes[j] = *reinterpret_cast<const v4u*>(p);
            else dma16(p, buf + (wave * kCount + j) * 1024);
        }
    }
    __device__ inline void request_scales(const AttnArgs& A, int head, int k0, int pid) {
        scale = 0.0f;
        if (I8 && wave == 0 && lane < BK && pid >= 0)
            scale = (kV ? A.vs : A.ks)[run_at(A, head, (uint32_t)pid, k0 + lane) / kRow];
    }
    // 8-bit codes: what was requested goes to LDS (bf16 rows are copied there: wait for them)
    __device__ inline void land(uint8_t* buf, float* scales) {
        if constexpr (I8) {
#pragma unroll
            for (int j = 0; j < kCount; ++j) {
                const int row = row_of(j), c = lane % kLanes;
                v4u w[2];
                codes_to_bf16(codes[j], w);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *reinterpret_cast<v4u*>(buf + row * HD * 2 + (((2 * c + e) ^ swizzle(row)) << 4)) = w[e];
            }
            if (wave == 0 && lane < BK) scales[lane] = scale;
        }
    }
};

// Every copy of this wave has landed (rows of bf16), and its reads of the tile at hand are done: in attn_keys_kernel, whose
// waves meet no barrier, the next copies go where that tile lies
template <bool I8>
__device__ inline void landed() {
    asm volatile("" ::: "memory");  // (no read moves behind the wait)
    if constexpr (!I8) QE_WAIT_VMCNT_LDS(0);
    asm volatile("" ::: "memory");
}

// What a lane's row sees of the 32 keys from k0 on, before the sequence's end is taken into account
struct RowMask {
    int token;             // of the sequence
    const uint32_t* bits;  // its tree row, or NULL
    int words;
    uint32_t w0, w1;  // the row's first words (trees of up to 64 tokens: all there are)
    __device__ inline void init(const AttnArgs& A, const Seq& q, int row) {
        token = min(row / A.group, q.n - 1);
        bits = A.tree ? A.tree + (size_t)(q.first + token) * A.tree_words : nullptr;
        words = A.tree_words;
        w0 = A.tree ? bits[0] : 0u;
        w1 = A.tree && words > 1 ? bits[1] : 0u;
    }
    __device__ inline uint32_t word(int w) const {
        return w < 0 ? ~0u : w >= words ? 0u : w == 0 ? w0 : w == 1 ? w1 : bits[w];
    }
    __device__ inline uint32_t of(int rel) const {  // rel: k0 less the keys before the new tokens
        if (!bits) {
            const int n = token + 1 - rel;
            return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
        }
        const int w = rel >> 5, sh = rel & 31;
        return (uint32_t)(((uint64_t)word(w + 1) << 32 | word(w)) >> sh);
    }
};

template <int HD>
struct Rows {
    v8bf q[HD / 16];
    v16f o[HD / 32];
    float m, l;
};

// S^T of NS x 32 keys
template <int HD, int NS, bool I8>
__device__ inline void attn_scores(const uint8_t* kbuf, const float* ksb, const Rows<HD>& R, v16f (&s)[NS]) {
    const int lane = threadIdx.x % kWave, r = lane % 32, h = lane / 32;
    const uint8_t* kp = kbuf + r * HD * 2;
    const int kx = (h ^ k_swizzle<HD>(r)) << 4;
#pragma unroll
    for (int b = 0; b < NS; ++b) {
        s[b] = (v16f)(0.0f);
#pragma unroll
        for (int c = 0; c < HD / 16; ++c) {
            const v8bf kf = *reinterpret_cast<const v8bf*>(kp + b * 32 * HD * 2 + (kx ^ (c << 5)));
            s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, R.q[c], s[b], 0, 0, 0);
        }
    }
    if constexpr (I8) {
#pragma unroll
        for (int b = 0; b < NS; ++b)
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const v4f f = *reinterpret_cast<const v4f*>(ksb + 32 * b + 8 * a + 4 * h);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[b][4 * a + i] *= f[i];
            }
    }
}

// Keys that the lane's row does not see
template <int NS>
__device__ inline void attn_mask(const uint32_t (&seen)[NS], v16f (&s)[NS]) {
    const int h = (threadIdx.x % kWave) / 32;
#pragma unroll
    for (int b = 0; b < NS; ++b) {
        const uint32_t w = seen[b] >> (4 * h);
#pragma unroll
        for (int i = 0; i < 16; ++i) s[b][i] = (w >> (8 * (i / 4) + i % 4)) & 1u ? s[b][i] : -__builtin_inff();
    }
}

template <int NS>
__device__ inline float attn_max(const v16f (&s)[NS]) {
    float mx = s[0][0];
#pragma unroll
    for (int b = 0; b < NS; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[b][i]);
    return mx;
}

// The running maximum (with lift_of on it) moves where the scores (their greatest in this lane: mx) exceed it by far
template <int HD>
__device__ inline void attn_rescale(float mx, float sc, float lift, Rows<HD>& R) {
    mx = half_max(mx) * sc + lift;
    if (__any(mx > R.m + kLazy)) {
        const float m = fmaxf(R.m, mx), f = __builtin_amdgcn_exp2f(R.m - m);
        R.m = m;
        R.l *= f;
#pragma unroll
        for (int d = 0; d < HD / 32; ++d) R.o[d] *= f;
    }
}

// Whether so many bytes of values hold an infinity or a NaN
template <int BYTES>
__device__ inline bool attn_unbounded(const uint8_t* vbuf) {
    v2us top = {0, 0};
#pragma unroll
    for (int i = 0; i < BYTES / (kWave * 16); ++i) {
        const v4u w = *reinterpret_cast<const v4u*>(vbuf + (i * kWave + threadIdx.x % kWave) * 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) top = __builtin_elementwise_max(top, __builtin_bit_cast(v2us, w[e] & 0x7fff7fffu));
    }
    return __any(top[0] >= 0x7f80 || top[1] >= 0x7f80);
}

// The products of such a tile, a key at a time: what a weight of zero belongs to is left out (the matrix cores would make
// a NaN of 0 x infinity, in rows that do not see the key)
template <int HD, int NS>
__device__ inline void attn_values_each(const uint8_t* vbuf, const v8bf (&p)[NS][2], Rows<HD>& R) {
    const int lane = threadIdx.x % kWave, h = lane / 32;
    for (int j = 0; j < 32 * NS; ++j) {
        const int at = (j >> 5) * 8 + ((j >> 3) & 3) * 2 + ((j >> 1) & 1);  // of the pair of weights with key j's
        uint32_t u = 0;
#pragma unroll
        for (int b = 0; b < NS; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (8 * b + 4 * e + i == at) u = __builtin_bit_cast(v4u, p[b][e])[i];
        const float w = __shfl(__uint_as_float(j & 1 ? u & 0xffff0000u : u << 16), lane % 32 + ((j >> 2) & 1) * 32, kWave);
#pragma unroll
        for (int d = 0; d < HD / 32; ++d)
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const int piece = (4 * d + a) ^ v_swizzle<HD>(j);
                const v2u x = *reinterpret_cast<const v2u*>(vbuf + j * HD * 2 + (piece << 4) + 8 * h);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v = __uint_as_float(e & 1 ? x[e / 2] & 0xffff0000u : x[e / 2] << 16);
                    R.o[d][4 * a + e] = w == 0.0f ? R.o[d][4 * a + e] : __builtin_fmaf(w, v, R.o[d][4 * a + e]);
                }
            }
    }
}

// Weights of the scores and their products with V.  kMasked: some rows may not see all the tile's keys, and what those
// hold, infinities and NaN too, must not reach them (looking for those takes 1 us of a call with a tile of 64 to mask)
template <int HD, int NS, bool I8, bool kMasked>
__device__ inline void attn_values(const uint8_t* vbuf, const float* vsb, float sc, const v16f (&s)[NS], Rows<HD>& R,
                                   bool look = true) {
    const int lane = threadIdx.x % kWave, h = lane / 32;
    v8bf p[NS][2];
#pragma unroll
    for (int b = 0; b < NS; ++b) {
        v16f w = s[b];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(w[i], sc, -R.m));
        if constexpr (I8) {
#pragma unroll
            for (int i = 0; i < 16; ++i) R.l += w[i];
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const v4f f = *reinterpret_cast<const v4f*>(vsb + 32 * b + 8 * a + 4 * h);
#pragma unroll
                for (int i = 0; i < 4; ++i) w[4 * a + i] = kMasked && w[4 * a + i] == 0.0f ? 0.0f : w[4 * a + i] * f[i];
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            v4u u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const v2f two = {w[8 * e + 2 * i], w[8 * e + 2 * i + 1]};
                const v2bf pk = __builtin_convertvector(two, v2bf);
                if constexpr (!I8) {
                    const v2bf one = {(__bf16)1.0f, (__bf16)1.0f};
                    R.l = __builtin_amdgcn_fdot2_f32_bf16(pk, one, R.l, false);
                }
                u[i] = __builtin_bit_cast(uint32_t, pk);
            }
            p[b][e] = __builtin_bit_cast(v8bf, u);
        }
    }
    if constexpr (kMasked && !I8) {
        if (look && __builtin_expect(attn_unbounded<NS * 32 * HD * 2>(vbuf), 0)) {
            attn_values_each<HD, NS>(vbuf, p, R);
            return;
        }
    }
    // V^T: lane l reads 4 keys of channel l % 32 at a time, through its group of 16 lanes
    const int g = (lane >> 4) & 1, i16 = lane & 15;
    const int vrow = 4 * h + (i16 >> 2);
    const uint8_t* vp = vbuf + vrow * HD * 2 + ((i16 & 1) << 3);
    const int vx = (((g << 1) | ((i16 >> 1) & 1)) ^ v_swizzle<HD>(vrow)) << 4;
#pragma unroll
    for (int b = 0; b < NS; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int d = 0; d < HD / 32; ++d) {
                const uint8_t* at = vp + (32 * b + 16 * e) * HD * 2 + (vx ^ (d << 6));
                typedef __attribute__((address_space(3))) v4s* lds4;
                const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(at));
                const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(at + 8 * HD * 2));
                const v8bf vf = __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                R.o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, p[b][e], R.o[d], 0, 0, 0);
            }
}

template <int HD>
__device__ inline void load_rows(const AttnArgs& A, const Seq& q, int head, int row, Rows<HD>& R) {
    const int h = (threadIdx.x % kWave) / 32;
    const int token = row / A.group, g = row - token * A.group;
    const uint16_t* p = A.q + (size_t)(q.first + token) * A.q_stride + (size_t)(head * A.group + g) * HD + 8 * h;
#pragma unroll
    for (int c = 0; c < HD / 16; ++c) {
        v4u w = {0, 0, 0, 0};
        if (token < q.n) w = *reinterpret_cast<const v4u*>(p + 16 * c);
        R.q[c] = __builtin_bit_cast(v8bf, w);
    }
#pragma unroll
    for (int d = 0; d < HD / 32; ++d) R.o[d] = (v16f)(0.0f);
    R.m = kLowest;
    R.l = 0.0f;
}

// 4 channels of a finished row
__device__ inline void store4(uint16_t* p, const float v[4], float f) {
    v2u w;
    w[0] = mx4_bf16_bits(v[0] * f) | (mx4_bf16_bits(v[1] * f) << 16);
    w[1] = mx4_bf16_bits(v[2] * f) | (mx4_bf16_bits(v[3] * f) << 16);
    *reinterpret_cast<v2u*>(p) = w;
}

// A tile of keys as one wave sees it
template <int BK, int NT, bool kRuns>
struct Tile {
    static constexpr int kGroups = BK / 16 / (NT / kWave);  // runs of 16 keys that the wave brings
    uint64_t at[kGroups];  // where they are (whole tiles of runs)
    uint64_t valid;        // keys that there are
    int pid;               // the page of key k0 + lane % BK, -1 where there is none (set for tiles that are not whole, and
                           // for every tile of codes)
    bool whole;
};

// The tiles of a sequence, one after the other
template <int HD, int BK, int NT, bool I8, bool kRuns>
struct Tiles {
    using T = Tile<BK, NT, kRuns>;
    Pages pages;
    Stage<HD, BK, NT, I8, false, kRuns> sk;
    Stage<HD, BK, NT, I8, true, kRuns> sv;
    int head, len, shift, ahead;  // ahead: the pages of the tile after, where every lane reads its own key's

    __device__ inline void early(const AttnArgs& A, int seq, int k0) { pages.early(A, seq, k0 >> A.page_shift); }
    __device__ inline void init(const AttnArgs& A, const Seq& q, int head_, int k0, int tid) {
        head = head_;
        len = q.len;
        shift = A.page_shift;
        sk.init(tid);
        sv.init(tid);
        if constexpr (kRuns) pages.init(len, shift);
        else ahead = page_at(k0);
    }
    __device__ inline int page_at(int k0) const {  // of the lane's key
        const int key = k0 + (int)(threadIdx.x % BK);
        if (key >= len) return -1;
        const int v = pages.read(key >> shift);
        return (uint32_t)v < (uint32_t)pages.n_pages ? v : -1;
    }
    // step: from this tile to the next one asked for
    __device__ inline void locate(const AttnArgs& A, int k0, int step, T& t) {
        constexpr uint64_t kAll = BK == 64 ? ~0ull : (1ull << (BK & 63)) - 1;
        if constexpr (kRuns) {
            pages.seek(k0 >> shift);
            t.whole = pages.whole(k0, BK, shift, len);
            t.valid = kAll;
            if (t.whole) {
#pragma unroll
                for (int g = 0; g < T::kGroups; ++g) {
                    const int key = k0 + 16 * (sk.wave * T::kGroups + g);
                    t.at[g] = sk.run_at(A, head, (uint32_t)pages.page(key >> shift), key);
                }
            } else {
                t.valid = pages.keys(k0, BK, shift, len);
            }
            if (I8 || !t.whole) {
                const int i = threadIdx.x % BK;
                const int pg = __shfl(pages.now, ((k0 + i) >> shift) - pages.base, kWave);
                t.pid = t.valid >> i & 1 ? pg : -1;
            }
        } else {
            t.pid = ahead;
            ahead = page_at(k0 + step);
            t.valid = __ballot(t.pid >= 0) & kAll;
            t.whole = t.valid == kAll;
        }
    }
    template <bool kV, class S>
    __device__ inline void request(const AttnArgs& A, S& s, int k0, const T& t, uint32_t buf) {
        if (kRuns && t.whole) s.request_runs(A, t.at, buf);
        else s.request_keys(A, head, k0, t.pid, buf);
        if constexpr (I8) s.request_scales(A, head, k0, t.pid);
    }
};

// Workgroup -> key head (fastest, so that a head's tiles meet in one L2), tile of rows (the last, longest one first), piece,
// sequence (pieces last would leave the pieces that only long sequences have to the end: 8 trees of 7 to 48 tokens over
// 1100 to 4000 keys, 8-bit cache: 52 us in place of 39 with 6 pieces; trees and lengths all alike: no difference)
template <int HD, int NW, bool I8, bool kRuns>
__global__ __launch_bounds__(NW* kWave, 2) void attn_rows_kernel(AttnArgs A) {
    constexpr int BK = 64, NT = NW * kWave, TILE = BK * HD * 2;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[4 * TILE];
    __shared__ __attribute__((aligned(16))) float scales[I8 ? 4 * BK : 4];
    int id = blockIdx.x;
    const int head = id % A.n_kv;
    id /= A.n_kv;
    const int tile = A.row_tiles - 1 - id % A.row_tiles;
    id /= A.row_tiles;
    const int split = id % A.splits, seq = id / A.splits, lo = split * A.chunk;
    Tiles<HD, BK, NT, I8, kRuns> tiles;
    tiles.early(A, seq, lo);
    const Seq q = seq_of(A, seq);
    const int row0 = tile * (32 * NW), rows = q.n * A.group;
    if (row0 >= rows) return;
    const int last = min(row0 + 32 * NW, rows) - 1;
    if (split > 0 && lo >= q.len) return;  // (no such piece: the join knows the length)
    int hi = A.tree ? q.len : min(q.len, q.ctx + last / A.group + 1);
    if (A.splits > 1) hi = min(hi, lo + A.chunk);

    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid % kWave;
    const int wrow = row0 + 32 * wave, row = wrow + lane % 32;
    Rows<HD> R;
    load_rows<HD>(A, q, head, row, R);
    RowMask mask;
    mask.init(A, q, row);
    const int all = wrow >= rows ? 0 : q.ctx + (A.tree ? 0 : wrow / A.group + 1);  // keys that every row of the wave sees
    const auto seen_at = [&](int k0, uint64_t valid, uint32_t (&seen)[2]) {
        seen[0] = (uint32_t)valid & mask.of(k0 - q.ctx);
        seen[1] = (uint32_t)(valid >> 32) & mask.of(k0 + 32 - q.ctx);
    };

    const float lift = lift_of(q.len);

    uint8_t *kbuf = smem, *vbuf = smem + 2 * TILE;
    float *ksb = scales, *vsb = scales + 2 * BK;
    const uint32_t klds = lds_addr(kbuf), vlds = lds_addr(vbuf);
    if (lo < hi) {
        tiles.init(A, q, head, lo, tid);
        Tile<BK, NT, kRuns> t;
        tiles.locate(A, lo, BK, t);
        tiles.template request<false>(A, tiles.sk, lo, t, klds);
        tiles.template request<true>(A, tiles.sv, lo, t, vlds);
        landed<I8>();
        tiles.sk.land(kbuf, ksb);
        tiles.sv.land(vbuf, vsb);
        __syncthreads();
        int buf = 0, k0 = lo;
        bool more;
        Tile<BK, NT, kRuns> t2;
        const auto begin = [&] {  // the next tile is on its way while this one is computed
            more = k0 + BK < hi;
            if (more) {
                tiles.locate(A, k0 + BK, BK, t2);
                tiles.template request<false>(A, tiles.sk, k0 + BK, t2, klds + (buf ^ 1) * TILE);
                tiles.template request<true>(A, tiles.sv, k0 + BK, t2, vlds + (buf ^ 1) * TILE);
            }
        };
        const auto end = [&] {
            landed<I8>();
            buf ^= 1;
            if (more) {
                tiles.sk.land(kbuf + buf * TILE, ksb + buf * BK);
                tiles.sv.land(vbuf + buf * TILE, vsb + buf * BK);
            }
            t = t2;
            k0 += BK;
            __syncthreads();
        };
        v16f s[2];
        // tiles that need no mask first, in a loop of their own (where both forms meet, the compiler copies the
        // running rows); after the first that does, the rest are masked
        while (k0 < hi && k0 + BK <= all && t.whole) {
            begin();
            attn_scores<HD, 2, I8>(kbuf + buf * TILE, ksb + buf * BK, R, s);
            attn_rescale(attn_max<2>(s), A.sc, lift, R);
            attn_values<HD, 2, I8, false>(vbuf + buf * TILE, vsb + buf * BK, A.sc, s, R);
            end();
        }
        // a wave without rows only loads (64 sequences of 8 tokens over 512 to 8000 keys, 64 heads: 278 -> 257 us); every
        // wave meets one barrier per tile, whichever of the loops it is in
        while (wrow >= rows && k0 < hi) {
            begin();
            end();
        }
        while (k0 < hi) {
            uint32_t seen[2];
            seen_at(k0, t.valid, seen);
            begin();
            attn_scores<HD, 2, I8>(kbuf + buf * TILE, ksb + buf * BK, R, s);
            attn_mask<2>(seen, s);
            attn_rescale(attn_max<2>(s), A.sc, lift, R);
            attn_values<HD, 2, I8, true>(vbuf + buf * TILE, vsb + buf * BK, A.sc, s, R);
            end();
        }
    }
    const float l = half_sum(R.l);
    if (row >= rows) return;
    const int token = q.first + row / A.group, hq = head * A.group + row % A.group, h = lane / 32;
    if (A.splits > 1) {
        const size_t at = ((size_t)split * A.T + token) * A.n_heads + hq;
        if (h == 0) A.part_ml[at] = make_float2(R.m, l);
#pragma unroll
        for (int d = 0; d < HD / 32; ++d)
#pragma unroll
            for (int a = 0; a < 4; ++a)
                *reinterpret_cast<v4f*>(A.part_o + at * HD + 32 * d + 8 * a + 4 * h) =
                    v4f{R.o[d][4 * a], R.o[d][4 * a + 1], R.o[d][4 * a + 2], R.o[d][4 * a + 3]};
    } else {
        const float f = l > 0.0f ? 1.0f / l : 0.0f;
        uint16_t* p = A.out + (size_t)token * A.out_stride + (size_t)hq * HD + 4 * h;
#pragma unroll
        for (int d = 0; d < HD / 32; ++d)
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const float v[4] = {R.o[d][4 * a], R.o[d][4 * a + 1], R.o[d][4 * a + 2], R.o[d][4 * a + 3]};
                store4(p + 32 * d + 8 * a, v, f);
            }
    }
}

// At most 32 rows: waves take tiles of 32 keys in turn.  Rows of bf16 are copied to the other of two buffers while a tile
// is computed; codes wait in registers, so that one buffer does, and two workgroups fit a CU (64 sequences, 64 heads, 8192
// keys: 130 us and 5 of the join, with two buffers 205 in all)
template <int HD, bool I8, bool kRuns>
__global__ __launch_bounds__(256, I8 || HD == 64 ? 2 : 1) void attn_keys_kernel(AttnArgs A) {
    constexpr int BK = 32, NW = 4, STEP = NW * BK, TILE = BK * HD * 2, OLD = HD + 4, BUFS = I8 ? 1 : 2;
    constexpr int REGION = 2 * BUFS * TILE > 32 * OLD * 4 ? 2 * BUFS * TILE : (32 * OLD * 4 + 1023) / 1024 * 1024;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[NW * REGION];
    __shared__ __attribute__((aligned(16))) float scales_all[I8 ? NW * 2 * BK : 4];
    __shared__ float2 ml[NW][32];
    int id = blockIdx.x;
    const int head = id % A.n_kv;
    id /= A.n_kv;
    const int seq = id % A.n_seq, split = id / A.n_seq, lo = split * A.chunk;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid % kWave;
    int k0 = lo + wave * BK;
    Tiles<HD, BK, kWave, I8, kRuns> tiles;
    tiles.early(A, seq, k0);
    const Seq q = seq_of(A, seq);
    const int rows = q.n * A.group;
    if (rows == 0 || (split > 0 && lo >= q.len)) return;
    const int hi = A.splits > 1 ? min(q.len, lo + A.chunk) : q.len;

    const int row = lane % 32;
    Rows<HD> R;
    load_rows<HD>(A, q, head, row, R);
    RowMask mask;
    mask.init(A, q, row);
    const int all = q.ctx + (A.tree ? 0 : 1);
    const bool hidden = A.tree || all < q.len;  // there may be keys that some rows do not see

    const float lift = lift_of(q.len);

    uint8_t* mine = smem + wave * REGION;
    float* scales = scales_all + (I8 ? wave * 2 * BK : 0);
    uint8_t *kbuf = mine, *vbuf = mine + BUFS * TILE;
    float *ksb = scales, *vsb = scales + BK;
    const uint32_t klds = lds_addr(kbuf), vlds = lds_addr(vbuf);
    if (k0 < hi) {
        tiles.init(A, q, head, k0, lane);
        Tile<BK, kWave, kRuns> t, t2;
        tiles.locate(A, k0, STEP, t);
        tiles.template request<false>(A, tiles.sk, k0, t, klds);
        tiles.template request<true>(A, tiles.sv, k0, t, vlds);
        landed<I8>();
        tiles.sk.land(kbuf, ksb);
        tiles.sv.land(vbuf, vsb);
        int buf = 0;
        bool more;
        const auto begin = [&] {
            more = k0 + STEP < hi;
            if (more) {
                tiles.locate(A, k0 + STEP, STEP, t2);
                tiles.template request<false>(A, tiles.sk, k0 + STEP, t2, klds + (buf ^ 1) * TILE);
                tiles.template request<true>(A, tiles.sv, k0 + STEP, t2, vlds + (buf ^ 1) * TILE);
            }
        };
        const auto end = [&] {
            landed<I8>();
            if (!I8) buf ^= 1;
            if (more) {
                tiles.sk.land(kbuf, ksb);
                tiles.sv.land(vbuf, vsb);
            }
            t = t2;
            k0 += STEP;
        };
        v16f s[1];
        while (k0 < hi && k0 + BK <= all && t.whole) {
            begin();
            attn_scores<HD, 1, I8>(kbuf + buf * TILE, ksb, R, s);
            attn_rescale(attn_max<1>(s), A.sc, lift, R);
            attn_values<HD, 1, I8, false>(vbuf + buf * TILE, vsb, A.sc, s, R);
            end();
        }
        while (k0 < hi) {
            const uint32_t seen[1] = {(uint32_t)t.valid & mask.of(k0 - q.ctx)};
            begin();
            attn_scores<HD, 1, I8>(kbuf + buf * TILE, ksb, R, s);
            attn_mask<1>(seen, s);
            attn_rescale(attn_max<1>(s), A.sc, lift, R);
            attn_values<HD, 1, I8, true>(vbuf + buf * TILE, vsb, A.sc, s, R, hidden);
            end();
        }
    }
    // join: every wave's region holds its unnormalised rows
    const float l = half_sum(R.l);
    const int h = lane / 32;
    float* o = reinterpret_cast<float*>(mine);
    QE_WAIT_LDS();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int d = 0; d < HD / 32; ++d)
#pragma unroll
        for (int a = 0; a < 4; ++a)
            *reinterpret_cast<v4f*>(o + row * OLD + 32 * d + 8 * a + 4 * h) =
                v4f{R.o[d][4 * a], R.o[d][4 * a + 1], R.o[d][4 * a + 2], R.o[d][4 * a + 3]};
    if (h == 0) ml[wave][row] = make_float2(R.m, l);
    __syncthreads();
    const int r = tid / 8, c0 = tid % 8 * 4;  // 4 channels at a time of a row
    if (r >= rows) return;
    float M = kLowest, L = 0.0f, w[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i) M = fmaxf(M, ml[i][r].x);
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        w[i] = __builtin_amdgcn_exp2f(ml[i][r].x - M);
        L += w[i] * ml[i][r].y;
    }
    const int token = q.first + r / A.group, hq = head * A.group + r % A.group;
    const size_t at = ((size_t)split * A.T + token) * A.n_heads + hq;
    const float f = L > 0.0f ? 1.0f / L : 0.0f;
    if (A.splits > 1 && tid % 8 == 0) A.part_ml[at] = make_float2(M, L);
#pragma unroll
    for (int c = c0; c < HD; c += 32) {
        v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const v4f x = *reinterpret_cast<const v4f*>(reinterpret_cast<const float*>(smem + i * REGION) + r * OLD + c);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += w[i] * x[e];
        }
        if (A.splits > 1) {
            *reinterpret_cast<v4f*>(A.part_o + at * HD + c) = v;
        } else {
            const float u[4] = {v[0], v[1], v[2], v[3]};
            store4(A.out + (size_t)token * A.out_stride + (size_t)hq * HD + c, u, f);
        }
    }
}

// The pieces of one token and query head, by kPar groups of HD / 4 lanes that take every kPar-th piece in order, 8 pieces
// of a group requested at once (one at a time, each a trip to memory: 18 us for 32 pieces, now 4)
template <int HD, int kPar>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs A) {
    constexpr int kLanes = HD / 4, kRows = 256 / (kLanes * kPar), kBatch = 8;
    const int lane = threadIdx.x % kWave, c = lane % kLanes, part = lane / kLanes % kPar;
    const unsigned per_seq = ((unsigned)A.max_q * A.n_heads + kRows - 1) / kRows;
    const int seq = (int)(blockIdx.x / per_seq);
    const int r = (int)(blockIdx.x - seq * per_seq) * kRows + threadIdx.x / (kLanes * kPar);  // row of the sequence
    const Seq q = seq_of(A, seq);
    if (r >= q.n * A.n_heads) return;
    const int n = min(A.splits, (q.len + A.chunk - 1) / A.chunk);
    const size_t step = (size_t)A.T * A.n_heads, first = (size_t)q.first * A.n_heads + r;
    float M = kLowest, L = 0.0f;
    v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s0 = 0; s0 < n; s0 += kPar * kBatch) {
        v4f x[kBatch];
        float2 p[kBatch];
        float m = M;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int s = s0 + k * kPar + part;
            p[k] = make_float2(kLowest, 0.0f);
            x[k] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            if (s < n) {
                p[k] = A.part_ml[s * step + first];
                x[k] = *reinterpret_cast<const v4f*>(A.part_o + (s * step + first) * HD + 4 * c);
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) m = fmaxf(m, p[k].x);
        const float f = __builtin_amdgcn_exp2f(M - m);
        M = m;
        L *= f;
        v *= f;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const float w = __builtin_amdgcn_exp2f(p[k].x - M);
            L += w * p[k].y;
            v += w * x[k];
        }
    }
#pragma unroll
    for (int off = kLanes; off < kLanes * kPar; off <<= 1) {
        const float m = __shfl_xor(M, off, kWave), top = fmaxf(M, m);
        const float w = __builtin_amdgcn_exp2f(M - top), w2 = __builtin_amdgcn_exp2f(m - top);
        M = top;
        L = w * L + w2 * __shfl_xor(L, off, kWave);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = w * v[i] + w2 * __shfl_xor(v[i], off, kWave);
    }
    const float f = L > 0.0f ? 1.0f / L : 0.0f;
    if (part == 0) {
        const float u[4] = {v[0], v[1], v[2], v[3]};
        const int token = r / A.n_heads, hq = r - token * A.n_heads;
        store4(A.out + (size_t)(q.first + token) * A.out_stride + (size_t)hq * HD + 4 * c, u, f);
    }
}

template <int HD, int kPar>
void launch_join(const AttnArgs& A, hipStream_t st) {
    constexpr int kRows = 256 / (HD / 4 * kPar);
    hipLaunchKernelGGL((attn_join_kernel<HD, kPar>), dim3(((unsigned)A.max_q * A.n_heads + kRows - 1) / kRows * A.n_seq),
                       dim3(256), 0, st, A);
}

template <int HD, bool I8, bool kRuns>
void launch_hd(const AttnArgs& A, const AttnPlan& P, hipStream_t st) {
    const unsigned grid = (unsigned)((size_t)A.n_kv * P.row_tiles * A.n_seq * P.splits);
    if (P.few_rows) hipLaunchKernelGGL((attn_keys_kernel<HD, I8, kRuns>), dim3(grid), dim3(256), 0, st, A);
    else hipLaunchKernelGGL((attn_rows_kernel<HD, 4, I8, kRuns>), dim3(grid), dim3(256), 0, st, A);
    if (P.splits > 8) launch_join<HD, 64 / (HD / 4)>(A, st);
    else if (P.splits > 1) launch_join<HD, 1>(A, st);
}

template <int HD>
void launch_any(const AttnArgs& A, const AttnPlan& P, bool i8, hipStream_t st) {
    const bool runs = A.page_shift >= 4;
    if (i8 && runs) launch_hd<HD, true, true>(A, P, st);
    else if (i8) launch_hd<HD, true, false>(A, P, st);
    else if (runs) launch_hd<HD, false, true>(A, P, st);
    else launch_hd<HD, false, false>(A, P, st);
}

}  // namespace

// How many pieces: as many as fill the workgroups that run at once (few rows: 1 to 3 per CU, by LDS and registers; many
// rows: two, and some more, as sequences differ), of 128 keys or more.
//   Few rows, up to 384 keys: one, as the join costs what two or three tiles do (12 heads on 2, one sequence: 256 keys 6.3
//   us, in two pieces 7.8; 384 keys 7.3 and 7.9; 512 keys 8.2, in four 8.0).
//   Few rows, as many sequences and heads as run at once already: pieces for two rounds (where several workgroups share a
//   CU: four), of 512 keys or more, so that long sequences do not end alone (64 sequences of 512 to 8000 keys, 64 heads,
//   8-bit cache: 150 -> 135 us, with heads of 64 channels 99 -> 76; bf16, 48 sequences: 199 -> 182).
//   (The times of a tile and of a join below are those of bf16 heads of 128 channels; other forms take the same rule.)
//   Many rows: no more than pay.  A piece's rows are written and read back as float32 (8 bytes a channel at the copy
//   rate), 64 keys take a workgroup 2 us where two share a CU, and the join's launch 6: pieces cost `join` each and leave
//   whole / pieces to wait for, least at the root of their quotient.  Where every sequence has rows for all its row tiles,
//   no more than run at once, 2 per CU; where some have not, the call's tokens bound the workgroups that have work, their
//   lengths are unlike, and more of them even the CUs out (4000 keys, 28 heads, 8 trees of 48 tokens: 49 us with 5 pieces,
//   54 with 6, 60 with 7; 16 of 8 to 20 tokens with 64 heads: 59 with 5, 77 with 4; 8 of 7 to 48, 8-bit cache: 34 with
//   8, 39 with 6).  A sequence much longer than the others is still shared by 256 workgroups, or in pieces of 8192 keys.
AttnPlan attn_plan(const qe_kv_cache* cache, int n_heads, int T, int n_seq, int max_q, int max_kv) {
    AttnPlan P;
    const long group = n_heads / cache->n_kv_heads, rows = max_q * group;
    P.few_rows = rows <= 32;
    P.row_tiles = P.few_rows ? 1 : (int)((rows + 127) / 128);
    // workgroups with rows: every sequence's last tile may be a partial one
    const long tiles = (long)n_seq * P.row_tiles, filled = std::min(tiles, T * group / 128 + n_seq);
    const long base = cache->n_kv_heads * filled;
    const bool i8 = cache->dtype == QE_I8, narrow = cache->head_dim == 64;
    const long at_once = !P.few_rows ? (filled < tiles ? 720 : 512) : i8 ? (narrow ? 768 : 512) : narrow ? 512 : 256;
    long pieces = std::min(at_once / base, (max_kv + 127) / 128L);
    if (P.few_rows && max_kv <= 384) pieces = 1;
    if (P.few_rows && at_once < 2 * base)
        pieces = std::min(((at_once > 256 ? 4 : 2) * at_once + base - 1) / base, max_kv / 512L);
    if (!P.few_rows) {
        const double join = std::min((double)n_seq * max_q, (double)T) * n_heads * cache->head_dim * 8 / 5e6;  // us
        const double whole = max_kv / 64.0 * 2.0;
        pieces = std::max(1L, std::min(pieces, std::lround(std::sqrt(whole / join))));
        if (whole / pieces + pieces * join + 6.0 > whole) pieces = 1;
    }
    const long alone = (long)cache->n_kv_heads * P.row_tiles;  // workgroups of one sequence
    pieces = std::max({pieces, std::min((max_kv + 8191) / 8192L, (255 + alone) / alone), 1L});
    P.chunk = (int)std::max(((max_kv + pieces - 1) / pieces + 127) / 128 * 128, 128L);
    P.splits = std::max(1, (int)(((long)max_kv + P.chunk - 1) / P.chunk));
    return P;
}

size_t attn_partial_bytes(const AttnPlan& P, int head_dim, int T, int n_heads) {
    return P.splits > 1 ? align256((size_t)P.splits * T * n_heads * 8) + (size_t)P.splits * T * n_heads * head_dim * 4 : 0;
}

hipError_t launch_attention(const AttnLaunch& L, const AttnPlan& P, hipStream_t st) {
    AttnArgs A = {};
    const qe_kv_cache* c = L.cache;
    A.q = L.q;
    A.q_stride = L.q_stride;
    A.k = reinterpret_cast<const uint8_t*>(c->k);
    A.v = reinterpret_cast<const uint8_t*>(c->v);
    A.ks = c->k_scale;
    A.vs = c->v_scale;
    A.q_start = L.q_start;
    A.kv_len = L.kv_len;
    A.pages = L.pages;
    A.tree = L.tree;
    A.tree_words = L.tree_words;
    A.T = L.T;
    A.n_heads = L.n_heads;
    A.n_kv = c->n_kv_heads;
    A.group = L.n_heads / c->n_kv_heads;
    A.n_seq = L.n_seq;
    A.max_pages = L.max_pages;
    A.n_pages = c->n_pages;
    while (1 << A.page_shift < c->page_size) ++A.page_shift;
    A.max_q = L.max_q;
    A.max_kv = L.max_kv;
    A.row_tiles = P.row_tiles;
    A.splits = P.splits;
    A.chunk = P.chunk;
    A.sc = L.scale * 1.4426950408889634f;
    A.out = L.out;
    A.out_stride = L.out_stride;
    A.part_ml = reinterpret_cast<float2*>(L.ws);
    A.part_o = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(L.ws) +
                                        align256((size_t)P.splits * L.T * L.n_heads * 8));
    const bool i8 = c->dtype == QE_I8;
    if (c->head_dim == 128) launch_any<128>(A, P, i8, st);
    else launch_any<64>(A, P, i8, st);
    return hipGetLastError();
}

}  // namespace qe
