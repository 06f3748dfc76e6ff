// Attention of new tokens over the paged cache: o = softmax(scale q K^T + mask) V, causal or along a tree of drafts.
//
// Transposed products keep a query in one lane of a half wave: S^T = K Q^T puts query l % 32 in lane l with 16 of the
// keys of a 32-key block, 8 (i / 4) + 4 (l / 32) + i % 4, so the softmax needs one exchange between the lane halves per
// tile (the maximum), its weights are the B operand of O^T = V^T P^T as they lie (V^T is read from LDS in the same key
// order by transposing reads), and the running factors of O^T are per lane.
//
//   m' = max(m, max_j s_j), taken over only when it exceeds m by 8 (in units of log2): until then the weights
//   2^(s - m) are at most 2^8, which costs no precision in a floating-point sum;
//   l' = l 2^(m - m') + sum_j 2^(s_j - m'), o' = o 2^(m - m') + sum_j 2^(s_j - m') v_j, all in float32
//
// The weights are rounded to bf16 for the matrix cores (at most 2^-8 relative each, as the values they multiply were); l is summed
// from the rounded weights (8-bit cache: from the unrounded ones, as the values' scales go into the weights), so
// that what is divided by is the sum of what was multiplied.
//
// Rows of a sequence and key head are its tokens times its group of query heads.  Two forms:
//   many rows: a wave has 32 rows, the waves of a workgroup share tiles of 64 keys
//   few rows (at most 32): every wave has them all, and its own tiles of 32 keys in turn; the waves' results join in LDS
// Long sequences of few workgroups are split into pieces of `chunk` keys whose unnormalised results join in a second
// kernel, in order.  Keys past the sequence or of a page outside the cache are never read: their rows come from a zero
// constant, so that whatever those places hold stays out of the products.
#include <algorithm>

#include "qe_cache.h"
#include "qe_dma.h"
#include "qe_mx4.h"

namespace qe {

namespace {

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));

constexpr float kLowest = -3.402823466e38f;
constexpr float kLazy = 8.0f;

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

// A sequence's new tokens [first, first + n) and keys (clamped to what the arguments allow)
struct Seq {
    int first, n, len, ctx;  // ctx: keys before the new tokens (may be negative)
};
__device__ inline Seq seq_of(const AttnArgs& A, int s) {
    Seq q;
    q.first = min(max(A.q_start[s], 0), A.T);
    const int n = min(max(A.q_start[s + 1], q.first), A.T) - q.first;
    q.n = min(n, A.max_q);
    const long cap = min((long)A.max_kv, (long)A.max_pages << A.page_shift);
    q.len = (int)min((long)max(A.kv_len[s], 0), cap);
    q.ctx = q.len - n;
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

// Tiles of BK keys brought to LDS by NT threads (whole waves)
template <int HD, int BK, int NT, bool I8>
struct Stage {
    static constexpr int kTileBytes = BK * HD * 2;
    static constexpr int kDma = kTileBytes / 1024 / (NT / kWave);  // 1 KB copies of a wave
    static constexpr int kUnits = BK * HD / 16 / NT;               // 16 codes each
    static constexpr int kRegs = I8 ? kUnits : 1;
    // keys that one copy, or a wave's 16-byte loads of codes, cover: with pages of at least so many places, and every
    // key of the tile there, they share a base address, and the lanes' offsets stay the same from tile to tile
    static constexpr int kLanes = I8 ? HD / 16 : HD / 8;
    static constexpr int kRun = kWave / kLanes;
    v4u rk[kRegs], rv[kRegs];
    float rks, rvs;
    uint32_t ko[I8 ? 1 : kDma], vo;
    int wave, lane;

    __device__ inline void init(int tid) {
        wave = NT == kWave ? 0 : __builtin_amdgcn_readfirstlane(tid / kWave);
        lane = tid % kWave;
        const int r = lane / kLanes, c = lane % kLanes;
        if constexpr (I8) {
            vo = lane * 16;
        } else {
#pragma unroll
            for (int j = 0; j < kDma; ++j)
                ko[j] = r * HD * 2 + ((c ^ k_swizzle<HD>((wave * kDma + j) * kRun + r)) << 4);
            vo = r * HD * 2 + ((c ^ v_swizzle<HD>(r)) << 4);  // (a run is a multiple of the swizzle's period)
        }
    }

    // pid: the page of key k0 + lane % BK, -1 where there is none; whole: every key is there
    __device__ inline void request(const AttnArgs& A, int head, int k0, int pid, bool whole, uint32_t kbuf, uint32_t vbuf) {
        const int mask = (1 << A.page_shift) - 1;
        const bool runs = whole && mask + 1 >= kRun;
        if constexpr (!I8) {
            if (runs) {
#pragma unroll
                for (int j = 0; j < kDma; ++j) {
                    const int piece = wave * kDma + j, row = piece * kRun;
                    const uint32_t pg = __builtin_amdgcn_readlane(pid, row);
                    const uint64_t at = ((((uint64_t)pg * A.n_kv + head) << A.page_shift) + ((k0 + row) & mask)) * (HD * 2);
                    dma16_at(A.k + at, ko[j], kbuf + piece * 1024);
                    dma16_at(A.v + at, vo, vbuf + piece * 1024);
                }
                return;
            }
#pragma unroll
            for (int j = 0; j < kDma; ++j) {
                const int piece = wave * kDma + j;
                const int row = piece * kRun + lane / kLanes, c = lane % kLanes;
                const int pg = __shfl(pid, row % BK, kWave);
                const size_t at = ((((size_t)(uint32_t)pg * A.n_kv + head) << A.page_shift) + ((k0 + row) & mask)) * (HD * 2);
                const void* pk = A.k + at + ((c ^ k_swizzle<HD>(row)) << 4);
                const void* pv = A.v + at + ((c ^ v_swizzle<HD>(row)) << 4);
                dma16(pg < 0 ? (const void*)kZero16 : pk, kbuf + piece * 1024);
                dma16(pg < 0 ? (const void*)kZero16 : pv, vbuf + piece * 1024);
            }
        } else {
            if (runs) {
#pragma unroll
                for (int j = 0; j < kUnits; ++j) {
                    const int row = (j * (NT / kWave) + wave) * kRun;
                    const uint32_t pg = __builtin_amdgcn_readlane(pid, row);
                    const uint64_t at = ((((uint64_t)pg * A.n_kv + head) << A.page_shift) + ((k0 + row) & mask)) * HD;
                    rk[j] = *reinterpret_cast<const v4u*>(A.k + at + vo);
                    rv[j] = *reinterpret_cast<const v4u*>(A.v + at + vo);
                }
            } else {
#pragma unroll
                for (int j = 0; j < kUnits; ++j) {
                    const int row = (j * (NT / kWave) + wave) * kRun + lane / kLanes, c = lane % kLanes;
                    const int pg = __shfl(pid, row % BK, kWave);
                    const size_t at =
                        ((((size_t)(uint32_t)pg * A.n_kv + head) << A.page_shift) + ((k0 + row) & mask)) * HD + c * 16;
                    const uint8_t* pk = pg < 0 ? (const uint8_t*)kZero16 : A.k + at;
                    const uint8_t* pv = pg < 0 ? (const uint8_t*)kZero16 : A.v + at;
                    rk[j] = *reinterpret_cast<const v4u*>(pk);
                    rv[j] = *reinterpret_cast<const v4u*>(pv);
                }
            }
            rks = rvs = 0.0f;
            if (wave == 0 && lane < BK && pid >= 0) {
                const size_t at = (((size_t)pid * A.n_kv + head) << A.page_shift) + ((k0 + lane) & mask);
                rks = A.ks[at];
                rvs = A.vs[at];
            }
        }
    }
    // what was requested is in LDS (for this wave; a barrier orders the others)
    __device__ inline void land(uint8_t* kbuf, uint8_t* vbuf, float* ksb, float* vsb) {
        if constexpr (!I8) {
            QE_WAIT_VMCNT(0);
            asm volatile("" ::: "memory");
        } else {
#pragma unroll
            for (int j = 0; j < kUnits; ++j) {
                const int row = (j * (NT / kWave) + wave) * kRun + lane / kLanes, c = lane % kLanes;
                v4u w[2];
                codes_to_bf16(rk[j], w);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *reinterpret_cast<v4u*>(kbuf + row * HD * 2 + (((2 * c + e) ^ k_swizzle<HD>(row)) << 4)) = w[e];
                codes_to_bf16(rv[j], w);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *reinterpret_cast<v4u*>(vbuf + row * HD * 2 + (((2 * c + e) ^ v_swizzle<HD>(row)) << 4)) = w[e];
            }
            if (wave == 0 && lane < BK) {
                ksb[lane] = rks;
                vsb[lane] = rvs;
            }
            asm volatile("" ::: "memory");
        }
    }
};

// What a lane's row sees of the 32 keys from k0 on, before the sequence's end is taken into account
struct RowMask {
    int token;             // of the sequence
    const uint32_t* bits;  // its tree row, or NULL
    int words;
    __device__ inline uint32_t word(int w) const { return w < 0 ? ~0u : w >= words ? 0u : bits[w]; }
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

// One tile of NS x 32 keys into a wave's rows
template <int HD, int NS, bool I8, bool kMasked>
__device__ inline void attn_tile(const uint8_t* kbuf, const uint8_t* vbuf, const float* ksb, const float* vsb,
                                 float sc, const uint32_t (&seen)[NS], Rows<HD>& R) {
    const int lane = threadIdx.x % kWave, r = lane % 32, h = lane / 32;
    v16f s[NS];
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
        if constexpr (I8) {
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const v4f f = *reinterpret_cast<const v4f*>(ksb + 32 * b + 8 * a + 4 * h);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[b][4 * a + i] *= f[i];
            }
        }
    }
    if constexpr (kMasked) {
#pragma unroll
        for (int b = 0; b < NS; ++b) {
            const uint32_t w = seen[b] >> (4 * h);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                s[b][i] = (w >> (8 * (i / 4) + i % 4)) & 1u ? s[b][i] : -__builtin_inff();
        }
    }
    float mx = s[0][0];
#pragma unroll
    for (int b = 0; b < NS; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[b][i]);
    mx = half_max(mx) * sc;
    if (__any(mx > R.m + kLazy)) {
        const float m = fmaxf(R.m, mx), f = __builtin_amdgcn_exp2f(R.m - m);
        R.m = m;
        R.l *= f;
#pragma unroll
        for (int d = 0; d < HD / 32; ++d) R.o[d] *= f;
    }
    v8bf p[NS][2];
#pragma unroll
    for (int b = 0; b < NS; ++b) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[b][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][i], sc, -R.m));
        if constexpr (I8) {
#pragma unroll
            for (int i = 0; i < 16; ++i) R.l += s[b][i];
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const v4f f = *reinterpret_cast<const v4f*>(vsb + 32 * b + 8 * a + 4 * h);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[b][4 * a + i] *= f[i];
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            v4u w;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const v2f two = {s[b][8 * e + 2 * i], s[b][8 * e + 2 * i + 1]};
                const v2bf pk = __builtin_convertvector(two, v2bf);
                if constexpr (!I8) {
                    const v2bf one = {(__bf16)1.0f, (__bf16)1.0f};
                    R.l = __builtin_amdgcn_fdot2_f32_bf16(pk, one, R.l, false);
                }
                w[i] = __builtin_bit_cast(uint32_t, pk);
            }
            p[b][e] = __builtin_bit_cast(v8bf, w);
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

__device__ inline int page_of(const AttnArgs& A, const int32_t* pages, int key, int len) {
    if (key >= len) return -1;
    const int p = pages[key >> A.page_shift];
    return (uint32_t)p < (uint32_t)A.n_pages ? p : -1;
}

// 4 channels of a finished row
__device__ inline void store4(uint16_t* p, const float v[4], float f) {
    v2u w;
    w[0] = mx4_bf16_bits(v[0] * f) | (mx4_bf16_bits(v[1] * f) << 16);
    w[1] = mx4_bf16_bits(v[2] * f) | (mx4_bf16_bits(v[3] * f) << 16);
    *reinterpret_cast<v2u*>(p) = w;
}

// Workgroup -> key head (fastest, so that a head's tiles meet in one L2), tile of rows (the last, longest one first),
// sequence, piece
template <int HD, int NW, bool I8>
__global__ __launch_bounds__(NW* kWave, NW == 4 ? 2 : 1) void attn_rows_kernel(AttnArgs A) {
    constexpr int BK = 64, NT = NW * kWave, TILE = BK * HD * 2;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[4 * TILE];
    __shared__ __attribute__((aligned(16))) float scales[I8 ? 4 * BK : 4];
    int id = blockIdx.x;
    const int head = id % A.n_kv;
    id /= A.n_kv;
    const int tile = A.row_tiles - 1 - id % A.row_tiles;
    id /= A.row_tiles;
    const int seq = id % A.n_seq, split = id / A.n_seq;
    const Seq q = seq_of(A, seq);
    const int row0 = tile * (32 * NW), rows = q.n * A.group;
    if (row0 >= rows) return;
    const int last = min(row0 + 32 * NW, rows) - 1;
    const int lo = split * A.chunk;
    if (split > 0 && lo >= q.len) return;  // (no such piece: the join knows the length)
    int hi = A.tree ? q.len : min(q.len, q.ctx + last / A.group + 1);
    if (A.splits > 1) hi = min(hi, lo + A.chunk);

    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid % kWave;
    const int wrow = row0 + 32 * wave, row = wrow + lane % 32;
    Rows<HD> R;
    load_rows<HD>(A, q, head, row, R);
    RowMask mask;
    mask.token = min(row / A.group, q.n - 1);
    mask.bits = A.tree ? A.tree + (size_t)(q.first + mask.token) * A.tree_words : nullptr;
    mask.words = A.tree_words;
    const int all = wrow >= rows ? 0 : q.ctx + (A.tree ? 0 : wrow / A.group + 1);  // keys that every row of the wave sees

    const int32_t* pages = A.pages + (size_t)seq * A.max_pages;
    Stage<HD, BK, NT, I8> st;
    st.init(tid);
    const uint32_t lds0 = lds_addr(smem);
    if (lo < hi) {
        int pid = page_of(A, pages, lo + lane, q.len);
        uint64_t valid = __ballot(pid >= 0);
        st.request(A, head, lo, pid, ~valid == 0, lds0, lds0 + 2 * TILE);
        pid = page_of(A, pages, lo + BK + lane, q.len);
        st.land(smem, smem + 2 * TILE, scales, scales + 2 * BK);
        __syncthreads();
        int buf = 0, k0 = lo;
        bool more;
        uint64_t valid_next;
        const auto begin = [&] {  // the next tile's rows are on their way while this one is computed
            more = k0 + BK < hi;
            valid_next = __ballot(pid >= 0);
            const int nb = buf ^ 1;
            if (more) {
                st.request(A, head, k0 + BK, pid, ~valid_next == 0, lds0 + nb * TILE, lds0 + (2 + nb) * TILE);
                pid = page_of(A, pages, k0 + 2 * BK + lane, q.len);
            }
        };
        const auto end = [&] {
            const int nb = buf ^ 1;
            if (more) st.land(smem + nb * TILE, smem + (2 + nb) * TILE, scales + nb * BK, scales + (2 + nb) * BK);
            valid = valid_next;
            k0 += BK;
            buf = nb;
            __syncthreads();
        };
        // tiles that need no mask first, in a loop of their own (where both forms meet, the compiler copies the running
        // rows); after the first that does, the rest are masked
        while (k0 < hi && k0 + BK <= all && ~valid == 0) {
            begin();
            const uint32_t seen[2] = {~0u, ~0u};
            attn_tile<HD, 2, I8, false>(smem + buf * TILE, smem + (2 + buf) * TILE, scales + buf * BK,
                                        scales + (2 + buf) * BK, A.sc, seen, R);
            end();
        }
        while (k0 < hi) {
            begin();
            // (a piece ends at a multiple of the tile, or where the sequence or the tile's last row ends)
            const uint32_t seen[2] = {(uint32_t)valid & mask.of(k0 - q.ctx),
                                      (uint32_t)(valid >> 32) & mask.of(k0 + 32 - q.ctx)};
            attn_tile<HD, 2, I8, true>(smem + buf * TILE, smem + (2 + buf) * TILE, scales + buf * BK,
                                       scales + (2 + buf) * BK, A.sc, seen, R);
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

// At most 32 rows: waves take tiles of 32 keys in turn
template <int HD, bool I8>
__global__ __launch_bounds__(256) void attn_keys_kernel(AttnArgs A) {
    constexpr int BK = 32, NW = 4, TILE = BK * HD * 2, OLD = HD + 4;
    static_assert(32 * OLD * 4 <= 4 * TILE + 1024, "");
    constexpr int REGION = 4 * TILE > 32 * OLD * 4 ? 4 * TILE : (32 * OLD * 4 + 1023) / 1024 * 1024;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[NW * REGION];
    __shared__ __attribute__((aligned(16))) float scales_all[I8 ? NW * 4 * BK : 4];
    __shared__ float2 ml[NW][32];
    int id = blockIdx.x;
    const int head = id % A.n_kv;
    id /= A.n_kv;
    const int seq = id % A.n_seq, split = id / A.n_seq;
    const Seq q = seq_of(A, seq);
    const int rows = q.n * A.group;
    const int lo = split * A.chunk;
    if (rows == 0 || (split > 0 && lo >= q.len)) return;
    const int hi = A.splits > 1 ? min(q.len, lo + A.chunk) : q.len;

    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid % kWave;
    const int row = lane % 32;
    Rows<HD> R;
    load_rows<HD>(A, q, head, row, R);
    RowMask mask;
    mask.token = min(row / A.group, q.n - 1);
    mask.bits = A.tree ? A.tree + (size_t)(q.first + mask.token) * A.tree_words : nullptr;
    mask.words = A.tree_words;
    const int all = q.ctx + (A.tree ? 0 : 1);

    const int32_t* pages = A.pages + (size_t)seq * A.max_pages;
    Stage<HD, BK, kWave, I8> st;
    st.init(lane);
    uint8_t* mine = smem + wave * REGION;
    float* scales = scales_all + (I8 ? wave * 4 * BK : 0);
    const uint32_t lds0 = lds_addr(mine);
    int k0 = lo + wave * BK;
    if (k0 < hi) {
        int pid = page_of(A, pages, k0 + row, q.len);
        uint32_t valid = (uint32_t)__ballot(pid >= 0);
        st.request(A, head, k0, pid, ~valid == 0, lds0, lds0 + 2 * TILE);
        pid = page_of(A, pages, k0 + NW * BK + row, q.len);
        st.land(mine, mine + 2 * TILE, scales, scales + 2 * BK);
        int buf = 0;
        bool more;
        uint32_t valid_next;
        const auto begin = [&] {
            more = k0 + NW * BK < hi;
            valid_next = (uint32_t)__ballot(pid >= 0);
            const int nb = buf ^ 1;
            if (more) {
                st.request(A, head, k0 + NW * BK, pid, ~valid_next == 0, lds0 + nb * TILE, lds0 + (2 + nb) * TILE);
                pid = page_of(A, pages, k0 + 2 * NW * BK + row, q.len);
            }
        };
        const auto end = [&] {
            const int nb = buf ^ 1;
            if (more) st.land(mine + nb * TILE, mine + (2 + nb) * TILE, scales + nb * BK, scales + (2 + nb) * BK);
            valid = valid_next;
            k0 += NW * BK;
            buf = nb;
        };
        while (k0 < hi && k0 + BK <= all && ~valid == 0) {
            begin();
            const uint32_t seen[1] = {~0u};
            attn_tile<HD, 1, I8, false>(mine + buf * TILE, mine + (2 + buf) * TILE, scales + buf * BK,
                                        scales + (2 + buf) * BK, A.sc, seen, R);
            end();
        }
        while (k0 < hi) {
            begin();
            const uint32_t seen[1] = {valid & mask.of(k0 - q.ctx)};
            attn_tile<HD, 1, I8, true>(mine + buf * TILE, mine + (2 + buf) * TILE, scales + buf * BK,
                                       scales + (2 + buf) * BK, A.sc, seen, R);
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

// The pieces of one token and query head, in order: a wave each
template <int HD>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs A) {
    const long id = (long)blockIdx.x * 4 + threadIdx.x / kWave;
    const int lane = threadIdx.x % kWave;
    const long token = id / A.n_heads;
    const int hq = (int)(id - token * A.n_heads);
    if (token >= A.T) return;
    int a = 0, b = A.n_seq;  // the last sequence that starts at or before the token
    while (b - a > 1) {
        const int mid = (a + b) / 2;
        if (A.q_start[mid] <= token) a = mid;
        else b = mid;
    }
    const Seq q = seq_of(A, a);
    if (token < q.first || token >= q.first + q.n) return;
    const int n = min(A.splits, (q.len + A.chunk - 1) / A.chunk);
    constexpr int V = HD / kWave;
    float M = kLowest, L = 0.0f, v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.0f;
    for (int s = 0; s < n; ++s) M = fmaxf(M, A.part_ml[((size_t)s * A.T + token) * A.n_heads + hq].x);
    for (int s = 0; s < n; ++s) {
        const size_t at = ((size_t)s * A.T + token) * A.n_heads + hq;
        const float2 p = A.part_ml[at];
        const float w = __builtin_amdgcn_exp2f(p.x - M);
        L += w * p.y;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += w * A.part_o[at * HD + V * lane + i];
    }
    const float f = L > 0.0f ? 1.0f / L : 0.0f;
    uint16_t* p = A.out + (size_t)token * A.out_stride + (size_t)hq * HD + V * lane;
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = (uint16_t)mx4_bf16_bits(v[i] * f);
}

template <int HD, bool I8>
void launch_hd(const AttnArgs& A, const AttnPlan& P, hipStream_t st) {
    const unsigned grid = (unsigned)((size_t)A.n_kv * P.row_tiles * A.n_seq * P.splits);
    if (P.few_rows) hipLaunchKernelGGL((attn_keys_kernel<HD, I8>), dim3(grid), dim3(256), 0, st, A);
    else hipLaunchKernelGGL((attn_rows_kernel<HD, 4, I8>), dim3(grid), dim3(256), 0, st, A);
    if (P.splits > 1)
        hipLaunchKernelGGL(attn_join_kernel<HD>, dim3((unsigned)(((size_t)A.T * A.n_heads + 3) / 4)), dim3(256), 0, st, A);
}

}  // namespace

AttnPlan attn_plan(const qe_kv_cache* cache, int n_heads, int n_seq, int max_q, int max_kv) {
    AttnPlan P;
    const long rows = (long)max_q * (n_heads / cache->n_kv_heads);
    P.few_rows = rows <= 32;
    P.row_tiles = P.few_rows ? 1 : (int)((rows + 127) / 128);
    const long base = (long)n_seq * cache->n_kv_heads * P.row_tiles;
    const long want = 1024, least = 256;
    const long pieces = std::max(1L, std::min((want + base - 1) / base, (max_kv + least - 1) / least));
    P.chunk = (int)(((max_kv + pieces - 1) / pieces + 127) / 128 * 128);
    P.chunk = std::max(P.chunk, 128);
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
    if (c->head_dim == 128) {
        if (i8) launch_hd<128, true>(A, P, st);
        else launch_hd<128, false>(A, P, st);
    } else {
        if (i8) launch_hd<64, true>(A, P, st);
        else launch_hd<64, false>(A, P, st);
    }
    return hipGetLastError();
}

}  // namespace qe
