// Verification of drafted tokens against the target's probabilities, from given random numbers.
//
//   chain (with the drafts' distributions): row i is taken while u_i q_i(x_i) < p_{i-1}(x_i); after the first row that is
//     not, the next token is drawn from max(p - q, 0), after the last from p
//   tree: at a node, its children in row order; c is taken if u_c rest < p(x_c), rest = 1 - the rejected siblings'
//     probabilities (a token that was already rejected there has none left); with no child taken, the next token is drawn
//     from p without the rejected tokens
//   draw: the smallest j with R_0 + .. + R_j > u_0 sum R
//
// Comparisons and sums in 64 bits: the probabilities are float32, and a sum over a vocabulary in 32 bits would move the
// drawn token.  Only one row of p (and of the drafts') per sequence is read whole, the one where the walk ends; so the
// first kernel's workgroups (one per sequence and piece of the vocabulary) each walk for themselves, from the rows'
// gathered probabilities in LDS, then sum their piece; the second kernel finds the piece and the token in it.
//
// Bound by trips to memory that wait for each other, four in the walk (starts; rows' tokens and random numbers; their
// probabilities; the last row) and three in the draw (sums and starts; random number and tokens; the piece), the float64
// scans with their barriers between, and two launches: a chain of 5 rows over 32000 entries 7.4 + 8.1 us, 32 trees of 33 rows
// over 131072 11.8 + 9.0 (17 MB of rows, 3 us at the copy rate).  One kernel with a workgroup per sequence saves the second
// launch but reads a row on one CU: 11 us in place of 14 at 8000 entries, the same at 32000, 38 in place of 17 at 131072.
// Trees of many rows are bound by the look for a token that a sibling has too, every pair of rows in every workgroup: 64
// rows 8.3 us, 1024 rows 470 (32000 or 131072 entries).
#include <algorithm>

#include "qe_cache.h"

namespace qe {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;                  // entries of a thread
constexpr int kPiece = kThreads * kPer;   // entries of a piece
constexpr int kMaxPieces = kVerifyMaxVocab / kPiece;

struct VerifyArgs {
    const float *p, *d;
    int64_t p_stride, d_stride;
    int vocab, n_rows, n_seq, max_rows, pieces;
    const int32_t *row_start, *token, *parent;
    const float* u;
    int32_t *taken, *path, *next;
    double* sums;   // [n_seq][pieces][2]: of what is drawn from, and of p
    int32_t* last;  // [n_seq]: the row (of the sequence) where the walk ended
};

struct SeqRows {
    int first, n;
};
__device__ inline SeqRows rows_of(const VerifyArgs& A, int s) {
    SeqRows r;
    r.first = min(max(A.row_start[s], 0), A.n_rows);
    r.n = min(min(max(A.row_start[s + 1], r.first), A.n_rows) - r.first, A.max_rows);
    return r;
}

// What the next token is drawn from: entry j of the last row's distribution
__device__ inline double residual(const float* p, const float* d, int j) {
    const double v = (double)p[j];
    return d ? fmax(v - (double)d[j], 0.0) : v;
}

// Bits of the piece's tokens that were refused at the last row: every child of it
__device__ inline void drop_bit(int above, int cur, int token, int base, uint32_t* bits) {
    const int at = token - base;
    if (above == cur && at >= 0 && at < kPiece) atomicOr(&bits[at >> 5], 1u << (at & 31));
}

// A double from the lane that a data-parallel move names (0 where there is none, and in the rows left out)
template <int kCtrl, int kRows>
__device__ inline double moved(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, kCtrl, kRows, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), kCtrl, kRows, 0xF, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Sums over the wave's lanes up to and with this one: within rows of 16, then the rows before (lane moves: through LDS, each
// of the six steps is a trip there, and the draw took 9.9 us in place of 9.1)
__device__ inline double wave_scan(double v) {
    v += moved<0x111, 0xF>(v);  // from 1, 2, 4, 8 lanes below
    v += moved<0x112, 0xF>(v);
    v += moved<0x114, 0xF>(v);
    v += moved<0x118, 0xF>(v);
    v += moved<0x142, 0xA>(v);  // lane 15 of rows 0 and 2 to the row above
    v += moved<0x143, 0xC>(v);  // lane 31 to the upper half
    return v;
}

// Sums over the threads up to and with this one (*all: over all of them), in a fixed order
__device__ inline double block_scan(double mine, double* red, double* all) {
    const double v = wave_scan(mine);
    if (threadIdx.x % kWave == kWave - 1) red[threadIdx.x / kWave] = v;
    __syncthreads();
    double before = 0.0, sum = 0.0;
#pragma unroll
    for (int i = 0; i < kThreads / kWave; ++i) {
        if (i == threadIdx.x / kWave) before = sum;
        sum += red[i];
    }
    __syncthreads();
    *all = sum;
    return before + v;
}

__device__ inline double block_sum(double v, double* red) {
    double all;
    block_scan(v, red, &all);
    return all;
}

__global__ __launch_bounds__(kThreads) void verify_walk_kernel(VerifyArgs A) {
    __shared__ int par[kVerifyMaxRows], tok[kVerifyMaxRows];
    __shared__ float uu[kVerifyMaxRows], pt[kVerifyMaxRows];
    __shared__ uint32_t bits[kPiece / 32];
    __shared__ double red[kThreads / kWave];
    __shared__ int s_cur;
    const int seq = blockIdx.x / A.pieces, piece = blockIdx.x % A.pieces, tid = threadIdx.x;
    for (int i = tid; i < kPiece / 32; i += kThreads) bits[i] = 0;
    const SeqRows r = rows_of(A, seq);
    if (r.n <= 0) {
        if (piece == 0 && tid == 0) {
            A.taken[seq] = 0;
            A.next[seq] = -1;
        }
        return;
    }
    for (int i = tid; i < r.n; i += kThreads) {
        const int x = A.token[r.first + i];
        int above = A.parent ? A.parent[r.first + i] : i - 1;
        if (above >= i || i == 0) above = -1;
        par[i] = above;
        tok[i] = x;
        uu[i] = A.u[r.first + i];
        pt[i] = -1.0f;  // a token outside the vocabulary is never taken
        if (above >= 0 && x >= 0 && x < A.vocab) {
            pt[i] = A.p[(size_t)(r.first + above) * A.p_stride + x];
            if (A.d && !((double)uu[i] * (double)A.d[(size_t)(r.first + i) * A.d_stride + x] < (double)pt[i])) pt[i] = -1.0f;
        }
    }
    __syncthreads();
    if (!A.d && A.parent) {  // a token that a sibling before it has: refused with it
        for (int at = tid; at < r.n * r.n; at += kThreads) {
            const int i = at / r.n, j = at - i * r.n;
            if (j > 0 && j < i && par[j] == par[i] && tok[j] == tok[i]) pt[i] = -1.0f;
        }
        __syncthreads();
    }
    int steps = 0;
    if (tid < kWave) {
        int cur = 0;
        bool on = r.n > 1;
        while (on) {
            on = false;
            double rest = 1.0;
            for (int b = (cur + 1) & ~(kWave - 1); b < r.n && !on; b += kWave) {
                const int i = b + tid;
                const bool child = i < r.n && i > cur && par[i] == cur;
                const float my_p = child ? pt[i] : 0.0f, my_u = child ? uu[i] : 0.0f;
                for (uint64_t m = __ballot(child); m; m &= m - 1) {
                    const int l = __ffsll((unsigned long long)m) - 1;
                    const double pc = (double)__int_as_float(__builtin_amdgcn_readlane(__float_as_int(my_p), l));
                    const double uc = (double)__int_as_float(__builtin_amdgcn_readlane(__float_as_int(my_u), l));
                    const bool take = A.d ? pc >= 0.0 : uc * rest < pc;
                    if (take) {
                        cur = b + l;
                        if (piece == 0 && tid == 0) A.path[r.first + steps] = cur;
                        ++steps;
                        on = true;
                        break;
                    }
                    if (pc > 0.0) rest -= pc;
                }
            }
        }
        if (tid == 0) s_cur = cur;
        if (piece == 0) {
            for (int i = steps + tid; i < r.n; i += kWave) A.path[r.first + i] = -1;
            if (tid == 0) {
                A.taken[seq] = steps;
                A.last[seq] = cur;
            }
        }
    }
    __syncthreads();
    const int cur = s_cur, base = piece * kPiece;
    if (!A.d) {
        for (int i = cur + 1 + tid; i < r.n; i += kThreads) drop_bit(par[i], cur, tok[i], base, bits);
        __syncthreads();
    }
    const float* p = A.p + (size_t)(r.first + cur) * A.p_stride;
    const float* d = A.d && cur + 1 < r.n ? A.d + (size_t)(r.first + cur + 1) * A.d_stride : nullptr;
    double sum = 0.0, all = 0.0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int at = k * kThreads + tid;
        if (base + at >= A.vocab) continue;
        all += (double)p[base + at];
        if (!(bits[at >> 5] >> (at & 31) & 1u)) sum += residual(p, d, base + at);
    }
    sum = block_sum(sum, red);
    all = block_sum(all, red);
    if (tid == 0) {
        double* o = A.sums + ((size_t)seq * A.pieces + piece) * 2;
        o[0] = sum;
        o[1] = all;
    }
}

// The pieces of a thread, at most kMaxPieces / kThreads consecutive ones: the sum of all, and, given a goal, the first
// piece whose end lies past it (into *at and *before)
constexpr int kPieces = kMaxPieces / kThreads;
__device__ inline double scan_pieces(const double (&s)[kPieces], double* red, double (&before)[kPieces]) {
    double mine = 0.0, all;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) mine += s[k];
    double c = block_scan(mine, red, &all) - mine;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        before[k] = c;
        c += s[k];
    }
    return all;
}

// The least `first` below `none` and the greatest `last` above -1 over the threads, both growing with the thread (one LDS
// atomic per wave: 4096 on one address took 30 us)
__device__ inline void first_and_last(int first, int none, int last, int* at_first, int* at_last) {
    const uint64_t f = __ballot(first < none), l = __ballot(last >= 0);
    const int lo = f ? __builtin_amdgcn_readlane(first, __builtin_ctzll(f)) : none;
    const int hi = l ? __builtin_amdgcn_readlane(last, 63 - __builtin_clzll(l)) : -1;
    if (threadIdx.x % kWave == 0) {
        if (f) atomicMin(at_first, lo);
        if (l) atomicMax(at_last, hi);
    }
}

__global__ __launch_bounds__(kThreads) void verify_draw_kernel(VerifyArgs A) {
    __shared__ double R[kPiece + kThreads];  // a thread's 16 entries at 17 k: no two lanes of a group in one bank
    __shared__ double red[kThreads / kWave];
    __shared__ uint32_t bits[kPiece / 32];
    __shared__ double s_before;
    __shared__ int s_piece, s_some, s_found, s_positive;
    const int seq = blockIdx.x, tid = threadIdx.x;
    // (what does not depend on the rows is requested with them: each wait is a trip to memory)
    const double* sums = A.sums + (size_t)seq * A.pieces * 2;
    const int per = (A.pieces + kThreads - 1) / kThreads;
    double s[kPieces], s_p[kPieces], before[kPieces];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        const int i = tid * per + k;
        const bool in = k < per && i < A.pieces;
        s[k] = in ? sums[2 * i] : 0.0;
        s_p[k] = in ? sums[2 * i + 1] : 0.0;
    }
    const int cur = A.last[seq];
    const SeqRows r = rows_of(A, seq);
    if (r.n <= 0) return;
    const double u = (double)A.u[r.first];
    int my_above = -1, my_token = -1;  // of row tid
    if (!A.d && tid < r.n) {
        my_above = A.parent ? A.parent[r.first + tid] : tid - 1;
        my_token = A.token[r.first + tid];
    }
    for (int i = tid; i < kPiece / 32; i += kThreads) bits[i] = 0;
    if (tid == 0) {
        s_piece = A.pieces;
        s_some = -1;
        s_found = kPiece;
        s_positive = -1;
    }
    double z = scan_pieces(s, red, before);
    const bool plain = !(z > 0.0);  // nothing left to draw from (all of p was refused, up to its rounding): p itself
    if (plain) {
#pragma unroll
        for (int k = 0; k < kPieces; ++k) s[k] = s_p[k];
        z = scan_pieces(s, red, before);
    }
    if (!(z > 0.0)) {  // no distribution
        if (tid == 0) A.next[seq] = -1;
        return;
    }
    const double goal = u * z;
    int past = A.pieces, some = -1;
#pragma unroll
    for (int k = 0; k < kPieces; ++k)
        if (s[k] > 0.0) {
            some = tid * per + k;
            if (before[k] + s[k] > goal) past = min(past, some);
        }
    first_and_last(past, A.pieces, some, &s_piece, &s_some);
    __syncthreads();
    const int piece = s_piece < A.pieces ? s_piece : s_some;  // (no piece reaches the goal: the last with any weight)
#pragma unroll
    for (int k = 0; k < kPieces; ++k)
        if (k < per && tid * per + k == piece) s_before = before[k];
    const int base = piece * kPiece;
    if (!A.d && !plain) {
        if (tid > cur) drop_bit(my_above, cur, my_token, base, bits);
        for (int i = tid + kThreads; i < r.n; i += kThreads)
            if (i > cur) drop_bit(A.parent ? A.parent[r.first + i] : i - 1, cur, A.token[r.first + i], base, bits);
    }
    __syncthreads();
    const float* p = A.p + (size_t)(r.first + cur) * A.p_stride;
    const float* d = A.d && !plain && cur + 1 < r.n ? A.d + (size_t)(r.first + cur + 1) * A.d_stride : nullptr;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int at = k * kThreads + tid;
        double v = 0.0;
        if (base + at < A.vocab && !(bits[at >> 5] >> (at & 31) & 1u)) v = residual(p, d, base + at);
        R[at + at / kPer] = v;
    }
    __syncthreads();
    double mine = 0.0, all;
#pragma unroll
    for (int k = 0; k < kPer; ++k) mine += R[tid * (kPer + 1) + k];
    double c = s_before + (block_scan(mine, red, &all) - mine);
    int found = kPiece, positive = -1;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const double v = R[tid * (kPer + 1) + k];
        c += v;
        if (v > 0.0) {
            positive = tid * kPer + k;
            if (c > goal) found = min(found, positive);
        }
    }
    first_and_last(found, kPiece, positive, &s_found, &s_positive);
    __syncthreads();
    // (a piece whose entries sum to a little less here than in the other order: its last entry)
    if (tid == 0) A.next[seq] = base + (s_found < kPiece ? s_found : max(s_positive, 0));
}

}  // namespace

int verify_chunks(int vocab) { return (vocab + kPiece - 1) / kPiece; }

hipError_t launch_verify(const float* p, int64_t p_stride, const float* draft_p, int64_t draft_stride, int vocab,
                         const int32_t* row_start, int n_rows, const int32_t* token, const int32_t* parent,
                         const float* u, int n_seq, int max_rows, int32_t* taken, int32_t* path, int32_t* next, void* ws,
                         hipStream_t st) {
    VerifyArgs A = {};
    A.p = p;
    A.d = draft_p;
    A.p_stride = p_stride;
    A.d_stride = draft_stride;
    A.vocab = vocab;
    A.n_rows = n_rows;
    A.n_seq = n_seq;
    A.max_rows = max_rows;
    A.pieces = verify_chunks(vocab);
    A.row_start = row_start;
    A.token = token;
    A.parent = parent;
    A.u = u;
    A.taken = taken;
    A.path = path;
    A.next = next;
    A.sums = reinterpret_cast<double*>(ws);
    A.last = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(ws) + align256((size_t)n_seq * A.pieces * 16));
    hipLaunchKernelGGL(verify_walk_kernel, dim3((unsigned)((size_t)A.pieces * n_seq)), dim3(kThreads), 0, st, A);
    hipLaunchKernelGGL(verify_draw_kernel, dim3((unsigned)n_seq), dim3(kThreads), 0, st, A);
    return hipGetLastError();
}

}  // namespace qe
