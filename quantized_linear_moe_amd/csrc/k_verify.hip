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
#include <algorithm>

#include "qe_cache.h"

namespace qe {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;                  // entries of a thread
constexpr int kPiece = kThreads * kPer;   // entries of a piece

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

// Bits of the piece's tokens that were rejected at the last row (tree: every child of it)
__device__ inline void drop_bits(const VerifyArgs& A, const SeqRows& r, int cur, int base, uint32_t* bits) {
    for (int i = threadIdx.x; i < kPiece / 32; i += kThreads) bits[i] = 0;
    __syncthreads();
    if (!A.d)
        for (int i = cur + 1 + threadIdx.x; i < r.n; i += kThreads) {
            const int above = A.parent ? A.parent[r.first + i] : i - 1;
            const int at = A.token[r.first + i] - base;
            if (above == cur && at >= 0 && at < kPiece) atomicOr(&bits[at >> 5], 1u << (at & 31));
        }
    __syncthreads();
}

__device__ inline double block_sum(double v, double* red) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
    if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = v;
    __syncthreads();
    const double s = ((red[0] + red[1]) + red[2]) + red[3];
    __syncthreads();
    return s;
}

__global__ __launch_bounds__(kThreads) void verify_walk_kernel(VerifyArgs A) {
    __shared__ int par[kVerifyMaxRows], tok[kVerifyMaxRows];
    __shared__ float uu[kVerifyMaxRows], pt[kVerifyMaxRows];
    __shared__ uint32_t bits[kPiece / 32];
    __shared__ double red[kThreads / kWave];
    __shared__ int s_cur;
    const int seq = blockIdx.x / A.pieces, piece = blockIdx.x % A.pieces, tid = threadIdx.x;
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
    if (!A.d && A.parent) {
        bool again[kVerifyMaxRows / kThreads];
#pragma unroll
        for (int k = 0; k < kVerifyMaxRows / kThreads; ++k) {
            const int i = tid + k * kThreads;
            again[k] = false;
            for (int j = 1; j < i && i < r.n; ++j) again[k] = again[k] || (par[j] == par[i] && tok[j] == tok[i]);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kVerifyMaxRows / kThreads; ++k)
            if (again[k]) pt[tid + k * kThreads] = -1.0f;
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
                    const double pc = (double)__shfl(my_p, l, kWave), uc = (double)__shfl(my_u, l, kWave);
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
    drop_bits(A, r, cur, base, bits);
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

__global__ __launch_bounds__(kThreads) void verify_draw_kernel(VerifyArgs A) {
    __shared__ double R[kPiece + kThreads];  // a thread's 16 entries at 17 k: no two lanes of a group in one bank
    __shared__ double head[kThreads / kWave];
    __shared__ uint32_t bits[kPiece / 32];
    __shared__ double s_before, s_goal;
    __shared__ int s_piece, s_found, s_positive;
    const int seq = blockIdx.x, tid = threadIdx.x;
    const SeqRows r = rows_of(A, seq);
    if (r.n <= 0) return;
    const int cur = A.last[seq];
    const double* sums = A.sums + (size_t)seq * A.pieces * 2;
    if (tid == 0) {
        // nothing left to draw from (all of p's mass was rejected, up to its rounding): from p itself
        double z = 0.0;
        for (int i = 0; i < A.pieces; ++i) z += sums[2 * i];
        int which = 0;
        if (!(z > 0.0)) {
            which = 1;
            z = 0.0;
            for (int i = 0; i < A.pieces; ++i) z += sums[2 * i + 1];
        }
        const double goal = (double)A.u[r.first] * z;
        double before = 0.0;
        int at = -1, some = -1;
        double some_before = 0.0;
        for (int i = 0; i < A.pieces && z > 0.0; ++i) {
            const double s = sums[2 * i + which];
            if (s > 0.0) {
                some = i;
                some_before = before;
            }
            if (before + s > goal) {
                at = i;
                break;
            }
            before += s;
        }
        s_piece = z > 0.0 ? 2 * (at >= 0 ? at : some) + which : -1;
        s_before = at >= 0 ? before : some_before;
        s_goal = goal;
        s_found = kPiece;
        s_positive = -1;
    }
    __syncthreads();
    if (s_piece < 0) {  // no distribution
        if (tid == 0) A.next[seq] = -1;
        return;
    }
    const int base = (s_piece >> 1) * kPiece;
    const bool plain = s_piece & 1;
    drop_bits(A, r, cur, base, bits);
    const float* p = A.p + (size_t)(r.first + cur) * A.p_stride;
    const float* d = A.d && !plain && cur + 1 < r.n ? A.d + (size_t)(r.first + cur + 1) * A.d_stride : nullptr;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int at = k * kThreads + tid;
        double v = 0.0;
        if (base + at < A.vocab && (plain || !(bits[at >> 5] >> (at & 31) & 1u))) v = residual(p, d, base + at);
        R[at + at / kPer] = v;
    }
    __syncthreads();
    double mine = 0.0;
    for (int k = 0; k < kPer; ++k) mine += R[tid * (kPer + 1) + k];
    double before = mine;  // sums of the threads up to this one: within the wave, then the waves before it
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const double o = __shfl_up(before, off, kWave);
        if (tid % kWave >= off) before += o;
    }
    if (tid % kWave == kWave - 1) head[tid / kWave] = before;
    __syncthreads();
    double c = s_before;
    for (int i = 0; i < tid / kWave; ++i) c += head[i];
    c += before - mine;
    for (int k = 0; k < kPer; ++k) {
        const double v = R[tid * (kPer + 1) + k];
        c += v;
        if (v > 0.0) {
            atomicMax(&s_positive, tid * kPer + k);
            if (c > s_goal) {
                atomicMin(&s_found, tid * kPer + k);
                break;
            }
        }
    }
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
