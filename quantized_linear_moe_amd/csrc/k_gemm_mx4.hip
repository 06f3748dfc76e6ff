// Product of two microscaled 4-bit operands on the scaled matrix instruction of gfx950, with both
// low-rank corrections of a QE linear in the same accumulators.
//
//   y[t][i] = sum_j a[t][j] w[i][j] + u[t] . B_s[:, i] + v[t] . B_{e_t}[:, i]
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 32 rows by 32 columns over 64 channels: a lane's 32
// codes (16 bytes) are one scale block, whose scale byte it supplies beside them, so the scaling
// costs no separate work.  The codes enter the matrix core as stored: no unpacking.  Products are
// exact and sums float32.  The adapter terms are bf16 32x32x16 steps on the same accumulators
// (same lane layout), so they need no pass over y.
//
// Two kernels: tiles through LDS for prompts (bound by the matrix cores when large), and weight
// streaming for up to 64 tokens (bound by the reads of the weights).

#include <algorithm>

#include "qe_dma.h"
#include "qe_internal.h"
#include "qe_mx4.h"

namespace qe {

namespace {

// an MFMA operand of 4-bit codes: the instruction reads the first 4 of the builtin's 8 registers
__device__ inline v8i mx_operand(v4i c) { return v8i{c[0], c[1], c[2], c[3], 0, 0, 0, 0}; }

// H: half of a 128-wide K step; its two blocks' scales are bytes 2H + lane/32 of the K step's dword,
// moved to byte 2H by a shift of 8 * (lane / 32)
template <int H>
__device__ inline v16f mx_mfma(v4i a, uint32_t sa, v4i b, uint32_t sb, v16f c) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(a), mx_operand(b), c, 4, 4, 2 * H, (int)sa,
                                                           2 * H, (int)sb);
}

// row of accumulator register i in its 32-row block (the column is lane % 32)
__device__ inline int acc_row(int i, int lane) { return 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3); }

__device__ inline void store_out(float* y, size_t idx, float v, bool y_bf16) {
    if (y_bf16) reinterpret_cast<uint16_t*>(y)[idx] = (uint16_t)mx4_bf16_bits(v);
    else y[idx] = v;
}

constexpr int TS_NS = 4;  // K steps in the LDS ring of the tile kernel

}  // namespace

// ------------------------------------------------------------------ tiles
// BM tokens x BN channels per workgroup of 4 waves (2 x 2), 128 channels of K per step.  Code rows and
// weight tiles go global -> LDS by DMA through a ring of TS_NS steps, TS_NS - 1 ahead.  Each wave
// holds BM/64 x BN/64 blocks of 32 x 32.  The fragments of the next half step are requested before the MFMAs
// of the current one, and the barrier that frees a ring slot stands between the two halves of a step,
// with the second half's fragments already in registers: the matrix cores meet it with work queued.
// Code rows of a step are 64 bytes, four 16-byte chunks stored at chunk ^ ((row >> 1) & 3) so that 8
// consecutive rows reach all banks.
template <int BM, int BN>
__global__ __launch_bounds__(256, 1) void gemm_mx4_kernel(Mx4Gemm G, int n_tm, int ksplit) {
    constexpr int MB = BM / 64, NB = BN / 64;              // 32x32 blocks per wave
    constexpr int A_ST = BM * 64, B_ST = BN * 64;          // codes per step
    constexpr int STAGE = A_ST + B_ST + BM * 4 + BN * 4;   // + scales
    constexpr int AD = BM / 64, BD = BN / 64;              // 1 KB copies per wave
    constexpr int SQ = BM / 64 + BN / 64, SD = (SQ + 3) / 4;  // 256-byte scale copies: in all, per wave
    constexpr int OPS = AD + BD + SD;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[TS_NS * STAGE];
    __shared__ int s_tok[BM];
    __shared__ int s_ex[BM];

    // tile order: see gemm_w4_tile (each XCD walks a contiguous range of groups of 8 token tiles)
    int tm, tn;
    {
        const int total = gridDim.x, n_tn = total / n_tm;
        int L = blockIdx.x;
        if ((total & 7) == 0) L = (L & 7) * (total >> 3) + (L >> 3);
        constexpr int GM = 8;
        const int per_group = GM * n_tn;
        const int g = L / per_group, first = g * GM, gs = min(n_tm - first, GM), r = L - g * per_group;
        tm = first + r % gs;
        tn = r / gs;
    }
    const int m0 = tm * BM, n0 = tn * BN;
    const int tid = threadIdx.x, wid = tid >> 6, lane = tid & 63, lr = lane & 31, lh = lane >> 5;
    const int wm = wid & 1, wn = wid >> 1;
    const int T = G.T, KB = G.d_in / 128, NBT = (G.d_out + 31) / 32;
    const int ky = blockIdx.y;
    const int kb0 = (int)((long)ky * KB / ksplit), nk = (int)((long)(ky + 1) * KB / ksplit) - kb0;

    const bool routed = G.v != nullptr;
    for (int r = tid; r < BM; r += 256) {
        const int pos = min(m0 + r, T - 1);
        const int tk = G.perm ? G.perm[pos] : pos;
        s_tok[r] = tk;
        s_ex[r] = (routed && m0 + r < T) ? min(max(G.expert[tk], 0), G.n_r - 1) : -1;
    }
    __syncthreads();

    const uint32_t lds0 = lds_addr(smem);
    // copy sources; A copy q covers rows 16q..16q+15: lane i fetches the chunk stored at slot i%4
    const uint8_t* a_src[AD];
#pragma unroll
    for (int p = 0; p < AD; ++p) {
        const int r = 16 * (wid + 4 * p) + (lane >> 2), c = (lane & 3) ^ ((r >> 1) & 3);
        a_src[p] = G.codes + (size_t)s_tok[r] * (G.d_in / 2) + (size_t)kb0 * 64 + c * 16;
    }
    const uint8_t* b_src[BD];  // B copy q: half step q & 1 of channel block q >> 1
#pragma unroll
    for (int p = 0; p < BD; ++p) {
        const int q = wid + 4 * p, nb = min(n0 / 32 + (q >> 1), NBT - 1);
        b_src[p] = G.w_tiled + (((size_t)nb * KB + kb0) * 2 + (q & 1)) * 1024 + lane * 16;
    }
    const uint8_t* s_src[SD];  // scale copies: 64 rows of A each, then 64 channels of B each
    int s_dst[SD], s_step[SD];
#pragma unroll
    for (int p = 0; p < SD; ++p) {
        const int q = (wid + 4 * p) % SQ;  // fewer copies than waves: repeated, the same bytes
        if (q < BM / 64) {
            s_src[p] = G.scales + (size_t)s_tok[q * 64 + lane] * (G.d_in / 32) + (size_t)kb0 * 4;
            s_step[p] = 4;
        } else {
            const int nb = min(n0 / 32 + (q - BM / 64) * 2 + lh, NBT - 1);
            s_src[p] = reinterpret_cast<const uint8_t*>(G.w_scale + ((size_t)nb * KB + kb0) * 32 + lr);
            s_step[p] = 128;
        }
        s_dst[p] = A_ST + B_ST + q * 256;
    }
    auto issue = [&](int slot, int i) {
        const uint32_t base = lds0 + slot * STAGE;
#pragma unroll
        for (int p = 0; p < AD; ++p) dma16(a_src[p] + (size_t)i * 64, base + (wid + 4 * p) * 1024);
#pragma unroll
        for (int p = 0; p < BD; ++p) dma16(b_src[p] + (size_t)i * 2048, base + A_ST + (wid + 4 * p) * 1024);
#pragma unroll
        for (int p = 0; p < SD; ++p) dma4(s_src[p] + (size_t)i * s_step[p], base + s_dst[p]);
    };
    struct Frag {
        v4i a[MB], b[NB];
    };
    struct Scale {
        uint32_t a[MB], b[NB];
    };
    auto read = [&](Frag& f, int slot, int h) {
        const uint8_t* st = smem + slot * STAGE;
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            const int row = (wm * MB + m) * 32 + lr;
            f.a[m] = *reinterpret_cast<const v4i*>(st + row * 64 + (((h * 2 + lh) ^ ((row >> 1) & 3)) << 4));
        }
#pragma unroll
        for (int n = 0; n < NB; ++n)
            f.b[n] = *reinterpret_cast<const v4i*>(st + A_ST + ((wn * NB + n) * 2 + h) * 1024 + lane * 16);
    };
    auto read_scales = [&](Scale& s, int slot) {
        const uint8_t* st = smem + slot * STAGE + A_ST + B_ST;
#pragma unroll
        for (int m = 0; m < MB; ++m)
            s.a[m] = *reinterpret_cast<const uint32_t*>(st + ((wm * MB + m) * 32 + lr) * 4) >> (8 * lh);
#pragma unroll
        for (int n = 0; n < NB; ++n)
            s.b[n] = *reinterpret_cast<const uint32_t*>(st + BM * 4 + ((wn * NB + n) * 32 + lr) * 4) >> (8 * lh);
    };

    v16f acc[MB][NB];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int n = 0; n < NB; ++n) acc[m][n] = v16f{};

#pragma unroll
    for (int st = 0; st < TS_NS - 1; ++st) issue(st, min(st, nk - 1));
    QE_WAIT_VMCNT_LDS((TS_NS - 2) * OPS);
    QE_WG_BARRIER();
    Frag f0, f1;
    Scale s;
    read(f0, 0, 0);
    read_scales(s, 0);
    for (int i = 0; i < nk; ++i) {
        const int slot = i % TS_NS;
        // refills the slot of step i - 1: every wave had its last fragments before the barrier below
        // (past the end a repeat of the last step, never used)
        issue((i + TS_NS - 1) % TS_NS, min(i + TS_NS - 1, nk - 1));
        read(f1, slot, 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int n = 0; n < NB; ++n) acc[m][n] = mx_mfma<0>(f0.a[m], s.a[m], f0.b[n], s.b[n], acc[m][n]);
        __builtin_amdgcn_sched_barrier(0);
        // step i + 1 has landed (later ones may be in flight) and this wave's reads of step i are done
        QE_WAIT_VMCNT_LDS((TS_NS - 2) * OPS);
        QE_WG_BARRIER();
        Scale sn;
        read(f0, (i + 1) % TS_NS, 0);
        read_scales(sn, (i + 1) % TS_NS);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int n = 0; n < NB; ++n) acc[m][n] = mx_mfma<1>(f1.a[m], s.a[m], f1.b[n], s.b[n], acc[m][n]);
        s = sn;
    }
    QE_WAIT_VMCNT(0);  // no copy may land after the workgroup has given its LDS back

    // ---- adapter terms (of the first K split)
    int tok[MB], ch[NB];
#pragma unroll
    for (int m = 0; m < MB; ++m) tok[m] = s_tok[(wm * MB + m) * 32 + lr];
#pragma unroll
    for (int n = 0; n < NB; ++n) ch[n] = min(n0 + (wn * NB + n) * 32 + lr, G.d_out - 1);
    if (G.u && ky == 0) {
        for (int k = 0; k < G.rs_pad; k += 16) {
            v8bf a[MB], b[NB];
#pragma unroll
            for (int m = 0; m < MB; ++m)
                a[m] = *reinterpret_cast<const v8bf*>(G.u + (size_t)tok[m] * G.rs_pad + k + lh * 8);
#pragma unroll
            for (int n = 0; n < NB; ++n)
                b[n] = *reinterpret_cast<const v8bf*>(G.bt_s + (size_t)ch[n] * G.rs_pad + k + lh * 8);
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[m], b[n], acc[m][n], 0, 0, 0);
        }
    }
    if (routed && ky == 0) {
        int ex[MB];
        uint32_t present = 0;  // experts of this wave's rows
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            ex[m] = s_ex[(wm * MB + m) * 32 + lr];
            for (int e = 0; e < G.n_r; ++e)
                if (__ballot(ex[m] == e)) present |= 1u << e;
        }
        for (int k = 0; k < G.rr_pad; k += 16) {
            v8bf a[MB];
#pragma unroll
            for (int m = 0; m < MB; ++m)
                a[m] = *reinterpret_cast<const v8bf*>(G.v + (size_t)tok[m] * G.rr_pad + k + lh * 8);
            for (uint32_t left = present; left; left &= left - 1) {
                const int e = __builtin_ctz(left);
                v8bf b[NB];
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    b[n] = *reinterpret_cast<const v8bf*>(G.bt_r + ((size_t)e * G.d_out + ch[n]) * G.rr_pad + k + lh * 8);
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    const v8bf am = ex[m] == e ? a[m] : v8bf{};
#pragma unroll
                    for (int n = 0; n < NB; ++n)
                        acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(am, b[n], acc[m][n], 0, 0, 0);
                }
            }
        }
    }

    // ---- out
    float* part = ksplit > 1 ? G.part + (size_t)ky * T * G.d_out : nullptr;
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int r = (wm * MB + m) * 32 + acc_row(i, lane);
            if (m0 + r >= T) continue;
            const size_t row = (size_t)s_tok[r] * G.d_out;
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const int c = n0 + (wn * NB + n) * 32 + lr;
                if (c >= G.d_out) continue;
                if (part) part[row + c] = acc[m][n][i];
                else store_out(G.y, row + c, acc[m][n][i], G.y_bf16);
            }
        }
}

// ------------------------------------------------------------------ weight streaming
// Up to 32 * TB tokens: a workgroup takes 32 channels (and a K split); its 8 waves take the 128-wide K
// steps in turn, each loading its weight fragments (one contiguous 2 KB per step) and the token rows
// straight into registers, 4 steps at a time; the adapter terms are more steps, dealt to the waves
// alike.  The waves' sums meet in LDS and are added in wave order.
constexpr int SW = 8;  // waves
constexpr int SU = 4;  // K steps requested together by a wave

template <int TB>
__global__ __launch_bounds__(64 * SW) void stream_mx4_kernel(Mx4Gemm G, int ksplit) {
    __shared__ float red[SW][TB * 16][64];
    const int tid = threadIdx.x, wid = tid >> 6, lane = tid & 63, lr = lane & 31, lh = lane >> 5;
    const int nb = blockIdx.x, ky = blockIdx.y;
    const int T = G.T, KB = G.d_in / 128;
    const int kb0 = (int)((long)ky * KB / ksplit), kb1 = (int)((long)(ky + 1) * KB / ksplit);

    const v4i* w = reinterpret_cast<const v4i*>(G.w_tiled) + (size_t)nb * KB * 128 + lane;
    const uint32_t* ws = G.w_scale + (size_t)nb * KB * 32 + lr;
    const uint8_t* a[TB];
    const uint8_t* as[TB];
    int tok[TB];
#pragma unroll
    for (int b = 0; b < TB; ++b) {  // rows past the last token repeat it and are not written
        tok[b] = min(b * 32 + lr, T - 1);
        a[b] = G.codes + (size_t)tok[b] * (G.d_in / 2) + lh * 16;
        as[b] = G.scales + (size_t)tok[b] * (G.d_in / 32);
    }
    v16f acc[TB];
#pragma unroll
    for (int b = 0; b < TB; ++b) acc[b] = v16f{};

    for (int kb = kb0 + wid; kb < kb1; kb += SW * SU) {
        v4i wf[SU][2], af[SU][TB][2];
        uint32_t wsc[SU], asc[SU][TB];
#pragma unroll
        for (int s = 0; s < SU; ++s) {  // steps past the end repeat the last one and are not used
            const int k = min(kb + s * SW, kb1 - 1);
            wf[s][0] = w[(size_t)k * 128];
            wf[s][1] = w[(size_t)k * 128 + 64];
            wsc[s] = ws[(size_t)k * 32];
#pragma unroll
            for (int b = 0; b < TB; ++b) {
                af[s][b][0] = *reinterpret_cast<const v4i*>(a[b] + (size_t)k * 64);
                af[s][b][1] = *reinterpret_cast<const v4i*>(a[b] + (size_t)k * 64 + 32);
                asc[s][b] = *reinterpret_cast<const uint32_t*>(as[b] + (size_t)k * 4);
            }
        }
#pragma unroll
        for (int s = 0; s < SU; ++s) {
            if (kb + s * SW >= kb1) break;
            const uint32_t sw = wsc[s] >> (8 * lh);
#pragma unroll
            for (int b = 0; b < TB; ++b) {
                const uint32_t sa = asc[s][b] >> (8 * lh);
                acc[b] = mx_mfma<0>(af[s][b][0], sa, wf[s][0], sw, acc[b]);
                acc[b] = mx_mfma<1>(af[s][b][1], sa, wf[s][1], sw, acc[b]);
            }
        }
    }

    const int ch = min(nb * 32 + lr, G.d_out - 1);
    int turn = 0;  // adapter steps, dealt to the waves in turn
    if (G.u && ky == 0) {
        for (int k = 0; k < G.rs_pad; k += 16, ++turn) {
            if (turn % SW != wid) continue;
            const v8bf b = *reinterpret_cast<const v8bf*>(G.bt_s + (size_t)ch * G.rs_pad + k + lh * 8);
#pragma unroll
            for (int q = 0; q < TB; ++q) {
                const v8bf ua = *reinterpret_cast<const v8bf*>(G.u + (size_t)tok[q] * G.rs_pad + k + lh * 8);
                acc[q] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ua, b, acc[q], 0, 0, 0);
            }
        }
    }
    if (G.v && ky == 0) {
        int ex[TB];
        uint32_t present = 0;
#pragma unroll
        for (int q = 0; q < TB; ++q) {
            ex[q] = q * 32 + lr < T ? min(max(G.expert[tok[q]], 0), G.n_r - 1) : -1;
            for (int e = 0; e < G.n_r; ++e)
                if (__ballot(ex[q] == e)) present |= 1u << e;
        }
        for (uint32_t left = present; left; left &= left - 1) {
            const int e = __builtin_ctz(left);
            for (int k = 0; k < G.rr_pad; k += 16, ++turn) {
                if (turn % SW != wid) continue;
                const v8bf b = *reinterpret_cast<const v8bf*>(G.bt_r + ((size_t)e * G.d_out + ch) * G.rr_pad + k + lh * 8);
#pragma unroll
                for (int q = 0; q < TB; ++q) {
                    v8bf va = *reinterpret_cast<const v8bf*>(G.v + (size_t)tok[q] * G.rr_pad + k + lh * 8);
                    if (ex[q] != e) va = v8bf{};
                    acc[q] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(va, b, acc[q], 0, 0, 0);
                }
            }
        }
    }

#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (b * 32 + 8 * (i >> 2) < T) red[wid][b * 16 + i][lane] = acc[b][i];
    __syncthreads();
    float* part = ksplit > 1 ? G.part + (size_t)ky * T * G.d_out : nullptr;
    for (int e = tid; e < TB * 16 * 64; e += 64 * SW) {
        const int i = e >> 6, l = e & 63;
        const int t = (i >> 4) * 32 + acc_row(i & 15, l), c = nb * 32 + (l & 31);
        if (t >= T || c >= G.d_out) continue;
        float s = red[0][i][l];
#pragma unroll
        for (int q = 1; q < SW; ++q) s += red[q][i][l];
        const size_t o = (size_t)t * G.d_out + c;
        if (part) part[o] = s;
        else store_out(G.y, o, s, G.y_bf16);
    }
}

// ------------------------------------------------------------------ K splits
// y = the sum of the splits' partials, in split order; 4 outputs per thread (d_out % 16 == 0)
__global__ __launch_bounds__(256) void mx4_finish_kernel(const float* __restrict__ part, int ksplit, size_t n,
                                                         float* __restrict__ y, bool y_bf16) {
    const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    v4f s = *reinterpret_cast<const v4f*>(part + i);
    for (int k = 1; k < ksplit; ++k) s += *reinterpret_cast<const v4f*>(part + k * n + i);
    if (y_bf16) {
        *reinterpret_cast<v2u*>(reinterpret_cast<uint16_t*>(y) + i) =
            v2u{mx4_bf16_bits(s[0]) | (mx4_bf16_bits(s[1]) << 16), mx4_bf16_bits(s[2]) | (mx4_bf16_bits(s[3]) << 16)};
    } else {
        *reinterpret_cast<v4f*>(y + i) = s;
    }
}

Mx4Plan mx4_plan(int T, int d_in, int d_out) {
    Mx4Plan P{0, 1};
    const int KB = d_in / 128;
    if (T <= 0) return P;
    if (T <= kMxMaxTStream) {
        const int wgs = (d_out + 31) / 32;
        P.ksplit = std::max(1, std::min(512 / wgs, KB / SW));
        return P;
    }
    auto tiles = [&](int b) { return (long)((T + b - 1) / b) * ((d_out + b - 1) / b); };
    P.kind = tiles(256) >= 256 ? 256 : tiles(128) >= 192 ? 128 : 64;
    const long n = tiles(P.kind);
    if (n < 256) P.ksplit = (int)std::max(1l, std::min(512 / n, (long)KB / 8));
    return P;
}

hipError_t launch_mx4_gemm(const Mx4Gemm& G, const Mx4Plan& P, hipStream_t st) {
    if (G.T <= 0) return hipSuccess;
    if (P.kind == 0) {
        const dim3 grid((G.d_out + 31) / 32, P.ksplit), block(64 * SW);
        if (G.T <= 32) hipLaunchKernelGGL(stream_mx4_kernel<1>, grid, block, 0, st, G, P.ksplit);
        else hipLaunchKernelGGL(stream_mx4_kernel<2>, grid, block, 0, st, G, P.ksplit);
    } else {
        const int n_tm = (G.T + P.kind - 1) / P.kind, n_tn = (G.d_out + P.kind - 1) / P.kind;
        const dim3 grid((unsigned)((size_t)n_tm * n_tn), P.ksplit);
        if (P.kind == 256) hipLaunchKernelGGL((gemm_mx4_kernel<256, 256>), grid, dim3(256), 0, st, G, n_tm, P.ksplit);
        else if (P.kind == 128) hipLaunchKernelGGL((gemm_mx4_kernel<128, 128>), grid, dim3(256), 0, st, G, n_tm, P.ksplit);
        else hipLaunchKernelGGL((gemm_mx4_kernel<64, 64>), grid, dim3(256), 0, st, G, n_tm, P.ksplit);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || P.ksplit == 1) return e;
    const size_t n = (size_t)G.T * G.d_out;
    hipLaunchKernelGGL(mx4_finish_kernel, dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, st, G.part, P.ksplit, n,
                       G.y, G.y_bf16);
    return hipGetLastError();
}

}  // namespace qe
