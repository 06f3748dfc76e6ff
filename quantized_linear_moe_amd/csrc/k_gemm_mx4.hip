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
#include <type_traits>

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

}  // namespace

// ------------------------------------------------------------------ tiles
// BM tokens x BN channels per workgroup of WM x WN waves, 128 channels of K per step.  Codes and scales
// go global -> LDS by DMA through a ring of NS steps, NS - 1 ahead; each wave holds MB x NB blocks of
// 32 x 32.  The fragments of a half step are read while the MFMAs of the one before run, and the barrier
// that frees a ring slot stands between the two halves of a step, when the second half's fragments are
// already in registers: the matrix cores meet it with work at hand.
//
// Adapter terms are more steps of the same ring: a row's 32 ranks of u (or v) and of B_s (or of one
// expert's B_e) have the 64 bytes of 128 codes, 16 ranks per half, multiplied in bf16.  A routed step is
// masked to its expert's rows; only experts that some row of the tile uses are met.
//
// Operands that come as rows (adapters; activations unless TA) are copied 16 rows of 64 bytes at a time,
// a row's four chunks of 16 stored at chunk ^ ((row >> 2) & 3), so that the fragment reads of 16
// neighbouring rows reach all 64 banks.  TA: the activations come as tiles like the weights
// (mx4_tile_kernel, in the order of perm), every copy contiguous.  Otherwise their scales, one dword per row
// and step, are copied four steps at a time, 16 rows per copy, into four slots of their own: step by step
// every row's dword would be a memory request of its own, as many as the codes make.
//
// What bounds the large tile, 4096 x 8192 -> 29568 without corrections, in a long loop (us; 1.98e12
// operations): 498 in 4 x 2 waves (64 x 128 channels each), 505 in 2 x 4, 508 in 2 x 2 of 128 x 128; without
// the stores of y 451, without the copies' traffic 450, without both 429; the same products on registers
// alone 300 (6.6 POP/s).  The clock is 1.77 GHz in both; the matrix cores are busy 52 % of the cycles here and
// 92 % there, and the waves wait in 28 % of theirs (LDS bank conflicts: none).  Tiles in turn in resident
// workgroups, the next one's first copies behind the stores of the last, took out the stalls between tiles
// but no time.  With both corrections 535, into bf16 500.
template <int BM, int BN, int WM, int WN, bool TA, int NS>
__global__ __launch_bounds__(64 * WM * WN, 1) void gemm_mx4_kernel(Mx4Gemm G, int n_tm, int n_off, int ksplit) {
    constexpr int NW = WM * WN;
    constexpr int MB = BM / 32 / WM, NB = BN / 32 / WN;    // 32x32 blocks per wave
    constexpr int A_ST = BM * 64, B_ST = BN * 64;          // codes per step
    constexpr int A_SC = TA ? BM * 4 : 0, STAGE = A_ST + B_ST + A_SC + BN * 4;  // + scales
    constexpr int ROWSC = NS * STAGE, ROWSC_SLOT = TA ? 0 : BM * 16;  // scales by rows: 4 slots of 4 steps
    constexpr int AD = BM / 16 / NW, BD = BN / 16 / NW;    // 1 KB copies per wave
    constexpr int SQ = BM / 64 + BN / 64, SD = (SQ + NW - 1) / NW;  // 256-byte scale copies: in all, per wave
    constexpr int OPS = AD + BD + SD;
    static_assert(BM % (16 * NW) == 0 && BN % (16 * NW) == 0, "whole copies per wave");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[ROWSC + 4 * ROWSC_SLOT];
    __shared__ int s_tok[BM];  // the token of every row (its position in tiled form is the row's own)
    __shared__ int s_ex[BM];   // its routed expert, -1 past the last token
    __shared__ uint32_t s_present;

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
    const int m0 = tm * BM, n0 = n_off + tn * BN;
    const int tid = threadIdx.x, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63, lr = lane & 31, lh = lane >> 5;
    const int wm = wid % WM, wn = wid / WM;
    const int T = G.T, KB = G.d_in / 128, NBT = (G.d_out + 31) / 32, NBA = (T + 31) / 32;
    const int ky = blockIdx.y;
    const int kb0 = (int)((long)ky * KB / ksplit), nk = (int)((long)(ky + 1) * KB / ksplit) - kb0;
    const bool routed = G.v != nullptr && ky == 0;  // the first K split has the adapter terms

    const uint32_t lds0 = lds_addr(smem);
    const int row_chunk = (lane & 3) ^ ((lane >> 4) & 3);  // of row lane / 4, the chunk that slot lane % 4 holds
    const uint8_t *a_src[AD], *b_src[BD], *s_src[SD], *r_src[SD][4];
    auto scale_copy = [&](int p) { return (wid + NW * p) % SQ; };  // fewer copies than waves: repeated, the same bytes
#pragma unroll
    for (int p = 0; p < BD; ++p) {  // B copy q: half step q & 1 of channel block q >> 1
        const int q = wid + NW * p, nb = min(n0 / 32 + (q >> 1), NBT - 1);
        b_src[p] = G.w_tiled + (((size_t)nb * KB + kb0) * 2 + (q & 1)) * 1024 + lane * 16;
    }
#pragma unroll
    for (int p = 0; p < SD; ++p) {  // scale copies: 64 rows of A each, then 64 channels of B each
        const int q = scale_copy(p);
        if (q >= BM / 64) {
            const int nb = min(n0 / 32 + (q - BM / 64) * 2 + lh, NBT - 1);
            s_src[p] = reinterpret_cast<const uint8_t*>(G.w_scale + ((size_t)nb * KB + kb0) * 32 + lr);
        } else {
            const int mb = min(m0 / 32 + q * 2 + lh, NBA - 1);
            s_src[p] = G.scales + ((size_t)mb * KB + kb0) * 128 + lr * 4;  // (TA)
        }
    }
    // scales by rows: quarter k (16 rows) of copy p for the steps 4g..4g+3 (past the end: the last step's)
    auto issue_row_scales = [&](int p, int k, int g) {
        const uint8_t* src = k == 0 ? r_src[p][0] : k == 1 ? r_src[p][1] : k == 2 ? r_src[p][2] : r_src[p][3];
        dma4(src + 4 * min(4 * g + (lane & 3), nk - 1),
             lds0 + ROWSC + (g & 3) * ROWSC_SLOT + (scale_copy(p) * 64 + k * 16) * 16);
    };
    // copy c of step j of the codes into the ring slot at LDS address `base` (AD of A, BD of B, SD of scales);
    // its source moves on (more != 0).  Of the scales by rows, step j copies a quarter of the group of four
    // steps after its own.
    auto issue = [&](int c, uint32_t base, int more, int j) {
        if (c < AD) {
            dma16(a_src[c], base + (wid + NW * c) * 1024);
            a_src[c] += more * (TA ? 2048 : 64);
        } else if (c < AD + BD) {
            const int p = c - AD;
            dma16(b_src[p], base + A_ST + (wid + NW * p) * 1024);
            b_src[p] += more * 2048;
        } else {
            const int p = c - AD - BD, q = scale_copy(p);
            if (!TA && q < BM / 64) {
                issue_row_scales(p, j & 3, (j >> 2) + 1);
            } else {
                dma4(s_src[p], base + A_ST + B_ST + (q - (TA ? 0 : BM / 64)) * 256);
                s_src[p] += more * 128;
            }
        }
    };
    const int first = min(NS - 1, nk);  // steps of codes among the first NS - 1 of the ring
    // The tile's tokens, then their routed experts.  Copies that do not wait for them go first: the
    // weights, and tiled activations.
    auto issue_first = [&](int c0, int c1) {
        for (int st = 0; st < first; ++st)
#pragma unroll
            for (int c = 0; c < OPS; ++c)
                if (c >= c0 && c < c1) issue(c, lds0 + st * STAGE, st + 1 < nk, st);
    };
    if constexpr (TA) {
#pragma unroll
        for (int p = 0; p < AD; ++p) {
            const int q = wid + NW * p, mb = min(m0 / 32 + (q >> 1), NBA - 1);
            a_src[p] = G.codes + (((size_t)mb * KB + kb0) * 2 + (q & 1)) * 1024 + lane * 16;
        }
        issue_first(0, OPS);
    } else {
        issue_first(AD, AD + BD);
    }
    if (tid == 0) s_present = 0;
    for (int r = tid; r < BM; r += 64 * NW) {
        const int pos = min(m0 + r, T - 1);
        s_tok[r] = G.perm ? G.perm[pos] : pos;
    }
    QE_WAIT_LDS();  // (no __syncthreads: it would also wait for the copies)
    QE_WG_BARRIER();
    if constexpr (!TA) {
#pragma unroll
        for (int p = 0; p < AD; ++p)
            a_src[p] = G.codes + (size_t)s_tok[16 * (wid + NW * p) + (lane >> 2)] * (G.d_in / 2) + (size_t)kb0 * 64 + row_chunk * 16;
#pragma unroll
        for (int p = 0; p < SD; ++p) {
            const int q = scale_copy(p);
            if (q >= BM / 64) continue;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                r_src[p][k] = G.scales + (size_t)s_tok[q * 64 + k * 16 + (lane >> 2)] * (G.d_in / 32) + (size_t)kb0 * 4;
#pragma unroll
            for (int k = 0; k < 4; ++k) issue_row_scales(p, k, 0);
        }
        issue_first(0, AD);
        issue_first(AD + BD, OPS);
    }
    if (routed) {
        for (int r = tid; r < BM; r += 64 * NW) {
            const int e = m0 + r < T ? min(max(G.expert[s_tok[r]], 0), G.n_r - 1) : -1;
            s_ex[r] = e;
            if (e >= 0) atomicOr(&s_present, 1u << e);
        }
        QE_WAIT_LDS();
        QE_WG_BARRIER();
    }
    const uint32_t present = __builtin_amdgcn_readfirstlane(s_present);
    // Adapter steps follow the nk steps of codes: the shared expert's, then those of every present expert in
    // turn.  `turn` walks them; the experts of the steps in the ring wait in `queue`.
    const int se = G.u && ky == 0 ? G.rs_pad / 32 : 0, re = G.rr_pad / 32;
    const int nt = nk + se + __popc(present) * re;
    struct {
        int s, k;
        uint32_t left;
    } turn = {0, 0, present};
    int queue[NS];
    const uint16_t *ad_x, *ad_bt;  // the rows of the adapter step being copied
    int ad_pad;
    int ad_tok[AD], ad_ch[BD];
#pragma unroll
    for (int p = 0; p < AD; ++p) ad_tok[p] = s_tok[16 * (wid + NW * p) + (lane >> 2)];
#pragma unroll
    for (int p = 0; p < BD; ++p) ad_ch[p] = min(n0 + 16 * (wid + NW * p) + (lane >> 2), G.d_out - 1);
    auto next_adapter = [&]() {  // (after the last one: the last again, into slots that nothing reads)
        int e = -1;
        if (turn.s < se) {
            ad_x = G.u + turn.s * 32;
            ad_bt = G.bt_s + turn.s * 32;
            ad_pad = G.rs_pad;
            ++turn.s;
        } else if (turn.left) {
            e = __builtin_ctz(turn.left);
            ad_x = G.v + turn.k;
            ad_bt = G.bt_r + (size_t)e * G.d_out * G.rr_pad + turn.k;
            ad_pad = G.rr_pad;
            turn.k += 32;
            if (turn.k == G.rr_pad) {
                turn.k = 0;
                turn.left &= turn.left - 1;
            }
        }
#pragma unroll
        for (int q = 0; q + 1 < NS; ++q) queue[q] = queue[q + 1];
        queue[NS - 1] = e;
    };
    // copy c of that step (the scales' are repeated: every step makes the same number of copies)
    auto issue_adapter = [&](int c, uint32_t base, int j) {
        if (c < AD) dma16(ad_x + (size_t)ad_tok[c] * ad_pad + row_chunk * 8, base + (wid + NW * c) * 1024);
        else if (c < AD + BD) dma16(ad_bt + (size_t)ad_ch[c - AD] * ad_pad + row_chunk * 8, base + A_ST + (wid + NW * (c - AD)) * 1024);
        else issue(c, base, 0, j);
    };
    for (int st = first; st < NS - 1; ++st) {  // (fewer steps of codes than the ring holds)
        if (nt > nk) {
            next_adapter();
#pragma unroll
            for (int c = 0; c < OPS; ++c) issue_adapter(c, lds0 + st * STAGE, st);
        } else {
#pragma unroll
            for (int c = 0; c < OPS; ++c) issue(c, lds0 + st * STAGE, 0, st);
        }
    }
    int ex[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) ex[m] = routed ? s_ex[(wm * MB + m) * 32 + lr] : -1;

    // fragments and scales of the slot at offset `st`, numbered so that their reads can be spread between
    // MFMAs: MB of A, then NB of B.  offa, offb: the fragments' places, as tiles or as rows
    v4i fa[2][MB], fb[2][NB];
    uint32_t ra[MB], rb[NB], sa[MB], sb[NB];  // scale dwords as read, and with the lane's blocks in bytes 0 and 2
    const int swz = (lr >> 2) & 3, rows_a = (wm * MB * 32 + lr) * 64, rows_b = A_ST + (wn * NB * 32 + lr) * 64;
    const int row_a[2] = {rows_a + ((lh ^ swz) << 4), rows_a + (((2 + lh) ^ swz) << 4)};
    const int row_b[2] = {rows_b + ((lh ^ swz) << 4), rows_b + (((2 + lh) ^ swz) << 4)};
    const int tile_a = wm * MB * 2048 + lane * 16, tile_b = A_ST + wn * NB * 2048 + lane * 16;
    const int code_a[2] = {TA ? tile_a : row_a[0], TA ? tile_a + 1024 : row_a[1]}, code_b[2] = {tile_b, tile_b + 1024};
    const int off_sa = TA ? A_ST + B_ST + (wm * MB * 32 + lr) * 4 : ROWSC + (wm * MB * 32 + lr) * 16;
    const int off_sb = A_ST + B_ST + A_SC + (wn * NB * 32 + lr) * 4;
    auto read = [&](int q, int st, int h, int offa, int offb) {
        if (q < MB) fa[h][q] = *reinterpret_cast<const v4i*>(smem + st + offa + q * 2048);
        else if (q < MB + NB) fb[h][q - MB] = *reinterpret_cast<const v4i*>(smem + st + offb + (q - MB) * 2048);
    };
    auto read_scale = [&](int q, int st, int j) {  // of step j
        if (q < MB) {
            const int o = TA ? st + q * 128 : ((j >> 2) & 3) * ROWSC_SLOT + (j & 3) * 4 + q * 512;
            ra[q] = *reinterpret_cast<const uint32_t*>(smem + off_sa + o);
        } else if (q < MB + NB) {
            rb[q - MB] = *reinterpret_cast<const uint32_t*>(smem + st + off_sb + (q - MB) * 128);
        }
    };

    v16f acc[MB][NB];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int n = 0; n < NB; ++n) acc[m][n] = v16f{};

    QE_WAIT_VMCNT_LDS(TA ? (NS - 2) * OPS : 0);  // rows: the first copies were not issued step by step
    QE_WG_BARRIER();
#pragma unroll
    for (int q = 0; q < MB + NB; ++q) {
        read(q, 0, 0, code_a[0], code_b[0]);
        read_scale(q, 0, 0);
    }
    constexpr int NM = MB * NB;  // MFMAs of a half step
    constexpr int RQ = (MB + NB + NM - 1) / NM, CQ = (OPS + NM - 1) / NM;
    int st = 0, st_next = STAGE, st_fill = (NS - 1) * STAGE;  // slots of steps i, i + 1 and i + NS - 1
    // One step.  A wave issues in order, so whatever stands between two MFMAs for longer than one takes is
    // lost to the matrix cores: reads and copies go one or two to an MFMA, fenced so that they stay there.
    // kStep: 0 codes, copying codes; 1 codes, copying an adapter step; 2 adapter.  The slot refilled is that
    // of step i - 1: every wave had its last fragments before the barrier (past the end: a repeat, never used).
    auto step = [&](auto kind, int i) {
        constexpr int kStep = decltype(kind)::value;
        const int more = i + NS < nk;
        int e = -1;
        if constexpr (kStep != 0) next_adapter();  // step i's own expert is now first in the queue
        if constexpr (kStep == 2) {
            e = queue[0];
        } else {
#pragma unroll
            for (int m = 0; m < MB; ++m) sa[m] = ra[m] >> (8 * lh);
#pragma unroll
            for (int n = 0; n < NB; ++n) sb[n] = rb[n] >> (8 * lh);
        }
        auto mfma = [&](auto half, int q) {
            constexpr int H = decltype(half)::value;
            const int m = q / NB, n = q % NB;
            if constexpr (kStep == 2) {
                const v4i a = e < 0 || ex[m] == e ? fa[H][m] : v4i{0, 0, 0, 0};
                acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a),
                                                                    __builtin_bit_cast(v8bf, fb[H][n]), acc[m][n], 0, 0, 0);
            } else {
                acc[m][n] = mx_mfma<H>(fa[H][m], sa[m], fb[H][n], sb[n], acc[m][n]);
            }
        };
        const int here_a = kStep == 2 ? row_a[1] : code_a[1], here_b = kStep == 2 ? row_b[1] : code_b[1];
        const bool codes_next = kStep == 0 || (kStep == 1 && i + 1 < nk);
        const int next_a = codes_next ? code_a[0] : row_a[0], next_b = codes_next ? code_b[0] : row_b[0];
#pragma unroll
        for (int q = 0; q < NM; ++q) {
            mfma(std::integral_constant<int, 0>{}, q);
#pragma unroll
            for (int r = 0; r < RQ; ++r) read(q * RQ + r, st, 1, here_a, here_b);
#pragma unroll
            for (int r = 0; r < CQ; ++r)
                if (q * CQ + r < OPS) {
                    if constexpr (kStep == 0) issue(q * CQ + r, lds0 + st_fill, more, i + NS - 1);
                    else issue_adapter(q * CQ + r, lds0 + st_fill, i + NS - 1);
                }
            __builtin_amdgcn_sched_barrier(0);
        }
        // step i + 1 has landed (later ones may be in flight) and this wave's reads of step i are done
        QE_WAIT_VMCNT_LDS((NS - 2) * OPS);
        QE_WG_BARRIER();
#pragma unroll
        for (int q = 0; q < NM; ++q) {
            mfma(std::integral_constant<int, 1>{}, q);
#pragma unroll
            for (int r = 0; r < RQ; ++r) {
                read(q * RQ + r, st_next, 0, next_a, next_b);
                if constexpr (kStep != 2) read_scale(q * RQ + r, st_next, i + 1);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        st = st_next;
        st_next = st_next == (NS - 1) * STAGE ? 0 : st_next + STAGE;
        st_fill = st_fill == (NS - 1) * STAGE ? 0 : st_fill + STAGE;
    };
    int i = 0;
    for (const int end = nt == nk ? nk : nk - (NS - 1); i < end; ++i) step(std::integral_constant<int, 0>{}, i);
    for (; i < nk; ++i) step(std::integral_constant<int, 1>{}, i);
    for (; i < nt; ++i) step(std::integral_constant<int, 2>{}, i);
    QE_WAIT_VMCNT_LDS(0);  // no copy may land after the workgroup has given its LDS back

    // ---- out: every wave turns one row of 32x32 blocks at a time into whole rows through its own part of
    // the ring, and stores 16 bytes per lane, past the caches (nothing here reads y again)
    QE_WG_BARRIER();  // the copies of every wave have landed
    constexpr int COLS = NB * 32, PITCH = COLS * 4 + 16;  // channels and LDS bytes of a row
    static_assert(NW * 32 * PITCH <= NS * STAGE, "the ring holds the waves' rows");
    uint8_t* flip = smem + wid * 32 * PITCH;
    const int c0 = n0 + wn * COLS;
    auto out = [&](auto kind) {
        constexpr int kOut = decltype(kind)::value;  // 0 partial sums, 1 float32, 2 bf16
        constexpr int E = kOut == 2 ? 8 : 4, LPR = COLS / E, RPI = 64 / LPR;  // elements per lane, lanes per row, rows per store
        float* base = kOut == 0 ? G.part + (size_t)ky * T * G.d_out : G.y;
        const int c = lane % LPR * E;
#pragma unroll
        for (int m = 0; m < MB; ++m) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    *reinterpret_cast<float*>(flip + acc_row(j, lane) * PITCH + (n * 32 + lr) * 4) = acc[m][n][j];
#pragma unroll
            for (int j = 0; j < 32 / RPI; ++j) {
                const int r = j * RPI + lane / LPR, q = (wm * MB + m) * 32 + r;
                const v4f* p = reinterpret_cast<const v4f*>(flip + r * PITCH + c * 4);
                const v4f lo = p[0];
                if (m0 + q >= T || c0 + c >= G.d_out) continue;
                const size_t o = (size_t)s_tok[q] * G.d_out + c0 + c;
                if constexpr (kOut == 2) {
                    const v4f hi = p[1];
                    const v4u w = v4u{mx4_bf16_bits(lo[0]) | (mx4_bf16_bits(lo[1]) << 16),
                                      mx4_bf16_bits(lo[2]) | (mx4_bf16_bits(lo[3]) << 16),
                                      mx4_bf16_bits(hi[0]) | (mx4_bf16_bits(hi[1]) << 16),
                                      mx4_bf16_bits(hi[2]) | (mx4_bf16_bits(hi[3]) << 16)};
                    __builtin_nontemporal_store(w, reinterpret_cast<v4u*>(reinterpret_cast<uint16_t*>(base) + o));
                } else if constexpr (kOut == 1) {
                    __builtin_nontemporal_store(lo, reinterpret_cast<v4f*>(base + o));
                } else {
                    *reinterpret_cast<v4f*>(base + o) = lo;
                }
            }
        }
    };
    if (ksplit > 1) out(std::integral_constant<int, 0>{});
    else if (G.y_bf16) out(std::integral_constant<int, 2>{});
    else out(std::integral_constant<int, 1>{});
}

// ------------------------------------------------------------------ weight streaming
// Up to 32 * TB tokens: a workgroup takes 32 channels; its waves take the 128-wide K steps in turn, each
// loading its weight fragments (one contiguous 2 KB per step) and the token rows straight into registers,
// SU steps at a time; the adapter terms are more steps, dealt to the waves alike.  The waves' sums meet in
// LDS and are added in wave order; a split of K over workgroups would need a second launch.  Bound by the
// reads of the weights: 8192 -> 29568, 1 token 23.5 us (5.5 TB/s); 29568 -> 8192, 8 tokens with both
// corrections 25.6.  (8 waves, or 2 or 8 steps together: no faster.)
constexpr int SW = 16;  // waves
constexpr int SU = 4;   // K steps requested together by a wave

template <int TB>
__global__ __launch_bounds__(64 * SW) void stream_mx4_kernel(Mx4Gemm G) {
    __shared__ float red[SW][16][64];
    const int tid = threadIdx.x, wid = tid >> 6, lane = tid & 63, lr = lane & 31, lh = lane >> 5;
    const int nb = blockIdx.x, T = G.T, KB = G.d_in / 128;

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

    for (int kb = wid; kb < KB; kb += SW * SU) {
        v4i wf[SU][2], af[SU][TB][2];
        uint32_t wsc[SU], asc[SU][TB];
#pragma unroll
        for (int s = 0; s < SU; ++s) {  // steps past the end repeat the last one and are not used
            const int k = min(kb + s * SW, KB - 1);
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
            if (kb + s * SW >= KB) break;
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
    if (G.u) {
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
    if (G.v) {
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
    for (int b = 0; b < TB; ++b) {
        if (b > 0) __syncthreads();
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (b * 32 + 8 * (i >> 2) < T) red[wid][i][lane] = acc[b][i];
        __syncthreads();
        for (int e = tid; e < 16 * 64; e += 64 * SW) {
            const int i = e >> 6, l = e & 63;
            const int t = b * 32 + acc_row(i, l), c = nb * 32 + (l & 31);
            if (t >= T || c >= G.d_out) continue;
            float s = red[0][i][l];
#pragma unroll
            for (int q = 1; q < SW; ++q) s += red[q][i][l];
            store_out(G.y, (size_t)t * G.d_out + c, s, G.y_bf16);
        }
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

// Which kernel.  Times are us per call with both corrections (8 experts, ranks 32), weights not in the caches.
//   * Weight streaming re-reads the token rows for every 32 channels, about T row requests per step and CU; the
//     weights themselves bound it up to 12 tokens.  8192 -> 29568: 8 tokens 26 streamed, 29 in 64 x 128 tiles;
//     16 tokens 34, 31; 32 tokens 53, 36.  29568 -> 8192 (a quarter of the steps per CU): 16 tokens 28, 33;
//     32 tokens 46, 35.  8192 -> 1024: 32 tokens 13, 15.
//   * 256 x 256 tiles, one per CU, where they give every CU one, or 128 x 128 tiles would need a second round of
//     two per CU: 512 x 8192 -> 29568 80 (128 x 128: 132), 512 x 3584 -> 18944 35 (44), 1024 x 1536 -> 8960 24
//     (30); 1024 x 8192 -> 8192, where they would not, 52 (49); 2048 x 4096 -> 4096 35 (32).  Not for up to
//     128 tokens: 100 x 3584 -> 151936 118 (103), 64 of them 93 (64 x 128: 69).
//   * 128 x 128 tiles, two per CU: 128 x 8192 -> 29568 42, in 64 x 128 tiles 59; 512 x 8192 -> 8192 31, 34.  Fewer of
//     them with long sums, split where half the CUs would be idle: 640 x 18944 -> 3584 47 (64 x 128: 61),
//     320 x 18944 -> 3584 in 3 splits 35 (40), 256 x 29568 -> 8192 in 2 60 (73), 128 x 29568 -> 8192 in 4 48 (52);
//     with 8192 tile steps 256 x 8192 -> 8192 28 (24), with 7168 256 x 14336 -> 4096 27 (24).
//   * 64 x 128 tiles: 32 x 8192 -> 29568 36, in 128 x 128 tiles 43.  Long sums in few tiles are split:
//     64 x 29568 -> 8192 80 unsplit, 53 in 2, 41 in 4.
//   * 64 x 64 tiles, split until there are about 512: 128 x 18944 -> 3584 40 unsplit, 23 split.
Mx4Plan mx4_plan(int T, int d_in, int d_out) {
    Mx4Plan P{0, 0, 1};
    const int KB = d_in / 128, wgs = (int)(((long)d_out + 31) / 32);
    if (T <= 12 || (T <= kMxMaxTStream && (long)((wgs + 255) / 256) * KB * T <= 3800)) return P;
    auto tiles = [&](int bm, int bn) { return ((long)T + bm - 1) / bm * (((long)d_out + bn - 1) / bn); };
    const long t128x128 = tiles(128, 128), t64x128 = tiles(64, 128), t64x64 = tiles(64, 64);
    if (KB >= 8 && T > 128 && (tiles(256, 256) >= 256 || t128x128 > 512)) P = {256, 256, 1};
    else if (T > 64 && t128x128 >= 192) P = {128, 128, 1};
    else if (T > 64 && t128x128 * KB >= 11000) P = {128, 128, (int)std::max(1l, std::min(256 / t128x128, 4l))};
    else if (t64x128 >= 200) P = {64, 128, 1};
    else if (t64x128 >= 50 && KB >= 64) P = {64, 128, (int)std::min(512 / t64x128, 4l)};
    else P = {64, 64, (int)std::max(1l, std::min(512 / std::min(t64x64, 512l), (long)KB / 8))};
    return P;
}

// Columns of 256-channel tiles for the large-tile launch: one tile runs per CU, so a last round that fills
// few of the 256 CUs is given to 128 x 128 tiles instead (two per CU, a quarter of the work each).
static int mx4_main_columns(int n_tm, int n_tn) {
    const long n = (long)n_tm * n_tn, rounds = n / 256, rest = n - rounds * 256;
    const int main = (int)(rounds * 256 / n_tm);
    // (main 0: a column has more tiles than the full rounds)
    return rest == 0 || rest > 96 || main == 0 ? n_tn : main;
}

hipError_t launch_mx4_gemm(const Mx4Gemm& G, const Mx4Plan& P, hipStream_t st) {
    if (G.T <= 0) return hipSuccess;
    if (P.bm == 0) {
        const dim3 grid((G.d_out + 31) / 32), block(64 * SW);
        if (G.T <= 32) hipLaunchKernelGGL(stream_mx4_kernel<1>, grid, block, 0, st, G);
        else hipLaunchKernelGGL(stream_mx4_kernel<2>, grid, block, 0, st, G);
        return hipGetLastError();
    }
    Mx4Gemm H = G;
    const bool tiled = !G.codes || mx4_tiled(P, G.d_in);
    if (tiled) {
        if (G.codes) {
            const hipError_t e = launch_mx4_tile(G.codes, G.scales, G.perm, G.T, G.d_in, G.a_tiled, G.a_scale, st);
            if (e != hipSuccess) return e;
        }
        H.codes = G.a_tiled;
        H.scales = reinterpret_cast<const uint8_t*>(G.a_scale);
    }
    // one launch: tiles of channels n_off, n_off + bn, ... (columns of them) by all tokens
    auto launch = [&](auto kernel, int bm, int bn, int threads, int n_off, int columns) {
        const int n_tm = (G.T + bm - 1) / bm;
        hipLaunchKernelGGL(kernel, dim3((unsigned)((size_t)n_tm * columns), P.ksplit), dim3(threads), 0, st, H, n_tm,
                           n_off, P.ksplit);
    };
    const int columns = (G.d_out + P.bn - 1) / P.bn;
    if (P.bm == 256) {
        const int main = mx4_main_columns((G.T + 255) / 256, columns);
        launch(gemm_mx4_kernel<256, 256, 4, 2, true, 4>, 256, 256, 512, 0, main);
        if (main * 256 < G.d_out)
            launch(gemm_mx4_kernel<128, 128, 2, 2, true, 4>, 128, 128, 256, main * 256, (G.d_out - main * 256 + 127) / 128);
    } else if (P.bm == 128) {
        if (tiled) launch(gemm_mx4_kernel<128, 128, 2, 2, true, 4>, 128, 128, 256, 0, columns);
        else launch(gemm_mx4_kernel<128, 128, 2, 2, false, 4>, 128, 128, 256, 0, columns);
    } else if (P.bn == 128) {
        launch(gemm_mx4_kernel<64, 128, 2, 2, false, 4>, 64, 128, 256, 0, columns);
    } else {
        launch(gemm_mx4_kernel<64, 64, 2, 2, false, 4>, 64, 64, 256, 0, columns);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || P.ksplit == 1) return e;
    const size_t n = (size_t)G.T * G.d_out;
    hipLaunchKernelGGL(mx4_finish_kernel, dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, st, G.part, P.ksplit, n,
                       G.y, G.y_bf16);
    return hipGetLastError();
}

}  // namespace qe
