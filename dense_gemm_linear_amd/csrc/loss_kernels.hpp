// Kernels of the linear head's losses (loss.hip holds the rest and launches
// them).  With z = scale * X W^T over the vocabulary (X [T, D], W [V, D] bf16)
// four products are needed, none of which may leave z in memory:
//
//   ROLE_LSE   z tile of X W^T -> per row and tile column: maximum and
//              sum of exp(z - maximum) over the columns other than the row's
//              label, the pieces of a log-sum-exp, and the label's z apart.
//              (With both in one sum, the loss lse - z[label] of a label of
//              probability near 1 would be the difference of two equal
//              numbers; apart, it is log(1 + exp(lse_others - z[label])),
//              exact to a few units of the last place of z.)
//   ROLE_GRAD  the same z tile again, for one piece of the vocabulary:
//              G = a exp(z - lse), and b at the label's column, rounded to
//              bf16 for the two products below (to nearest: at most 2^-8 of
//              the value, as the gradients themselves are rounded).
//   ROLE_DX    dX += G W over the piece's columns, fp32 planes.
//   ROLE_DW    dW = G^T X for the piece's rows of W.
//
// X and W are taken as they lie in memory; no operand is laid out first.  An
// operand whose contraction axis is contiguous (X and W in the logits, G in
// dX) is staged in LDS as the A operand of gemm_ab_kernel is.  One whose
// contraction axis is its row index (W in dX; G and X in dW) is staged as rows
// of the other axis and read with gfx950's transposing LDS read, which hands
// each lane four values of one column: a transposed copy of W alone would cost
// 4 bytes of traffic per weight and direction.
#pragma once

#include "kernels.hpp"

namespace dg {

enum { ROLE_LSE = 0, ROLE_GRAD = 1, ROLE_DX = 2, ROLE_DW = 3 };

// One kept row: what its gradient needs, in compact row order.
struct RowInfo {
    float lse;
    float a;      // factor of exp(z - lse): dloss * scale * (1 + 2 z_loss lse)
    float b;      // the gradient at the label's column
    int label;    // column of W, -1: none
};

struct LossArgs {
    const uint8_t* A;      // X compact [n, lda] (LSE, GRAD), G [n, lda] (DX, DW)
    const uint8_t* B;      // W [., ldb] from the piece's first row (LSE, GRAD, DX), X compact (DW)
    int64_t lda_b, ldb_b;  // row pitches in bytes
    const int* n_kept;     // rows of X that take part (device)
    int M, N, K;           // M: DW only (the piece's rows of W); K: not for DW (n)
    int tiles_n;
    int splits, kt_per;    // DX: K slices, k-tiles per slice
    float scale;
    const RowInfo* rows;
    float2* part;          // LSE: [tiles_n][ldpart] (maximum, sum)
    int64_t ldpart;
    float* zlabel;         // LSE: z at the label, compact rows
    int v0;                // GRAD: first column of the piece
    float* planes;         // DX: [splits][plane_rows][ldplane]
    int64_t plane;         // elements of one plane
    int64_t ldplane;
    int first;             // DX: the first piece writes, later ones add
    uint16_t* C;           // GRAD: G; DW: dW
    int64_t ldc;
    int c_vec;
};

// Tile shape: TM x TN outputs, WM x WN waves, ST stages of KTB bytes of K,
// OCC waves per SIMD to leave registers for.
template <int TM_, int TN_, int WM_, int WN_, int ST_, int KTB_, int OCC_>
struct LossShape {
    static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, ST = ST_, KTB = KTB_, OCC = OCC_;
    static constexpr int R = 16;
    static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
    static constexpr int MR = TM / WM / R, NR = TN / WN / R;
    static constexpr int A_BUF = TM * KTB, B_BUF = TN * KTB, STAGE = A_BUF + B_BUF;
    static constexpr int A_DMA = A_BUF / 1024 / WAVES, B_DMA = B_BUF / 1024 / WAVES;
    static constexpr int LOADS = A_DMA + B_DMA;
    static constexpr int KT = KTB / 2;                 // k-tile in elements
    static constexpr int WCOLS = TN / WN;
    static constexpr int SROW = WCOLS * 2 + 16;
    static constexpr int ROWS_LDS = TM * 16;           // RowInfo of the tile's rows
    static constexpr int CH = fit_stage_rows(MR, WAVES, R, SROW, ST * STAGE - ROWS_LDS);
    static constexpr int LDS = ST * STAGE;
    static_assert(MR >= 1 && NR >= 1 && MR * WM * R == TM && NR * WN * R == TN, "tile shape");
    static_assert(A_DMA >= 1 && B_DMA >= 1 && A_DMA * 1024 * WAVES == A_BUF &&
                      B_DMA * 1024 * WAVES == B_BUF, "DMA split");
    static_assert(WAVES * CH * R * SROW + ROWS_LDS <= LDS && LDS <= 160 * 1024, "LDS budget");
    static_assert(TM * 4 + WN * TM * 8 <= LDS, "LSE reduction space");
};

typedef short s16x4 __attribute__((ext_vector_type(4)));

// gfx950's transposing LDS read of 16-bit values: in each group of 16 lanes,
// lane i supplies the address of four values, (row i / 4, columns 4 (i % 4)
// ..), of a 4 x 16 block and receives column i, rows 0 .. 3.
//
// The pointer is restrict so that the read carries alias information, as an
// ordinary load does by its type: without any, the compiler waits before it
// for every LDS DMA in flight (vmcnt(0) in front of each group of reads),
// which empties the pipeline k_loop fills.  What those loads write and when it
// may be read is k_loop's own barrier.
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
__device__ __forceinline__ s16x4 lds_read_tr16(lds_s16x4* __restrict p)
{
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
}

// Rows of a transposed operand's stage: TW columns of 2 bytes, 32-byte unit u
// of k row r stored at unit u ^ tr_key(r).  A fragment read takes rows 8 g +
// 4 h + 0 .. 3 for lane group g: the two groups served together read rows
// {0-3, 8-11} (+16), and the key sends those eight to eight different 32-byte
// spans of the 256 bytes the banks cover.
__host__ __device__ constexpr uint32_t tr_key(uint32_t row) { return (row & 3u) | ((row >> 1) & 4u); }

// Maximum / sum over the 16 lanes of a row group, in every lane of it.
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float x)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float row16_max(float x)
{
    x = fmaxf(x, dpp_f32<0x128>(x));   // row_ror:8, 4, 2, 1
    x = fmaxf(x, dpp_f32<0x124>(x));
    x = fmaxf(x, dpp_f32<0x122>(x));
    return fmaxf(x, dpp_f32<0x121>(x));
}
__device__ __forceinline__ float row16_sum(float x)
{
    x += dpp_f32<0x128>(x);
    x += dpp_f32<0x124>(x);
    x += dpp_f32<0x122>(x);
    return x + dpp_f32<0x121>(x);
}

constexpr float kLog2e = 1.44269504088896340736f;

// exp(z - m): the difference first, so that a large common part of z and m
// leaves no error in the exponent (one hardware exponential, 1 ulp).
__device__ __forceinline__ float exp_diff(float z, float m)
{
    return __builtin_amdgcn_exp2f((z - m) * kLog2e);
}

template <class S, int ROLE>
__global__ __launch_bounds__(S::THREADS, S::OCC) void loss_gemm_kernel(LossArgs p)
{
    using AT = Atom<DT_BF16, 16>;
    using KTL = KTile<S::KTB>;
    using acc_t = AT::acc_t;
    constexpr int TM = S::TM, TN = S::TN, WN = S::WN, R = 16, KTB = S::KTB, KT = S::KT;
    constexpr int MR = S::MR, NR = S::NR, A_DMA = S::A_DMA, B_DMA = S::B_DMA;
    constexpr int A_BUF = S::A_BUF, STAGE = S::STAGE, WAVES = S::WAVES, ST = S::ST;
    constexpr int STEPS = KTB / 64;
    constexpr bool TRA = ROLE == ROLE_DW, TRB = ROLE == ROLE_DX || ROLE == ROLE_DW;
    static_assert(!TRA || TM >= 128, "a transposed operand's unit key needs 8 units a row");
    static_assert(!TRB || TN >= 128, "a transposed operand's unit key needs 8 units a row");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];

    const int n = *p.n_kept;
    const int M = ROLE == ROLE_DW ? p.M : n;
    const int tiles_m = (M + TM - 1) / TM;
    // the grid is sized for every row of X; n may be less
    const int grid = tiles_m * p.tiles_n;
    int slice = 0, wg = (int)blockIdx.x;
    if constexpr (ROLE == ROLE_DX) {
        if (grid == 0)
            return;
        slice = wg / grid;
        wg -= slice * grid;
        if (slice >= p.splits)
            return;
    } else if (wg >= grid) {
        return;
    }
    int tm, tn;
    tile_raster<DG_GROUP_M>(xcd_remap(wg, grid), tiles_m, p.tiles_n, tm, tn);
    const int m0 = tm * TM, n0 = tn * TN;
    const int rows = min(TM, M - m0);

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int lc = lane & 15, lg = lane >> 4;

    // K range in elements and k-tiles
    const int K = ROLE == ROLE_DW ? n : p.K;
    int kt0 = 0, nkt = (K + KT - 1) / KT, k_end = K;
    if constexpr (ROLE == ROLE_DX) {
        kt0 = slice * p.kt_per;
        const int kt_end = min(nkt, kt0 + p.kt_per);
        nkt = max(0, kt_end - kt0);
        k_end = min(K, kt_end * KT);
    }

    // ---- loads.  Plain operand: rows of K, KTB bytes a k-tile, chunk c of
    // row r at c ^ key(r); rows past the bound read zero, chunks past K go out
    // of range.  Transposed operand: the k-tile's KT rows, the descriptor
    // rebased to them, so that no offset grows with K and rows past K read
    // zero; columns past the matrix hold other rows' values and only reach
    // outputs that are not stored.
    uint32_t a_goff[A_DMA], a_col[A_DMA], b_goff[B_DMA], b_col[B_DMA];
#pragma unroll
    for (int i = 0; i < A_DMA; ++i) {
        if constexpr (TRA) {
            const uint32_t at = (uint32_t)(wave + WAVES * i) * 1024u + (uint32_t)lane * 16u;
            const uint32_t r = at / (TM * 2), c = at % (TM * 2) / 16;
            a_goff[i] = r * (uint32_t)p.lda_b + ((c ^ (tr_key(r) << 1)) << 4);
            a_col[i] = 0;
        } else {
            const ADma d = a_dma_lane<KTB>(wave + WAVES * i, lane, p.lda_b);
            a_goff[i] = d.goff;
            a_col[i] = d.col;
        }
    }
#pragma unroll
    for (int i = 0; i < B_DMA; ++i) {
        if constexpr (TRB) {
            const uint32_t at = (uint32_t)(wave + WAVES * i) * 1024u + (uint32_t)lane * 16u;
            const uint32_t r = at / (TN * 2), c = at % (TN * 2) / 16;
            b_goff[i] = r * (uint32_t)p.ldb_b + ((c ^ (tr_key(r) << 1)) << 4);
            b_col[i] = 0;
        } else {
            const ADma d = a_dma_lane<KTB>(wave + WAVES * i, lane, p.ldb_b);
            b_goff[i] = d.goff;
            b_col[i] = d.col;
        }
    }
    const int brows = min(TN, p.N - n0);
    const uint8_t* a_base = TRA ? p.A + (int64_t)m0 * 2 : p.A + (int64_t)m0 * p.lda_b;
    const uint8_t* b_base = TRB ? p.B + (int64_t)n0 * 2 : p.B + (int64_t)n0 * p.ldb_b;
    // a transposed operand's bytes from its base to the end of row K - 1
    // (G's rows are padded: its last, partial 16 bytes are read whole)
    const int64_t a_span = TRA ? (int64_t)(k_end - 1) * p.lda_b + (int64_t)(p.M - m0 + 7) / 8 * 16 : 0;
    const int64_t b_span = TRB ? (int64_t)(k_end - 1) * p.ldb_b + (int64_t)(p.N - n0) * 2 : 0;
    const rsrc_t ra = make_rsrc(
        a_base, TRA ? 0u : (uint32_t)((int64_t)(rows - 1) * p.lda_b + (int64_t)(K + 7) / 8 * 16));
    const rsrc_t rb = make_rsrc(b_base, TRB ? 0u : (uint32_t)((int64_t)(brows - 1) * p.ldb_b + (int64_t)K * 2));
    const int kb_end = k_end * 2;                    // bytes of K a plain operand may read
    const int last_full = kb_end / KTB;

    auto rebase = [&](const uint8_t* base, int64_t span, int64_t off) __attribute__((always_inline)) {
        const int64_t left = span - off;
        return make_rsrc(base + off, left <= 0 ? 0u : (uint32_t)min(left, (int64_t)0x7FFFFFFF));
    };
    auto load = [&](int kt_local, int stage, int part, int nparts, auto nomask_c)
                    __attribute__((always_inline)) {
        constexpr bool NOMASK = decltype(nomask_c)::value;
        const int kt = kt0 + kt_local;
        const bool mask = kt >= last_full;
        uint8_t* base = lds + stage * STAGE;
        const rsrc_t rat = TRA ? rebase(a_base, a_span, (int64_t)kt * KT * p.lda_b) : ra;
        const rsrc_t rbt = TRB ? rebase(b_base, b_span, (int64_t)kt * KT * p.ldb_b) : rb;
        auto one = [&](rsrc_t r, uint8_t* dst, uint32_t goff, uint32_t col, auto tr)
                       __attribute__((always_inline)) {
            if constexpr (decltype(tr)::value) {
                dma16(r, dst, goff, 0);
            } else if constexpr (NOMASK) {
                dma16(r, dst, goff, (uint32_t)kt * KTB);
            } else {
                uint32_t off = goff + (uint32_t)kt * KTB;
                if (mask && (int)((uint32_t)kt * KTB + col) >= kb_end)
                    off = kOOB;
                dma16(r, dst, off, 0);
            }
        };
#pragma unroll
        for (int i = 0; i < A_DMA; ++i)
            if (i % nparts == part)
                one(rat, base + (wave + WAVES * i) * 1024, a_goff[i], a_col[i],
                    std::integral_constant<bool, TRA>{});
#pragma unroll
        for (int i = 0; i < B_DMA; ++i)
            if ((A_DMA + i) % nparts == part)
                one(rbt, base + A_BUF + (wave + WAVES * i) * 1024, b_goff[i], b_col[i],
                    std::integral_constant<bool, TRB>{});
    };

    // ---- fragments.  Plain: one 16-byte read, K values 8 lg .. 8 lg + 7 of
    // row lc.  Transposed: two reads of K rows 8 lg + 4 h + 0 .. 3; the unit of
    // atom i differs from atom 0's in bits 5-7 of the address, by XOR.
    const uint32_t swz = KTL::key((uint32_t)lc);
    const uint32_t row0 = (uint32_t)(wm * (TM / S::WM)), col0 = (uint32_t)(wn * S::WCOLS);
    constexpr int PA = TRA ? 1 : STEPS, PB = TRB ? 1 : STEPS;
    LdsBases<S::LDS> a_at[PA], b_at[PB];
    const uint32_t key = tr_key((uint32_t)(8 * lg + (lc >> 2)));
    if constexpr (TRA) {
        a_at[0].init((uint32_t)(8 * lg + (lc >> 2)) * (TM * 2) + (((row0 >> 4) ^ key) << 5) +
                     (uint32_t)(lc & 3) * 8);
    } else {
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            a_at[s].init((row0 + (uint32_t)lc) * KTB + (((uint32_t)AT::a_chunk(s, lane, 0) ^ swz) << 4));
    }
    if constexpr (TRB) {
        b_at[0].init((uint32_t)(8 * lg + (lc >> 2)) * (TN * 2) + (((col0 >> 4) ^ key) << 5) +
                     (uint32_t)(lc & 3) * 8);
    } else {
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            b_at[s].init((col0 + (uint32_t)lc) * KTB + (((uint32_t)AT::a_chunk(s, lane, 0) ^ swz) << 4));
    }
    auto tr_frag = [&](const LdsBases<S::LDS>& at, uint32_t c, int i, int pitch)
                       __attribute__((always_inline)) {
        i32x4 v;
        const uint32_t c1 = c + 4u * (uint32_t)pitch;
        const s16x4 lo = lds_read_tr16(
            (lds_s16x4*)(lds + (at.b[c >> 16] ^ ((uint32_t)i << 5)) + (c & 0xFFFFu)));
        const s16x4 hi = lds_read_tr16(
            (lds_s16x4*)(lds + (at.b[c1 >> 16] ^ ((uint32_t)i << 5)) + (c1 & 0xFFFFu)));
        typedef int i32x2 __attribute__((ext_vector_type(2)));
        const i32x2 l2 = __builtin_bit_cast(i32x2, lo), h2 = __builtin_bit_cast(i32x2, hi);
        v[0] = l2[0];
        v[1] = l2[1];
        v[2] = h2[0];
        v[3] = h2[1];
        return v;
    };

    i32x4 af[frag_sets(ST, STEPS)][MR], bf[frag_sets(ST, STEPS)][NR];
    acc_t acc[MR][NR];
#pragma unroll
    for (int mi = 0; mi < MR; ++mi)
#pragma unroll
        for (int j = 0; j < NR; ++j)
            acc[mi][j] = zero_acc<AT>();

    auto read = [&](int stage, int s, int set, int g, int G) __attribute__((always_inline)) {
        constexpr int NF = MR + NR;
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            if (f * G / NF != g)
                continue;
            if (f < NR) {
                if constexpr (TRB)
                    bf[set][f] = tr_frag(b_at[0], (uint32_t)(stage * STAGE + A_BUF + s * 32 * TN * 2), f,
                                         TN * 2);
                else
                    bf[set][f] = *reinterpret_cast<const i32x4*>(
                        lds + b_at[s % PB].at((uint32_t)(stage * STAGE + A_BUF + f * R * KTB)));
            } else {
                const int mi = f - NR;
                if constexpr (TRA)
                    af[set][mi] = tr_frag(a_at[0], (uint32_t)(stage * STAGE + s * 32 * TM * 2), mi, TM * 2);
                else
                    af[set][mi] = *reinterpret_cast<const i32x4*>(
                        lds + a_at[s % PA].at((uint32_t)(stage * STAGE + mi * R * KTB)));
            }
        }
    };
    auto mma = [&](int, int, int set, int g, int G) __attribute__((always_inline)) {
#pragma unroll
        for (int a = 0; a < MR * NR; ++a) {
            if (a * G / (MR * NR) != g)
                continue;
            const int mi = a / NR, j = a % NR;
            acc[mi][j] = mfma_bf16(af[set][mi], bf[set][j], acc[mi][j]);
        }
    };
    k_loop<ST, STEPS, S::LOADS, step_groups(MR * NR)>(nkt, min(nkt, last_full - kt0), load, read, mma);

    // ---- outputs.  Lane l holds, in element e of atom (mi, j), row
    // 16 mi + 4 lg + e of the wave's block and column 16 j + lc.
    if constexpr (ROLE == ROLE_LSE) {
        int* lab = reinterpret_cast<int*>(lds);
        float2* red = reinterpret_cast<float2*>(lds + TM * 4);
        for (int r = tid; r < TM; r += S::THREADS)
            lab[r] = r < rows ? p.rows[m0 + r].label : -1;
        __syncthreads();
        const int col_w = n0 + (int)col0;
#pragma unroll
        for (int mi = 0; mi < MR; ++mi) {
            const int r4 = (int)row0 + mi * R + 4 * lg;
            const i32x4 l4 = *reinterpret_cast<const i32x4*>(lab + r4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float z[NR];
#pragma unroll
                for (int j = 0; j < NR; ++j) {
                    z[j] = acc[mi][j][e] * p.scale;
                    z[j] = col_w + j * R + lc < p.N ? z[j] : -INFINITY;
                }
                // the label's column, in the one lane that holds it
                const uint32_t d = (uint32_t)(l4[e] - (col_w + lc));
                if (d < (uint32_t)(NR * R) && (d & 15u) == 0) {
                    float zl = z[0];
#pragma unroll
                    for (int j = 1; j < NR; ++j)
                        zl = (int)(d >> 4) == j ? z[j] : zl;
#pragma unroll
                    for (int j = 0; j < NR; ++j)
                        z[j] = (int)(d >> 4) == j ? -INFINITY : z[j];
                    p.zlabel[m0 + r4 + e] = zl;
                }
                float m = z[0];
#pragma unroll
                for (int j = 1; j < NR; ++j)
                    m = fmaxf(m, z[j]);
                m = row16_max(m);
                const float ms = m == -INFINITY ? 0.f : m;   // a block of no column, or all -inf
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < NR; ++j)
                    s += exp_diff(z[j], ms);
                s = row16_sum(s);
                if (lc == 0)
                    red[wn * TM + r4 + e] = make_float2(m, s);
            }
        }
        __syncthreads();
        for (int r = tid; r < rows; r += S::THREADS) {
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < WN; ++w)
                m = fmaxf(m, red[w * TM + r].x);
            const float ms = m == -INFINITY ? 0.f : m;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < WN; ++w) {
                const float2 v = red[w * TM + r];
                // an empty block's sum is 0 (exp(-inf)); its maximum stays out
                s += v.x == -INFINITY ? v.y : v.y * exp_diff(v.x, ms);
            }
            p.part[(int64_t)tn * p.ldpart + m0 + r] = make_float2(m, s);
        }
    } else if constexpr (ROLE == ROLE_GRAD) {
        float4* info = reinterpret_cast<float4*>(lds + S::LDS - S::ROWS_LDS);
        for (int r = tid; r < TM; r += S::THREADS)
            info[r] = *reinterpret_cast<const float4*>(p.rows + m0 + min(r, rows - 1));
        __syncthreads();
        const int col_w = n0 + (int)col0;
#pragma unroll
        for (int mi = 0; mi < MR; ++mi)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 ri = info[(int)row0 + mi * R + 4 * lg + e];
                const int label = __float_as_int(ri.w) - p.v0;
#pragma unroll
                for (int j = 0; j < NR; ++j) {
                    const int col = col_w + j * R + lc;
                    const float zz = acc[mi][j][e] * p.scale;
                    const float g = col == label ? ri.z : ri.y * exp_diff(zz, ri.x);
                    acc[mi][j][e] = col < p.N ? g : 0.f;   // columns of no weight row: zero
                }
            }
        GemmArgs c;
        c.C = p.C;
        c.ldc = p.ldc;
        c.N = (int)p.ldc;              // whole tiles: G's pitch is a multiple of the tile
        c.c_vec = 1;
        store_c_tile<DT_BF16, AT, MR, NR, S::CH, S::SROW, S::WCOLS, false>(
            c, acc, lds + wave * (S::CH * R * S::SROW), m0, rows, col_w, (int)row0, lane, 1.f, 1.f);
    } else if constexpr (ROLE == ROLE_DX) {
        float* plane = p.planes + (int64_t)slice * p.plane + (int64_t)m0 * p.ldplane + n0;
        const rsrc_t rp = make_rsrc(plane, (uint32_t)(((int64_t)(rows - 1) * p.ldplane + (p.N - n0)) * 4));
        const uint32_t pitch = (uint32_t)p.ldplane * 4u;
#pragma unroll
        for (int mi = 0; mi < MR; ++mi) {
            uint32_t base[NR];
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                const int col = (int)col0 + j * R + lc;
                base[j] = n0 + col < p.N
                              ? (row0 + (uint32_t)(mi * R + 4 * lg)) * pitch + (uint32_t)col * 4u
                              : kOOB;
            }
            if (!p.first) {
#pragma unroll
                for (int j = 0; j < NR; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float old = __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b32(
                            rp, (int)(base[j] + (uint32_t)e * pitch), 0, 0));
                        acc[mi][j][e] += old;
                    }
            }
#pragma unroll
            for (int j = 0; j < NR; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v = acc[mi][j][e];
                    store4(rp, base[j] + (uint32_t)e * pitch, __float_as_uint(v));
                }
        }
    } else {
        GemmArgs c;
        c.C = p.C;
        c.ldc = p.ldc;
        c.N = p.N;
        c.c_vec = p.c_vec;
        store_c_tile<DT_BF16, AT, MR, NR, S::CH, S::SROW, S::WCOLS, false>(
            c, acc, lds + wave * (S::CH * R * S::SROW), m0, rows, n0 + (int)col0, (int)row0, lane, 1.f,
            1.f);
    }
}

}  // namespace dg
