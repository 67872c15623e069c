// Kernels of the linear head's losses (loss.hip holds the rest and launches
// them).  With z = scale * X W^T over the vocabulary (X [T, D], W [V, D] bf16)
// four products are needed, none of which may leave z in memory:
//
//   ROLE_LSE   z tile of X W^T -> per row and tile column: a reference m and
//              the sum of 2^(z / ln 2 - m) over the columns other than the
//              row's label, the pieces of a log-sum-exp, and the label's z
//              apart.  m is the maximum of z / ln 2 rounded up to an integer:
//              the sums of two sets of columns then join by a power of two,
//              which rounds nothing.
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

// dW of more rows than one tile: rows are in the order of their target's group of
// this many columns, and G's rows end in as many more, the rests of the row's
// targets in that group.
constexpr int kRestCols = 256;

// One kept row: what its gradient needs, in compact row order.
struct RowInfo {
    float lse2;   // lse / ln 2
    float a;      // factor of exp(z - lse): dloss * scale * (1 + 2 z_loss lse)
    float b;      // the gradient at the label's column
    int label;    // column of W, -1: none
};

// K slices of dX.  The workspace holds S planes of T rows; where only n of the
// rows are kept, the same memory holds S T / n planes of n, and further slices
// take the place of the missing tiles (652 rows kept of 6520: the slices chosen
// for 6520 rows left five sixths of the CUs without work).
struct DxSlices {
    int S, T;
    int tm, tiles_n;       // tile rows, tile columns
    int items;             // tiles x S of all T rows
    int most;              // slices of at least 8 k-tiles
    __device__ __forceinline__ int count(int n) const
    {
        const int tiles = (n + tm - 1) / tm * tiles_n;
        const int64_t room = (int64_t)S * T / max(n, 1);
        return max(S, min(most, (int)min(room, (int64_t)(items / max(tiles, 1)))));
    }
};

struct LossArgs {
    const uint8_t* A;      // X compact [n, lda] (LSE, GRAD), G [n, lda] (DX, DW)
    const uint8_t* B;      // W [., ldb] from the piece's first row (LSE, GRAD, DX), X compact (DW)
    int64_t lda_b, ldb_b;  // row pitches in bytes
    const int* n_kept;     // rows of X that take part (device); null (few rows, LSE): n of them
    int n;
    const int64_t* labels; // few rows, LSE: the rows' labels, or with lead non-null the
    const int* lead;       // columns of their largest targets, [n][2]; A is X itself then
    int M, N, K;           // M: DW only (the piece's rows of W); K: not for DW (n)
    int tiles_n;
    DxSlices slices;       // DX
    float scale;
    const RowInfo* rows;
    float2* part;          // LSE: [tiles_n][ldpart] (reference, sum)
    int64_t ldpart;
    float* zlabel;         // LSE: the label's sum over d, with scale's sign; compact rows
    int v0;                // LSE, GRAD: the vocabulary's column of B's first row; DW: of M's
    float* planes;         // DX: [slices][n][ldplane]
    int64_t ldplane;
    int first;             // DX: the first piece writes, later ones add
    uint16_t* C;           // GRAD: G; DW: dW
    int c_cols;            // GRAD: columns of G from C on that may be written (whole tiles)
    int64_t ldc;
    int c_vec;             // DW: 1 C's rows take 16-byte stores, 2 and non-temporal ones
    int w_nt;              // few rows, GRAD and DX: W with the non-temporal hint
    int64_t half_b;        // few rows, GRAD and DW: bytes from G to its second half
    // DW of more rows: G's columns of rests, and the first row of each group
    const uint8_t* rest;
    const int* group;
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
    // After the k-tile stages: RowInfo of the tile's rows, twice (this tile's
    // and the next one's); then, one tile at a time, each wave's block of 16
    // rows of output or the row sums of the wave columns.
    static constexpr int ROWS_AT = ST * STAGE, ROWS_LDS = TM * 16 > 1024 ? TM * 16 : 1024;
    static constexpr int OUT_AT = ROWS_AT + 2 * ROWS_LDS;
    static constexpr int OUT_LDS = WAVES * R * SROW > WN * TM * 8 ? WAVES * R * SROW : WN * TM * 8;
    static constexpr int LDS = OUT_AT + OUT_LDS;
    // workgroups a CU holds
    static constexpr int PER_CU = (160 * 1024 / LDS < 4 * OCC / WAVES || OCC == 1) ? 160 * 1024 / LDS
                                                                                  : 4 * OCC / WAVES;
    static_assert(MR >= 1 && NR >= 1 && MR * WM * R == TM && NR * WN * R == TN, "tile shape");
    static_assert(A_DMA >= 1 && B_DMA >= 1 && A_DMA * 1024 * WAVES == A_BUF &&
                      B_DMA * 1024 * WAVES == B_BUF, "DMA split");
    static_assert(LDS <= 160 * 1024, "LDS budget");
    static_assert(ROWS_LDS <= 1024 * WAVES, "one RowInfo load a wave");
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

// Maximum / sum over the four lanes that share lane % 16, in each of them.
__device__ __forceinline__ float quad_max(float x)
{
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float quad_sum(float x)
{
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

constexpr float kLog2e = 1.44269504088896340736f;

// (reference, sum) pairs of two sets of columns -> of both.  References are
// integers (-inf: a set of no column, or of -inf only, with sum 0 or NaN).
__device__ __forceinline__ float2 lse_merge(float2 a, float2 b)
{
    const float m = fmaxf(a.x, b.x);
    if (m == -INFINITY)
        return make_float2(m, a.y + b.y);
    // 2^(reference - m): differences of integers, far below fp32's range at most
    return make_float2(m, __builtin_amdgcn_ldexpf(a.y, (int)fmaxf(a.x - m, -4096.f)) +
                              __builtin_amdgcn_ldexpf(b.y, (int)fmaxf(b.x - m, -4096.f)));
}

// A wave's (MR 16) x WCOLS block of accumulators as bf16 into rows of C from
// (row0, col_w) on, through its own LDS region, CH atom rows at a time: a lane
// holds four consecutive columns (one 8-byte LDS write) and stores 16-byte
// pieces of rows, or single elements where C's rows do not allow that.  Rows
// past `rows` and columns past N are not stored.  c_vec: 16-byte pieces, 2 with
// the non-temporal hint.
template <int MR, int NR, int CH, int SROW>
__device__ __forceinline__ void store_bf16_block(uint16_t* C, int64_t ldc, int N, int c_vec,
                                                 const f32x4 (&acc)[MR][NR], uint8_t* stage, int m0,
                                                 int rows, int row0, int col_w, int lane)
{
    constexpr int WCOLS = NR * 16, PPR = WCOLS / 8;
    const int lc = lane & 15, lg = lane >> 4;
    const rsrc_t rc = make_rsrc(C + (int64_t)m0 * ldc + col_w,
                                (uint32_t)(((int64_t)(rows - 1) * ldc + max(N - col_w, 0)) * 2));
    const uint32_t pitch = (uint32_t)ldc * 2u;
    static_for<MR / CH>([&](auto cc_c) __attribute__((always_inline)) {
        constexpr int cc = decltype(cc_c)::value;
#pragma unroll
        for (int ml = 0; ml < CH; ++ml)
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                uint2 v;
                const f32x4 a = acc[cc * CH + ml][j];
                const float a0 = a[0], a1 = a[1], a2 = a[2], a3 = a[3];
                v.x = (uint32_t)bf16_rne(a0) | (uint32_t)bf16_rne(a1) << 16;
                v.y = (uint32_t)bf16_rne(a2) | (uint32_t)bf16_rne(a3) << 16;
                *reinterpret_cast<uint2*>(stage + (ml * 16 + lc) * SROW + (j * 16 + 4 * lg) * 2) = v;
            }
        wave_lds_order();
        const int r0 = row0 + cc * CH * 16;
        if (c_vec) {
#pragma unroll
            for (int q0 = 0; q0 < CH * 16 * PPR; q0 += 64) {
                // (past the last piece: the last one again)
                const int q = CH * 16 * PPR % 64 == 0 ? q0 + lane : min(q0 + lane, CH * 16 * PPR - 1);
                const int r = q / PPR, c = q % PPR * 8;
                const i32x4 v = *reinterpret_cast<const i32x4*>(stage + r * SROW + c * 2);
                const uint32_t off = (uint32_t)(r0 + r) * pitch + (uint32_t)c * 2u;
                // N is a multiple of 8 wherever c_vec is given
                if (c_vec == 2)
                    store16_nt(rc, col_w + c < N ? off : kOOB, v);
                else
                    store16(rc, col_w + c < N ? off : kOOB, v);
            }
        } else {
            for (int q = lane; q < CH * 16 * WCOLS; q += 64) {
                const int r = q / WCOLS, c = q % WCOLS;
                if (col_w + c < N)
                    store2(rc, (uint32_t)(r0 + r) * pitch + (uint32_t)c * 2u,
                           *reinterpret_cast<const uint16_t*>(stage + r * SROW + c * 2));
            }
        }
        wave_lds_order();
    });
}

// FEW: few rows (at most one tile of them).
//   LSE   their selection would take longer than what it saves: A is X itself
//         and every row is computed (a row's X reaches its own logits only),
//         labels are read where they are needed, and W, read once, is loaded
//         with the non-temporal hint.
//   GRAD  G is stored in two bf16 halves, the rounded value and the rounded
//         rest (16 bits of it together), and
//   DW    sums both: the product is bound by writing dW, not by its K.
// With more rows the second half's products would take as long as the first's
// again.  Rounding G to bf16 is as large an error as rounding dW itself, over any
// number of rows, as the errors and the products add up alike, and nearly all of it
// comes from the columns that are some row's target, where |dz| is largest.  DW
// takes the rests of those alone (p.rest): rows lie in the order of their target's
// group of 256 columns, so the ones with a target in a tile's columns are a
// range of rows, further k-tiles of the same loop with the rests at the targets and
// zeros elsewhere (3686 rows: 115 k-tiles, and 19 rows a tile on average).  The norm of
// dW's error at 1100 x 11001 x 520 is that of one rounding, and 1.44 times it
// without; gradients and loss of 1024 x 50257 x 512 take 281 us, 276 without, of
// 528 x 11007 x 1024 with half of the rows kept 77, 73.
//   GRAD, DX  load W with the non-temporal hint where it is larger than the
//         Infinity Cache (w_nt), which then cannot hand it from one to the other.
// Workgroup `block` of `blocks`; lds: S::LDS bytes.
template <class S, int ROLE, bool FEW>
__device__ __forceinline__ void loss_product(const LossArgs& p, uint8_t* lds, int block, int blocks)
{
    constexpr bool FEWX = FEW && ROLE == ROLE_LSE;        // X not selected
    constexpr bool HALVES = FEW && ROLE == ROLE_DW, RESTS = !FEW && ROLE == ROLE_DW;
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

    const int n = FEWX ? p.n : *p.n_kept;
    const int M = ROLE == ROLE_DW ? p.M : n;
    const int tiles_m = (M + TM - 1) / TM;
    // A persistent grid: workgroup b takes items b, b + blocks, ...  The grid
    // is sized for every row of X; n may be less.
    const int tiles = tiles_m * p.tiles_n;
    const int nslices = ROLE == ROLE_DX ? p.slices.count(n) : 1;
    const int items = tiles * nslices;
    int item = block;
    if (item >= items)
        return;

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int lc = lane & 15, lg = lane >> 4;

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
    // ---- the item: output tile, K range (elements and k-tiles), operands
    const int K = ROLE == ROLE_DW ? n : p.K;
    const int all_kt = (K + KT - 1) / KT;
    int slice = 0, m0 = 0, n0 = 0, rows = 0;
    int kt0 = 0, nkt = HALVES ? 2 * all_kt : all_kt, kb_end = K * 2, last_full = 0;
    const uint8_t *a_base = nullptr, *b_base = nullptr;
    int64_t a_span = 0, b_span = 0;
    const uint8_t* e_base = nullptr;                 // RESTS: the tile's rows of rests
    int64_t e_span = 0;
    int e_row = 0;
    uint32_t a_bytes = 0, b_bytes = 0;
    auto set_item = [&](int it) __attribute__((always_inline)) {
        // Each XCD a contiguous run of items.  dX: slices outermost, so that the
        // tiles of a slice, which read the same columns of G and rows of W, share
        // an L2 (1024 x 50257 x 512, gradient of X: 129 us against 155 with each
        // slice's tiles spread over the XCDs, which read G four times from memory).
        int t = xcd_remap(it, items), tm, tn;
        if constexpr (ROLE == ROLE_DX) {
            slice = t / tiles;
            t -= slice * tiles;
        }
        tile_raster<DG_GROUP_M>(t, tiles_m, p.tiles_n, tm, tn);
        m0 = tm * TM;
        n0 = tn * TN;
        rows = min(TM, M - m0);
        int k_end = K;
        if constexpr (ROLE == ROLE_DX) {
            const int kt_per = (all_kt + nslices - 1) / nslices;
            kt0 = slice * kt_per;
            const int kt_end = min(all_kt, kt0 + kt_per);
            nkt = max(0, kt_end - kt0);
            k_end = min(K, kt_end * KT);
        }
        kb_end = k_end * 2;                        // bytes of K a plain operand may read
        last_full = kb_end / KTB;
        a_base = TRA ? p.A + (int64_t)m0 * 2 : p.A + (int64_t)m0 * p.lda_b;
        b_base = TRB ? p.B + (int64_t)n0 * 2 : p.B + (int64_t)n0 * p.ldb_b;
        // a transposed operand's bytes from its base to the end of row K - 1
        // (G's rows are padded: its last, partial 16 bytes are read whole)
        if constexpr (TRA)
            a_span = (int64_t)(k_end - 1) * p.lda_b + (int64_t)(p.M - m0 + 7) / 8 * 16;
        else
            a_bytes = (uint32_t)((int64_t)(rows - 1) * p.lda_b + (int64_t)(K + 7) / 8 * 16);
        if constexpr (RESTS) {
            const int v = p.v0 + m0;                   // tiles do not cross groups
            e_row = __builtin_amdgcn_readfirstlane(p.group[v / kRestCols]);
            const int e_rows = __builtin_amdgcn_readfirstlane(p.group[v / kRestCols + 1]) - e_row;
            e_base = p.rest + e_row * p.lda_b + v % kRestCols * 2;
            e_span = (e_rows - 1) * p.lda_b + TM * 2;
            nkt = all_kt + (e_rows + KT - 1) / KT;
        }
        if constexpr (TRB)
            b_span = (int64_t)(k_end - 1) * p.ldb_b + (int64_t)(p.N - n0) * 2;
        else
            b_bytes = (uint32_t)((int64_t)(min(TN, p.N - n0) - 1) * p.ldb_b + (int64_t)K * 2);
    };
    auto rebase = [&](const uint8_t* base, int64_t span, int64_t off) __attribute__((always_inline)) {
        // (in 32-bit halves, which stay in scalar registers: 64-bit compares take
        // vector ones, and the 256 x 256 tile has none left)
        const int64_t left = span - off;
        const int hi = (int)(left >> 32);
        const uint32_t lo = min((uint32_t)left, 0x7FFFFFFFu);
        return make_rsrc(base + off, hi < 0 ? 0u : hi > 0 ? 0x7FFFFFFFu : lo);
    };
    auto load = [&](int kt_local, int stage, int part, int nparts, auto nomask_c)
                    __attribute__((always_inline)) {
        constexpr bool NOMASK = decltype(nomask_c)::value;
        const int kt = kt0 + kt_local;
        const bool mask = kt >= last_full;
        uint8_t* base = lds + stage * STAGE;
        // the second half of G against the same rows of X, or the rests against
        // the rows of the tile's targets (past the last of them: zeros)
        const bool second = (HALVES || RESTS) && kt >= all_kt;
        const int64_t row = (int64_t)(second ? kt - all_kt : kt) * KT;
        const rsrc_t rat =
            TRA ? rebase(RESTS && second ? e_base : a_base + (HALVES && second ? p.half_b : 0),
                         RESTS && second ? e_span : a_span, row * p.lda_b)
                : make_rsrc(a_base, a_bytes);
        const rsrc_t rbt = TRB ? rebase(b_base, b_span, ((RESTS && second ? e_row : 0) + row) * p.ldb_b)
                               : make_rsrc(b_base, b_bytes);
        auto one = [&](rsrc_t r, uint8_t* dst, uint32_t goff, uint32_t col, auto tr, auto nt)
                       __attribute__((always_inline)) {
            uint32_t off = goff, soff = 0;
            if constexpr (decltype(tr)::value) {
            } else if constexpr (NOMASK) {
                soff = (uint32_t)kt * KTB;
            } else {
                off = goff + (uint32_t)kt * KTB;
                if (mask && (int)((uint32_t)kt * KTB + col) >= kb_end)
                    off = kOOB;
            }
            if (decltype(nt)::value && (FEWX || p.w_nt))
                dma16_nt(r, dst, off, soff);
            else
                dma16(r, dst, off, soff);
        };
#pragma unroll
        for (int i = 0; i < A_DMA; ++i)
            if (i % nparts == part)
                one(rat, base + (wave + WAVES * i) * 1024, a_goff[i], a_col[i],
                    std::integral_constant<bool, TRA>{}, std::false_type{});
#pragma unroll
        for (int i = 0; i < B_DMA; ++i)
            if ((A_DMA + i) % nparts == part)
                one(rbt, base + A_BUF + (wave + WAVES * i) * 1024, b_goff[i], b_col[i],
                    std::integral_constant<bool, TRB>{},
                    std::integral_constant<bool, FEW && ROLE != ROLE_DW>{});
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
            acc[mi][j] = mfma_bf16(bf[set][j], af[set][mi], acc[mi][j]);
        }
    };
    // ---- outputs.  The products are formed with the operands exchanged, so
    // that lane l holds, in element e of atom (mi, j), row 16 mi + lc of the
    // wave's block and column 16 j + 4 lg + e: four consecutive columns of one
    // row.  A row's reductions then run inside the lane and over four lanes
    // (with the rows in the elements they took 8 cross-lane steps for every row
    // of 4 values, and the log-sum-exp of a 256 x 256 tile 6 us), and the
    // stores take 8 or 16 bytes a lane.
    auto output = [&](int m0, int n0, int rows, int slice, int parity, bool idle)
                      __attribute__((always_inline)) {
    if (ROLE != ROLE_LSE && idle)
        return;
    // the lane again, as a value of its own: what the outputs derive from it
    // would otherwise be kept in registers through the K loop
    int ol = lane;
    asm volatile("" : "+v"(ol));
    const int lc = ol & 15, lg = ol >> 4;
    const int col_w = n0 + (int)col0;
    [[maybe_unused]] const uint8_t* info = lds + S::ROWS_AT + parity * S::ROWS_LDS;
    uint8_t* out_lds = lds + S::OUT_AT;
    if constexpr (ROLE == ROLE_LSE) {
        [[maybe_unused]] const int* lab = reinterpret_cast<const int*>(info + 12);
        float2* red = reinterpret_cast<float2*>(out_lds);
        // z / ln 2 = acc * c with c >= 0: a negative scale turns acc's sign
        const float c = fabsf(p.scale) * kLog2e;
        if (p.scale < 0.f) {
#pragma unroll
            for (int mi = 0; mi < MR; ++mi)
#pragma unroll
                for (int j = 0; j < NR; ++j)
                    acc[mi][j] = -acc[mi][j];
        }
        auto rows_of = [&](auto full_c) __attribute__((always_inline)) {
            constexpr bool FULL = decltype(full_c)::value;   // every column of the block is in W
#pragma unroll
            for (int mi = 0; mi < MR; ++mi) {
                const int r = (int)row0 + mi * R + lc;
                float x[NR][4];
#pragma unroll
                for (int j = 0; j < NR; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[j][e] = acc[mi][j][e];
                        if (!FULL && col_w + j * R + 4 * lg + e >= p.N)
                            x[j][e] = -INFINITY;
                    }
                // the label's column, in the one lane that holds it
                int label;
                if constexpr (FEWX) {
                    const int64_t at = min(m0 + r, n - 1);
                    const int64_t y = p.lead ? p.lead[2 * at + 1] : p.labels[at];
                    label = y >= 0 && y < (1 << 30) ? (int)y : -1;
                } else {
                    label = lab[4 * r];
                }
                const uint32_t d = (uint32_t)(label - p.v0 - col_w);
                if (d < (uint32_t)(NR * R) && (int)(d >> 2 & 3u) == lg) {
                    float xl = 0.f;
#pragma unroll
                    for (int j = 0; j < NR; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const bool at = d == (uint32_t)(j * R + 4 * lg + e);
                            xl = at ? x[j][e] : xl;
                            x[j][e] = at ? -INFINITY : x[j][e];
                        }
                    p.zlabel[m0 + r] = xl;
                }
                float m = x[0][0];
#pragma unroll
                for (int j = 0; j < NR; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        m = fmaxf(m, x[j][e]);
                m = quad_max(m);
                // no column of it: reference -inf, 0 in its place below.  With
                // scale 0 every column counts the same.
                const bool none = m == -INFINITY;
                m = none ? 0.f : ceilf(m * c);
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < NR; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float t = __builtin_amdgcn_exp2f(fmaf(x[j][e], c, -m));
                        s += p.scale == 0.f && x[j][e] == -INFINITY ? 0.f : t;
                    }
                s = quad_sum(s);
                if (lg == 0)
                    red[wn * TM + r] = make_float2(none ? -INFINITY : m, s);
            }
        };
        if (idle) {
        } else if (col_w + S::WCOLS <= p.N) {
            rows_of(std::true_type{});
        } else {
            rows_of(std::false_type{});
        }
        // LDS only: the next item's loads stay in flight
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(63));
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        for (int r = wave * 64 + ol; r < rows; r += S::THREADS) {
            float2 v = red[r];
#pragma unroll
            for (int w = 1; w < WN; ++w)
                v = lse_merge(v, red[w * TM + r]);
            p.part[(int64_t)(n0 / TN) * p.ldpart + m0 + r] = v;
        }
    } else if constexpr (ROLE == ROLE_GRAD) {
        const float c = p.scale * kLog2e;
        const bool full = col_w + S::WCOLS <= p.N;
#pragma unroll
        for (int mi = 0; mi < MR; ++mi) {
            const float4 ri = reinterpret_cast<const float4*>(info)[(int)row0 + mi * R + lc];
#pragma unroll
            for (int j = 0; j < NR; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[mi][j][e] = ri.y * __builtin_amdgcn_exp2f(fmaf(acc[mi][j][e], c, -ri.x));
            const uint32_t d = (uint32_t)(__float_as_int(ri.w) - p.v0 - col_w);
            if (d < (uint32_t)(NR * R) && (int)(d >> 2 & 3u) == lg) {
#pragma unroll
                for (int j = 0; j < NR; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[mi][j][e] = d == (uint32_t)(j * R + 4 * lg + e) ? ri.z : acc[mi][j][e];
            }
            if (!full) {                       // columns of no weight row: zero
#pragma unroll
                for (int j = 0; j < NR; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[mi][j][e] = col_w + j * R + 4 * lg + e < p.N ? acc[mi][j][e] : 0.f;
            }
        }
        // whole tiles: G's pitch is a multiple of the tile
        store_bf16_block<MR, NR, 1, S::SROW>(p.C, p.ldc, p.c_cols, 1, acc,
                                                 out_lds + wave * (R * S::SROW), m0, rows,
                                                 (int)row0, col_w, ol);
        if (FEW && p.half_b) {
#pragma unroll
            for (int mi = 0; mi < MR; ++mi)
#pragma unroll
                for (int j = 0; j < NR; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float g = acc[mi][j][e];
                        acc[mi][j][e] = g - bf16_to_f32(bf16_rne(g));
                    }
            store_bf16_block<MR, NR, 1, S::SROW>(p.C + p.half_b / 2, p.ldc, p.c_cols, 1, acc,
                                                 out_lds + wave * (R * S::SROW), m0, rows,
                                                 (int)row0, col_w, ol);
        }
    } else if constexpr (ROLE == ROLE_DX) {
        float* plane = p.planes + ((int64_t)slice * n + m0) * p.ldplane + n0;
        const rsrc_t rp = make_rsrc(plane, (uint32_t)(((int64_t)(rows - 1) * p.ldplane + (p.N - n0)) * 4));
        const uint32_t pitch = (uint32_t)p.ldplane * 4u;
#pragma unroll
        for (int mi = 0; mi < MR; ++mi) {
            uint32_t off[NR];
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                const int col = (int)col0 + j * R + 4 * lg;
                off[j] = n0 + col < p.N ? (row0 + (uint32_t)(mi * R + lc)) * pitch + (uint32_t)col * 4u
                                        : kOOB;
            }
            if (!p.first) {
                i32x4 old[NR];
#pragma unroll
                for (int j = 0; j < NR; ++j)
                    old[j] = load16(rp, off[j]);
#pragma unroll
                for (int j = 0; j < NR; ++j)
                    acc[mi][j] += __builtin_bit_cast(f32x4, old[j]);
            }
#pragma unroll
            for (int j = 0; j < NR; ++j)
                store16(rp, off[j], __builtin_bit_cast(i32x4, acc[mi][j]));
        }
    } else {
        // (only the few rows' instance has the non-temporal stores)
        store_bf16_block<MR, NR, 1, S::SROW>(p.C, p.ldc, p.N, FEW ? p.c_vec : p.c_vec & 1, acc,
                                                 out_lds + wave * (R * S::SROW), m0, rows,
                                                 (int)row0, col_w, ol);
    }
    };

    auto nothing = [](int, int, int, int, int) {};

    // The first k-tiles of an item, and its rows' RowInfo (by LDS DMA too, so
    // that nothing waits for it before the first barrier; rows past n: zeros,
    // which reach no row that is kept).
    auto preload = [&](int parity) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < ST - 1; ++t)
            load(t, t, 0, 1, std::false_type{});
        if constexpr ((ROLE == ROLE_LSE && !FEWX) || ROLE == ROLE_GRAD)
            if (wave * 64 < TM)
                dma16(make_rsrc(p.rows + m0, (uint32_t)rows * 16u),
                      lds + S::ROWS_AT + parity * S::ROWS_LDS + wave * 1024, (uint32_t)lane * 16u + (uint32_t)wave * 1024u, 0);
    };
    set_item(item);
    preload(0);
    for (int parity = 0;; parity ^= 1) {
#pragma unroll
        for (int mi = 0; mi < MR; ++mi)
#pragma unroll
            for (int j = 0; j < NR; ++j)
                acc[mi][j] = zero_acc<AT>();
        // Waves whose rows all lie past the last one only load and keep the
        // barriers' count: a row of tiles is half empty on average.
        const bool idle = ROLE != ROLE_DW && (int)row0 >= rows;
        if (!idle)
            k_loop<ST, STEPS, S::LOADS, step_groups(MR * NR), true>(nkt, min(nkt, last_full - kt0),
                                                                    load, read, mma);
        else
            k_loop<ST, STEPS, S::LOADS, step_groups(MR * NR), true>(nkt, min(nkt, last_full - kt0),
                                                                    load, nothing, nothing);
        // the next item's loads go out before this one's outputs
        const int o_m0 = m0, o_n0 = n0, o_rows = rows, o_slice = slice;
        item += blocks;
        const bool more = item < items;
        if (more) {
            set_item(item);
            preload(parity ^ 1);
        }
        output(o_m0, o_n0, o_rows, o_slice, parity, idle);
        if (!more)
            break;
    }
}

template <class S, int ROLE, bool FEW = false>
__global__ __launch_bounds__(S::THREADS, S::OCC) void loss_gemm_kernel(LossArgs p)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
    loss_product<S, ROLE, FEW>(p, lds, (int)blockIdx.x, (int)gridDim.x);
}

// dX and dW of the vocabulary in one launch, the first x_blocks workgroups for
// dX.  They share nothing but the G they read.
template <class S, bool FEW>
__global__ __launch_bounds__(S::THREADS, S::OCC) void loss_pair_kernel(LossArgs x, LossArgs w, int x_blocks)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
    if ((int)blockIdx.x < x_blocks)
        loss_product<S, ROLE_DX, false>(x, lds, (int)blockIdx.x, x_blocks);
    else
        loss_product<S, ROLE_DW, FEW>(w, lds, (int)blockIdx.x - x_blocks, (int)gridDim.x - x_blocks);
}

}  // namespace dg
