// Products of rows that lie sorted by group, each group with a weight of its
// own, and of all rows with one weight beside each group's low-rank pair.
// With rows p of group g at offsets[g] <= p < offsets[g + 1]:
//
//   GROUP_FWD    Y[p] = act(W_g x) * mul[p], x = X[p] or X[order[p] / k]
//   GROUP_DX     dX[p] = sum_n dY[p][n] W_g[n]
//   GROUP_DW     dW_g = sum over its p of dY[p] x^T; zeros for a group of no row
//   GROUP_ADAPT  Y[order[p]] = W x + B_g u[p], u = scale_g A_g x in two bf16
//                halves from the kernel before; the second term as further k-tiles
//
// Operands are taken as they lie in memory and staged in LDS k-tile by k-tile
// (k_loop): one whose contraction axis is contiguous as gemm_ab_kernel stages
// A, the others as rows that gfx950's transposing LDS read turns (dX's W, both
// of dW's; see loss_kernels.hpp).  Rows of X are picked up by the loads
// themselves: every lane of an LDS DMA has an offset of its own, so that rows in
// any order cost what sorted ones cost, and no sorted copy of X is made.
//
// How many rows a group has is known on the device only.  Every workgroup
// turns the offsets into the groups' first tiles (a scan over at most 512
// groups in LDS, under 2 us) and walks a persistent range of tiles; no host
// synchronisation, no table from another launch.
#pragma once

#include "group.hpp"
#include "loss_kernels.hpp"

namespace dg {

// FWD without act and mul is an instance of its own (GATED has them).
enum { GROUP_FWD = 0, GROUP_DX = 1, GROUP_DW = 2, GROUP_ADAPT = 3, GROUP_GATED = 4 };

struct GroupArgs {
    const uint8_t* A;      // X (FWD, ADAPT), dY (DX, DW)
    int64_t lda_b;         // pitches in bytes
    const uint8_t* B;      // W (FWD, DX, ADAPT), sorted X (DW)
    int64_t ldb_b, b_group;// bytes between two groups' W
    const int* offsets;    // [groups + 1]
    int groups;
    int S;                 // sorted rows that the buffers hold
    const int* order;      // FWD: null, A's rows are sorted
    uint32_t k_mul;        // slot -> row of X (divide_by)
    uint32_t a_bytes;      // order given: bytes of X
    int M, N, K;           // M: DW's rows; N: columns of the output; K: not for DW
    int tiles_n;
    uint16_t* C;
    int64_t ldc, c_group;  // c_group: DW, elements between two groups' dW
    int c_vec;             // 16-byte stores of C's rows, 2: non-temporal
    int b_nt;              // B is read once: non-temporal loads
    int act;               // GATED
    const uint16_t* mul;
    int64_t ld_mul;
    int mul_vec;           // mul's rows take 8-byte loads
    const uint8_t* U;      // ADAPT: [S][2][R]
    const uint8_t* LB;     // ADAPT: [groups][N][ldlb]
    int64_t ldlb_b, lb_group;
    int R;
    int units, pack;       // set by the launch, which knows the tile: units of 16 ranks an
                           // adapter, and whether adapters share k-tiles of them
};

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr int kTableLds = ((int)kMaxGroups + 4) * 4 + 64;

// Tile shape: TM x TN outputs, WM x WN waves, ST stages of KTB bytes of K, OCC
// waves per SIMD to leave registers for.
template <int TM_, int TN_, int WM_, int WN_, int ST_, int KTB_, int OCC_>
struct GroupShape {
    static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, ST = ST_, KTB = KTB_, OCC = OCC_;
    static constexpr int R = 16;
    static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
    static constexpr int MR = TM / WM / R, NR = TN / WN / R;
    static constexpr int A_BUF = TM * KTB, B_BUF = TN * KTB, STAGE = A_BUF + B_BUF;
    static constexpr int A_DMA = A_BUF / 1024 / WAVES, B_DMA = B_BUF / 1024 / WAVES;
    static constexpr int LOADS = A_DMA + B_DMA;
    static constexpr int KT = KTB / 2;
    static constexpr int WCOLS = TN / WN;
    static constexpr int SROW = WCOLS * 2 + 16;
    static constexpr int REST_KT = 8;    // DW, see there
    // after the stages: the waves' output blocks, the groups' table
    static constexpr int OUT_AT = ST * STAGE, OUT_LDS = WAVES * R * SROW;
    static constexpr int TABLE_AT = OUT_AT + OUT_LDS;
    static constexpr int TABLE_LDS = kTableLds;
    static constexpr int LDS = TABLE_AT + TABLE_LDS;
    static constexpr int PER_CU = (160 * 1024 / LDS < 4 * OCC / WAVES || OCC == 1) ? 160 * 1024 / LDS
                                                                                  : 4 * OCC / WAVES;
    static_assert(MR >= 1 && NR >= 1 && MR * WM * R == TM && NR * WN * R == TN, "tile shape");
    static_assert(A_DMA >= 1 && B_DMA >= 1 && A_DMA * 1024 * WAVES == A_BUF &&
                      B_DMA * 1024 * WAVES == B_BUF, "DMA split");
    static_assert(LDS <= 160 * 1024, "LDS budget");
};

// The groups' table in LDS.  first(i): where entry i begins, counted in units of
// `unit` rows (rounded up per group, and `more` of them each); first(count): the end.  With COMPACT only
// groups that have rows are entries, id(i) says which group entry i is, and the
// unit is a row; else entry i is group i.  Offsets that are not ascending or lie
// outside [0, S] are taken as the nearest that are, so that no index derived
// from them leaves the buffers.
struct GroupTable {
    int* entry;            // [kMaxGroups + 1], COMPACT: first << 10 | id
    int* sums;             // [16]
    int count, shift;
    __device__ __forceinline__ void at(uint8_t* lds)
    {
        entry = reinterpret_cast<int*>(lds);
        sums = entry + kMaxGroups + 4;
    }
    __device__ __forceinline__ int first(int i) const { return (int)((uint32_t)entry[i] >> shift); }
    __device__ __forceinline__ int id(int i) const { return entry[i] & 1023; }
};

// Rows of group g: [lo, hi).
__device__ __forceinline__ int2 group_rows(const int* offsets, int g, int S)
{
    const int lo = min(max(offsets[g], 0), S);
    return make_int2(lo, min(max(offsets[g + 1], lo), S));
}

template <int THREADS, bool COMPACT>
__device__ __forceinline__ void build_table(GroupTable& t, const int* offsets, int groups, int S, int unit, int more)
{
    constexpr int WAVES = THREADS / 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int each = (groups + THREADS - 1) / THREADS;
    const int g0 = min(groups, tid * each), g1 = min(groups, g0 + each);
    auto units = [&](int g) {
        const int2 r = group_rows(offsets, g, S);
        return COMPACT ? (int)(r.y > r.x) : (r.y - r.x + unit - 1) / unit + more;
    };
    int n = 0;
    for (int g = g0; g < g1; ++g)
        n += units(g);
    int upto = n;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int y = __shfl_up(upto, d);
        upto += lane >= d ? y : 0;
    }
    if (lane == 63)
        t.sums[wave] = upto;
    __syncthreads();
    int at = upto - n, all = 0;
    for (int w = 0; w < WAVES; ++w) {
        at += w < wave ? t.sums[w] : 0;
        all += t.sums[w];
    }
    for (int g = g0; g < g1; ++g) {
        if constexpr (COMPACT) {
            const int2 r = group_rows(offsets, g, S);
            if (r.y > r.x) {
                t.entry[at] = r.x << 10 | g;
                ++at;
                // (an entry ends where the next begins, the last at its own end)
                if (at == all)
                    t.entry[all] = r.y << 10;
            }
        } else {
            t.entry[g] = at;
            at += units(g);
        }
    }
    if (!COMPACT && tid == 0)
        t.entry[groups] = all;
    t.shift = COMPACT ? 10 : 0;
    t.count = COMPACT ? all : groups;
    __syncthreads();
}

// The last entry i with first(i) <= x, for first(0) <= x < first(count) (the
// same x in every lane).  Two ballots over 64 entries at most.
__device__ __forceinline__ int find_entry(const GroupTable& t, int x, int lane)
{
    const int step = t.count / 64 + 1;
    int i = min(lane * step, t.count);
    const int block = __popcll(__ballot(lane * step <= t.count && t.first(i) <= x)) - 1;
    if (step == 1)
        return block;
    i = min(block * step + lane, t.count);
    return block * step + __popcll(__ballot(lane < step && block * step + lane <= t.count && t.first(i) <= x)) - 1;
}

// A wave's block of accumulators as bf16 into rows of C, through its own LDS
// region, 16 rows at a time: a lane holds four consecutive columns of one row
// (one 8-byte LDS write) and stores 16-byte pieces of rows, or single elements
// where C's rows do not allow that.  finish(mi, j, r, col, v) turns the four sums of
// block (mi, j), row r of the tile, columns col .. col + 3, into outputs; row_of(r) is
// C's row, or negative: not stored.
template <int MR, int NR, int SROW, class Finish, class RowOf>
__device__ __forceinline__ void store_group_block(uint16_t* C, int64_t ldc, int N, int c_vec,
                                                  const f32x4 (&acc)[MR][NR], uint8_t* stage, int row0,
                                                  int col_w, int lane, Finish&& finish, RowOf&& row_of)
{
    constexpr int WCOLS = NR * 16, PPR = WCOLS / 8;
    const int lc = lane & 15, lg = lane >> 4;
    static_for<MR>([&](auto mi_c) __attribute__((always_inline)) {
        constexpr int mi = decltype(mi_c)::value;
        const int r0 = row0 + mi * 16;
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            f32x4 v = acc[mi][j];
            finish(mi, j, r0 + lc, col_w + j * 16 + 4 * lg, v);
            uint2 o;
            const float v0 = v[0], v1 = v[1], v2 = v[2], v3 = v[3];
            o.x = (uint32_t)bf16_rne(v0) | (uint32_t)bf16_rne(v1) << 16;
            o.y = (uint32_t)bf16_rne(v2) | (uint32_t)bf16_rne(v3) << 16;
            *reinterpret_cast<uint2*>(stage + lc * SROW + (j * 16 + 4 * lg) * 2) = o;
        }
        wave_lds_order();
        if (c_vec) {
#pragma unroll
            for (int q0 = 0; q0 < 16 * PPR; q0 += 64) {
                const int q = q0 + lane;
                const int r = q / PPR, c = q % PPR * 8;
                const int to = q < 16 * PPR ? row_of(r0 + r) : -1;
                if (to >= 0 && col_w + c < N) {
                    const i32x4 v = *reinterpret_cast<const i32x4*>(stage + r * SROW + c * 2);
                    *reinterpret_cast<i32x4*>(C + to * ldc + col_w + c) = v;
                }
            }
        } else {
            for (int q = lane; q < 16 * WCOLS; q += 64) {
                const int r = q / WCOLS, c = q % WCOLS;
                const int to = row_of(r0 + r);
                if (to >= 0 && col_w + c < N)
                    C[to * ldc + col_w + c] = *reinterpret_cast<const uint16_t*>(stage + r * SROW + c * 2);
            }
        }
        wave_lds_order();
    });
}

__device__ __forceinline__ uint2 load8(rsrc_t r, uint32_t off)
{
    return __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, 0, 0));
}

__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p)
{
    const uint64_t v = (uint64_t)p;
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
    return (const uint8_t*)((uint64_t)hi << 32 | lo);
}

// The kernel's arguments, read again from memory where they are used: as values of
// the start they would stay in scalar registers through the K loop, which has none
// left (the 256 x 256 tiles spilled 90 of them to vector registers, and those to
// memory inside the loop).
typedef const __attribute__((address_space(4))) GroupArgs* KernelArgs;
__device__ __forceinline__ KernelArgs kernel_args()
{
    KernelArgs a = (KernelArgs)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(a));
    return a;
}

// k_loop for items whose k-tiles follow one another without a break: k-tiles 0 ..
// ST - 2 are in flight at the start, and load(kt ..) for kt from `end` (a multiple of
// ST) on loads the next item's, which are left in flight at the end; nothing is
// drained.  Waits count what was issued behind a k-tile's loads (vector memory
// operations of a wave complete in the order of their issue): the k-tiles after it,
// and with `stored` at least STORES stores of the item before, issued between the
// last of its loads and this loop.
template <int ST, int LOADS, int G, int STORES, class Load, class Read, class Mma>
__device__ __forceinline__ void k_stream(int end, bool stored, Load& load, Read& read, Mma& mma)
{
    constexpr int NS = frag_sets(ST, 1);
    static_assert((ST - 2) * LOADS + STORES <= 63, "pipeline depth vs vmcnt");
    if (stored)
        DG_STAGE_BARRIER((ST - 2) * LOADS + STORES);
    else
        DG_STAGE_BARRIER((ST - 2) * LOADS);
#pragma unroll
    for (int g = 0; g < G; ++g)
        read(0, 0, 0, g, G);
    auto phase = [&](int t, auto sc, auto extra) __attribute__((always_inline)) {
        constexpr int si = decltype(sc)::value;
        DG_STAGE_BARRIER((ST - 3) * LOADS + decltype(extra)::value);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            read((si + 1) % ST, 0, (si + 1) % NS, g, G);
            mma(si, 0, si % NS, g, G);
            load(t + ST - 1, (si + ST - 1) % ST, g, G, std::false_type{});
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    int kt = 0;
    if (stored) {
        // the k-tiles loaded before the stores
        static_for<ST>([&](auto i) __attribute__((always_inline)) {
            constexpr int I = decltype(i)::value;
            phase(I, i, std::integral_constant<int, I < ST - 2 ? STORES : 0>{});
        });
        kt = ST;
    }
    for (; kt < end; kt += ST)
        static_for<ST>([&](auto i) __attribute__((always_inline)) {
            phase(kt + decltype(i)::value, i, std::integral_constant<int, 0>{});
        });
}

template <class S, int ROLE>
__global__ __launch_bounds__(S::THREADS, S::OCC) void group_gemm_kernel(GroupArgs p)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
    using AT = Atom<DT_BF16, 16>;
    using KTL = KTile<S::KTB>;
    using acc_t = AT::acc_t;
    constexpr int TM = S::TM, TN = S::TN, WN = S::WN, R = 16, KTB = S::KTB, KT = S::KT;
    constexpr int MR = S::MR, NR = S::NR, A_DMA = S::A_DMA, B_DMA = S::B_DMA;
    constexpr int A_BUF = S::A_BUF, STAGE = S::STAGE, WAVES = S::WAVES, ST = S::ST;
    constexpr int STEPS = KTB / 64, CHUNKS = KTB / 16;
    constexpr bool TRA = ROLE == GROUP_DW, TRB = ROLE == GROUP_DX || ROLE == GROUP_DW;
    constexpr bool STREAM = ROLE == GROUP_DW;
    constexpr bool ADAPT = ROLE == GROUP_ADAPT, GATHER = ROLE == GROUP_FWD || ROLE == GROUP_GATED || ADAPT;
    static_assert(!TRA || TM >= 128, "a transposed operand's unit key needs 8 units a row");
    static_assert(!TRB || TN >= 128, "a transposed operand's unit key needs 8 units a row");

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int lc = lane & 15, lg = lane >> 4;

    // ---- the tiles
    GroupTable table;
    table.at(lds + S::TABLE_AT);
    build_table<S::THREADS, ADAPT>(table, p.offsets, p.groups, p.S, ROLE == GROUP_DW ? KT : TM,
                                   ROLE == GROUP_DW ? S::REST_KT : 0);
    const int w_tiles = ROLE == GROUP_DW ? (p.M + TM - 1) / TM * p.tiles_n : 0;   // DW: tiles of a group
    // (offsets that are not ascending may claim more rows than there are: nothing is done)
    const int items = __builtin_amdgcn_readfirstlane(
        ROLE == GROUP_DW ? p.groups * w_tiles
        : ADAPT          ? (p.S + TM - 1) / TM * p.tiles_n
        : table.first(p.groups) <= p.S / TM + p.groups ? table.first(p.groups) * p.tiles_n : 0);
    // DW: a tile takes as long as its group has rows.  Each XCD has a run of tiles
    // of the same cost, counted in k-tiles (with REST_KT for a tile's start and its
    // output), which its workgroups take in turn.  (Items b, b + G, ... as for the
    // others gave an XCD one group: 8 groups of 342 to 2185 rows, 8192 in all, of 4096 x
    // 4096 took 419 us where equal groups took 262; a run of equal cost for each
    // workgroup 337, but equal groups 313, as tiles that share operands are apart.)
    int item = (int)blockIdx.x, end = items, step = (int)gridDim.x;
    if constexpr (ROLE == GROUP_DW) {
        const int parts = step % 8 == 0 ? 8 : 1;
        const int64_t all = (int64_t)__builtin_amdgcn_readfirstlane(table.first(p.groups)) * w_tiles;
        auto start = [&](int i) __attribute__((always_inline)) {
            if (i >= parts)
                return items;
            const int64_t x = all / parts * i + all % parts * i / parts;      // i / parts of all
            const int g = __builtin_amdgcn_readfirstlane(find_entry(table, (int)(x / w_tiles), lane));
            const int first = __builtin_amdgcn_readfirstlane(table.first(g));
            const int cost = __builtin_amdgcn_readfirstlane(table.first(g + 1)) - first;
            return g * w_tiles + (int)((x - (int64_t)first * w_tiles + cost - 1) / cost);
        };
        end = start(item % parts + 1);
        item = start(item % parts) + item / parts;
        step /= parts;
    }
    if (item >= end)
        return;

    // ---- loads.  Plain operand: rows of K, KTB bytes a k-tile, chunk c of row
    // r at c ^ key(r); rows past the bound read zero, chunks past K go out of
    // range.  Transposed operand: the k-tile's KT rows, the descriptor rebased
    // to them, rows past K read zero; columns past the matrix hold other rows'
    // values and only reach outputs that are not stored.
    // Chunk i of a wave lies A_ROWS i (B_ROWS i) rows further: a multiple of 16, so
    // that the swizzles are the first chunk's.  For a plain operand one offset in a
    // vector register serves all, with the descriptor's base moved; rows picked up
    // by order, and those of a transposed operand, whose descriptor moves with the
    // k-tiles, have an offset each.  (With offsets for all, the 256 x 256 tiles
    // spilled them into the K loop.)
    constexpr int A_ROWS = WAVES * 1024 / (TRA ? TM * 2 : KTB), B_ROWS = WAVES * 1024 / (TRB ? TN * 2 : KTB);
    static_assert(A_ROWS % 16 == 0 && B_ROWS % 16 == 0, "swizzles repeat");
    constexpr int A_OFFS = GATHER || TRA ? A_DMA : 1, B_OFFS = TRB ? B_DMA : 1;
    uint32_t a_goff[A_OFFS], b_goff[B_OFFS], a_col = 0, b_col = 0;
    auto tr_offset = [&](int width, int64_t ld_b) __attribute__((always_inline)) {
        const uint32_t at = (uint32_t)wave * 1024u + (uint32_t)lane * 16u;
        const uint32_t r = at / (uint32_t)(width * 2), c = at % (uint32_t)(width * 2) / 16;
        return r * (uint32_t)ld_b + ((c ^ (tr_key(r) << 1)) << 4);
    };
    if constexpr (TRA) {
        a_goff[0] = tr_offset(TM, p.lda_b);
#pragma unroll
        for (int i = 1; i < A_OFFS; ++i)
            a_goff[i] = a_goff[0] + (uint32_t)(i * A_ROWS) * (uint32_t)p.lda_b;
    } else {
        const ADma d = a_dma_lane<KTB>(wave, lane, p.lda_b);
        a_goff[0] = d.goff;
        a_col = d.col;
#pragma unroll
        for (int i = 1; i < A_OFFS; ++i)
            a_goff[i] = a_goff[0] + (uint32_t)(i * A_ROWS) * (uint32_t)p.lda_b;
    }
    if constexpr (TRB) {
        b_goff[0] = tr_offset(TN, p.ldb_b);
#pragma unroll
        for (int i = 1; i < B_OFFS; ++i)
            b_goff[i] = b_goff[0] + (uint32_t)(i * B_ROWS) * (uint32_t)p.ldb_b;
    } else {
        const ADma d = a_dma_lane<KTB>(wave, lane, p.ldb_b);
        b_goff[0] = d.goff;
        b_col = d.col;
    }
    // (as values of their own: where they are the low halves of 64-bit products, the
    // compiler keeps both halves)
#pragma unroll
    for (int i = 0; i < A_OFFS; ++i)
        asm volatile("" : "+v"(a_goff[i]));
#pragma unroll
    for (int i = 0; i < B_OFFS; ++i)
        asm volatile("" : "+v"(b_goff[i]));
    // ---- the item: its group, output tile, K range, operands
    const int plain_kt = (p.K + KT - 1) / KT;          // not DW
    int group = 0, m0 = 0, n0 = 0, rows = 0, nkt = plain_kt;
    const int kb_end = ROLE == GROUP_DW ? 0 : p.K * 2;
    const int last_full = ROLE == GROUP_DW ? 0 : kb_end / KTB;
    const uint8_t *a_base = nullptr, *b_base = nullptr;
    // plain: bytes of the tile's rows; transposed: bytes of the last k-tile, and of those
    // before it
    int a_span = 0, b_span = 0, a_full = 0, b_full = 0;
    const int a_step = KT * (int)p.lda_b, b_step = KT * (int)p.ldb_b;         // TRA, TRB
    const int a_rows = A_ROWS * (int)p.lda_b, b_rows = B_ROWS * (int)p.ldb_b;
    uint32_t a_bytes = 0;                                                     // GATHER
    // STREAM: what the loads turn to behind the present item's k-tiles
    struct Operands {
        const uint8_t *a, *b;
        int a_span, b_span, a_full, b_full, nkt;
    };
    Operands next = {nullptr, nullptr, 0, 0, 0, 0, 0};
    int stream_end = -1, k_off = 0;
    // ADAPT: the first of the table's entries that the tile's rows touch, and all their
    // units of 16 ranks
    int units = 0, entry0 = 0;
    auto set_item = [&](int it) __attribute__((always_inline)) {
        const KernelArgs q = kernel_args();
        int t = ROLE == GROUP_DW ? it : xcd_remap(it, items), tm, tn;

        int last_row;
        if constexpr (ROLE == GROUP_DW) {
            group = t / w_tiles;
            tile_raster<DG_GROUP_M>(t - group * w_tiles, w_tiles / q->tiles_n, q->tiles_n, tm, tn);
            const int2 r = group_rows(q->offsets, group, q->S);
            const int lo = __builtin_amdgcn_readfirstlane(r.x);
            const int n = __builtin_amdgcn_readfirstlane(r.y) - lo;
            m0 = tm * TM;
            rows = min(TM, q->M - m0);
            nkt = (n + KT - 1) / KT;
            a_base = q->A + lo * q->lda_b + (int64_t)m0 * 2;
            a_span = (n - 1) % KT * (int)q->lda_b + (q->M - m0) * 2;
            a_full = a_step - (int)q->lda_b + (q->M - m0) * 2;
            b_base = q->B + lo * q->ldb_b;
            b_span = (n - 1) % KT * (int)q->ldb_b;
            last_row = 0;
        } else if constexpr (ADAPT) {
            tile_raster<DG_GROUP_M>(t, items / q->tiles_n, q->tiles_n, tm, tn);
            m0 = tm * TM;
            last_row = q->S;
        } else {
            group = __builtin_amdgcn_readfirstlane(find_entry(table, t / q->tiles_n, lane));
            const int first = __builtin_amdgcn_readfirstlane(table.first(group));
            const int tiles = __builtin_amdgcn_readfirstlane(table.first(group + 1)) - first;
            const int2 r = group_rows(q->offsets, group, q->S);
            tile_raster<8>(t - first * q->tiles_n, tiles, q->tiles_n, tm, tn);
            m0 = __builtin_amdgcn_readfirstlane(r.x) + tm * TM;
            last_row = __builtin_amdgcn_readfirstlane(r.y);
        }
        n0 = tn * TN;
        if constexpr (ROLE != GROUP_DW) {
            rows = min(TM, last_row - m0);
            a_base = q->A + (int64_t)m0 * q->lda_b;
            a_span = (rows - 1) * (int)q->lda_b + q->K * 2;
            a_bytes = (uint32_t)a_span;
            b_base = q->B + group * q->b_group;
        }
        if constexpr (GATHER) {
            if (ADAPT || q->order) {
                a_base = q->A;
                a_bytes = q->a_bytes;
#pragma unroll
                for (int i = 0; i < A_DMA; ++i) {
                    const int r = KTL::ROWS_PER_LOAD * (wave + WAVES * i) + lane / CHUNKS;
                    const uint32_t slot = (uint32_t)q->order[m0 + min(r, rows - 1)];
                    const uint32_t row = q->k_mul ? __umulhi(slot, q->k_mul) : slot;
                    a_goff[i] = r < rows && slot < (uint32_t)q->S ? row * (uint32_t)q->lda_b + a_col : kOOB;
                }
            }
        }
        if constexpr (ADAPT) {
            entry0 = 0;
            int over = 0;
            if (table.count > 0 && m0 < table.first(table.count)) {
                const int end = min(m0 + rows, table.first(table.count));
                entry0 = max(0, find_entry(table, max(m0, table.first(0)), lane));
                over = end > table.first(0) ? find_entry(table, end - 1, lane) - entry0 + 1 : 0;
            }
            entry0 = __builtin_amdgcn_readfirstlane(entry0);
            over = __builtin_amdgcn_readfirstlane(over);
            units = over * q->units;
        }
        if constexpr (TRB) {
            b_base += (int64_t)n0 * 2;
            if constexpr (ROLE == GROUP_DX)
                b_span = (q->K - 1) % KT * (int)q->ldb_b;
            b_span += (q->N - n0) * 2;
            b_full = b_step - (int)q->ldb_b + (q->N - n0) * 2;
        } else {
            b_base += (int64_t)n0 * q->ldb_b;
            b_span = (min(TN, q->N - n0) - 1) * (int)q->ldb_b + q->K * 2;
        }
        // Said to be uniform, which they are: where the compiler computed one of
        // them in vector registers, every load would run a loop over its values.
        a_base = uniform(a_base);
        b_base = uniform(b_base);
        a_bytes = (uint32_t)__builtin_amdgcn_readfirstlane((int)a_bytes);
        a_span = __builtin_amdgcn_readfirstlane(a_span);
        b_span = __builtin_amdgcn_readfirstlane(b_span);
        a_full = __builtin_amdgcn_readfirstlane(a_full);
        b_full = __builtin_amdgcn_readfirstlane(b_full);
        if constexpr (ROLE == GROUP_DW)
            nkt = __builtin_amdgcn_readfirstlane(nkt);
    };
    // Rows i rows_b bytes behind the tile's first; or the rows of k-tile kt, none behind
    // the last one.
    auto plain_rsrc = [&](const uint8_t* base, int span, int behind) __attribute__((always_inline)) {
        return make_rsrc(base + behind, (uint32_t)max(span - behind, 0));
    };
    auto tr_rsrc = [&](const uint8_t* base, int span, int full, int kt) __attribute__((always_inline)) {
        return make_rsrc(base, (uint32_t)(kt + 1 < nkt ? full : kt < nkt ? span : 0));
    };
    auto load = [&](int kt, int stage, int part, int nparts, auto nomask_c) __attribute__((always_inline)) {
        constexpr bool NOMASK = decltype(nomask_c)::value;
        const bool mask = kt >= last_full;
        uint8_t* base = lds + stage * STAGE;
        if constexpr (STREAM) {
            if (part == 0 && kt == stream_end) {           // the next item's k-tiles
                a_base = next.a;
                b_base = next.b;
                a_span = next.a_span;
                b_span = next.b_span;
                a_full = next.a_full;
                b_full = next.b_full;
                nkt = next.nkt;
                k_off = stream_end;
            }
        }
        auto one = [&](rsrc_t r, uint8_t* dst, uint32_t goff, uint32_t col, auto tr, int nt)
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
            if (nt)
                dma16_nt(r, dst, off, soff);
            else
                dma16(r, dst, off, soff);
        };
#pragma unroll
        for (int i = 0; i < A_DMA; ++i)
            if (i % nparts == part)
                one(GATHER ? make_rsrc(a_base, a_bytes)
                    : TRA  ? tr_rsrc(a_base, a_span, a_full, kt - k_off)
                           : plain_rsrc(a_base, a_span, i * a_rows),
                    base + (wave + WAVES * i) * 1024, a_goff[i % A_OFFS], a_col,
                    std::integral_constant<bool, TRA>{}, 0);
#pragma unroll
        for (int i = 0; i < B_DMA; ++i)
            if ((A_DMA + i) % nparts == part)
                one(TRB ? tr_rsrc(b_base, b_span, b_full, kt - k_off) : plain_rsrc(b_base, b_span, i * b_rows),
                    base + A_BUF + (wave + WAVES * i) * 1024, b_goff[i % B_OFFS], b_col,
                    std::integral_constant<bool, TRB>{}, TM <= 64 && !TRA ? p.b_nt : 0);
        // a transposed operand's base goes on with the k-tiles (part by part, then
        // tile by tile: load is called in that order)
        if (part == nparts - 1) {
            if constexpr (TRA)
                a_base += a_step;
            if constexpr (TRB)
                b_base += b_step;
        }
    };

    // ---- fragments, as in loss_product
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
        // (formed at the read: hoisted out of the K loop, the 12 fragments' addresses
        // in two halves of LDS took 24 registers and others were spilled for them)
        uint32_t x = at.b[c >> 16], y = at.b[c1 >> 16];
        asm volatile("" : "+v"(x));
        if (c1 >> 16 != c >> 16)
            asm volatile("" : "+v"(y));
        else
            y = x;
        const s16x4 lo = lds_read_tr16((lds_s16x4*)(lds + (x ^ ((uint32_t)i << 5)) + (c & 0xFFFFu)));
        const s16x4 hi = lds_read_tr16((lds_s16x4*)(lds + (y ^ ((uint32_t)i << 5)) + (c1 & 0xFFFFu)));
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
    // operands exchanged: a lane holds four consecutive columns of one row
    auto mma = [&](int, int, int set, int g, int G) __attribute__((always_inline)) {
#pragma unroll
        for (int a = 0; a < MR * NR; ++a) {
            if (a * G / (MR * NR) != g)
                continue;
            const int mi = a / NR, j = a % NR;
            acc[mi][j] = mfma_bf16(bf[set][j], af[set][mi], acc[mi][j]);
        }
    };
    // GATED: the multipliers of blocks of 16 rows, AHEAD of them on their way, the first
    // ones before the next item's loads (39200 rows of 2048 x 512 with SiLU: 144 us, 189
    // where they were read as they were used, one block after the other).
    constexpr bool MUL = ROLE == GROUP_GATED;
    constexpr int AHEAD = MR < 2 ? MR : 2;
    uint2 mulv[MUL ? AHEAD + 1 : 1][MUL ? NR : 1];
    auto load_mul = [&](int mi, int m0, int n0, int rows) __attribute__((always_inline)) {
        const KernelArgs q = kernel_args();
        int ol = lane;
        asm volatile("" : "+v"(ol));
        const rsrc_t r = make_rsrc(uniform(reinterpret_cast<const uint8_t*>(q->mul + (int64_t)m0 * q->ld_mul)),
                                   (uint32_t)((rows - 1) * (int)q->ld_mul + q->N) * 2u);
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            const int col = n0 + (int)col0 + j * R + 4 * (ol >> 4);
            const int at = ((int)row0 + mi * R + (ol & 15)) * (int)q->ld_mul + col;
            mulv[mi % (AHEAD + 1)][j] = load8(r, col < q->N ? (uint32_t)at * 2u : kOOB);
        }
    };
    auto output = [&](int group, int m0, int n0, int rows) __attribute__((always_inline)) {
        const KernelArgs q = kernel_args();
        // the lane again, as a value of its own, so that what the outputs derive
        // from it is not kept in registers through the K loop
        int ol = lane;
        asm volatile("" : "+v"(ol));
        const int col_w = n0 + (int)col0;
        uint8_t* stage = lds + S::OUT_AT + wave * (R * S::SROW);
        if constexpr (ADAPT) {
            store_group_block<MR, NR, S::SROW>(
                q->C, q->ldc, q->N, q->c_vec, acc, stage, (int)row0, col_w, ol,
                [](int, int, int, int, f32x4&) {},
                [&](int r) __attribute__((always_inline)) {
                    const int to = r < rows ? q->order[m0 + r] : -1;
                    return to < q->S ? to : -1;
                });
        } else if constexpr (ROLE == GROUP_GATED) {
            auto gated = [&](auto cls, auto vec) __attribute__((always_inline)) {
                constexpr bool VEC = decltype(vec)::value;
                store_group_block<MR, NR, S::SROW>(
                    q->C + (int64_t)m0 * q->ldc, q->ldc, q->N, q->c_vec, acc, stage, (int)row0, col_w, ol,
                    [&](int mi, int j, int r, int col, f32x4& v) __attribute__((always_inline)) {
                        if (VEC && j == 0 && mi + AHEAD < MR)
                            load_mul(mi + AHEAD, m0, n0, rows);
                        float f[4] = {1.f, 1.f, 1.f, 1.f};
                        if constexpr (VEC) {
                            const uint2 u = mulv[mi % (AHEAD + 1)][j];
                            f[0] = __uint_as_float(u.x << 16);
                            f[1] = __uint_as_float(u.x & 0xFFFF0000u);
                            f[2] = __uint_as_float(u.y << 16);
                            f[3] = __uint_as_float(u.y & 0xFFFF0000u);
                        } else if (q->mul && r < rows && col < q->N) {
                            const uint16_t* from = q->mul + (int64_t)(m0 + r) * q->ld_mul + col;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                f[e] = bf16_to_f32(from[min(e, q->N - 1 - col)]);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float a = activate_c<decltype(cls)::value>(q->act, v[e]);
                            v[e] = VEC || q->mul ? a * f[e] : a;
                        }
                    },
                    [&](int r) __attribute__((always_inline)) { return r < rows ? r : -1; });
            };
            auto activated = [&](auto vec) __attribute__((always_inline)) {
                switch (act_class(q->act)) {
                case 1:
                    gated(std::integral_constant<int, 1>{}, vec);
                    break;
                case 2:
                    gated(std::integral_constant<int, 2>{}, vec);
                    break;
                default:
                    gated(std::integral_constant<int, 0>{}, vec);
                }
            };
            if (q->mul_vec)
                activated(std::true_type{});
            else
                activated(std::false_type{});
        } else {
            store_bf16_block<MR, NR, 1, S::SROW>(q->C + group * q->c_group, q->ldc, q->N, q->c_vec, acc, stage,
                                                 m0, rows, (int)row0, col_w, ol);
        }
    };

    // (but DW:) Round r of the grid takes items r G .. r G + G - 1, rotated by 8 r: a group's
    // last, partly filled row of tiles comes up every few items, and without the
    // rotation the same workgroups would get it in every round.  (8: an XCD's
    // workgroups keep to its run of tiles.)
    int round = 0;
    auto next_item = [&]() __attribute__((always_inline)) {
        if constexpr (ROLE == GROUP_DW)
            return (item += step) < end;
        const int G = (int)gridDim.x;
        ++round;
        const int left = items - round * G;
        if (left <= 0)
            return false;
        if (left >= G && G % 8 == 0) {
            item = round * G + ((int)blockIdx.x + 8 * round) % G;
            return true;
        }
        item = round * G + (int)blockIdx.x;
        return item < items;
    };
    auto nothing = [](int, int, int, int, int) {};
    auto preload = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < ST - 1; ++t)
            load(t, t, 0, 1, std::false_type{});
    };
    if constexpr (STREAM) {
        // The k-tiles of all items in one stream: while the last ones of an item are
        // multiplied the first ones of the next are on their way, and its own loop
        // begins without a wait (8192 rows in 32 equal groups of 1024 x 2048, 8 k-tiles a
        // tile: 256 x 128 tiles 84 -> 76 us, 128 x 128 79 -> 74).
        static_assert(STEPS == 1 && ST >= 3);
        constexpr int STORES = MR * (16 * (S::WCOLS / 8) / 64);       // of a wave's 16-byte stores
        bool stored = false;
        set_item(item);
        preload();
        for (;;) {
            const int o_group = group, o_m0 = m0, o_n0 = n0, o_rows = rows;
            const Operands here = {a_base, b_base, a_span, b_span, a_full, b_full, nkt};
            const bool more = next_item();
            stream_end = max(1, (nkt + ST - 1) / ST) * ST;
            if (more)
                set_item(item);
            next = Operands{a_base, b_base, a_span, b_span, a_full, b_full, more ? nkt : 0};
            a_base = here.a;
            b_base = here.b;
            a_span = here.a_span;
            b_span = here.b_span;
            a_full = here.a_full;
            b_full = here.b_full;
            nkt = here.nkt;
            k_off = 0;
#pragma unroll
            for (int mi = 0; mi < MR; ++mi)
#pragma unroll
                for (int j = 0; j < NR; ++j)
                    acc[mi][j] = zero_acc<AT>();
            k_stream<ST, S::LOADS, step_groups(MR * NR), STORES>(stream_end, stored, load, read, mma);
            output(o_group, o_m0, o_n0, o_rows);
            if (!more)
                break;
            stored = p.c_vec != 0;
        }
        // (loads of no item are still on their way into LDS)
        __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
        return;
    }
    set_item(item);
    preload();
    for (;;) {
#pragma unroll
        for (int mi = 0; mi < MR; ++mi)
#pragma unroll
            for (int j = 0; j < NR; ++j)
                acc[mi][j] = zero_acc<AT>();
        // waves whose rows all lie past the last one only load
        const bool idle = ROLE != GROUP_DW && (int)row0 >= rows;
        const int nomask = min(nkt, last_full);
        if (!idle)
            k_loop<ST, STEPS, S::LOADS, step_groups(MR * NR), true>(nkt, nomask, load, read, mma);
        else
            k_loop<ST, STEPS, S::LOADS, step_groups(MR * NR), true>(nkt, nomask, load, nothing, nothing);
        if constexpr (ADAPT) {
            if constexpr (TM <= 64)
            if (p.R <= 32 && units > p.units * (TM / 8)) {
                // A few rows and ranks, and an adapter for every eighth row or more: a thread
                // takes a column of B at a time, the lanes of a wave neighbouring ones, whose
                // ranks lie together in memory, for each row with its own adapter.  Sums in fp32
                // through LDS into the accumulators' layout.  They take the same time however
                // many adapters the rows have, where the matrix steps, below, take one of all
                // rows for each (28672 x 2048, 32 rows of 16 ranks in 32 x 64 tiles: 33.0 to 33.7
                // us; 31.0 for one adapter, 32.8 for 4, 34.5 for 8, 41.7 for 32; 16 rows in 16 x 32
                // tiles 31.6 to 32.4, and 31.6 for one, 32.0 for 2, 33.0 for 4, 36.2 for 16; 3000
                // rows of 264 x 1024, 64 adapters, two in a 64 x 64 tile: 21.6 and 17.4).
                const KernelArgs q = kernel_args();
                float* delta = reinterpret_cast<float*>(lds);                  // [TM][TN + 4]
                float* u_lds = delta + TM * (TN + 4);                          // [TM][32]
                int* row_id = reinterpret_cast<int*>(u_lds + TM * 32);         // [TM]
                static_assert((TM * (TN + 4) + TM * 33) * 4 <= S::OUT_AT, "fits the stages");
                for (int r = tid; r < TM; r += S::THREADS)
                    row_id[r] = -1;
                for (int i = tid; i < rows * 4; i += S::THREADS) {
                    const int r = i / 4, k = i % 4 * 8;
                    if (k < q->R) {
                        const uint16_t* u = reinterpret_cast<const uint16_t*>(q->U) + (int64_t)(m0 + r) * 2 * q->R + k;
                        const i32x4 hi = *reinterpret_cast<const i32x4*>(u);
                        const i32x4 lo = *reinterpret_cast<const i32x4*>(u + q->R);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            u_lds[r * 32 + k + 2 * e] =
                                __uint_as_float((uint32_t)hi[e] << 16) + __uint_as_float((uint32_t)lo[e] << 16);
                            u_lds[r * 32 + k + 2 * e + 1] = __uint_as_float((uint32_t)hi[e] & 0xFFFF0000u) +
                                                            __uint_as_float((uint32_t)lo[e] & 0xFFFF0000u);
                        }
                    }
                }
                __syncthreads();
                const int over = units / q->units;
                for (int e = tid; e < over; e += S::THREADS) {
                    const int id = table.id(entry0 + e);
                    const int hi = min(table.first(entry0 + e + 1) - m0, rows);
                    for (int r = max(table.first(entry0 + e) - m0, 0); r < hi; ++r)
                        row_id[r] = id;
                }
                __syncthreads();
                constexpr int EACH = TM * TN / S::THREADS, B = EACH < 8 ? EACH : 8;
                static_assert(EACH % B == 0, "columns a thread");
                for (int i0 = 0; i0 < EACH; i0 += B) {
                    float sum[B] = {};
                    for (int k = 0; k < q->R; k += 16) {
                        i32x4 w[B][2];
#pragma unroll
                        for (int i = 0; i < B; ++i) {
                            const int at = (i0 + i) * S::THREADS + tid, r = at / TN, c = at % TN;
                            const int id = row_id[r];
                            const bool in = id >= 0 && n0 + c < q->N;
                            const uint8_t* from = q->LB + (in ? id * q->lb_group + (n0 + c) * q->ldlb_b + k * 2 : 0);
                            w[i][0] = *reinterpret_cast<const i32x4*>(from);
                            w[i][1] = *reinterpret_cast<const i32x4*>(from + (in && k + 8 < q->R ? 16 : 0));
                        }
#pragma unroll
                        for (int i = 0; i < B; ++i) {
                            const int r = ((i0 + i) * S::THREADS + tid) / TN;
                            const float* u = u_lds + r * 32 + k;
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (k + 8 * h < q->R)
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        sum[i] = fmaf(u[8 * h + 2 * e], __uint_as_float((uint32_t)w[i][h][e] << 16), sum[i]);
                                        sum[i] = fmaf(u[8 * h + 2 * e + 1],
                                                      __uint_as_float((uint32_t)w[i][h][e] & 0xFFFF0000u), sum[i]);
                                    }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < B; ++i) {
                        const int at = (i0 + i) * S::THREADS + tid, r = at / TN;
                        delta[r * (TN + 4) + at % TN] = row_id[r] >= 0 ? sum[i] : 0.f;
                    }
                }
                __syncthreads();
                // (rows that have none take zeros, and a row's NaN stays its own)
#pragma unroll
                for (int mi = 0; mi < MR; ++mi)
#pragma unroll
                    for (int j = 0; j < NR; ++j)
                        acc[mi][j] += *reinterpret_cast<const f32x4*>(
                            delta + ((int)row0 + mi * R + lc) * (TN + 4) + (int)col0 + j * R + 4 * lg);
                __syncthreads();
                units = 0;
            }
            // Behind the k-tiles of X and W: the ranks of the adapters that the tile's rows
            // have, in units of 16.  One step of the matrix cores holds a unit: the rows'
            // inner values, upper halves and then lower ones, against the same columns of B
            // twice.  As many k-tiles as there are stages at a time, all their loads and
            // then their products (as a second pipelined loop they had registers of the
            // first spilled; straight from memory in the fragments' layout, neighbouring
            // lanes in different rows, 4095 rows of 64 ranks took 24 us longer).  A unit's
            // products are formed apart and added to the rows of its adapter only: zeros in
            // the other rows' inner values would not keep an infinity or NaN of one request's
            // adapter out of the others' rows.
            const KernelArgs q = kernel_args();
            for (int u0 = 0; u0 < units; u0 += ST * STEPS) {
                // (lanes as values of their own, so that nothing that hangs on them lives
                // through the loop before)
                int ol = lane;
                asm volatile("" : "+v"(ol));
                // lane i: unit u0 + i; behind the last one: no row, no rank
                const int each = q->units, u = u0 + min(ol, ST * STEPS - 1);
                const int at = min(u, units - 1) / each;
                const int v_lo = table.first(entry0 + at) - m0;
                const int v_hi = u < units ? table.first(entry0 + at + 1) - m0 : v_lo;
                const int v_id = table.id(entry0 + at);
                const int v_rank = u < units ? (u - at * each) * 16 : q->R;
                const int cols = min(TN, q->N - n0);
                const rsrc_t ru = make_rsrc(uniform(q->U + (int64_t)m0 * q->R * 4), (uint32_t)(rows * q->R * 4));
                const int r0 = KTL::ROWS_PER_LOAD * wave + ol / CHUNKS;
                const int c = (int)((uint32_t)(ol % CHUNKS) ^ KTL::key((uint32_t)r0));
#pragma unroll 1
                for (int t = 0; t < ST && u0 + t * STEPS < units; ++t) {
                    const int id = __builtin_amdgcn_readlane(v_id, t * STEPS);
                    int rank = __builtin_amdgcn_readlane(v_rank, t * STEPS);
                    const uint8_t* from = q->LB + (int64_t)n0 * q->ldlb_b;
                    uint32_t at = 0, records = (uint32_t)((cols - 1) * (int)q->ldlb_b + q->R * 2);
                    if (q->pack) {                      // any adapter by a 32-bit offset
                        records = 0x7FFFFFFFu;
                        at = (uint32_t)id * (uint32_t)q->lb_group;
                    } else {                            // a k-tile is of one adapter
                        from += id * q->lb_group;
                    }
                    if constexpr (STEPS == 2) {
                        const int id1 = __builtin_amdgcn_readlane(v_id, t * STEPS + 1);
                        const int rank1 = __builtin_amdgcn_readlane(v_rank, t * STEPS + 1);
                        rank = c < 4 ? rank : rank1;
                        at = c < 4 || !q->pack ? at : (uint32_t)id1 * (uint32_t)q->lb_group;
                    }
                    rank += c % 2 * 8;
                    const rsrc_t rl = make_rsrc(uniform(from), records);
                    uint8_t* base = lds + t * STAGE;
#pragma unroll
                    for (int n = 0; n < A_DMA; ++n)
                        dma16(ru, base + (wave + WAVES * n) * 1024,
                              rank < q->R ? (uint32_t)(((r0 + n * A_ROWS) * 2 + c / 2 % 2) * q->R + rank) * 2u : kOOB,
                              0);
#pragma unroll
                    for (int n = 0; n < B_DMA; ++n) {
                        const int r = r0 + n * B_ROWS;
                        dma16(rl, base + A_BUF + (wave + WAVES * n) * 1024,
                              rank < q->R && r < cols ? at + (uint32_t)r * (uint32_t)q->ldlb_b + (uint32_t)rank * 2u
                                                      : kOOB,
                              0);
                    }
                }
                // An infinity of B counts against the upper halves only: against a lower one,
                // zero or of the other sign, it would turn the row's infinity into NaN.  Every
                // lane looks at the pieces that it loaded, before the others may (stages that
                // hold no units have something of before, which nobody reads).
                __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
                asm volatile("" ::: "memory");
                auto piece = [&](int t, int n) __attribute__((always_inline)) {
                    return reinterpret_cast<i32x4*>(lds + t * STAGE + A_BUF + (wave + WAVES * n) * 1024 + ol * 16);
                };
                u16x2 largest = {0, 0};
#pragma unroll
                for (int t = 0; t < ST; ++t)
#pragma unroll
                    for (int n = 0; n < B_DMA; ++n) {
                        const i32x4 w = *piece(t, n);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            largest = __builtin_elementwise_max(largest,
                                                                __builtin_bit_cast(u16x2, w[e] & 0x7FFF7FFF));
                    }
                if (c / 2 % 2 && max(largest[0], largest[1]) >= 0x7F80)
#pragma unroll 1
                    for (int t = 0; t < ST; ++t)
#pragma unroll 1
                        for (int n = 0; n < B_DMA; ++n) {
                            i32x4 w = *piece(t, n);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t v = (uint32_t)w[e];
                                w[e] = (int)(((v & 0x7F80u) == 0x7F80u ? 0u : v & 0xFFFFu) |
                                             ((v & 0x7F800000u) == 0x7F800000u ? 0u : v & 0xFFFF0000u));
                            }
                            *piece(t, n) = w;
                        }
                DG_STAGE_BARRIER(0);
#pragma unroll 1
                for (int i = 0; i < ST * STEPS && !idle; ++i) {
                    const int lo = __builtin_amdgcn_readlane(v_lo, i), hi = __builtin_amdgcn_readlane(v_hi, i);
                    if (hi <= lo)
                        continue;
                    const int s = i % STEPS;
                    const uint8_t* base = lds + i / STEPS * STAGE;
                    const uint32_t chunk = ((uint32_t)(4 * s + (ol >> 4)) ^ KTL::key((uint32_t)(ol % 16))) << 4;
                    const uint8_t* wp = base + A_BUF + (col0 + (uint32_t)(ol % 16)) * KTB + chunk;
                    const uint8_t* up = base + (row0 + (uint32_t)(ol % 16)) * KTB + chunk;
                    i32x4 wf[NR];
#pragma unroll
                    for (int j = 0; j < NR; ++j)
                        wf[j] = *reinterpret_cast<const i32x4*>(wp + j * R * KTB);
#pragma unroll
                    for (int mi = 0; mi < MR; ++mi) {
                        const int r = (int)row0 + mi * R;
                        if (r >= hi || r + R <= lo)
                            continue;
                        const i32x4 uf = *reinterpret_cast<const i32x4*>(up + mi * R * KTB);
                        if (r >= lo && r + R <= hi) {        // all 16 rows are its own
#pragma unroll
                            for (int j = 0; j < NR; ++j)
                                acc[mi][j] = mfma_bf16(wf[j], uf, acc[mi][j]);
                            continue;
                        }
                        const bool own = r + ol % 16 >= lo && r + ol % 16 < hi;
                        acc_t v[NR];
#pragma unroll
                        for (int j = 0; j < NR; ++j)
                            v[j] = mfma_bf16(wf[j], uf, zero_acc<AT>());
                        if (own)
#pragma unroll
                            for (int j = 0; j < NR; ++j)
                                acc[mi][j] += v[j];
                    }
                }
                DG_STAGE_BARRIER(0);
            }
        }
        if constexpr (MUL) {
            if (!idle && kernel_args()->mul_vec) {
#pragma unroll
                for (int mi = 0; mi < AHEAD; ++mi)
                    load_mul(mi, m0, n0, rows);
            } else {                           // (or they would be kept from the item before)
#pragma unroll
                for (int mi = 0; mi < AHEAD; ++mi)
#pragma unroll
                    for (int j = 0; j < NR; ++j)
                        mulv[mi][j] = make_uint2(0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        // the next item's loads go out before this one's outputs
        const int o_group = group, o_m0 = m0, o_n0 = n0, o_rows = rows;
        const bool more = next_item();
        if (more) {
            set_item(item);
            preload();
        }
        if (!idle)
            output(o_group, o_m0, o_n0, o_rows);
        if (!more)
            break;
    }
}

}  // namespace dg
