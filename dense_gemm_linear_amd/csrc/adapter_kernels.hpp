// Kernels of linear_adapters beside the grouped product: the inner values of rows
// that many requests' adapters have, the whole of it for one token, and for few
// rows in slices of K.
#pragma once

#include "group_kernels.hpp"

namespace dg {

// ---------------------------------------------------------------------------
// Adapters' inner values: u[p] = scale_g A_g x for every sorted row p of a
// group, as two bf16 halves (the rounded value and the rounded rest: 16 bits of
// it together, so that what rounding takes from u is far below the rounding of
// Y).  One workgroup takes 16 MB rows of one group and 16 NR ranks.  Its 8 waves
// split K in chunks of 64 values, a whole line of every row, and keep two chunks
// in flight in registers: eight lanes a line, which is how memory gives them up
// (loads in the fragments' layout, with neighbouring lanes in different rows, came
// at 15 bytes a clock and CU).  The waves turn them in LDS of their own, without
// barriers, and add their sums at the end in a fixed order.
// The group whose rows sorted position x is among: the number of groups that end
// at or before it (`groups`: none, as for a row in front of the first group's, which a
// range of a larger table's offsets has).
__device__ __forceinline__ int row_group(const int* offsets, int groups, int x, int lane)
{
    int n = x < offsets[0] ? groups : 0;
    for (int g = 0; g < groups; g += 64)
        n += __popcll(__ballot(g + lane < groups && offsets[min(g + lane, groups - 1) + 1] <= x));
    return __builtin_amdgcn_readfirstlane(n);
}

struct InnerArgs {
    const uint8_t* X;
    int64_t ldx_b;
    uint32_t x_bytes;
    const int* offsets;
    const int* order;
    int groups, S;
    const uint8_t* A;      // [groups][R][lda]
    int64_t lda_b, a_group;
    const float* scale;
    int R, K;
    uint16_t* U;           // [S][2][R]
};

// u in its two halves.  A finite value that would round to infinity has the largest
// finite one as its upper half, which leaves a finite rest.
__device__ __forceinline__ void store_inner(uint16_t* to, int R, float v)
{
    uint16_t hi = bf16_rne(v);
    if ((hi & 0x7FFFu) == 0x7F80u && fabsf(v) < INFINITY)
        --hi;
    const float rest = v - bf16_to_f32(hi);      // infinite v: none
    to[0] = hi;
    to[R] = fabsf(rest) < INFINITY ? bf16_rne(rest) : 0;
}

template <int NR, int MB>
__global__ __launch_bounds__(512) void adapter_inner_kernel(InnerArgs p)
{
    constexpr int WAVES = 8, ROWS = 16 * (MB + NR), LOADS = ROWS / 8;
    constexpr int PART = MB * NR * 1024 > ROWS * 128 ? MB * NR * 1024 : ROWS * 128;
    using KTL = KTile<128>;
    __shared__ __attribute__((aligned(16))) uint8_t lds[WAVES * PART + kTableLds];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lc = lane & 15, lg = lane >> 4;
    const int block = (int)blockIdx.x;
    GroupTable table;
    table.at(lds + WAVES * PART);
    build_table<64 * WAVES, false>(table, p.offsets, p.groups, p.S, 16 * MB, 0);
    if (block >= table.first(p.groups))
        return;
    const int group = __builtin_amdgcn_readfirstlane(find_entry(table, block, lane));
    const int2 gr = group_rows(p.offsets, group, p.S);
    const int m0 = __builtin_amdgcn_readfirstlane(gr.x + (block - table.first(group)) * 16 * MB);
    const int rows = min(16 * MB, __builtin_amdgcn_readfirstlane(gr.y) - m0);
    const int r0 = (int)blockIdx.y * 16 * NR;

    // load i: rows 8 i .. 8 i + 7 of the chunk's 16 MB rows of X and 16 NR of A
    const int lr = lane >> 3;
    const uint32_t lk = (uint32_t)(lane & 7) * 16u;
    uint32_t x_off[2 * MB];
#pragma unroll
    for (int i = 0; i < 2 * MB; ++i)
        x_off[i] = (uint32_t)p.order[m0 + min(8 * i + lr, rows - 1)];
    const rsrc_t rx = make_rsrc(p.X, p.x_bytes);
    const rsrc_t ra = make_rsrc(uniform(p.A + group * p.a_group + r0 * p.lda_b),
                                (uint32_t)((int64_t)(min(16 * NR, p.R - r0) - 1) * p.lda_b + p.K * 2));
    const int chunks = (p.K + 63) / 64;
    i32x4 got[2][LOADS];
    auto load_a = [&](int c, auto set) __attribute__((always_inline)) {
        const uint32_t k = (uint32_t)c * 128u + lk;
        const bool in = (int)k < p.K * 2;
#pragma unroll
        for (int i = 0; i < 2 * NR; ++i)
            got[decltype(set)::value][2 * MB + i] =
                load16(ra, in ? (uint32_t)(8 * i + lr) * (uint32_t)p.lda_b + k : kOOB);
    };
    auto load_x = [&](int c, auto set) __attribute__((always_inline)) {
        const uint32_t k = (uint32_t)c * 128u + lk;
        const bool in = (int)k < p.K * 2;
#pragma unroll
        for (int i = 0; i < 2 * MB; ++i)
            got[decltype(set)::value][i] = load16(rx, in ? x_off[i] + k : kOOB);
    };
    f32x4 acc[MB][NR];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int j = 0; j < NR; ++j)
            acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    uint8_t* own = lds + wave * PART;
    auto multiply = [&](auto set) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const uint32_t r = (uint32_t)(8 * i + lr);
            *reinterpret_cast<i32x4*>(own + r * 128 + (((uint32_t)(lane & 7) ^ KTL::key(r)) << 4)) =
                got[decltype(set)::value][i];
        }
        wave_lds_order();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const uint32_t c = ((uint32_t)(4 * s + lg) ^ KTL::key((uint32_t)lc)) << 4;
            i32x4 x[MB], a[NR];
#pragma unroll
            for (int m = 0; m < MB; ++m)
                x[m] = *reinterpret_cast<const i32x4*>(own + (16 * m + lc) * 128 + c);
#pragma unroll
            for (int j = 0; j < NR; ++j)
                a[j] = *reinterpret_cast<const i32x4*>(own + (16 * (MB + j) + lc) * 128 + c);
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int j = 0; j < NR; ++j)
                    acc[m][j] = mfma_bf16(x[m], a[j], acc[m][j]);
        }
        wave_lds_order();
    };
    constexpr std::integral_constant<int, 0> S0{};
    constexpr std::integral_constant<int, 1> S1{};
    // A's loads first: those of X wait for the rows' numbers
    load_a(wave, S0);
    load_a(wave + WAVES, S1);
#pragma unroll
    for (int i = 0; i < 2 * MB; ++i)
        x_off[i] = 8 * i + lr < rows && x_off[i] < (uint32_t)p.S ? x_off[i] * (uint32_t)p.ldx_b : kOOB;
    load_x(wave, S0);
    load_x(wave + WAVES, S1);
    for (int c = wave; c < chunks; c += 2 * WAVES) {
        // (a chunk past K is zeros)
        multiply(S0);
        load_a(c + 2 * WAVES, S0);
        load_x(c + 2 * WAVES, S0);
        multiply(S1);
        load_a(c + 3 * WAVES, S1);
        load_x(c + 3 * WAVES, S1);
    }
    f32x4* part = reinterpret_cast<f32x4*>(lds);
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int j = 0; j < NR; ++j)
            part[(wave * MB * NR + m * NR + j) * 64 + lane] = acc[m][j];
    __syncthreads();
    const float scale = p.scale ? p.scale[group] : 1.f;
    for (int b = wave; b < MB * NR; b += WAVES) {
        f32x4 sum = part[b * 64 + lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w)
            sum += part[(w * MB * NR + b) * 64 + lane];
        const int rank = r0 + 16 * (b % NR) + lc;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 16 * (b / NR) + 4 * lg + e;
            if (r < rows && rank < p.R)
                store_inner(p.U + (int64_t)(m0 + r) * 2 * p.R + rank, p.R, sum[e] * scale);
        }
    }
}

__device__ __forceinline__ float dot8(i32x4 a, i32x4 b, float sum)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sum = fmaf(__uint_as_float((uint32_t)a[i] << 16), __uint_as_float((uint32_t)b[i] << 16), sum);
        sum = fmaf(__uint_as_float((uint32_t)a[i] & 0xFFFF0000u), __uint_as_float((uint32_t)b[i] & 0xFFFF0000u),
                   sum);
    }
    return sum;
}
__device__ __forceinline__ float lanes_sum(float x)
{
#pragma unroll
    for (int d = 32; d; d >>= 1)
        x += __shfl_xor(x, d);
    return x;
}

// The same for few rows: a workgroup a row and 16 ranks, a wave a rank, 512
// values of K at a time over its lanes.  The row's group is found by counting the
// offsets in front.  A whole call of 8 rows of 16 ranks, 14336 x 4096: 31.0 us, 32.9 with the
// kernel above; 64 rows of 28672 x 4096 67.9 and 70.1, 200 of 14336 x 4096 61.1 and 64.0.
__global__ __launch_bounds__(1024) void adapter_inner_row_kernel(InnerArgs p)
{
    const int lane = threadIdx.x & 63;
    const int m0 = (int)blockIdx.x;
    const int r = (int)blockIdx.y * 16 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const uint32_t row = (uint32_t)p.order[m0];
    const int group = row_group(p.offsets, p.groups, m0, lane);
    if (group >= p.groups || r >= p.R)
        return;
    const rsrc_t rx = make_rsrc(uniform(p.X + (row < (uint32_t)p.S ? row * p.ldx_b : 0)), (uint32_t)p.K * 2u);
    const rsrc_t ra = make_rsrc(uniform(p.A + group * p.a_group + r * p.lda_b), (uint32_t)p.K * 2u);
    constexpr int UN = 8;
    float sum = 0.f;
    for (int k0 = lane * 16; k0 < p.K * 2 + lane * 16; k0 += 1024 * UN) {
        i32x4 x[UN], a[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const uint32_t off = (uint32_t)(k0 + 1024 * u);          // (past K: zeros)
            a[u] = load16(ra, off);
            x[u] = load16(rx, off);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < UN; ++u)
            sum = dot8(a[u], x[u], sum);
    }
    sum = lanes_sum(sum);
    if (lane == 0)
        store_inner(p.U + (int64_t)m0 * 2 * p.R + r, p.R, sum * (p.scale ? p.scale[group] : 1.f));
}

// ---------------------------------------------------------------------------
// One token: y = W x + scale_g B_g (A_g x), all in one launch.  Bound by reading W
// (11008 x 4096: 90 MB, 13.6 us at the rate of a streaming read), so that the matrix
// cores have nothing to offer: a wave takes ROWS rows of W, 512 values of K at a
// time over its lanes, in fp32.  Every workgroup forms the inner values itself, a
// row of A a wave next to its rows of W (128 KiB for 16 ranks, from the L2, against
// 256 KiB of W): the launch that does it apart took 7 us of 26.
struct TokenArgs {
    const uint16_t* X;
    const uint16_t* W;
    int64_t ldw;
    const uint16_t* A;
    int64_t lda, a_group;
    const uint16_t* B;
    int64_t ldb, b_group;
    const float* scale;
    const int* offsets;
    int groups, N, K, R;
    uint16_t* Y;
};

template <int ROWS, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void adapter_token_kernel(TokenArgs p)
{
    __shared__ float inner[kMaxRank];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int n0 = ((int)blockIdx.x * WAVES + wave) * ROWS;
    const int K = p.K;
    constexpr int UN = 4;
    const rsrc_t rx = make_rsrc(p.X, (uint32_t)K * 2u);
    const rsrc_t rw = make_rsrc(uniform(reinterpret_cast<const uint8_t*>(p.W + (int64_t)min(n0, p.N - 1) * p.ldw)),
                                n0 < p.N ? (uint32_t)((min(ROWS, p.N - n0) - 1) * (int)p.ldw + K) * 2u : 0u);
    const int group = row_group(p.offsets, p.groups, 0, lane);
    const bool has = group < p.groups;
    // rank `wave`, if there is one; a row past the last reads zeros
    auto rank_row = [&](int r) __attribute__((always_inline)) {
        const bool in = has && r < p.R;
        return make_rsrc(uniform(reinterpret_cast<const uint8_t*>(p.A + (in ? group * p.a_group + r * p.lda : 0))),
                         in ? (uint32_t)K * 2u : 0u);
    };
    const rsrc_t ra = rank_row(wave);
    float acc[ROWS] = {}, rank = 0.f;
    for (int k0 = lane * 8; k0 < K + lane * 8; k0 += 512 * UN) {
        i32x4 x[UN], w[UN][ROWS], a[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int k = k0 + 512 * u;
            // (past a row's end the next row begins)
            const uint32_t off = k < K ? (uint32_t)k * 2u : kOOB;
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
                w[u][r] = load16_nt(rw, k < K ? off + (uint32_t)r * (uint32_t)p.ldw * 2u : kOOB);
            x[u] = load16(rx, off);
            a[u] = load16(ra, off);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            rank = dot8(a[u], x[u], rank);
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
                acc[r] = dot8(w[u][r], x[u], acc[r]);
        }
    }
    const float scale = has && p.scale ? p.scale[group] : 1.f;
    rank = lanes_sum(rank);
    if (lane == 0)
        inner[wave] = rank * scale;
    for (int r = wave + WAVES; r < p.R; r += WAVES) {
        const rsrc_t rr = rank_row(r);
        float s = 0.f;
        for (int k = lane * 8; k < K; k += 512)
            s = dot8(load16(rr, (uint32_t)k * 2u), load16(rx, (uint32_t)k * 2u), s);
        s = lanes_sum(s);
        if (lane == 0)
            inner[r] = s * scale;
    }
    __syncthreads();
    if (has)
        for (int r = lane; r < p.R; r += 64)
#pragma unroll
            for (int i = 0; i < ROWS; ++i)
                if (n0 + i < p.N)
                    acc[i] = fmaf(inner[r], bf16_to_f32(p.B[group * p.b_group + (n0 + i) * p.ldb + r]), acc[i]);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const float y = lanes_sum(acc[i]);
        if (lane == 0 && n0 + i < p.N)
            p.Y[n0 + i] = bf16_rne(y);
    }
}

// ---------------------------------------------------------------------------
// Few rows: W x over slices of K, so that all CUs read W, with the inner values
// formed by further workgroups of the same launch; a second launch adds the slices
// and the adapters' terms.  A CU's loads bring 45 to 60 KB a microsecond into LDS
// whatever the tile, and without slices a decode batch has too few tiles (48 rows of
// 11008 x 4096, 16 adapters of 16 ranks: 35.2 -> 28.4 us; 40 of 4096 x 4096 24.7 -> 16.7).
struct SplitArgs {
    const uint8_t* X;
    int64_t ldx_b;
    const uint8_t* W;
    int64_t ldw_b;
    int T, N, K;
    int tiles_m, slices, kts;      // kts: k-tiles a slice
    int main;                      // workgroups of the product; behind them the inner values'
    int nt;                        // W is read once
    float* planes;                 // [slices][T][pitch]
    int pitch;
    // inner values
    const int* offsets;
    const int* order;
    int groups, R;
    const uint8_t* A;
    int64_t lda_b, a_group;
    const float* scale;
    float* U;                      // [T][R], by sorted position
};

// A workgroup a row and 16 ranks, a wave four of them, 512 values of K at a time over
// its lanes.
__device__ __forceinline__ void split_inner(const SplitArgs& p, int b, int wave, int lane)
{
    const int per_row = (p.R + 15) / 16;
    const int at = b / per_row, r0 = b % per_row * 16 + wave * 4;
    const uint32_t row = (uint32_t)__builtin_amdgcn_readfirstlane(p.order[at]);
    const int group = row_group(p.offsets, p.groups, at, lane);
    if (group >= p.groups || r0 >= p.R || row >= (uint32_t)p.T)
        return;
    const rsrc_t rx = make_rsrc(uniform(p.X + row * p.ldx_b), (uint32_t)p.K * 2u);
    // (R is a multiple of 8: all four are there)
    const uint8_t* a = p.A + group * p.a_group + r0 * p.lda_b;
    rsrc_t ra[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
        ra[r] = make_rsrc(uniform(a + r * p.lda_b), (uint32_t)p.K * 2u);
    constexpr int UN = 2;
    float sum[4] = {};
    for (int k0 = lane * 16; k0 < p.K * 2 + lane * 16; k0 += 1024 * UN) {
        i32x4 x[UN], w[UN][4];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const uint32_t off = (uint32_t)(k0 + 1024 * u);          // (past K: zeros)
            x[u] = load16(rx, off);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                w[u][r] = load16(ra[r], off);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < UN; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                sum[r] = dot8(w[u][r], x[u], sum[r]);
    }
    const float scale = p.scale ? p.scale[group] : 1.f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const float v = lanes_sum(sum[r]);
        if (lane == 0)
            p.U[(int64_t)at * p.R + r0 + r] = v * scale;
    }
}

template <class S>
__global__ __launch_bounds__(S::THREADS, S::OCC) void adapter_split_kernel(SplitArgs p)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S::OUT_AT];
    using AT = Atom<DT_BF16, 16>;
    using KTL = KTile<S::KTB>;
    using acc_t = AT::acc_t;
    constexpr int TM = S::TM, TN = S::TN, WN = S::WN, R = 16, KTB = S::KTB, WAVES = S::WAVES, ST = S::ST;
    constexpr int MR = S::MR, NR = S::NR, A_DMA = S::A_DMA, B_DMA = S::B_DMA, A_BUF = S::A_BUF, STAGE = S::STAGE;
    constexpr int STEPS = KTB / 64;
    static_assert(WAVES == 4, "split_inner's ranks");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    if ((int)blockIdx.x >= p.main) {
        split_inner(p, (int)blockIdx.x - p.main, wave, lane);
        return;
    }
    const int wm = wave / WN, wn = wave % WN;
    const int lc = lane & 15, lg = lane >> 4;
    const int t = xcd_remap((int)blockIdx.x, p.main);
    const int tm = t % p.tiles_m, slice = t / p.tiles_m % p.slices, tn = t / p.tiles_m / p.slices;
    const int m0 = tm * TM, n0 = tn * TN, k0 = slice * p.kts * KTB;
    const int rows = min(TM, p.T - m0), cols = min(TN, p.N - n0);
    const int kb_end = min(p.K * 2 - k0, p.kts * KTB), nkt = (kb_end + KTB - 1) / KTB, last_full = kb_end / KTB;
    const uint8_t* a_base = uniform(p.X + (int64_t)m0 * p.ldx_b + k0);
    const uint8_t* b_base = uniform(p.W + (int64_t)n0 * p.ldw_b + k0);
    const int a_span = (rows - 1) * (int)p.ldx_b + kb_end, b_span = (cols - 1) * (int)p.ldw_b + kb_end;
    constexpr int ROWS = WAVES * 1024 / KTB;           // between two chunks of a wave
    static_assert(ROWS % 16 == 0, "swizzles repeat");
    const int a_rows = ROWS * (int)p.ldx_b, b_rows = ROWS * (int)p.ldw_b;
    const ADma da = a_dma_lane<KTB>(wave, lane, p.ldx_b), db = a_dma_lane<KTB>(wave, lane, p.ldw_b);
    auto load = [&](int kt, int stage, int part, int nparts, auto nomask_c) __attribute__((always_inline)) {
        constexpr bool NOMASK = decltype(nomask_c)::value;
        uint8_t* to = lds + stage * STAGE + wave * 1024;
        auto offset = [&](const ADma& d) __attribute__((always_inline)) {
            if constexpr (NOMASK)
                return d.goff;
            return (int)((uint32_t)kt * KTB + d.col) < kb_end ? d.goff + (uint32_t)kt * KTB : kOOB;
        };
        const uint32_t soff = NOMASK ? (uint32_t)kt * KTB : 0u;
#pragma unroll
        for (int i = 0; i < A_DMA; ++i)
            if (i % nparts == part)
                dma16(make_rsrc(a_base + i * a_rows, (uint32_t)max(a_span - i * a_rows, 0)), to + WAVES * i * 1024,
                      offset(da), soff);
#pragma unroll
        for (int i = 0; i < B_DMA; ++i)
            if ((A_DMA + i) % nparts == part) {
                const rsrc_t r = make_rsrc(b_base + i * b_rows, (uint32_t)max(b_span - i * b_rows, 0));
                if (p.nt)
                    dma16_nt(r, to + A_BUF + WAVES * i * 1024, offset(db), soff);
                else
                    dma16(r, to + A_BUF + WAVES * i * 1024, offset(db), soff);
            }
    };
    const uint32_t swz = KTL::key((uint32_t)lc);
    const uint32_t row0 = (uint32_t)(wm * (TM / S::WM)), col0 = (uint32_t)(wn * S::WCOLS);
    LdsBases<S::OUT_AT> a_at[STEPS], b_at[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const uint32_t chunk = ((uint32_t)AT::a_chunk(s, lane, 0) ^ swz) << 4;
        a_at[s].init((row0 + (uint32_t)lc) * KTB + chunk);
        b_at[s].init((col0 + (uint32_t)lc) * KTB + chunk);
    }
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
            if (f < NR)
                bf[set][f] = *reinterpret_cast<const i32x4*>(
                    lds + b_at[s].at((uint32_t)(stage * STAGE + A_BUF + f * R * KTB)));
            else
                af[set][f - NR] = *reinterpret_cast<const i32x4*>(
                    lds + a_at[s].at((uint32_t)(stage * STAGE + (f - NR) * R * KTB)));
        }
    };
    auto mma = [&](int, int, int set, int g, int G) __attribute__((always_inline)) {
#pragma unroll
        for (int a = 0; a < MR * NR; ++a)
            if (a * G / (MR * NR) == g)
                acc[a / NR][a % NR] = mfma_bf16(bf[set][a % NR], af[set][a / NR], acc[a / NR][a % NR]);
    };
    k_loop<ST, STEPS, S::LOADS, step_groups(MR * NR)>(nkt, min(nkt, last_full), load, read, mma);
    // a lane holds four consecutive columns of a row; the pitch is a multiple of 4
    float* to = p.planes + ((int64_t)slice * p.T + m0) * p.pitch;
#pragma unroll
    for (int mi = 0; mi < MR; ++mi)
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            const int r = (int)row0 + mi * R + lc, c = n0 + (int)col0 + j * R + 4 * lg;
            if (r < rows && c < p.pitch)
                *reinterpret_cast<f32x4*>(to + (int64_t)r * p.pitch + c) = acc[mi][j];
        }
}

struct JoinArgs {
    const float* planes;
    int slices, T, N, pitch;
    const int* offsets;
    const int* order;
    int groups, R;
    const float* U;
    const uint16_t* B;
    int64_t ldb, b_group;
    uint16_t* Y;
    int64_t ldy;
};

// y = the sum of the slices, in their order, and u B^T.  A workgroup 256 columns of four
// rows, a thread a column, with NP pieces of 8 ranks of B at a time, in registers for as
// long as the rows are of one adapter.
constexpr int kJoinRows = 4;
template <int NP>
__global__ __launch_bounds__(256) void adapter_join_kernel(JoinArgs p)
{
    __shared__ __attribute__((aligned(16))) float u[kJoinRows][kMaxRank];
    const int at = (int)blockIdx.x * kJoinRows, lane = threadIdx.x & 63;
    int token[kJoinRows], group[kJoinRows];
#pragma unroll
    for (int i = 0; i < kJoinRows; ++i) {
        token[i] = at + i < p.T ? __builtin_amdgcn_readfirstlane(p.order[at + i]) : -1;
        group[i] = at + i < p.T ? row_group(p.offsets, p.groups, at + i, lane) : p.groups;
    }
    for (int i = (int)threadIdx.x; i < min(kJoinRows, p.T - at) * p.R; i += 256)
        u[i / p.R][i % p.R] = p.U[(int64_t)at * p.R + i];
    __syncthreads();
    const int c = (int)blockIdx.y * 256 + (int)threadIdx.x;
    if (c >= p.N)
        return;
    const int64_t step = (int64_t)p.T * p.pitch;
    float sum[kJoinRows] = {};
    for (int s0 = 0; s0 < p.slices; s0 += 4) {
        float v[kJoinRows][4];
#pragma unroll
        for (int i = 0; i < kJoinRows; ++i) {
            const float* from = p.planes + (int64_t)((uint32_t)token[i] < (uint32_t)p.T ? token[i] : 0) * p.pitch + c;
#pragma unroll
            for (int s = 0; s < 4; ++s)
                v[i][s] = from[min(s0 + s, p.slices - 1) * step];
        }
#pragma unroll
        for (int i = 0; i < kJoinRows; ++i)
#pragma unroll
            for (int s = 0; s < 4; ++s)
                sum[i] += s0 + s < p.slices ? v[i][s] : 0.f;
    }
    for (int r0 = 0; r0 < p.R; r0 += 8 * NP) {
        i32x4 w[NP] = {};
        int held = -1;
#pragma unroll
        for (int i = 0; i < kJoinRows; ++i) {
            if (group[i] >= p.groups)
                continue;
            if (group[i] != held) {
                held = group[i];
                const uint16_t* b = p.B + held * p.b_group + c * p.ldb + r0;
#pragma unroll
                for (int q = 0; q < NP; ++q)
                    if (r0 + 8 * q < p.R)
                        w[q] = *reinterpret_cast<const i32x4*>(b + 8 * q);
            }
#pragma unroll
            for (int q = 0; q < NP; ++q)
                if (r0 + 8 * q < p.R)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float* v = &u[i][r0 + 8 * q + 2 * e];
                        sum[i] = fmaf(v[0], __uint_as_float((uint32_t)w[q][e] << 16), sum[i]);
                        sum[i] = fmaf(v[1], __uint_as_float((uint32_t)w[q][e] & 0xFFFF0000u), sum[i]);
                    }
        }
    }
#pragma unroll
    for (int i = 0; i < kJoinRows; ++i)
        if ((uint32_t)token[i] < (uint32_t)p.T)
            p.Y[token[i] * p.ldy + c] = bf16_rne(sum[i]);
}

}  // namespace dg
