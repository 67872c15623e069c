// Rows sorted by group and back: the slots' stable sort, the rows' copy into
// that order, their weighted join and its gradient.  All of it moves memory;
// nothing is multiplied but by a weight.
#include "group.hpp"
#include "kernels.hpp"

#include <algorithm>

namespace dg {
namespace {

// ---------------------------------------------------------------------------
// Sort.  A stable counting sort of S slots by group id, ids outside [0, groups)
// behind the rest as a group of their own (`none`).  One workgroup of 16 waves
// takes a chunk of up to 8192 slots, every wave a contiguous part of it, 64 slots
// at a time:
//   1. a slot's number among its wave's slots of the same group: those of the
//      steps before (a count per wave and group in LDS) and those of the lower
//      lanes, which log2(groups) ballots tell (LDS atomics on the counts took
//      longer the fewer groups there were: 12 us for 8190 slots of 8 groups, 7 now);
//   2. thread g adds up group g's counts: rows of all lower groups, then of the
//      chunks and waves before;
//   3. each slot's position is the sum of both.
// Integers only: the result does not depend on any order of execution.  More
// chunks than one get their counts from a launch before, and many chunks the sums
// over the chunks before from one between.
constexpr int kSortWaves = 16;
constexpr int kSortBatch = 8;          // slots a lane at most
constexpr int kSortMost = kSortWaves * 64 * kSortBatch;
// Slots that one workgroup takes: 2048 in 4.3 us, 4096 in 5.8, 8192 in 9 to 14; two
// launches over chunks of 1024 take 6.8 to 7.4.
constexpr int kSortOne = 4096;
// Chunks from which on their counts are summed apart (from 32 on: 65536 slots of 128
// groups 12.0 us, 9.7 so; 131072 15.8 and 11.6; 524288 25.5 and 21.7).
constexpr int kSortScan = 97;

struct SortArgs {
    const int64_t* ids;
    int64_t ld;
    int k;
    uint32_t k_mul;        // 2^32 / k rounded up; 0: k is 1
    int dense;             // the pitch of ids is k
    int S, groups;
    int chunk;
    int* counts;           // [chunks][groups + 1], null: one chunk
    int* totals;           // [groups + 1], counts are sums already; null: they are not
    int* offsets;
    int* order;
    int* place;
};

__device__ __forceinline__ int slot_group(const SortArgs& p, int s)
{
    int64_t at = s;
    if (!p.dense) {
        const int t = p.k_mul ? (int)__umulhi((uint32_t)s, p.k_mul) : s;
        at = t * p.ld + (s - t * p.k);
    }
    const int64_t id = p.ids[at];
    return id >= 0 && id < p.groups ? (int)id : p.groups;
}

__device__ __forceinline__ int wave_scan(int x, int lane)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int y = __shfl_up(x, d);
        x += lane >= d ? y : 0;
    }
    return x;
}

// A wave's slots: [w0, w1) of the workgroup's chunk.
struct WavePart {
    int w0, w1;
};
__device__ __forceinline__ WavePart wave_part(const SortArgs& p, int wave)
{
    const int s0 = (int)blockIdx.x * p.chunk, s1 = min(p.S, s0 + p.chunk);
    const int part = (s1 - s0 + kSortWaves * 64 - 1) / (kSortWaves * 64) * 64;
    WavePart w;
    w.w0 = min(s1, s0 + wave * part);
    w.w1 = min(s1, w.w0 + part);
    return w;
}

// Step 1: the groups of a wave's slots and their numbers; `count` is the wave's
// counts, zeros before.
__device__ __forceinline__ void number_slots(const SortArgs& p, const WavePart& w, int lane, int* count,
                                             int (&id)[kSortBatch], int (&number)[kSortBatch])
{
#pragma unroll
    for (int i = 0; i < kSortBatch; ++i)
        id[i] = w.w0 + i * 64 + lane < w.w1 ? slot_group(p, w.w0 + i * 64 + lane) : 0;
    const int bits = 32 - __clz(p.groups);
#pragma unroll
    for (int i = 0; i < kSortBatch; ++i) {
        if (w.w0 + i * 64 >= w.w1)
            break;
        const bool in = w.w0 + i * 64 + lane < w.w1;
        const int g = id[i];
        uint64_t same = __ballot(in);
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot((g >> b) & 1);
            same &= (g >> b) & 1 ? set : ~set;
        }
        const int rank = __popcll(same & ((UINT64_C(1) << lane) - 1));
        number[i] = count[g] + rank;
        wave_lds_order();
        if (in && rank == 0)
            count[g] = number[i] + __popcll(same);
        wave_lds_order();
    }
}

__global__ __launch_bounds__(1024) void group_count_kernel(SortArgs p)
{
    __shared__ int count[kSortWaves][kMaxGroups + 1];
    const int lane = threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    for (int g = lane; g <= p.groups; g += 64)
        count[wave][g] = 0;
    wave_lds_order();
    int id[kSortBatch], number[kSortBatch];
    number_slots(p, wave_part(p, wave), lane, count[wave], id, number);
    __syncthreads();
    for (int g = threadIdx.x; g <= p.groups; g += 1024) {
        int n = 0;
        for (int w = 0; w < kSortWaves; ++w)
            n += count[w][g];
        p.counts[(int64_t)blockIdx.x * (p.groups + 1) + g] = n;
    }
}

// One workgroup a group: its chunks' counts become the sums of those before.
__global__ __launch_bounds__(256) void group_scan_kernel(SortArgs p, int chunks)
{
    __shared__ int sums[4];
    const int g = (int)blockIdx.x, lane = threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    int total = 0;
    for (int c0 = 0; c0 < chunks; c0 += 256) {
        const int c = c0 + (int)threadIdx.x;
        int* at = p.counts + (int64_t)c * (p.groups + 1) + g;
        const int n = c < chunks ? *at : 0;
        const int upto = wave_scan(n, lane);
        if (lane == 63)
            sums[wave] = upto;
        __syncthreads();
        int before = total + upto - n;
        for (int w = 0; w < 4; ++w) {
            before += w < wave ? sums[w] : 0;
            total += sums[w];
        }
        if (c < chunks)
            *at = before;
        __syncthreads();
    }
    if (threadIdx.x == 0)
        p.totals[g] = total;
}

__global__ __launch_bounds__(1024) void group_place_kernel(SortArgs p)
{
    __shared__ int next[kSortWaves][kMaxGroups + 1];
    __shared__ int sums[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int G = p.groups;
    for (int g = lane; g <= G; g += 64)
        next[wave][g] = 0;
    wave_lds_order();
    const WavePart w = wave_part(p, wave);
    int id[kSortBatch], number[kSortBatch];
    number_slots(p, w, lane, next[wave], id, number);
    __syncthreads();
    // rows of group g in all, and in the chunks before
    auto totals = [&](int g, int& before) {
        int total = 0;
        before = 0;
        if (p.totals) {
            before = p.counts[(int64_t)blockIdx.x * (G + 1) + g];
            return p.totals[g];
        }
        if (p.counts) {
            // (16 loads in flight, whatever the number of chunks)
            const int chunks = (int)gridDim.x;
            for (int c0 = 0; c0 < chunks; c0 += 16) {
                int n[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    n[i] = p.counts[(int64_t)min(c0 + i, chunks - 1) * (G + 1) + g];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    before += c0 + i < (int)blockIdx.x ? n[i] : 0;
                    total += c0 + i < chunks ? n[i] : 0;
                }
            }
        } else {
#pragma unroll
            for (int v = 0; v < kSortWaves; ++v)
                total += next[v][g];
        }
        return total;
    };
    auto starts = [&](int g, int at) {
        int n[kSortWaves];
#pragma unroll
        for (int v = 0; v < kSortWaves; ++v)
            n[v] = next[v][g];
#pragma unroll
        for (int v = 0; v < kSortWaves; ++v) {
            next[v][g] = at;
            at += n[v];
        }
    };
    // thread g: group g, and behind all others `none` (group G)
    int before = 0;
    const int rows = tid <= G ? totals(tid, before) : 0;
    const int total = tid < G ? rows : 0;
    const int upto = wave_scan(total, lane);
    if (lane == 63)
        sums[wave] = upto;
    __syncthreads();
    int base = 0, all = 0;
    for (int v = 0; v < kSortWaves; ++v) {
        base += v < wave ? sums[v] : 0;
        all += sums[v];
    }
    if (tid <= G) {
        const int first = tid < G ? base + upto - total : all;
        starts(tid, first + before);
        if (blockIdx.x == 0)
            p.offsets[tid] = first;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSortBatch; ++i) {
        const int slot = w.w0 + i * 64 + lane;
        if (slot < w.w1) {
            const int at = next[wave][id[i]] + number[i];
            p.order[at] = slot;
            p.place[slot] = id[i] < G ? at : -1;
        }
    }
}

// ---------------------------------------------------------------------------
// Rows.  Pieces of 16 bytes; rows and their starts may have any alignment (the
// hardware takes unaligned vector accesses).  The last piece of a row whose
// length is no multiple of 16 bytes begins 16 bytes before its end: both
// pieces write the same values where they overlap.
typedef i32x4 i32x4_u __attribute__((aligned(1)));

// The row of this thread, TPR (64 or 256) of which take one: the same in a whole
// wave, so that what hangs on it alone is loaded by scalar loads.
template <int TPR>
__device__ __forceinline__ int my_row()
{
    static_assert(TPR == 64 || TPR == 256, "whole waves");
    return TPR == 256 ? (int)blockIdx.x
                      : (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
}

__device__ __forceinline__ i32x4 load_piece(const void* p) { return *static_cast<const i32x4_u*>(p); }
__device__ __forceinline__ void store_piece(void* p, i32x4 v) { *static_cast<i32x4_u*>(p) = v; }
// Non-temporal accesses.  Loads of the experts' rows in the join and its gradient,
// their last use: as good in a layer (8190 rows of 4096: gather, two products and
// join 383 us, 385 without), and the rows that other kernels left in the caches are
// not pushed out (gather and join alone 40 us against 42, 65536 rows of 2048 120
// against 140).  Stores of sorted rows where these fill the Infinity Cache, so that
// the product that reads them would not find them there: 120 -> 105 us, the layer even
// (755 -> 750); below that they cost the product more than they save (8190 rows of
// 4096: 393 us against 385).
constexpr int64_t kCacheBytes = INT64_C(256) << 20;
__device__ __forceinline__ i32x4 load_piece_nt(const void* p)
{
    return __builtin_nontemporal_load(static_cast<const i32x4_u*>(p));
}
template <bool NT>
__device__ __forceinline__ void store_sorted(void* p, i32x4 v)
{
    if constexpr (NT)
        __builtin_nontemporal_store(v, static_cast<i32x4_u*>(p));
    else
        store_piece(p, v);
}

struct GatherArgs {
    const uint8_t* X;
    int64_t ldx_b;
    const int* place;
    int T, k, S;
    int row_b, pieces;
    uint8_t* Xs;
    int64_t ldxs_b;
};

// TPR threads a row.  A token's row is read once and written to each of its
// slots' places (a copy by sorted position reads it k times).
template <int TPR, bool NT>
__global__ __launch_bounds__(256) void group_gather_kernel(GatherArgs p)
{
    const int t = my_row<TPR>();
    if (t >= p.T)
        return;
    const uint8_t* from = p.X + t * p.ldx_b;
    const int* place = p.place + (int64_t)t * p.k;
    if (p.row_b < 16) {
        for (int j = 0; j < p.k; ++j)
            if ((uint32_t)place[j] < (uint32_t)p.S)
                for (int b = (int)threadIdx.x % TPR; b < p.row_b; b += TPR)
                    p.Xs[place[j] * p.ldxs_b + b] = from[b];
        return;
    }
    for (int q = (int)threadIdx.x % TPR; q < p.pieces; q += TPR) {
        const int at = min(q * 16, p.row_b - 16);
        const i32x4 v = load_piece(from + at);
        for (int j = 0; j < p.k; ++j) {
            const int to = place[j];
            if ((uint32_t)to < (uint32_t)p.S)
                store_sorted<NT>(p.Xs + to * p.ldxs_b + at, v);
        }
    }
}

struct PickArgs {
    const uint16_t* X;
    int64_t ldx;
    const int* offsets;
    const int* order;
    uint32_t k_mul;
    int S, groups, K;
    uint16_t* Xs;
};

// The same by sorted position, for whom the places are not at hand: rows of K
// (a multiple of 8) values, 16-byte aligned.
template <int TPR>
__global__ __launch_bounds__(256) void group_pick_kernel(PickArgs p)
{
    const int at = my_row<TPR>();
    if (at >= min(p.S, p.offsets[p.groups]))
        return;
    const uint32_t slot = (uint32_t)p.order[at];
    if (slot >= (uint32_t)p.S)
        return;
    const int64_t row = p.k_mul ? __umulhi(slot, p.k_mul) : slot;
    const i32x4* from = reinterpret_cast<const i32x4*>(p.X + row * p.ldx);
    i32x4* to = reinterpret_cast<i32x4*>(p.Xs + (int64_t)at * p.K);
    for (int q = (int)threadIdx.x % TPR; q < p.K / 8; q += TPR)
        to[q] = from[q];
}

struct CombineArgs {
    const uint16_t* Y;
    int64_t ldy;
    const int* place;
    const float* weights;
    int64_t ldw;
    int T, k, S, D, pieces;
    uint16_t* out;
    int64_t ldo;
    const uint16_t* dout;
    int64_t lddo;
    uint16_t* dY;
    int64_t lddy;
    float* dweights;
};

__device__ __forceinline__ void unpack8(i32x4 v, float (&f)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float((uint32_t)v[i] << 16);
        f[2 * i + 1] = __uint_as_float((uint32_t)v[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ i32x4 pack8(const float (&f)[8])
{
    i32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = (int)((uint32_t)bf16_rne(f[2 * i]) | (uint32_t)bf16_rne(f[2 * i + 1]) << 16);
    return v;
}

// out[t] = sum_j w[t][j] Y[place[t][j]], j ascending, in fp32, rounded once.  TPR
// threads a row; B slots of P pieces at a time, whose loads are all in flight: with
// one after the other (8192 x 8 slots of 2048) the rows came at 3 TB/s.
template <int TPR, int B, int P>
__global__ __launch_bounds__(256) void group_combine_kernel(CombineArgs p)
{
    const int t = my_row<TPR>();
    if (t >= p.T)
        return;
    const int* place = p.place + (int64_t)t * p.k;
    const float* w = p.weights ? p.weights + t * p.ldw : nullptr;
    uint16_t* out = p.out + t * p.ldo;
    const int q0 = (int)threadIdx.x % TPR;
    if (p.D < 8) {
        for (int d = q0; d < p.D; d += TPR) {
            float s = 0.f;
            for (int j = 0; j < p.k; ++j)
                if ((uint32_t)place[j] < (uint32_t)p.S)
                    s = fmaf(w ? w[j] : 1.f, bf16_to_f32(p.Y[place[j] * p.ldy + d]), s);
            out[d] = bf16_rne(s);
        }
        return;
    }
    for (int q = q0; q < p.pieces; q += TPR * P) {
        float sum[P][8] = {};
        // a slot that takes no part reads the first row and counts nothing; a piece
        // past the row is its last one again
        for (int j0 = 0; j0 < p.k; j0 += B) {
            i32x4 v[B][P];
            float wj[B];
            bool in[B];
            int from[B];
#pragma unroll
            for (int i = 0; i < B; ++i)
                from[i] = place[min(j0 + i, p.k - 1)];
            if (w) {
#pragma unroll
                for (int i = 0; i < B; ++i)
                    wj[i] = w[min(j0 + i, p.k - 1)];
            } else {
#pragma unroll
                for (int i = 0; i < B; ++i)
                    wj[i] = 1.f;
            }
#pragma unroll
            for (int i = 0; i < B; ++i) {
                in[i] = j0 + i < p.k && (uint32_t)from[i] < (uint32_t)p.S;
                const uint16_t* y = p.Y + (in[i] ? from[i] : 0) * p.ldy;
#pragma unroll
                for (int u = 0; u < P; ++u)
                    v[i][u] = load_piece_nt(y + min((q + u * TPR) * 8, p.D - 8));
            }
#pragma unroll
            for (int i = 0; i < B; ++i)
                if (in[i])
#pragma unroll
                    for (int u = 0; u < P; ++u) {
                        float y[8];
                        unpack8(v[i][u], y);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            sum[u][e] = fmaf(wj[i], y[e], sum[u][e]);
                    }
        }
#pragma unroll
        for (int u = 0; u < P; ++u)
            if (q + u * TPR < p.pieces)
                store_piece(out + min((q + u * TPR) * 8, p.D - 8), pack8(sum[u]));
    }
}

// One wave a slot (t, j): dY[place] = w dout[t], dw = <dout[t], Y[place]>.  The
// slots of a token share a workgroup, and its dout comes from the L1.
template <bool NT>
__global__ __launch_bounds__(256) void group_combine_grad_kernel(CombineArgs p, uint32_t k_mul)
{
    const int s = my_row<64>();
    const int lane = threadIdx.x & 63;
    if (s >= p.T * p.k)
        return;
    const int t = k_mul ? (int)__umulhi((uint32_t)s, k_mul) : s;
    const int at = p.place[s];
    if ((uint32_t)at >= (uint32_t)p.S) {
        if (p.dweights && lane == 0)
            p.dweights[s] = 0.f;
        return;
    }
    const float w = p.weights ? p.weights[t * p.ldw + (s - t * p.k)] : 1.f;
    const uint16_t* dout = p.dout + t * p.lddo;
    const uint16_t* y = p.Y + at * p.ldy;
    uint16_t* dy = p.dY ? p.dY + at * p.lddy : nullptr;
    float sum = 0.f;
    if (p.D < 8) {
        if (lane < p.D) {
            const float d = bf16_to_f32(dout[lane]);
            if (p.dweights)
                sum = d * bf16_to_f32(y[lane]);
            if (dy)
                dy[lane] = bf16_rne(w * d);
        }
    } else {
        for (int q = lane; q < p.pieces; q += 64) {
            // (the last piece counts what the one before it has not)
            const int c = min(q * 8, p.D - 8);
            float d[8], r[8];
            unpack8(load_piece(dout + c), d);
            if (p.dweights) {
                unpack8(load_piece_nt(y + c), r);
                float part = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    part = c + i >= q * 8 ? fmaf(d[i], r[i], part) : part;
                sum += part;
            }
            if (dy) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    r[i] = w * d[i];
                store_sorted<NT>(dy + c, pack8(r));
            }
        }
    }
    if (!p.dweights)
        return;
#pragma unroll
    for (int d = 32; d; d >>= 1)
        sum += __shfl_xor(sum, d);
    if (lane == 0)
        p.dweights[s] = sum;
}


template <class Args, class... More>
hipError_t launch(void (*kernel)(Args, More...), int64_t grid, int block, hipStream_t s, Args a, More... more)
{
    void* list[] = {&a, &more...};
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3((unsigned)grid), dim3((unsigned)block),
                           list, 0, s);
}

}  // namespace

SortPlan sort_plan(int64_t S, int64_t groups)
{
    SortPlan p = {S, 1, 0};
    if (S > kSortOne) {
        // chunks of 1024 to 8192 slots, fewer than kSortScan of them if that does
        p.chunk = std::min<int64_t>(kSortMost, cdiv(cdiv(S, kSortScan - 1), 1024) * 1024);
        p.chunks = cdiv(S, p.chunk);
        p.bytes = (p.chunks + 1) * (groups + 1) * 4;
    }
    return p;
}

hipError_t group_sort(const SortCall& c)
{
    const SortPlan pl = sort_plan(c.T * c.k, c.groups);
    SortArgs a;
    a.ids = c.ids;
    a.ld = c.ld_ids;
    a.k = (int)c.k;
    a.k_mul = divide_by(c.k);
    a.dense = c.ld_ids == c.k;
    a.S = (int)(c.T * c.k);
    a.groups = (int)c.groups;
    a.chunk = (int)pl.chunk;
    a.counts = pl.chunks > 1 ? static_cast<int*>(c.ws) : nullptr;
    a.offsets = c.offsets;
    a.order = c.order;
    a.place = c.place;
    a.totals = nullptr;
    if (pl.chunks > 1) {
        hipError_t e = launch(group_count_kernel, pl.chunks, 1024, c.stream, a);
        if (e == hipSuccess && pl.chunks >= kSortScan) {
            a.totals = a.counts + pl.chunks * (c.groups + 1);
            e = launch(group_scan_kernel, c.groups + 1, 256, c.stream, a, (int)pl.chunks);
        }
        if (e != hipSuccess)
            return e;
    }
    return launch(group_place_kernel, pl.chunks, 1024, c.stream, a);
}

// Stored past the caches: see kCacheBytes.  Not where rows start inside 64 bytes, whose
// ends would go to memory as parts of lines (8192 x 8 rows of 2056: gather 78 us, 66 through
// the caches, gradient 134 and 116; past 1 GB, 7992 a row, 285 and 293, 509 and 537).
static bool past_caches(const void* rows, int64_t pitch_b, int64_t bytes)
{
    return bytes >= kCacheBytes && ((uintptr_t)rows | (uint64_t)pitch_b) % 64 == 0;
}

hipError_t group_gather(const GatherCall& c)
{
    GatherArgs a;
    a.X = c.X;
    a.ldx_b = c.ldx_b;
    a.place = c.place;
    a.T = (int)c.T;
    a.k = (int)c.k;
    a.S = (int)(c.T * c.k);
    a.row_b = (int)c.row_b;
    a.pieces = (int)cdiv(c.row_b, 16);
    a.Xs = c.Xs;
    a.ldxs_b = c.ldxs_b;
    if (a.pieces <= 64)
        return launch(group_gather_kernel<64, false>, cdiv(c.T, 4), 256, c.stream, a);
    if (!past_caches(c.Xs, c.ldxs_b, c.T * c.k * c.row_b))
        return launch(group_gather_kernel<256, false>, c.T, 256, c.stream, a);
    return launch(group_gather_kernel<256, true>, c.T, 256, c.stream, a);
}

hipError_t group_pick(const PickCall& c)
{
    PickArgs a;
    a.X = c.X;
    a.ldx = c.ldx;
    a.offsets = c.offsets;
    a.order = c.order;
    a.k_mul = divide_by(c.k);
    a.S = (int)c.S;
    a.groups = (int)c.groups;
    a.K = (int)c.K;
    a.Xs = c.Xs;
    if (c.K <= 1024)
        return launch(group_pick_kernel<64>, cdiv(c.S, 4), 256, c.stream, a);
    return launch(group_pick_kernel<256>, c.S, 256, c.stream, a);
}

static CombineArgs combine_args(const CombineCall& c)
{
    CombineArgs a;
    a.Y = c.Y;
    a.ldy = c.ldy;
    a.place = c.place;
    a.weights = c.weights;
    a.ldw = c.ld_weights;
    a.T = (int)c.T;
    a.k = (int)c.k;
    a.S = (int)(c.T * c.k);
    a.D = (int)c.D;
    a.pieces = (int)cdiv(c.D, 8);
    a.out = c.out;
    a.ldo = c.ldo;
    a.dout = c.dout;
    a.lddo = c.lddo;
    a.dY = c.dY;
    a.lddy = c.lddy;
    a.dweights = c.dweights;
    return a;
}

hipError_t group_combine(const CombineCall& c)
{
    const CombineArgs a = combine_args(c);
    if (a.pieces <= 64)
        return c.k <= 2 ? launch(group_combine_kernel<64, 2, 1>, cdiv(c.T, 4), 256, c.stream, a)
                        : launch(group_combine_kernel<64, 8, 1>, cdiv(c.T, 4), 256, c.stream, a);
    return c.k <= 2   ? launch(group_combine_kernel<256, 2, 2>, c.T, 256, c.stream, a)
           : c.k <= 4 ? launch(group_combine_kernel<256, 4, 2>, c.T, 256, c.stream, a)
                      : launch(group_combine_kernel<256, 8, 1>, c.T, 256, c.stream, a);
}

hipError_t group_combine_grad(const CombineCall& c)
{
    if (!past_caches(c.dY, c.lddy * 2, c.T * c.k * c.D * 2))
        return launch(group_combine_grad_kernel<false>, cdiv(c.T * c.k, 4), 256, c.stream, combine_args(c),
                      divide_by(c.k));
    return launch(group_combine_grad_kernel<true>, cdiv(c.T * c.k, 4), 256, c.stream, combine_args(c),
                  divide_by(c.k));
}

}  // namespace dg
