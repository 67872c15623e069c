// The linear head's losses: row selection, targets, the joins of the partial
// log-sum-exps, the sparse columns of the gradient, and the launches around
// the products of loss_kernels.hpp.
//
// Rows that are out (ignored labels, rows without a target) leave the
// products: the kept rows of X are copied together first (memory-bound, T D
// values against T V D multiply-adds), which skips the ignored rows' work and
// keeps whatever their X holds, NaN included, out of every sum over rows.
// How many are kept is known on the device only: grids are sized for every
// row and surplus workgroups return.
#include "loss.hpp"

#include <math.h>
#include <string.h>

#include <tuple>

#include "internal.hpp"
#include "loss_kernels.hpp"

namespace dg {
namespace {

constexpr int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
constexpr int64_t cdiv(int64_t x, int64_t a) { return (x + a - 1) / a; }

// Rows counted per entry of the chunk table, and up to how many rows one
// workgroup counts the rows in front of it by itself (32 KiB of labels, L2).
constexpr int kChunk = 1024;
constexpr int64_t kOwnCount = 4096;
constexpr int kSelRows = 4;      // rows one workgroup of the selection moves, one a wave

// dW of more rows than one tile wants them in the order of their target's group
// of columns (kRestCols).  Up to kOwnCount rows each workgroup counts, for its
// rows, those that come before; of more, a table holds how many rows of each chunk
// of kOwnCount lie in each group, and what lies in front of those (place).
constexpr int kGroupPass = 4096; // groups one workgroup of that count holds in LDS

// Row state: out, kept, or kept with a target outside the vocabulary (loss
// and gradient NaN).
enum { ROW_OUT = 0, ROW_KEPT = 1, ROW_BAD = 2 };

struct RowSource {
    const int64_t* labels;       // cross entropy
    int64_t ignore_index, V;
    const int* flag;             // distillation: [T][2] row state, lead column
};

__device__ __forceinline__ int row_state(const RowSource& s, int64_t t, int& label)
{
    if (s.flag) {
        const int f = s.flag[2 * t];
        label = s.flag[2 * t + 1];
        return f;
    }
    const int64_t y = s.labels[t];
    if (y == s.ignore_index)
        return ROW_OUT;
    const bool in = y >= 0 && y < s.V;
    label = in ? (int)y : -1;
    return in ? ROW_KEPT : ROW_BAD;
}

__device__ __forceinline__ int wave_sum(int x)
{
#pragma unroll
    for (int d = 32; d; d >>= 1)
        x += __shfl_xor(x, d);
    return x;
}
__device__ __forceinline__ float wave_sum(float x)
{
#pragma unroll
    for (int d = 32; d; d >>= 1)
        x += __shfl_xor(x, d);
    return x;
}
__device__ __forceinline__ float wave_max(float x)
{
#pragma unroll
    for (int d = 32; d; d >>= 1)
        x = fmaxf(x, __shfl_xor(x, d));
    return x;
}

// What rounding took from a value kept in bf16.
__device__ __forceinline__ float bf16_rest(float x) { return x - bf16_to_f32(bf16_rne(x)); }

// Kept rows in [t0, t1), counted by a workgroup of 256 threads.
__device__ __forceinline__ int count_kept(const RowSource& src, int64_t t0, int64_t t1, int* red)
{
    int c = 0, label;
    for (int64_t t = t0 + threadIdx.x; t < t1; t += 256)
        c += row_state(src, t, label) != ROW_OUT;
    c = wave_sum(c);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = c;
    __syncthreads();
    return red[0] + red[1] + red[2] + red[3];
}

// The group of a kept row's target (no target in the vocabulary: the first).
__device__ __forceinline__ int row_group(int label) { return max(label, 0) / kRestCols; }

// place[group][chunk]: kept rows of one chunk of kOwnCount rows in each group.
// Integer sums in LDS: their order does not matter.
__global__ __launch_bounds__(1024) void loss_group_count_kernel(RowSource src, int64_t T, int groups, int* place)
{
    __shared__ int found[kGroupPass];
    const int64_t t0 = (int64_t)blockIdx.x * kOwnCount, t1 = min(T, t0 + kOwnCount);
    const int g0 = blockIdx.y * kGroupPass, n = min(groups - g0, kGroupPass);
    for (int g = threadIdx.x; g < n; g += 1024)
        found[g] = 0;
    __syncthreads();
    for (int64_t t = t0 + threadIdx.x; t < t1; t += 1024) {
        int label;
        const bool kept = row_state(src, t, label) != ROW_OUT;
        const int g = row_group(label) - g0;
        if (kept && g >= 0 && g < n)
            atomicAdd(&found[g], 1);
    }
    __syncthreads();
    for (int g = threadIdx.x; g < n; g += 1024)
        place[(int64_t)(g0 + g) * gridDim.x + blockIdx.x] = found[g];
}

// The counts -> what lies in front of them, by one workgroup, 8 a thread at a
// time; and the groups' first rows.
__global__ __launch_bounds__(1024) void loss_group_place_kernel(int* place, int64_t n, int chunks, int* group,
                                                                int groups, int* n_kept)
{
    __shared__ int sums[16];
    int before = 0;
    for (int64_t i0 = 0; i0 < n; i0 += 8192) {
        int v[8], mine = 0;
        const int64_t i = i0 + (int64_t)threadIdx.x * 8;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            v[u] = i + u < n ? place[i + u] : 0;
            mine += v[u];
        }
        int run = mine;                        // up to and with this lane
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(run, d);
            run += (int)(threadIdx.x & 63) >= d ? o : 0;
        }
        if ((threadIdx.x & 63) == 63)
            sums[threadIdx.x >> 6] = run;
        __syncthreads();
        int at = before + run - mine;
#pragma unroll
        for (int w = 0; w < 16; ++w) {
            at += w < (int)(threadIdx.x >> 6) ? sums[w] : 0;
            before += sums[w];
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (i + u < n) {
                place[i + u] = at;
                if ((i + u) % chunks == 0)
                    group[(i + u) / chunks] = at;
            }
            at += v[u];
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        group[groups] = before;
        *n_kept = before;
    }
}

__global__ __launch_bounds__(256) void loss_count_kernel(RowSource src, int64_t T, int* chunks)
{
    __shared__ int red[4];
    const int64_t t0 = (int64_t)blockIdx.x * kChunk;
    const int c = count_kept(src, t0, min(T, t0 + kChunk), red);
    if (threadIdx.x == 0)
        chunks[blockIdx.x] = c;
}

struct SelectArgs {
    RowSource src;
    int64_t T;
    const int* chunks;           // kept rows per kChunk rows, or null: count them here
    const uint8_t* X;
    int64_t ldx_b;
    uint8_t* Xc;                 // [n][D] compact
    int64_t row_b;               // D * 2
    int* n_kept;
    int* map;                    // compact row -> row
    int* pos;                    // row -> compact row, -1: out
    RowInfo* rows;
    // forward
    float* zlabel;
    float* loss;
    float* lse_out;
    // gradient
    const float* loss_in;
    const float* lse_in;
    const float* dloss;
    int64_t dloss_stride;
    float scale, z_loss;
    // BY_GROUP
    const int* place;            // [groups][chunks], or null: count them here
    int n_chunks, groups;
    int* group;                  // [groups + 1]: first rows
    uint8_t* rest;               // G's columns of rests
    int64_t rest_b;              // G's pitch
};

// 4 rows a workgroup: how many kept rows lie in front of them, each row's
// place, what the row's gradient needs, and the copy of the kept rows.  BY_GROUP:
// in the order of the targets' groups, and the rests of G there; without a table
// the workgroups past those of the rows find the groups' first rows, four each.
template <bool BY_GROUP>
__global__ __launch_bounds__(256) void loss_select_kernel(SelectArgs p)
{
    __shared__ int red[4];
    __shared__ int place[kSelRows];
    __shared__ int front[4][kSelRows + 1];
    __shared__ uint32_t left[kSelRows];      // the row's rest, bf16, and its column in the group
    __shared__ int column[kSelRows];
    const int64_t t0 = (int64_t)blockIdx.x * kSelRows;
    int before = 0;
    if constexpr (BY_GROUP) {
        // rows that come before (group, row) of each of the four
        const int64_t row_blocks = (p.T + kSelRows - 1) / kSelRows;
        const bool firsts = (int64_t)blockIdx.x >= row_blocks;
        int g[kSelRows], c[kSelRows + 1] = {0, 0, 0, 0, 0};
        int64_t upto[kSelRows];
#pragma unroll
        for (int r = 0; r < kSelRows; ++r) {
            if (firsts) {
                g[r] = (int)((int64_t)blockIdx.x - row_blocks) * kSelRows + r;
                upto[r] = 0;
            } else {
                int label = -1;
                if (t0 + r < p.T)
                    row_state(p.src, t0 + r, label);
                g[r] = row_group(label);
                upto[r] = t0 + r;
            }
        }
        const int64_t c0 = p.place ? t0 / kOwnCount * kOwnCount : 0, c1 = p.place ? t0 + kSelRows : p.T;
        const int64_t c_end = min(p.T, c1);
        for (int64_t t1 = c0 + threadIdx.x; t1 - threadIdx.x < c_end; t1 += 1024) {
            int at[4];                       // four rows a lane at once; -1: none
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t t = t1 + u * 256;
                int label = -1;
                const bool kept = t < c_end && row_state(p.src, t, label) != ROW_OUT;
                at[u] = kept ? row_group(label) : -1;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t t = t1 + u * 256;
#pragma unroll
                for (int r = 0; r < kSelRows; ++r)
                    c[r] += __popcll(__ballot((at[u] == g[r] && t < upto[r]) ||
                                              (!p.place && at[u] >= 0 && at[u] < g[r])));
                c[kSelRows] += __popcll(__ballot(at[u] >= 0));
            }
        }
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int r = 0; r <= kSelRows; ++r)
                front[threadIdx.x >> 6][r] = c[r];
        __syncthreads();
        const int r = threadIdx.x;
        if (firsts) {
            const int at = (int)((int64_t)blockIdx.x - row_blocks) * kSelRows + r;
            if (r < kSelRows && at <= p.groups)
                p.group[at] = front[0][r] + front[1][r] + front[2][r] + front[3][r];
            return;
        }
        if (r < kSelRows) {
            before = front[0][r] + front[1][r] + front[2][r] + front[3][r];
            if (p.place)
                before += p.place[(r == 0 ? g[0] : r == 1 ? g[1] : r == 2 ? g[2] : g[3]) * (int64_t)p.n_chunks +
                                  t0 / kOwnCount];
        }
        if (r == 0 && blockIdx.x == 0 && !p.place)
            *p.n_kept = front[0][kSelRows] + front[1][kSelRows] + front[2][kSelRows] + front[3][kSelRows];
    } else if (p.chunks) {
        const int64_t c0 = t0 / kChunk;
        int c = 0;
        for (int64_t i = threadIdx.x; i < c0; i += 256)
            c += p.chunks[i];
        c = wave_sum(c);
        if ((threadIdx.x & 63) == 0)
            red[threadIdx.x >> 6] = c;
        __syncthreads();
        before = red[0] + red[1] + red[2] + red[3];
        before += count_kept(p.src, c0 * kChunk, t0, red);
    } else {
        before = count_kept(p.src, 0, t0, red);
    }
    if (threadIdx.x < 64) {
        const int64_t t = t0 + threadIdx.x;
        const bool mine = threadIdx.x < kSelRows && t < p.T;
        int label = -1;
        const int st = mine ? row_state(p.src, t, label) : ROW_OUT;
        const uint64_t kept = __ballot(st != ROW_OUT);
        const int at = BY_GROUP ? before : before + __popcll(kept & ((1ull << threadIdx.x) - 1));
        if (mine) {
            place[threadIdx.x] = st != ROW_OUT ? at : -1;
            p.pos[t] = st != ROW_OUT ? at : -1;
            if (st != ROW_OUT) {
                RowInfo ri = {0.f, 0.f, 0.f, label};
                if (p.lse_in) {
                    const float lse = p.lse_in[t];
                    const float g = p.dloss[t * p.dloss_stride] * p.scale;
                    const float extra = 2.f * p.z_loss * lse;
                    ri.lse2 = lse * kLog2e;
                    ri.a = g * (1.f + extra);
                    if (p.loss_in) {
                        // p - 1 = expm1(-nll), exact for p near 1 too
                        const float nll = p.loss_in[t] - p.z_loss * lse * lse;
                        ri.b = g * (expm1f(-nll) + extra * expf(-nll));
                    } else {
                        ri.label = -1;         // distillation: sparse columns come after
                        ri.b = g;
                    }
                    if (st == ROW_BAD)
                        ri.a = ri.b = NAN;
                    if (BY_GROUP)
                        left[threadIdx.x] = ri.label >= 0 ? bf16_rne(bf16_rest(ri.b)) : 0u;
                }
                if (p.zlabel)
                    p.zlabel[at] = NAN;        // stays for a target outside the vocabulary
                p.rows[at] = ri;
                p.map[at] = (int)t;
            } else if (p.loss) {
                p.loss[t] = 0.f;
                p.lse_out[t] = 0.f;
            }
        }
        if (BY_GROUP && mine)
            column[threadIdx.x] = max(label, 0) % kRestCols;
        if (!BY_GROUP && threadIdx.x == 0 && t0 + kSelRows >= p.T)
            *p.n_kept = before + __popcll(kept);
    }
    __syncthreads();
    const int r = threadIdx.x >> 6;
    if (t0 + r >= p.T || place[r] < 0)
        return;
    if constexpr (BY_GROUP) {
        // (distillation's come with its sparse columns)
        const int lane = threadIdx.x & 63, c = column[r];
        const uint32_t v = left[r] << (c & 1) * 16;
        const uint2 w = make_uint2(c / 4 == lane && !(c & 2) ? v : 0u, c / 4 == lane && c & 2 ? v : 0u);
        *reinterpret_cast<uint2*>(p.rest + place[r] * p.rest_b + lane * 8) = w;
    }
    const uint8_t* from = p.X + (t0 + r) * p.ldx_b;
    uint8_t* to = p.Xc + place[r] * p.row_b;
    for (int64_t b = (threadIdx.x & 63) * 16; b < p.row_b; b += 4096) {
        i32x4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (b + u * 1024 < p.row_b)
                v[u] = *reinterpret_cast<const i32x4*>(from + b + u * 1024);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (b + u * 1024 < p.row_b)
                *reinterpret_cast<i32x4*>(to + b + u * 1024) = v[u];
    }
}

struct JoinArgs {
    const float2* part;          // [tiles_n][ldpart]
    int64_t ldpart;
    int tiles_n;
    const int* n_kept;
    const int* map;
    RowSource src;               // few rows: their states
    int few;                     // few rows: how many; none moved
    const float* zlabel;
    float scale, z_loss;         // scale without its sign
    float* loss;
    float* lse;
};

// Joins the tile columns' (reference, sum) pairs of one row by a workgroup of
// THREADS, R rows in all; red: a pair of LDS for each thread.
template <int R, int THREADS = 256>
__device__ __forceinline__ float2 join_row(const JoinArgs& p, int row, bool valid, float2* red)
{
    constexpr int Q = THREADS / R;
    const int q = threadIdx.x / R;
    float2 acc = make_float2(-INFINITY, 0.f);
    if (valid)
        for (int t = q; t < p.tiles_n; t += 4 * Q) {
            float2 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                v[u] = t + u * Q < p.tiles_n ? p.part[(int64_t)(t + u * Q) * p.ldpart + row]
                                             : make_float2(-INFINITY, 0.f);
            acc = lse_merge(acc, lse_merge(lse_merge(v[0], v[1]), lse_merge(v[2], v[3])));
        }
    red[threadIdx.x] = acc;
    __syncthreads();
#pragma unroll
    for (int half = Q / 2; half; half /= 2) {
        if (q < half)
            red[threadIdx.x] = lse_merge(red[threadIdx.x], red[threadIdx.x + half * R]);
        __syncthreads();
    }
    return red[threadIdx.x % R];
}

// lse and the label's negative log-probability from the joined pair and the
// label's sum over d.  others = (reference + log2 sum) ln 2; its distance to the
// label's z from the sum itself, so that what they share cancels before it is
// rounded.
__device__ __forceinline__ void lse_finish(float2 v, float xl, float scale, float& nll, float& lse)
{
    constexpr float kLn2 = 0.69314718055994530942f;
    const float logs = logf(v.y), zl = xl * scale;
    const bool none = v.x == -INFINITY && v.y == 0.f;     // one column: no others
    const float others = none ? -INFINITY : fmaf(v.x, kLn2, logs);
    const float d = none ? -INFINITY : fmaf(fmaf(-xl, scale * kLog2e, v.x), kLn2, logs);
    nll = fmaxf(d, 0.f) + log1pf(expf(-fabsf(d))) + (d != d ? d : 0.f);
    // no label column (NaN), or one of z = -inf: lse of all that was summed
    lse = d != d || zl == -INFINITY ? others : zl + nll;
}

// Cross entropy's last step, and distillation's for many rows (loss: the lead's
// negative log-probability then).  R rows a workgroup, 256 / R threads a row: 16
// rows read whole 128-byte lines of the table where there are many; few rows
// get all threads (one row of 393 pairs: 16 threads took 11 us, 256 take 4).
template <int R>
__global__ __launch_bounds__(256) void loss_join_kernel(JoinArgs p)
{
    __shared__ float2 red[256];
    const int n = p.few ? p.few : *p.n_kept;
    const int row = blockIdx.x * R + threadIdx.x % R;
    if (blockIdx.x * R >= n)
        return;
    const float2 v = join_row<R>(p, row, row < n, red);
    if (threadIdx.x >= R || row >= n)
        return;
    float xl = p.zlabel[row];
    if (p.few) {
        int label;
        const int st = row_state(p.src, row, label);
        if (st == ROW_OUT) {
            p.loss[row] = p.lse[row] = 0.f;
            return;
        }
        if (st == ROW_BAD)
            xl = NAN;
    }
    float nll, l;
    lse_finish(v, xl, p.scale, nll, l);
    const int t = p.few ? row : p.map[row];
    p.loss[t] = nll + p.z_loss * l * l;
    p.lse[t] = l;
}

// ---------------------------------------------------------------------------
// Distillation targets.  One wave a row: q = softmax(scale * teacher) over the
// row's filled slots; slots that name one column together count once, in the
// first of them (the leader); the row's lead is the column of the largest q.
// For a leader, rest = 1 - (its q) is the sum of the other slots' q, so that
// p - q of a column that both sides are sure of keeps its digits.  With logp the lead
// is the column of the largest |p - q|.
struct TargetArgs {
    const int64_t* index;
    const float* teacher;
    int64_t ld_index, ld_teacher, T, V;
    int k;
    float scale;
    float* q;                    // [T][k]: q of the slot, 0 where it is empty
    float* qsum;                 // [T][k]: q of the slot's column, all its slots
    float* rest;                 // [T][k]: 1 - qsum
    int* leader;                 // [T][k]: column, or -1: empty or not the first
    int* flag;                   // [T][2]: row state, lead column
    const float* logp;           // gradient, dW of more rows: [T][k], else null
};

// p - q with q = 1 - rest: near p = q = 1 both sides are taken from 1.
__device__ __forceinline__ float target_dz(float logp, float qsum, float rest)
{
    return rest < 0.5f ? expm1f(logp) + rest : expf(logp) - qsum;
}

// The wave's largest value and its slot, the lowest among equals.
__device__ __forceinline__ void first_largest(float& best, int& slot)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const float ob = __shfl_xor(best, d);
        const int os = __shfl_xor(slot, d);
        if (ob > best || (ob == best && os < slot)) {
            best = ob;
            slot = os;
        }
    }
}

__global__ __launch_bounds__(64) void loss_target_kernel(TargetArgs p)
{
    __shared__ __attribute__((aligned(16))) int idx[kMaxLossSlots];
    __shared__ __attribute__((aligned(16))) float qs[kMaxLossSlots];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x;
    const int k4 = (p.k + 3) / 4;
    if (lane < 4 * k4 - p.k) {               // fill the last group of four
        idx[p.k + lane] = -2;
        qs[p.k + lane] = 0.f;
    }
    float m = -INFINITY;
    bool bad = false, any = false;
    for (int j = lane; j < p.k; j += 64) {
        const int64_t i = p.index[t * p.ld_index + j];
        const float z = p.teacher[t * p.ld_teacher + j] * p.scale;
        const bool filled = i >= 0 && p.teacher[t * p.ld_teacher + j] != -INFINITY;
        const bool in = filled && i < p.V;
        any |= filled;
        bad |= filled && (!in || !(fabsf(z) < INFINITY));
        idx[j] = in ? (int)i : -1;
        qs[j] = filled ? z : -INFINITY;
        if (in)
            m = fmaxf(m, z);
    }
    m = wave_max(m);
    any = __any(any);
    bad = __any(bad);
    __syncthreads();
    float s = 0.f;
    for (int j = lane; j < p.k; j += 64)
        s += idx[j] >= 0 ? expf(qs[j] - m) : 0.f;
    s = wave_sum(s);
    __syncthreads();
    for (int j = lane; j < p.k; j += 64)
        qs[j] = idx[j] >= 0 ? expf(qs[j] - m) / s : 0.f;
    __syncthreads();
    // the lead: the largest q, the lowest slot among equals
    float best = -1.f;
    int slot = p.k;
    for (int j = lane; j < p.k; j += 64)
        if (idx[j] >= 0 && qs[j] > best) {
            best = qs[j];
            slot = j;
        }
    first_largest(best, slot);
    if (lane == 0) {
        p.flag[2 * t] = !any ? ROW_OUT : bad ? ROW_BAD : ROW_KEPT;
        p.flag[2 * t + 1] = slot < p.k ? idx[slot] : -1;
    }
    if (p.logp) {
        best = -1.f;
        slot = p.k;
    }
    for (int j = lane; j < p.k; j += 64) {
        const int me = idx[j];
        bool first = me >= 0;
        float rest = 0.f, sum = 0.f;
        // every slot against every other, four to an LDS read (one at a time,
        // 106 slots took 21 us)
#pragma unroll 4
        for (int i = 0; i < k4; ++i) {
            const i32x4 c = reinterpret_cast<const i32x4*>(idx)[i];
            const f32x4 v = reinterpret_cast<const f32x4*>(qs)[i];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const bool same = c[u] == me;
                const float x = v[u];
                first = first && !(same && 4 * i + u < j);
                rest += same ? 0.f : x;
                sum += same ? x : 0.f;
            }
        }
        p.q[t * p.k + j] = qs[j];
        p.qsum[t * p.k + j] = sum;
        p.rest[t * p.k + j] = rest;
        p.leader[t * p.k + j] = first ? me : -1;
        if (p.logp && first) {
            const float d = fabsf(target_dz(p.logp[t * p.k + j], sum, rest));
            if (d > best) {
                best = d;
                slot = j;
            }
        }
    }
    if (p.logp) {
        first_largest(best, slot);
        if (lane == 0)
            p.flag[2 * t + 1] = slot < p.k ? idx[slot] : -1;
    }
}

struct PickArgs {
    const uint8_t* W;
    int64_t ldw_b;
    const uint8_t* Xc;
    int64_t row_b;
    int64_t ldx_b;
    const int* pos;              // null: Xc is X itself
    const int64_t* index;
    int64_t ld_index, V;
    const float* teacher;
    int64_t ld_teacher;
    const float* q;
    const int* flag;
    int k;
    float scale;
    const float* zlabel;
    float* loss;                 // in: the lead's negative log-probability; out: the loss
    float* logp;                 // [T][k]
};

__device__ __forceinline__ float dot8(i32x4 a, i32x4 b, float s)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = (uint32_t)a[i], y = (uint32_t)b[i];
        s = fmaf(__uint_as_float(x << 16), __uint_as_float(y << 16), s);
        s = fmaf(__uint_as_float(x & 0xFFFF0000u), __uint_as_float(y & 0xFFFF0000u), s);
    }
    return s;
}

// The student's log-probabilities at a row's slots, and the row's loss: a
// workgroup a row, four slots at a time a wave, each a dot product of the row of
// X with the slot's row of W.  JOIN (few rows): the row's join here too, instead
// of in a launch of its own, and 16 waves instead of 4, as few workgroups leave
// the CUs to them (56 rows of 100 slots, D = 2656: 42 us with 4).
template <bool JOIN>
__global__ __launch_bounds__(JOIN ? 1024 : 256) void loss_pick_kernel(PickArgs p, JoinArgs jn)
{
    constexpr int THREADS = JOIN ? 1024 : 256;
    __shared__ float z[kMaxLossSlots];
    __shared__ float2 red[JOIN ? THREADS : 1];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // few rows: none moved
    const int at = p.pos ? p.pos[t] : p.flag[2 * t] == ROW_OUT ? -1 : (int)t;
    float* out = p.logp + t * p.k;
    if (at < 0) {
        for (int j = threadIdx.x; j < p.k; j += THREADS)
            out[j] = 0.f;
        if (JOIN && threadIdx.x == 0)
            p.loss[t] = jn.lse[t] = 0.f;
        return;
    }
    float2 joined = make_float2(0.f, 0.f);
    if constexpr (JOIN)
        joined = join_row<1, THREADS>(jn, (int)t, true, red);
    const uint8_t* x = p.Xc + at * p.ldx_b;
    const int lead = p.flag[2 * t + 1];
    for (int j0 = 4 * wave; j0 < p.k; j0 += THREADS / 16) {
        const uint8_t* w[4];
        int use[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t i = j0 + u < p.k ? p.index[t * p.ld_index + j0 + u] : -1;
            use[u] = i >= 0 && i < p.V;
            w[u] = p.W + (use[u] ? i : 0) * p.ldw_b;
        }
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        for (int64_t b = lane * 16; b < p.row_b; b += 1024) {
            const i32x4 xv = *reinterpret_cast<const i32x4*>(x + b);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                s[u] = dot8(xv, *reinterpret_cast<const i32x4*>(w[u] + b), s[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            s[u] = wave_sum(s[u]);
            if (lane == 0 && j0 + u < p.k)
                z[j0 + u] = s[u] * p.scale;
        }
    }
    __syncthreads();
    if (wave != 0)
        return;
    // the lead's own log-probability is the well-conditioned one of the join;
    // the others' follow from their distance to it
    const float xl = p.zlabel[at], zl = xl * fabsf(p.scale);
    float lead_nll;
    if constexpr (JOIN) {
        float lse;
        lse_finish(joined, lead >= 0 ? xl : NAN, jn.scale, lead_nll, lse);
        if (lane == 0)
            jn.lse[t] = lse;
    } else {
        lead_nll = p.loss[t];
    }
    float mx = -INFINITY;
    for (int j = lane; j < p.k; j += 64) {
        const int64_t i = p.index[t * p.ld_index + j];
        const float te = p.teacher[t * p.ld_teacher + j];
        if (i >= 0 && i < p.V && te != -INFINITY)
            mx = fmaxf(mx, te * p.scale);
    }
    mx = wave_max(mx);
    float es = 0.f;
    for (int j = lane; j < p.k; j += 64) {
        const int64_t i = p.index[t * p.ld_index + j];
        const float te = p.teacher[t * p.ld_teacher + j];
        if (i >= 0 && i < p.V && te != -INFINITY)
            es += expf(te * p.scale - mx);
    }
    const float log_es = logf(wave_sum(es));
    float part = 0.f;
    for (int j = lane; j < p.k; j += 64) {
        const int64_t i = p.index[t * p.ld_index + j];
        const float te = p.teacher[t * p.ld_teacher + j];
        if (i < 0 || te == -INFINITY) {
            out[j] = 0.f;
            continue;
        }
        const float lp = i >= p.V ? NAN : i == lead ? -lead_nll : (z[j] - zl) - lead_nll;
        out[j] = lp;
        const float qj = p.q[t * p.k + j];
        if (qj > 0.f)
            part += qj * ((te * p.scale - mx) - log_es - lp);
    }
    part = wave_sum(part);
    if (lane == 0)
        p.loss[t] = p.flag[2 * t] == ROW_BAD ? NAN : part;
}

// Distillation: the sparse columns of the gradient piece, p - q in place of
// p.  One wave a kept row.  What rounding them to bf16 takes away is kept for
// dX where it counts (lost).
struct SparseArgs {
    const int* n_kept;
    const int* map;
    const RowInfo* rows;
    const int* leader;
    const float *qsum, *rest, *logp;
    int k;
    int64_t v0, vp;
    uint16_t* G;
    int64_t ldg, half_b;         // half_b 0: G has one half
    float* lost;                 // [T][k]
    const int* flag;             // dW of more rows: the lead's column,
    uint16_t* lead_rest;         // and G's columns of rests, of the lead's group; else null
};
__global__ __launch_bounds__(256) void loss_sparse_kernel(SparseArgs p)
{
    const int row = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= *p.n_kept)
        return;
    const int64_t t = p.map[row];
    const float g = p.rows[row].b;
    constexpr int U = kMaxLossSlots / 64;
    const int lane = threadIdx.x & 63;
    int cols[U];
    float d[U], most = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int j = lane + 64 * u;
        const int64_t i = t * p.k + j;
        cols[u] = j < p.k ? p.leader[i] : -1;
        d[u] = cols[u] >= 0 ? target_dz(p.logp[i], p.qsum[i], p.rest[i]) : 0.f;
        most = fmaxf(most, fabsf(d[u]));
    }
    most = wave_max(most);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = t * p.k + lane + 64 * u, col = cols[u];
        if (col < p.v0 || col >= p.v0 + p.vp)
            continue;
        uint16_t* at = p.G + row * p.ldg + (col - p.v0);
        *at = bf16_rne(g * d[u]);
        if (p.half_b)
            at[p.half_b / 2] = bf16_rne(bf16_rest(g * d[u]));
        // (the row lies with its lead's group, whose other targets come for nothing)
        if (p.lead_rest && col / kRestCols == row_group(p.flag[2 * t + 1]))
            p.lead_rest[row * p.ldg + col % kRestCols] = bf16_rne(bf16_rest(g * d[u]));
        // Below 1 / (4 sqrt k) of the row's largest: all of them together hold at
        // most 1/16 of its square, and their roundings add 3 % to the error's
        // norm at most; each one more is a row of W to read.
        p.lost[i] = d[u] * d[u] * (16.f * p.k) >= most * most ? bf16_rest(g * d[u]) : 0.f;
    }
}

// dX: the sum of the K slices' planes in slice order, rounded once; zero for
// rows that are out.
// A row of dX is often little more than one or two columns' worth of W, the
// target's: what rounding G to bf16 took from those is added here in fp32, rest
// times the column's row of W.  (Without it the roundings of G and of dX
// together are 1.4 times the latter, and up to 2.5 times where one target
// makes up a row.)
struct DxArgs {
    const float* planes;
    DxSlices slices;
    const int* n_kept;
    int64_t ldplane;
    const int* pos;
    const RowInfo* rows;
    const uint16_t* W;
    int64_t ldw;
    int k;                       // distillation: slots, else 0
    const int* leader;
    const float* lost;
    uint16_t* dX;
    int64_t lddx, D;
    int vec;                     // dX's rows start on 8 bytes
};
// P > 1: a workgroup takes 1024 / P columns of a row, and P threads share the
// planes of each four of them (few rows in many planes: 48 x 2048 in 24 took 14
// us by one thread, 56 x 2656 takes 4.9 by eight).  P = 1: a workgroup a row (4096
// x 4096 in 2 planes takes 28 us; 39 where 1024 columns were a workgroup each,
// which all read the row's targets again).
template <int P>
__global__ __launch_bounds__(256) void loss_dx_kernel(DxArgs p)
{
    constexpr int QUADS = 256 / P;
    __shared__ int col[kMaxLossSlots];
    __shared__ float rest[kMaxLossSlots];
    __shared__ int used[4];
    __shared__ f32x4 sums[P > 1 ? 256 : 1];
    const int blocks = P > 1 ? (int)((p.D + 4 * QUADS - 1) / (4 * QUADS)) : 1;
    const int64_t t = blockIdx.x / blocks;
    const int at = p.pos[t];
    int n = 0;
    if (at >= 0) {
        if (p.k == 0) {
            const RowInfo ri = p.rows[at];
            if (threadIdx.x == 0) {
                col[0] = ri.label;
                rest[0] = bf16_rest(ri.b);
            }
            n = ri.label >= 0;
        } else {
            // the slots with something lost, in slot order
            const int j = threadIdx.x;
            const int c = j < p.k ? p.leader[t * p.k + j] : -1;
            const float r = c >= 0 ? p.lost[t * p.k + j] : 0.f;
            const uint64_t has = __ballot(r != 0.f);
            if ((j & 63) == 0)
                used[j >> 6] = __popcll(has);
            __syncthreads();
            int before = 0;
            for (int w = 0; w < 4; ++w) {
                before += w < (j >> 6) ? used[w] : 0;
                n += used[w];
            }
            if (r != 0.f) {
                const int to = before + __popcll(has & ((1ull << (j & 63)) - 1));
                col[to] = c;
                rest[to] = r;
            }
        }
    }
    __syncthreads();
    const int part = threadIdx.x / QUADS;
    const int kept = *p.n_kept, slices = p.slices.count(kept);
    const int64_t plane = kept * p.ldplane;
    auto columns = [&](int64_t d) {
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
        if (at >= 0 && d < p.D) {
            const float* from = p.planes + at * p.ldplane + d;
            for (int i = part; i < slices; i += 4 * P) {
                f32x4 v[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    v[u] = i + u * P < slices ? *reinterpret_cast<const f32x4*>(from + (i + u * P) * plane)
                                              : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    s += v[u];
            }
            for (int i = part; i < n; i += 4 * P) {
                uint2 w[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (i + u * P < n)
                        w[u] = *reinterpret_cast<const uint2*>(p.W + col[i + u * P] * p.ldw + d);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (i + u * P >= n)
                        continue;
                    const float r = rest[i + u * P];
                    s[0] = fmaf(r, __uint_as_float(w[u].x << 16), s[0]);
                    s[1] = fmaf(r, __uint_as_float(w[u].x & 0xFFFF0000u), s[1]);
                    s[2] = fmaf(r, __uint_as_float(w[u].y << 16), s[2]);
                    s[3] = fmaf(r, __uint_as_float(w[u].y & 0xFFFF0000u), s[3]);
                }
            }
        }
        if constexpr (P > 1) {
            sums[threadIdx.x] = s;
            __syncthreads();
            if (part != 0)
                return;
            for (int u = 1; u < P; ++u)
                s += sums[threadIdx.x + u * QUADS];
        }
        if (d >= p.D)
            return;
        const float s0 = s[0], s1 = s[1], s2 = s[2], s3 = s[3];
        const uint16_t o[4] = {bf16_rne(s0), bf16_rne(s1), bf16_rne(s2), bf16_rne(s3)};
        uint16_t* to = p.dX + t * p.lddx + d;
        if (p.vec) {
            *reinterpret_cast<uint2*>(to) =
                make_uint2((uint32_t)o[0] | (uint32_t)o[1] << 16, (uint32_t)o[2] | (uint32_t)o[3] << 16);
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                to[u] = o[u];
        }
    };
    // one group of columns a workgroup where the planes are shared out, else
    // the whole row
    if constexpr (P > 1) {
        columns((int64_t)(blockIdx.x % blocks) * 4 * QUADS + threadIdx.x % QUADS * 4);
    } else {
        for (int64_t d = threadIdx.x * 4; d < p.D; d += 1024)
            columns(d);
    }
}

// ---------------------------------------------------------------------------
// Launches.
//
// Tile shapes.  kt and epi are what one round (every CU holding its fill of
// workgroups) measured on MI355X, in microseconds: kt for each 32 values of K,
// epi for the rest of a tile; kt1 where there is at most one workgroup a CU.
// Those of Few and Low are one guess for both, which dX's K slices alone go by:
// over 32 sizes of 16 to 64 rows dX then takes at most 8.5 % more than with the
// best of 12 numbers of slices, 3 % on average.  few_shape takes Slim, FewSlim and
// LowSlim by size, so they have none.
//   Big   taken where its tiles fill the CUs: twice the work of Tall, four
//         times that of the others, in 1.0 to 1.6 times their time (4095 x
//         50257 x 4096 logits: 1291 us; the next best shape 1414).
//   Line  for the logits: two stages of whole 128-byte lines of X and W.
//         Against four of 64 bytes (Mid): 597 x 50257 x 4096 298 us : 357,
//         100 x 50257 x 2048 41 : 46, 528 x 11007 x 1024 26 : 29.  Deeper
//         rings of 64-byte k-tiles gained nothing (31 to 33 us there).
//   Wide  for the logits where its tiles make one or two rounds: three stages of
//         whole lines, one workgroup a CU (400 x 11008 x 1024 forward 21.7 us
//         against 24.9 with Line, 300 x 30000 x 2048 48 against 55 with Big).
//   Deep  for the logits where its tiles make one round: four stages of whole
//         lines (215 x 9904 x 3832 forward 48 us against 54 with Wide).
//   Mid   for dX and dW, whose transposed operands are whole lines anyway.
//   Few, Low  up to 64 and 32 rows, where the product is a read of W: the
//         tile that just covers the rows keeps the most of it in flight (forward
//         of 48 x 50257 x 4096, whose W no cache holds: 82 us against 93 to 109 of
//         the others; 30 rows 78 against 79 to 87).
//   Slim, FewSlim, LowSlim  for up to 128, 64 and 32 rows of vocabularies that
//         make no full round of the 128-column tiles: 64 columns and deeper
//         rings (121 x 10399 x 3272 forward 41 us against 66, 48 x 16000 x 4096
//         31 : 41, 1 x 5000 x 4096 19 : 31).
using Big = LossShape<256, 256, 2, 4, 4, 64, 1>;
using Tall = LossShape<256, 128, 4, 2, 4, 64, 2>;
using Mid = LossShape<128, 128, 2, 2, 4, 64, 2>;
using Line = LossShape<128, 128, 2, 2, 2, 128, 2>;
using Wide = LossShape<128, 192, 2, 4, 3, 128, 2>;
using Deep = LossShape<128, 128, 2, 2, 4, 128, 1>;
using Slim = LossShape<128, 64, 2, 2, 6, 128, 1>;
using FewSlim = LossShape<64, 64, 1, 4, 4, 128, 2>;
using LowSlim = LossShape<32, 64, 1, 4, 5, 128, 2>;
using Few = LossShape<64, 128, 1, 4, 3, 128, 2>;
using Low = LossShape<32, 128, 1, 4, 3, 128, 2>;
enum { SHAPE_BIG = 0, SHAPE_TALL, SHAPE_MID, SHAPE_LINE, SHAPE_WIDE, SHAPE_DEEP, SHAPE_FEW, SHAPE_LOW,
       SHAPE_SLIM, SHAPE_FEW_SLIM, SHAPE_LOW_SLIM };
struct ShapeCost {
    int tm, tn, per_cu;
    double kt = 0.0, kt1 = 0.0, epi = 0.0;
};
constexpr ShapeCost kShapes[] = {{Big::TM, Big::TN, Big::PER_CU, 0.72, 0.72, 9.0},
                                 {Tall::TM, Tall::TN, Tall::PER_CU, 0.48, 0.48, 4.5},
                                 {Mid::TM, Mid::TN, Mid::PER_CU, 0.64, 0.50, 0.5},
                                 {Line::TM, Line::TN, Line::PER_CU, 0.56, 0.47, 1.0},
                                 {Wide::TM, Wide::TN, Wide::PER_CU, 0.36, 0.32, 2.0},
                                 {Deep::TM, Deep::TN, Deep::PER_CU, 0.30, 0.29, 2.0},
                                 {Few::TM, Few::TN, Few::PER_CU, 0.5, 0.4, 2.0},
                                 {Low::TM, Low::TN, Low::PER_CU, 0.5, 0.4, 2.0},
                                 {Slim::TM, Slim::TN, Slim::PER_CU},
                                 {FewSlim::TM, FewSlim::TN, FewSlim::PER_CU},
                                 {LowSlim::TM, LowSlim::TN, LowSlim::PER_CU}};
constexpr int kPlanCus = 256;            // the workspace must not depend on the device
constexpr double kLaunchUs = 5.0;        // a further launch, start to start
constexpr double kPlaneBytesPerUs = 2.0e6;

// Estimated time of a product of rows x cols outputs over k values.
double product_us(int shape, int64_t rows, int64_t cols, int64_t k, int splits, int cus)
{
    const ShapeCost& s = kShapes[shape];
    const int64_t items = cdiv(rows, s.tm) * cdiv(cols, s.tn) * splits;
    const int64_t kts = cdiv(cdiv(k, 32), splits);
    const int64_t full = items / (cus * s.per_cu), left = items % (cus * s.per_cu);
    return full * (kts * s.kt + s.epi) + (left ? kts * (left > cus ? s.kt : s.kt1) + s.epi : 0.0);
}

// Shape of the logits of few rows (one tile of them).
int few_shape(int64_t rows, int64_t cols, int cus)
{
    if (rows <= Low::TM)
        return cols <= (int64_t)LowSlim::TN * LowSlim::PER_CU * cus ? SHAPE_LOW_SLIM : SHAPE_LOW;
    if (rows <= Few::TM)
        return cols <= (int64_t)FewSlim::TN * FewSlim::PER_CU * cus ? SHAPE_FEW_SLIM : SHAPE_FEW;
    return cols <= (int64_t)Slim::TN * cus ? SHAPE_SLIM : cols <= (int64_t)Deep::TN * cus ? SHAPE_DEEP
                                                                                        : SHAPE_LINE;
}

// Shape of a product whose outputs are rows x cols, by the estimate.
int pick_shape(bool logits, int64_t rows, int64_t cols, int64_t k, int cus)
{
    constexpr int kLogits[] = {SHAPE_TALL, SHAPE_LINE, SHAPE_WIDE, SHAPE_DEEP};
    constexpr int kOthers[] = {SHAPE_TALL, SHAPE_MID};
    int best = SHAPE_BIG;
    for (const int* i = logits ? kLogits : kOthers; i != (logits ? kLogits + 4 : kOthers + 2); ++i)
        if (product_us(*i, rows, cols, k, 1, cus) < product_us(best, rows, cols, k, 1, cus))
            best = *i;
    return best;
}

// A product over a range of the vocabulary, v values of it: the first `main`
// of them with one shape, in whole rounds of tiles, and the rest with the shape that
// suits so few, when two launches are estimated to take less than one (597
// rows x 50257: 591 large tiles are 2.3 rounds; 510 of them and the rest in
// smaller tiles).  main == v: one launch.
struct RangePlan {
    int shape, rest_shape;
    int64_t main;
};
RangePlan plan_range(int64_t t, int64_t v, int64_t k, int64_t other, bool by_rows, int cus)
{
    // by_rows (dW): outputs are v x other; else (logits) t x v
    auto us = [&](int sh, int64_t n) {
        return by_rows ? product_us(sh, n, other, k, 1, cus) : product_us(sh, t, n, k, 1, cus);
    };
    auto pick = [&](int64_t n) {
        return by_rows ? pick_shape(false, n, other, k, cus) : pick_shape(true, t, n, k, cus);
    };
    RangePlan p;
    p.shape = p.rest_shape = pick(v);
    p.main = v;
    double best = us(p.shape, v);
    const ShapeCost& b = kShapes[SHAPE_BIG];
    const int64_t across = by_rows ? cdiv(other, b.tn) : cdiv(t, b.tm);
    const int64_t step = by_rows ? b.tm : b.tn;
    for (int64_t rounds = v / step * across / cus; rounds >= 1; --rounds) {
        const int64_t main = rounds * cus / across * step;
        if (main <= 0 || main >= v)
            continue;
        const int rest = pick(v - main);
        const double two = us(SHAPE_BIG, main) + us(rest, v - main) + kLaunchUs;
        if (two < best) {
            best = two;
            p.shape = SHAPE_BIG;
            p.rest_shape = rest;
            p.main = main;
        }
        break;                   // fewer rounds only leave more to the smaller tiles
    }
    return p;
}

template <class S, int ROLE, bool FEW = false>
hipError_t go(const LossArgs& a, int64_t tiles_m, int cus, hipStream_t s)
{
    LossArgs copy = a;
    copy.tiles_n = (int)cdiv(a.N, S::TN);
    const int64_t items = tiles_m * copy.tiles_n * (ROLE == ROLE_DX ? a.slices.most : 1);
    if (items > INT32_MAX)
        return hipErrorInvalidValue;
    const int64_t grid = std::min<int64_t>(items, (int64_t)cus * S::PER_CU);
    void* args[] = {&copy};
    return hipLaunchKernel(reinterpret_cast<const void*>(&loss_gemm_kernel<S, ROLE, FEW>), dim3((unsigned)grid),
                           dim3(S::THREADS), args, 0, s);
}

template <int ROLE, bool FEW = false>
hipError_t launch_role(int shape, const LossArgs& a, int64_t rows, int cus, hipStream_t s)
{
    // (few rows' logits have launches of their own)
    if constexpr (ROLE == ROLE_DX) {
        if (shape == SHAPE_LOW)
            return go<Low, ROLE, FEW>(a, cdiv(rows, Low::TM), cus, s);
        if (shape == SHAPE_FEW)
            return go<Few, ROLE, FEW>(a, cdiv(rows, Few::TM), cus, s);
    }
    if constexpr (!FEW) {
        if (shape == SHAPE_BIG)
            return go<Big, ROLE>(a, cdiv(rows, Big::TM), cus, s);
    }
    if (shape == SHAPE_TALL)
        return go<Tall, ROLE, FEW>(a, cdiv(rows, Tall::TM), cus, s);
    if constexpr (ROLE == ROLE_LSE || ROLE == ROLE_GRAD) {
        if (shape == SHAPE_WIDE)
            return go<Wide, ROLE>(a, cdiv(rows, Wide::TM), cus, s);
        if (shape == SHAPE_DEEP)
            return go<Deep, ROLE>(a, cdiv(rows, Deep::TM), cus, s);
    }
    using Other = std::conditional_t<ROLE == ROLE_LSE || ROLE == ROLE_GRAD, Line, Mid>;
    return go<Other, ROLE, FEW>(a, cdiv(rows, Other::TM), cus, s);
}

// dX and dW of the vocabulary in one launch, half of the workgroups for each.  In
// launches of their own both mostly wait for memory, with one or two tiles a CU.
template <class S, bool FEW>
hipError_t go_pair(const LossArgs& x, const LossArgs& w, int cus, hipStream_t s)
{
    LossArgs xc = x, wc = w;
    xc.tiles_n = (int)cdiv(x.N, S::TN);
    wc.tiles_n = (int)cdiv(w.N, S::TN);
    int half = cus * S::PER_CU / 2;          // xc's slices make at most so many items
    const int64_t w_items = cdiv(w.M, S::TM) * wc.tiles_n;
    const int64_t grid = half + std::min<int64_t>(w_items, (int64_t)cus * S::PER_CU - half);
    void* args[] = {&xc, &wc, &half};
    return hipLaunchKernel(reinterpret_cast<const void*>(&loss_pair_kernel<S, FEW>), dim3((unsigned)grid),
                           dim3(S::THREADS), args, 0, s);
}

// The logits of few rows.
template <int ROLE>
hipError_t launch_few(int shape, const LossArgs& a, int cus, hipStream_t s)
{
    switch (shape) {
    case SHAPE_LOW_SLIM:
        return go<LowSlim, ROLE, true>(a, 1, cus, s);
    case SHAPE_LOW:
        return go<Low, ROLE, true>(a, 1, cus, s);
    case SHAPE_FEW_SLIM:
        return go<FewSlim, ROLE, true>(a, 1, cus, s);
    case SHAPE_FEW:
        return go<Few, ROLE, true>(a, 1, cus, s);
    case SHAPE_SLIM:
        return go<Slim, ROLE, true>(a, 1, cus, s);
    case SHAPE_DEEP:
        return go<Deep, ROLE, true>(a, 1, cus, s);
    }
    return go<Line, ROLE, true>(a, 1, cus, s);
}

// Launches a kernel; the status of this launch, not an earlier sticky error.
template <class... P, class... A>
hipError_t launch(void (*kernel)(P...), dim3 grid, int block, hipStream_t s, A... args)
{
    std::tuple<P...> held(args...);
    return std::apply(
        [&](auto&... a) {
            void* list[] = {&a...};
            return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3((unsigned)block), list,
                                   0, s);
        },
        held);
}
template <class... P, class... A>
hipError_t launch(void (*kernel)(P...), int64_t grid, int block, hipStream_t s, A... args)
{
    return launch(kernel, dim3((unsigned)grid), block, s, args...);
}

#define DG_TRY(x)                    \
    do {                             \
        const hipError_t e_ = (x);   \
        if (e_ != hipSuccess)        \
            return e_;               \
    } while (0)

// Distillation: the targets' kernel.  Returns where the rows' states are.
hipError_t row_targets(const LossCall& c, const LossPlan& pl, bool by_group, RowSource* out)
{
    uint8_t* ws = c.ws;
    RowSource& src = *out;
    src = {c.labels, c.ignore_index, c.V, nullptr};
    if (c.slots) {
        TargetArgs t;
        t.index = c.index;
        t.teacher = c.teacher;
        t.ld_index = c.ld_index;
        t.ld_teacher = c.ld_teacher;
        t.T = c.T;
        t.V = c.V;
        t.k = (int)c.slots;
        t.scale = c.scale;
        t.q = reinterpret_cast<float*>(ws + pl.off_q);
        t.qsum = reinterpret_cast<float*>(ws + pl.off_qsum);
        t.rest = reinterpret_cast<float*>(ws + pl.off_rest);
        t.leader = reinterpret_cast<int*>(ws + pl.off_lead);
        t.flag = reinterpret_cast<int*>(ws + pl.off_flag);
        t.logp = by_group ? c.logp_in : nullptr;
        src.flag = t.flag;
        DG_TRY(launch(loss_target_kernel, c.T, 64, c.stream, t));
    }
    return hipSuccess;
}

hipError_t select_rows(const LossCall& c, const LossPlan& pl, const RowSource& src, bool backward, bool by_group)
{
    uint8_t* ws = c.ws;
    int* chunks = nullptr;
    int* n_kept = reinterpret_cast<int*>(ws + pl.off_count);
    int* group = reinterpret_cast<int*>(ws + pl.off_group);
    int* place = nullptr;
    const int groups = (int)pl.groups, n_chunks = (int)cdiv(c.T, kOwnCount);
    if (by_group && c.T > kOwnCount) {
        place = reinterpret_cast<int*>(ws + pl.off_place);
        DG_TRY(launch(loss_group_count_kernel, dim3((unsigned)n_chunks, (unsigned)cdiv(groups, kGroupPass)), 1024,
                      c.stream, src, c.T, groups, place));
        DG_TRY(launch(loss_group_place_kernel, dim3(1), 1024, c.stream, place, (int64_t)groups * n_chunks, n_chunks,
                      group, groups, n_kept));
    } else if (c.T > kOwnCount) {
        chunks = reinterpret_cast<int*>(ws + pl.off_chunks);
        DG_TRY(launch(loss_count_kernel, cdiv(c.T, kChunk), 256, c.stream, src, c.T, chunks));
    }
    SelectArgs a;
    a.src = src;
    a.T = c.T;
    a.chunks = chunks;
    a.X = reinterpret_cast<const uint8_t*>(c.X);
    a.ldx_b = c.ldx * 2;
    a.Xc = ws + pl.off_x;
    a.row_b = c.D * 2;
    a.n_kept = n_kept;
    a.map = reinterpret_cast<int*>(ws + pl.off_map);
    a.pos = reinterpret_cast<int*>(ws + pl.off_pos);
    a.rows = reinterpret_cast<RowInfo*>(ws + pl.off_rows);
    a.zlabel = backward ? nullptr : reinterpret_cast<float*>(ws + pl.off_zlabel);
    a.loss = c.loss;
    a.lse_out = c.lse;
    a.loss_in = c.loss_in;
    a.lse_in = c.lse_in;
    a.dloss = c.dloss;
    a.dloss_stride = c.dloss_stride;
    a.scale = c.scale;
    a.z_loss = c.z_loss;
    a.place = place;
    a.n_chunks = n_chunks;
    a.groups = groups;
    a.group = group;
    a.rest = ws + pl.off_g + pl.piece * 2;
    a.rest_b = pl.ldg * 2;
    const int64_t firsts = place ? 0 : cdiv(groups + 1, kSelRows);
    return by_group ? launch(loss_select_kernel<true>, cdiv(c.T, kSelRows) + firsts, 256, c.stream, a)
                    : launch(loss_select_kernel<false>, cdiv(c.T, kSelRows), 256, c.stream, a);
}

LossArgs product_args(const LossCall& c, const LossPlan& pl)
{
    LossArgs a;
    memset(&a, 0, sizeof a);
    a.n_kept = reinterpret_cast<const int*>(c.ws + pl.off_count);
    a.rows = reinterpret_cast<const RowInfo*>(c.ws + pl.off_rows);
    a.scale = c.scale;
    return a;
}

}  // namespace

static LossPlan make_plan(int64_t T, int64_t V, int64_t D, int64_t slots, bool backward)
{
    LossPlan p;
    memset(&p, 0, sizeof p);
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t o = at;
        at = round_up(at + bytes, 256);
        return o;
    };
    p.rows_pad = round_up(T, 256);
    p.few = T <= Line::TM;
    // Rows of the large tables: stores and reads stop at the last kept row, so
    // that few rows need no more (one row of 50257 x 512 asks for 1 MB, 49 with 256)
    p.rows = p.few ? T : p.rows_pad;
    p.off_count = take(256);
    p.off_chunks = take(cdiv(T, kChunk) * 4);
    p.off_map = take(p.rows_pad * 4);
    p.off_pos = take(p.rows_pad * 4);
    p.off_rows = take(p.rows_pad * 16);
    p.off_x = take(T * D * 2);
    if (slots) {
        p.off_q = take(T * slots * 4);
        p.off_qsum = take(T * slots * 4);
        p.off_rest = take(T * slots * 4);
        p.off_lead = take(T * slots * 4);
        p.off_flag = take(T * 8);
    }
    const int64_t shared = at;
    p.tiles_n_max = cdiv(V, T <= Line::TM ? 64 : 128);
    p.off_part = take(p.tiles_n_max * p.rows * 8);
    p.off_zlabel = take(p.rows_pad * 4);
    p.bytes = at;
    if (backward) {
        at = shared;
        // G of one piece, or its two halves: at most 256 MiB (the Infinity Cache's
        // size), at least 256 columns; at most 2^21 columns, as the pitches of X
        // and W (a tile's rows stay within a 31-bit offset).  Fewer pieces make fuller rounds of tiles and
        // fewer passes over dX's planes: 2048 x 131072 x 4096 measured 5351,
        // 5316, 5222 and 5172 us with 64, 128, 256 and 512 MiB.
        const int64_t row_b = p.rows * (p.few ? 4 : 2);
        int64_t piece = (INT64_C(256) << 20) / row_b / 256 * 256;
        piece = std::max<int64_t>(piece, 256);
        piece = std::min<int64_t>(piece, INT64_C(1) << 21);
        piece = std::min(piece, round_up(V, 256));
        p.piece = piece;
        // dX: shape and K slices by the estimate, the planes' traffic included
        // (each slice writes one, the last kernel reads them, and every
        // further piece reads and writes them again)
        const int64_t passes = 2 * cdiv(V, piece);
        // (One tile of rows never takes Big: a round of Mid holds as many columns of
        // outputs, two tiles a CU, and costs less.)
        double best = 0.0;
        for (int sh = T <= 32 ? SHAPE_LOW : T <= 64 ? SHAPE_FEW : p.few ? SHAPE_TALL : SHAPE_BIG;
             sh <= (T <= 32 ? SHAPE_LOW : T <= 64 ? SHAPE_FEW : SHAPE_MID); ++sh)
            for (int sp = 1; sp <= 64 && (sp == 1 || piece / sp >= 256); ++sp) {
                const double us = cdiv(V, piece) * product_us(sh, T, D, piece, sp, kPlanCus) +
                                  (double)(passes * sp * T * D * 4) / kPlaneBytesPerUs;
                if (best == 0.0 || us < best) {
                    best = us;
                    p.dx_shape = sh;
                    p.splits = sp;
                }
            }
        // Both gradients of a small vocabulary in one launch, dX in as many
        // slices as give half of the workgroups one tile each, when a slice is
        // at most 128 k-tiles: of 38 such sizes 37 then took 1 to 14 % less for
        // their gradients (400 x 11008 x 1024: 55.7 us, 50.1) and one 2 % more; with
        // longer slices 6 % less to 9 % more (148 x 57039 x 2896: 372, 405).
        // Few rows, whose dW is stores more than sums: at most 16 k-tiles (14 of
        // 38 sizes: 1 to 10 % less, 30 x 5000 x 512 30.5 us, 27.9; the others up
        // to 13 % less, 1 x 43021 x 2160, and 9 % more, 100 x 11008 x 4096).
        const int64_t pair_tiles = cdiv(T, Mid::TM) * cdiv(D, Mid::TN);
        const int64_t pair_slices = std::min(kPlanCus / pair_tiles, piece / 256);
        if (V <= piece && pair_slices >= 1 && cdiv(cdiv(V, Mid::KT), pair_slices) <= (p.few ? 16 : 128))
            p.pair = (int)pair_slices;
        p.ldg = piece + (p.few ? 0 : kRestCols);
        p.off_g = take(row_b * p.ldg);
        if (!p.few) {
            p.groups = cdiv(V, kRestCols);
            p.off_group = take((p.groups + 1) * 4);
            p.off_place = take(T > kOwnCount ? p.groups * cdiv(T, kOwnCount) * 4 : 0);
        }
        p.off_planes = take((int64_t)std::max(p.splits, p.pair) * T * D * 4);
        p.bytes = std::max(p.bytes, at);
    }
    return p;
}

// A call asks for its plan two or three times, and a program calls with the
// same sizes again and again: each thread keeps the last few.
LossPlan loss_plan(int64_t T, int64_t V, int64_t D, int64_t slots, bool backward)
{
    struct Entry {
        int64_t T, V, D, slots, backward;
        LossPlan plan;
    };
    thread_local Entry kept[4];
    thread_local int next = 0;
    for (const Entry& e : kept)
        if (e.T == T && e.V == V && e.D == D && e.slots == slots && e.backward == backward)
            return e.plan;
    Entry& e = kept[next];
    next = (next + 1) % 4;
    e = {T, V, D, slots, backward, make_plan(T, V, D, slots, backward)};
    return e.plan;
}

hipError_t loss_forward(const LossCall& c)
{
    const LossPlan pl = loss_plan(c.T, c.V, c.D, c.slots, false);
    uint8_t* ws = c.ws;
    RowSource src;
    DG_TRY(row_targets(c, pl, false, &src));
    // Rows that one tile holds are not selected: W is read for one of them as
    // for all, and the launch takes longer than the rest could save (one row of
    // 50257 x 512: 20 us with it, 16 without).
    const bool few = c.T <= Line::TM;
    if (!few)
        DG_TRY(select_rows(c, pl, src, false, false));
    LossArgs a = product_args(c, pl);
    a.A = few ? reinterpret_cast<const uint8_t*>(c.X) : ws + pl.off_x;
    a.lda_b = few ? c.ldx * 2 : c.D * 2;
    a.n = (int)c.T;
    a.labels = c.labels;
    a.lead = src.flag;
    a.B = reinterpret_cast<const uint8_t*>(c.W);
    a.ldb_b = c.ldw * 2;
    a.N = (int)c.V;
    a.K = (int)c.D;
    a.part = reinterpret_cast<float2*>(ws + pl.off_part);
    a.ldpart = pl.rows;
    a.zlabel = reinterpret_cast<float*>(ws + pl.off_zlabel);
    const RangePlan rp = few ? RangePlan{few_shape(c.T, c.V, c.cus), 0, c.V}
                             : plan_range(c.T, c.V, c.D, 0, false, c.cus);
    int64_t tiles = 0;                       // tile columns so far
    for (int64_t v0 = 0; v0 < c.V; v0 += rp.main) {
        const int shape = v0 == 0 ? rp.shape : rp.rest_shape;
        LossArgs m = a;
        m.v0 = (int)v0;
        m.N = (int)(v0 == 0 ? rp.main : c.V - v0);
        m.B = a.B + v0 * a.ldb_b;
        m.part = a.part + tiles * a.ldpart;
        DG_TRY(few ? launch_few<ROLE_LSE>(shape, m, c.cus, c.stream)
                   : launch_role<ROLE_LSE>(shape, m, c.T, c.cus, c.stream));
        tiles += cdiv(m.N, kShapes[shape].tn);
        if (v0 != 0)
            break;
    }
    JoinArgs j;
    j.part = a.part;
    j.ldpart = a.ldpart;
    j.tiles_n = (int)tiles;
    j.n_kept = a.n_kept;
    j.map = reinterpret_cast<const int*>(ws + pl.off_map);
    j.src = src;
    j.few = few ? (int)c.T : 0;
    j.zlabel = a.zlabel;
    j.scale = fabsf(c.scale);
    j.z_loss = c.slots ? 0.f : c.z_loss;
    j.loss = c.loss;
    j.lse = c.lse;
    auto join = [&](auto r) {
        constexpr int R = decltype(r)::value;
        return launch(loss_join_kernel<R>, cdiv(c.T, R), 256, c.stream, j);
    };
    if (!few || !c.slots)
        DG_TRY(c.T >= 2048 ? join(std::integral_constant<int, 16>{})
               : c.T >= 256 ? join(std::integral_constant<int, 4>{})
                            : join(std::integral_constant<int, 1>{}));
    if (!c.slots)
        return hipSuccess;
    PickArgs k;
    k.W = a.B;
    k.ldw_b = a.ldb_b;
    k.Xc = a.A;
    k.row_b = c.D * 2;
    k.ldx_b = a.lda_b;
    k.pos = few ? nullptr : reinterpret_cast<const int*>(ws + pl.off_pos);
    k.index = c.index;
    k.ld_index = c.ld_index;
    k.V = c.V;
    k.teacher = c.teacher;
    k.ld_teacher = c.ld_teacher;
    k.q = reinterpret_cast<const float*>(ws + pl.off_q);
    k.flag = reinterpret_cast<const int*>(ws + pl.off_flag);
    k.k = (int)c.slots;
    k.scale = c.scale;
    k.zlabel = a.zlabel;
    k.loss = c.loss;
    k.logp = c.logp;
    return few ? launch(loss_pick_kernel<true>, c.T, 1024, c.stream, k, j)
               : launch(loss_pick_kernel<false>, c.T, 256, c.stream, k, j);
}

hipError_t loss_backward(const LossCall& c)
{
    const LossPlan pl = loss_plan(c.T, c.V, c.D, c.slots, true);
    uint8_t* ws = c.ws;
    RowSource src;
    const bool by_group = c.dW && !pl.few;
    DG_TRY(row_targets(c, pl, by_group, &src));
    DG_TRY(select_rows(c, pl, src, true, by_group));
    const int* pos = reinterpret_cast<const int*>(ws + pl.off_pos);
    const int* map = reinterpret_cast<const int*>(ws + pl.off_map);
    const RowInfo* rows = reinterpret_cast<const RowInfo*>(ws + pl.off_rows);
    // few rows: G in two halves where dW is asked for; W past the Infinity Cache
    // with the non-temporal hint (both gradients at 48 x 50257 x 4096, 412 MB: 275
    // us against 302; 30 x 131072 x 4096: 562 against 635; but 48 x 50257 x 2048,
    // 206 MB: 144 against 133)
    const bool few = pl.few;
    const int64_t half_b = few && c.dW ? pl.rows * pl.piece * 2 : 0;
    const int w_nt = few && c.V * c.D * 2 > (INT64_C(256) << 20);
    uint16_t* G = reinterpret_cast<uint16_t*>(ws + pl.off_g);
    const bool pair = pl.pair && c.dX && c.dW;
    const ShapeCost& dxs = kShapes[pair ? SHAPE_MID : pl.dx_shape];
    const int splits = pair ? pl.pair : pl.splits;
    DxSlices slices;
    slices.S = splits;
    slices.T = (int)c.T;
    slices.tm = dxs.tm;
    slices.tiles_n = (int)cdiv(c.D, dxs.tn);
    slices.items = (int)(cdiv(c.T, dxs.tm) * slices.tiles_n * splits);
    slices.most = (int)std::max<int64_t>(splits, pl.piece / 256);
    const uint8_t* Xc = ws + pl.off_x;
    float* planes = reinterpret_cast<float*>(ws + pl.off_planes);
    for (int64_t v0 = 0; v0 < c.V; v0 += pl.piece) {
        const int64_t vp = std::min(pl.piece, c.V - v0);
        const uint8_t* W = reinterpret_cast<const uint8_t*>(c.W) + v0 * c.ldw * 2;
        const RangePlan gp = few ? RangePlan{few_shape(c.T, vp, c.cus), 0, vp}
                                 : plan_range(c.T, vp, c.D, 0, false, c.cus);
        for (int64_t u = 0; u < vp; u += gp.main) {
            const int shape = u == 0 ? gp.shape : gp.rest_shape;
            LossArgs a = product_args(c, pl);
            a.A = Xc;
            a.lda_b = c.D * 2;
            a.B = W + u * c.ldw * 2;
            a.ldb_b = c.ldw * 2;
            a.N = (int)(u == 0 ? gp.main : vp - u);
            a.K = (int)c.D;
            a.v0 = (int)(v0 + u);
            a.C = G + u;
            a.ldc = pl.ldg;
            a.c_cols = (int)(pl.piece - u);
            a.half_b = half_b;
            a.w_nt = w_nt;
            DG_TRY(few ? launch_few<ROLE_GRAD>(shape, a, c.cus, c.stream)
                       : launch_role<ROLE_GRAD>(shape, a, c.T, c.cus, c.stream));
            if (u != 0)
                break;
        }
        if (c.slots) {
            SparseArgs k;
            k.n_kept = reinterpret_cast<const int*>(ws + pl.off_count);
            k.map = map;
            k.rows = rows;
            k.leader = reinterpret_cast<const int*>(ws + pl.off_lead);
            k.qsum = reinterpret_cast<const float*>(ws + pl.off_qsum);
            k.rest = reinterpret_cast<const float*>(ws + pl.off_rest);
            k.logp = c.logp_in;
            k.k = (int)c.slots;
            k.v0 = v0;
            k.vp = vp;
            k.G = G;
            k.ldg = pl.ldg;
            k.half_b = half_b;
            k.lost = reinterpret_cast<float*>(ws + pl.off_q);
            k.flag = src.flag;
            k.lead_rest = by_group ? G + pl.piece : nullptr;
            DG_TRY(launch(loss_sparse_kernel, cdiv(c.T, 4), 256, c.stream, k));
        }
        LossArgs dx = product_args(c, pl);
        if (c.dX) {
            LossArgs& d = dx;
            d.A = reinterpret_cast<const uint8_t*>(G);
            d.lda_b = pl.ldg * 2;
            d.B = W;
            d.ldb_b = c.ldw * 2;
            d.N = (int)c.D;
            d.K = (int)vp;
            d.slices = slices;
            d.planes = planes;
            d.ldplane = c.D;
            d.first = v0 == 0;
            d.w_nt = w_nt;
            if (pair) {
                // with dW, below
            } else if (w_nt) {
                DG_TRY((launch_role<ROLE_DX, true>(pl.dx_shape, d, c.T, c.cus, c.stream)));
            } else {
                DG_TRY(launch_role<ROLE_DX>(pl.dx_shape, d, c.T, c.cus, c.stream));
            }
        }
        if (c.dW) {
            const RangePlan wp = few || pair ? RangePlan{SHAPE_MID, 0, vp}
                                     : plan_range(c.T, vp, c.T, c.D, true, c.cus);
            for (int64_t u = 0; u < vp; u += wp.main) {
                LossArgs d = product_args(c, pl);
                d.A = reinterpret_cast<const uint8_t*>(G + u);
                d.lda_b = pl.ldg * 2;
                d.B = Xc;
                d.ldb_b = c.D * 2;
                d.M = (int)(u == 0 ? wp.main : vp - u);
                d.v0 = (int)(v0 + u);        // (whole groups)
                d.rest = reinterpret_cast<const uint8_t*>(G + pl.piece);
                d.group = reinterpret_cast<const int*>(ws + pl.off_group);
                d.N = (int)c.D;
                d.C = c.dW + (v0 + u) * c.lddw;
                d.ldc = c.lddw;
                d.c_vec = ((uintptr_t)c.dW & 15u) == 0 && c.lddw % 8 == 0;
                // With few rows dW is bound by writing it; past half of the
                // Infinity Cache the non-temporal hint helps (48 x 50257 x 2048,
                // 206 MB: 112 us against 130), below it does not (1 x 50257 x
                // 1024, 103 MB: 47 against 43).
                if (half_b && d.c_vec && c.V * c.D * 2 > (INT64_C(128) << 20))
                    d.c_vec = 2;
                d.half_b = half_b;
                const int shape = u == 0 ? wp.shape : wp.rest_shape;
                if (pair) {
                    DG_TRY((few ? go_pair<Mid, true>(dx, d, c.cus, c.stream)
                                : go_pair<Mid, false>(dx, d, c.cus, c.stream)));
                    break;
                }
                DG_TRY((few ? go<Mid, ROLE_DW, true>(d, cdiv(d.M, Mid::TM), c.cus, c.stream)
                            : launch_role<ROLE_DW>(shape, d, d.M, c.cus, c.stream)));
                if (u != 0)
                    break;
            }
        }
    }
    if (c.dX) {
        DxArgs d;
        d.planes = planes;
        d.slices = slices;
        d.n_kept = reinterpret_cast<const int*>(ws + pl.off_count);
        d.ldplane = c.D;
        d.pos = pos;
        d.rows = rows;
        d.W = c.W;
        d.ldw = c.ldw;
        d.k = (int)c.slots;
        d.leader = reinterpret_cast<const int*>(ws + pl.off_lead);
        d.lost = reinterpret_cast<const float*>(ws + pl.off_q);
        d.dX = c.dX;
        d.lddx = c.lddx;
        d.D = c.D;
        d.vec = ((uintptr_t)c.dX & 7u) == 0 && c.lddx % 4 == 0;
        if (c.T <= Line::TM && splits >= 8)
            DG_TRY(launch(loss_dx_kernel<8>, c.T * cdiv(c.D, 128), 256, c.stream, d));
        else
            DG_TRY(launch(loss_dx_kernel<1>, c.T, 256, c.stream, d));
    }
    return hipSuccess;
}

}  // namespace dg
