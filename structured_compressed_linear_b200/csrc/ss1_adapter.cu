// Low-rank adapters of many requests beside one projection, and their gradients.
//
// Row m of the batch uses adapter a = index[m] (none if a is outside [0, count)):
//
//     H[m] = X[m] A[a]^T                       [R]      A [count, R, K]
//     out[m] = Y[m] + scale[a] H[m] B[a]^T     [N]      B [count, N, R]
//
// and, for a gradient dY of out,
//
//     G[m] = scale[a] dY[m] B[a]               [R]
//     dX_out[m] = dX[m] + G[m] A[a]            [K]
//     dA[a] = sum over its rows of G[m]^T X[m],    dB[a] = scale[a] sum over its rows of dY[m]^T H[m]
//
// A rank is small beside K and N, so these passes move bytes: the forward reads X and Y and writes
// out, the backward reads dY, X and dX and writes dX. H and G are float32: rounding them would
// add an error of the size of the output's own rounding, and they are R columns only.
//
// The plan lists the rows by adapter (stable, so sums over an adapter's rows have one order), and
// tiles of up to kTile rows of one adapter.
#include "ss1_adapter.cuh"
#include "ptx_sm100.cuh"

#include <algorithm>

namespace ss1 {
namespace ada {

using namespace op;

// ---- plan ------------------------------------------------------------------------------------

// One CTA. Every warp counts its own contiguous share of the rows by adapter (lanes with the same
// adapter find one another by a ballot for each bit of its number: one __match_any_sync takes a step for every
// different value, 18 us for 8192 rows of 32 adapters in random order), the counts are scanned over
// adapters and warps, and each row's place is what comes before it: rows keep their order within an
// adapter. The first AHEAD index words of a lane are loaded together, and their places within the warp kept:
// one memory latency, and one walk; rows beyond are walked twice. AHEAD is 8 where 32 warps (fewer beside many
// adapters) cover all rows so, since code that is not fetched yet is what a small plan waits for: 3.2 us against 4.4
// with 16 at 300 rows, 4.4 against 5.7 at 8192; 16 beyond: 16,384 rows 7.8 us against 10.2 with 8.

__device__ __forceinline__ int plan_group(const int32_t* __restrict__ index, int row, int end, int n) {
    if (row >= end) return -1;
    const int a = index[row];
    return (unsigned)a < (unsigned)n ? a : n;
}

template <int AHEAD>
__global__ void __launch_bounds__(1024) plan_kernel(const int32_t* __restrict__ index, int M, int n, PlanView plan) {
    extern __shared__ int cnt[];   // [warps][n + 1], then [n + 2] first rows and [n + 2] first tiles
    wait_for_previous();
    let_next_start();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const int groups = n + 1;      // group n: rows without an adapter
    int* first = cnt + warps * groups;
    int* first_tile = first + n + 2;
    const int share = (M + warps - 1) / warps;
    const int begin = min(M, warp * share), end = min(M, begin + share);
    int ahead[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) ahead[i] = plan_group(index, begin + i * 32 + lane, end, n);
    for (int i = threadIdx.x; i < warps * groups; i += blockDim.x) cnt[i] = 0;
    __syncthreads();
    int* mine = cnt + warp * groups;
    const int bits = 32 - __clz(n);           // of the numbers 0 .. n
    auto peers = [&](int a) {                  // lanes with this lane's group; -1 (no row) is a group of its own
        const int one = __shfl_sync(0xFFFFFFFFu, a, 0);
        if (__all_sync(0xFFFFFFFFu, a == one)) return 0xFFFFFFFFu;      // a request's rows mostly come together
        unsigned same = __ballot_sync(0xFFFFFFFFu, a >= 0);
        if (a < 0) same = ~same;
        for (int b = 0; b < bits; ++b) {
            const unsigned set = __ballot_sync(0xFFFFFFFFu, (a >> b) & 1);
            same &= (a >> b) & 1 ? set : ~set;
        }
        return same;
    };
    // the row's number among the warp's rows of its group so far
    auto count = [&](int a) {
        const unsigned same = peers(a);
        const int before = a >= 0 ? mine[a] + __popc(same & ((1u << lane) - 1u)) : 0;
        __syncwarp();
        if (a >= 0 && lane == __ffs(same) - 1) mine[a] += __popc(same);
        __syncwarp();
        return before;
    };
    int nth[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) nth[i] = begin + i * 32 < end ? count(ahead[i]) : 0;
    for (int at = begin + AHEAD * 32; at < end; at += 32) count(plan_group(index, at + lane, end, n));
    __syncthreads();
    // totals, then their exclusive sums (one warp, 32 groups at a time), with the tiles' beside them
    for (int a = warp; a < groups; a += warps) {       // a warp a group, a lane a warp's count
        const int c = lane < warps ? cnt[lane * groups + a] : 0;
        int s = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
            if (lane >= o) s += u;
        }
        if (lane < warps) cnt[lane * groups + a] = s - c;
        if (lane == 31) first[a] = s;
    }
    __syncthreads();
    if (warp == 0) {
        int rows = 0, tiles = 0;
        for (int at = 0; at < groups; at += 32) {
            const int a = at + lane;
            const int c = a < groups ? first[a] : 0;
            const int t = (c + kTile - 1) / kTile;
            int cs = c, ts = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int cu = __shfl_up_sync(0xFFFFFFFFu, cs, o), tu = __shfl_up_sync(0xFFFFFFFFu, ts, o);
                if (lane >= o) { cs += cu; ts += tu; }
            }
            if (a < groups) {
                first[a] = rows + cs - c;
                first_tile[a] = tiles + ts - t;
            }
            rows += __shfl_sync(0xFFFFFFFFu, cs, 31);
            tiles += __shfl_sync(0xFFFFFFFFu, ts, 31);
        }
        if (lane == 0) {
            first[groups] = rows;
            first_tile[groups] = tiles;
        }
    }
    __syncthreads();
    for (int a = threadIdx.x; a <= groups; a += blockDim.x) {
        plan.first[a] = first[a];
        plan.first_tile[a] = first_tile[a];
    }
    for (int i = threadIdx.x; i < plan.max_tiles; i += blockDim.x) {
        int4 t = make_int4(-1, 0, 0, 0);
        if (i < first_tile[groups]) {
            int lo = 0, hi = groups - 1;               // the last group whose first tile is at or before i and that has rows
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (first_tile[mid] <= i) lo = mid;
                else hi = mid - 1;
            }
            const int at = first[lo] + (i - first_tile[lo]) * kTile;
            t = make_int4(lo < n ? lo : -1, at, min(kTile, first[lo + 1] - at), 0);
        }
        plan.tiles[i] = t;
    }
    int* so_far = cnt + warp * groups;         // rows of the group in the warps before this one; then its own ones too
    auto put = [&](int a, int row, int number) {
        const int to = first[a] + number;
        if (SS1_IN(to, M, kSitePlan)) plan.rows[to] = row;
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (ahead[i] >= 0) put(ahead[i], begin + i * 32 + lane, so_far[ahead[i]] + nth[i]);
    if (begin + AHEAD * 32 >= end) return;    // the whole warp
    __syncwarp();
    // the second walk counts on from the first AHEAD rounds
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) count(ahead[i]);
    for (int at = begin + AHEAD * 32; at < end; at += 32) {
        const int a = plan_group(index, at + lane, end, n);
        const int number = count(a);
        if (a >= 0) put(a, at + lane, number);
    }
}

cudaError_t launch_plan(const int32_t* index, int64_t M, int n, PlanView plan, cudaStream_t st) {
    // counters of every warp beside one another in the 48 KB that need no opt-in
    int warps = (48 * 1024 / 4 - 2 * (n + 2)) / (n + 1);
    warps = warps > 32 ? 32 : warps;
    const size_t smem = ((size_t)warps * (n + 1) + 2 * (n + 2)) * sizeof(int);
    return launch_dependent(M <= (int64_t)warps * 32 * 8 ? &plan_kernel<8> : &plan_kernel<16>, dim3(1), dim3((unsigned)(warps * 32)), smem, st, index, (int)M, n, plan);
}

namespace {

int64_t sub_tiles(const Call& c) {
    const int64_t tiles = c.plan.rows ? c.plan.max_tiles : (c.M + kTile - 1) / kTile;
    return tiles * (kTile / 32);
}

// ---- general path: any type, size and alignment, on the CUDA cores -----------------------------

constexpr int kRanks = 16;   // ranks a thread sums at a time

// Sums of kRanks values over the CTA's threads; the result is in the first kRanks threads' return value.
__device__ __forceinline__ float cta_sums(float (&s)[kRanks], float (*buf)[kRanks]) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
#pragma unroll
    for (int r = 0; r < kRanks; ++r) {
        const float v = warp_sum(s[r]);
        if (lane == 0) buf[warp][r] = v;
    }
    __syncthreads();
    float v = 0.0f;
    if (threadIdx.x < kRanks)
        for (int w = 0; w < warps; ++w) v += buf[w][threadIdx.x];
    return v;
}

// P[m, r] = f * sum_c U[m, c] * table_a[c, r] (table element (a, c, r) at a * stride + c * cs + r * rs), f = scale[a]
// or 1; 0 for a row without an adapter.
template <typename T>
__global__ void __launch_bounds__(256) row_products_kernel(const T* __restrict__ U, const T* __restrict__ table,
                                                           const int32_t* __restrict__ index, const float* __restrict__ scale,
                                                           float* __restrict__ P, int64_t M, int C, int R, int n, int cs, int rs,
                                                           int site_u, int site_t) {
    __shared__ float buf[8][kRanks];
    const int64_t m = blockIdx.x;
    const int r0 = blockIdx.y * kRanks, ranks = min(kRanks, R - r0);
    const int a = index ? index[m] : 0;
    const bool some = (unsigned)a < (unsigned)n;
    float s[kRanks];
#pragma unroll
    for (int r = 0; r < kRanks; ++r) s[r] = 0.0f;
    if (some) {
        const int64_t base = (int64_t)a * C * R;
        for (int c = threadIdx.x; c < C; c += blockDim.x) {
            const float u = SS1_IN(m * C + c, M * C, site_u) ? to_f(U[m * C + c]) : 0.0f;
#pragma unroll
            for (int r = 0; r < kRanks; ++r) {
                const int64_t at = base + (int64_t)c * cs + (int64_t)(r0 + r) * rs;
                if (r < ranks && SS1_IN(at, (int64_t)n * C * R, site_t)) s[r] = fmaf(u, to_f(table[at]), s[r]);
            }
        }
    }
    const float v = cta_sums(s, buf);
    if (threadIdx.x < ranks && SS1_IN(m * R + r0 + threadIdx.x, M * R, kSiteAdaH))
        P[m * R + r0 + threadIdx.x] = some ? v * (scale ? scale[a] : 1.0f) : 0.0f;
}

// out[m, c] = in[m, c] + f * sum_r P[m, r] * table_a[c, r]; in may be out itself, or null (0).
template <typename T>
__global__ void __launch_bounds__(256) row_update_kernel(const float* __restrict__ P, const T* __restrict__ table,
                                                         const int32_t* __restrict__ index, const float* __restrict__ scale,
                                                         const T* in, T* out, int64_t M, int C, int R, int n, int cs, int rs,
                                                         int site_t) {
    __shared__ float p[kMaxRank];
    const int64_t m = blockIdx.y;
    const int a = index ? index[m] : 0;
    const bool some = (unsigned)a < (unsigned)n;
    const float f = some && scale ? scale[a] : 1.0f;
    if (some)
        for (int r = threadIdx.x; r < R; r += blockDim.x) p[r] = f * P[m * R + r];
    __syncthreads();
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= C || !SS1_IN(m * C + c, M * C, kSiteAdaY)) return;
    float v = 0.0f;
    if (some) {
        const int64_t base = (int64_t)a * C * R + (int64_t)c * cs;
        for (int r = 0; r < R; ++r)
            if (SS1_IN(base + (int64_t)r * rs, (int64_t)n * C * R, site_t)) v = fmaf(p[r], to_f(table[base + (int64_t)r * rs]), v);
    }
    if (in) {
        if (some) out[m * C + c] = from_f<T>(to_f(in[m * C + c]) + v);
        else out[m * C + c] = in[m * C + c];
    } else {
        out[m * C + c] = from_f<T>(v);
    }
}

// The same three sums for more rows, with rows of one adapter together: each element of a table or of P that is
// read serves many rows or columns. A sub-tile is 32 rows of one of the plan's tiles.
constexpr int kSub = 32, kSubs = kTile / kSub;
constexpr int kWide = 128;    // columns of a stage

struct SubTile {
    int adapter, first, rows;
};
__device__ __forceinline__ SubTile sub_tile(const PlanView& plan, int i, int M, int n) {
    SubTile t{0, i / kSubs * kTile, min(kTile, M - i / kSubs * kTile)};
    if (plan.rows) {
        const int4 p = plan.tiles[i / kSubs];
        t = SubTile{p.x < n ? p.x : -1, p.y, p.y < 0 ? 0 : min(p.z, min(kTile, M - p.y))};
    }
    t.first += i % kSubs * kSub;
    t.rows = min(kSub, t.rows - i % kSubs * kSub);
    return t;
}
__device__ __forceinline__ int64_t plan_row(const PlanView& plan, int place, int M) {
    const int m = plan.rows ? plan.rows[place] : place;
    return (unsigned)m < (unsigned)M ? m : -1;
}

// P of a sub-tile and kRanks ranks a CTA. Stages of kWide columns of U and the table in shared memory as float; a lane is
// a row, a warp takes every eighth column and sums all ranks (16 multiply-adds for five shared-memory
// reads); the warps' sums meet at the end. The next stage's elements are loaded before this one's sums. Where
// the sub-tiles are few, a cluster's CTAs share the columns and their sums meet in distributed shared memory.
template <typename T>
__global__ void __launch_bounds__(256) tile_products_kernel(const T* __restrict__ U, const T* __restrict__ table, PlanView plan,
                                                            const float* __restrict__ scale, float* __restrict__ P, int M, int C, int R,
                                                            int n, int cs, int rs, int splits, int site_u, int site_t) {
    __shared__ float u[kSub][kWide + 1];
    __shared__ __align__(16) float t[kWide][kRanks];
    __shared__ float part[8][kRanks][kSub + 1];
    float* sums = &u[0][0];                    // once the last stage is over
    __shared__ int64_t rows[kSub];
    const SubTile tile = sub_tile(plan, blockIdx.x / splits, M, n);
    if (tile.rows <= 0) return;                // the whole cluster, here and below
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, split = blockIdx.x % splits;
    const int stages = (C + kWide - 1) / kWide, per = (stages + splits - 1) / splits;
    const int from = min(C, split * per * kWide), to = min(C, from + per * kWide);
    const int r0 = blockIdx.y * kRanks, ranks = min(kRanks, R - r0);
    if (tid < kSub) rows[tid] = tid < tile.rows ? plan_row(plan, tile.first + tid, M) : -1;
    __syncthreads();
    if (tile.adapter < 0) {        // rows without an adapter
        for (int i = split * 256 + tid; i < tile.rows * ranks; i += splits * 256) {
            const int64_t m = rows[i / ranks];
            if (m >= 0 && SS1_IN(m * R + r0 + i % ranks, (int64_t)M * R, kSiteAdaH)) P[m * R + r0 + i % ranks] = 0.0f;
        }
        return;
    }
    const int64_t base = (int64_t)tile.adapter * C * R;
    [[maybe_unused]] const int64_t tsize = (int64_t)n * C * R;
    // this thread's elements of a stage: of U a column of every second row, of the table along its contiguous side
    constexpr int kMyU = kSub * kWide / 256, kMyT = kWide * kRanks / 256, kStep = 256 / kWide;
    const int uc = tid % kWide, ur = tid / kWide;
    int tc[kMyT], tr[kMyT];
#pragma unroll
    for (int i = 0; i < kMyT; ++i) {
        const int e = tid + i * 256;
        tc[i] = rs == 1 ? e / kRanks : e % kWide;
        tr[i] = rs == 1 ? e % kRanks : e / kWide;
    }
    T nu[kMyU], nt[kMyT];
    auto fetch = [&](int c0) {
#pragma unroll
        for (int i = 0; i < kMyU; ++i) {
            const int64_t m = rows[ur + kStep * i];
            nu[i] = m >= 0 && c0 + uc < C && SS1_IN(m * C + c0 + uc, (int64_t)M * C, site_u) ? U[m * C + c0 + uc] : from_f<T>(0.0f);
        }
#pragma unroll
        for (int i = 0; i < kMyT; ++i) {
            const int64_t at = base + (int64_t)(c0 + tc[i]) * cs + (int64_t)(r0 + tr[i]) * rs;
            nt[i] = tr[i] < ranks && c0 + tc[i] < C && SS1_IN(at, tsize, site_t) ? table[at] : from_f<T>(0.0f);
        }
    };
    float s[kRanks];
#pragma unroll
    for (int r = 0; r < kRanks; ++r) s[r] = 0.0f;
    fetch(from);
    for (int c0 = from; c0 < to; c0 += kWide) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kMyU; ++i) u[ur + kStep * i][uc] = to_f(nu[i]);
#pragma unroll
        for (int i = 0; i < kMyT; ++i) t[tc[i]][tr[i]] = to_f(nt[i]);
        __syncthreads();
        if (c0 + kWide < to) fetch(c0 + kWide);
#pragma unroll
        for (int k = 0; k < kWide / 8; ++k) {
            const int c = k * 8 + warp;
            const float x = u[lane][c];
            const float4* row = reinterpret_cast<const float4*>(t[c]);
#pragma unroll
            for (int r = 0; r < kRanks / 4; ++r) {
                const float4 v = row[r];
                s[4 * r] = fmaf(x, v.x, s[4 * r]);
                s[4 * r + 1] = fmaf(x, v.y, s[4 * r + 1]);
                s[4 * r + 2] = fmaf(x, v.z, s[4 * r + 2]);
                s[4 * r + 3] = fmaf(x, v.w, s[4 * r + 3]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRanks; ++r) part[warp][r][lane] = s[r];
    __syncthreads();
    const float f = scale ? scale[tile.adapter] : 1.0f;
    for (int i = tid; i < kSub * kRanks; i += 256) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) v += part[w][i % kRanks][i / kRanks];
        sums[i] = v;
    }
    if (splits > 1) ptx::cluster_sync();
    else __syncthreads();
    for (int i = split * 256 + tid; i < kSub * kRanks; i += splits * 256) {
        const int r = i % kRanks;
        float v = 0.0f;
        if (splits > 1)
            for (int k = 0; k < splits; ++k) v += ptx::ld_cluster_f32(ptx::map_to_rank(sums + i, k));
        else
            v = sums[i];
        const int64_t m = rows[i / kRanks];
        if (m >= 0 && r < ranks && SS1_IN(m * R + r0 + r, (int64_t)M * R, kSiteAdaH)) P[m * R + r0 + r] = f * v;
    }
    if (splits > 1) ptx::cluster_sync();       // nobody leaves while its sums are being read
}

// out of `subs` sub-tiles of a tile and 256 columns: a thread is a column, its table row in registers kRanks at a time
// (and kept for all of them where R is no more), P's rows in shared memory, 32 rows at a time.
template <typename T>
__global__ void __launch_bounds__(256) tile_update_kernel(const float* __restrict__ P, const T* __restrict__ table, PlanView plan,
                                                          const float* __restrict__ scale, const T* in, T* out, int M, int C, int R, int n,
                                                          int cs, int rs, int subs, int site_t) {
    __shared__ __align__(16) float p[kSub][kRanks];
    __shared__ int64_t rows[kSub];
    const int cols = (C + 255) / 256;      // CTAs side by side
    const int tid = threadIdx.x, c = blockIdx.x % cols * 256 + tid;
    [[maybe_unused]] const int64_t total = (int64_t)M * C, tsize = (int64_t)n * C * R;
    float w[kRanks];
    for (int sub = 0; sub < subs; ++sub) {      // 1, or all of a tile's
        const SubTile tile = sub_tile(plan, blockIdx.x / cols * subs + sub, M, n);
        if (tile.rows <= 0) return;
        __syncthreads();
        if (tid < kSub) rows[tid] = tid < tile.rows ? plan_row(plan, tile.first + tid, M) : -1;
        __syncthreads();
        if (tile.adapter < 0) {
            if (in == out) return;
            T v[kSub];
#pragma unroll
            for (int i = 0; i < kSub; ++i)
                v[i] = in && c < C && rows[i] >= 0 && SS1_IN(rows[i] * C + c, total, kSiteAdaY) ? in[rows[i] * C + c] : from_f<T>(0.0f);
#pragma unroll
            for (int i = 0; i < kSub; ++i)
                if (c < C && rows[i] >= 0 && SS1_IN(rows[i] * C + c, total, kSiteAdaY)) out[rows[i] * C + c] = v[i];
            continue;
        }
        const float f = scale ? scale[tile.adapter] : 1.0f;
        const int64_t base = (int64_t)tile.adapter * C * R + (int64_t)c * cs;
        float v[kSub];
#pragma unroll
        for (int i = 0; i < kSub; ++i)
            v[i] = in && c < C && rows[i] >= 0 && SS1_IN(rows[i] * C + c, total, kSiteAdaY) ? to_f(in[rows[i] * C + c]) : 0.0f;
        for (int r0 = 0; r0 < R; r0 += kRanks) {
            if (r0 > 0) __syncthreads();
            for (int i = tid; i < kSub * kRanks; i += 256) {
                const int64_t m = rows[i / kRanks];
                const int r = r0 + i % kRanks;
                p[i / kRanks][i % kRanks] = m >= 0 && r < R ? f * P[m * R + r] : 0.0f;
            }
            if (R > kRanks || sub == 0) {
#pragma unroll
                for (int r = 0; r < kRanks; ++r) {
                    const int64_t at = base + (int64_t)(r0 + r) * rs;
                    w[r] = c < C && r0 + r < R && SS1_IN(at, tsize, site_t) ? to_f(table[at]) : 0.0f;
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
                const float4* row = reinterpret_cast<const float4*>(p[i]);
#pragma unroll
                for (int r = 0; r < kRanks / 4; ++r) {
                    const float4 x = row[r];
                    v[i] = fmaf(x.x, w[4 * r], v[i]);
                    v[i] = fmaf(x.y, w[4 * r + 1], v[i]);
                    v[i] = fmaf(x.z, w[4 * r + 2], v[i]);
                    v[i] = fmaf(x.w, w[4 * r + 3], v[i]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kSub; ++i)
            if (c < C && rows[i] >= 0 && SS1_IN(rows[i] * C + c, total, kSiteAdaY)) out[rows[i] * C + c] = from_f<T>(v[i]);
    }
}

// D_a[c, r] = f * sum over adapter a's rows of U[m, c] P[m, r], dA and dB in one launch (each CTA of either), for one
// share of the rows (blockIdx.z): element (share, a, c, r) at share * n * C * R + a * C * R + c * cs + r * rs of D, or of
// `out` where there is one share. A thread is a column; 32 rows' P lie in shared memory, and 32 rows of U are on
// their way at a time.
template <typename T>
struct ColumnSums {
    const T* U;
    const float* P;
    const float* scale;
    float* D;
    T* out;
    int C, cs, rs, shares, blocks, site;     // blocks: of 128 columns; 0: not wanted
};

template <typename T>
__global__ void __launch_bounds__(128) column_sums_kernel(const ColumnSums<T> da, const ColumnSums<T> db, PlanView plan, int64_t M, int R,
                                                          int n) {
    const bool second = (int)blockIdx.x >= da.blocks;
    const ColumnSums<T>& d = second ? db : da;
    const T* __restrict__ U = d.U;
    const float* __restrict__ P = d.P;
    const int C = d.C, cs = d.cs, rs = d.rs, shares = d.shares;
    [[maybe_unused]] const int site_u = d.site;
    if ((int)blockIdx.z >= shares) return;
    __shared__ __align__(16) float p[kSub][kRanks];
    __shared__ int64_t rows[kSub];
    const int a = blockIdx.y % n, r0 = (blockIdx.y / n) * kRanks, ranks = min(kRanks, R - r0);
    const int c = ((int)blockIdx.x - (second ? da.blocks : 0)) * 128 + threadIdx.x;
    const int begin = plan.rows ? max(0, plan.first[a]) : 0, end = plan.rows ? min((int)M, plan.first[a + 1]) : (int)M;
    const int per = (max(0, end - begin) + shares - 1) / shares;
    const int from = begin + (int)blockIdx.z * per, to = min(end, from + per);
    float s[kRanks];
#pragma unroll
    for (int r = 0; r < kRanks; ++r) s[r] = 0.0f;
    for (int at = from; at < to; at += kSub) {
        __syncthreads();
        if (threadIdx.x < kSub) rows[threadIdx.x] = at + (int)threadIdx.x < to ? plan_row(plan, at + threadIdx.x, (int)M) : -1;
        __syncthreads();
        T u[kSub];
#pragma unroll
        for (int i = 0; i < kSub; ++i)
            u[i] = rows[i] >= 0 && c < C && SS1_IN(rows[i] * C + c, M * C, site_u) ? U[rows[i] * C + c] : from_f<T>(0.0f);
        for (int i = threadIdx.x; i < kSub * kRanks; i += 128) {
            const int64_t m = rows[i / kRanks];
            const int r = i % kRanks;
            p[i / kRanks][r] = m >= 0 && r < ranks ? P[m * R + r0 + r] : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSub; ++i) {
            const float x = to_f(u[i]);
            const float4* row = reinterpret_cast<const float4*>(p[i]);
#pragma unroll
            for (int r = 0; r < kRanks / 4; ++r) {
                const float4 v = row[r];
                s[4 * r] = fmaf(x, v.x, s[4 * r]);
                s[4 * r + 1] = fmaf(x, v.y, s[4 * r + 1]);
                s[4 * r + 2] = fmaf(x, v.z, s[4 * r + 2]);
                s[4 * r + 3] = fmaf(x, v.w, s[4 * r + 3]);
            }
        }
    }
    if (c >= C) return;
    const float f = d.scale ? d.scale[a] : 1.0f;
    const int64_t size = (int64_t)n * C * R;
    const int64_t base = (int64_t)blockIdx.z * size + (int64_t)a * C * R + (int64_t)c * cs;
#pragma unroll
    for (int r = 0; r < kRanks; ++r)
        if (r < ranks && SS1_IN(base + (int64_t)(r0 + r) * rs, size * shares, kSiteAdaPart)) {
            if (shares == 1) d.out[base + (int64_t)(r0 + r) * rs] = from_f<T>(f * s[r]);
            else d.D[base + (int64_t)(r0 + r) * rs] = f * s[r];
        }
}

// The shares' partial sums of dA (blockIdx.y 0) and dB, added in share order; one share has written its result itself.
template <typename T>
__global__ void __launch_bounds__(256) add_shares_kernel(const ColumnSums<T> da, const ColumnSums<T> db, int R, int n) {
    const ColumnSums<T>& d = blockIdx.y ? db : da;
    const int64_t size = (int64_t)n * d.C * R, i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (d.blocks == 0 || d.shares == 1 || i >= size) return;
    float s = 0.0f;
    for (int k = 0; k < d.shares; ++k) s += d.D[k * size + i];
    d.out[i] = from_f<T>(s);
}

// A CTA takes one row while that reads no more than kAloneWork elements of A and B; beyond, 32 rows of an adapter
// together, with a plan. Measured forward, us, a row / 32 rows: float32 333 x 1001 x 770, rank 6 (3.5 M elements) 9.9 / 16.6;
// 200 x 1024 x 1024, rank 16 (6.5 M) 14.7 / 16.6; bf16 200 x 3001 x 5001, rank 16 (26 M) 31 / 25; float32
// 1024 x 1024 x 1024, rank 16 (34 M) 46 / 13.
constexpr int64_t kAloneWork = 1 << 23;
bool alone(const Call& c) { return c.M <= 65535 && c.M * c.R * (c.K + c.N) <= kAloneWork; }

// P[m] = f U[m] T_a and out[m] = in[m] + f P[m] T_a, whichever way suits the rows.
template <typename T>
cudaError_t products(const Call& c, const void* U, const void* table, const float* scale, float* P, int64_t C, int cs, int rs, int site_u,
                     int site_t, cudaStream_t st) {
    const unsigned ranks = (unsigned)((c.R + kRanks - 1) / kRanks);
    if (alone(c))
        row_products_kernel<T><<<dim3((unsigned)c.M, ranks), 256, 0, st>>>((const T*)U, (const T*)table, c.index, scale, P, c.M, (int)C, c.R,
                                                                          c.n, cs, rs, site_u, site_t);
    else {
        // two CTAs for each of 148 SMs, at least two stages each, clusters of a portable size
        const int64_t subs = sub_tiles(c), stages = (C + kWide - 1) / kWide;
        int64_t splits = 296 / (subs * ranks);
        splits = splits > stages / 2 ? stages / 2 : splits;
        splits = splits > 8 ? 8 : (splits < 1 ? 1 : splits);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(subs * splits), ranks);
        cfg.blockDim = dim3(256);
        cfg.stream = st;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)splits;
        at[0].val.clusterDim.y = 1;
        at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, &tile_products_kernel<T>, (const T*)U, (const T*)table, c.plan, scale, P, (int)c.M, (int)C, c.R, c.n,
                                  cs, rs, (int)splits, site_u, site_t);
    }
    return cudaGetLastError();
}
template <typename T>
cudaError_t update(const Call& c, const float* P, const void* table, const float* scale, const void* in, void* out, int64_t C, int cs, int rs,
                   int site_t, cudaStream_t st) {
    const unsigned cols = (unsigned)((C + 255) / 256);
    if (alone(c))
        row_update_kernel<T><<<dim3(cols, (unsigned)c.M), 256, 0, st>>>(P, (const T*)table, c.index, scale, (const T*)in, (T*)out, c.M, (int)C,
                                                                       c.R, c.n, cs, rs, site_t);
    else {
        // a whole tile a CTA (its table row read once) where that still gives eight CTAs for each of 148 SMs: bf16
        // 4000 x 4001 x 4003, rank 16, 134 us against 147; 32 rows a CTA elsewhere: float32 1024 x 1024 x 1024 13 against 25
        const int subs = sub_tiles(c) / kSubs * cols >= 148 * 8 ? kSubs : 1;
        const int64_t ctas = sub_tiles(c) / subs * cols;
        if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
        tile_update_kernel<T><<<(unsigned)ctas, 256, 0, st>>>(P, (const T*)table, c.plan, scale, (const T*)in, (T*)out, (int)c.M, (int)C, c.R,
                                                             c.n, cs, rs, subs, site_t);
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t forward_general(const Call& c, const void* X, const void* Y, void* out, float* H, cudaStream_t st) {
    const cudaError_t e = products<T>(c, X, c.A, nullptr, H, c.K, 1, (int)c.K, kSiteAdaX, kSiteAdaA, st);
    if (e != cudaSuccess) return e;
    return update<T>(c, H, c.B, c.scale, Y, out, c.N, c.R, 1, kSiteAdaB, st);
}

// dA = G^T X and dB = s dY^T H, whichever are wanted.
template <typename T>
cudaError_t column_sums(const Call& c, const void* dY, const void* X, const float* H, const float* G, void* dA, void* dB, float* part_a,
                        float* part_b, cudaStream_t st) {
    const int sa = general_shares(c.M, c.K, c.R, c.n), sb = general_shares(c.M, c.N, c.R, c.n);
    const ColumnSums<T> da{(const T*)X, G, nullptr, part_a, (T*)dA, (int)c.K, 1, (int)c.K, sa, dA ? (int)((c.K + 127) / 128) : 0, kSiteAdaX};
    const ColumnSums<T> db{(const T*)dY, H, c.scale, part_b, (T*)dB, (int)c.N, c.R, 1, sb, dB ? (int)((c.N + 127) / 128) : 0, kSiteAdaY};
    const int shares = std::max(dA ? sa : 1, dB ? sb : 1);
    const dim3 grid((unsigned)(da.blocks + db.blocks), (unsigned)(c.n * ((c.R + kRanks - 1) / kRanks)), (unsigned)shares);
    column_sums_kernel<T><<<grid, 128, 0, st>>>(da, db, c.plan, c.M, c.R, c.n);
    const int64_t size = (int64_t)c.n * std::max(dA ? c.K : 0, dB ? c.N : 0) * c.R;
    if (shares > 1) add_shares_kernel<T><<<dim3((unsigned)((size + 255) / 256), 2), 256, 0, st>>>(da, db, c.R, c.n);
    return cudaGetLastError();
}

template <typename T>
cudaError_t backward_general(const Call& c, const void* dY, const void* X, const float* H, const void* dX_in, void* dX,
                             void* dA, void* dB, float* G, float* part_a, float* part_b, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (dX || dA) e = products<T>(c, dY, c.B, c.scale, G, c.N, c.R, 1, kSiteAdaY, kSiteAdaB, st);
    if (e == cudaSuccess && dX) e = update<T>(c, G, c.A, nullptr, dX_in, dX, c.K, 1, (int)c.K, kSiteAdaA, st);
    if (e == cudaSuccess && (dA || dB)) e = column_sums<T>(c, dY, X, H, G, dA, dB, part_a, part_b, st);
    return e;
}

constexpr size_t align_up(size_t v) { return (v + 255) & ~(size_t)255; }

bool sizes_ok(int64_t M, int64_t K, int64_t N, int R, int n, int dtype) {
    if (M < 0 || M > (1 << 30) || K < 1 || N < 1 || K > (1 << 24) || N > (1 << 24)) return false;
    if (R < 1 || R > kMaxRank || n < 1 || n > kMaxCount || !dtype_ok(dtype)) return false;
    return (K > N ? K : N) * R * n <= (int64_t)1 << 38;   // what one grid of 256 elements a CTA covers
}

// The workspaces: the plan, then what the path needs. They hold either path's, so that a workspace's size
// does not depend on the alignment of the other pointers.
struct Sizes {
    size_t plan;
    size_t rows, sums_a, sums_b;                        // general path: H or G; the partial sums of dA and dB
    size_t packed, wide_b, turned_a, part_a, part_b;    // tensor-core path
    size_t forward() const { return plan + (rows > packed + wide_b ? rows : packed + wide_b); }
    size_t backward() const {
        const size_t a = rows + sums_a + sums_b, b = 2 * packed + wide_b + turned_a + part_a + part_b;
        return plan + (a > b ? a : b);
    }
};
Sizes workspace_of(int64_t M, int64_t K, int64_t N, int R, int n) {
    Sizes s = {};
    s.plan = align_up(plan_bytes(M, n));
    s.rows = align_up((size_t)M * R * sizeof(float));
    const size_t a = (size_t)n * K * R, b = (size_t)n * N * R;
    s.sums_a = align_up(general_shares(M, K, R, n) * a * sizeof(float));
    s.sums_b = align_up(general_shares(M, N, R, n) * b * sizeof(float));
    s.packed = align_up((size_t)M * mma_rank(R) * 2 * sizeof(uint16_t));
    s.wide_b = R % 8 ? align_up((size_t)n * N * ((R + 7) / 8 * 8) * sizeof(uint16_t)) : 0;
    s.turned_a = align_up((size_t)n * K * ((R + 7) / 8 * 8) * sizeof(uint16_t));
    s.part_a = align_up((size_t)(mma_runs(M, K, n) + n) * K * R * sizeof(float));
    s.part_b = align_up((size_t)(mma_runs(M, N, n) + n) * N * R * sizeof(float));
    return s;
}

// The tensor-core path takes bf16 rows on 16-byte boundaries (and B's rows too, where R allows it), and as
// many tiles and column ranges as a grid's second dimension.
bool mma_shape(const ss1_adapters& ad, int64_t M) {
    return ad.dtype == SS1_DTYPE_BF16 && ad.K % 8 == 0 && ad.N % 8 == 0 && aligned(ad.A, 16) && (ad.R % 8 || aligned(ad.B, 16)) &&
           max_tiles(M, ad.count) <= 32768 && ad.K <= 1 << 22 && ad.N <= 1 << 22;
}

// What the calls have in common; `status` other than SS1_OK refuses.
int check(const ss1_adapters* ad, int64_t M) {
    if (!ad || !sizes_ok(M, ad->K, ad->N, ad->R, ad->count, ad->dtype)) return SS1_ERR_INVALID_ARG;
    if (M == 0) return SS1_OK;
    if (!ad->index && ad->count != 1) return SS1_ERR_INVALID_ARG;
    if (!ad->A || !ad->B) return SS1_ERR_INVALID_ARG;
    const size_t e = dtype_size(ad->dtype);
    if (!aligned(ad->A, e) || !aligned(ad->B, e) || !aligned(ad->scale, 4) || !aligned(ad->index, 4) || !aligned(ad->plan, 256))
        return SS1_ERR_MISALIGNED;
    return SS1_OK;
}

Call call_of(const ss1_adapters& ad, int64_t M) {
    Call c;
    c.A = ad.A; c.B = ad.B; c.scale = ad.scale; c.index = ad.index;
    c.M = M; c.K = ad.K; c.N = ad.N; c.R = ad.R; c.n = ad.count;
    c.plan = PlanView{};
    c.planned = false;
    return c;
}

// c.plan: the caller's plan, or one made at `ws`; none where every row uses adapter 0.
cudaError_t plan_of(const ss1_adapters& ad, int64_t M, void* ws, Call& c, cudaStream_t st) {
    if (!ad.index) return cudaSuccess;
    c.plan = plan_view(ad.plan ? const_cast<void*>(ad.plan) : ws, M, ad.count);
    c.planned = ad.plan == nullptr;
    return ad.plan ? cudaSuccess : launch_plan(ad.index, M, ad.count, c.plan, st);
}

// A forward runs a row a cluster up to kFewRows rows, while these read no more than kFewWork elements of A and B
// (each row reads its own). Measured as graph replays, that and the tensor-core kernels (with their
// plan), us: K = N = 4096, R = 16, 24 adapters: 5.3 / 13.9 at 48 rows, 6.4 / 14.2 at 64, 15.8 / 14.8 at 192;
// K = 4096, N = 14336, R = 16: 8.6 / 13.9 at 48 rows, 16.7 / 14.7 at 96; R = 64, N = 4096: 9.2 / 14.3 at 16 rows,
// 15.0 / 14.4 at 48. One adapter of rank 8 on 768 x 2304 (no plan): 4.6 / 6.5 at 64 rows, 7.5 / 7.2 at 96.
constexpr int64_t kFewRows = 64, kFewWork = 1 << 24;

bool rows_shape(const ss1_adapters& ad, int64_t M) {
    return M <= kFewRows && M * ad.R * (ad.K + ad.N) <= kFewWork && ad.K % 8 == 0 && ad.N % 8 == 0 && ad.R % 8 == 0 && aligned(ad.A, 16) && aligned(ad.B, 16);
}

}  // namespace

int general_shares(int64_t M, int64_t C, int R, int n) {
    // enough CTAs for the machine, at least 64 rows a share
    const int64_t ctas = (C + 127) / 128 * n * ((R + kRanks - 1) / kRanks);
    int64_t s = 592 / ctas;
    if (s > M / 64) s = M / 64;
    return (int)(s < 1 ? 1 : (s > 16 ? 16 : s));
}

size_t plan_bytes(int64_t M, int n) {
    return (2 * ((size_t)(n + 2 + 3) / 4 * 4) + 4 * (size_t)max_tiles(M, n) + (size_t)M) * sizeof(int32_t);
}

PlanView plan_view(void* plan, int64_t M, int n) {
    PlanView v;
    v.first = static_cast<int32_t*>(plan);
    v.max_tiles = max_tiles(M, n);
    v.first_tile = v.first + (n + 2 + 3) / 4 * 4;
    v.tiles = reinterpret_cast<int4*>(v.first_tile + (n + 2 + 3) / 4 * 4);
    v.rows = reinterpret_cast<int32_t*>(v.tiles + v.max_tiles);
    return v;
}

}  // namespace ada
}  // namespace ss1

using namespace ss1;
using namespace ss1::op;
using namespace ss1::ada;

extern "C" SS1_API int ss1_adapter_plan_bytes(int64_t M, int count, size_t* bytes) {
    if (!bytes || !sizes_ok(M, 1, 1, 1, count, SS1_DTYPE_FP32)) return SS1_ERR_INVALID_ARG;
    *bytes = plan_bytes(M, count);
    return SS1_OK;
}

extern "C" SS1_API int ss1_adapter_plan(const int32_t* index, int64_t M, int count, void* plan, size_t bytes_of_plan, void* stream) {
    if (!sizes_ok(M, 1, 1, 1, count, SS1_DTYPE_FP32)) return SS1_ERR_INVALID_ARG;
    if (!plan || (M > 0 && !index) || bytes_of_plan < plan_bytes(M, count)) return SS1_ERR_INVALID_ARG;
    if (!aligned(plan, 256) || !aligned(index, 4)) return SS1_ERR_MISALIGNED;
    if (launch_plan(index, M, count, plan_view(plan, M, count), static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return SS1_ERR_CUDA;
    }
    return SS1_OK;
}

extern "C" SS1_API int ss1_adapter_workspace(int64_t M, int64_t K, int64_t N, int R, int count, int dtype, size_t* forward_bytes,
                                             size_t* backward_bytes) {
    if (!sizes_ok(M, K, N, R, count, dtype)) return SS1_ERR_INVALID_ARG;
    const Sizes s = workspace_of(M, K, N, R, count);
    if (forward_bytes) *forward_bytes = s.forward();
    if (backward_bytes) *backward_bytes = s.backward();
    return SS1_OK;
}

extern "C" SS1_API int ss1_adapter_forward(const ss1_adapters* ad, const void* X, const void* Y, void* out, float* H, int64_t M,
                                           void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = check(ad, M);
    if (rc != SS1_OK || M == 0) return rc;
    if (!X || !Y || !out) return SS1_ERR_INVALID_ARG;
    const size_t e = dtype_size(ad->dtype);
    if (!aligned(X, e) || !aligned(Y, e) || !aligned(out, e) || !aligned(H, 4) || !aligned(workspace, 256)) return SS1_ERR_MISALIGNED;
    const Sizes s = workspace_of(M, ad->K, ad->N, ad->R, ad->count);
    if (!workspace || workspace_bytes < s.forward()) return SS1_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    Call c = call_of(*ad, M);
    cudaError_t err = cudaSuccess;
    const bool vec = aligned(X, 16) && aligned(Y, 16) && aligned(out, 16);
    if (vec && rows_shape(*ad, M)) {
        if (rows_forward(c, X, Y, out, H, ad->dtype, st) != cudaSuccess) { cudaGetLastError(); return SS1_ERR_CUDA; }
        return SS1_OK;
    }
    if (vec && mma_shape(*ad, M)) {
        err = plan_of(*ad, M, ws, c, st);
        const MmaSpace w{ws + s.plan, nullptr, ws + s.plan + s.packed, nullptr, nullptr, nullptr};
        if (err == cudaSuccess) err = mma_forward(c, X, Y, out, H, w, st);
        if (err != cudaSuccess) { cudaGetLastError(); return SS1_ERR_CUDA; }
        return SS1_OK;
    }
    if (!H) H = reinterpret_cast<float*>(ws + s.plan);
    if (!alone(c)) err = plan_of(*ad, M, ws, c, st);
    if (err == cudaSuccess)
        err = ad->dtype == SS1_DTYPE_BF16 ? forward_general<__nv_bfloat16>(c, X, Y, out, H, st)
                                                        : forward_general<float>(c, X, Y, out, H, st);
    if (err != cudaSuccess) { cudaGetLastError(); return SS1_ERR_CUDA; }
    return SS1_OK;
}

// `test`: the time-out test, on the tensor-core path or not at all.
static int adapter_backward(const ss1_adapters* ad, const void* dY, const void* X, const float* H, const void* dX_in, void* dX, void* dA,
                            void* dB, int64_t M, void* workspace, size_t workspace_bytes, const Watch* test, void* stream) {
    const int rc = check(ad, M);
    if (rc != SS1_OK) return rc;
    const size_t e = dtype_size(ad->dtype);
    if (!aligned(dY, e) || !aligned(X, e) || !aligned(H, 4) || !aligned(dX_in, e) || !aligned(dX, e) || !aligned(dA, e) ||
        !aligned(dB, e) || !aligned(workspace, 256))
        return SS1_ERR_MISALIGNED;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    if (M == 0) {   // no rows: the adapters' gradients are zero
        if (dA) err = cudaMemsetAsync(dA, 0, (size_t)ad->count * ad->R * ad->K * e, st);
        if (err == cudaSuccess && dB) err = cudaMemsetAsync(dB, 0, (size_t)ad->count * ad->R * ad->N * e, st);
        if (err != cudaSuccess) { cudaGetLastError(); return SS1_ERR_CUDA; }
        return SS1_OK;
    }
    if (!dX && !dA && !dB) return SS1_OK;
    if (!dY || (dA && !X) || (dB && !H) || (dX_in && !dX)) return SS1_ERR_INVALID_ARG;
    const Sizes s = workspace_of(M, ad->K, ad->N, ad->R, ad->count);
    if (!workspace || workspace_bytes < s.backward()) return SS1_ERR_INVALID_ARG;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    Call c = call_of(*ad, M);
    const bool mma = mma_shape(*ad, M) && aligned(dY, 16) && aligned(X, 16) && aligned(dX_in, 16) && aligned(dX, 16);
    if (test && !mma) return SS1_ERR_UNSUPPORTED_SHAPE;
    err = plan_of(*ad, M, ws, c, st);
    if (err == cudaSuccess && mma) {
        uint8_t* at = ws + s.plan;
        MmaSpace w;
        w.packed_g = at; at += s.packed;
        w.packed_h = at; at += s.packed;
        w.wide_b = at; at += s.wide_b;
        w.turned_a = at; at += s.turned_a;
        w.part_a = reinterpret_cast<float*>(at); at += s.part_a;
        w.part_b = reinterpret_cast<float*>(at);
        err = mma_backward(c, dY, X, H, dX_in, dX, dA, dB, w, test, st);
        if (err != cudaSuccess) { cudaGetLastError(); return SS1_ERR_CUDA; }
        return SS1_OK;
    }
    float* G = reinterpret_cast<float*>(ws + s.plan);
    float* part_a = reinterpret_cast<float*>(ws + s.plan + s.rows);
    float* part_b = reinterpret_cast<float*>(ws + s.plan + s.rows + s.sums_a);
    if (err == cudaSuccess)
        err = ad->dtype == SS1_DTYPE_BF16 ? backward_general<__nv_bfloat16>(c, dY, X, H, dX_in, dX, dA, dB, G, part_a, part_b, st)
                                          : backward_general<float>(c, dY, X, H, dX_in, dX, dA, dB, G, part_a, part_b, st);
    if (err != cudaSuccess) { cudaGetLastError(); return SS1_ERR_CUDA; }
    return SS1_OK;
}

extern "C" SS1_API int ss1_adapter_backward(const ss1_adapters* ad, const void* dY, const void* X, const float* H, const void* dX_in,
                                            void* dX, void* dA, void* dB, int64_t M, void* workspace, size_t workspace_bytes,
                                            void* stream) {
    return adapter_backward(ad, dY, X, H, dX_in, dX, dA, dB, M, workspace, workspace_bytes, nullptr, stream);
}

extern "C" SS1_API int ss1_test_adapter_timeout(const ss1_adapters* ad, const void* dY, const void* X, const float* H, const void* dX_in,
                                                void* dX, void* dA, void* dB, int64_t M, void* workspace, size_t workspace_bytes,
                                                int site, int64_t limit_ns, void* stream) {
    if (site < kTimeoutG || site > kTimeoutDa || limit_ns < 1 || limit_ns > 2000000000 || M < 1 || !dX || !dA || !dB)
        return SS1_ERR_INVALID_ARG;
    const Watch watch{(uint64_t)limit_ns, site};
    return adapter_backward(ad, dY, X, H, dX_in, dX, dA, dB, M, workspace, workspace_bytes, &watch, stream);
}

extern "C" SS1_API int ss1_adapter_status(int32_t* detail) {
    int32_t v = 0;
    if (mma_status(&v) != cudaSuccess) { cudaGetLastError(); return SS1_ERR_CUDA; }
    if (detail) *detail = v;
    return v == 0 ? SS1_OK : SS1_ERR_DEVICE_TIMEOUT;
}
