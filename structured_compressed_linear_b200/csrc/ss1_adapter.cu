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

namespace ss1 {
namespace ada {

using namespace op;

// ---- plan ------------------------------------------------------------------------------------

// One CTA. Every warp counts its own contiguous share of the rows by adapter (lanes with the same
// adapter find one another by a ballot for each bit of its number: one __match_any_sync takes a step for every
// different value, 18 us for 8192 rows of 32 adapters in random order), the counts are scanned over
// adapters and warps, and each row's place is what comes before it: rows keep their order within an
// adapter. The first kAhead index words of a lane are loaded together, and their places within the warp kept
// (32 warps cover 16,384 rows that way): one memory latency, and one walk; rows beyond are walked twice.
constexpr int kAhead = 16;

__device__ __forceinline__ int plan_group(const int32_t* __restrict__ index, int row, int end, int n) {
    if (row >= end) return -1;
    const int a = index[row];
    return (unsigned)a < (unsigned)n ? a : n;
}

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
    int ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) ahead[i] = plan_group(index, begin + i * 32 + lane, end, n);
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
    int nth[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) nth[i] = begin + i * 32 < end ? count(ahead[i]) : 0;
    for (int at = begin + kAhead * 32; at < end; at += 32) count(plan_group(index, at + lane, end, n));
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
    for (int i = 0; i < kAhead; ++i)
        if (ahead[i] >= 0) put(ahead[i], begin + i * 32 + lane, so_far[ahead[i]] + nth[i]);
    if (begin + kAhead * 32 >= end) return;    // the whole warp
    __syncwarp();
    // the second walk counts on from the first kAhead rounds
#pragma unroll
    for (int i = 0; i < kAhead; ++i) count(ahead[i]);
    for (int at = begin + kAhead * 32; at < end; at += 32) {
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
    return launch_dependent(&plan_kernel, dim3(1), dim3((unsigned)(warps * 32)), smem, st, index, (int)M, n, plan);
}

namespace {

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
    const int64_t m = blockIdx.y + (int64_t)blockIdx.z * 65535;
    if (m >= M) return;
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

// D_a[c, r] = f * sum over adapter a's rows of U[m, c] P[m, r], for one share of the rows (blockIdx.z):
// element (share, a, c, r) at share * n * C * R + a * C * R + c * cs + r * rs.
template <typename T>
__global__ void __launch_bounds__(128) column_sums_kernel(const T* __restrict__ U, const float* __restrict__ P, PlanView plan,
                                                          const float* __restrict__ scale, float* __restrict__ D, int64_t M,
                                                          int C, int R, int n, int cs, int rs, int site_u) {
    const int a = blockIdx.y % n, r0 = (blockIdx.y / n) * kRanks, ranks = min(kRanks, R - r0);
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= C) return;
    const int begin = plan.rows ? plan.first[a] : 0, end = plan.rows ? plan.first[a + 1] : (int)M;
    const int shares = gridDim.z, per = (end - begin + shares - 1) / shares;
    const int from = begin + (int)blockIdx.z * per, to = min(end, from + per);
    float s[kRanks];
#pragma unroll
    for (int r = 0; r < kRanks; ++r) s[r] = 0.0f;
    for (int i = from; i < to; ++i) {
        const int64_t m = plan.rows ? plan.rows[i] : i;
        if ((uint64_t)m >= (uint64_t)M || !SS1_IN(m * C + c, M * C, site_u)) continue;
        const float u = to_f(U[m * C + c]);
#pragma unroll
        for (int r = 0; r < kRanks; ++r)
            if (r < ranks) s[r] = fmaf(u, P[m * R + r0 + r], s[r]);
    }
    const float f = scale ? scale[a] : 1.0f;
    const int64_t size = (int64_t)n * C * R;
    const int64_t base = (int64_t)blockIdx.z * size + (int64_t)a * C * R + (int64_t)c * cs;
#pragma unroll
    for (int r = 0; r < kRanks; ++r)
        if (r < ranks && SS1_IN(base + (int64_t)(r0 + r) * rs, size * shares, kSiteAdaPart)) D[base + (int64_t)(r0 + r) * rs] = f * s[r];
}

// out[i] = the shares' partial sums, added in share order.
template <typename T>
__global__ void __launch_bounds__(256) add_shares_kernel(const float* __restrict__ part, T* __restrict__ out, int64_t size,
                                                         int shares) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= size) return;
    float s = 0.0f;
    for (int k = 0; k < shares; ++k) s += part[k * size + i];
    out[i] = from_f<T>(s);
}

template <typename T>
cudaError_t forward_general(const Call& c, const void* X, const void* Y, void* out, float* H, cudaStream_t st) {
    const dim3 grid((unsigned)c.M, (unsigned)((c.R + kRanks - 1) / kRanks));
    row_products_kernel<T><<<grid, 256, 0, st>>>((const T*)X, (const T*)c.A, c.index, nullptr, H, c.M, (int)c.K, c.R, c.n, 1,
                                                 (int)c.K, kSiteAdaX, kSiteAdaA);
    const dim3 egrid((unsigned)((c.N + 255) / 256), (unsigned)(c.M < 65535 ? c.M : 65535), (unsigned)((c.M + 65534) / 65535));
    row_update_kernel<T><<<egrid, 256, 0, st>>>(H, (const T*)c.B, c.index, c.scale, (const T*)Y, (T*)out, c.M, (int)c.N, c.R, c.n,
                                                c.R, 1, kSiteAdaB);
    return cudaGetLastError();
}

template <typename T>
cudaError_t column_sums(const Call& c, const void* U, const float* P, const float* scale, void* D, float* part, int64_t C, int cs,
                        int rs, int site, cudaStream_t st) {
    const int shares = general_shares(c.M, C, c.R, c.n);
    const dim3 grid((unsigned)((C + 127) / 128), (unsigned)(c.n * ((c.R + kRanks - 1) / kRanks)), (unsigned)shares);
    column_sums_kernel<T><<<grid, 128, 0, st>>>((const T*)U, P, c.plan, scale, part, c.M, (int)C, c.R, c.n, cs, rs, site);
    const int64_t size = (int64_t)c.n * C * c.R;
    add_shares_kernel<T><<<(unsigned)((size + 255) / 256), 256, 0, st>>>(part, (T*)D, size, shares);
    return cudaGetLastError();
}

template <typename T>
cudaError_t backward_general(const Call& c, const void* dY, const void* X, const float* H, const void* dX_in, void* dX,
                             void* dA, void* dB, float* G, float* part, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (dX || dA) {
        const dim3 grid((unsigned)c.M, (unsigned)((c.R + kRanks - 1) / kRanks));
        row_products_kernel<T><<<grid, 256, 0, st>>>((const T*)dY, (const T*)c.B, c.index, c.scale, G, c.M, (int)c.N, c.R, c.n, c.R,
                                                     1, kSiteAdaY, kSiteAdaB);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess && dX) {
        const dim3 grid((unsigned)((c.K + 255) / 256), (unsigned)(c.M < 65535 ? c.M : 65535), (unsigned)((c.M + 65534) / 65535));
        row_update_kernel<T><<<grid, 256, 0, st>>>(G, (const T*)c.A, c.index, nullptr, (const T*)dX_in, (T*)dX, c.M, (int)c.K, c.R,
                                                   c.n, 1, (int)c.K, kSiteAdaA);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess && dA) e = column_sums<T>(c, X, G, nullptr, dA, part, c.K, 1, (int)c.K, kSiteAdaX, st);
    if (e == cudaSuccess && dB) e = column_sums<T>(c, dY, H, c.scale, dB, part, c.N, c.R, 1, kSiteAdaY, st);
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
    size_t rows, part;                                  // general path: H or G; the partial sums of dA or dB
    size_t packed, wide_b, turned_a, part_a, part_b;    // tensor-core path
    size_t forward() const { return plan + (rows > packed + wide_b ? rows : packed + wide_b); }
    size_t backward() const {
        const size_t a = rows + part, b = 2 * packed + wide_b + turned_a + part_a + part_b;
        return plan + (a > b ? a : b);
    }
};
Sizes workspace_of(int64_t M, int64_t K, int64_t N, int R, int n) {
    Sizes s = {};
    s.plan = align_up(plan_bytes(M, n));
    s.rows = align_up((size_t)M * R * sizeof(float));
    const size_t a = (size_t)n * K * R, b = (size_t)n * N * R;
    const size_t ga = general_shares(M, K, R, n) * a, gb = general_shares(M, N, R, n) * b;
    s.part = align_up((ga > gb ? ga : gb) * sizeof(float));
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
    return c;
}

// c.plan: the caller's plan, or one made at `ws`; none where every row uses adapter 0.
cudaError_t plan_of(const ss1_adapters& ad, int64_t M, void* ws, Call& c, cudaStream_t st) {
    if (!ad.index) return cudaSuccess;
    c.plan = plan_view(ad.plan ? const_cast<void*>(ad.plan) : ws, M, ad.count);
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
    err = ad->dtype == SS1_DTYPE_BF16 ? forward_general<__nv_bfloat16>(c, X, Y, out, H, st)
                                                        : forward_general<float>(c, X, Y, out, H, st);
    if (err != cudaSuccess) { cudaGetLastError(); return SS1_ERR_CUDA; }
    return SS1_OK;
}

extern "C" SS1_API int ss1_adapter_backward(const ss1_adapters* ad, const void* dY, const void* X, const float* H, const void* dX_in,
                                            void* dX, void* dA, void* dB, int64_t M, void* workspace, size_t workspace_bytes,
                                            void* stream) {
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
    err = plan_of(*ad, M, ws, c, st);
    if (err == cudaSuccess && mma_shape(*ad, M) && aligned(dY, 16) && aligned(X, 16) && aligned(dX_in, 16) &&
        aligned(dX, 16)) {
        uint8_t* at = ws + s.plan;
        MmaSpace w;
        w.packed_g = at; at += s.packed;
        w.packed_h = at; at += s.packed;
        w.wide_b = at; at += s.wide_b;
        w.turned_a = at; at += s.turned_a;
        w.part_a = reinterpret_cast<float*>(at); at += s.part_a;
        w.part_b = reinterpret_cast<float*>(at);
        err = mma_backward(c, dY, X, H, dX_in, dX, dA, dB, w, st);
        if (err != cudaSuccess) { cudaGetLastError(); return SS1_ERR_CUDA; }
        return SS1_OK;
    }
    float* G = reinterpret_cast<float*>(ws + s.plan);
    float* part = reinterpret_cast<float*>(ws + s.plan + s.rows);
    if (err == cudaSuccess)
        err = ad->dtype == SS1_DTYPE_BF16 ? backward_general<__nv_bfloat16>(c, dY, X, H, dX_in, dX, dA, dB, G, part, st)
                                          : backward_general<float>(c, dY, X, H, dX_in, dX, dA, dB, G, part, st);
    if (err != cudaSuccess) { cudaGetLastError(); return SS1_ERR_CUDA; }
    return SS1_OK;
}
