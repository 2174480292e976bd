// Layer norm over the rows of X [M, K], and its backward pass.
//
//     mean = (1/K) sum_k x_k,   rstd = 1 / sqrt((1/K) sum_k (x_k - mean)^2 + eps),
//     xhat = (x - mean) rstd,   y = xhat w + b
//     g = dy w,   dx = rstd (g - mean_k(g) - xhat mean_k(g xhat)),
//     dw = sum_m dy xhat,       db = sum_m dy
//
// Both passes move bytes: forward reads X once and writes Y once, backward reads X and dY once and
// writes dX once; the weights and statistics are small. So a row is read into registers once and
// everything is computed from there: the variance from the deviations (a second pass over the
// registers, not over memory), never from sum x^2 - mean^2, which loses all digits where |mean|
// is large. All sums are float32.
#include "ss1_ops.cuh"

namespace ss1 {
namespace {

using namespace op;

constexpr int kUnit = 8;   // elements a thread takes at a time: 16 bytes of bf16, 32 of float

// Eight elements of a row. Vector form: consecutive, from 8 * (unit * width + t); scalar form (rows
// that do not start on 16-byte boundaries): strided by the width, so that a warp's loads stay
// together. `n` is what is left of the row from the unit's first element.
template <bool VEC>
__device__ __forceinline__ int unit_first(int unit, int width, int t) {
    return VEC ? (unit * width + t) * kUnit : unit * width * kUnit + t;
}

template <typename T, bool VEC>
__device__ __forceinline__ void load_unit(const T* __restrict__ p, int64_t base, int64_t total, int first, int width,
                                          int K, float (&f)[kUnit], int site) {
    if (VEC) {
        Raw8<T> r;
        if (first < K && SS1_SPAN_IN(base + first, kUnit, total, site)) r.load(p + base + first);
        else r.zero();
        r.get(f);
    } else {
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
            const int k = first + i * width;
            f[i] = k < K && SS1_IN(base + k, total, site) ? to_f(p[base + k]) : 0.0f;
        }
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_unit(T* __restrict__ p, int64_t base, int64_t total, int first, int width, int K,
                                           const float (&f)[kUnit], int site) {
    if (VEC) {
        Raw8<T> r;
        r.set(f);
        if (first < K && SS1_SPAN_IN(base + first, kUnit, total, site)) r.store(p + base + first);
    } else {
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
            const int k = first + i * width;
            if (k < K && SS1_IN(base + k, total, site)) p[base + k] = from_f<T>(f[i]);
        }
    }
}

// Sum over the `width` threads of a row (one warp, or all warps of the CTA), the same in every
// thread. `buf` holds one float per warp.
__device__ __forceinline__ float row_sum(float v, int width, float* buf) {
    v = warp_sum(v);
    if (width == 32) return v;
    const int warps = width / 32;
    __syncthreads();   // the buffer's last use is over
    if (threadIdx.x % 32 == 0) buf[threadIdx.x / 32] = v;
    __syncthreads();
    return warp_sum(threadIdx.x % 32 < warps ? buf[threadIdx.x % 32] : 0.0f);
}

// ---- forward ---------------------------------------------------------------------------------

// One row per warp (`width` 32, several rows a CTA) or per CTA (`width` = blockDim.x), held in NU
// units a thread.
template <typename T, typename W, bool VEC, int NU>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const T* __restrict__ X, const W* __restrict__ w,
                                                        const W* __restrict__ b, T* __restrict__ Y,
                                                        float* __restrict__ mean_out, float* __restrict__ rstd_out,
                                                        int64_t M, int K, float eps, int width) {
    __shared__ float buf[32];
    const int t = width == 32 ? threadIdx.x % 32 : threadIdx.x;
    const int64_t row = width == 32 ? (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32 : blockIdx.x;
    if (row >= M) return;   // whole warps, and only where a row is a warp's
    const int64_t base = row * K, total = M * K;
    float x[NU][kUnit];
    float s = 0.0f;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
        load_unit<T, VEC>(X, base, total, unit_first<VEC>(u, width, t), width, K, x[u], kSiteNormX);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) s += x[u][i];
    }
    const float mean = row_sum(s, width, buf) / (float)K;
    float q = 0.0f;
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
            const int first = unit_first<VEC>(u, width, t);
            const bool in = VEC ? first < K : first + i * width < K;
            const float d = in ? x[u][i] - mean : 0.0f;
            x[u][i] = d;
            q = fmaf(d, d, q);
        }
    const float rstd = 1.0f / sqrtf(row_sum(q, width, buf) / (float)K + eps);
#pragma unroll
    for (int u = 0; u < NU; ++u) {
        const int first = unit_first<VEC>(u, width, t);
        float wv[kUnit], bv[kUnit];
#pragma unroll
        for (int i = 0; i < kUnit; ++i) { wv[i] = 1.0f; bv[i] = 0.0f; }
        if (w) load_unit<W, VEC>(w, 0, K, first, width, K, wv, kSiteNormW);
        if (b) load_unit<W, VEC>(b, 0, K, first, width, K, bv, kSiteNormW);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) x[u][i] = fmaf(x[u][i] * rstd, wv[i], bv[i]);
        store_unit<T, VEC>(Y, base, total, first, width, K, x[u], kSiteNormY);
    }
    if (t == 0) {
        if (mean_out) mean_out[row] = mean;
        if (rstd_out) rstd_out[row] = rstd;
    }
}

// Rows that are too wide for the registers of one CTA: three passes over the row, the last two of
// which find it in L2.
template <typename T, typename W>
__global__ void __launch_bounds__(1024) norm_fwd_wide_kernel(const T* __restrict__ X, const W* __restrict__ w,
                                                             const W* __restrict__ b, T* __restrict__ Y,
                                                             float* __restrict__ mean_out, float* __restrict__ rstd_out,
                                                             int64_t M, int64_t K, float eps) {
    __shared__ float buf[32];
    const int64_t row = blockIdx.x;
    const T* x = X + row * K;
    float s = 0.0f;
    for (int64_t k = threadIdx.x; k < K; k += blockDim.x) s += SS1_IN(row * K + k, M * K, kSiteNormX) ? to_f(x[k]) : 0.0f;
    const float mean = row_sum(s, blockDim.x, buf) / (float)K;
    float q = 0.0f;
    for (int64_t k = threadIdx.x; k < K; k += blockDim.x) {
        const float d = to_f(x[k]) - mean;
        q = fmaf(d, d, q);
    }
    const float rstd = 1.0f / sqrtf(row_sum(q, blockDim.x, buf) / (float)K + eps);
    for (int64_t k = threadIdx.x; k < K; k += blockDim.x) {
        const float v = fmaf((to_f(x[k]) - mean) * rstd, w ? to_f(w[k]) : 1.0f, b ? to_f(b[k]) : 0.0f);
        if (SS1_IN(row * K + k, M * K, kSiteNormY)) Y[row * K + k] = from_f<T>(v);
    }
    if (threadIdx.x == 0) {
        if (mean_out) mean_out[row] = mean;
        if (rstd_out) rstd_out[row] = rstd;
    }
}

template <typename T, typename W, bool VEC, int NU>
cudaError_t fwd_launch(const void* X, const void* w, const void* b, void* Y, float* mean, float* rstd, int64_t M, int K,
                       float eps, int width, int threads, cudaStream_t st) {
    const int64_t rows = width == 32 ? threads / 32 : 1;
    const int64_t grid = (M + rows - 1) / rows;
    norm_fwd_kernel<T, W, VEC, NU><<<(unsigned)grid, threads, 0, st>>>((const T*)X, (const W*)w, (const W*)b, (T*)Y, mean,
                                                                      rstd, M, K, eps, width);
    return cudaGetLastError();
}

// Widest row of the register kernels: 1024 threads of four units.
constexpr int64_t kFwdWidest = 1024 * 4 * kUnit;

template <typename T, typename W, bool VEC>
cudaError_t fwd_shape(const void* X, const void* w, const void* b, void* Y, float* mean, float* rstd, int64_t M, int64_t K,
                      float eps, cudaStream_t st) {
    if (K > kFwdWidest) {
        norm_fwd_wide_kernel<T, W><<<(unsigned)M, 1024, 0, st>>>((const T*)X, (const W*)w, (const W*)b, (T*)Y, mean, rstd, M,
                                                                K, eps);
        return cudaGetLastError();
    }
    const int units = (int)((K + kUnit - 1) / kUnit);
    // one warp a row while the row fits its registers; 8 rows a CTA
#define SS1_NORM_WARP(nu) \
    if (units <= 32 * nu) return fwd_launch<T, W, VEC, nu>(X, w, b, Y, mean, rstd, M, (int)K, eps, 32, 256, st)
    SS1_NORM_WARP(1);
    SS1_NORM_WARP(2);
    SS1_NORM_WARP(3);
    SS1_NORM_WARP(4);
    SS1_NORM_WARP(5);
#undef SS1_NORM_WARP
    const int per = units <= 1024 ? 1 : (units <= 2048 ? 2 : 4);
    const int threads = ((units + per - 1) / per + 31) / 32 * 32;
    if (per == 1) return fwd_launch<T, W, VEC, 1>(X, w, b, Y, mean, rstd, M, (int)K, eps, threads, threads, st);
    if (per == 2) return fwd_launch<T, W, VEC, 2>(X, w, b, Y, mean, rstd, M, (int)K, eps, threads, threads, st);
    return fwd_launch<T, W, VEC, 4>(X, w, b, Y, mean, rstd, M, (int)K, eps, threads, threads, st);
}

// ---- backward --------------------------------------------------------------------------------

constexpr int64_t kBwdWidest = 1024 * kUnit;   // widest row that one CTA holds at a unit a thread
constexpr int kBwdThreads = 512;               // threads a CTA aims at: several row groups where rows are narrow
constexpr int kBwdCtas = 296;                  // CTAs at most (two for each of 148 SMs); each writes one partial sum

int bwd_group_threads(int64_t K) { return (int)(((K + kUnit - 1) / kUnit + 31) / 32 * 32); }
int bwd_groups(int64_t K) {
    const int n = kBwdThreads / bwd_group_threads(K);
    return n < 1 ? 1 : (n > 8 ? 8 : n);
}
// Rows of the partial sums [parts, 2, K].
int64_t bwd_parts(int64_t M, int64_t K) {
    if (K > kBwdWidest) return M < 64 ? M : 64;
    const int64_t need = (M + bwd_groups(K) - 1) / bwd_groups(K);
    return need < kBwdCtas ? need : kBwdCtas;
}

// Both sums over one row: within the group's warps, through `buf` (two floats a warp, two sets in
// turn, so that one barrier a row is enough).
__device__ __forceinline__ float2 group_sums(float a, float b, int warps, int warp, float2* buf, int bar, int width) {
    a = warp_sum(a);
    b = warp_sum(b);
    if (warps == 1) return make_float2(a, b);
    if (threadIdx.x % 32 == 0) buf[warp] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(width) : "memory");
    const float2 v = (int)(threadIdx.x % 32) < warps ? buf[threadIdx.x % 32] : make_float2(0.f, 0.f);
    return make_float2(warp_sum(v.x), warp_sum(v.y));
}

// A CTA is `groups` groups of `width` threads; group g of CTA c takes rows c * groups + g and so on
// in steps of the grid. A thread keeps one unit of columns all the way: its sums of dw and db stay in
// registers over all rows, the groups' are added in shared memory in group order, and each CTA
// writes one partial row. The next row's loads are issued before the present row's sums.
template <typename T, typename W, bool VEC>
__global__ void __launch_bounds__(1024) norm_bwd_kernel(const T* __restrict__ dY, const T* __restrict__ X,
                                                        const float* __restrict__ mean, const float* __restrict__ rstd,
                                                        const W* __restrict__ w, T* __restrict__ dX,
                                                        float* __restrict__ part, int64_t M, int K, int width, int groups) {
    extern __shared__ float col[];                    // [2][K] where groups > 1
    __shared__ float2 buf[2][8][32];
    const int g = threadIdx.x / width, t = threadIdx.x % width;
    const int first = unit_first<VEC>(0, width, t);
    const int64_t total = M * K;
    float wv[kUnit], sw[kUnit], sb[kUnit], x[kUnit], dy[kUnit], nx[kUnit], ndy[kUnit];
#pragma unroll
    for (int i = 0; i < kUnit; ++i) { wv[i] = 1.0f; sw[i] = 0.0f; sb[i] = 0.0f; }
    if (w) load_unit<W, VEC>(w, 0, K, first, width, K, wv, kSiteNormW);
    const int64_t step = (int64_t)gridDim.x * groups;
    int64_t row = (int64_t)blockIdx.x * groups + g;
    if (row < M) {
        load_unit<T, VEC>(X, row * K, total, first, width, K, nx, kSiteNormX);
        load_unit<T, VEC>(dY, row * K, total, first, width, K, ndy, kSiteNormX);
    }
    for (int turn = 0; row < M; row += step, turn ^= 1) {
        const float mu = mean[row], rs = rstd[row];
#pragma unroll
        for (int i = 0; i < kUnit; ++i) { x[i] = nx[i]; dy[i] = ndy[i]; }
        if (row + step < M) {
            load_unit<T, VEC>(X, (row + step) * K, total, first, width, K, nx, kSiteNormX);
            load_unit<T, VEC>(dY, (row + step) * K, total, first, width, K, ndy, kSiteNormX);
        }
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
            const bool in = VEC ? first < K : first + i * width < K;
            const float xh = in ? (x[i] - mu) * rs : 0.0f;   // dy is 0 behind the row's end
            sw[i] = fmaf(dy[i], xh, sw[i]);
            sb[i] += dy[i];
            x[i] = xh;
            dy[i] *= wv[i];
            a += dy[i];
            b = fmaf(dy[i], xh, b);
        }
        if (!dX) continue;
        const float2 s = group_sums(a, b, width / 32, t / 32, buf[turn][g], 1 + g, width);
        const float ma = s.x / (float)K, mb = s.y / (float)K;
#pragma unroll
        for (int i = 0; i < kUnit; ++i) x[i] = rs * (dy[i] - ma - x[i] * mb);
        store_unit<T, VEC>(dX, row * K, total, first, width, K, x, kSiteNormY);
    }
    if (!part) return;
    float* mine = part + (int64_t)blockIdx.x * 2 * K;
    const int64_t parts = (int64_t)gridDim.x * 2 * K;
    if (groups > 1) {
        for (int k = threadIdx.x; k < 2 * K; k += blockDim.x) col[k] = 0.0f;
        for (int turn = 0; turn < groups; ++turn) {
            __syncthreads();
            if (g != turn) continue;
#pragma unroll
            for (int i = 0; i < kUnit; ++i) {
                const int k = VEC ? first + i : first + i * width;
                if (k < K) { col[k] += sw[i]; col[K + k] += sb[i]; }
            }
        }
        __syncthreads();
        for (int k = threadIdx.x; k < 2 * K; k += blockDim.x)
            if (SS1_IN(mine + k - part, parts, kSiteNormPart)) mine[k] = col[k];
        return;
    }
#pragma unroll
    for (int i = 0; i < kUnit; ++i) {
        const int k = VEC ? first + i : first + i * width;
        if (k < K && SS1_SPAN_IN(mine + k - part, K + 1, parts, kSiteNormPart)) { mine[k] = sw[i]; mine[K + k] = sb[i]; }
    }
}

// Rows wider than kBwdWidest: dX a row per CTA in two passes, and the column sums apart.
template <typename T, typename W>
__global__ void __launch_bounds__(1024) norm_bwd_wide_kernel(const T* __restrict__ dY, const T* __restrict__ X,
                                                             const float* __restrict__ mean, const float* __restrict__ rstd,
                                                             const W* __restrict__ w, T* __restrict__ dX, int64_t M, int64_t K) {
    __shared__ float buf[32];
    const int64_t row = blockIdx.x;
    const float mu = mean[row], rs = rstd[row];
    float a = 0.0f, b = 0.0f;
    for (int64_t k = threadIdx.x; k < K; k += blockDim.x) {
        const bool in = SS1_IN(row * K + k, M * K, kSiteNormX);
        const float gk = in ? to_f(dY[row * K + k]) * (w ? to_f(w[k]) : 1.0f) : 0.0f;
        a += gk;
        b = fmaf(gk, in ? (to_f(X[row * K + k]) - mu) * rs : 0.0f, b);
    }
    const float ma = row_sum(a, blockDim.x, buf) / (float)K;
    const float mb = row_sum(b, blockDim.x, buf) / (float)K;
    for (int64_t k = threadIdx.x; k < K; k += blockDim.x) {
        if (!SS1_IN(row * K + k, M * K, kSiteNormY)) continue;
        const float gk = to_f(dY[row * K + k]) * (w ? to_f(w[k]) : 1.0f);
        dX[row * K + k] = from_f<T>(rs * (gk - ma - (to_f(X[row * K + k]) - mu) * rs * mb));
    }
}

template <typename T>
__global__ void __launch_bounds__(256) norm_bwd_columns_kernel(const T* __restrict__ dY, const T* __restrict__ X,
                                                               const float* __restrict__ mean, const float* __restrict__ rstd,
                                                               float* __restrict__ part, int64_t M, int64_t K) {
    const int64_t k = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (k >= K) return;
    float sw = 0.0f, sb = 0.0f;
    for (int64_t row = blockIdx.y; row < M; row += gridDim.y) {
        if (!SS1_IN(row * K + k, M * K, kSiteNormX)) continue;
        const float dy = to_f(dY[row * K + k]);
        sw = fmaf(dy, (to_f(X[row * K + k]) - mean[row]) * rstd[row], sw);
        sb += dy;
    }
    if (!SS1_SPAN_IN((int64_t)blockIdx.y * 2 * K + k, K + 1, (int64_t)gridDim.y * 2 * K, kSiteNormPart)) return;
    part[(int64_t)blockIdx.y * 2 * K + k] = sw;
    part[(int64_t)blockIdx.y * 2 * K + K + k] = sb;
}

// dw and db: the partial rows added in a fixed order, 32 columns a CTA, 32 threads a column.
template <typename W>
__global__ void __launch_bounds__(1024) norm_bwd_sum_kernel(const float* __restrict__ part, W* __restrict__ dw,
                                                            W* __restrict__ db, int64_t parts, int64_t K) {
    __shared__ float acc[32][33];
    const int64_t j = (int64_t)blockIdx.x * 32 + threadIdx.x;   // column of [2 K]: dw, then db
    float s = 0.0f;
    if (j < 2 * K)
        for (int64_t p = threadIdx.y; p < parts; p += 32)
            if (SS1_IN(p * 2 * K + j, parts * 2 * K, kSiteNormPart)) s += part[p * 2 * K + j];
    acc[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    s = warp_sum(acc[threadIdx.x][threadIdx.y]);   // warp y adds column y of the CTA
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x != 0 || c >= 2 * K) return;
    if (c < K) { if (dw) dw[c] = from_f<W>(s); }
    else if (db) db[c - K] = from_f<W>(s);
}

template <typename T, typename W, bool VEC>
cudaError_t bwd_shape(const void* dY, const void* X, const float* mean, const float* rstd, const void* w, void* dX, void* dw,
                      void* db, int64_t M, int64_t K, float* ws, cudaStream_t st) {
    float* part = dw || db ? ws : nullptr;
    const int64_t parts = bwd_parts(M, K);
    if (M > 0 && K > kBwdWidest) {
        if (dX) norm_bwd_wide_kernel<T, W><<<(unsigned)M, 1024, 0, st>>>((const T*)dY, (const T*)X, mean, rstd, (const W*)w,
                                                                       (T*)dX, M, K);
        if (part) norm_bwd_columns_kernel<T><<<dim3((unsigned)((K + 255) / 256), (unsigned)parts), 256, 0, st>>>(
            (const T*)dY, (const T*)X, mean, rstd, part, M, K);
    } else if (M > 0) {
        const int width = bwd_group_threads(K), groups = bwd_groups(K);
        const size_t smem = groups > 1 ? 2 * (size_t)K * sizeof(float) : 0;   // K <= 2048 there: 16 KB
        norm_bwd_kernel<T, W, VEC><<<(unsigned)parts, width * groups, smem, st>>>(
            (const T*)dY, (const T*)X, mean, rstd, (const W*)w, (T*)dX, part, M, (int)K, width, groups);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !(dw || db)) return e;
    norm_bwd_sum_kernel<W><<<(unsigned)((2 * K + 31) / 32), dim3(32, 32), 0, st>>>(part, (W*)dw, (W*)db, parts, K);
    return cudaGetLastError();
}

bool sizes_ok(int64_t M, int64_t K, int dtype, int w_dtype) {
    if (M < 0 || K < 1 || M > 0x7FFFFFFF || K > (1 << 30)) return false;
    // weights have the rows' type, or are float32 beside bf16 rows
    return dtype_ok(dtype) && dtype_ok(w_dtype) && (w_dtype == dtype || w_dtype == SS1_DTYPE_FP32);
}

}  // namespace
}  // namespace ss1

using namespace ss1;
using namespace ss1::op;

extern "C" SS1_API int ss1_layernorm_forward(const void* X, const void* weight, const void* bias, void* Y, float* mean,
                                             float* rstd, int64_t M, int64_t K, float eps, int dtype, int w_dtype,
                                             void* stream) {
    if (!sizes_ok(M, K, dtype, w_dtype) || !(eps >= 0.0f)) return SS1_ERR_INVALID_ARG;
    if (M == 0) return SS1_OK;
    if (!X || !Y) return SS1_ERR_INVALID_ARG;
    const size_t e = dtype_size(dtype), we = dtype_size(w_dtype);
    if (!aligned(X, e) || !aligned(Y, e) || !aligned(weight, we) || !aligned(bias, we) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return SS1_ERR_MISALIGNED;
    // 8-element loads: every row, and the weights, on a 16-byte boundary
    const bool vec = K % 8 == 0 && aligned(X, 16) && aligned(Y, 16) && aligned(weight, 16) && aligned(bias, 16);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    using bf16 = __nv_bfloat16;
    cudaError_t err;
    if (dtype == SS1_DTYPE_FP32)
        err = vec ? fwd_shape<float, float, true>(X, weight, bias, Y, mean, rstd, M, K, eps, st)
                  : fwd_shape<float, float, false>(X, weight, bias, Y, mean, rstd, M, K, eps, st);
    else if (w_dtype == SS1_DTYPE_FP32)
        err = vec ? fwd_shape<bf16, float, true>(X, weight, bias, Y, mean, rstd, M, K, eps, st)
                  : fwd_shape<bf16, float, false>(X, weight, bias, Y, mean, rstd, M, K, eps, st);
    else
        err = vec ? fwd_shape<bf16, bf16, true>(X, weight, bias, Y, mean, rstd, M, K, eps, st)
                  : fwd_shape<bf16, bf16, false>(X, weight, bias, Y, mean, rstd, M, K, eps, st);
    if (err != cudaSuccess) { cudaGetLastError(); return SS1_ERR_CUDA; }
    return SS1_OK;
}

extern "C" SS1_API int ss1_layernorm_backward_workspace(int64_t M, int64_t K, size_t* bytes) {
    if (!bytes || !sizes_ok(M, K, SS1_DTYPE_FP32, SS1_DTYPE_FP32)) return SS1_ERR_INVALID_ARG;
    *bytes = (size_t)bwd_parts(M, K) * 2 * (size_t)K * sizeof(float);
    return SS1_OK;
}

extern "C" SS1_API int ss1_layernorm_backward(const void* dY, const void* X, const float* mean, const float* rstd,
                                              const void* weight, void* dX, void* dweight, void* dbias, int64_t M,
                                              int64_t K, int dtype, int w_dtype, void* workspace, size_t workspace_bytes,
                                              void* stream) {
    if (!sizes_ok(M, K, dtype, w_dtype)) return SS1_ERR_INVALID_ARG;
    const size_t e = dtype_size(dtype), we = dtype_size(w_dtype);
    if (!aligned(dY, e) || !aligned(X, e) || !aligned(dX, e) || !aligned(weight, we) || !aligned(dweight, we) ||
        !aligned(dbias, we) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(workspace, 16))
        return SS1_ERR_MISALIGNED;
    if (!dX && !dweight && !dbias) return SS1_OK;
    if (M > 0) {
        if (!dY || !X || !mean || !rstd) return SS1_ERR_INVALID_ARG;
        const size_t need = (size_t)bwd_parts(M, K) * 2 * (size_t)K * sizeof(float);
        if ((dweight || dbias) && (!workspace || workspace_bytes < need)) return SS1_ERR_INVALID_ARG;
    } else if (!dweight && !dbias) {
        return SS1_OK;
    }
    const bool vec = K % 8 == 0 && aligned(dY, 16) && aligned(X, 16) && aligned(dX, 16) && aligned(weight, 16);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    float* ws = static_cast<float*>(workspace);
    using bf16 = __nv_bfloat16;
    cudaError_t err;
    if (dtype == SS1_DTYPE_FP32)
        err = vec ? bwd_shape<float, float, true>(dY, X, mean, rstd, weight, dX, dweight, dbias, M, K, ws, st)
                  : bwd_shape<float, float, false>(dY, X, mean, rstd, weight, dX, dweight, dbias, M, K, ws, st);
    else if (w_dtype == SS1_DTYPE_FP32)
        err = vec ? bwd_shape<bf16, float, true>(dY, X, mean, rstd, weight, dX, dweight, dbias, M, K, ws, st)
                  : bwd_shape<bf16, float, false>(dY, X, mean, rstd, weight, dX, dweight, dbias, M, K, ws, st);
    else
        err = vec ? bwd_shape<bf16, bf16, true>(dY, X, mean, rstd, weight, dX, dweight, dbias, M, K, ws, st)
                  : bwd_shape<bf16, bf16, false>(dY, X, mean, rstd, weight, dX, dweight, dbias, M, K, ws, st);
    if (err != cudaSuccess) { cudaGetLastError(); return SS1_ERR_CUDA; }
    return SS1_OK;
}
