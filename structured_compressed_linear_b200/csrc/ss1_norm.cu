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
#include "ptx_sm100.cuh"

namespace ss1 {
namespace {

using namespace op;

constexpr int kUnit = 8;   // elements a thread takes at a time: 16 bytes of bf16, 32 of float

// Eight elements of a row, a thread's unit. kRow8: consecutive (bf16 rows on 16-byte boundaries); kRow44: twice four
// consecutive ones, half the unit's columns apart, so that a warp's 16-byte pieces of float rows lie side by
// side; kRow1: strided by the width (rows that do not start on 16-byte boundaries), so that its elements do. They
// are worked on as four pairs.
enum Form { kRow1, kRow8, kRow44 };
template <typename T, bool VEC>
constexpr Form form_of() { return !VEC ? kRow1 : (sizeof(T) == 4 ? kRow44 : kRow8); }

template <Form F>
__device__ __forceinline__ int unit_first(int unit, int width, int t) {
    return F == kRow8 ? (unit * width + t) * kUnit : unit * width * kUnit + (F == kRow44 ? t * 4 : t);
}
template <Form F>
__device__ __forceinline__ int unit_at(int first, int width, int i) {      // column of the unit's element i
    return F == kRow8 ? first + i : (F == kRow44 ? first + (i < 4 ? i : width * 4 + i - 4) : first + i * width);
}

template <Form F>
__device__ __forceinline__ bool unit_in(int first, int width, int i, int K) {      // does element i lie inside the row?
    return (F == kRow8 ? first : unit_at<F>(first, width, F == kRow44 ? i & 4 : i)) < K;
}

// `p` is the row (or the weights), `left` what `total` leaves behind it; elements past K are `other`.
template <typename T, Form F>
__device__ __forceinline__ void load_unit(const T* __restrict__ p, [[maybe_unused]] int64_t left, int first, int width, int K, F2 (&f)[4],
                                          float other, int site) {
    if constexpr (F == kRow8) {
        if (first < K && SS1_SPAN_IN(first, kUnit, left, site)) {
            Raw8<T> r;
            r.load(p + first);
            r.get(f);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = F2::both(other);
        }
    } else if constexpr (F == kRow44) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = unit_at<F>(first, width, 4 * h);
            float4 v = make_float4(other, other, other, other);
            if (k < K && SS1_SPAN_IN(k, 4, left, site)) v = *reinterpret_cast<const float4*>(p + k);
            f[2 * h] = F2::of(v.x, v.y);
            f[2 * h + 1] = F2::of(v.z, v.w);
        }
    } else {
        float v[kUnit];
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
            const int k = unit_at<F>(first, width, i);
            v[i] = k < K && SS1_IN(k, left, site) ? to_f(p[k]) : other;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = F2::of(v[2 * i], v[2 * i + 1]);
    }
}

template <typename T, Form F>
__device__ __forceinline__ void store_unit(T* __restrict__ p, [[maybe_unused]] int64_t left, int first, int width, int K,
                                           const F2 (&f)[4], int site) {
    if constexpr (F == kRow8) {
        Raw8<T> r;
        r.set(f);
        if (first < K && SS1_SPAN_IN(first, kUnit, left, site)) r.store(p + first);
    } else if constexpr (F == kRow44) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = unit_at<F>(first, width, 4 * h);
            if (k < K && SS1_SPAN_IN(k, 4, left, site))
                *reinterpret_cast<float4*>(p + k) = make_float4(f[2 * h].lo(), f[2 * h].hi(), f[2 * h + 1].lo(), f[2 * h + 1].hi());
        }
    } else {
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
            const int k = unit_at<F>(first, width, i);
            if (k < K && SS1_IN(k, left, site)) p[k] = from_f<T>(i % 2 ? f[i / 2].hi() : f[i / 2].lo());
        }
    }
}

// Rows on their way: every thread copies the units that it will work on into places of its own
// in shared memory, some rows ahead, and reads them back itself. So the bytes in flight cost no
// registers, and a thread waits for its own copies only, without a barrier. Pieces are 16 bytes a
// thread (vector rows) or 4 (scalar rows of float), threads side by side. Scalar rows of bf16 have none:
// no copy is as small as an element, and those rows are loaded when their turn comes.
template <typename T>
constexpr int unit_bytes() { return kUnit * (int)sizeof(T); }
template <typename T, bool VEC>
constexpr bool in_ring() { return VEC || sizeof(T) == 4; }

// `first` as unit_first gives it, from the start of the row at `p`; nothing is read where the row is not `ok`, or behind
// its end (zeros instead). FULL: every unit lies inside the row.
template <typename T, Form F, bool FULL>
__device__ __forceinline__ void unit_ahead(uint32_t ring, int threads, const T* p, [[maybe_unused]] int64_t left, int first, int width, int K,
                                           bool ok, const T* any, int site) {
    if constexpr (F != kRow1) {
#pragma unroll
        for (int i = 0; i < unit_bytes<T>() / 16; ++i) {
            const int k = unit_at<F>(first, width, i * (16 / (int)sizeof(T)));
            const bool in = ok && (FULL || k < K) && SS1_SPAN_IN(k, 16 / (int)sizeof(T), left, site);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ring + (i * threads + threadIdx.x) * 16),
                         "l"(in ? p + k : any), "r"(in ? 16 : 0)
                         : "memory");
        }
    } else {
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
            const int k = unit_at<F>(first, width, i);
            const bool in = ok && k < K && SS1_IN(k, left, site);
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(ring + (i * threads + threadIdx.x) * 4),
                         "l"(in ? p + k : any), "r"(in ? 4 : 0)
                         : "memory");
        }
    }
}

template <typename T, Form F>
__device__ __forceinline__ void unit_back(const uint8_t* ring, int threads, F2 (&f)[4]) {
    if constexpr (F == kRow8) {
        Raw8<T> r;
        r.a = *reinterpret_cast<const uint4*>(ring + threadIdx.x * 16);
        r.get(f);
    } else if constexpr (F == kRow44) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 v = *reinterpret_cast<const float4*>(ring + (h * threads + threadIdx.x) * 16);
            f[2 * h] = F2::of(v.x, v.y);
            f[2 * h + 1] = F2::of(v.z, v.w);
        }
    } else {
        const float* v = reinterpret_cast<const float*>(ring) + threadIdx.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = F2::of(v[2 * i * threads], v[(2 * i + 1) * threads]);
    }
}

// Sum over the `width` threads of a row (one warp, or all warps of the CTA), the same in every
// thread. `buf` holds one float per warp, zeros behind the last; uses of one buffer lie a barrier apart.
__device__ __forceinline__ float row_sum(float v, int width, float* buf) {
    v = warp_sum(v);
    if (width == 32) return v;
    if (threadIdx.x % 32 == 0) buf[threadIdx.x / 32] = v;
    __syncthreads();
    if (width > 256) return warp_sum(buf[threadIdx.x % 32]);
    const float4 a = *reinterpret_cast<const float4*>(buf);
    v = (a.x + a.y) + (a.z + a.w);
    if (width > 128) {
        const float4 b = *reinterpret_cast<const float4*>(buf + 4);
        v += (b.x + b.y) + (b.z + b.w);
    }
    return v;
}

// ---- forward ---------------------------------------------------------------------------------

// CTAs meant to be on an SM: about 768 threads of up to 85 registers; rows of more than 256 threads 1024 of 64
constexpr int fwd_ctas(int threads) { return threads <= 256 ? 768 / threads : 1024 / threads; }
// Rows ahead: what keeps about 64 KB in flight on an SM beside the rows being read, one to three (128 KB: 5 % slower).
template <typename T>
constexpr int fwd_ahead(int units, int threads) {
    const int rows = 65536 / (fwd_ctas(threads) * units * unit_bytes<T>() * threads);
    return rows > 3 ? 3 : (rows < 1 ? 1 : rows);
}

// One row per warp (WARP: several rows a CTA) or per CTA, held in NU units a thread; the grid walks the
// rows. THREADS is what the CTA has at most. Enough rows are on an SM at once for one row's sums (two
// trees with a barrier each, where a row is a CTA's) to pass behind the others' work. What is left to
// bound it is issue slots: so sums and products go in pairs, FULL rows (all units inside) carry no
// predicates, and where warps share a CTA the weights lie converted in shared memory. 16384 x 1280: bf16 15.5 us,
// 84 MB at 5.4 TB/s; float 29.7 us, 5.7 TB/s.
template <typename T, typename W, bool VEC, bool WARP, bool FULL, int NU, int THREADS>
__global__ void __launch_bounds__(THREADS, fwd_ctas(THREADS)) norm_fwd_kernel(const T* __restrict__ X, const W* __restrict__ w,
                                                                             const W* __restrict__ b, T* __restrict__ Y,
                                                                             float* __restrict__ mean_out, float* __restrict__ rstd_out,
                                                                             int64_t M, int K, float eps) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ __align__(16) float buf[2][32];
    wait_for_previous();

    constexpr Form F = form_of<T, VEC>();
    constexpr bool kRing = in_ring<T, VEC>(), kShared = WARP && VEC;
    constexpr int kDepth = fwd_ahead<T>(NU, THREADS), kPlace = unit_bytes<T>() * THREADS, kRow = NU * kPlace;
    __shared__ __align__(16) float weights[kShared ? 2 : 1][kShared ? NU * 2 : 1][kShared ? 128 : 4];   // [w, b][half unit][lane * 4]
    const int width = WARP ? 32 : blockDim.x, t = WARP ? threadIdx.x % 32 : threadIdx.x;
    const int64_t step = WARP ? (int64_t)gridDim.x * (THREADS / 32) : gridDim.x, stride = step * K;
    int64_t row = WARP ? (int64_t)blockIdx.x * (THREADS / 32) + threadIdx.x / 32 : blockIdx.x;
    const uint32_t place = ptx::smem_u32(ring);
    const T* in = X + row * K;              // the row that is worked on, and the next one to be copied
    const T* from = in;
    T* out = Y + row * K;
    int64_t from_row = row;
    auto ahead = [&](int slot) {
        if (!kRing) return;
        if (from_row < M) {
#pragma unroll
            for (int u = 0; u < NU; ++u)
                unit_ahead<T, F, FULL>(place + slot * kRow + u * kPlace, THREADS, from, (M - from_row) * K, unit_first<F>(u, width, t),
                                         width, K, true, X, kSiteNormX);
        }
        from += stride;
        from_row += step;
        ptx::cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kDepth; ++i) ahead(i);
    if (kShared) {
        for (int i = threadIdx.x; i < NU * 256; i += THREADS) {      // element i of the row: unit, lane, half, place in the half
            const int u = i / 256, l = F == kRow44 ? i / 4 % 32 : i / 8 % 32, h = F == kRow44 ? i / 128 % 2 : i / 4 % 2;
            weights[0][u * 2 + h][l * 4 + i % 4] = w && i < K ? to_f(w[i]) : 1.0f;
            weights[kShared][u * 2 + h][l * 4 + i % 4] = b && i < K ? to_f(b[i]) : 0.0f;
        }
        __syncthreads();
    }
    if (!WARP) {
        if (threadIdx.x < 64) buf[threadIdx.x / 32][threadIdx.x % 32] = 0.0f;
        __syncthreads();
    }
    const float inv = 1.0f / (float)K;
    for (int slot = 0; row < M; slot = slot + 1 == kDepth ? 0 : slot + 1) {     // together: all that meet at a barrier
        [[maybe_unused]] const int64_t left = (M - row) * K;
        F2 x[NU][4];
        F2 s = F2::both(0.0f);
        if (kRing) ptx::cp_async_wait<kDepth - 1>();
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            if (kRing) {
                unit_back<T, F>(ring + slot * kRow + u * kPlace, THREADS, x[u]);
            } else {
                load_unit<T, F>(in, left, unit_first<F>(u, width, t), width, K, x[u], 0.0f, kSiteNormX);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) s = s + x[u][i];
        }
        ahead(slot);
        const float mean = row_sum(s.lo() + s.hi(), width, buf[0]) * inv;
        const F2 less = F2::both(-mean);
        F2 q = F2::both(0.0f);
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int first = unit_first<F>(u, width, t);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[u][i] = x[u][i] + less;
            if (!FULL) {          // what lies behind the row's end deviates by nothing
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[u][i] = F2::of(unit_in<F>(first, width, 2 * i, K) ? x[u][i].lo() : 0.0f,
                                     unit_in<F>(first, width, 2 * i + 1, K) ? x[u][i].hi() : 0.0f);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) q = fma2(x[u][i], x[u][i], q);
        }
        const float rstd = rsqrtf(row_sum(q.lo() + q.hi(), width, buf[1]) * inv + eps);
        const F2 by = F2::both(rstd);
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int first = unit_first<F>(u, width, t);
            F2 wv[4], bv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[u][i] = x[u][i] * by;
            if (kShared) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float4 wh = *reinterpret_cast<const float4*>(&weights[0][u * 2 + h][t * 4]);
                    const float4 bh = *reinterpret_cast<const float4*>(&weights[kShared][u * 2 + h][t * 4]);
                    x[u][2 * h] = fma2(x[u][2 * h], F2::of(wh.x, wh.y), F2::of(bh.x, bh.y));
                    x[u][2 * h + 1] = fma2(x[u][2 * h + 1], F2::of(wh.z, wh.w), F2::of(bh.z, bh.w));
                }
            } else if (w) {
                load_unit<W, F>(w, K, first, width, K, wv, 1.0f, kSiteNormW);
                if (b) {
                    load_unit<W, F>(b, K, first, width, K, bv, 0.0f, kSiteNormW);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[u][i] = fma2(x[u][i], wv[i], bv[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[u][i] = x[u][i] * wv[i];
                }
            } else if (b) {
                load_unit<W, F>(b, K, first, width, K, bv, 0.0f, kSiteNormW);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[u][i] = x[u][i] + bv[i];
            }
            store_unit<T, F>(out, left, first, width, FULL ? 1 << 30 : K, x[u], kSiteNormY);
        }
        if (t == 0) {
            if (mean_out) mean_out[row] = mean;
            if (rstd_out) rstd_out[row] = rstd;
        }
        in += stride;
        out += stride;
        row += step;
    }
}

// Rows that are too wide for the registers of one CTA: three passes over the row, the last two of
// which find it in L2.
template <typename T, typename W>
__global__ void __launch_bounds__(1024) norm_fwd_wide_kernel(const T* __restrict__ X, const W* __restrict__ w,
                                                             const W* __restrict__ b, T* __restrict__ Y,
                                                             float* __restrict__ mean_out, float* __restrict__ rstd_out,
                                                             int64_t M, int64_t K, float eps) {
    __shared__ __align__(16) float buf[2][32];   // 32 warps: every place is written
    const int64_t row = blockIdx.x;
    const T* x = X + row * K;
    float s = 0.0f;
    for (int64_t k = threadIdx.x; k < K; k += blockDim.x) s += SS1_IN(row * K + k, M * K, kSiteNormX) ? to_f(x[k]) : 0.0f;
    const float mean = row_sum(s, blockDim.x, buf[0]) / (float)K;
    float q = 0.0f;
    for (int64_t k = threadIdx.x; k < K; k += blockDim.x) {
        const float d = to_f(x[k]) - mean;
        q = fmaf(d, d, q);
    }
    const float rstd = 1.0f / sqrtf(row_sum(q, blockDim.x, buf[1]) / (float)K + eps);
    for (int64_t k = threadIdx.x; k < K; k += blockDim.x) {
        const float v = fmaf((to_f(x[k]) - mean) * rstd, w ? to_f(w[k]) : 1.0f, b ? to_f(b[k]) : 0.0f);
        if (SS1_IN(row * K + k, M * K, kSiteNormY)) Y[row * K + k] = from_f<T>(v);
    }
    if (threadIdx.x == 0) {
        if (mean_out) mean_out[row] = mean;
        if (rstd_out) rstd_out[row] = rstd;
    }
}

template <typename T, typename W, bool VEC, bool WARP, bool FULL, int NU, int THREADS>
cudaError_t fwd_launch(const void* X, const void* w, const void* b, void* Y, float* mean, float* rstd, int64_t M, int K,
                       float eps, int threads, cudaStream_t st) {
    auto* fn = &norm_fwd_kernel<T, W, VEC, WARP, FULL, NU, THREADS>;
    constexpr int smem = in_ring<T, VEC>() ? fwd_ahead<T>(NU, THREADS) * NU * unit_bytes<T>() * THREADS : 0;
    if (smem > 0) {
        const cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(fn), smem);
        if (e != cudaSuccess) return e;
    }
    const int64_t rows = WARP ? threads / 32 : 1, need = (M + rows - 1) / rows, most = 148 * fwd_ctas(THREADS);
    return launch_dependent(fn, dim3((unsigned)(need < most ? need : most)), dim3((unsigned)threads), smem, st, (const T*)X, (const W*)w,
                            (const W*)b, (T*)Y, mean, rstd, M, K, eps);
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
    // one warp a row while the row fits its registers
#define SS1_NORM_WARP(nu) \
    if (VEC && units == 32 * nu) return fwd_launch<T, W, VEC, true, VEC, nu, 256>(X, w, b, Y, mean, rstd, M, (int)K, eps, 256, st); \
    if (units <= 32 * nu) return fwd_launch<T, W, VEC, true, false, nu, 256>(X, w, b, Y, mean, rstd, M, (int)K, eps, 256, st)
    SS1_NORM_WARP(1);
    SS1_NORM_WARP(2);
    SS1_NORM_WARP(3);
    SS1_NORM_WARP(4);
    SS1_NORM_WARP(5);
#undef SS1_NORM_WARP
    const int threads = ((units + 3) / 4 + 31) / 32 * 32;
#define SS1_NORM_CTA(most) \
    if (VEC && units == 4 * threads && threads <= most) \
        return fwd_launch<T, W, VEC, false, VEC, 4, most>(X, w, b, Y, mean, rstd, M, (int)K, eps, threads, st); \
    if (threads <= most) return fwd_launch<T, W, VEC, false, false, 4, most>(X, w, b, Y, mean, rstd, M, (int)K, eps, threads, st)
    SS1_NORM_CTA(64);
    SS1_NORM_CTA(128);
    SS1_NORM_CTA(256);
    SS1_NORM_CTA(512);
#undef SS1_NORM_CTA
    return fwd_launch<T, W, VEC, false, false, 4, 1024>(X, w, b, Y, mean, rstd, M, (int)K, eps, threads, st);
}

// ---- backward --------------------------------------------------------------------------------

constexpr int kBwdThreads = 512;                   // threads of a CTA at most, one CTA an SM: 128 registers each, without spills
constexpr int kBwdCtas = 148;                      // CTAs at most; each writes one partial sum
constexpr int64_t kBwdWidest = 512 * 2 * kUnit;    // widest row that a CTA holds

// Rows up to 4096 wide: a unit a thread, two rows a turn; wider ones: two units, one row.
constexpr int64_t kBwdPairs = 512 * kUnit;
int bwd_group_threads(int64_t K) {
    const int64_t each = K <= kBwdPairs ? kUnit : 2 * kUnit;
    return (int)(((K + each - 1) / each + 31) / 32 * 32);
}
int bwd_groups(int64_t K) {
    const int n = kBwdThreads / bwd_group_threads(K);
    return n > 15 ? 15 : n;                        // a named barrier each
}
// Rows of the partial sums [parts, 2, K]. Where one CTA does, it writes the sums themselves, and the second launch is
// saved: up to kBwdAlone elements. 1 x 768: 4.3 us against 5.3; 16 x 4096 (65,536 elements) already 18 against 7.7.
constexpr int64_t kBwdAlone = 1 << 13;
int64_t bwd_parts(int64_t M, int64_t K) {
    if (K > kBwdWidest) return M < 64 ? M : 64;
    if (M * K <= kBwdAlone) return M < 1 ? M : 1;
    const int64_t need = (M + bwd_groups(K) - 1) / bwd_groups(K);
    return need < kBwdCtas ? need : kBwdCtas;
}

// A CTA is `groups` groups of `width` threads; group g of CTA c takes ROWS rows at a time, from row
// (c * groups + g) * ROWS in steps of the grid. A thread keeps its columns all the way: its sums of dw and
// db stay in registers over all rows, the groups' are added through shared memory in group order, and each CTA
// writes one partial row. A row's two sums take two trees and a barrier of its group; two rows a
// turn share them. One CTA an SM leaves a thread 128 registers, which the sums of its columns need; what
// bounds it is issue slots, then bytes. 16384 x 1280: bf16 29 us, 126 MB at 4.4 TB/s; float 42.4 us, 5.9 TB/s.
template <typename T>
constexpr int bwd_ahead() { return sizeof(T) == 2 ? 2 : 1; }    // turns ahead: 32 or 64 KB each (one more is 2 % slower)

template <typename T, typename W, bool VEC, int UNITS, int ROWS>
__global__ void __launch_bounds__(kBwdThreads) norm_bwd_kernel(const T* __restrict__ dY, const T* __restrict__ X,
                                                               const float* __restrict__ mean, const float* __restrict__ rstd,
                                                               const W* __restrict__ w, T* __restrict__ dX, float* __restrict__ part,
                                                               W* __restrict__ dw, W* __restrict__ db, int64_t M, int K, int width,
                                                               int groups) {
    static_assert(UNITS * ROWS == 2, "one turn's pieces");
    extern __shared__ __align__(16) uint8_t ring[];             // the turns ahead, later [groups][2][K] sums
    __shared__ __align__(16) float4 buf[2][15][16];             // a row's two sums of each warp, for two rows
    constexpr Form F = form_of<T, VEC>();
    constexpr bool kRing = in_ring<T, VEC>();
    constexpr int kDepth = bwd_ahead<T>(), kPlace = unit_bytes<T>() * kBwdThreads, kTurn = 4 * kPlace;
    wait_for_previous();

    const int g = threadIdx.x / width, t = threadIdx.x % width, warps = width / 32, warp = t / 32;
    for (int i = threadIdx.x; i < 2 * 15 * 16; i += blockDim.x) (&buf[0][0][0])[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
    const float inv = 1.0f / (float)K;
    const int64_t total = M * K, step = (int64_t)gridDim.x * groups * ROWS;
    F2 sw[UNITS][4], sb[UNITS][4], wv[UNITS][4];
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) { sw[u][i] = sb[u][i] = F2::both(0.0f); wv[u][i] = F2::both(1.0f); }
        if (w) load_unit<W, F>(w, K, unit_first<F>(u, width, t), width, K, wv[u], 0.0f, kSiteNormW);
    }
    int64_t row = ((int64_t)blockIdx.x * groups + g) * ROWS, from = row;
    const uint32_t place = ptx::smem_u32(ring);
    auto ahead = [&](int slot) {
        if (!kRing) return;
        if (from < M) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {                       // the turn's two units: two rows', or one row's
                const int64_t r = from + (ROWS == 2 ? e : 0), at = r * K;
                const int first = unit_first<F>(ROWS == 2 ? 0 : e, width, t);
                unit_ahead<T, F, false>(place + slot * kTurn + e * 2 * kPlace, kBwdThreads, X + at, total - at, first, width, K, r < M, X,
                                          kSiteNormX);
                unit_ahead<T, F, false>(place + slot * kTurn + (e * 2 + 1) * kPlace, kBwdThreads, dY + at, total - at, first, width, K,
                                          r < M, dY, kSiteNormX);
            }
        }
        from += step;
        ptx::cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kDepth; ++i) ahead(i);
    float mu[ROWS], rs[ROWS], next_mu[ROWS], next_rs[ROWS];      // statistics a turn ahead; 0 behind the last row
    auto look_up = [&](int64_t r0) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            next_mu[r] = r0 + r < M ? mean[r0 + r] : 0.0f;
            next_rs[r] = r0 + r < M ? rstd[r0 + r] : 0.0f;
        }
    };
    look_up(row);
    for (int turn = 0, slot = 0; row < M; row += step, turn ^= 1, slot = slot + 1 == kDepth ? 0 : slot + 1) {
        F2 x[2][4], dy[2][4];
        if (kRing) ptx::cp_async_wait<kDepth - 1>();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (kRing) {
                unit_back<T, F>(ring + slot * kTurn + e * 2 * kPlace, kBwdThreads, x[e]);
                unit_back<T, F>(ring + slot * kTurn + (e * 2 + 1) * kPlace, kBwdThreads, dy[e]);
            } else {
                const int64_t r = row + (ROWS == 2 ? e : 0);
                const int k = r < M ? K : 0;
                const int first = unit_first<F>(ROWS == 2 ? 0 : e, width, t);
                load_unit<T, F>(X + r * K, total - r * K, first, width, k, x[e], 0.0f, kSiteNormX);
                load_unit<T, F>(dY + r * K, total - r * K, first, width, k, dy[e], 0.0f, kSiteNormX);
            }
        }
        ahead(slot);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) { mu[r] = next_mu[r]; rs[r] = next_rs[r]; }
        look_up(row + step);
        F2 a[ROWS], b[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) a[r] = b[r] = F2::both(0.0f);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = ROWS == 2 ? e : 0, u = ROWS == 2 ? 0 : e;
            const F2 by = F2::both(rs[r]);
            const int first = unit_first<F>(u, width, t);
#pragma unroll
            for (int i = 0; i < 4; ++i) {     // behind the row's end dy and xh are 0, whatever the mean is
                const F2 xh = (x[e][i] + F2::of(unit_in<F>(first, width, 2 * i, K) ? -mu[r] : 0.0f,
                                                unit_in<F>(first, width, 2 * i + 1, K) ? -mu[r] : 0.0f)) *
                              by;
                sw[u][i] = fma2(dy[e][i], xh, sw[u][i]);
                sb[u][i] = sb[u][i] + dy[e][i];
                x[e][i] = xh;
                dy[e][i] = dy[e][i] * wv[u][i];
                a[r] = a[r] + dy[e][i];
                b[r] = fma2(dy[e][i], xh, b[r]);
            }
        }
        if (!dX) continue;
        float4 s = make_float4(a[0].lo() + a[0].hi(), b[0].lo() + b[0].hi(), a[ROWS - 1].lo() + a[ROWS - 1].hi(),
                               b[ROWS - 1].lo() + b[ROWS - 1].hi());
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s.x += __shfl_xor_sync(0xFFFFFFFFu, s.x, o);
            s.y += __shfl_xor_sync(0xFFFFFFFFu, s.y, o);
            if (ROWS == 2) {
                s.z += __shfl_xor_sync(0xFFFFFFFFu, s.z, o);
                s.w += __shfl_xor_sync(0xFFFFFFFFu, s.w, o);
            }
        }
        if (warps > 1) {      // two buffers in turn: one barrier a turn is enough
            if (threadIdx.x % 32 == 0) buf[turn][g][warp] = s;
            asm volatile("bar.sync %0, %1;" ::"r"(1 + g), "r"(width) : "memory");
            F2 p = F2::both(0.0f), q = p;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                if (k % 4 == 0 && k >= warps) break;
                const float4 v = buf[turn][g][k];
                p = p + F2::of(v.x, v.y);
                if (ROWS == 2) q = q + F2::of(v.z, v.w);
            }
            s = make_float4(p.lo(), p.hi(), q.lo(), q.hi());
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = ROWS == 2 ? e : 0;
            const F2 ma = F2::both(-(r ? s.z : s.x) * inv), mb = F2::both(-(r ? s.w : s.y) * inv), by = F2::both(rs[r]);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[e][i] = (fma2(x[e][i], mb, dy[e][i]) + ma) * by;
            if (row + r < M)
                store_unit<T, F>(dX + (row + r) * K, total - (row + r) * K, unit_first<F>(ROWS == 2 ? 0 : e, width, t), width, K, x[e],
                                   kSiteNormY);
        }
    }
    if (!part && !dw && !db) return;
    // every group's sums side by side over the ring's memory, then a thread adds its columns' in group order
    float* to = part + (int64_t)blockIdx.x * 2 * K;
    [[maybe_unused]] const int64_t parts = (int64_t)(gridDim.x - blockIdx.x) * 2 * K;
    float* col = reinterpret_cast<float*>(ring) + (int64_t)g * 2 * K;
    if (kRing) ptx::cp_async_wait<0>();
    __syncthreads();
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
            const int k = unit_at<F>(unit_first<F>(u, width, t), width, i);
            if (k < K) {
                col[k] = i % 2 ? sw[u][i / 2].hi() : sw[u][i / 2].lo();
                col[K + k] = i % 2 ? sb[u][i / 2].hi() : sb[u][i / 2].lo();
            }
        }
    __syncthreads();
    for (int k = threadIdx.x; k < 2 * K; k += blockDim.x) {
        float v = 0.0f;
        for (int o = 0; o < groups; ++o) v += reinterpret_cast<float*>(ring)[(int64_t)o * 2 * K + k];
        if (part) {
            if (SS1_IN(k, parts, kSiteNormPart)) to[k] = v;
        } else if (k < K) {                    // the only CTA
            if (dw) dw[k] = from_f<W>(v);
        } else if (db) {
            db[k - K] = from_f<W>(v);
        }
    }
}

// Rows wider than kBwdWidest: dX a row per CTA in two passes, and the column sums apart.
template <typename T, typename W>
__global__ void __launch_bounds__(1024) norm_bwd_wide_kernel(const T* __restrict__ dY, const T* __restrict__ X,
                                                             const float* __restrict__ mean, const float* __restrict__ rstd,
                                                             const W* __restrict__ w, T* __restrict__ dX, int64_t M, int64_t K) {
    __shared__ __align__(16) float buf[2][32];   // 32 warps: every place is written
    const int64_t row = blockIdx.x;
    const float mu = mean[row], rs = rstd[row];
    float a = 0.0f, b = 0.0f;
    for (int64_t k = threadIdx.x; k < K; k += blockDim.x) {
        const bool in = SS1_IN(row * K + k, M * K, kSiteNormX);
        const float gk = in ? to_f(dY[row * K + k]) * (w ? to_f(w[k]) : 1.0f) : 0.0f;
        a += gk;
        b = fmaf(gk, in ? (to_f(X[row * K + k]) - mu) * rs : 0.0f, b);
    }
    const float ma = row_sum(a, blockDim.x, buf[0]) / (float)K;
    const float mb = row_sum(b, blockDim.x, buf[1]) / (float)K;
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
    wait_for_previous();
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

template <typename T, typename W, bool VEC, int UNITS, int ROWS>
cudaError_t bwd_rows(const void* dY, const void* X, const float* mean, const float* rstd, const void* w, void* dX, float* part, void* dw,
                     void* db, int64_t M, int K, int ctas, cudaStream_t st) {
    auto* fn = &norm_bwd_kernel<T, W, VEC, UNITS, ROWS>;
    const int width = bwd_group_threads(K), groups = bwd_groups(K);
    // the turns ahead, and the groups' sums over them: a group has at most 16 columns a thread
    constexpr int most_sums = 2 * kBwdThreads * UNITS * kUnit * (int)sizeof(float);
    constexpr int turns = in_ring<T, VEC>() ? bwd_ahead<T>() * 4 * unit_bytes<T>() * kBwdThreads : 0, smem = turns > most_sums ? turns : most_sums;
    const cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(fn), smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(fn, dim3((unsigned)ctas), dim3((unsigned)(width * groups)), smem, st, (const T*)dY, (const T*)X, mean, rstd,
                            (const W*)w, (T*)dX, part, (W*)dw, (W*)db, M, K, width, groups);
}

template <typename T, typename W, bool VEC>
cudaError_t bwd_shape(const void* dY, const void* X, const float* mean, const float* rstd, const void* w, void* dX, void* dw,
                      void* db, int64_t M, int64_t K, float* ws, cudaStream_t st) {
    const int64_t parts = bwd_parts(M, K);
    const bool direct = parts == 1 && K <= kBwdWidest;
    float* part = (dw || db) && !direct ? ws : nullptr;
    if (M > 0 && K > kBwdWidest) {
        if (dX) norm_bwd_wide_kernel<T, W><<<(unsigned)M, 1024, 0, st>>>((const T*)dY, (const T*)X, mean, rstd, (const W*)w,
                                                                       (T*)dX, M, K);
        if (part) norm_bwd_columns_kernel<T><<<dim3((unsigned)((K + 255) / 256), (unsigned)parts), 256, 0, st>>>(
            (const T*)dY, (const T*)X, mean, rstd, part, M, K);
    } else if (M > 0) {
        auto* rows = K <= kBwdPairs ? &bwd_rows<T, W, VEC, 1, 2> : &bwd_rows<T, W, VEC, 2, 1>;
        const cudaError_t e = rows(dY, X, mean, rstd, w, dX, part, direct ? dw : nullptr, direct ? db : nullptr, M, (int)K, (int)parts, st);
        if (e != cudaSuccess) return e;
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !(dw || db) || direct) return e;
    return launch_dependent(&norm_bwd_sum_kernel<W>, dim3((unsigned)((2 * K + 31) / 32)), dim3(32, 32), 0, st, (const float*)part, (W*)dw,
                            (W*)db, parts, K);
}

size_t bwd_workspace(int64_t M, int64_t K) {
    const int64_t parts = bwd_parts(M, K);
    return parts == 1 && K <= kBwdWidest ? 0 : (size_t)parts * 2 * (size_t)K * sizeof(float);
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
    *bytes = bwd_workspace(M, K);
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
        const size_t need = bwd_workspace(M, K);
        if ((dweight || dbias) && need > 0 && (!workspace || workspace_bytes < need)) return SS1_ERR_INVALID_ARG;
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
