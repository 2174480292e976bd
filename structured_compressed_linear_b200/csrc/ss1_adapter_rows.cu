// The adapters' forward for a few rows (decode): one launch, one row a cluster.
//
// A decode batch reads every used adapter once and little else, so what counts is latency: the two
// products of a row depend on one another, and a second launch costs more than either. A cluster of
// eight CTAs takes a row (several clusters a row where the batch is small: each repeats the first
// product and takes its own columns of the second). CTA c sums its eighth of K for all ranks, the
// partial H meet in distributed shared memory, and each CTA finishes its share of the columns. B and Y
// are asked into L2 at the start, beside the first product. Rows need no plan: each looks its adapter up.
// 48 rows of 24 adapters, 4096 x 4096, rank 16: 5.3 us as graph replays, of which the bytes (7.3 MB) take 1.1.
#include "ss1_adapter.cuh"
#include "ptx_sm100.cuh"

namespace ss1 {
namespace ada {
namespace {

using namespace op;

constexpr int kThreads = 256, kWarps = kThreads / 32, kCluster = 8;

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

template <typename T>
__global__ void __launch_bounds__(kThreads) rows_kernel(const T* __restrict__ X, const T* __restrict__ A, const T* __restrict__ B,
                                                        const int32_t* __restrict__ index, const float* __restrict__ scale,
                                                        const T* Y, T* out, float* __restrict__ H, int M, int K, int N, int R, int n) {
    __shared__ float part[kMaxRank], h[kMaxRank];
    wait_for_previous();
    let_next_start();
    const int m = blockIdx.y, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int rank = blockIdx.x % kCluster, groups = gridDim.x / kCluster, group = blockIdx.x / kCluster;
    const int a = index ? index[m] : 0;
    // this CTA's columns of the second product, in eights
    const int eights = N / 8, shares = groups * kCluster, per = (eights + shares - 1) / shares;
    const int c0 = min(N, (int)blockIdx.x * per * 8), c1 = min(N, c0 + per * 8);
    const int64_t row = (int64_t)m * N;
    if ((unsigned)a >= (unsigned)n) {          // the whole cluster: the row stays as it is
        if (H && group == 0 && rank == 0)
            for (int r = tid; r < R; r += kThreads) H[(int64_t)m * R + r] = 0.0f;
        if (Y == out) return;
        for (int c = c0 + tid * 8; c < c1; c += kThreads * 8) {
            Raw8<T> v;
            if (!SS1_SPAN_IN(row + c, 8, (int64_t)M * N, kSiteAdaY)) continue;
            v.load(Y + row + c);
            v.store(out + row + c);
        }
        return;
    }
    const T* Ba = B + (int64_t)a * N * R;
    {   // lines of 128 bytes of this CTA's part of B, and of Y
        constexpr int line = 128 / sizeof(T);
        for (int64_t i = (int64_t)c0 * R + tid * line; i < (int64_t)c1 * R; i += kThreads * line) prefetch_l2(Ba + i);
        for (int i = c0 + tid * line; i < c1; i += kThreads * line) prefetch_l2(Y + row + i);
    }
    // H: eights of K dealt to the cluster's CTAs, ranks to the warps
    const int keights = K / 8, kper = (keights + kCluster - 1) / kCluster;
    const int k0 = min(keights, rank * kper), k1 = min(keights, k0 + kper);
    const T* x = X + (int64_t)m * K;
    const T* Aa = A + (int64_t)a * R * K;
    constexpr int kRanks = 2;                  // of a warp at a time
    for (int r0 = warp * kRanks; r0 < R; r0 += kWarps * kRanks) {
        float s[kRanks] = {};
#pragma unroll 2
        for (int k = k0 + lane; k < k1; k += 32) {
            Raw8<T> u, v[kRanks];
            const bool ok = SS1_SPAN_IN((int64_t)m * K + k * 8, 8, (int64_t)M * K, kSiteAdaX);
            if (ok) u.load(x + k * 8);
            else u.zero();
#pragma unroll
            for (int r = 0; r < kRanks; ++r) {
                if (r0 + r < R && SS1_SPAN_IN(((int64_t)a * R + r0 + r) * K + k * 8, 8, (int64_t)n * R * K, kSiteAdaA))
                    v[r].load(Aa + (int64_t)(r0 + r) * K + k * 8);
                else v[r].zero();
            }
            float f[8], g[8];
            u.get(f);
#pragma unroll
            for (int r = 0; r < kRanks; ++r) {
                v[r].get(g);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[r] = fmaf(f[i], g[i], s[r]);
            }
        }
#pragma unroll
        for (int r = 0; r < kRanks; ++r) {
            const float v = warp_sum(s[r]);
            if (lane == 0 && r0 + r < R) part[r0 + r] = v;
        }
    }
    ptx::cluster_sync();
    const float f = scale ? scale[a] : 1.0f;
    if (tid < R) {
        float v[kCluster], s = 0.0f;
#pragma unroll
        for (int k = 0; k < kCluster; ++k) v[k] = ptx::ld_cluster_f32(ptx::map_to_rank(part + tid, k));
#pragma unroll
        for (int k = 0; k < kCluster; ++k) s += v[k];
        if (H && group == 0 && rank == 0 && SS1_IN((int64_t)m * R + tid, (int64_t)M * R, kSiteAdaH)) H[(int64_t)m * R + tid] = s;
        h[tid] = f * s;
    }
    // nobody leaves while its sums are being read; this also makes h visible to the CTA
    ptx::cluster_sync();
    // one column a thread, B's row of it in eights of ranks
    for (int c = c0 + tid; c < c1; c += kThreads) {
        float s = 0.0f;
        for (int r = 0; r < R; r += 8) {
            Raw8<T> v;
            if (SS1_SPAN_IN(((int64_t)a * N + c) * R + r, 8, (int64_t)n * N * R, kSiteAdaB)) v.load(Ba + (int64_t)c * R + r);
            else v.zero();
            float g[8];
            v.get(g);
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(h[r + i], g[i], s);
        }
        if (SS1_IN(row + c, (int64_t)M * N, kSiteAdaY)) out[row + c] = from_f<T>(to_f(Y[row + c]) + s);
    }
}

template <typename T>
cudaError_t launch(const Call& c, const void* X, const void* Y, void* out, float* H, cudaStream_t st) {
    // clusters a row: about two CTAs for each of 148 SMs in all, at least 128 columns a CTA
    int groups = (int)(296 / (kCluster * c.M));
    const int most = (int)(c.N / (128 * kCluster));
    groups = groups > most ? most : groups;
    groups = groups < 1 ? 1 : groups;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(kCluster * groups), (unsigned)c.M);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kCluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, &rows_kernel<T>, (const T*)X, (const T*)c.A, (const T*)c.B, c.index, c.scale, (const T*)Y, (T*)out, H,
                              (int)c.M, (int)c.K, (int)c.N, c.R, c.n);
}

}  // namespace

cudaError_t rows_forward(const Call& c, const void* X, const void* Y, void* out, float* H, int dtype, cudaStream_t st) {
    return dtype == SS1_DTYPE_BF16 ? launch<__nv_bfloat16>(c, X, Y, out, H, st) : launch<float>(c, X, Y, out, H, st);
}

}  // namespace ada
}  // namespace ss1
