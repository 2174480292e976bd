// One AdamW step (Loshchilov & Hutter, "Decoupled Weight Decay Regularization") over many tensors in
// one launch, the moments in float32 or in 8 bits.
//
//     g' = g * grad_scale
//     m  = beta1 m + (1 - beta1) g',     v = beta2 v + (1 - beta2) g'^2
//     p  = p (1 - lr decay) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
//
// 8-bit moments: blocks of 256 consecutive elements of a tensor share one float scale, a power of
// two, so that scaling rounds nothing: the smallest 2^e (e >= -126) that brings the block's largest
// magnitude to 448 or below. Held are the E4M3 codes of m / scale and of sqrt(v) / scale: the root
// needs half of v's exponent range, and it is what the update divides by. A positive root keeps at
// least the smallest code: rounded to 0 it would make the next update m / eps. The update itself
// uses the unrounded new moments.
//
// Memory-bound: bf16 weights with a float32 master copy move 28 bytes an element with float32
// moments, 16 with 8-bit ones. Every float32 operation is rounded on its own (no fused multiply-
// add), so that the codes are those of the same formula written with elementwise operations.
#include "ss1_ops.cuh"

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <math.h>

namespace ss1 {
namespace {

using namespace op;

constexpr int kBlock = 256;              // elements of one scale: one warp, eight a lane
constexpr int kWarps = 8;
constexpr int kChunk = kBlock * kWarps * 4;   // elements of a CTA: four blocks a warp

enum : uint32_t { kParamBf16 = 1, kGradBf16 = 2, kAligned = 4 };

struct Entry {
    void* p;
    const void* g;
    float* master;
    void* m;
    void* v;
    float* m_scale;
    float* v_scale;
    int64_t n;
};

// The launch's tensors travel as kernel parameters (32,764 bytes at most): no copy to the device, and
// a captured launch keeps them.
template <int N>
struct Table {
    Entry t[N];
    int32_t first[N];    // the tensor's first chunk
    uint8_t flags[N];
    int32_t count;
};

struct Factors {
    float beta1, rest1, beta2, rest2, keep, step, root, eps, grad;
};
constexpr int kFactors = sizeof(Factors) / sizeof(float);

// Eight elements from `at` on, `n` of them inside the tensor; 0 in the others.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int64_t at, int n, bool vec, float (&f)[8]) {
    if (vec && n == 8) {
        Raw8<T> r;
        r.load_once(p + at);
        r.get(f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = i < n ? to_f(p[at + i]) : 0.0f;
    }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, int64_t at, int n, bool vec, const float (&f)[8]) {
    if (vec && n == 8) {
        Raw8<T> r;
        r.set(f);
        r.store(p + at);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[at + i] = from_f<T>(f[i]);
    }
}

__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int64_t at, int n, bool vec) {
    if (vec && n == 8) return __ldcs(reinterpret_cast<const uint2*>(p + at));
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) w[i / 4] |= (uint32_t)p[at + i] << (8 * (i % 4));
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void store_codes(uint8_t* p, int64_t at, int n, bool vec, uint2 c) {
    if (vec && n == 8) {
        *reinterpret_cast<uint2*>(p + at) = c;
        return;
    }
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[at + i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
}

__device__ __forceinline__ void decode8(uint2 c, float scale, float (&f)[8]) {
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_fp8x2_storage_t two = (__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i % 2)));
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3);
        const float2 x = __half22float2(__half2(h));
        f[2 * i] = __fmul_rn(x.x, scale);
        f[2 * i + 1] = __fmul_rn(x.y, scale);
    }
}

// The block's scale from the largest magnitude (the bits of its absolute value) over the warp.
__device__ __forceinline__ float block_scale(const float (&f)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    // top = 1.f * 2^ex: 448 is 1.75 * 2^8
    const int ex = (int)(top >> 23) - 127;
    const int e = (top & 0x7FFFFFu) <= 0x600000u ? ex - 8 : ex - 7;
    return __uint_as_float((uint32_t)(max(e, -126) + 127) << 23);
}

__device__ __forceinline__ uint2 encode8(const float (&f)[8], float scale) {
    // 1 / scale, exactly: scale = 2^e with -126 <= e <= 121
    const float inv = __uint_as_float((254u << 23) - __float_as_uint(scale));
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = make_float2(__fmul_rn(f[2 * i], inv), __fmul_rn(f[2 * i + 1], inv));
        w[i / 2] |= (uint32_t)__nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3) << (16 * (i % 2));
    }
    return make_uint2(w[0], w[1]);
}

template <int N, int BITS>
__global__ void __launch_bounds__(kWarps * 32) adamw_kernel(const __grid_constant__ Table<N> table, const Factors host,
                                                            const float* __restrict__ device) {
    Factors f = host;
    if (device) {
        float* to = reinterpret_cast<float*>(&f);
#pragma unroll
        for (int i = 0; i < kFactors; ++i) to[i] = __ldg(device + i);
    }
    // the tensor whose chunks contain this CTA's: the last one that starts at or before it
    int lo = 0, hi = table.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (table.first[mid] <= (int)blockIdx.x) lo = mid;
        else hi = mid - 1;
    }
    const Entry& t = table.t[lo];
    const uint32_t flags = table.flags[lo];
    const bool vec = flags & kAligned;
    const int64_t start = (int64_t)((int)blockIdx.x - table.first[lo]) * kChunk;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    for (int64_t block = start / kBlock + warp; block < (start + kChunk) / kBlock && block * kBlock < t.n; block += kWarps) {
        const int64_t at = block * kBlock + lane * 8;
        const int64_t left = t.n - at;
        int n = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
        if (n > 0 && !SS1_SPAN_IN(at, n, t.n, kSiteAdamTensor)) n = 0;
        float g[8], p[8], m[8], v[8];
        if (flags & kGradBf16) load8((const __nv_bfloat16*)t.g, at, n, vec, g);
        else load8((const float*)t.g, at, n, vec, g);
        if (t.master) load8((const float*)t.master, at, n, vec, p);
        else if (flags & kParamBf16) load8((const __nv_bfloat16*)t.p, at, n, vec, p);
        else load8((const float*)t.p, at, n, vec, p);
        if (BITS == 32) {
            load8((const float*)t.m, at, n, vec, m);
            load8((const float*)t.v, at, n, vec, v);
        } else {
            const uint2 mc = load_codes((const uint8_t*)t.m, at, n, vec), vc = load_codes((const uint8_t*)t.v, at, n, vec);
            decode8(mc, t.m_scale[block], m);
            decode8(vc, t.v_scale[block], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], v[i]);
        }
        float root[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float gi = __fmul_rn(g[i], f.grad);
            m[i] = __fadd_rn(__fmul_rn(m[i], f.beta1), __fmul_rn(gi, f.rest1));
            v[i] = __fadd_rn(__fmul_rn(v[i], f.beta2), __fmul_rn(__fmul_rn(gi, gi), f.rest2));
            root[i] = __fsqrt_rn(v[i]);
            const float den = __fadd_rn(__fmul_rn(root[i], f.root), f.eps);
            p[i] = __fsub_rn(__fmul_rn(p[i], f.keep), __fmul_rn(__fdiv_rn(m[i], den), f.step));
        }
        if (t.master) store8(t.master, at, n, vec, p);
        if (flags & kParamBf16) store8((__nv_bfloat16*)t.p, at, n, vec, p);
        else store8((float*)t.p, at, n, vec, p);
        if (BITS == 32) {
            store8((float*)t.m, at, n, vec, m);
            store8((float*)t.v, at, n, vec, v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)   // lanes behind the tensor's end take no part in the block's maximum
                if (i >= n) m[i] = root[i] = 0.0f;
            const float ms = block_scale(m), vs = block_scale(root);
            uint2 mc = encode8(m, ms), vc = encode8(root, vs);
            uint32_t w[2] = {vc.x, vc.y};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (root[i] > 0.0f && !((w[i / 4] >> (8 * (i % 4))) & 0xFFu)) w[i / 4] |= 1u << (8 * (i % 4));
            store_codes((uint8_t*)t.m, at, n, vec, mc);
            store_codes((uint8_t*)t.v, at, n, vec, make_uint2(w[0], w[1]));
            if (lane == 0 && SS1_IN(block, (t.n + kBlock - 1) / kBlock, kSiteAdamScale)) {
                t.m_scale[block] = ms;
                t.v_scale[block] = vs;
            }
        }
    }
}

template <int N>
cudaError_t launch(const ss1_adamw_tensor* tensors, int64_t count, int bits, const Factors& f,
                   const float* device, cudaStream_t st) {
    static_assert(sizeof(Table<N>) + sizeof(Factors) + 16 <= 32764, "kernel parameters");
    Table<N> table;
    table.count = 0;
    int64_t chunks = 0;
    for (int64_t i = 0; i < count; ++i) {
        const ss1_adamw_tensor& t = tensors[i];
        if (t.numel == 0) continue;
        const bool pb = t.param_dtype == SS1_DTYPE_BF16, gb = t.grad_dtype == SS1_DTYPE_BF16;
        const size_t state = bits == 32 ? 16 : 8;
        const bool vec = aligned(t.param, 16) && aligned(t.grad, 16) && aligned(t.master, 16) && aligned(t.exp_avg, state) &&
                         aligned(t.exp_avg_sq, state);
        const int k = table.count++;
        table.t[k] = Entry{t.param, t.grad, t.master, t.exp_avg, t.exp_avg_sq, t.avg_scale, t.sq_scale, t.numel};
        table.first[k] = (int32_t)chunks;
        table.flags[k] = (uint8_t)((pb ? kParamBf16 : 0) | (gb ? kGradBf16 : 0) | (vec ? kAligned : 0));
        chunks += (t.numel + kChunk - 1) / kChunk;
    }
    if (table.count == 0) return cudaSuccess;
    if (bits == 32) adamw_kernel<N, 32><<<(unsigned)chunks, kWarps * 32, 0, st>>>(table, f, device);
    else adamw_kernel<N, 8><<<(unsigned)chunks, kWarps * 32, 0, st>>>(table, f, device);
    return cudaGetLastError();
}

constexpr int kSmall = 32, kLarge = 440;   // tensors of one launch: the parameters are copied at every launch

bool hyper_ok(const ss1_adamw_hyper* h) {
    return h && h->step >= 1 && isfinite(h->lr) && h->beta1 >= 0.0 && h->beta1 < 1.0 && h->beta2 >= 0.0 && h->beta2 < 1.0 &&
           h->eps >= 0.0 && isfinite(h->eps) && isfinite(h->weight_decay) && isfinite(h->grad_scale);
}

Factors factors(const ss1_adamw_hyper& h) {
    Factors f;
    f.beta1 = (float)h.beta1;
    f.rest1 = (float)(1.0 - h.beta1);
    f.beta2 = (float)h.beta2;
    f.rest2 = (float)(1.0 - h.beta2);
    f.keep = (float)(1.0 - h.lr * h.weight_decay);
    f.step = (float)(h.lr / (1.0 - pow(h.beta1, (double)h.step)));
    f.root = (float)(1.0 / sqrt(1.0 - pow(h.beta2, (double)h.step)));
    f.eps = (float)h.eps;
    f.grad = (float)h.grad_scale;
    return f;
}

}  // namespace
}  // namespace ss1

using namespace ss1;
using namespace ss1::op;

extern "C" SS1_API int ss1_adamw_factors(const ss1_adamw_hyper* hyper, float* out) {
    static_assert(kFactors == SS1_ADAMW_FACTORS, "header");
    if (!out || !hyper_ok(hyper)) return SS1_ERR_INVALID_ARG;
    const Factors f = factors(*hyper);
    const float* from = reinterpret_cast<const float*>(&f);
    for (int i = 0; i < kFactors; ++i) out[i] = from[i];
    return SS1_OK;
}

extern "C" SS1_API int ss1_adamw_step(const ss1_adamw_tensor* tensors, int64_t count, int state_bits,
                                      const ss1_adamw_hyper* hyper, const float* device_factors, void* stream) {
    if (count < 0 || (count > 0 && !tensors) || (state_bits != 32 && state_bits != 8)) return SS1_ERR_INVALID_ARG;
    if (!device_factors && !hyper_ok(hyper)) return SS1_ERR_INVALID_ARG;
    if (!aligned(device_factors, 4)) return SS1_ERR_MISALIGNED;
    // everything is checked before the first launch, so that a refused call has changed nothing
    for (int64_t i = 0; i < count; ++i) {
        const ss1_adamw_tensor& t = tensors[i];
        if (t.numel < 0 || t.numel > (int64_t)1 << 40 || !dtype_ok(t.param_dtype) || !dtype_ok(t.grad_dtype))
            return SS1_ERR_INVALID_ARG;
        if (t.master && t.param_dtype != SS1_DTYPE_BF16) return SS1_ERR_INVALID_ARG;
        if (t.numel == 0) continue;
        if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq) return SS1_ERR_INVALID_ARG;
        if (state_bits == 8 && (!t.avg_scale || !t.sq_scale)) return SS1_ERR_INVALID_ARG;
        if (!aligned(t.param, dtype_size(t.param_dtype)) || !aligned(t.grad, dtype_size(t.grad_dtype)) ||
            !aligned(t.master, 4) || (state_bits == 32 && (!aligned(t.exp_avg, 4) || !aligned(t.exp_avg_sq, 4))) ||
            (state_bits == 8 && (!aligned(t.avg_scale, 4) || !aligned(t.sq_scale, 4))))
            return SS1_ERR_MISALIGNED;
    }
    Factors f = {};
    if (!device_factors) f = factors(*hyper);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    for (int64_t at = 0; at < count;) {
        // as many tensors as one launch takes, and no more chunks than its grid can count
        int64_t end = at, chunks = 0;
        for (; end < count && end - at < kLarge; ++end) {
            const int64_t c = (tensors[end].numel + kChunk - 1) / kChunk;
            if (end > at && chunks + c > 0x7FFFFFFF) break;
            chunks += c;
        }
        const cudaError_t e = end - at <= kSmall ? launch<kSmall>(tensors + at, end - at, state_bits, f, device_factors, st)
                                                 : launch<kLarge>(tensors + at, end - at, state_bits, f, device_factors, st);
        if (e != cudaSuccess) { cudaGetLastError(); return SS1_ERR_CUDA; }
        at = end;
    }
    return SS1_OK;
}
